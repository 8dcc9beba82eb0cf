"""What is asked once a device (csrc/aq_device.h), and that the experts' kernels
ask in that way (no GPU: the class is compiled alone)."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "quantized_matmul_affine_gb300", "csrc")
PROGRAM = r"""
#include "aq_device.h"
#include <cstdio>
int main() {
    aq::PerDevice p;
    int calls = 0;
    auto ask = [&](bool answer) { return [&calls, answer] { ++calls; return answer; }; };
    // a device's answer is its own, whichever came first, and is asked for once
    const bool a = !p(1, ask(false)) && p(0, ask(true)) && p(63, ask(true)) && !p(62, ask(false));
    const bool b = calls == 4;
    const bool c = !p(1, ask(true)) && p(0, ask(false)) && p(63, ask(false)) && !p(62, ask(true)) && calls == 4;
    // devices past the bits are asked every time, and stand for no other
    const bool d = p(64, ask(true)) && !p(64, ask(false)) && p(127, ask(true)) && calls == 7;
    const bool e = p(0, ask(false)) && !p(1, ask(true)) && calls == 7;
    std::printf("%d%d%d%d%d\n", a, b, c, d, e);
}
"""


def test_answers_are_a_devices_own(tmp_path):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "per_device.cpp", tmp_path / "per_device"
    src.write_text(PROGRAM)
    subprocess.run([cc, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout == "11111\n"


def test_experts_kernels_ask_every_device():
    """Attributes of the experts' kernels are set each time or once a device,
    never once a process."""
    for name in ("aq_moe.cu", "aq_moe.cuh", "aq_embed.cu"):
        text = open(os.path.join(CSRC, name)).read()
        assert "call_once" not in text, name
        kept = re.findall(r"static\s+([\w:<>]+)\s+\w+\s*(?:\{|;|=)", text)  # (functions have parentheses)
        assert set(kept) <= {"PerDevice", "std::atomic<uint64_t>"}, (name, kept)  # a bit a device
