"""include/aq.h compiles alone and after the standard headers, as C and as C++."""
import os
import shutil
import subprocess

import pytest

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
BEFORE = ["", "complex.h", "math.h", "tgmath.h", "iso646.h", "time.h", "signal.h", "errno.h", "inttypes.h", "stdatomic.h"]


@pytest.mark.parametrize("before", BEFORE)
@pytest.mark.parametrize("lang,std", [("c", "c99"), ("c", "c11"), ("c++", "c++17")])
def test_compiles_after(before, lang, std, tmp_path):
    cc = shutil.which("gcc" if lang == "c" else "g++")
    if cc is None:
        pytest.skip("no compiler")
    if before in ("stdatomic.h", "tgmath.h") and (lang, std) != ("c", "c11"):
        pytest.skip("a header of C11")
    src = tmp_path / "one.src"
    src.write_text((f"#include <{before}>\n" if before else "") + '#include "aq.h"\n#include "aq.h"\n'
                   "int f(const aq_experts *x, const aq_router *r) { return (int)(x->inner + r->K); }\n")
    subprocess.run([cc, "-x", lang, f"-std={std}", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", INCLUDE, "-c",
                    str(src), "-o", str(tmp_path / "one.o")], check=True)
