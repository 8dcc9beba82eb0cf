"""Several samples of one prompt through a small quantised decoder.

A prompt is read once into a paged 4-bit KV cache; its pages are then forked
into a row for each sample.  A decode step gives every row a token's room
(copying the shared partial page where it is written), projects q, k and v
with the quantised weights, appends k and v, and attends - the prompt's keys
once for all samples.  In the end the worse half of the samples is freed and
the pool compacted.

    python examples/serve_samples.py [samples] [prompt tokens] [steps]

The model is random: the example shows the calls, and checks that sharing,
forking and compacting change no result.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_matmul_affine_gb300 as aq  # noqa: E402

HIDDEN, HEADS, KV, DIM, LAYERS, PAGE, BITS, GROUP = 1024, 8, 2, 128, 2, 32, 4, 64


class Layer:
    """Attention of one decoder layer: quantised q, k, v and output projections."""

    def __init__(self, gen):
        def weight(n, k):
            w = torch.randn(n, k, device="cuda", generator=gen) * k ** -0.5
            return aq.aq_quantize(w.half(), BITS)

        self.qkv = [weight(HEADS * DIM, HIDDEN), weight(KV * DIM, HIDDEN), weight(KV * DIM, HIDDEN)]
        self.out = weight(HIDDEN, HEADS * DIM)

    def __call__(self, x, cache, layer, cu, start, table, attend):
        q, k, v = aq.aq_matmul_multi(x, self.qkv, BITS)
        aq.aq_cache_append(cache, layer, k.view(-1, KV, DIM), v.view(-1, KV, DIM), cu, start, table)
        o = attend(q.view(-1, HEADS, DIM), layer)
        return x + aq.aq_matmul(o.reshape(-1, HEADS * DIM), *self.out, BITS)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def main(samples=6, prompt=75, steps=5, seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layers = [Layer(gen) for _ in range(LAYERS)]
    width = -(-(prompt + steps) // PAGE)
    n_pages = width * samples + 4
    cache = aq.AqCache.empty(LAYERS, n_pages, KV, DIM, PAGE, BITS, GROUP)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    lens = torch.zeros(samples, dtype=torch.int32, device="cuda")
    table = torch.full((samples, width), -1, dtype=torch.int32, device="cuda")
    everyone = torch.arange(samples + 1, dtype=torch.int32, device="cuda")
    scale = DIM ** -0.5

    # the prompt, into row 0: its tokens see those before them
    add = torch.zeros_like(lens)
    add[0] = prompt
    assert aq.aq_cache_grow(cache, refs, table, lens, add)[3].tolist()[0] == 0
    x = torch.randn(prompt, HIDDEN, device="cuda", generator=gen).half()
    cu = ints(0, *[prompt] * samples)
    zero = torch.zeros_like(lens)

    def causal(q, layer):  # 64 tokens a call: the last L of the sequence so far
        parts = []
        for t0 in range(0, prompt, 64):
            t1 = min(prompt, t0 + 64)
            parts.append(aq.aq_attention_batch(q[None, t0:t1].contiguous(), cache, layer, table[:1],
                                               ints(t1), scale)[0])
        return torch.cat(parts)

    for i, layer in enumerate(layers):
        x = layer(x, cache, i, cu, zero, table, causal)

    # every other row becomes a copy of row 0: the same pages, none copied
    parent = torch.zeros_like(lens)
    parent[0] = -1
    assert aq.aq_cache_fork(cache, refs, table, lens, parent, torch.full_like(lens, -1))[3].tolist()[0] == 0

    group, shared = ints(0, samples), ints(prompt)
    x = torch.randn(samples, HIDDEN, device="cuda", generator=gen).half()
    for _ in range(steps):
        start = lens.clone()
        status = aq.aq_cache_grow(cache, refs, table, lens, torch.ones_like(lens))[3]

        def attend(q, layer):
            q = q[:, None]
            o = aq.aq_attention_batch(q, cache, layer, table, lens, scale, group, shared)
            alone = aq.aq_attention_batch(q, cache, layer, table, lens, scale)
            torch.testing.assert_close(o, alone, rtol=1e-2, atol=4e-3)
            return o

        for i, layer in enumerate(layers):
            x = layer(x, cache, i, everyone, start, table, attend)
        assert status.tolist()[0] == 0

    # the worse half ends, the pool closes its gaps: the others' rows are the same
    before = aq.aq_cache_read(cache, 1, everyone * (prompt + steps), zero, table,
                              samples * (prompt + steps), torch.float16)
    score = x.float().square().mean(1)
    keep = torch.where(score >= score.median(), -1, 0).int()
    freed = aq.aq_cache_trim(cache, refs, table, lens, keep)[3].tolist()
    live, moved = aq.aq_cache_compact(cache, refs, table, lens)[2].tolist()[2:]
    after = aq.aq_cache_read(cache, 1, everyone * (prompt + steps), zero,
                             torch.where(table >= 0, table, 0), samples * (prompt + steps), torch.float16)
    for a, b in zip(before, after):
        a, b = (t.view(samples, prompt + steps, -1)[keep < 0] for t in (a, b))
        assert torch.equal(a, b)
    assert int((refs > 0).sum()) == live and not refs[live:].any() and aq.aq_device_error() == 0
    print(f"{samples} samples of a {prompt}-token prompt, {steps} steps: {freed[2]} pages freed, "
          f"{live} live, {moved} moved")
    return live


if __name__ == "__main__":
    main(*[int(a) for a in sys.argv[1:]])
