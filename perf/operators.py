"""Cases that measure the paged quantised KV cache and the attention that reads it.

The cache is a pool of pages [layers][n_pages][KV][record].  The record of one page and one KV head
holds P cached rows of K and of V in the affine format (4 or 8 bit codes, LSB first; a value is
scale * code + bias, one fp16 scale and bias per group of values along the head dimension):

    K codes [P][D*bits/32] words | V codes [P][D*bits/32] words |
    K (scale, bias) [P][D/group] | V (scale, bias) [P][D/group]

A sequence is a row of `table` (int32 [B][max_pages], page numbers, -1 where it has none) and its
length in `lens`; `refs` counts the rows that hold a page (0: the page is free).

Four operators, one kind of case each:
  attend   softmax attention of L new tokens a sequence over the cache, for a batch whose groups share
           the first tokens of their sequences;
  append   quantising new K and V rows into their pages, and reading rows back as floats;
  beam     one step of the page tables of a beam search: the losers are freed, the winners forked into
           their rows, every row grown by a token (shared partial pages are copied);
  compact  moving live pages to the front of the pool, tables and counts with them.
"""
import math

import torch

own = False

# (query heads, KV heads, head dimension): a 5120-wide decoder's 40 heads of 128, the 16 heads of 256
# over 8 of a 12B decoder, small heads, one query head per KV head, one KV head for all
HEADS = {"40x128": (40, 8, 128), "16x256": (16, 8, 256), "12x64": (12, 2, 64), "8x64": (8, 8, 64),
         "16x128": (16, 1, 128)}


def listed():
    return [
        # one user, a short prompt: the first decode steps of a chat, where latency counts
        attend("attend_one", 1, 1, 0, 0, 37, "40x128", 4, 64, 16, "fp16", shape="even"),
        # several drafted tokens a sequence to verify, three system prompts in one batch, odd lengths
        attend("attend_draft", 11, 5, 3, 1001, 333, "12x64", 8, 32, 32, "fp16"),
        # a batch of unrelated conversations of up to 8k rows on the 12B decoder's heads
        attend("attend_ragged", 24, 1, 0, 0, 8192, "16x256", 4, 64, 64, "bf16"),
        # a small batch of chats behind one system prompt
        attend("attend_prompt", 8, 1, 1, 4096, 777, "40x128", 4, 64, 64, "bf16"),
        # a full batch that answers questions about one document
        attend("attend_document", 64, 1, 1, 8191, 1024, "40x128", 4, 64, 64, "bf16"),
        # the largest: 128 samples over a 32k-token context
        attend("attend_samples", 128, 1, 1, 32768, 1024, "40x128", 8, 64, 64, "fp16"),
        # a decode step's new rows of a full batch
        append("append_step", 64, 64, "40x128", 4, 64, 64, "bf16"),
        # prompts of unequal lengths, 16k tokens together
        append("append_prompts", 13, 16384, "40x128", 4, 64, 64, "bf16"),
        # one request with four beams
        beam("beam_request", 1, 4, 500, 40, "16x256", 4, 64, 64, 2),
        # 64 requests with eight beams each, four layers' pages
        beam("beam_batch", 64, 8, 2048, 256, "40x128", 4, 64, 64, 4),
        # a small pool after its first requests have ended
        compact("compact_small", 256, 9, "12x64", 8, 32, 32, 1),
        # a pool of 1.2 GB with 40 % holes
        compact("compact_pool", 8192, 160, "40x128", 4, 64, 64, 2),
    ]


def attend(name, batch, tokens, groups, shared, own_rows, heads, bits, group, page, dtype, shape="ragged"):
    return dict(name=name, kind="attend", batch=batch, tokens=tokens, groups=groups, shared=shared, own_rows=own_rows, heads=heads,
                bits=bits, group=group, page=page, dtype=dtype, shape=shape)


def append(name, batch, total, heads, bits, group, page, dtype):
    return dict(name=name, kind="append", batch=batch, total=total, heads=heads, bits=bits, group=group, page=page, dtype=dtype)


def beam(name, requests, width, prompt, generated, heads, bits, group, page, layers):
    return dict(name=name, kind="beam", requests=requests, width=width, prompt=prompt, generated=generated, heads=heads, bits=bits,
                group=group, page=page, layers=layers)


def compact(name, n_pages, batch, heads, bits, group, page, layers):
    return dict(name=name, kind="compact", n_pages=n_pages, batch=batch, heads=heads, bits=bits, group=group, page=page, layers=layers)


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    heads = rng.choice(sorted(HEADS))
    bits, dtype = rng.choice((4, 8)), rng.choice(("fp16", "bf16"))
    group = rng.choice([g for g in (32, 64, 128) if HEADS[heads][2] % g == 0])
    page = rng.choice((16, 32, 64, 128))
    kind = rng.choice(("attend", "attend", "attend", "append", "beam", "compact"))
    if kind == "attend":
        while True:
            batch, tokens = log(1, 128), rng.choice((1, 1, 1, 2, 3, 5, 8))
            groups = rng.choice((0, 1, 1, min(3, batch))) if batch > 1 else 0
            shared = log(64, 32768) if groups else 0
            own_rows = log(16, 2048 if groups else 8192)
            c = attend("", batch, tokens, groups, shared, own_rows, heads, bits, group, page, dtype)
            w = work(c)
            if w["bytes"] < 250e6 and w["flops"] < 80e9:
                break
    elif kind == "append":
        batch = log(1, 64)
        c = append("", batch, max(batch, log(1, 16000)), heads, bits, group, page, dtype)
    elif kind == "beam":
        c = beam("", log(1, 64), rng.randint(2, 8), log(30, 2000), log(5, 250), heads, bits, group, page, rng.randint(1, 3))
    else:
        n = log(64, 8000)
        c = compact("", n, rng.randint(2, min(160, n // 8)), heads, bits, group, page, rng.randint(1, 2))
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------- inputs


def _record(case):
    _, kv, d = HEADS[case["heads"]]
    return case["page"] * (2 * d * case["bits"] // 8 + 8 * (d // case["group"]))


def _pool(case, layers, n_pages, gen):
    """Pages with codes of every value; scales and biases as a quantiser of rows of about unit size leaves them."""
    _, kv, d = HEADS[case["heads"]]
    rec, codes = _record(case), 2 * case["page"] * d * case["bits"] // 8
    pool = torch.empty(layers, n_pages, kv, rec, dtype=torch.uint8, device="cuda")
    for layer in pool:  # one layer at a time: the random numbers are wider than what is kept of them
        layer[..., :codes] = torch.randint(0, 256, (n_pages, kv, codes), dtype=torch.uint8, device="cuda", generator=gen)
        s = torch.rand(n_pages, kv, (rec - codes) // 4, device="cuda", generator=gen) * (3.4 / 2 ** case["bits"]) + 1.7 / 2 ** case["bits"]
        b = -(2 ** (case["bits"] - 1)) * s + 0.1 * torch.randn(s.shape, device="cuda", generator=gen)
        layer[..., codes:] = torch.stack((s, b), -1).half().view(n_pages, kv, -1).view(torch.uint8)
    return pool


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _attend_lengths(case, seed):
    """Per sequence its group (or -1) and its length, new tokens included; first sequences of the groups."""
    r = torch.Generator().manual_seed(seed)
    batch, tokens, groups = case["batch"], case["tokens"], case["groups"]
    share = [case["shared"] - 37 * g for g in range(groups)]  # prompts of unequal lengths
    share = [max(1, s) for s in share]
    starts = [round(g * batch / groups) for g in range(groups)] + [batch] if groups else [0]
    lens = []
    for b in range(batch):
        own_rows = case["own_rows"] if case["shape"] == "even" else 1 + int(case["own_rows"] * torch.rand(1, generator=r).item())
        g = next((g for g in range(groups) if starts[g] <= b < starts[g + 1]), -1)
        lens.append((share[g] if g >= 0 else 0) + max(own_rows, tokens))
    if batch > 8:  # an empty slot of the batch: its rows have nothing to attend to
        lens[batch - 2] = 0
    return starts, share, lens


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed + 1)
    h, kv, d = HEADS[case["heads"]]
    page = case["page"]
    state = {"case": case}
    if case["kind"] == "attend":
        starts, share, lens = _attend_lengths(case, seed)
        width = -(-max(lens) // page) + 1
        table, used = torch.full((case["batch"], width), -1, dtype=torch.int32), 0
        fulls, first = [s // page for s in share], {}
        for b, n in enumerate(lens):
            have = -(-n // page)
            g = next((g for g in range(case["groups"]) if starts[g] <= b < starts[g + 1]), -1)
            same = min(fulls[g], have) if g >= 0 else 0
            if g >= 0 and g not in first:  # the group's first sequence: all its pages are its own
                first[g], same = b, 0
            elif same:
                table[b, :same] = table[first[g], :same]
            table[b, same:have] = torch.arange(used, used + have - same, dtype=torch.int32)
            used += have - same
        n_pages = used + 3
        order = torch.randperm(n_pages, generator=cpu).int()
        table = torch.where(table >= 0, order[table.clamp(min=0).long()], table)
        pool = _pool(case, 1, n_pages, gen)
        # the partial page at a shared prefix's end is every sequence's own, with the same rows in it
        rec, rb, sg = _record(case), d * case["bits"] // 8, 4 * (d // case["group"])
        for g in range(case["groups"]):
            part = share[g] % page
            for b in range(starts[g], starts[g + 1]):
                if not part or b == first[g] or lens[b] == 0:
                    continue
                src, dst = int(table[first[g], fulls[g]]), int(table[b, fulls[g]])
                for at, n in ((0, rb), (page * rb, rb), (2 * page * rb, sg), (2 * page * rb + page * sg, sg)):
                    pool[0, dst, :, at:at + part * n] = pool[0, src, :, at:at + part * n]
        dt = torch.float16 if case["dtype"] == "fp16" else torch.bfloat16
        state |= {"pool": pool, "table": table.cuda(), "lens": _ints(lens), "starts": _ints(starts) if share else None,
                  "shared": _ints(share) if share else None, "scale": d ** -0.5, "widest": max(lens) if not share else max(max(lens) - min(share), 1),
                  "q": torch.randn(case["batch"], case["tokens"], h, d, device="cuda", generator=gen).to(dt)}
    elif case["kind"] == "append":
        cuts = torch.randperm(case["total"] - 1, generator=cpu)[:case["batch"] - 1].sort().values + 1 if case["total"] > 1 else torch.empty(0)
        cu = torch.cat((torch.zeros(1), cuts, torch.tensor([case["total"]]))).int()
        start = torch.randint(0, 300, (len(cu) - 1,), generator=cpu).int()
        have = (start + cu.diff() + page - 1) // page
        n_pages = int(have.sum()) + 3
        order = torch.randperm(n_pages, generator=cpu).int()
        table, used = torch.full((len(start), int(have.max()) + 1), -1, dtype=torch.int32), 0
        for b, n in enumerate(have.tolist()):
            table[b, :n] = order[used:used + n]
            used += n
        dt = torch.float16 if case["dtype"] == "fp16" else torch.bfloat16
        # a fused projection's output [tokens][q, k and v heads]; rows and channels of unequal size, as caches have them
        x = torch.randn(case["total"], h + 2 * kv, d, device="cuda", generator=gen)
        x *= torch.rand(1, h + 2 * kv, d, device="cuda", generator=gen) * 2 + 0.1
        x = x.to(dt)
        state |= {"pool": _pool(case, 1, n_pages, gen), "table": table.cuda(), "cu": cu.cuda(), "start": start.cuda(),
                  "k": x[:, h:h + kv], "v": x[:, h + kv:]}
    elif case["kind"] == "beam":
        req, width = case["requests"], case["width"]
        lens, rows, used = [], [], 0
        for r in range(req):
            prompt = 1 + int(case["prompt"] * (0.5 + 0.5 * torch.rand(1, generator=cpu).item()))
            n = prompt + 1 + int(case["generated"] * torch.rand(1, generator=cpu).item())
            same, have = prompt // page, -(-n // page)
            for w in range(width):
                rows.append(list(range(used, used + same)) + list(range(used + same + w * (have - same), used + same + (w + 1) * (have - same))))
                lens.append(n)
            used += same + width * (have - same)
        most = -(-(case["prompt"] + case["generated"] + 3) // page)  # pages of the longest row there can be
        n_pages = req * (case["prompt"] // page + 2 + width * (case["generated"] // page + 4))
        order = torch.randperm(n_pages, generator=cpu).int()
        wide = most + 2
        table = torch.tensor([r + [-1] * (wide - len(r)) for r in rows], dtype=torch.int32)
        table = torch.where(table >= 0, order[table.clamp(min=0).long()], table)
        refs = torch.bincount(table[table >= 0].long(), minlength=n_pages).int()
        keep, parent = [], []
        for r in range(req):  # half of a request's beams lose; each of them becomes a copy of a winner
            order = torch.randperm(width, generator=cpu).tolist()
            wins, lost = order[: width - width // 2], set(order[width - width // 2:])
            for w in range(width):
                keep.append(0 if w in lost else -1)
                parent.append(r * width + wins[int(torch.randint(0, len(wins), (1,), generator=cpu))] if w in lost else -1)
        state |= {"pool": _pool(case, case["layers"], n_pages, gen), "table": table.cuda(), "refs": refs.cuda(), "lens": _ints(lens),
                  "keep": _ints(keep), "parent": _ints(parent), "whole": _ints([-1] * len(lens)), "add": _ints([1] * len(lens))}
    else:
        n, batch = case["n_pages"], case["batch"]
        live = torch.randperm(n, generator=cpu)[: _live(case)].int()
        # the live pages dealt to the sequences in uneven runs; each sequence also holds the first pages of its left neighbour
        cuts = [round(len(live) * ((b + 1) / batch) ** 1.5) for b in range(batch - 1)]
        runs = [x.tolist() for x in torch.tensor_split(live, cuts)]
        rows = [runs[b - 1][: len(runs[b - 1]) // 4] + runs[b] if b else runs[b] for b in range(batch)]
        wide = max(len(r) for r in rows) + 1
        table = torch.tensor([[int(p) for p in r] + [-1] * (wide - len(r)) for r in rows], dtype=torch.int32)
        refs = torch.bincount(table[table >= 0].long(), minlength=n).int()
        lens = [max(0, len(r) * page - int(torch.randint(0, page, (1,), generator=cpu))) for r in rows]
        state |= {"pool": _pool(case, case["layers"], n, gen), "table": table.cuda(), "refs": refs.cuda(), "lens": _ints(lens)}
    return state


def _live(case):
    return case["n_pages"] * 6 // 10


# ---------------------------------------------------------------------------------------------- one pass


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    return {"attend": _attend, "append": _append, "beam": _beam, "compact": _compact}[case["kind"]](state, case)


def _run_own(state, case):
    import quantized_matmul_affine_gb300 as aq

    cache = aq.AqCache(state["pool"], case["page"], HEADS[case["heads"]][2], case["bits"], case["group"])
    if case["kind"] == "attend":
        return aq.aq_attention_batch(state["q"], cache, 0, state["table"], state["lens"], scale=state["scale"],
                                     group_start=state["starts"], shared=state["shared"])
    if case["kind"] == "append":
        aq.aq_cache_append(cache, 0, state["k"], state["v"], state["cu"], state["start"], state["table"])
        return aq.aq_cache_read(cache, 0, state["cu"], state["start"], state["table"], case["total"], state["k"].dtype)
    if case["kind"] == "beam":
        refs, table, lens, freed = aq.aq_cache_trim(cache, state["refs"], state["table"], state["lens"], state["keep"], in_place=False)
        refs, table, lens, forked = aq.aq_cache_fork(cache, refs, table, lens, state["parent"], state["whole"])
        refs, table, lens, grown = aq.aq_cache_grow(cache, refs, table, lens, state["add"])
        return {"refs": refs, "table": table, "lens": lens, "status": [freed, forked, grown], "pool": state["pool"].view(torch.int64)}
    refs, table, status = aq.aq_cache_compact(cache, state["refs"], state["table"], state["lens"], in_place=False)
    return {"refs": refs, "table": table, "status": status, "pool": state["pool"].view(torch.int64)}


def _parts(pool, case):
    """One layer's pages as K words, V words, K (scale, bias), V (scale, bias): [n_pages][KV][P][...]."""
    _, _, d = HEADS[case["heads"]]
    n, kv, page = pool.shape[0], pool.shape[1], case["page"]
    codes = page * d * case["bits"] // 8
    side = page * 4 * (d // case["group"])
    cut = [pool[..., :codes], pool[..., codes:2 * codes], pool[..., 2 * codes:2 * codes + side], pool[..., 2 * codes + side:]]
    return [x.reshape(n, kv, page, -1) for x in cut]


def _rows(words, side, pages, slots, case):
    """Cached rows as fp32 [...][KV][D], for pages and slots of shape [...]."""
    _, kv, d = HEADS[case["heads"]]
    w = words[pages, :, slots].contiguous().view(torch.int32)
    shifts = torch.arange(0, 32, case["bits"], device=w.device, dtype=torch.int32)
    codes = ((w[..., None] >> shifts) & (2 ** case["bits"] - 1)).float().view(*w.shape[:-1], -1, case["group"])
    sb = side[pages, :, slots].contiguous().view(torch.float16).float().view(*w.shape[:-1], -1, 2)
    return (codes * sb[..., :1] + sb[..., 1:]).flatten(-2)


def _softmax_part(q, k, v, seen):
    """Largest score, sum and unnormalised output: q [N][KV][M][D], k and v [N][S][KV][D], seen [N][M][S]."""
    s = torch.einsum("nkmd,nskd->nkms", q, k).masked_fill_(~seen[:, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    return top, p.sum(-1, keepdim=True), torch.einsum("nkms,nskd->nkmd", p, v)


def _attend(state, case):
    h, kv, d = HEADS[case["heads"]]
    rep, page, table, lens = h // kv, case["page"], state["table"].long(), state["lens"].long()
    batch, tokens = case["batch"], case["tokens"]
    kw, vw, ks, vs = _parts(state["pool"][0], case)
    # rows [B][KV][L * rep][D]; a row of token l sees the first lens - (L - 1 - l) keys
    q = state["q"].float().view(batch, tokens, kv, rep, d).permute(0, 2, 1, 3, 4).reshape(batch, kv, tokens * rep, d) * state["scale"]
    sees = (lens[:, None] - (tokens - 1) + torch.arange(tokens, device=lens.device)).repeat_interleave(rep, 1)
    first = torch.zeros_like(lens)
    if state["shared"] is not None:
        starts, shared = state["starts"].long(), state["shared"].long()
        group = torch.bucketize(torch.arange(batch, device=lens.device), starts[1:], right=True)
        first = shared[group]
    # every sequence's own keys
    at = first[:, None] + torch.arange(state["widest"], device=lens.device)
    pages = table.gather(1, (at // page).clamp(max=table.shape[1] - 1)).clamp(min=0)
    top, total, out = _softmax_part(q, _rows(kw, ks, pages, at % page, case), _rows(vw, vs, pages, at % page, case),
                                    at[:, None] < sees[..., None])
    if state["shared"] is not None:  # the groups' shared keys, once a group
        members = starts[:-1, None] + torch.arange(int(-(-batch // case["groups"]) + 1), device=lens.device)
        real, members = members < starts[1:, None], members.clamp(max=batch - 1)
        at = torch.arange(case["shared"], device=lens.device).expand(len(shared), -1)
        pages = table[starts[:-1]].gather(1, at // page).clamp(min=0)
        g, m = members.shape
        gq = q[members].transpose(1, 2).reshape(g, kv, m * tokens * rep, d)
        seen = (at[:, None] < sees[members].view(g, -1, 1)) & (at[:, None] < shared[:, None, None])
        gt, gs, go = _softmax_part(gq, _rows(kw, ks, pages, at % page, case), _rows(vw, vs, pages, at % page, case), seen)
        back = [x.view(g, kv, m, tokens * rep, -1).transpose(1, 2)[real] for x in (gt, gs, go)]  # in the batch's order
        both = torch.maximum(top, back[0])
        both = torch.where(both == float("-inf"), torch.zeros_like(both), both)
        a, b = torch.exp(top - both), torch.exp(back[0] - both)
        total, out = total * a + back[1] * b, out * a + back[2] * b
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    return out.view(batch, kv, tokens, rep, d).permute(0, 2, 1, 3, 4).reshape(batch, tokens, h, d).to(state["q"].dtype)


def _append(state, case):
    _, kv, d = HEADS[case["heads"]]
    page, bits, most = case["page"], case["bits"], 2 ** case["bits"] - 1
    t = torch.arange(case["total"], device="cuda")
    seq = torch.bucketize(t, state["cu"][1:].long(), right=True)
    at = state["start"].long()[seq] + t - state["cu"].long()[seq]
    pages, slots = state["table"].long()[seq, at // page], at % page
    kw, vw, ks, vs = _parts(state["pool"][0], case)
    codes, side = page * d * bits // 8, page * 4 * (d // case["group"])
    flat = state["pool"][0]
    read = []
    for n, x in enumerate((state["k"], state["v"])):
        w = x.float().reshape(case["total"], kv, -1, case["group"])
        low, high = w.amin(-1, keepdim=True), w.amax(-1, keepdim=True)
        s, b = ((high - low) / most).half(), low.half()
        q = torch.where(s > 0, torch.round((w - b.float()) / s.float()).clamp(0, most), torch.zeros_like(w)).int()
        shifts = torch.arange(0, 32, bits, device="cuda", dtype=torch.int32)
        words = (q.view(case["total"], kv, -1, 32 // bits) << shifts).sum(-1, dtype=torch.int32)
        bytes_, pairs = words.view(torch.uint8), torch.cat((s, b), -1).view(case["total"], kv, -1).view(torch.uint8)
        for data, at0, each in ((bytes_, n * codes, d * bits // 8), (pairs, 2 * codes + n * side, 4 * (d // case["group"]))):
            cols = at0 + slots[:, None] * each + torch.arange(each, device="cuda")
            flat[pages[:, None, None], torch.arange(kv, device="cuda")[:, None], cols[:, None]] = data
    kw, vw, ks, vs = _parts(state["pool"][0], case)
    return [_rows(kw, ks, pages, slots, case).to(state["k"].dtype), _rows(vw, vs, pages, slots, case).to(state["v"].dtype)]


def _status(*v):
    return torch.stack([torch.as_tensor(x, device="cuda").to(torch.int32) for x in v])


def _beam(state, case):
    page, lens, table, refs = case["page"], state["lens"], state["table"], state["refs"]
    spot = torch.arange(table.shape[1], device="cuda", dtype=torch.int32)
    row = torch.arange(len(lens), device="cuda", dtype=torch.int32)
    n = refs.shape[0]

    def tally(pages, weight):  # how often each page is named
        return torch.zeros(n, dtype=torch.int32, device="cuda").index_add_(0, pages.clamp(min=0).flatten().long(), weight.flatten().int())

    # the rows with keep >= 0 give back the pages past that length
    left = torch.where(state["keep"] >= 0, torch.minimum(state["keep"], lens), lens)
    gone = (spot >= ((left + page - 1) // page)[:, None]) & (spot < ((lens + page - 1) // page)[:, None])
    less = refs - tally(table, gone)
    freed = _status(0, 0, ((refs > 0) & (less == 0)).sum(), 0)
    refs, table, lens = less, torch.where(gone, torch.full_like(table, -1), table), left
    # the rows with a parent take its pages
    child = state["parent"] >= 0
    kept = torch.where(child, lens[state["parent"].clamp(min=0).long()], lens)
    takes = child[:, None] & (spot < ((kept + page - 1) // page)[:, None])
    table = torch.where(takes, table[state["parent"].clamp(min=0).long()], table)
    refs, lens = refs + tally(table, takes), kept
    forked = _status(0, 0, takes.sum(), 0)
    # every row grows; a shared partial page is copied, but by the last of its rows if all of them grow
    have, want = (lens + page - 1) // page, (lens + state["add"] + page - 1) // page
    part = (state["add"] > 0) & (lens % page != 0)
    last_page = table.gather(1, (lens // page).clamp(max=table.shape[1] - 1)[:, None].long())[:, 0]
    growing = tally(last_page, part)
    keeper = torch.full((n,), -1, dtype=torch.int32, device="cuda").scatter_reduce_(
        0, last_page.clamp(min=0).long(), torch.where(part, row, torch.full_like(row, -1)), "amax")
    where = last_page.clamp(min=0).long()
    copies = part & (refs[where] > 1) & ~((growing[where] >= refs[where]) & (keeper[where] == row))
    need = want - have + copies
    base = need.cumsum(0) - need
    free = torch.cumsum((refs == 0).int(), 0)  # the k-th free page is the first with free == k + 1
    new = (spot >= have[:, None]) & (spot < want[:, None])
    rank = base[:, None] + copies[:, None].int() + spot - have[:, None]
    fresh = torch.searchsorted(free, (rank + 1).clamp(min=1)).int()
    copied = torch.searchsorted(free, (base + 1).int()).int()
    swap = copies[:, None] & (spot == (lens // page)[:, None])
    refs = refs - tally(last_page, copies) + tally(copied, copies) + tally(fresh.clamp(max=n - 1), new)
    table = torch.where(new, fresh, torch.where(swap, copied[:, None], table))
    src, dst, held = last_page[copies].long(), copied[copies].long(), (lens % page)[copies]
    # only the rows that the sequence holds: their bytes in the record's four parts
    _, _, d = HEADS[case["heads"]]
    each, side = d * case["bits"] // 8, 4 * (d // case["group"])
    at = torch.arange(state["pool"].shape[-1], device="cuda")
    rest = at - 2 * page * each
    slot = torch.where(rest < 0, at % (page * each) // each, rest % (page * side) // side)
    pool = state["pool"]
    pool[:, dst] = torch.where(slot < held[:, None, None], pool[:, src], pool[:, dst])
    grown = _status(0, 0, need.sum(), copies.sum())
    return {"refs": refs, "table": table, "lens": lens + state["add"], "status": [freed, forked, grown], "pool": state["pool"].view(torch.int64)}


def _compact(state, case):
    refs, table = state["refs"], state["table"]
    n = refs.shape[0]
    page = torch.arange(n, device="cuda")
    live = refs > 0
    count = live.sum()
    holes = (~live & (page < count)).nonzero()[:, 0]
    movers = (live & (page >= count)).nonzero()[:, 0].flip(0)  # the last live page fills the first hole
    to = page.clone()
    to[movers] = holes
    fresh = refs.clone()
    fresh[holes], fresh[movers] = refs[movers], 0
    used = torch.arange(table.shape[1], device="cuda") < ((state["lens"] + case["page"] - 1) // case["page"])[:, None]
    table = torch.where(used, to[table.clamp(min=0).long()].int(), table)
    state["pool"][:, holes] = state["pool"][:, movers]
    return {"refs": fresh, "table": table, "status": _status(0, 0, count, holes.shape[0]), "pool": state["pool"].view(torch.int64)}


# ---------------------------------------------------------------------------------------------- bytes and operations


def work(case):
    h, kv, d = HEADS[case["heads"]]
    row = kv * (2 * d * case["bits"] // 8 + 8 * (d // case["group"]))  # one cached token of one layer
    if case["kind"] == "attend":
        starts, share, lens = _attend_lengths(case, 0)
        part = [next((share[g] for g in range(case["groups"]) if starts[g] <= b < starts[g + 1]), 0) for b in range(case["batch"])]
        keys = sum(share) + sum(max(0, n - s) for n, s in zip(lens, part))
        rows = case["batch"] * case["tokens"] * h
        return {"bytes": keys * row + 2 * 2 * rows * d + 4 * (keys // case["page"] + 2 * case["batch"]),
                "flops": 4 * d * h * case["tokens"] * sum(lens)}
    if case["kind"] == "append":  # rows in, codes and scales out and in again, rows out
        return {"bytes": case["total"] * (2 * 2 * 2 * kv * d + 2 * row), "flops": case["total"] * 2 * kv * d * 8}
    if case["kind"] == "beam":
        rows = case["requests"] * case["width"]
        each = case["page"] * row * case["layers"]
        # the losers' rows and their winners' partial pages are shared: one copy for each loser, of half a page on average
        held = 0.75 * case["prompt"] / case["page"] + 0.5 * case["generated"] / case["page"] + 1
        return {"bytes": case["requests"] * (case["width"] // 2) * each * (1 - 1 / case["page"]) + rows * 8 * held + 8 * rows, "flops": 0}
    each = case["page"] * row * case["layers"]
    moved = _live(case) * (case["n_pages"] - _live(case)) / case["n_pages"]
    return {"bytes": moved * 2 * each + 8 * case["n_pages"] + 8 * _live(case) * 1.25, "flops": 0}


# ---------------------------------------------------------------------------------------------- 64 bits


def _exact_rows(pool, case, which, pages, slots):
    """Rows [n][KV][D] of K (0) or V (1) in 64 bits, code by code from the record's bytes."""
    _, kv, d = HEADS[case["heads"]]
    page, bits, group = case["page"], case["bits"], case["group"]
    each, side = d * bits // 8, 4 * (d // group)
    at = torch.arange(d, device=pool.device) * bits
    heads = torch.arange(kv, device=pool.device)[None, :, None]
    byte = pool[pages[:, None, None], heads, which * page * each + slots[:, None, None] * each + at // 8]
    codes = (byte.to(torch.int64) >> (at % 8)) & (2 ** bits - 1)
    cols = 2 * page * each + which * page * side + slots[:, None, None] * side + torch.arange(side, device=pool.device)
    pair = pool[pages[:, None, None], heads, cols].contiguous().view(torch.float16).double().view(len(pages), kv, -1, 2)
    return codes.double() * pair[..., 0].repeat_interleave(group, -1) + pair[..., 1].repeat_interleave(group, -1)


def exact(case, seed):
    if case["kind"] not in ("attend", "append"):
        return None  # pages and counts: whole numbers
    state = prepare(case, seed)
    h, kv, d = HEADS[case["heads"]]
    page, table = case["page"], state["table"].long()
    if case["kind"] == "append":
        out = []
        for x in (state["k"], state["v"]):
            w = x.double().reshape(case["total"], kv, -1, case["group"])
            low, high = w.amin(-1, keepdim=True), w.amax(-1, keepdim=True)
            s, b = ((high - low) / (2 ** case["bits"] - 1)).half().double(), low.half().double()
            level = torch.where(s > 0, ((w - b) / s).round().clamp(0, 2 ** case["bits"] - 1), torch.zeros_like(w))
            out.append((s * level + b).reshape(case["total"], kv, d))
        return out
    q, lens = state["q"].double(), state["lens"].tolist()
    out = torch.zeros(case["batch"], case["tokens"], h, d, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        at = torch.arange(n, device="cuda")
        k = _exact_rows(state["pool"][0], case, 0, table[b, at // page], at % page)
        v = _exact_rows(state["pool"][0], case, 1, table[b, at // page], at % page)
        s = torch.einsum("lkrd,nkd->lkrn", q[b].view(case["tokens"], kv, h // kv, d), k) * state["scale"]
        limit = n - (case["tokens"] - 1) + torch.arange(case["tokens"], device="cuda")
        s = s.masked_fill(at >= limit[:, None, None, None], float("-inf"))
        p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e300))
        o = torch.einsum("lkrn,nkd->lkrd", p, v) / p.sum(-1, keepdim=True).clamp(min=1e-300)
        out[b] = o.reshape(case["tokens"], h, d)
    return out
