"""Cases that measure what a quantised decoder picks by index: the experts of a mixture and the token's
row of the embedding table, both in the affine format.

A weight stack holds E matrices [N][K] of codes (LSB first, `bits` each), with one fp16 scale and bias per
group of values along K: w = scale * code + bias.  A layer has three: gate and up [E][inner][hidden], down
[E][hidden][inner].

Four operators, one kind of case each:
  route    router logits, the k largest experts of each token (ties to the lowest index, listed in ascending
           order) and their weights;
  experts  y[t] = sum_j w[t][j] * down(silu(gate(x[t])) * up(x[t])) over the experts that are given for each
           token; -1 is none;
  layer    both in one call;
  embed    rows of a quantised table by token, times a factor; -1 is a row of zeros.
"""
import math

import torch

own = False


def listed():
    return [
        # one token of a chat: the router of many small experts, where latency counts
        route("route_one", 1, 2048, 128, 8, "softmax", "bf16"),
        # a full decode batch on a wide model, selection by scores with a learned bias
        route("route_batch", 256, 5120, 256, 8, "sigmoid", "fp16"),
        # one user's decode step: 8 of 128 small experts
        layer("layer_one", 1, 2048, 768, 128, 8, "softmax", 4, 64, "bf16"),
        # a few drafted tokens to verify, 3-bit experts, their number no power of two
        layer("layer_draft", 5, 2048, 1408, 60, 4, "softmax", 3, 64, "fp16"),
        # a small batch on few large experts of a 4096-wide model
        layer("layer_large", 8, 4096, 13824, 8, 2, "softmax", 4, 64, "bf16"),
        # a decode batch of unrelated chats on a 5120-wide model
        layer("layer_batch", 33, 5120, 1536, 64, 6, "sigmoid", 4, 64, "bf16"),
        # the largest: a full batch, every expert busy, 6-bit codes in groups of 32
        layer("layer_full", 256, 2048, 768, 128, 8, "softmax", 6, 32, "bf16"),
        # one token, two experts of 8 bits, routed by the caller
        experts("experts_one", 1, 4096, 1536, 16, 2, 0.0, 8, 32, "fp16"),
        # a batch whose experts lie half on this card and half elsewhere
        experts("experts_share", 48, 2048, 1024, 64, 8, 0.5, 4, 128, "bf16"),
        # a decode step's token
        embed("embed_one", 1, 128256, 4096, 4, 64, "bf16"),
        # prompts of 16k tokens together
        embed("embed_prompt", 16384, 128256, 4096, 4, 64, "bf16"),
    ]


def route(name, tokens, hidden, count, top, score, dtype):
    return dict(name=name, kind="route", tokens=tokens, hidden=hidden, count=count, top=top, score=score, dtype=dtype)


def layer(name, tokens, hidden, inner, count, top, score, bits, group, dtype):
    return dict(name=name, kind="layer", tokens=tokens, hidden=hidden, inner=inner, count=count, top=top, score=score, bits=bits,
                group=group, dtype=dtype)


def experts(name, tokens, hidden, inner, count, top, absent, bits, group, dtype):
    return dict(name=name, kind="experts", tokens=tokens, hidden=hidden, inner=inner, count=count, top=top, absent=absent, bits=bits,
                group=group, dtype=dtype)


def embed(name, tokens, vocabulary, hidden, bits, group, dtype):
    return dict(name=name, kind="embed", tokens=tokens, vocabulary=vocabulary, hidden=hidden, bits=bits, group=group, dtype=dtype)


def draw(rng):
    def log(lo, hi, step=1):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step

    bits, dtype = rng.choice((2, 3, 3, 4, 4, 4, 5, 6, 8)), rng.choice(("fp16", "bf16"))
    group = rng.choice((32, 64, 64, 128))
    step = max(group, 64)
    kind = rng.choice(("route", "layer", "layer", "layer", "experts", "embed"))
    hidden = log(512, 5120, step)
    score = rng.choice(("softmax", "sigmoid"))
    if kind == "route":
        count = log(4, 256)
        c = route("", log(1, 256), hidden, count, rng.randint(1, min(8, count)), score, dtype)
    elif kind == "embed":
        c = embed("", log(1, 16000), log(1000, 128256), hidden, bits, group, dtype)
    else:
        while True:
            count = log(4, 200)
            top = rng.randint(1, min(8, count))
            sizes = (log(1, 256), hidden, log(128, 4096, step), count, top)
            c = layer("", *sizes, score, bits, group, dtype) if kind == "layer" else \
                experts("", *sizes, rng.choice((0.0, 0.25, 0.75)), bits, group, dtype)
            if 3 * count * c["hidden"] * c["inner"] * bits / 8 < 600e6 and work(c)["flops"] < 19e9:
                break
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------- inputs


def _type(case):
    return torch.float16 if case["dtype"] == "fp16" else torch.bfloat16


def _stack(case, count, rows, cols, gen):
    """Codes of every value; scales and biases as a quantiser of centred rows leaves them."""
    bits, size = case["bits"], (count, rows, cols // case["group"])
    words = torch.randint(-2 ** 31, 2 ** 31, (count, rows, cols * bits // 32), dtype=torch.int32, device="cuda", generator=gen)
    s = (torch.rand(size, device="cuda", generator=gen) + 0.5) * (3.4 / 2 ** bits) * cols ** -0.5
    b = -(2 ** bits - 1) / 2 * s + 0.05 * cols ** -0.5 * torch.randn(size, device="cuda", generator=gen)
    return words, s.half(), b.half()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    state, tokens, hidden = {"case": case}, case["tokens"], case["hidden"]
    if case["kind"] == "embed":
        words, s, b = _stack(case, 1, case["vocabulary"], hidden, gen)
        # frequent tokens come first in a vocabulary; the last slots of a padded batch have none
        ids = (torch.rand(tokens, device="cuda", generator=gen) ** 3 * case["vocabulary"]).int().clamp(max=case["vocabulary"] - 1)
        if tokens > 8:
            ids[-2:] = -1
        return state | {"table": (words[0], s[0], b[0]), "ids": ids, "factor": hidden ** 0.5}
    # activations behind a norm: unit size, a few channels much larger
    gain = 0.5 + torch.rand(hidden, device="cuda", generator=gen)
    gain[torch.randint(0, hidden, (max(1, hidden // 256),), device="cuda", generator=gen)] *= 8
    state["x"] = (randn(tokens, hidden) * gain).to(_type(case))
    if case["kind"] != "experts":
        # some experts are liked more than others
        liked = 0.6 + 0.8 * torch.rand(case["count"], 1, device="cuda", generator=gen)
        state["router"] = (randn(case["count"], hidden) * liked * hidden ** -0.5).to(_type(case))
        state["bias"] = 0.1 * randn(case["count"]) if case["score"] == "sigmoid" else None
        state["factor"] = 2.5 if case["score"] == "sigmoid" else 1.0
    else:
        order = torch.rand(tokens, case["count"], device="cuda", generator=gen).argsort(1)[:, : case["top"]]
        away = torch.rand(tokens, case["top"], device="cuda", generator=gen) < case["absent"]
        state["ids"] = order.int().masked_fill(away, -1).contiguous()
        state["weights"] = torch.softmax(randn(tokens, case["top"]), -1)
    if case["kind"] != "route":
        for name, rows, cols in (("gate", case["inner"], hidden), ("up", case["inner"], hidden), ("down", hidden, case["inner"])):
            state[name] = _stack(case, case["count"], rows, cols, gen)
    if own:  # what a program makes once for its layer
        import quantized_matmul_affine_gb300 as aq

        if "router" in state:
            state["own_router"] = aq.AqRouter(state["router"], case["top"], bias=state["bias"], score=case["score"], scale=state["factor"])
        if "gate" in state:
            state["own_experts"] = aq.AqExperts(state["gate"], state["up"], state["down"], case["bits"], case["group"])
    return state


# ---------------------------------------------------------------------------------------------- one pass


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["kind"] == "embed":
        return _embed(state, case)
    if case["kind"] == "experts":
        return _experts(state, case, state["ids"], state["weights"])
    ids, weights = _route(state, case)
    if case["kind"] == "route":
        return {"ids": ids, "weights": weights}
    return {"y": _experts(state, case, ids, weights), "ids": ids, "weights": weights}


def _run_own(state, case):
    import quantized_matmul_affine_gb300 as aq

    if case["kind"] == "embed":
        return aq.aq_embed(state["ids"], *state["table"], case["bits"], case["group"], _type(case), scale=state["factor"])
    if case["kind"] == "experts":
        return aq.aq_moe_experts(state["x"], state["own_experts"], state["ids"], state["weights"])
    if case["kind"] == "route":
        ids, weights = aq.aq_moe_route(state["x"], state["own_router"])
        return {"ids": ids, "weights": weights}
    y, ids, weights = aq.aq_moe(state["x"], state["own_router"], state["own_experts"])
    return {"y": y, "ids": ids, "weights": weights}


def _values(stack, case, dtype=torch.float32):
    """The values of packed rows [..., K * bits / 32]."""
    words, s, b = stack
    bits, k = case["bits"], words.shape[-1] * 32 // case["bits"]
    if 32 % bits == 0:
        shifts = torch.arange(0, 32, bits, dtype=torch.int32, device=words.device)
        codes = (words[..., None] >> shifts) & (2 ** bits - 1)
    else:  # codes that may lie in two words
        at = torch.arange(k, device=words.device) * bits
        wide = words.long() & 0xFFFFFFFF
        both = wide | torch.nn.functional.pad(wide[..., 1:], (0, 1)) << 32
        codes = (both[..., at // 32] >> (at % 32)) & (2 ** bits - 1)
    codes = codes.reshape(*words.shape[:-1], -1, case["group"]).to(dtype)
    return (codes * s.to(dtype)[..., None] + b.to(dtype)[..., None]).flatten(-2)


def _route(state, case):
    # next to the border between two experts 32 bits do not tell which is larger
    logits = state["x"].double() @ state["router"].double().T
    if case["score"] == "softmax":
        score = torch.softmax(logits, -1)
        order = logits
    else:
        score = 1 / (1 + torch.exp(-logits))
        order = score + state["bias"].double()
    ids = order.sort(dim=-1, descending=True, stable=True).indices[:, : case["top"]].sort(-1).values
    weights = score.gather(1, ids)
    return ids.int(), (weights / weights.sum(-1, keepdim=True) * state["factor"]).float()


def _experts(state, case, ids, weights):
    x = state["x"].float()
    y = torch.zeros_like(x)
    for e in torch.unique(ids).tolist():
        if e < 0:
            continue
        t, j = (ids == e).nonzero(as_tuple=True)
        gate, up, down = (_values([part[e] for part in state[name]], case) for name in ("gate", "up", "down"))
        g = x[t] @ gate.T
        h = g / (1 + torch.exp(-g)) * (x[t] @ up.T)
        y.index_add_(0, t, weights[t, j, None] * (h @ down.T))
    return y.to(state["x"].dtype)


def _embed(state, case):
    ids = state["ids"].long()
    rows = _values([part[ids.clamp(min=0)] for part in state["table"]], case) * state["factor"]
    return rows.masked_fill_((ids < 0)[:, None], 0).to(_type(case))


# ---------------------------------------------------------------------------------------------- bytes and operations


def work(case):
    tokens, hidden = case["tokens"], case["hidden"]
    if case["kind"] == "embed":
        return {"bytes": tokens * (4 + hidden * (case["bits"] / 8 + 4 / case["group"] + 2)), "flops": 3 * tokens * hidden}
    routed = 8 * tokens * case["top"]
    router = {"bytes": 2 * hidden * (tokens + case["count"]) + routed, "flops": 2 * tokens * hidden * case["count"]}
    if case["kind"] == "route":
        return router
    here = 1 - case.get("absent", 0.0)
    # experts that some token picks, were all liked the same
    busy = case["count"] * (1 - (1 - case["top"] * here / case["count"]) ** tokens)
    each = 3 * hidden * case["inner"]
    total = {"bytes": busy * each * (case["bits"] / 8 + 4 / case["group"]) + 4 * tokens * hidden + routed,
             "flops": 2 * each * tokens * case["top"] * here}
    if case["kind"] == "layer":
        total["bytes"] += 2 * hidden * case["count"]
        total["flops"] += router["flops"]
    return total


# ---------------------------------------------------------------------------------------------- 64 bits


def _exact_matrix(stack, case):
    """The same values in 64 bits, each code put together from the bits of the row's bytes."""
    words, s, b = stack
    bits = case["bits"]
    data = words.contiguous().view(torch.uint8)
    at = torch.arange(words.shape[-1] * 32 // bits, device=words.device) * bits
    codes = 0
    for i in range(bits):
        codes = codes + (((data[..., (at + i) // 8].to(torch.int32) >> ((at + i) % 8).int()) & 1) << i)
    return codes.double() * s.double().repeat_interleave(case["group"], -1) + b.double().repeat_interleave(case["group"], -1)


def exact(case, seed):
    state = prepare(case, seed)
    if case["kind"] == "embed":
        out = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
        for part in torch.arange(case["tokens"], device="cuda").split(2048):
            part = part[state["ids"][part] >= 0]
            rows = state["ids"][part].long()
            out[part] = _exact_matrix([p[rows] for p in state["table"]], case) * state["factor"]
        return out
    x = state["x"].double()
    if case["kind"] == "experts":
        ids, weights = state["ids"].long(), state["weights"].double()
    else:
        logits = torch.stack([(x * row.double()).sum(-1) for row in state["router"]], -1)
        likes = logits if case["score"] == "softmax" else torch.sigmoid(logits) + state["bias"].double()
        rest, chosen = likes.clone(), []
        for _ in range(case["top"]):  # argmax gives the lowest of equal ones
            best = (rest == rest.amax(-1, keepdim=True)).int().argmax(-1)
            chosen.append(best)
            rest[torch.arange(len(x), device="cuda"), best] = float("-inf")
        ids = torch.stack(chosen, -1).sort(-1).values
        picked = logits.gather(1, ids)
        weights = torch.exp(picked - picked.amax(-1, keepdim=True)) if case["score"] == "softmax" else torch.sigmoid(picked)
        weights = weights / weights.sum(-1, keepdim=True) * state["factor"]
        if case["kind"] == "route":
            return {"ids": None, "weights": weights}
    y = torch.zeros_like(x)
    for e in range(case["count"]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        gate, up, down = (_exact_matrix([p[e] for p in state[name]], case) for name in ("gate", "up", "down"))
        g = x[t] @ gate.T
        out = weights[t, j, None] * ((g * torch.sigmoid(g) * (x[t] @ up.T)) @ down.T)
        for n, at in enumerate(t.tolist()):
            y[at] += out[n]
    return y if case["kind"] == "experts" else {"y": y, "ids": None, "weights": weights}
