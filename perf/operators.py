"""What the serving operators around BitLinear cost: the cases that are measured, and their plain forms.

Four operators that a decoder layer built on this library runs between its BitLinear products:

``layer``      residual addition, RMS normalisation and per-token activation codes in one pass
               (``bitnet_act_quant_residual_norm``), alone or followed by the ternary product
               (``bitnet_residual_norm_bitlinear_forward``);
``append``     K and V states written into a paged 8-bit cache, one scale for each block of tokens
               and head (``bitnet_kv_cache_append``);
``read``       cached states read back as bf16 (``bitnet_kv_cache_read``);
``attention``  attention of new tokens over that cache (``bitnet_kv_attention``).

With ``own`` false, ``run`` computes them with elementary torch operations in fp32; with ``own``
true it makes the calls that a program makes of the library.

The cache.  Codes are int8 [pages, kv_heads, page_tokens, head_dim]; scales float
[pages, kv_heads, page_tokens / scale_tokens], the step d of a block of ``scale_tokens`` tokens of
one head (a token's state is code * d).  A sequence's token at position p lies in page
page_table[sequence, p // page_tokens].  ``q_start`` [batch + 1] says which rows of the packed new
tokens belong to a sequence, ``kv_len`` [batch] its length with these tokens: they are its last.

Writing tokens into a block (fp32): mx = max(|x| of the block's new tokens and this head, 1e-5);
g_old = 127 * d_old, or 0 where the block's first token is among the new ones; mx > g_old sets
g = mx, d = g / 127, else g = g_old, d = d_old; s = 127 / g; new codes are round(x * s), old ones
round(c * (d_old * s)) where d changed.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
Q8 = 127.0
FLOOR = 1e-5                      # the smallest maximum that a scale is made of
SQRT7 = float(np.float32(math.sqrt(7.0)))
EPS = 1e-5                        # of the RMS normalisation


def listed():
    """Sizes are those of the workloads in synth.py (hidden 2048 and 4096), heads of 64 or 128."""
    return [
        # one token's residual + norm + INT8 codes: decoding with batch 1, where latency counts
        dict(name="layer_token", op="layer", tokens=1, width=2048, bits=8, out=0),
        # a 4096-token prompt at hidden 2048
        dict(name="layer_prompt", op="layer", tokens=4096, width=2048, bits=8, out=0),
        # an odd number of tokens at hidden 4096, the largest pass over the residual stream
        dict(name="layer_wide", op="layer", tokens=16383, width=4096, bits=8, out=0),
        # INT4 activations straight into the fused Q/K/V product (16 + 2 * 2 heads of 128)
        dict(name="layer_qkv_int4", op="layer", tokens=4096, width=2048, bits=4, out=2560),
        # one new token for each of 64 running sequences of ragged lengths
        dict(name="append_tokens", op="append", batch=64, prefix=4000, ragged=1, new=1,
             kv_heads=8, head_dim=128, page=64, block=16),
        # prompts continued at an odd position: a partly filled block and page first
        dict(name="append_prompt", op="append", batch=3, prefix=1001, ragged=1, new=4099,
             kv_heads=8, head_dim=128, page=64, block=16),
        # the last 257 tokens of some sequences, heads of 64
        dict(name="read_tail", op="read", batch=5, prefix=1000, ragged=1, new=257, kv_heads=4,
             head_dim=64, page=32, block=32),
        # whole sequences out of the cache (to hand one over, or to compute on in bf16)
        dict(name="read_whole", op="read", batch=4, prefix=0, ragged=1, new=16384, kv_heads=8,
             head_dim=128, page=64, block=64),
        # one token over a short cache: the smallest attention call
        dict(name="attention_short", op="attention", batch=1, prefix=300, ragged=0, new=1,
             q_heads=16, kv_heads=2, head_dim=128, page=64, block=16),
        # decoding a batch of ragged sequences, four query heads to a key head
        dict(name="attention_batch", op="attention", batch=32, prefix=8000, ragged=1, new=1,
             q_heads=32, kv_heads=8, head_dim=128, page=64, block=16),
        # one token over a very long cache: few rows, a long axis
        dict(name="attention_long", op="attention", batch=1, prefix=131072, ragged=0, new=1,
             q_heads=32, kv_heads=8, head_dim=128, page=128, block=64),
        # a prompt chunk behind 1000 cached tokens, causal: the matrix-product bound form
        dict(name="attention_prompt", op="attention", batch=1, prefix=1000, ragged=0, new=6001,
             q_heads=16, kv_heads=2, head_dim=128, page=64, block=16),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["layer", "append", "read", "attention", "attention", "attention"])
    if op == "layer":
        out = rng.choice([0, 0, 0, 1280, 2048, 2560])
        width = 128 * _log(rng, 2, 40)
        return dict(op=op, tokens=_log(rng, 1, 8192), width=width,
                    bits=rng.choice([4, 8]) if out else 8, out=out)
    head_dim = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    case = dict(op=op, batch=1, prefix=0, ragged=rng.randint(0, 1), new=1)
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    layout = dict(kv_heads=kv_heads, head_dim=head_dim, page=page,
                  block=rng.choice([b for b in (16, 32, 64, 128) if b <= page]))
    if op == "append":
        case["batch"] = _log(rng, 1, 64)
        case["prefix"] = _log(rng, 1, 4000)
        case["new"] = rng.choice([1, _log(rng, 1, 12288 // case["batch"] + 1)])
        return {**case, **layout}
    if op == "read":
        case["batch"] = _log(rng, 1, 16)
        case["new"] = _log(rng, 1, 60000 // case["batch"])
        case["prefix"] = rng.choice([0, _log(rng, 1, 3000)])
        return {**case, **layout}
    group = rng.choice([1, 2, 4, 7, 8])
    case["q_heads"] = group * kv_heads
    kind = rng.choice(["token", "token", "draft", "prompt"])
    if kind == "prompt":
        case["batch"] = rng.choice([1, 1, 2])
        case["new"] = _log(rng, 20, 2500)
        case["prefix"] = rng.choice([0, _log(rng, 1, 2500)])
    else:
        case["batch"] = _log(rng, 1, 48)
        case["new"] = 1 if kind == "token" else rng.randint(2, 9)
        case["prefix"] = _log(rng, 1, min(60000, 200000 // case["batch"]))
    return {**case, **layout}


# ---------------------------------------------------------------------------------------------
# sizes
# ---------------------------------------------------------------------------------------------
def _lengths(case):
    """(new tokens, length with them) of each sequence: from a quarter of the largest up, where
    the batch is ragged."""
    new, total = [], []
    for i in range(case["batch"]):
        f = 1.0 - (0.75 * ((0.6180339887 * i) % 1.0) if case["ragged"] else 0.0)
        n = max(1, int(round(case["new"] * f))) if case["new"] > 1 else 1
        new.append(n)
        total.append(n + int(case["prefix"] * f))
    return new, total


def _pages(case):
    return [-(-length // case["page"]) for length in _lengths(case)[1]]


def work(case):
    if case["op"] == "layer":
        M, K, N = case["tokens"], case["width"], case["out"]
        moved = M * K * (2 + 2 + 2) + 2 * K
        if N:
            return {"bytes": moved + N * K // 4 + 2 * M * N, "flops": 2 * M * K * N + 12 * M * K}
        return {"bytes": moved + M * K + 8 * M, "flops": 12 * M * K}
    new, total = _lengths(case)
    width, T = case["kv_heads"] * case["head_dim"], sum(new)
    if case["op"] == "append":  # states in, codes out, the step of each touched block
        blocks = sum((length - 1) // case["block"] - (length - n) // case["block"] + 1
                     for n, length in zip(new, total))
        return {"bytes": 2 * T * width * 3 + 2 * blocks * case["kv_heads"] * 8,
                "flops": 2 * T * width * 3}
    if case["op"] == "read":
        return {"bytes": 2 * T * width * 3 + 2 * T * case["kv_heads"] * 4 / case["block"],
                "flops": 2 * T * width}
    cached = sum(total) * 2 * (width + 4 * case["kv_heads"] / case["block"])
    seen = sum(n * (length - n) + n * (n + 1) // 2 for n, length in zip(new, total))
    return {"bytes": cached + T * case["q_heads"] * (4 * case["head_dim"] + 4),
            "flops": 4 * seen * case["q_heads"] * case["head_dim"]}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _states(gen, shape, outliers):
    """bf16 states [tokens, heads, head_dim], near Gaussian; keys have some channels that are much
    larger than the others, as after a product with trained weights."""
    x = torch.randn(shape, generator=gen, device=DEVICE)
    if outliers:
        gain = torch.ones(shape[1:], device=DEVICE)
        gain[:, ::29] = 6.0
        x *= gain
    return x.bfloat16()


def _pack_ternary(q):
    """Offset codes q + 1, weight 16g + 4p + j of a row at bits 8j + 2p of its word g."""
    N, K = q.shape
    u = (q + 1).to(torch.uint8).view(N, K // 16, 4, 4)  # word, p, j
    return (u[:, :, 0] | u[:, :, 1] << 2 | u[:, :, 2] << 4 | u[:, :, 3] << 6).reshape(N, K // 4)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    if case["op"] == "layer":
        M, K, N = case["tokens"], case["width"], case["out"]
        s = {"case": case}
        s["x"] = torch.randn((M, K), generator=gen, device=DEVICE).mul_(0.3).bfloat16()
        r = torch.randn((M, K), generator=gen, device=DEVICE)
        r[:, :: max(1, K // 9)] *= 20.0  # the residual stream's few large features
        s["r"] = r.bfloat16()
        s["gain"] = (1 + 0.2 * torch.randn(K, generator=gen, device=DEVICE)).bfloat16()
        if N:
            q = torch.randint(-1, 2, (N, K), generator=gen, device=DEVICE, dtype=torch.int8)
            s["q"], s["Wp"] = q, _pack_ternary(q)
            s["gamma"] = torch.full((1,), 0.016, device=DEVICE)
        return s
    H, D, P, S = case["kv_heads"], case["head_dim"], case["page"], case["block"]
    new, total = _lengths(case)
    pages, B = _pages(case), case["batch"]
    count = sum(pages) + 3  # some pages belong to nobody
    s = {"case": case}
    order = torch.randperm(count, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.zeros((B, max(pages)), dtype=torch.int32, device=DEVICE)
    at = 0
    for b in range(B):
        table[b, : pages[b]] = order[at : at + pages[b]]
        at += pages[b]
    s["page_table"] = table
    s["q_start"] = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=DEVICE)
    s["kv_len"] = torch.tensor(total, dtype=torch.int32, device=DEVICE)
    s["max_new"], s["tokens"] = max(new), sum(new)
    for which, outliers in (("k", True), ("v", False)):  # a cache that earlier calls have filled
        x = _states(gen, (count * P, H, D), outliers).view(count, P, H, D).transpose(1, 2)
        blocks = x.reshape(count, H, P // S, S * D)
        step = blocks.abs().amax(-1).float().clamp_(min=FLOOR) / Q8
        s[which + "_scales"] = step.contiguous()
        codes = torch.round(blocks.float() / step[..., None])
        s[which + "_codes"] = codes.to(torch.int8).view(count, H, P, D)
    if case["op"] == "append":
        # Q, K and V come out of one product: the states are column slices of its rows
        width = H * D
        qkv = torch.empty((s["tokens"], 4 * width), dtype=torch.bfloat16, device=DEVICE)
        qkv[:, : 2 * width] = 0
        qkv[:, 2 * width : 3 * width] = _states(gen, (s["tokens"], H, D), True).flatten(1)
        qkv[:, 3 * width :] = _states(gen, (s["tokens"], H, D), False).flatten(1)
        s["k"], s["v"] = qkv[:, 2 * width : 3 * width], qkv[:, 3 * width :]
        # the tokens whose stored state the call may change: the new ones and those before them
        # in the first block
        back = [min(length, n + S - 1) for n, length in zip(new, total)]
        s["read_start"] = torch.tensor([0] + list(np.cumsum(back)), dtype=torch.int32,
                                       device=DEVICE)
        s["read_tokens"] = sum(back)
    if case["op"] == "attention":
        s["q"] = _states(gen, (s["tokens"], case["q_heads"], D), False).flatten(1)
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "layer":
        return _plain_layer(state)
    if op == "append":
        for which in ("k", "v"):
            _plain_append(state, state[which], state[which + "_codes"], state[which + "_scales"])
        return _plain_read(state, state["read_start"], state["read_tokens"])
    if op == "read":
        return _plain_read(state, state["q_start"], state["tokens"])
    return _plain_attention(state)


def _run_own(state):
    from bit_activation_linear_b200 import binding as B
    case = state["case"]
    if case["op"] == "layer":
        if case["out"]:
            h, y = B.bitnet_residual_norm_bitlinear_forward(
                state["x"], state["r"], state["gain"], EPS, state["Wp"], state["gamma"],
                case["bits"])
            return {"h": h, "y": y}
        h, codes, scales, rowsum = B.bitnet_act_quant_residual_norm(
            state["x"], state["r"], state["gain"], EPS, case["bits"])
        values = torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device)
        torch.mul(codes, scales.unsqueeze(1), out=values)
        return {"h": h, "values": values}
    cache = state.get("cache")
    if cache is None:  # the program's handle on its cache
        cache = state["cache"] = B.KvCache(state["k_codes"], state["v_codes"], state["k_scales"],
                                           state["v_scales"])
    if case["op"] == "append":
        B.bitnet_kv_cache_append(cache, state["k"], state["v"], state["q_start"],
                                 state["kv_len"], state["page_table"])
        k, v = B.bitnet_kv_cache_read(cache, state["read_tokens"], state["read_start"],
                                      state["kv_len"], state["page_table"])
        return {"k": k, "v": v}
    if case["op"] == "read":
        k, v = B.bitnet_kv_cache_read(cache, state["tokens"], state["q_start"], state["kv_len"],
                                      state["page_table"])
        return {"k": k, "v": v}
    y, lse = B.bitnet_kv_attention(cache, state["q"], case["q_heads"], state["q_start"],
                                   state["kv_len"], state["page_table"], state["max_new"],
                                   causal=True, want_lse=True)
    return {"y": y, "lse": lse}


def _plain_layer(state):
    case = state["case"]
    h = (state["x"].float() + state["r"].float()).bfloat16()
    y = h.float()
    rinv = 1.0 / torch.sqrt(y.square().mean(-1, keepdim=True) + EPS)
    y = y * rinv * state["gain"].float()
    if case["bits"] == 8:
        g = y.abs().amax(-1, keepdim=True).clamp(min=FLOOR)
        codes, step = torch.round(y * (Q8 / g)), g / Q8
    else:
        g = y.abs().double().mean(-1, keepdim=True).clamp(min=FLOOR).float()
        codes, step = torch.round(y * (SQRT7 / g)).clamp(-8, 7), g / SQRT7
    if not case["out"]:
        return {"h": h, "values": (codes * step).bfloat16()}
    acc = codes @ state["q"].float().t()
    return {"h": h, "y": (acc * (step * state["gamma"])).bfloat16()}


def _places(state, start, tokens):
    """(sequence, page, offset in the page) of each of the packed tokens."""
    t = torch.arange(tokens, device=DEVICE)
    seq = torch.searchsorted(start[1:], t, right=True)
    count = start[1:] - start[:-1]
    position = state["kv_len"][seq] - count[seq] + (t - start[seq])
    P = state["case"]["page"]
    page = state["page_table"][seq, position // P].long()
    return seq, page, position % P


def _plain_append(state, x, codes, scales):
    case = state["case"]
    H, D, P, S = case["kv_heads"], case["head_dim"], case["page"], case["block"]
    x = x.float().view(-1, H, D)
    start = state["q_start"].long()
    _, page, offset = _places(state, start, state["tokens"])
    per_page = P // S
    slot = page * per_page + offset // S
    slots = scales.shape[0] * per_page
    # the largest new state of each block and head, and the blocks that begin with a new token
    mx = torch.zeros((slots, H), device=DEVICE)
    mx.scatter_reduce_(0, slot[:, None].expand(-1, H), x.abs().amax(-1), "amax")
    mx = mx.clamp(min=FLOOR)
    fresh = torch.zeros(slots, device=DEVICE)
    fresh.scatter_reduce_(0, slot, (offset % S == 0).float(), "amax")
    d_old = scales.transpose(1, 2).reshape(slots, H)
    g_old = torch.where(fresh[:, None] > 0, 0.0, d_old * Q8)
    grown = mx > g_old
    g = torch.where(grown, mx, g_old)
    d = torch.where(grown, g / Q8, d_old)
    s = Q8 / g
    # tokens that were there before, in the block of each sequence's first new token
    first = slot[start[:-1]]
    factor = torch.where(grown & (fresh[:, None] == 0), d_old * s, 1.0)[first]
    blocks = codes.view(-1, H, per_page, S, D)
    old = blocks[first // per_page, :, first % per_page].float()
    blocks[first // per_page, :, first % per_page] = torch.round(
        old * factor[:, :, None, None]).to(torch.int8)
    codes[page, :, offset] = torch.round(x * s[slot][:, :, None]).to(torch.int8)
    new_steps = d[slot]
    scales[page, :, offset // S] = new_steps


def _plain_read(state, start, tokens):
    case = state["case"]
    _, page, offset = _places(state, start.long(), tokens)
    out = {}
    for which in ("k", "v"):
        step = state[which + "_scales"][page, :, offset // case["block"]]
        value = state[which + "_codes"][page, :, offset].float() * step[:, :, None]
        out[which] = value.bfloat16().flatten(1)
    return out


def _plain_attention(state):
    case = state["case"]
    H, D, S = case["kv_heads"], case["head_dim"], case["block"]
    G, B, n = case["q_heads"] // H, case["batch"], state["max_new"]
    start, length = state["q_start"].long(), state["kv_len"].long()
    count = start[1:] - start[:-1]
    table = state["page_table"].long()

    def gathered(which):  # [batch, kv_heads, tokens, head_dim]
        step = state[which + "_scales"][table].repeat_interleave(S, dim=3)
        value = state[which + "_codes"][table].float() * step[..., None]
        return value.transpose(1, 2).reshape(B, H, -1, D)

    i = torch.arange(n, device=DEVICE)
    row = (start[:-1, None] + i).clamp(max=state["tokens"] - 1)       # [batch, n]
    q = state["q"].float().view(-1, H, G, D)[row]                     # [batch, n, H, G, D]
    q = q.permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D)
    score = (q @ gathered("k").transpose(2, 3)) * (1.0 / math.sqrt(D))
    position = (length - count)[:, None] + i                          # [batch, n]
    column = torch.arange(score.shape[-1], device=DEVICE)
    seen = (column <= position[..., None]) & (column < length[:, None, None])
    seen = seen[:, None, :, None, :].expand(B, 1, n, G, -1).reshape(B, 1, n * G, -1)
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    y = (p @ gathered("v")) / torch.where(total == 0, 1.0, total)
    lse = torch.where(total == 0, -math.inf, top + torch.log(total))
    y = y.view(B, H, n, G, D).permute(0, 2, 1, 3, 4)
    lse = lse.view(B, H, n, G).permute(0, 2, 1, 3)
    t = torch.arange(state["tokens"], device=DEVICE)
    seq = torch.searchsorted(start[1:], t, right=True)
    at = (seq, t - start[seq])
    return {"y": y[at].reshape(-1, H * G * D).bfloat16(),
            "lse": lse[at].reshape(-1, H * G).contiguous()}


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layer":
        h = (s["x"].double() + s["r"].double()).to(torch.bfloat16)
        y = h.double()
        y = y / (y.pow(2).sum(1, keepdim=True) / y.shape[1] + EPS).sqrt() * s["gain"].double()
        if case["bits"] == 8:
            step = torch.maximum(y.abs().max(1, keepdim=True)[0], torch.tensor(FLOOR)) / 127
            codes = (y / step).round()
        else:
            step = torch.maximum(y.abs().mean(1, keepdim=True), torch.tensor(FLOOR)) / 7 ** 0.5
            codes = (y / step).round().clamp(-8, 7)
        value = codes * step
        if case["out"]:
            value = value @ s["q"].double().t() * s["gamma"].double()
            return {"h": s["x"].double() + s["r"].double(), "y": value}
        return {"h": s["x"].double() + s["r"].double(), "values": value}
    H, D, P, S = case["kv_heads"], case["head_dim"], case["page"], case["block"]
    new, total = _lengths(case)

    def sequence(which, b):
        """The codes [tokens, H, D] and the steps [tokens, H] of one sequence, in 64 bits."""
        pages = s["page_table"][b, : -(-total[b] // P)].long()
        c = s[which + "_codes"][pages].double().transpose(1, 2).reshape(-1, H, D)[: total[b]]
        d = s[which + "_scales"][pages].double().transpose(1, 2).reshape(-1, H)
        return c, d.repeat_interleave(S, 0)[: total[b]]

    if case["op"] in ("append", "read"):
        out = {}
        for which in ("k", "v"):
            parts, at = [], 0
            for b in range(case["batch"]):
                c, d = sequence(which, b)
                first = total[b] - new[b]
                if case["op"] == "append":
                    x = s[which][at : at + new[b]].double().view(-1, H, D)
                    at += new[b]
                    for lo in range(first // S * S, total[b], S):
                        hi, mid = min(lo + S, total[b]), max(lo, first)
                        most = x[mid - first : hi - first].abs().amax((0, 2)).clamp(min=FLOOR)
                        before = d[lo] if mid > lo else torch.zeros_like(most)
                        step = torch.maximum(most / 127, before)
                        c[lo:mid] = (c[lo:mid] * (before / step)[:, None]).round()
                        c[mid:hi] = (x[mid - first : hi - first] / step[:, None]).round()
                        d[lo:hi] = step
                    first = max(0, first - S + 1)
                parts.append((c * d[..., None])[first:].reshape(-1, H * D))
            out[which] = torch.cat(parts)
        return out
    G = case["q_heads"] // H
    ys, lses, at = [], [], 0
    for b in range(case["batch"]):
        k, v = ((c * d[..., None]).transpose(0, 1) for c, d in (sequence("k", b),
                                                                sequence("v", b)))
        q = s["q"][at : at + new[b]].double().view(new[b], H, G, D)
        at += new[b]
        for lo in range(0, new[b], 512):
            rows = q[lo : lo + 512].permute(1, 0, 2, 3)          # H, rows, G, D
            score = torch.einsum("hrgd,hld->hrgl", rows, k) / D ** 0.5
            last = total[b] - new[b] + lo + torch.arange(rows.shape[1], device=DEVICE)
            score = score.masked_fill(
                torch.arange(total[b], device=DEVICE) > last[None, :, None, None], -math.inf)
            lses.append(torch.logsumexp(score, -1).permute(1, 0, 2).reshape(-1, H * G))
            y = torch.einsum("hrgl,hld->hrgd", torch.softmax(score, -1), v)
            ys.append(y.permute(1, 0, 2, 3).reshape(-1, H * G * D))
    return {"y": torch.cat(ys), "lse": torch.cat(lses)}
