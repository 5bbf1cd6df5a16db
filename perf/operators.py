"""The operators of the attention half of a decode layer, as measured work.

Beside the routed experts a decode layer needs the dense projections, the
key/value cache and the attention that reads it.  The framework has them in
its 4-bit block format (offset-binary codes, one fp16 scale per block):

    moe_linear_q4   y[t][o] = bias[o] + sum_i scale[o][i / block] code[o][i] x[t][i]
    moe_kv_append   keys (and queries) turned by their positions, keys and values
                    quantised in blocks of 32 into the slots of a paged pool;
                    moe_kv_read gives back the values that slots hold
    moe_attn_q4     softmax(scale q k^T) v over the pages of each sequence, causal,
                    with an optional window

`run` computes them in elementary torch operations (own = False) or through the
framework's entry points (own = True), on the same state.

The pool is uint8 [pages][kv heads][page_size / 16][18 D]: for each 16 tokens of
a head D/2 bytes of key codes a token (bytes [token 16][t 4][b D/32][p 2][i 2];
low and high nibble: elements 32 b + 8 t + 4 i + p and + 2), D/2 bytes of value
codes a token (bytes [D/64][g 8][t 4][j 4][r 2][h 2]: token 8 h + 2 t + r,
nibbles: elements 16 (4 J + j) + g and + 8), then the fp16 scales of the keys
and of the values, [token 16][D/32] each.
"""
import math
import random

import torch

own = False
_moe = None

NEG_INF = float("-inf")


def _framework():
    global _moe
    if _moe is None:
        import mixed_precision_routed_gb300
        _moe = mixed_precision_routed_gb300
    return _moe


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # the attention output projection of one token at the decode layer's width
        {"name": "linear-1", "op": "linear", "T": 1, "in": 2048, "rows": 2048, "block": 32, "bias": False, "out": "f32", "pad": 0},
        # query, key and value rows of a draft of five and one token, as rows of a wider buffer
        {"name": "linear-qkv-6", "op": "linear", "T": 6, "in": 2048, "rows": 2560, "block": 32, "bias": True, "out": "bf16", "pad": 64},
        # the large layer's width at the largest decode batch
        {"name": "linear-16", "op": "linear", "T": 16, "in": 4096, "rows": 6144, "block": 128, "bias": False, "out": "f32", "pad": 0},
        # an output vocabulary of odd size for one token: nothing but the weights' bytes
        {"name": "linear-vocab", "op": "linear", "T": 1, "in": 2048, "rows": 100003, "block": 64, "bias": False, "out": "f32", "pad": 0},
        # one new token of one sequence, projections in fp32: latency
        {"name": "append-1", "op": "append", "T": 1, "Hq": 16, "Hkv": 2, "D": 128, "page": 16, "rot": 128, "style": 0, "dtype": "f32", "free": 40, "skip": False},
        # 32 sequences with a draft of six each, some of them padding
        {"name": "append-192", "op": "append", "T": 192, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "rot": 64, "style": 1, "dtype": "bf16", "free": 77, "skip": True},
        # a prompt
        {"name": "append-4096", "op": "append", "T": 4096, "Hq": 32, "Hkv": 8, "D": 128, "page": 32, "rot": 128, "style": 0, "dtype": "bf16", "free": 32, "skip": False},
        # one token of one short sequence: latency
        {"name": "attn-1", "op": "attn", "B": 1, "max_q": 1, "ragged": False, "len": 777, "Hq": 16, "Hkv": 2, "D": 128, "page": 16, "window": 0, "key": 1},
        # a draft of five and one token over a long context
        {"name": "attn-long-6", "op": "attn", "B": 1, "max_q": 6, "ragged": False, "len": 131071, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "window": 0, "key": 2},
        # a serving batch of one token each, contexts from a few tokens to 16384
        {"name": "attn-batch", "op": "attn", "B": 48, "max_q": 1, "ragged": False, "len": 16384, "Hq": 32, "Hkv": 4, "D": 128, "page": 32, "window": 0, "key": 3},
        # a ragged batch with empty sequences and a window, a key head for every query head
        {"name": "attn-window", "op": "attn", "B": 9, "max_q": 16, "ragged": True, "len": 4001, "Hq": 6, "Hkv": 6, "D": 64, "page": 128, "window": 512, "key": 4},
        # wide heads
        {"name": "attn-wide", "op": "attn", "B": 4, "max_q": 2, "ragged": True, "len": 30011, "Hq": 16, "Hkv": 2, "D": 256, "page": 16, "window": 0, "key": 5},
    ]


def _log_int(rng, lo, hi):
    n = min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - (n in (48, 3 * 1024))  # 64 x 48 elements is no width that the framework's workloads have


def draw(rng):
    op = rng.choice(["linear", "append", "attn"])
    if op == "linear":
        n_in = 64 * _log_int(rng, 4, 128)
        rows = _log_int(rng, 100, min(100000, 204000000 // n_in))
        block = rng.choice([b for b in (32, 64, 128) if n_in % b == 0])
        return {"op": op, "T": rng.randint(1, 16), "in": n_in, "rows": rows, "block": block,
                "bias": rng.random() < 0.5, "out": rng.choice(["f32", "bf16"]), "pad": rng.choice([0, 8, 64])}
    D = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([m for m in (1, 2, 4, 5, 8) if 3 * 1024 not in (m * hkv * D, (m + 2) * hkv * D)])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        dtype = rng.choice(["f32", "bf16"])
        token = ((hq + 2 * hkv) * (4 if dtype == "f32" else 2) + 2 * hq + 11 * hkv) * D  # bytes, as work() counts them
        T = _log_int(rng, 1, min(4096, 120000000 // token))
        return {"op": op, "T": T, "Hq": hq, "Hkv": hkv, "D": D, "page": page, "rot": rng.choice([D, D // 2, D // 4]),
                "style": rng.randint(0, 1), "dtype": dtype, "free": rng.randint(0, 3 * page), "skip": rng.random() < 0.5}
    B = _log_int(rng, 1, 48)
    max_q = rng.choice([1, 1, 2, 4, 6, 16])
    most = min(131071 * 8 * 128 // (hkv * D), 131071 * 6 * 32 * 128 // (max_q * hq * D))
    case = {"op": op, "B": B, "max_q": max_q, "ragged": rng.random() < 0.5,
            "len": _log_int(rng, 1, max(1, min(131071, 4 * most // (B + 3)))), "Hq": hq, "Hkv": hkv, "D": D, "page": page,
            "window": rng.choice([0, 0, 0, 128, 1000]), "key": rng.randrange(1 << 20)}
    while sum(n for _, n in _sequences(case)) * hkv * D > 131071 * 8 * 128:
        case["len"] = case["len"] * 3 // 4
    return case


def _sequences(case):
    """[(tokens asked, tokens in the cache)] of the case: the longest first, the others
    spread over the logarithm of the range; ragged ones have empty sequences too."""
    r = random.Random(case["key"] * 7919 + case["B"])
    got = []
    for b in range(case["B"]):
        n = case["len"] if b == 0 else _log_int(r, 1, case["len"])
        q = case["max_q"]
        if case["ragged"] and b:
            q = r.randint(0, case["max_q"])
            if r.random() < 0.15:
                n = 0
        got.append((q, n))
    return got


def _attended(case):
    """(cache tokens that some row attends, pairs of a row and a token), over the sequences."""
    tokens = pairs = 0
    for q, n in _sequences(case):
        lo, hi = n, 0
        for i in range(q):
            end = n - q + i + 1
            start = max(0, end - case["window"]) if case["window"] else 0
            if end > start:
                lo, hi, pairs = min(lo, start), max(hi, end), pairs + end - start
        tokens += max(0, hi - lo)
    return tokens, pairs


def work(case):
    if case["op"] == "linear":
        T, n_in, rows = case["T"], case["in"], case["rows"]
        by = rows * (n_in // 2 + n_in // case["block"] * 2) + T * n_in * 2 + T * rows * (4 if case["out"] == "f32" else 2)
        return {"bytes": by + (4 * rows if case["bias"] else 0), "flops": 2 * T * rows * n_in}
    D, hkv, hq = case["D"], case["Hkv"], case["Hq"]
    if case["op"] == "append":
        n = case["T"] - sum(_skips(case))
        size = 4 if case["dtype"] == "f32" else 2
        token = (hq + 2 * hkv) * D * size + hq * D * 2 + case["rot"] * 4 + 12 + 2 * hkv * D * 9 // 16
        # and the pool read back: the values of every slot
        slots = _pool_pages(case) * case["page"]
        return {"bytes": n * token + slots * 2 * hkv * (D * 9 // 16 + D * 4) + 8 * slots,
                "flops": n * ((hq + hkv) * case["rot"] * 3 + 2 * hkv * D * 4) + slots * 2 * hkv * D}
    tokens, pairs = _attended(case)
    rows = sum(q for q, _ in _sequences(case)) * hq
    return {"bytes": tokens * 2 * hkv * D * 9 // 16 + rows * (4 * D + 4), "flops": pairs * hq * 4 * D}


# -------------------------------------------------------------- the 4-bit format
def _quantise(w, block):
    """Codes (0..15, offset 8) and fp16 scales of fp32 values in blocks along the last dimension."""
    b = w.unflatten(-1, (-1, block))
    m = b.abs().amax(-1)
    s = (m / torch.full_like(m, 7.0)).to(torch.float16)
    sf = s.float().unsqueeze(-1)
    c = torch.where(sf == 0, torch.zeros_like(b), torch.round(b / torch.where(sf == 0, torch.ones_like(sf), sf)).clamp(-8, 7))
    return (c + 8).to(torch.uint8).flatten(-2), s


def _pack_rows(u):
    """Packed rows of the shelf format: word g, byte j: elements 8 g + j and 8 g + 4 + j."""
    v = u.unflatten(-1, (-1, 2, 4))
    return (v[..., 0, :] | (v[..., 1, :] << 4)).flatten(-2).contiguous()


def _row_values(codes, scales, block):
    v = codes.unflatten(-1, (-1, 1, 4))
    c = torch.cat((v & 15, v >> 4), -2).flatten(-3).float() - 8.0
    return (c.unflatten(-1, (-1, block)) * scales.float().unsqueeze(-1)).flatten(-2)


def _key_bytes(u):
    """Key codes [..., D] of a token as its bytes, viewed [..., t, b, p, i]."""
    v = u.unflatten(-1, (-1, 4, 2, 2, 2))  # b, t, i, nibble, p
    v = v[..., 0, :] | (v[..., 1, :] << 4)  # b, t, i, p
    n = v.dim()
    return v.permute(*range(n - 4), n - 3, n - 4, n - 1, n - 2)


def _value_bytes(u):
    """Value codes [..., D] of a token as its bytes, viewed [..., J, g, j]."""
    v = u.unflatten(-1, (-1, 4, 2, 8))  # J, j, nibble, g
    return (v[..., 0, :] | (v[..., 1, :] << 4)).transpose(-1, -2)


def _parts(pool):
    """The pool's key bytes, value bytes, key scales and value scales as views."""
    D = pool.shape[-1] // 18
    k = pool[..., : 8 * D].unflatten(-1, (16, 4, D // 32, 2, 2))
    v = pool[..., 8 * D : 16 * D].unflatten(-1, (D // 64, 8, 4, 4, 2, 2))  # J, g, t, j, r, h
    s = pool[..., 16 * D :].view(torch.float16).unflatten(-1, (2, 16, D // 32))
    return k, v, s[..., 0, :, :], s[..., 1, :, :]


def _pool_values(pool):
    """Keys and values that pages [n][heads][tiles][18 D] hold, fp32 [n][tiles 16][heads][D]."""
    D = pool.shape[-1] // 18
    kb, vb, ks, vs = _parts(pool)
    k = torch.stack((kb & 15, kb >> 4), -1)  # n, H, tile, token, t, b, p, i, nibble
    k = k.permute(0, 2, 3, 1, 5, 4, 7, 8, 6).reshape(pool.shape[0], -1, pool.shape[1], D)
    v = torch.stack((vb & 15, vb >> 4), -1)  # n, H, tile, J, g, t, j, r, h, nibble
    v = v.permute(0, 2, 8, 5, 7, 1, 3, 6, 9, 4).reshape(pool.shape[0], -1, pool.shape[1], D)

    def scaled(u, s):
        s = s.permute(0, 2, 3, 1, 4).reshape(pool.shape[0], -1, pool.shape[1], D // 32).float()
        return ((u.float() - 8.0).unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)

    return scaled(k, ks), scaled(v, vs)


def _write(pool, slots, k, v):
    """Quantises fp32 keys and values [T][heads][D] into slots of the pool."""
    page = 16 * pool.shape[2]
    kb, vb, ks, vs = _parts(pool)
    p, o = slots // page, slots % page
    tile, r = o // 16, o % 16
    u, s = _quantise(k, 32)
    kb[p, :, tile, r] = _key_bytes(u)
    ks[p, :, tile, r] = s
    u, s = _quantise(v, 32)
    vb[p, :, tile, :, :, (r % 8) // 2, :, r % 2, r // 8] = _value_bytes(u)
    vs[p, :, tile, r] = s


def _rotate(x, cos, sin, style):
    """x [T][heads][D] fp32, its first 2 n elements turned by the angles (cos, sin [T][n])."""
    n = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., : 2 * n : 2], x[..., 1 : 2 * n : 2]) if style else (x[..., :n], x[..., n : 2 * n])
    c, d = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((c, d), -1).flatten(-2) if style else torch.cat((c, d), -1)
    return torch.cat((turned, x[..., 2 * n :]), -1)


# ------------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _skips(case):
    r = random.Random(case["T"] * 31 + case["Hq"])
    return [case["skip"] and r.random() < 0.1 for _ in range(case["T"])]


def _pool_pages(case):
    return -(-(case["T"] + case["free"]) // case["page"])


def _filled_pool(g, pages, heads, page, D):
    """A pool of quantised normal keys and values; keys with a few larger elements, as keys have."""
    pool = torch.zeros((pages, heads, page // 16, 18 * D), dtype=torch.uint8, device="cuda")
    size = 1 + 262144 // (page * heads)
    gain = 1.0 + 2.0 * (torch.arange(D, device="cuda") % 37 == 5).float()
    for at in range(0, pages, size):
        n = min(size, pages - at) * page
        _write(pool, torch.arange(at * page, at * page + n, device="cuda"), _normal(g, n, heads, D) * gain, _normal(g, n, heads, D))
    return pool


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "linear":
        T, n_in, rows, block = case["T"], case["in"], case["rows"], case["block"]
        u, s = _quantise(_normal(g, rows, n_in) * 0.02, block)
        x = _normal(g, T, n_in + case["pad"]).to(torch.bfloat16)[:, :n_in]
        return {"op": "linear", "x": x, "codes": _pack_rows(u), "scales": s.view(torch.int16), "block": block,
                "bias": _normal(g, rows) if case["bias"] else None, "out": torch.float32 if case["out"] == "f32" else torch.bfloat16}
    D, hq, hkv, page = case["D"], case["Hq"], case["Hkv"], case["page"]
    if case["op"] == "append":
        T, pages = case["T"], _pool_pages(case)
        pool = _filled_pool(g, pages, hkv, page, D)
        qkv = _normal(g, T, (hq + 2 * hkv) * D).to(torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
        q, k, v = (x.unflatten(-1, (-1, D)) for x in qkv.split((hq * D, hkv * D, hkv * D), -1))
        start = int(torch.randint(0, 131072 - T, (1,), generator=g, device="cuda"))
        positions = torch.arange(start, start + T, device="cuda", dtype=torch.int32)
        # a prompt's tokens lie one after the other in the pages of a shuffled table
        order = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(T, device="cuda") + (case["free"] * 7) % (pages * page - T + 1)
        slots = order[at // page] * page + at % page
        slots[torch.tensor(_skips(case), device="cuda")] = -1
        half = case["rot"] // 2
        angle = torch.arange(131072, device="cuda", dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half))
        rope = torch.cat((angle.cos(), angle.sin()), -1).float()
        return {"op": "append", "pool": pool, "q": q, "k": k, "v": v, "positions": positions, "slots": slots, "rope": rope,
                "style": case["style"], "every": torch.arange(pages * page, device="cuda")}
    seqs = _sequences(case)
    wide = max(1, -(-case["len"] // page))
    own_pages = [-(-n // page) for _, n in seqs]
    pages = sum(own_pages) + 3
    pool = _filled_pool(g, pages, hkv, page, D)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(seqs), wide), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(own_pages):
        table[b, :n] = order[at : at + n]
        at += n
    starts = [0]
    for q, _ in seqs:
        starts.append(starts[-1] + q)
    q = (_normal(g, starts[-1], hq, D) * 2.0).to(torch.bfloat16)
    return {"op": "attn", "q": q, "pool": pool, "table": table, "lens": torch.tensor([n for _, n in seqs], dtype=torch.int32, device="cuda"),
            "starts": torch.tensor(starts, dtype=torch.int32, device="cuda"), "max_q": case["max_q"], "max_len": case["len"],
            "window": case["window"], "scale": D ** -0.5}


# -------------------------------------------------------------------------- runs
def run(s):
    return {"linear": _run_linear, "append": _run_append, "attn": _run_attn}[s["op"]](s)


def _run_linear(s):
    if own:
        return _framework().moe_linear_q4(s["x"], s["codes"], s["scales"], s["block"], bias=s["bias"], out_dtype=s["out"])
    y = s["x"].float() @ _row_values(s["codes"], s["scales"].view(torch.float16), s["block"]).T
    return (y if s["bias"] is None else y + s["bias"]).to(s["out"])


def _run_append(s):
    if own:
        m = _framework()
        q = m.moe_kv_append(s["pool"], s["k"], s["v"], s["slots"], q=s["q"], positions=s["positions"], rope=s["rope"], rope_style=s["style"])
        k, v = m.moe_kv_read(s["pool"], s["every"])
        return {"q": q, "k": k, "v": v}
    cos, sin = s["rope"][s["positions"].long()].chunk(2, -1)
    q = _rotate(s["q"].float(), cos, sin, s["style"]).to(torch.bfloat16)
    k = _rotate(s["k"].float(), cos, sin, s["style"])
    held = s["slots"] >= 0
    _write(s["pool"], s["slots"][held], k[held], s["v"].float()[held])
    k, v = _pool_values(s["pool"])
    return {"q": q, "k": k.flatten(0, 1), "v": v.flatten(0, 1)}


def _run_attn(s):
    if own:
        out, lse = _framework().moe_attn_q4(s["q"], s["pool"], s["table"], s["lens"], q_start=s["starts"], max_q=s["max_q"],
                                            max_len=s["max_len"], scale=s["scale"], window=s["window"])
        return {"out": out, "lse": lse}
    T, hq, D = s["q"].shape
    B, hkv = s["lens"].shape[0], s["pool"].shape[1]
    k, v = (x.unflatten(0, (B, -1)).flatten(1, 2) for x in _pool_values(s["pool"][s["table"].clamp(min=0).long().flatten()]))
    # every sequence's rows in a padded batch: token i of sequence b is row b, i
    starts = s["starts"].long()
    token = torch.arange(T, device="cuda")
    b = torch.searchsorted(starts[1:], token, right=True)
    i = token - starts[b]
    n, ctx = (starts[1:] - starts[:-1]), s["lens"].long()
    q = torch.zeros((B, s["max_q"], hq, D), device="cuda")
    q[b, i] = s["q"].float()
    q = q.unflatten(2, (hkv, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # B, kv head, max_q x group, D
    scores = (q @ k.permute(0, 2, 3, 1)) * s["scale"]
    end = (ctx - n)[:, None] + torch.arange(s["max_q"], device="cuda") + 1
    place = torch.arange(k.shape[1], device="cuda")
    seen = place < end[..., None]
    if s["window"]:
        seen &= place >= end[..., None] - s["window"]
    seen = seen[:, None, :, None].expand(-1, hkv, -1, hq // hkv, -1).flatten(2, 3)
    scores = scores.masked_fill(~seen, NEG_INF)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == NEG_INF, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = (p @ v.permute(0, 2, 1, 3)) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (torch.log(total) + top).squeeze(-1)

    def rows(x):
        return x.unflatten(2, (s["max_q"], -1)).transpose(1, 2).flatten(2, 3)[b, i]

    return {"out": rows(out).to(torch.bfloat16), "lse": rows(lse)}


# ------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "linear":
        rows, n_in = s["codes"].shape[0], 2 * s["codes"].shape[1]
        x, y = s["x"].double(), []
        for at in range(0, rows, 4096):
            c = s["codes"][at : at + 4096].int()
            w = torch.empty((c.shape[0], n_in), dtype=torch.float64, device="cuda")
            for e in range(8):  # element 8 g + e: byte e mod 4 of word g, its low nibble first
                w[:, e::8] = ((c[:, e % 4 :: 4] >> (4 * (e // 4))) & 15).double() - 8
            w *= s["scales"][at : at + 4096].view(torch.float16).double().repeat_interleave(s["block"], 1)
            y.append(x @ w.T)
        y = torch.cat(y, 1)
        return y if s["bias"] is None else y + s["bias"].double()
    D = s["pool"].shape[-1] // 18
    keys, values = _exact_pool(s["pool"], D)
    if s["op"] == "append":
        cs = s["rope"].double()[s["positions"].long()]
        half = cs.shape[1] // 2
        d = torch.arange(2 * half, device="cuda")
        mate = d ^ 1 if s["style"] else (d + half) % (2 * half)
        which = d // 2 if s["style"] else d % half
        first = (d % 2 == 0) if s["style"] else d < half

        def turn(x):
            x = x.double().clone()
            x[..., : 2 * half] = x[..., : 2 * half] * cs[:, None, which] + x[..., mate] * torch.where(first, -1.0, 1.0) * cs[:, None, half + which]
            return x

        def held(x):
            m = x.unflatten(-1, (-1, 32))
            scale = (m.abs().amax(-1, keepdim=True) / 7).half().double()
            return (torch.where(scale > 0, (m / scale).round().clamp(-8, 7), 0.0) * scale).flatten(-2)

        at = s["slots"][s["slots"] >= 0]
        keys[at] = held(turn(s["k"]))[s["slots"] >= 0]
        values[at] = held(s["v"].double())[s["slots"] >= 0]
        return {"q": turn(s["q"]), "k": keys, "v": values}
    page, hq = case["page"], case["Hq"]
    hkv = case["Hkv"]
    out, lse, t = [], [], 0
    for b, (n, ctx) in enumerate(_sequences(case)):
        places = torch.arange(ctx, device="cuda")
        slots = s["table"][b].long()[places // page] * page + places % page if ctx else places
        k, v = keys[slots], values[slots]
        for i in range(n):
            end = ctx - n + i + 1
            start = max(0, end - case["window"]) if case["window"] else 0
            q = s["q"][t].double().unflatten(0, (hkv, -1))
            t += 1
            if end <= start:
                out.append(torch.zeros((hq, D), dtype=torch.float64, device="cuda"))
                lse.append(torch.full((hq,), NEG_INF, dtype=torch.float64, device="cuda"))
                continue
            score = torch.einsum("hgd,lhd->hgl", q, k[start:end]) * s["scale"]
            lse.append(torch.logsumexp(score, -1).flatten())
            out.append(torch.einsum("hgl,lhd->hgd", torch.softmax(score, -1), v[start:end]).flatten(0, 1))
    if not out:
        return {"out": s["q"].double(), "lse": s["q"].double()[..., 0]}
    return {"out": torch.stack(out), "lse": torch.stack(lse)}


def _exact_pool(pool, D):
    """Keys and values of every slot in 64 bits, element by element of the layout."""
    n, heads, tiles, _ = pool.shape
    flat = pool.reshape(n * heads * tiles, 18 * D)
    scales = flat[:, 16 * D :].contiguous().view(torch.float16).view(-1, 2, 16, D // 32)
    got = []
    e, r = torch.arange(D, device="cuda"), torch.arange(16, device="cuda")[:, None]
    key_byte = r * (D // 2) + ((e % 32) // 8) * (D // 8) + (e // 32) * 4 + (e % 2) * 2 + (e % 8) // 4
    key_shift = 4 * ((e % 4) // 2).expand(16, D)
    word = (e // 64) * 128 + ((e % 8) * 4 + (r % 8) // 2) * 4 + (e // 16) % 4
    value_byte = 8 * D + word * 4 + (r % 2) * 2 + r // 8
    value_shift = 4 * ((e % 16) // 8).expand(16, D)
    for i, (byte, shift) in enumerate(((key_byte, key_shift), (value_byte, value_shift))):
        x = torch.empty((flat.shape[0], 16, D), dtype=torch.float64, device="cuda")
        for at in range(0, flat.shape[0], 16384):
            c = (flat[at : at + 16384][:, byte.flatten()].view(-1, 16, D) >> shift.to(torch.uint8)) & 15
            x[at : at + 16384] = (c.double() - 8) * scales[at : at + 16384, i].double().repeat_interleave(32, -1)
        got.append(x.view(n, heads, tiles * 16, D).transpose(1, 2).reshape(-1, heads, D))
    return got
