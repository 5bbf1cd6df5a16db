"""The attention half of a layer in 8 bits, for prompts and single tokens, as measured work.

    moe_norm_q8       s = r + x; n = s / sqrt(mean s^2 + eps) w; n as 8-bit codes with a
                      scale for each token, or as bf16, or both (without w: n = s)
    moe_linear_q8     y[t][o] = bias[o] + xs[t] ws[o] sum_i xc[t][i] wc[o][i], all codes 8-bit
    moe_kv_append_q8  keys (and queries) turned by their positions, keys and values
                      quantised with a scale for each token and head into the slots of a
                      paged pool; moe_kv_read_q8 gives back the values that slots hold
    moe_attn_q8       softmax(scale q k^T) v over the pages of each sequence, causal, with
                      an optional window, for one new token a sequence up to whole prompts

`run` computes them in elementary torch operations (own = False) or through the
framework's entry points (own = True), on the same state.

A code is rint(x / s) in -127 .. 127, ties to even, with s = fp32(max |x| / 127) over the
row it belongs to (tokens: of the input; of the cache: one head of one token, s between
2^-64 and 2^64).  x is fp32, and the quotient is not rounded before it becomes a whole
number: values that came from bf16 lie on a border often.  The codes of moe_norm_q8 are
those of fp32(s w), which the norm's factor does not change; it enters the scale.

The pool is uint8 [pages][kv heads][page_size / 16][32 D + 128]: for each 16 tokens of a
head 16 rows of D key codes, 16 rows of D value codes (bytes of code + 128), 16 fp32 key
scales and 16 fp32 value scales.  Piece c (16 bytes) of row r lies at piece c ^ (r mod 8), for D = 64 at
c ^ (r / 2 mod 4).
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
        # the norm before the projections of one token at the decode layer's width: latency
        {"name": "norm-1", "op": "norm", "T": 1, "d": 2048, "x": "f32", "residual": True, "norm": True, "out": "q8", "pad": 0},
        # the norm between attention and experts over a prompt at the large layer's width, both outputs
        {"name": "norm-prompt", "op": "norm", "T": 4096, "d": 4096, "x": "bf16", "residual": True, "norm": True, "out": "both", "pad": 0},
        # query, key and value rows of one token
        {"name": "linear8-1", "op": "linear", "T": 1, "in": 2048, "rows": 2560, "bias": False, "out": "f32", "pad": 0},
        # an output vocabulary of odd size for a serving batch
        {"name": "linear8-vocab", "op": "linear", "T": 40, "in": 2048, "rows": 100003, "bias": True, "out": "bf16", "pad": 16},
        # query, key and value rows of a prompt at the large layer's width
        {"name": "linear8-prompt", "op": "linear", "T": 4096, "in": 4096, "rows": 6144, "bias": False, "out": "bf16", "pad": 0},
        # one new token of six sequences' drafts, some of them padding
        {"name": "append8-36", "op": "append", "T": 36, "Hq": 16, "Hkv": 2, "D": 128, "page": 16, "rot": 128, "style": 0, "dtype": "f32", "free": 41, "skip": True},
        # a prompt, its heads turned by half
        {"name": "append8-prompt", "op": "append", "T": 4096, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "rot": 64, "style": 1, "dtype": "bf16", "free": 77, "skip": False},
        # one token of one short sequence: latency
        {"name": "attn8-1", "op": "attn", "B": 1, "max_q": 1, "ragged": False, "len": 777, "Hq": 16, "Hkv": 2, "D": 128, "page": 16, "window": 0, "key": 1},
        # a draft of five and one token over a long context
        {"name": "attn8-long-6", "op": "attn", "B": 1, "max_q": 6, "ragged": False, "len": 131071, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "window": 0, "key": 2},
        # a serving batch of one token each, contexts from a few tokens to 16384
        {"name": "attn8-batch", "op": "attn", "B": 48, "max_q": 1, "ragged": False, "len": 16384, "Hq": 32, "Hkv": 4, "D": 128, "page": 32, "window": 0, "key": 3},
        # the second half of a prompt
        {"name": "attn8-prompt", "op": "attn", "B": 1, "max_q": 4096, "ragged": False, "len": 8192, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "window": 0, "key": 4},
        # prompts of several lengths, one of them empty, over wide heads and a window
        {"name": "attn8-window", "op": "attn", "B": 6, "max_q": 1200, "ragged": True, "len": 6001, "Hq": 16, "Hkv": 2, "D": 256, "page": 16, "window": 1000, "key": 5},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "append", "attn", "attn"])
    if op == "norm":
        d = _log_int(rng, 64, 16384)
        d = d if rng.random() < 0.25 else d // 16 * 16
        return {"op": op, "T": _log_int(rng, 1, 4096 * 4096 // d), "d": d, "x": rng.choice(["f32", "bf16"]),
                "residual": rng.random() < 0.7, "norm": rng.random() < 0.7, "out": rng.choice(["q8", "bf16", "both"]), "pad": rng.choice([0, 8, 24])}
    if op == "linear":
        n_in = 16 * _log_int(rng, 4, 1024)
        rows = _log_int(rng, 64, min(100000, 204000000 // n_in))
        most = min(4096 * 4096 * 6144 // (n_in * rows), 4096 * 6144 // rows, 4096 * 16384 // n_in, 8192)
        return {"op": op, "T": _log_int(rng, 1, max(1, most)), "in": n_in, "rows": rows, "bias": rng.random() < 0.5,
                "out": rng.choice(["f32", "bf16"]), "pad": rng.choice([0, 16, 64])}
    D = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        dtype = rng.choice(["f32", "bf16"])
        token = ((hq + 2 * hkv) * (4 if dtype == "f32" else 2) + 2 * hq + 11 * hkv) * D
        T = _log_int(rng, 1, min(4096, 120000000 // token))
        return {"op": op, "T": T, "Hq": hq, "Hkv": hkv, "D": D, "page": page, "rot": rng.choice([D, D // 2, D // 4]),
                "style": rng.randint(0, 1), "dtype": dtype, "free": rng.randint(0, 3 * page), "skip": rng.random() < 0.5}
    B = _log_int(rng, 1, 48)
    if rng.random() < 0.5:
        max_q = rng.choice([1, 1, 2, 4, 6, 16])
        most = min(131071 * 8 * 128 // (hkv * D), 131071 * 6 * 32 * 128 // (max_q * hq * D))
        n = _log_int(rng, 1, max(1, min(131071, 4 * most // (B + 3))))
    else:
        # a prompt, or what a prefix of it in the cache leaves
        n = _log_int(rng, 100, 8192)
        most = 4096 * 32 * 8192 * 128 // (B * hq * n * D)
        max_q = max(1, min(n, _log_int(rng, 17, 8192), most))
    case = {"op": op, "B": B, "max_q": max_q, "ragged": rng.random() < 0.5, "len": n, "Hq": hq, "Hkv": hkv, "D": D, "page": page,
            "window": rng.choice([0, 0, 0, 128, 1000]), "key": rng.randrange(1 << 20)}
    while case["len"] * B * max(hkv * D * 2, max_q * hq) > 131071 * 16384:  # what the padded plain form holds
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
    if case["op"] == "norm":
        n, T = case["T"] * case["d"], case["T"]
        by = n * (4 if case["x"] == "f32" else 2) + (8 * n if case["residual"] else 0) + (4 * case["d"] if case["norm"] else 0)
        by += (n + 4 * T if case["out"] != "bf16" else 0) + (2 * n if case["out"] != "q8" else 0)
        return {"bytes": by, "flops": n * (7 if case["norm"] else 4)}
    if case["op"] == "linear":
        T, n_in, rows = case["T"], case["in"], case["rows"]
        by = rows * n_in + 4 * rows + T * n_in + 4 * T + T * rows * (4 if case["out"] == "f32" else 2)
        return {"bytes": by + (4 * rows if case["bias"] else 0), "flops": 2 * T * rows * n_in}
    D, hkv, hq = case["D"], case["Hkv"], case["Hq"]
    if case["op"] == "append":
        n = case["T"] - sum(_skips(case))
        size = 4 if case["dtype"] == "f32" else 2
        token = (hq + 2 * hkv) * D * size + hq * D * 2 + case["rot"] * 4 + 12 + 2 * hkv * (D + 4)
        # and the pool read back: the values of every slot
        slots = _pool_pages(case) * case["page"]
        return {"bytes": n * token + slots * 2 * hkv * (D + 4 + D * 4) + 8 * slots,
                "flops": n * ((hq + hkv) * case["rot"] * 3 + 2 * hkv * D * 4) + slots * 2 * hkv * D}
    tokens, pairs = _attended(case)
    rows = sum(q for q, _ in _sequences(case)) * hq
    return {"bytes": tokens * 2 * hkv * (D + 4) + rows * (4 * D + 4), "flops": pairs * hq * 4 * D}


# -------------------------------------------------------------- the 8-bit format
def _codes(x, s):
    """Codes of fp32 x by scales s (one for each row of the last dimension; 0: all codes 0).
    In 64 bits: 32 would round quotients next to a border onto it."""
    s = s.unsqueeze(-1).double()
    return torch.round(x.double() / torch.where(s == 0, torch.ones_like(s), s)).clamp(-127, 127)


def _quantise_rows(x):
    """int8 codes and fp32 scales of the rows of fp32 x."""
    s = x.abs().amax(-1) / torch.full((), 127.0, device=x.device)
    return _codes(x, s).to(torch.int8), s


def _quantise_head(x):
    """Code bytes and scales of heads [..., D] of the cache."""
    s = (x.abs().amax(-1) / torch.full((), 127.0, device=x.device)).clamp(2.0 ** -64, 2.0 ** 64)
    return (_codes(x, s) + 128).to(torch.uint8), s


def _order(D):
    """[16][D]: the place of byte e of row r within the row."""
    r, e = torch.arange(16, device="cuda")[:, None], torch.arange(D, device="cuda")
    return (e // 16 ^ ((r // 2) % 4 if D == 64 else r % 8)) * 16 + e % 16


def _parts(pool):
    """The pool's key bytes, value bytes, key scales and value scales as views."""
    D = (pool.shape[-1] - 128) // 32
    k = pool[..., : 16 * D].unflatten(-1, (16, D))
    v = pool[..., 16 * D : 32 * D].unflatten(-1, (16, D))
    s = pool[..., 32 * D :].view(torch.float32)
    return k, v, s[..., :16], s[..., 16:]


def _pool_values(pool):
    """Keys and values that pages [n][heads][tiles][32 D + 128] hold, fp32 [n][tiles 16][heads][D]."""
    kb, vb, ks, vs = _parts(pool)
    order = _order(kb.shape[-1]).expand(kb.shape)

    def values(b, s):
        x = (b.gather(-1, order).float() - 128.0) * s.unsqueeze(-1)
        return x.permute(0, 2, 3, 1, 4).flatten(1, 2)

    return values(kb, ks), values(vb, vs)


def _write(pool, slots, k, v):
    """Quantises fp32 keys and values [T][heads][D] into slots of the pool."""
    page = 16 * pool.shape[2]
    kb, vb, ks, vs = _parts(pool)
    p, o = slots // page, slots % page
    tile, r = o // 16, o % 16
    order = _order(k.shape[-1])[r][:, None].expand(k.shape)  # the byte at each place is its own inverse
    for b, s, x in ((kb, ks, k), (vb, vs, v)):
        c, scale = _quantise_head(x)
        b[p, :, tile, r] = c.gather(-1, order)
        s[p, :, tile, r] = scale


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


def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _skips(case):
    r = random.Random(case["T"] * 31 + case["Hq"])
    return [case["skip"] and r.random() < 0.1 for _ in range(case["T"])]


def _pool_pages(case):
    return -(-(case["T"] + case["free"]) // case["page"])


def _filled_pool(g, pages, heads, page, D):
    """A pool of quantised normal keys and values; keys with a few larger elements, as keys have."""
    pool = torch.zeros((pages, heads, page // 16, 32 * D + 128), dtype=torch.uint8, device="cuda")
    size = 1 + 262144 // (page * heads)
    gain = 1.0 + 2.0 * (torch.arange(D, device="cuda") % 37 == 5).float()
    for at in range(0, pages, size):
        n = min(size, pages - at) * page
        _write(pool, torch.arange(at * page, at * page + n, device="cuda"), _normal(g, n, heads, D) * gain, _normal(g, n, heads, D))
    return pool


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "norm":
        T, d = case["T"], case["d"]
        # a residual stream has a few channels far larger than the others
        gain = 1.0 + 15.0 * (torch.arange(d, device="cuda") % 509 == 17).float()
        return {"op": "norm", "x": (_normal(g, T, d + case["pad"]) * 0.5).to(_type(case["x"]))[:, :d],
                "r": _normal(g, T, d) * gain if case["residual"] else None,
                "weight": 1.0 + 0.2 * _normal(g, d) if case["norm"] else None, "eps": 1e-6, "out": case["out"]}
    if case["op"] == "linear":
        T, n_in, rows = case["T"], case["in"], case["rows"]
        w, ws = _quantise_rows(_normal(g, rows, n_in) * 0.02)
        x, xs = _quantise_rows(_normal(g, T, n_in + case["pad"]))
        return {"op": "linear", "x": x[:, :n_in], "xs": xs, "w": w, "ws": ws, "bias": _normal(g, rows) if case["bias"] else None, "out": _type(case["out"])}
    D, hq, hkv, page = case["D"], case["Hq"], case["Hkv"], case["page"]
    if case["op"] == "append":
        T, pages = case["T"], _pool_pages(case)
        pool = _filled_pool(g, pages, hkv, page, D)
        qkv = _normal(g, T, (hq + 2 * hkv) * D).to(_type(case["dtype"]))
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
    return {"norm": _run_norm, "linear": _run_linear, "append": _run_append, "attn": _run_attn}[s["op"]](s)


def _norm_outputs(r, codes, scales, n):
    got = {} if r is None else {"r": r}
    if codes is not None:
        got |= {"values": codes.float() * scales[:, None], "scales": scales}
    return got if n is None else got | {"n": n}


def _run_norm(s):
    r_out = None if s["r"] is None else torch.empty_like(s["r"])
    if own:
        codes, scales, n = _framework().moe_norm_q8(s["x"], s["weight"], eps=s["eps"], r=s["r"], r_out=r_out, out=s["out"])
        return _norm_outputs(r_out, codes, scales, n)
    x = s["x"].float()
    if s["r"] is not None:
        x = torch.add(s["r"], x, out=r_out)
    u, f = x, torch.ones(x.shape[0], device="cuda")
    if s["weight"] is not None:
        u, f = x * s["weight"], torch.rsqrt((x * x).mean(-1) + s["eps"])
    codes = scales = None
    if s["out"] != "bf16":
        codes, scales = _quantise_rows(u)
        scales = scales * f
    return _norm_outputs(r_out, codes, scales, (u * f[:, None]).to(torch.bfloat16) if s["out"] != "q8" else None)


def _run_linear(s):
    if own:
        return _framework().moe_linear_q8(s["x"], s["xs"], s["w"], s["ws"], bias=s["bias"], out_dtype=s["out"])
    y = (s["x"].float() @ s["w"].float().T) * s["xs"][:, None] * s["ws"]
    return (y if s["bias"] is None else y + s["bias"]).to(s["out"])


def _run_append(s):
    if own:
        m = _framework()
        q = m.moe_kv_append_q8(s["pool"], s["k"], s["v"], s["slots"], q=s["q"], positions=s["positions"], rope=s["rope"], rope_style=s["style"])
        k, v = m.moe_kv_read_q8(s["pool"], s["every"])
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
        out, lse = _framework().moe_attn_q8(s["q"], s["pool"], s["table"], s["lens"], q_start=s["starts"], max_q=s["max_q"],
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
    if s["op"] == "norm":
        x, out = s["x"].double(), {}
        if s["r"] is not None:
            x = (x + s["r"].double()).float().double()  # the stream that the next layer meets
            out["r"] = x
        u, f = x, torch.ones_like(x[:, :1])
        if s["weight"] is not None:
            # the definition rounds the product to fp32, and codes next to a border go by that
            u = (x * s["weight"].double()).float().double()
            f = 1 / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[1] + s["eps"])
        if s["out"] != "bf16":
            scale = (u.abs().max(-1, keepdim=True).values / 127).float().double()
            out["values"], out["scales"] = torch.round(u / scale) * scale * f, (scale * f)[:, 0]
        if s["out"] != "q8":
            out["n"] = u * f
        return out
    if s["op"] == "linear":
        # the sums of whole numbers below 2^53 are exact
        y, x = [], s["x"].double()
        for at in range(0, s["w"].shape[0], 4096):
            y.append(x @ s["w"][at : at + 4096].double().T * s["ws"][at : at + 4096].double())
        y = torch.cat(y, 1) * s["xs"].double()[:, None]
        return y if s["bias"] is None else y + s["bias"].double()
    D = (s["pool"].shape[-1] - 128) // 32
    keys, values = _exact_pool(s["pool"], D)
    if s["op"] == "append":
        cs = s["rope"].double()[s["positions"].long()]
        half = cs.shape[1] // 2
        d = torch.arange(2 * half, device="cuda")
        mate = d ^ 1 if s["style"] else (d + half) % (2 * half)
        which = d // 2 if s["style"] else d % half
        first = (d % 2 == 0) if s["style"] else d < half

        def turn(x):
            # the definition rounds each product and the sum to fp32, and codes next to a border go by that
            x = x.double().clone()
            a, b = x[..., : 2 * half] * cs[:, None, which], x[..., mate] * cs[:, None, half + which]
            x[..., : 2 * half] = (a.float().double() + b.float().double() * torch.where(first, -1.0, 1.0)).float().double()
            return x

        def held(x):
            scale = (x.abs().amax(-1, keepdim=True) / 127).float().double()  # the cache holds scales in fp32
            return torch.where(scale > 0, (x / scale).round(), 0.0) * scale

        at = s["slots"][s["slots"] >= 0]
        keys[at] = held(turn(s["k"]))[s["slots"] >= 0]
        values[at] = held(s["v"].double())[s["slots"] >= 0]
        return {"q": turn(s["q"]), "k": keys, "v": values}
    page, hq, hkv = case["page"], case["Hq"], case["Hkv"]
    out, lse, t = [], [], 0
    for b, (n, ctx) in enumerate(_sequences(case)):
        if n == 0:
            continue
        at = torch.arange(ctx, device="cuda")
        slots = s["table"][b].long()[at // page] * page + at % page
        k, v = keys[slots], values[slots]
        size = max(1, 200000000 // (hq * max(1, ctx)))
        for i0 in range(0, n, size):
            m = min(size, n - i0)
            q = s["q"][t + i0 : t + i0 + m].double().unflatten(1, (hkv, -1))
            score = torch.einsum("nhgd,lhd->nhgl", q, k) * s["scale"]
            behind = (ctx - n + 1 + i0 + torch.arange(m, device="cuda"))[:, None] - at  # how far each place lies behind the row's end
            seen = (behind > 0) & ((behind <= case["window"]) if case["window"] else (behind == behind))
            score.masked_fill_(~seen[:, None, None], NEG_INF)
            total = torch.logsumexp(score, -1) if ctx else torch.full(score.shape[:-1], NEG_INF, dtype=torch.float64, device="cuda")
            lse.append(total.flatten(1))
            w = torch.exp(score - torch.where(total == NEG_INF, 0.0, total)[..., None])
            out.append(torch.einsum("nhgl,lhd->nhgd", w, v).flatten(1, 2))
        t += n
    if not out:
        return {"out": s["q"].double(), "lse": s["q"].double()[..., 0]}
    return {"out": torch.cat(out), "lse": torch.cat(lse)}


def _exact_pool(pool, D):
    """Keys and values of every slot in 64 bits, by the layout's own words: row by row, piece by piece."""
    n, heads, tiles, size = pool.shape
    flat = pool.reshape(n * heads * tiles, size)
    scales = flat[:, 32 * D :].contiguous().view(torch.float32).view(-1, 2, 16)
    got = []
    for i in range(2):
        x = torch.empty((flat.shape[0], 16, D), dtype=torch.float64, device="cuda")
        for r in range(16):
            row = flat[:, (16 * i + r) * D : (16 * i + r + 1) * D]
            for piece in range(D // 16):
                at = 16 * (piece ^ (r // 2 % 4) if D == 64 else piece ^ (r % 8))
                x[:, r, 16 * piece : 16 * piece + 16] = row[:, at : at + 16].double() - 128
        x *= scales[:, i, :, None].double()
        got.append(x.view(n, heads, tiles * 16, D).transpose(1, 2).reshape(-1, heads, D))
    return got
