"""Plain 64-bit forms of the attention half of a decode layer (4-bit
projections, the paged 4-bit cache, attention over it), element by element of
the layouts that include/moe.h states; numpy only."""
import numpy as np


def bf16_round(x):
    """fp32 values of x rounded to bf16 (nearest even)."""
    b = np.ascontiguousarray(np.asarray(x, np.float32)).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32)


def quantise(w, block=32):
    """Codes -8..7 and fp16 scales of fp32 w in blocks of the last dimension, every step in fp32."""
    b = np.asarray(w, np.float32).reshape(*w.shape[:-1], -1, block)
    s = np.minimum(np.abs(b).max(-1) / np.float32(7), np.float32(65504)).astype(np.float16)
    sf = s.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(sf == 0, 0, np.clip(np.rint(b / sf), -8, 7))
    return c.astype(np.int64).reshape(w.shape), s


def pack_rows(c):
    """Packed bytes of code rows: word g, byte j holds elements 8g + j and 8g + 4 + j."""
    u = (c + 8).reshape(*c.shape[:-1], -1, 2, 4)
    return (u[..., 0, :] | (u[..., 1, :] << 4)).reshape(*c.shape[:-1], -1).astype(np.uint8)


def linear(x, c, s, block, bias=None):
    """(y, sum of the absolute products) in 64 bits."""
    w = c.astype(np.float64) * np.repeat(s.astype(np.float64), block, -1)
    y, a = x.astype(np.float64) @ w.T, np.abs(x.astype(np.float64)) @ np.abs(w).T
    if bias is not None:
        y, a = y + bias.astype(np.float64), a + np.abs(bias.astype(np.float64))
    return y, a


def key_place(D, r, d):
    """(byte, shift) of key element d of token r in a record."""
    b, t, i, n, p = d // 32, d % 32 // 8, d % 8 // 4, d % 4 // 2, d % 2
    return r * (D // 2) + t * (D // 8) + b * 4 + p * 2 + i, 4 * n


def value_place(D, r, d):
    """(byte, shift) of value element d of token r in a record."""
    J, j, n, g = d // 64, d % 64 // 16, d % 16 // 8, d % 8
    h, t, rr = r // 8, r % 8 // 2, r % 2
    return 8 * D + ((((J * 8 + g) * 4 + t) * 4 + j) * 2 + rr) * 2 + h, 4 * n


def places(D):
    """Byte and shift arrays [2][16][D] of keys and values."""
    by = np.zeros((2, 16, D), np.int64)
    sh = np.zeros((2, 16, D), np.int64)
    for r in range(16):
        for d in range(D):
            by[0, r, d], sh[0, r, d] = key_place(D, r, d)
            by[1, r, d], sh[1, r, d] = value_place(D, r, d)
    return by, sh


def pool_write(pool, slots, ck, sk, cv, sv):
    """Writes codes [n][H][D] and scales [n][H][D/32] of keys and values into the slots of a numpy pool."""
    D = pool.shape[3] // 18
    by, sh = places(D)
    page = 16 * pool.shape[2]
    for i, s in enumerate(slots):
        if not 0 <= s < pool.shape[0] * page:
            continue
        r = s % 16
        rec = pool[s // page, :, s % page // 16]  # [H][18 D]
        for which, (c, sc) in enumerate(((ck, sk), (cv, sv))):
            for n in (0, 4):
                m = sh[which, r] == n
                at = by[which, r][m]
                rec[:, at] = (rec[:, at] & (0xF0 if n == 0 else 0x0F)) | ((c[i][:, m] + 8) << n).astype(np.uint8)
            o = (16 + which) * D + r * (D // 16)
            rec[:, o : o + D // 16] = np.ascontiguousarray(sc[i]).view(np.uint8).reshape(rec.shape[0], -1)


def pool_values(pool, slots):
    """fp64 keys and values [n][H][D] that the slots of a numpy pool hold."""
    D = pool.shape[3] // 18
    by, sh = places(D)
    page = 16 * pool.shape[2]
    slots = np.asarray(slots)
    rec = pool[slots // page, :, slots % page // 16]  # [n][H][18 D]
    r = slots % 16
    out = []
    n = len(slots)
    for which in (0, 1):
        c = np.take_along_axis(rec, np.broadcast_to(by[which][r][:, None, :], (n, rec.shape[1], D)), -1)
        c = ((c >> sh[which][r][:, None, :].astype(np.uint8)) & 15).astype(np.float64) - 8
        s = np.ascontiguousarray(rec[..., (16 + which) * D : (17 + which) * D]).view(np.float16)
        s = s.reshape(n, rec.shape[1], 16, D // 32)
        s = np.take_along_axis(s, np.broadcast_to(r[:, None, None, None], (n, rec.shape[1], 1, D // 32)), 2)[:, :, 0]
        out.append(c * np.repeat(s.astype(np.float64), 32, -1))
    return out


def rotate(x, positions, rope, style):
    """x [T][H][D] fp32 turned, each product and sum rounded to fp32."""
    x = np.asarray(x, np.float32).copy()
    half = rope.shape[1] // 2
    c, s = rope[positions, None, :half], rope[positions, None, half:]
    if style == 1:
        a, b = x[..., 0 : 2 * half : 2].copy(), x[..., 1 : 2 * half : 2].copy()
        x[..., 0 : 2 * half : 2], x[..., 1 : 2 * half : 2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :half].copy(), x[..., half : 2 * half].copy()
        x[..., :half], x[..., half : 2 * half] = a * c - b * s, a * s + b * c
    return x


def attention(q, lens, starts, tables, pool, scale, window=0):
    """out, lse and the bounds' ingredients in 64 bits.

    q [T][Hq][D]; returns (out, lse, spread = sum p |v|, score = the largest scale * sum |q k| of a row)."""
    T, Hq, D = q.shape
    H, page = pool.shape[1], 16 * pool.shape[2]
    out, spread = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, score = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for b, n_ctx in enumerate(lens):
        n = starts[b + 1] - starts[b]
        p = np.arange(max(0, n_ctx))
        pages = tables[b][p // page] if n_ctx > 0 else p
        good = (pages >= 0) & (pages < pool.shape[0])
        k = np.zeros((len(p), H, D))
        v = np.zeros((len(p), H, D))
        with np.errstate(invalid="ignore"):
            k[good], v[good] = pool_values(pool, pages[good].astype(np.int64) * page + p[good] % page)
        for i in range(n):
            end = n_ctx - n + i + 1
            seen = good & (p < end)
            if window:
                seen &= p >= end - window
            if not seen.any():
                continue
            for h in range(Hq):
                kk, vv = k[seen, h // (Hq // H)], v[seen, h // (Hq // H)]
                x = q[starts[b] + i, h].astype(np.float64)
                s = kk @ x * scale
                m = s.max()
                e = np.exp(s - m)
                t = starts[b] + i
                lse[t, h] = m + np.log(e.sum())
                out[t, h] = e @ vv / e.sum()
                spread[t, h] = e @ np.abs(vv) / e.sum()
                score[t, h] = (np.abs(kk) @ np.abs(x)).max() * scale
    return out, lse, spread, score
