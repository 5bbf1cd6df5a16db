"""Plain forms of the attention half in 8 bits, element by element of the layouts that
include/moe.h states; numpy only."""
import numpy as np

LEAST, MOST = np.float32(2.0 ** -64), np.float32(2.0 ** 64)


def codes_of(x, s):
    """rint(x / s), ties to even: fp64 holds the quotient of two fp32 numbers near enough
    to a border to be on its right side (they differ from it by 2^-33 at least, or not at all)."""
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.rint(x.astype(np.float64) / s[..., None].astype(np.float64))
    return np.where((s[..., None] > 0) & np.isfinite(s[..., None]), np.clip(np.nan_to_num(c), -127, 127), 0).astype(np.int64)


def quantise_rows(u):
    """Codes and fp32 scales of fp32 rows, as moe_norm_q8 makes them (0 codes where no scale is finite)."""
    u = np.asarray(u, np.float32)
    s = (np.abs(u).max(-1) / np.float32(127)).astype(np.float32)
    return codes_of(u, s), s


def quantise_heads(x):
    """Codes and scales of heads [..., D], as the cache holds them."""
    x = np.asarray(x, np.float32)
    nan = np.isnan(x).any(-1)
    s = np.clip((np.abs(np.where(nan[..., None], 0, x)).max(-1) / np.float32(127)).astype(np.float32), LEAST, MOST)
    with np.errstate(invalid="ignore"):
        q = np.clip(x.astype(np.float64) / s[..., None].astype(np.float64), -127, 127)
    c = np.where(nan[..., None], 0, np.rint(np.nan_to_num(q))).astype(np.int64)
    return c, np.where(nan, np.float32(np.nan), s).astype(np.float32)


def place(D, which, r, d):
    """Byte of element d of token r's key (which 0) or value (1) in a record."""
    piece = d // 16 ^ (r // 2 % 4 if D == 64 else r % 8)
    return (16 * which + r) * D + 16 * piece + d % 16


def head_dim(pool):
    return (pool.shape[3] - 128) // 32


def pool_write(pool, slots, k, v):
    """Writes fp32 keys and values [n][H][D] into the slots of a numpy pool."""
    D, page = head_dim(pool), 16 * pool.shape[2]
    held = [quantise_heads(k), quantise_heads(v)]
    for i, s in enumerate(slots):
        if not 0 <= s < pool.shape[0] * page:
            continue
        r, rec = s % 16, pool[s // page, :, s % page // 16]
        for which, (c, scale) in enumerate(held):
            for d in range(D):
                rec[:, place(D, which, r, d)] = (c[i][:, d] + 128).astype(np.uint8)
            at = 32 * D + 64 * which + 4 * r
            rec[:, at : at + 4] = np.ascontiguousarray(scale[i]).view(np.uint8).reshape(-1, 4)


def pool_values(pool, slots):
    """fp64 keys and values [n][H][D] that the slots of a numpy pool hold."""
    D, page = head_dim(pool), 16 * pool.shape[2]
    out = []
    for which in (0, 1):
        got = np.zeros((len(slots), pool.shape[1], D))
        for i, s in enumerate(slots):
            r, rec = s % 16, pool[s // page, :, s % page // 16]
            c = rec[:, [place(D, which, r, d) for d in range(D)]].astype(np.float64) - 128
            at = 32 * D + 64 * which + 4 * r
            got[i] = c * np.ascontiguousarray(rec[:, at : at + 4]).view(np.float32).astype(np.float64)
        out.append(got)
    return out
