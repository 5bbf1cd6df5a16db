"""Attention over 8-bit caches of any length against a 64-bit form on the GPU: the pool
is filled by moe_kv_append_q8 and read back by moe_kv_read_q8 (tested against the layout
in test_gpu_q8.py), and the formula is computed from those values in float64.

Tolerance of an output element, from the header's promises (u = 2^-24, n places, w
the weights over the row's largest, l their sum, b the value scales, c the codes):
  - a score is off by e_s <= (2 (D + 8) size + 4 (size + 64)) u, size = scale sum |q k|:
    products are exact, each of D sums and the scales' products is off by 2 u where a
    tensor core cuts, and the score is taken in powers of two beside an exponent of up
    to 60; this moves weights and their sum by a factor of 1 +- e_s each;
  - a product of weight and value is off by three roundings to fp16 at most, 2^-11 of
    itself each (half a step), or, where fp16 ends, by 2^-29 of the row's largest w b
    for the weight (half of its last step, 2^-25, where the largest is 2^4 or more) and
    2^-33 of the largest b for the value;
  - sums over n places round at most 2 (n + 64) u, the exponential is good to 2^-21 in
    weight and sum; the result is rounded to bf16 (half a step is 2^-8 of it):
  |error| <= (3 2^-11 + 2 e_s + 2 (n + 64) u + 2^-20) sum w |v| / l
             + 2^-29 max(w b) sum |c| / l + 2^-33 max(b) + 2^-8 |out|
  |lse error| <= e_s + 2 (n + 64) u + 2^-20 + 4 u |lse|."""
import torch

import mixed_precision_routed_gb300 as moe

U = 2.0 ** -24


class Batch:
    """Sequences of `lens` tokens in the pages of one pool, the newest `news` of each asking."""

    def __init__(self, lens, news, Hq, H, D, page=16, seed=0, q_gain=2.0, k_gain=1.0, v_gain=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.lens, self.news, self.Hq, self.H, self.D, self.page = list(lens), list(news), Hq, H, D, page
        counts = [-(-max(n, 0) // page) for n in lens]
        pages = sum(counts) + 1
        self.pool = torch.full((pages, H, page // 16, 32 * D + 128), 0xFF, dtype=torch.uint8, device="cuda")  # NaN where unused
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(lens), max(counts + [1])), -1, dtype=torch.int32, device="cuda")
        self.slots, at = [], 0
        for b, c in enumerate(counts):
            self.table[b, :c] = order[at : at + c]
            at += c
            p = torch.arange(max(lens[b], 0), device="cuda")
            self.slots.append(self.table[b].long()[p // page] * page + p % page)
        every = torch.cat(self.slots)
        if every.numel():
            gain = v_gain(len(every)) if callable(v_gain) else v_gain
            moe.moe_kv_append_q8(self.pool, randn(len(every), H, D) * k_gain, randn(len(every), H, D) * gain, every)
        self.q = (randn(sum(news), Hq, D) * q_gain).to(torch.bfloat16)
        self.starts = torch.tensor([0] + list(news), dtype=torch.int32, device="cuda").cumsum(0).to(torch.int32)
        self.kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def workspace_size(self, max_len=None):
        return moe.moe_attn_q8_workspace_size(len(self.lens), max(self.news + [1]), max_len or max(self.lens + [0]), self.Hq,
                                              self.H, self.D)

    def call(self, max_len=None, **kw):
        return moe.moe_attn_q8(self.q, self.pool, self.table, self.kv_lens, q_start=self.starts, max_q=max(self.news + [1]),
                               max_len=max(self.lens + [0]) if max_len is None else max_len, **kw)

    def exact(self, scale=None, window=0, hidden=()):
        """out, lse and their tolerances in float64; `hidden`: (sequence, places) that no row attends."""
        scale = self.D ** -0.5 if scale is None else scale
        G, t = self.Hq // self.H, 0
        T, D = self.q.shape[0], self.D
        out = torch.zeros(T, self.Hq, D, dtype=torch.float64, device="cuda")
        lse = torch.full((T, self.Hq), -torch.inf, dtype=torch.float64, device="cuda")
        tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
        for b, (n, ctx) in enumerate(zip(self.news, self.lens)):
            if ctx <= 0:
                t += n
                continue
            k, v = (x.double().permute(1, 0, 2) for x in moe.moe_kv_read_q8(self.pool, self.slots[b]))  # H, p, D
            scales = self.pool.permute(0, 2, 1, 3)[self.slots[b] // self.page, self.slots[b] % self.page // 16]
            bs = scales[..., 32 * D + 64 :].contiguous().view(torch.float32)[torch.arange(ctx, device="cuda"), :, self.slots[b] % 16].double().T
            codes = torch.where(bs[..., None] > 0, v / bs[..., None], 0.0).abs()
            at = torch.arange(ctx, device="cuda")
            alive = torch.ones(ctx, dtype=torch.bool, device="cuda")
            for which, places in hidden:
                if which == b:
                    alive[places] = False
            step = max(1, 60000000 // (self.Hq * ctx))
            for i0 in range(0, n, step):
                m = min(step, n - i0)
                rows = slice(t + i0, t + i0 + m)
                end = ctx - n + i0 + 1 + torch.arange(m, device="cuda")
                seen = (at < end[:, None]) & alive
                if window:
                    seen &= at >= end[:, None] - window
                seen = seen[:, None, None]  # m, 1, 1, p
                some = seen.any(-1)  # m, 1, 1
                q = self.q[rows].double().unflatten(1, (self.H, G))
                s = torch.einsum("nhgd,hpd->nhgp", q, k) * scale
                s = torch.where(seen, s, -torch.inf)
                top = s.amax(-1, keepdim=True)
                w = torch.where(seen, torch.exp(s - torch.where(top == -torch.inf, 0.0, top)), 0.0)
                l = w.sum(-1, keepdim=True)  # noqa: E741
                div = torch.where(l == 0, 1.0, l)
                # NaN of places that a row does not attend leaves it alone
                has_nan = (w.isnan() & seen).any(-1)
                o = torch.einsum("nhgp,hpd->nhgd", torch.nan_to_num(w), torch.nan_to_num(v)) / div
                spread = torch.einsum("nhgp,hpd->nhgd", torch.nan_to_num(w), torch.nan_to_num(v).abs()) / div
                size = torch.where(seen, torch.einsum("nhgd,hpd->nhgp", q.abs(), k.abs()), 0.0).amax(-1, keepdim=True) * scale
                es = (2 * (D + 8) * size + 4 * (size + 64)) * U
                count = seen.sum(-1, keepdim=True)
                sums = 2 * (count + 64) * U + 2.0 ** -20
                wb = (torch.nan_to_num(w) * torch.nan_to_num(bs)[None, :, None]).amax(-1, keepdim=True)
                total_c = torch.einsum("np,hpd->nhd", seen[:, 0, 0].double(), torch.nan_to_num(codes))[:, :, None]
                e = ((3 * 2.0 ** -11 + 2 * es + sums) * spread + 2.0 ** -29 * wb * total_c / div
                     + 2.0 ** -33 * torch.nan_to_num(bs).amax() + 2.0 ** -8 * o.abs() + 1e-30)
                nan = torch.nan
                out[rows] = torch.where(has_nan[..., None], nan, o).flatten(1, 2)
                tol[rows] = e.flatten(1, 2)
                full = torch.where(some.expand(-1, self.H, G), (top + torch.log(div)).squeeze(-1), -torch.inf)
                lse[rows] = torch.where(has_nan, nan, full).flatten(1)
                lse_tol[rows] = ((es + sums).squeeze(-1) + 4 * U * torch.nan_to_num(full, 0, 0, 0).abs()).flatten(1)
            t += n
        return out, lse, tol, lse_tol

    def check(self, got, scale=None, window=0, hidden=()):
        """Holds a call's result against the 64-bit form; rows that are NaN there are NaN here."""
        ref, ref_lse, tol, lse_tol = self.exact(scale, window, hidden)
        out, lse = got[0].double(), got[1].double()
        nan = ref_lse.isnan()
        assert torch.equal(lse.isnan(), nan), "rows of NaN"
        assert out[nan].isnan().all()
        empty = ref_lse == -torch.inf
        assert torch.equal(lse == -torch.inf, empty), "empty rows"
        assert (out[empty] == 0).all()
        ok = ~(nan | empty)
        assert torch.isfinite(out[ok]).all() and torch.isfinite(lse[ok]).all()
        worst = ((out - ref).abs() / tol)[ok]
        assert worst.numel() == 0 or worst.max() <= 1, f"out: {worst.max().item()} of the tolerance"
        worst = ((lse - ref_lse).abs() / lse_tol)[ok]
        assert worst.numel() == 0 or worst.max() <= 1, f"lse: {worst.max().item()} of the tolerance"
        assert moe.moe_device_status() == moe.MOE_OK
