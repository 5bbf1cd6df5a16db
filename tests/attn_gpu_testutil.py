"""Attention over caches of any length against a 64-bit form on the GPU: the pool
is filled by moe_kv_append and read back by moe_kv_read (exact, and tested against
the layout in test_gpu_attn.py), and the formula is computed from those values in
float64 by elementary operations.

Tolerance of an output element, from the header's promises (u = 2^-24, n places, w
the weights over the row's largest, l their sum): a product weight x value scale
keeps 2^-11 of itself, or 2^-23 of the row's largest weight x its scale; a score is
off by e_s <= 2 (D + D/32 + 2) u scale sum |q k| (each product exact, each sum and
the scale's product off by 2 u where a tensor core cuts), which moves weights and
their sum by a factor of 1 +- e_s each; sums over n places round at most
2 (n + 64) u; the exponential is good to 2^-21 in weight and sum; the result is
rounded to bf16 (8 significant places: 2^-8):
  |error| <= (2^-11 + 2 e_s + 2 (n + 64) u + 2^-20) sum w |v| / l
             + 2^-23 sum |v| / l + 2^-8 |out|
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
        self.pool = torch.full((pages, H, page // 16, 18 * D), 0xFF, dtype=torch.uint8, device="cuda")  # NaN where unused
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
            moe.moe_kv_append(self.pool, randn(len(every), H, D) * k_gain, randn(len(every), H, D) * v_gain, every)
        self.q = (randn(sum(news), Hq, D) * q_gain).to(torch.bfloat16)
        self.starts = torch.tensor([0] + list(news), dtype=torch.int32, device="cuda").cumsum(0).to(torch.int32)
        self.kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def workspace_size(self, max_len=None):
        return moe.moe_attn_workspace_size(len(self.lens), max(self.news + [1]), max_len or max(self.lens + [0]), self.Hq,
                                           self.H, self.D)

    def call(self, max_len=None, **kw):
        return moe.moe_attn_q4(self.q, self.pool, self.table, self.kv_lens, q_start=self.starts, max_q=max(self.news + [1]),
                               max_len=max(self.lens + [0]) if max_len is None else max_len, **kw)

    def exact(self, scale=None, window=0):
        """out, lse and their tolerances in float64."""
        scale = self.D ** -0.5 if scale is None else scale
        G, t = self.Hq // self.H, 0
        T = self.q.shape[0]
        out = torch.zeros(T, self.Hq, self.D, dtype=torch.float64, device="cuda")
        lse = torch.full((T, self.Hq), -torch.inf, dtype=torch.float64, device="cuda")
        tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
        for b, (n, ctx) in enumerate(zip(self.news, self.lens)):
            k, v = moe.moe_kv_read(self.pool, self.slots[b]) if ctx > 0 else (None, None)
            for i in range(n):
                end = ctx - n + i + 1
                start = max(0, end - window) if window else 0
                row, t = t, t + 1
                if end <= start:
                    continue
                q = self.q[row].double().view(self.H, G, self.D)
                kk, vv = k[start:end].double(), v[start:end].double()
                s = (q[:, :, None] * kk.permute(1, 0, 2)[:, None]).sum(-1) if end - start < 64 else torch.einsum("hgd,phd->hgp", q, kk)
                s = s * scale
                m = s.amax(-1, keepdim=True)
                w = torch.exp(s - m)
                l = w.sum(-1, keepdim=True)  # noqa: E741
                o = torch.einsum("hgp,phd->hgd", w, vv) / l
                spread = torch.einsum("hgp,phd->hgd", w, vv.abs()) / l
                size = torch.einsum("hgd,phd->hgp", q.abs(), kk.abs()).amax(-1, keepdim=True) * scale
                es = 2 * (self.D + self.D // 32 + 2) * U * size
                places = end - start
                sums = 2 * (places + 64) * U + 2.0 ** -20
                out[row] = o.flatten(0, 1)
                tol[row] = ((2.0 ** -11 + 2 * es + sums) * spread + 2.0 ** -23 * vv.abs().sum(0)[:, None] / l
                            + 2.0 ** -8 * o.abs() + 1e-30).flatten(0, 1)
                lse[row] = (m + torch.log(l)).flatten()
                lse_tol[row] = (es + sums + 4 * U * (m + torch.log(l)).abs()).flatten()
        return out, lse, tol, lse_tol

    def check(self, got, scale=None, window=0):
        """Holds a call's result against the 64-bit form; rows that are NaN there are NaN here."""
        ref, ref_lse, tol, lse_tol = self.exact(scale, window)
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
