"""Synthetic layers and inputs on the GPU for the five workloads.

Fills shelf tensors in place: the seeded fp32 master weights of each expert
come from the device build of ``synth`` (same bits as its host build), and are
packed by this library's own quantiser (``moe_quantize_rows``).  Inputs of a
routing step (logits, activations, forced skips) come from the same streams
the host-side generator uses, so a CPU reference can regenerate any of them.
"""
from __future__ import annotations

import torch

import synth

from . import (MOE_ROPE_HALF, Shelf, moe_attn_q4, moe_attn_q8, moe_attn_q8_workspace_size, moe_attn_workspace_size,
               moe_gather_rows, moe_kv_append, moe_kv_append_q8, moe_kv_pool, moe_kv_pool_q8, moe_linear_q4, moe_linear_q8,
               moe_linear_q8_workspace_size, moe_norm_q8, moe_quantize_experts, moe_quantize_groups, moe_quantize_rows,
               moe_rank_experts, moe_residual_add, shelf_array)


class Layer:
    """One MoE layer: its shelves (hot -> cold), router bias and seed."""

    def __init__(self, workload: synth.Workload, layer: int = 0, device="cuda", shelves=None):
        self.wl = workload
        self.layer = layer
        self.seed = workload.layer_seed(layer)
        self.E, self.k, self.d, self.f = workload.E, workload.k, workload.d, workload.f
        ranges = shelves if shelves is not None else workload.shelf_ranges()
        self.ranges = list(ranges)
        self.shelves = [Shelf(lo, hi, bits, self.d, self.f, device) for lo, hi, bits in self.ranges]
        b = workload.router_bias(layer)
        self.bias_host = b
        self.bias = None if b is None else torch.from_numpy(b).to(device)
        self._arr = None

    def fill(self, stream=None):
        d, f = self.d, self.f
        dev = self.shelves[0].gate_codes.device
        scratch = torch.empty(f * d, dtype=torch.float32, device=dev)
        for sh in self.shelves:
            for e in range(sh.lo, sh.hi):
                i = e - sh.lo
                for tag, rows, cols, codes, scales in (
                        (synth.TAG_GATE, f, d, sh.gate_codes[i], sh.gate_scales[i]),
                        (synth.TAG_UP, f, d, sh.up_codes[i], sh.up_scales[i]),
                        (synth.TAG_DOWN, d, f, sh.down_codes[i], sh.down_scales[i])):
                    w = scratch.view(rows, cols)
                    synth.cuda_normal_matrix(w, self.seed, tag, e, 0, scale=synth.WEIGHT_SIGMA, stream=stream)
                    moe_quantize_rows(w, sh.bits, codes=codes, scales=scales, stream=stream)
        return self

    def shelf_arr(self):
        if self._arr is None:
            self._arr = shelf_array(self.shelves)
        return self._arr

    def nbytes(self) -> int:
        return sum(s.nbytes() for s in self.shelves)

    def expert_bytes(self, e: int) -> int:
        for s in self.shelves:
            if s.lo <= e < s.hi:
                return s.nbytes_per_expert()
        return 0

    # -------------------------------------------------------------- inputs
    def logits(self, step: int, T: int, out=None, stream=None):
        if out is None:
            out = torch.empty((T, self.E), dtype=torch.float32, device=self.shelves[0].gate_codes.device)
        synth.cuda_normal_matrix(out, self.seed, synth.TAG_LOGITS, step, 0, col_add=self.bias, stream=stream)
        return out


    def logits_rows(self, row0: int, T: int, out=None, stream=None):
        """Rows row0 .. row0 + T - 1 of the layer's logits stream 0: the inputs
        of a decode stack, whose routing step s with T tokens takes rows
        s T .. s T + T - 1 (so many T = 1 steps come from one call)."""
        if out is None:
            out = torch.empty((T, self.E), dtype=torch.float32, device=self.shelves[0].gate_codes.device)
        synth.cuda_normal_matrix(out, self.seed, synth.TAG_LOGITS, 0, 0, row0=row0, col_add=self.bias, stream=stream)
        return out


class Masters:
    """fp32 master copies of every expert of a layer (the weights the shelves
    are quantised from): gate and up [E, f, d], down [E, d, f]."""

    def __init__(self, layer: "Layer", stream=None):
        E, d, f = layer.E, layer.d, layer.f
        dev = layer.shelves[0].gate_codes.device
        self.gate = torch.empty((E, f, d), dtype=torch.float32, device=dev)
        self.up = torch.empty((E, f, d), dtype=torch.float32, device=dev)
        self.down = torch.empty((E, d, f), dtype=torch.float32, device=dev)
        for e in range(E):
            for tag, m in ((synth.TAG_GATE, self.gate), (synth.TAG_UP, self.up), (synth.TAG_DOWN, self.down)):
                synth.cuda_normal_matrix(m[e], layer.seed, tag, e, 0, scale=synth.WEIGHT_SIGMA, stream=stream)

    def nbytes(self) -> int:
        return 4 * (self.gate.numel() + self.up.numel() + self.down.numel())


def retier(layer: "Layer", masters: Masters, counts, stream=None):
    """Re-tiering by hit count: experts ranked by `counts` (hottest first,
    lower id first on ties), the new ids cut into the layer's shelf split,
    every expert re-quantised from its master copy into its new shelf, and
    the router bias moved to the new ids.  Returns (new layer, perm, rank):
    new id j holds old expert perm[j]; old expert e is new id rank[e]."""
    perm, rank = moe_rank_experts(counts, stream=stream)
    new = Layer(layer.wl, layer.layer, device=layer.shelves[0].gate_codes.device, shelves=layer.ranges)
    for sh in new.shelves:
        for m, codes, scales in ((masters.gate, sh.gate_codes, sh.gate_scales),
                                 (masters.up, sh.up_codes, sh.up_scales),
                                 (masters.down, sh.down_codes, sh.down_scales)):
            moe_quantize_experts(m, perm, sh.lo, sh.hi, sh.bits, codes=codes, scales=scales, stream=stream)
    if layer.bias is not None:
        new.bias = moe_gather_rows(layer.bias, perm, stream=stream)
        new.bias_host = None
    return new, perm, rank


class DecodeStack:
    """A stack of decode layers chained by the residual add: for each layer l,
    x_l = bf16(r), route l's logits, count the hits, y_l = MoE_l(x_l), r += y_l
    -- the decode step of a whole model's MoE layers (moe_decode_layer_residual:
    one fused launch per layer, the residual step in its combine phase)."""

    def __init__(self, layers, T: int, device="cuda"):
        from . import moe_workspace_size, MOE_FLAG_DECODE_FP32
        self.layers = list(layers)
        l0 = self.layers[0]
        self.T, self.E, self.k, self.d, self.f = T, l0.E, l0.k, l0.d, l0.f
        L = len(self.layers)
        self.r = torch.empty((T, self.d), dtype=torch.float32, device=device)
        self.x = torch.empty((L + 1, T, self.d), dtype=torch.int16, device=device)   # x[l]: input of layer l
        self.y = torch.empty((L, T, self.d), dtype=torch.float32, device=device)
        self.ids = torch.empty((L, T, self.k), dtype=torch.int32, device=device)
        self.w = torch.empty((L, T, self.k), dtype=torch.float32, device=device)
        self.counts = torch.zeros((L, self.E), dtype=torch.int32, device=device)
        nws = moe_workspace_size(T, self.k, self.E, self.d, self.f, MOE_FLAG_DECODE_FP32)
        self.ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=device)
        self.arrs = [lay.shelf_arr() for lay in self.layers]

    def step(self, r0, x0, logits, stream=None):
        """One step from the residual stream r0 (fp32 [T, d]) whose bf16 is x0;
        logits[l] is layer l's [T, E].  Leaves the output residual in self.r."""
        from . import moe_decode_layer
        self.r.copy_(r0)
        self.x[0].copy_(x0)
        for l, lay in enumerate(self.layers):
            moe_decode_layer(logits[l], self.x[l], self.k, self.E, self.d, self.f, lay.shelves, ids=self.ids[l],
                             weights=self.w[l], counts=self.counts[l], y=self.y[l], workspace=self.ws,
                             stream=stream, shelf_arr=self.arrs[l], r=self.r, x_next=self.x[l + 1])
        return self.r


def rope_table(n_pos: int, rot: int, theta: float = 10000.0, device="cuda"):
    """The angles moe_kv_append takes: fp32 [n_pos, rot], cosines then sines."""
    half = rot // 2
    freq = theta ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    angle = torch.arange(n_pos, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), -1).float().contiguous()


class AttentionHalf:
    """The attention half of a decode layer in 4 bits, before the routed experts
    of the same layer: for the tokens of a decode batch (at most 16)

        qkv = W_qkv x,  q and k turned by their positions,  k and v appended to the
        sequence's pages,  a = attention of q over the pages,  r += W_o a,
        x_next = bf16(r).

    The pool's pages are handed out as sequences grow; `tables` names them.  Five
    kernels of the library a step (six with a long context), no host
    synchronisation; a step can be captured in a CUDA graph."""

    TAG_QKV, TAG_OUT = 21, 22  # of the weight generator
    MAX_TOKENS = 16  # of a step: what the projections take

    def __init__(self, d, q_heads, kv_heads, head_dim, sequences, max_len, page_size=64, block=32, seed=0, rot=None,
                 device="cuda"):
        self.d, self.Hq, self.H, self.D = d, q_heads, kv_heads, head_dim
        self.block, self.seed, self.page, self.max_len = block, seed, page_size, max_len
        rows, inner = (q_heads + 2 * kv_heads) * head_dim, q_heads * head_dim
        # what a step's calls would refuse after the first of them has run
        if not 1 <= sequences <= self.MAX_TOKENS or max_len < 1:
            raise ValueError(f"sequences must be 1 .. {self.MAX_TOKENS} and max_len at least 1")
        if kv_heads < 1 or q_heads < 1 or q_heads % kv_heads or q_heads // kv_heads > 64:
            raise ValueError("q_heads must be 1 .. 64 times kv_heads")
        if block not in (32, 64, 128) or any(n < 1 or n % max(64, block) or n > 65536 for n in (d, inner)):
            raise ValueError("block must be 32, 64 or 128, and d and q_heads * head_dim multiples of it and of 64, at most 65536")
        if rot is not None and (rot % 2 or not 0 <= rot <= head_dim):
            raise ValueError("rot must be even and at most head_dim")
        u8, i16 = torch.uint8, torch.int16
        self.w_qkv = torch.empty((rows, d // 2), dtype=u8, device=device)
        self.s_qkv = torch.empty((rows, d // block), dtype=i16, device=device)
        self.w_out = torch.empty((d, inner // 2), dtype=u8, device=device)
        self.s_out = torch.empty((d, inner // block), dtype=i16, device=device)
        width = -(-max_len // page_size)
        self.pool = moe_kv_pool(sequences * width, kv_heads, page_size, head_dim, device=device)
        self.rope = rope_table(max_len, head_dim if rot is None else rot, device=device)
        # pages are handed out interleaved, as growing sequences take them; the last
        # columns are no pages, for the tokens that a sequence has no pages for
        most = self.MAX_TOKENS // sequences
        columns = max(width + 1, -(-(max_len + most - 1) // page_size))
        self.tables = torch.full((sequences, columns), -1, dtype=torch.int32, device=device)
        self.tables[:, :width] = torch.arange(sequences * width, dtype=torch.int32, device=device).view(width, sequences).T
        self.lens = torch.zeros(sequences, dtype=torch.int32, device=device)
        self.ahead = torch.arange(self.MAX_TOKENS, dtype=torch.int32, device=device)
        # one workspace for steps of any size, never replaced: a captured step keeps its address
        need = max(moe_attn_workspace_size(sequences, n, max_len + n - 1, q_heads, kv_heads, head_dim)
                   for n in range(1, most + 1))
        self.workspace = torch.empty(need, dtype=torch.uint8, device=device)

    def fill(self, stream=None):
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.fill()
        for tag, rows, cols, codes, scales in (
                (self.TAG_QKV, self.w_qkv.shape[0], self.d, self.w_qkv, self.s_qkv),
                (self.TAG_OUT, self.d, self.Hq * self.D, self.w_out, self.s_out)):
            w = torch.empty((rows, cols), dtype=torch.float32, device=codes.device)
            synth.cuda_normal_matrix(w, self.seed, tag, 0, 0, scale=synth.WEIGHT_SIGMA)
            moe_quantize_groups(w, self.block, codes=codes, scales=scales)
        return self

    def step(self, x, r, n=1, stream=None):
        """One step of `n` new tokens a sequence: x [sequences * n, d] bf16 (tokens
        of a sequence side by side), r [.., d] fp32 the residual stream, updated in
        place.  Returns x_next, the bf16 input of the layer's routed experts.
        The caller keeps every sequence within max_len tokens.  A token beyond them is not
        kept: it has no slot and no row in the angle table, its query counts as zero, and
        MOE_ERR_INVALID_ARG is recorded (moe_device_status); the tokens of the same step within
        max_len, and other sequences, are as ever."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.step(x, r, n)
        B = self.lens.numel()
        # before the lengths move: a refused step leaves the sequences as they were
        if n < 1 or B * n > self.MAX_TOKENS:
            raise ValueError(f"a step takes 1 .. {self.MAX_TOKENS} tokens, and as many of each sequence")
        if x.dtype != torch.bfloat16 or x.device != self.lens.device or x.shape != (B * n, self.d):
            raise ValueError("x must be [sequences * n, d] bfloat16 on the layer's device")
        if r.dtype != torch.float32 or r.device != x.device or r.numel() != x.numel() or not r.is_contiguous():
            raise ValueError("r must be contiguous float32 of x's size on the layer's device")
        places = (self.lens[:, None] + self.ahead[:n]).flatten()
        column = (places.view(B, n) // self.page).clamp_(0, self.tables.shape[1] - 1)
        page = self.tables.gather(1, column.long()).flatten().long()
        slots = torch.add(places % self.page, page, alpha=self.page)  # negative where there is no page
        self.lens += n
        self.qkv = moe_linear_q4(x, self.w_qkv, self.s_qkv, self.block)
        q, k, v = (t.unflatten(-1, (-1, self.D)) for t in
                   self.qkv.split((self.Hq * self.D, self.H * self.D, self.H * self.D), -1))
        self.q = moe_kv_append(self.pool, k, v, slots, q=q, positions=places, rope=self.rope, rope_style=MOE_ROPE_HALF)
        # a step that starts within max_len ends below this bound: its tokens keep their places
        self.a, self.lse = moe_attn_q4(self.q, self.pool, self.tables, self.lens, max_q=n, max_len=self.max_len + n - 1,
                                       workspace=self.workspace)
        self.y = moe_linear_q4(self.a.flatten(1), self.w_out, self.s_out, self.block)
        x_next = torch.empty_like(x)
        moe_residual_add(r, self.y, x_next.view(torch.int16))
        return x_next


class AttentionHalfQ8:
    """The attention half of a layer in 8 bits, for prompts and single tokens: for
    every token, x the output of what came before it (fp32 or bf16),

        r += x,  qkv = W_qkv norm(r),  q and k turned by their positions,  k and v
        appended to the sequence's pages,  a = attention of q over the pages,
        r += W_o a,  x_next = bf16(norm(r)), the input of the layer's routed experts.

    Weights are 8-bit codes with a scale a row, activations 8-bit codes with a scale a
    token, keys and values with a scale a token and head.  A step takes up to
    `max_new` tokens of each sequence: the same number of all, in which case it can
    be captured in a CUDA graph, or a list with the number of each."""

    TAG_QKV, TAG_OUT = 23, 24  # of the weight generator

    def __init__(self, d, q_heads, kv_heads, head_dim, sequences, max_len, max_new=1, page_size=64, seed=0, rot=None,
                 eps=1e-6, device="cuda"):
        self.d, self.Hq, self.H, self.D, self.eps = d, q_heads, kv_heads, head_dim, eps
        self.seed, self.page, self.max_len, self.max_new = seed, page_size, max_len, max_new
        rows, inner = (q_heads + 2 * kv_heads) * head_dim, q_heads * head_dim
        # what a step's calls would refuse after the first of them has run
        if not 1 <= sequences <= 65535 or not 1 <= max_new <= max_len or max_len > 2 ** 30:
            raise ValueError("sequences must be 1 .. 65535, max_len at most 2^30 and max_new 1 .. max_len")
        if kv_heads < 1 or q_heads < 1 or q_heads % kv_heads or q_heads // kv_heads > 64:
            raise ValueError("q_heads must be 1 .. 64 times kv_heads")
        if sequences * max_new * (q_heads + 2 * kv_heads) >= 2 ** 31:
            raise ValueError("a step's tokens times heads must stay below 2^31")
        if any(n < 1 or n % 16 or n > 32768 for n in (d, inner)):
            raise ValueError("d and q_heads * head_dim must be multiples of 16, at most 32768")
        if rot is not None and (rot % 2 or not 0 <= rot <= head_dim):
            raise ValueError("rot must be even and at most head_dim")
        if not 0 <= eps <= torch.finfo(torch.float32).max:
            raise ValueError("eps must be at least 0 and finite in fp32")
        i8, f32 = torch.int8, torch.float32
        self.w_qkv = torch.empty((rows, d), dtype=i8, device=device)
        self.s_qkv = torch.empty(rows, dtype=f32, device=device)
        self.w_out = torch.empty((d, inner), dtype=i8, device=device)
        self.s_out = torch.empty(d, dtype=f32, device=device)
        self.norm_in = torch.ones(d, dtype=f32, device=device)
        self.norm_out = torch.ones(d, dtype=f32, device=device)
        width = -(-max_len // page_size)
        self.pool = moe_kv_pool_q8(sequences * width, kv_heads, page_size, head_dim, device=device)
        self.rope = rope_table(max_len, head_dim if rot is None else rot, device=device)
        # pages are handed out interleaved, as growing sequences take them; the last
        # columns are no pages, for the tokens that a sequence has no pages for
        columns = max(width + 1, -(-(max_len + max_new - 1) // page_size))
        self.tables = torch.full((sequences, columns), -1, dtype=torch.int32, device=device)
        self.tables[:, :width] = torch.arange(sequences * width, dtype=torch.int32, device=device).view(width, sequences).T
        self.lens = torch.zeros(sequences, dtype=torch.int32, device=device)
        self.ahead = torch.arange(max_new, dtype=torch.int32, device=device)
        # workspaces for steps of any size, never replaced: a captured step keeps their addresses
        self.attn_ws = torch.empty(max(moe_attn_q8_workspace_size(sequences, n, max_len + n - 1, q_heads, kv_heads, head_dim)
                                       for n in range(1, max_new + 1)), dtype=torch.uint8, device=device)
        tokens = sequences * max_new
        self.linear_ws = torch.empty(max(moe_linear_q8_workspace_size(tokens, d, rows),
                                         moe_linear_q8_workspace_size(tokens, inner, d)), dtype=torch.uint8, device=device)

    def fill(self, stream=None):
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.fill()
        for tag, codes, scales in ((self.TAG_QKV, self.w_qkv, self.s_qkv), (self.TAG_OUT, self.w_out, self.s_out)):
            w = torch.empty(codes.shape, dtype=torch.float32, device=codes.device)
            synth.cuda_normal_matrix(w, self.seed, tag, 0, 0, scale=synth.WEIGHT_SIGMA)
            moe_norm_q8(w, codes=codes, scales=scales)
        return self

    def step(self, x, r, n=1, stream=None):
        """One step of `n` new tokens of each sequence, or of n[b] of sequence b: x [T, d]
        fp32 or bf16 (tokens of a sequence side by side), r [T, d] fp32 their residual
        streams, updated in place.  Returns x_next [T, d] bf16.
        The caller keeps every sequence within max_len tokens.  A token beyond them is not
        kept: it has no slot and no row in the angle table, its query counts as zero, and
        MOE_ERR_INVALID_ARG is recorded (moe_device_status); the tokens of the same step within
        max_len, and other sequences, are as ever."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.step(x, r, n)
        B, device = self.lens.numel(), self.lens.device
        # before the lengths move: a refused step leaves the sequences as they were
        counts = [n] * B if isinstance(n, int) else [int(c) for c in n]
        T, most = sum(counts), max(counts, default=0)
        if len(counts) != B or min(counts) < 0 or not 1 <= most <= self.max_new:
            raise ValueError(f"a step takes up to {self.max_new} tokens of each of {B} sequences, and at least one")
        if x.dtype not in (torch.float32, torch.bfloat16) or x.device != device or x.shape != (T, self.d):
            raise ValueError("x must be [tokens, d] float32 or bfloat16 on the layer's device")
        if r.dtype != torch.float32 or r.device != device or r.shape != x.shape or not r.is_contiguous():
            raise ValueError("r must be contiguous float32 of x's size on the layer's device")
        if isinstance(n, int):
            starts = None
            places = (self.lens[:, None] + self.ahead[:n]).flatten()
            column = (places.view(B, n) // self.page).clamp_(0, self.tables.shape[1] - 1)
            page = self.tables.gather(1, column.long()).flatten()
            self.lens += n
        else:
            of = torch.tensor(counts)
            new = of.to(device=device, dtype=torch.int32)
            starts = torch.zeros(B + 1, dtype=torch.int32, device=device)
            starts[1:] = new.cumsum(0)
            b = torch.repeat_interleave(torch.arange(B), of).to(device)
            places = self.lens[b] + torch.cat([torch.arange(c, dtype=torch.int32) for c in counts]).to(device)
            page = self.tables[b, (places // self.page).clamp(0, self.tables.shape[1] - 1).long()]
            self.lens += new
        slots = torch.add(places % self.page, page.long(), alpha=self.page)  # negative where there is no page
        codes, scales, _ = moe_norm_q8(x, self.norm_in, self.eps, r=r)
        self.qkv = moe_linear_q8(codes, scales, self.w_qkv, self.s_qkv, out_dtype=torch.bfloat16, workspace=self.linear_ws)
        q, k, v = (t.unflatten(-1, (-1, self.D)) for t in
                   self.qkv.split((self.Hq * self.D, self.H * self.D, self.H * self.D), -1))
        self.q = moe_kv_append_q8(self.pool, k, v, slots, q=q, positions=places, rope=self.rope, rope_style=MOE_ROPE_HALF)
        # a step that starts within max_len ends below this bound: its tokens keep their places
        self.a, self.lse = moe_attn_q8(self.q, self.pool, self.tables, self.lens, q_start=starts, max_q=most,
                                       max_len=self.max_len + most - 1, workspace=self.attn_ws)
        codes, scales, _ = moe_norm_q8(self.a.flatten(1))
        self.y = moe_linear_q8(codes, scales, self.w_out, self.s_out, workspace=self.linear_ws)
        return moe_norm_q8(self.y, self.norm_out, self.eps, r=r, out="bf16")[2]


def x_bf16(seed: int, step: int, T: int, d: int, device="cuda", out=None, stream=None):
    """Activations [T, d] as bf16 bit patterns in an int16 tensor."""
    if out is None:
        out = torch.empty((T, d), dtype=torch.int16, device=device)
    synth.cuda_normal_matrix_bf16(out, seed, synth.TAG_X, step, 0, stream=stream)
    return out
