"""Device-memory plumbing around the C ABI for one layer and for the CE.

PyTorch allocates the buffers (inputs, weights, outputs, the saved buffer,
the workspace) and provides the stream; every computation is a call into
libmgb.so through `mgb`.
"""
from __future__ import annotations

import contextlib

import numpy as np
import torch

from . import mgb

WEIGHT_KEYS = ("w_qkv", "b_qkv", "w_o", "b_o", "w_1", "b_1", "w_2", "b_2",
               "ln1_g", "ln1_b", "ln2_g", "ln2_b")


def torch_dtype(name: str) -> torch.dtype:
    return torch.bfloat16 if name == "bf16" else torch.float32


def to_device(a: np.ndarray, dtype: torch.dtype, device="cuda") -> torch.Tensor:
    """float64 array of values exact in `dtype` -> device tensor (exact copy)."""
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(device=device, dtype=dtype)


class LayerRunner:
    """One layer's device buffers and the fwd/bwd calls."""

    def __init__(self, shape, arrays: dict, device="cuda"):
        self.shape = shape
        self.desc = mgb.block_desc(shape)
        self.dtype = torch_dtype(shape.dtype)
        self.w = {k: (to_device(arrays[k], self.dtype, device) if arrays.get(k) is not None else None)
                  for k in WEIGHT_KEYS}
        self.x = to_device(arrays["x"], self.dtype, device)
        saved, fwd, bwd = mgb.mgb_block_sizes(self.desc)
        self.saved = torch.empty(max(saved, 16), dtype=torch.uint8, device=device)
        self.ws = torch.empty(max(bwd, 16), dtype=torch.uint8, device=device)
        # float32: the forward's GEMMs keep their split operands here
        self.fwd_ws = torch.empty(fwd, dtype=torch.uint8, device=device) if fwd > 0 else None
        self.y = torch.empty_like(self.x)
        self.dx = torch.empty_like(self.x)
        self.grads = {k: (torch.empty_like(v) if v is not None else None) for k, v in self.w.items()}

    def fwd(self, stream=None):
        mgb.mgb_block_fwd(self.desc, self.w, self.x, self.y, self.saved, self.fwd_ws, stream)
        return self.y

    def bwd(self, dy: torch.Tensor, stream=None):
        mgb.mgb_block_bwd(self.desc, self.w, self.x, dy, self.saved, self.dx, self.grads, self.ws,
                          stream)
        return self.dx, self.grads


class CERunner:
    """Tied-embedding CE buffers and the fused fwd+bwd call."""

    def __init__(self, tokens: int, hidden: int, vocab: int, chunk: int, hidden_t: torch.Tensor,
                 emb_t: torch.Tensor, targets_t: torch.Tensor, grad_scale: float | None = None,
                 want_grads: bool = True, mode: int = mgb.MGB_CE_FUSED, emb_stream=None,
                 token_block: int = 0):
        dev = hidden_t.device
        self.desc = mgb.ce_desc(tokens, hidden, vocab, chunk,
                                grad_scale if grad_scale is not None else 1.0 / max(tokens, 1), mode,
                                token_block)
        # resident / blocked mode: d_emb (its last part) is left running on this
        # stream (the caller joins it)
        self.desc.emb_stream = emb_stream.cuda_stream if emb_stream is not None else None
        self.hidden, self.emb, self.targets = hidden_t, emb_t, targets_t
        # the blocked mode's rows per block as the library rounds them
        tb = token_block if token_block > 0 else mgb.CE_DEFAULT_TOKEN_BLOCK
        self.token_block = min((tb + 255) // 256 * 256, (tokens + 255) // 256 * 256)
        self.ws = torch.empty(max(mgb.mgb_vocab_ce_sizes(self.desc), 16), dtype=torch.uint8, device=dev)
        self.loss = torch.empty(max(tokens, 1), dtype=torch.float32, device=dev)
        self.lse = torch.empty(max(tokens, 1), dtype=torch.float32, device=dev)
        self.loss_mean = torch.empty(4, dtype=torch.float32, device=dev)
        self.d_hidden = torch.empty_like(hidden_t) if want_grads else None
        self.d_emb = torch.empty_like(emb_t) if want_grads else None

    def run(self, stream=None):
        mgb.mgb_vocab_ce_fwd_bwd(self.desc, self.hidden, self.emb, self.targets, self.loss,
                                 self.loss_mean, self.lse, self.d_hidden, self.d_emb, self.ws, stream)


def rope_table(positions: int, rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """The rotary table mgb_kv_append reads, [positions, rot_dim / 2, 2] float32:
    cos and sin of p * base^(-2 j / rot_dim), from float64 angles (a float32
    product p * frequency is off by up to 2^-24 p radians)."""
    j = torch.arange(rot_dim // 2, dtype=torch.float64)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * base ** (-2.0 * j / rot_dim)[None, :]
    return torch.stack((torch.cos(a), torch.sin(a)), dim=-1).to(device, torch.float32).contiguous()


DEVICE = "cuda"  # where a batch's lengths, offsets and block table lie: kernels read them


def _on(stream, device: torch.device):
    """Context with `stream` (None: the current one; a torch stream or a raw
    handle) as torch's current stream: what is allocated and filled inside is
    ordered with the kernels, and its memory goes back to that stream. The
    tensors' device becomes the current one."""
    if stream is None:
        return torch.cuda.device(device) if device.type == "cuda" else contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


class ServingBatch:
    """What all layers share in one step of running sequences: the lengths, the
    block table and the attention plan (made from the lengths as they are now: a
    step with others takes a new batch, or a replay of a captured one). Without `cu_seqlens` the step has one
    new token per sequence (decode); with it, the rows of whole prompts packed
    one behind the other (`tokens` rows, possibly more than they fill), whose
    lengths are their numbers of rows, or 0 for padding: a prompt that continues
    cached tokens is reported by mgb_device_status as MGB_ERR_INDEX and not
    cached, since its rows would attend to each other alone. A prompt's rows see
    each other as the shape's mask says; a decode step's row sees all of the
    cache, with either mask."""

    def __init__(self, shape, block_table: torch.Tensor, seq_lens: torch.Tensor,
                 cu_seqlens: torch.Tensor | None = None, tokens: int | None = None, stream=None):
        self.block_table, self.seq_lens, self.cu_seqlens = block_table, seq_lens, cu_seqlens
        n, dev = seq_lens.numel(), seq_lens.device
        for t in (seq_lens, cu_seqlens):
            if t is not None and (t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous()):
                raise ValueError("seq_lens and cu_seqlens must be contiguous int32 vectors")
        if block_table.dim() != 2 or block_table.shape[0] != n or (
                cu_seqlens is not None and (cu_seqlens.numel() != n + 1 or tokens is None)):
            raise ValueError("a batch of n sequences has n block-table rows and, packed, n + 1 row "
                             "offsets and a number of tokens")
        if dev.type != DEVICE or any(t.device != dev for t in (block_table, cu_seqlens) if t is not None):
            raise ValueError("seq_lens, cu_seqlens and the block table must be on one GPU device")
        self.tokens = n if cu_seqlens is None else tokens
        self.heads = (shape.n_q_heads, shape.n_kv_heads, shape.head_dim)
        self.causal = shape.causal
        with _on(stream, dev):
            if cu_seqlens is None:
                self.ws = torch.empty(mgb.mgb_attention_decode_ws_bytes(
                    n, shape.n_q_heads, shape.n_kv_heads, shape.head_dim), dtype=torch.uint8, device=dev)
                self.plan = mgb.mgb_attention_decode_prepare(
                    n, shape.n_q_heads, shape.n_kv_heads, shape.head_dim, seq_lens, self.ws)
            else:
                self.ws = torch.empty(mgb.mgb_attention_packed_ws_bytes(n, tokens), dtype=torch.uint8,
                                      device=dev)
                self.plan = mgb.mgb_attention_packed_prepare(n, tokens, shape.causal, cu_seqlens, self.ws)


class ServingLayer:
    """One layer for running sequences: its weights and its paged key/value
    pools ([n_pages, page_size, n_kv_heads, head_dim]; every layer has its own,
    the block table is shared). `rope`: the table of rope_table, or None."""

    def __init__(self, shape, arrays: dict, k_pool: torch.Tensor, v_pool: torch.Tensor,
                 rope: torch.Tensor | None = None, rope_interleaved: bool = False):
        self.shape, self.k_pool, self.v_pool = shape, k_pool, v_pool
        self.rope, self.rope_interleaved = rope, rope_interleaved
        self.dtype = torch_dtype(shape.dtype)
        self.mgb_dtype = mgb.MGB_BF16 if shape.dtype == "bf16" else mgb.MGB_F32
        if k_pool.dtype != self.dtype or tuple(k_pool.shape[2:]) != (shape.n_kv_heads, shape.head_dim):
            raise ValueError("the pools must be [n_pages, page_size, n_kv_heads, head_dim] of the "
                             "layer's dtype")
        if any(t is not None and t.device != k_pool.device for t in (v_pool, rope)):
            raise ValueError("the pools and rope must be on one device")
        if rope is not None and (rope.dtype != torch.float32 or rope.dim() != 3 or rope.shape[2] != 2
                                 or not rope.is_contiguous()):
            raise ValueError("rope must be [positions, rot_dim / 2, 2] float32, contiguous")
        self.w = {k: (to_device(arrays[k], self.dtype, k_pool.device) if arrays.get(k) is not None
                      else None) for k in WEIGHT_KEYS}

    def _gemm(self, epilogue, a, w, bias, c, c2=None, resid=None):
        m, k, n = a.shape[0], a.shape[1], w.shape[0]
        d = mgb.GemmExDesc(
            g=mgb.GemmDesc(m=m, n=n, k=k, a_major=mgb.MGB_K_MAJOR, b_major=mgb.MGB_K_MAJOR, lda=k, ldb=k,
                           ldc=n, dtype=self.mgb_dtype, c_f32=0, accumulate=0, alpha=1.0),
            epilogue=epilogue, glu_block=self.shape.glu_block, ldc2=c2.shape[1] if c2 is not None else 0,
            ldr=n, ldaux=0)
        mgb.mgb_gemm_ex(d, a, w, bias, c, c2=c2, resid=resid)
        return c

    def _norm(self, x, which):
        y = torch.empty_like(x)
        mgb.mgb_layernorm_fwd(x.shape[0], x.shape[1], self.mgb_dtype, self.shape.ln_eps, x,
                              self.w[f"ln{which}_g"], self.w[f"ln{which}_b"], y, None, None)
        return y

    def step(self, x: torch.Tensor, batch: ServingBatch, stream=None) -> torch.Tensor:
        """The layer's output [tokens, hidden] for the batch's new rows x, whose
        keys and values enter the cache. Rows of no sequence come out as the
        layer of a zero attention output. With `stream` the whole step, its
        temporaries included, runs on that stream, behind what the caller has
        ordered it after; the output belongs to it."""
        s = self.shape
        if tuple(x.shape) != (batch.tokens, s.hidden) or x.dtype != self.dtype or not x.is_contiguous():
            raise ValueError("x must be [batch.tokens, hidden] of the layer's dtype, contiguous")
        if any(t.device != x.device for t in (self.k_pool, batch.seq_lens)):
            raise ValueError("x, the layer's pools and the batch must be on one device")
        # (a packed plan serves any heads, a decode plan those it was cut for)
        if batch.cu_seqlens is None and batch.heads != (s.n_q_heads, s.n_kv_heads, s.head_dim):
            raise ValueError("the batch was prepared for other heads than the layer's")
        if batch.cu_seqlens is not None and bool(batch.causal) != bool(s.causal):
            raise ValueError("the batch was prepared for a causal mask, or without one, unlike the layer")
        if batch.tokens == 0:
            return torch.empty_like(x)
        with _on(stream, x.device):
            if stream is not None:  # either may belong to another stream and be freed before the step is done
                now = torch.cuda.current_stream(x.device)
                x.record_stream(now)
                batch.ws.record_stream(now)
            return self._step(x, batch)

    def _step(self, x: torch.Tensor, batch: ServingBatch) -> torch.Tensor:
        s, w, d = self.shape, self.w, self.shape.head_dim
        T, nq, nkv = x.shape[0], self.shape.n_q_heads, self.shape.n_kv_heads
        pre = s.norm_pos == "pre"
        width = (nq + 2 * nkv) * d
        new = lambda cols: torch.empty((T, cols), dtype=self.dtype, device=x.device)
        qkv = self._gemm(mgb.MGB_EPI_STORE, self._norm(x, 1) if pre else x, w["w_qkv"], w["b_qkv"], new(width))
        q, k, v = qkv, qkv[:, nq * d:], qkv[:, (nq + nkv) * d:]
        cache = mgb.kv_cache(self.k_pool, self.v_pool, batch.block_table)
        rot = 2 * self.rope.shape[1] if self.rope is not None else 0
        desc = mgb.kv_append_desc(T, batch.seq_lens.numel(), nq, rot, self.rope_interleaved,
                                  self.rope.shape[0] if rot else 0, whole=batch.cu_seqlens is not None)
        # queries and keys are rotated where they lie
        mgb.mgb_kv_append(desc, cache, batch.cu_seqlens, batch.seq_lens, self.rope, q, k, v, width, width,
                          q, width, k, width)
        o = torch.zeros((T, nq * d), dtype=self.dtype, device=x.device)
        if batch.cu_seqlens is None:
            mgb.mgb_attention_decode(batch.plan, cache, q, width, o, nq * d, None)
        else:
            mgb.mgb_attention_packed_fwd(batch.plan, nq, nkv, d, self.mgb_dtype, q, k, v, width, width, o,
                                         nq * d, None)
        h = self._gemm(mgb.MGB_EPI_BIAS_RESID, o, w["w_o"], w["b_o"], new(s.hidden), resid=x)
        if not pre:
            h = self._norm(h, 1)
        epi = mgb.MGB_EPI_BIAS_SWIGLU if s.act == "swiglu" else mgb.MGB_EPI_BIAS_GELU
        a = new(s.ffn)
        self._gemm(epi, self._norm(h, 2) if pre else h, w["w_1"], w["b_1"], new(w["w_1"].shape[0]), c2=a)
        y = self._gemm(mgb.MGB_EPI_BIAS_RESID, a, w["w_2"], w["b_2"], new(s.hidden), resid=h)
        return y if pre else self._norm(y, 2)
