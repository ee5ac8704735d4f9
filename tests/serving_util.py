"""Shared by the serving tests: caches with poisoned unused slots, and bounds
for attention results derived from the number formats.

Bounds. With bf16 inputs the products q k are exact in float32, so a score is
off by the float32 additions: at most d additions, each half a step, or a
whole one where the tensor core truncates, of sum |q k| / sqrt(d) -> d 2^-23
sum |q k| / sqrt(d); scaling to log2 units, subtracting the maximum and 2^x
(relative 2^-22) add 2^-22 (1 + |score|). A weight is then off by the relative
factor E1 = 2 (score error) + 2^-21 (numerator and denominator); in bf16 it is
also rounded, 2^-8. n additions in float32 add n 2^-23. So with A = sum p |v|
    |o - o_ref| <= (E + [bf16] 2^-8) A + half a step of the output,
and lse is off by the score error + n 2^-23 + a step of its own."""
import numpy as np
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from megatron_transformer_layer_fwd_gb300.inputs import round_to_bf16

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
MGB = {"bf16": mgb.MGB_BF16, "f32": mgb.MGB_F32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def values(rng, shape, dtype, scale=1.0):
    """float64 values exact in dtype."""
    x = rng.standard_normal(shape) * scale
    return round_to_bf16(x) if dtype == "bf16" else x.astype(np.float32).astype(np.float64)


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to("cuda", TORCH[dtype])


def host(t):
    return t.detach().double().cpu().numpy()


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Cache:
    """Pools whose slots beyond the sequences' lengths hold NaN, pages dealt
    out in random order, table entries that must not be read out of range."""

    def __init__(self, rng, lens, page, nkv, d, dtype, head_major=False, fill=True, extra=2,
                 unused_entry=-7):
        need = [(n + page - 1) // page for n in lens]
        self.n_pages, width = sum(need) + extra, max([1] + need)
        order = rng.permutation(self.n_pages)
        self.table = np.full((len(lens), width), unused_entry, dtype=np.int64)
        self.k = np.full((self.n_pages, page, nkv, d), np.nan)
        self.v = self.k.copy()
        at = 0
        for s, (n, m) in enumerate(zip(lens, need)):
            self.table[s, :m] = order[at:at + m]
            at += m
            if fill and n:
                p = np.arange(n)
                for x in (self.k, self.v):
                    x[self.table[s][p // page], p % page] = values(rng, (n, nkv, d), dtype)
        self.head_major = head_major
        self.tk, self.tv = (self._store(x, dtype) for x in (self.k, self.v))
        self.ttable = ints(self.table)
        self.desc = mgb.kv_cache(self.tk, self.tv, self.ttable)

    def _store(self, x, dtype):
        if self.head_major:
            return dev(np.swapaxes(x, 1, 2), dtype).transpose(1, 2)
        return dev(x, dtype)


def check_attention(o, lse, ref_o, ref_lse, weight_sum, qk_sum, n_keys, d, dtype):
    """o, ref_o [..., d]; lse, ref_lse [...]; weight_sum [..., d] = sum p |v|;
    qk_sum [...] = max over keys of sum |q k| / sqrt(d); n_keys [...]."""
    score = d * 2.0 ** -23 * qk_sum + 2.0 ** -22 * (1 + qk_sum)
    e = 2 * score + 2.0 ** -21 + n_keys * 2.0 ** -23
    tol = (e + (2.0 ** -8 if dtype == "bf16" else 0.0))[..., None] * weight_sum
    tol = tol + HALF_STEP[dtype] * (np.abs(ref_o) + tol) + 1e-30
    assert np.isfinite(o).all()
    bad = np.abs(o - ref_o) > tol
    assert not bad.any(), (np.abs(o - ref_o)[bad].max(), tol[bad].min(), int(bad.sum()))
    if lse is not None:
        dead = np.isneginf(ref_lse)
        assert np.isneginf(lse[dead]).all()
        with np.errstate(invalid="ignore"):
            err = np.abs(lse - ref_lse)[~dead]
        bound = (score + n_keys * 2.0 ** -23 + 2.0 ** -22 * (1 + np.abs(np.where(dead, 0, ref_lse))))[~dead]
        assert (err <= bound).all(), (err.max(), bound.min())
