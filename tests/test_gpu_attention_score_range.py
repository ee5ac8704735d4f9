"""Scores of any finite size in the serving attention kernels: weights that are
equal stay equal, and none overflows, up to scores near the types' lowest number."""
import numpy as np
import pytest
import torch

from tests.serving_util import TORCH, dev, values
from tests.test_gpu_attention_nonfinite import INF, _decode, _packed

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


def _check_mean(got, v, dtype):
    """got [.., d] = the mean of v's rows, from weights that are equal (to 2^-8 relative at
    most each in bf16): n additions in float32, and the output's half step."""
    n, v = v.shape[0], v.double()
    mean, size = v.mean(0), v.abs().mean(0)
    half = torch.finfo(TORCH[dtype]).eps / 2
    e = (n + 4) * 2.0 ** -23 + (2.0 ** -8 if dtype == "bf16" else 0.0)
    assert bool(((got.double() - mean).abs() <= size * e * (1 + half) + half * mean.abs()).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_of_the_lowest_scores(dtype, d):
    """Every score is close to the lowest finite number: equal weights."""
    rng = np.random.default_rng(42)
    n, nq, nkv, T = 4, 4, 1, 2048
    q, k, v = (dev(values(rng, s, dtype), dtype) for s in ((n, nq, d), (n, T, nkv, d), (n, T, nkv, d)))
    lens = [0, 1, 77, 1999]
    q.zero_()
    q[:, :, 0] = float(d) ** 0.5
    k[..., 0] = torch.finfo(TORCH[dtype]).min / 16
    want, wlse = _decode(q, k, v, lens, d)
    for s, m in enumerate(lens):
        k[s, m:], v[s, m:] = float("nan"), INF
    o, lse = _decode(q, k, v, lens, d)
    assert torch.equal(o, want) and torch.equal(lse, wlse)
    assert bool(o.isfinite().all()) and bool(lse[1:].isfinite().all()) and bool((o[0] == 0).all())
    _check_mean(o[3], v[3, :1999, 0], dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("size", [2.0 ** 20, 1e9, 1e30, 2e37])
@pytest.mark.parametrize("sign", [1, -1])
def test_packed_large_equal_scores(dtype, d, causal, size, sign):
    """Scores that are all the same large number, up to near the lowest of the type:
    every visible key has the same weight."""
    rng = np.random.default_rng(45)
    nq, nkv, cu = 2, 1, [0, 300, 333]
    x = dev(values(rng, (333, nq + 2 * nkv, d), dtype), dtype)
    x[:, :nq] = 0.0
    x[:, :nq, 0] = float(d) ** 0.5
    x[:, nq, 0] = sign * size
    o, lse = _packed(x, cu, nq, nkv, d, dtype, causal)
    score = float(x[0, 0, 0].double() * x[0, nq, 0].double()) / d ** 0.5
    for s, e in zip(cu[:-1], cu[1:]):
        for row in [s, s + 1, s + 31, s + 32, min(s + 130, e - 1), e - 1]:
            n = row + 1 - s if causal else e - s
            for h in range(nq):
                _check_mean(o[row, h], x[s:s + n, nq + 1], dtype)
                assert abs(float(lse[h, row]) - (score + np.log(n))) <= 2.0 ** -21 * abs(score)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1e9, 2e37])
def test_large_negative_scores_vanish_beside_others(dtype, d, size):
    """Keys 0 .. 99 with scores near the lowest number of the type, then the usual ones, in
    prompts and in a cache: the same as without those keys."""
    rng = np.random.default_rng(46)
    nq, nkv, T, cut = 2, 1, 400, 100
    x = dev(values(rng, (T, nq + 2 * nkv, d), dtype), dtype)
    x[:, :nq, 0], x[:, nq, 0] = 1.0, 0.0
    y = x.clone()
    y[:cut, nq, 0] = -size
    o, lse = _packed(y, [0, T], nq, nkv, d, dtype, False)
    q, k, v = y[:, :nq], y[None, :, nq:nq + 1], y[None, :, nq + 1:]
    od, ld = _decode(q[:1].contiguous(), k.contiguous(), v.contiguous(), [T], d)
    z = torch.cat([x[cut:], x[:cut]])                    # the usual keys first, then no others
    w, wl = _packed(z, [0, T - cut, T], nq, nkv, d, dtype, False)
    wd, wld = _decode(q[:1].contiguous(), z[None, :, nq:nq + 1].contiguous(), z[None, :, nq + 1:].contiguous(),
                      [T - cut], d)
    # the same keys elsewhere in the tiles: each side is off by at most the bounds of
    # serving_util, with its sum of weights times |v| at most max |v|
    f = x.double()
    qk = float((f[:, :nq].abs().flatten(0, 1) @ f[cut:, nq].abs().T).max()) / d ** 0.5
    score = d * 2.0 ** -23 * qk + 2.0 ** -22 * (1 + qk)
    e = 2 * score + 2.0 ** -21 + T * 2.0 ** -23 + (2.0 ** -8 if dtype == "bf16" else 0.0)
    half = torch.finfo(TORCH[dtype]).eps / 2
    tol = 2 * (e + half * (1 + e)) * float(f[:, nq + 1].abs().max())
    assert bool(((o[cut:].double() - w[:T - cut].double()).abs() <= tol).all())
    assert bool(((od.double() - wd.double()).abs() <= tol).all())
    ltol = 2 * (score + T * 2.0 ** -23 + 2.0 ** -22 * (1 + qk + np.log(T)))
    assert bool(((lse[:, cut:] - wl[:, :T - cut]).abs() <= ltol).all())
    assert bool(((ld - wld).abs() <= ltol).all())
