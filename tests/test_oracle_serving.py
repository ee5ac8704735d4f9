"""Pins of the serving oracle: rotations by closed forms, the paged cache by
explicit placement, packed attention by the dense oracle, decode attention by
the last rows of causal attention."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serving

RNG = np.random.default_rng(3)


def _rope(n, rot, base=10000.0):
    a = np.arange(n)[:, None] * base ** (-2.0 * np.arange(rot // 2) / rot)[None]
    return np.stack((np.cos(a), np.sin(a)), axis=-1)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,d", [(8, 8), (4, 10)])
def test_rotation(interleaved, rot, d):
    x = RNG.standard_normal((6, 3, d))
    y = serving.rope_rotate(x, _rope(6, rot), interleaved)
    np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-13)
    np.testing.assert_array_equal(y[0], x[0])               # position 0
    np.testing.assert_array_equal(y[..., rot:], x[..., rot:])
    z = x[:, :, :rot]
    z = z[..., 0::2] + 1j * z[..., 1::2] if interleaved else z[..., :rot // 2] + 1j * z[..., rot // 2:]
    w = z * np.exp(1j * np.arange(6)[:, None, None] * 10000.0 ** (-2.0 * np.arange(rot // 2) / rot))
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    np.testing.assert_allclose(a + 1j * b, w, atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_products_depend_on_the_distance_only(interleaved):
    q, k = RNG.standard_normal((2, 1, 1, 16))
    rope = _rope(50, 16)
    at = lambda x, p: serving.rope_rotate(x, rope[p:p + 1], interleaved)[0, 0]
    ref = at(q, 5) @ at(k, 2)
    for shift in (1, 17, 40):
        assert abs(at(q, 5 + shift) @ at(k, 2 + shift) - ref) < 1e-12
    assert abs(at(q, 9) @ at(k, 2) - ref) > 1e-3


def test_append_places_every_row_once():
    cu, lens = [0, 3, 3, 4, 9], [5, 7, 0, 5]   # 3 new of 5, none, padding, 5 of 5
    where = serving.append_positions(cu, lens, 11)
    assert where == [(0, 2), (0, 3), (0, 4), (-1, -1), (3, 0), (3, 1), (3, 2), (3, 3), (3, 4),
                     (-1, -1), (-1, -1)]
    table = np.array([[4, 1, 0], [2, 2, 2], [0, 0, 0], [3, 5, 6]])
    q, k, v = RNG.standard_normal((3, 11, 2, 4))
    pools = RNG.standard_normal((2, 7, 2, 2, 4))
    q2, k2, kp, vp = serving.kv_append(q, k, v, cu, lens, None, False, table, *pools)
    np.testing.assert_array_equal(q2, q)
    np.testing.assert_array_equal(k2, k)
    np.testing.assert_array_equal(kp[1, 0], k[0])          # position 2: second page, slot 0
    np.testing.assert_array_equal(vp[0, 0], v[2])          # position 4: third page, slot 0
    np.testing.assert_array_equal(kp[5, 1], k[7])
    changed = (kp != pools[0]).any(axis=(2, 3))
    assert changed.sum() == 8 and not changed[4].any() and not changed[2].any()


@pytest.mark.parametrize("causal", [False, True])
def test_packed_is_the_dense_oracle_per_sequence(causal):
    lens = [3, 0, 1, 6]
    cu = np.cumsum([0] + lens)
    q = RNG.standard_normal((12, 4, 8))
    k, v = RNG.standard_normal((2, 12, 2, 8))
    o, lse = serving.packed_attention(q, k, v, cu, causal)
    ref = torch.nn.functional.scaled_dot_product_attention(
        *(torch.from_numpy(np.moveaxis(np.repeat(x[4:10], r, axis=1), 1, 0).copy())
          for x, r in ((q, 1), (k, 2), (v, 2))), is_causal=causal).numpy()
    np.testing.assert_allclose(np.moveaxis(o[4:10], 1, 0), ref, atol=1e-12)
    np.testing.assert_allclose(o[3], np.repeat(v[3], 2, axis=0), atol=1e-14)  # a sequence of one
    assert np.isnan(o[10:]).all() and np.isfinite(o[:10]).all() and np.isfinite(lse[:, :10]).all()


def test_decode_is_the_last_row_of_causal_attention():
    n, nq, nkv, d, page = 7, 4, 2, 8, 3
    q = RNG.standard_normal((n, nq, d))
    k, v = RNG.standard_normal((2, n, nkv, d))
    table = np.array([[2, 0, 4], [1, 1, 1]])
    zeros = np.zeros((5, page, nkv, d))
    _, _, kp, vp = serving.kv_append(q, k, v, [0, n, n], [n, 0], None, False, table, zeros, zeros)
    o, lse = serving.packed_attention(q, k, v, [0, n])
    do, dl = serving.decode_attention(np.stack((q[-1], q[0])), kp, vp, table, [n, 0])
    np.testing.assert_allclose(do[0], o[-1], atol=1e-13)
    np.testing.assert_allclose(dl[0], lse[:, -1], atol=1e-13)
    assert (do[1] == 0).all() and np.isneginf(dl[1]).all()
    assert abs(oracle.serving.decode_attention(q[-1:], kp, vp, table, [n - 1])[0] - o[-1]).max() > 1e-3


@pytest.mark.parametrize("norm_pos,act", [("pre", "gelu"), ("post", "swiglu")])
def test_layer_without_rotation_is_the_block(norm_pos, act):
    from megatron_transformer_layer_fwd_gb300.inputs import LayerShape, layer_inputs
    shape = LayerShape(1, 6, 16, 4, 2, 4, 32, norm_pos=norm_pos, act=act, causal=True, glu_block=16)
    arr = layer_inputs(shape, seed=1, random_affine=True)
    y, _ = oracle.block_fwd(shape, arr, arr["x"])
    np.testing.assert_allclose(serving.layer_fwd(shape, arr, arr["x"]), y, atol=1e-12)
    # rotation by position: the first row of a sequence is at position 0, and a
    # causal row does not depend on the rows after it
    r = serving.layer_fwd(shape, arr, arr["x"], _rope(6, 4))
    np.testing.assert_allclose(r[0], y[0], atol=1e-12)
    assert np.abs(r[1:] - y[1:]).max() > 1e-9
    np.testing.assert_allclose(serving.layer_fwd(shape, arr, arr["x"][:4], _rope(6, 4)), r[:4], atol=1e-12)
