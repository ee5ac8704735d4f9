"""GPU tests of the operators for drafted tokens beside those in test_gpu_kv_tree.py and
test_gpu_tree_more.py: vectors next to each other."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from oracle import drafts
from tests.drafts_util import Batch, random_tree
from tests.serving_util import Cache, host, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


@pytest.mark.parametrize("lens_first", [True, False])
def test_accepted_indices_and_new_lengths_next_to_each_other(lens_first):
    rng = np.random.default_rng(80)
    b = Batch([(20, random_tree(rng, 9)), (0, random_tree(rng, 4)), (None, [-1]), (300, random_tree(rng, 30))])
    accepted = [8, 2, -1, 29]
    c = Cache(rng, b.lens, 16, 2, 64, "bf16")
    both = ints([-9] * 10)
    new, old = (both[1:5], both[5:9]) if lens_first else (both[5:9], both[1:5])
    old.copy_(ints(accepted))
    mgb.mgb_kv_accept(b.plan(4, 2, 64), c.desc, old, new)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    (kp, vp), lens = drafts.accept((c.k, c.v), c.table, b.cu, b.lens, b.trees, accepted)
    assert new.tolist() == lens and old.tolist() == accepted and both[0] == both[9] == -9
    for got, want in ((host(c.tk), kp), (host(c.tv), vp)):
        assert ((got == want) | (np.isnan(got) & np.isnan(want))).all()
