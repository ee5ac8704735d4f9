"""mgb_kv_accept turns down lengths laid over the accepted indices, wholly or in part
(no GPU needed: before any launch)."""
import pytest

from megatron_transformer_layer_fwd_gb300 import mgb
from tests.test_drafts_host import P, _accept, _plan, lib  # noqa: F401


@pytest.mark.parametrize("n", [1, 3, 200])
def test_new_lengths_over_the_accepted_indices(lib, n):  # noqa: F811
    plan = lambda: _plan(lib, n_seqs=n)
    for off in {0, 1, n - 1, n // 2, 1 - n}:
        if abs(off) < n:
            assert _accept(lib, plan=plan(), accepted=P, new_lens=P + 4 * off) == mgb.MGB_ERR_INVALID_ARG, off
