"""Shared by the tests of drafted tokens: trees, batches, plans."""
import numpy as np
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from tests.serving_util import ints


def random_tree(rng, m, branch=3, roots=1):
    """Parents of m drafted tokens, level by level, the first `roots` without one."""
    return [-1 if i < roots else int(max(0, (i - roots) // branch - rng.integers(0, 2))) for i in range(m)]


class Batch:
    """Row offsets, lengths and parents of sequences (ctx, tree); ctx None: padding."""

    def __init__(self, seqs, tail=0):
        self.trees = [t for _, t in seqs]
        self.lens = [0 if c is None else c + len(t) for c, t in seqs]
        self.cu = [0]
        for _, t in seqs:
            self.cu.append(self.cu[-1] + len(t))
        self.tokens = self.cu[-1] + tail
        self.parents = [p for t in self.trees for p in t] + [-7] * tail
        self.n = len(seqs)

    def plan(self, nq, nkv, d, guard=None, parents=True, cu=None, lens=None):
        n = mgb.mgb_attention_tree_ws_bytes(self.n, self.tokens, nq, nkv, d)
        ws = guard.empty((n,), torch.uint8) if guard else torch.empty(n, dtype=torch.uint8, device="cuda")
        ws.fill_(0xC3)   # whatever was there before
        return mgb.mgb_attention_tree_prepare(
            self.n, self.tokens, nq, nkv, d, ints(self.cu if cu is None else cu),
            ints(self.lens if lens is None else lens), ints(self.parents) if parents else None, ws)

    def live(self):
        """Rows that belong to a sequence."""
        on = np.zeros(self.tokens, dtype=bool)
        for s, n in enumerate(self.lens):
            on[self.cu[s]:self.cu[s + 1]] = n > 0
        return on
