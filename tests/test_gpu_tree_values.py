"""Tree attention on the GPU, where a wrong schedule or a lost value would show: shares of a single key
tile, repeated; NaN in keys that a row sees; weights far below the largest; values that say which key
they came from, over every grouping of heads and every split into shares."""
import numpy as np
import pytest
import torch

from . import step_reference as R
from .test_gpu_step import check_tree, reference_tree, run_tree, tree_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kc():
    from paged_kv_cache_block_gb300 import kvcache
    return kvcache


@pytest.mark.parametrize("Hq,Hkv,D,most", [(16, 1, 128, 8), (5, 1, 64, 24), (1, 1, 128, 1), (12, 2, 128, 63), (24, 2, 64, 30)])
def test_pieces_of_one_row_tile_and_one_key_tile_repeat(kc, Hq, Hkv, D, most):
    """One kv head, or a last row tile without a partner, over contexts within one key tile: every share is
    one piece in which the second chain has no tile and hands on its empty result at once, while the other
    warps may still be taking the share's start from the schedule."""
    rng = np.random.default_rng(70 + Hq)
    B = 60
    drafts = rng.integers(max(1, most - 12), most + 1, B).tolist()
    contexts = rng.integers(0, 128 - most, B).tolist()
    c = tree_case(70 + Hq, contexts, drafts, Hq, Hkv, D, 16, torch.bfloat16)
    out, lse, err = run_tree(kc, c)
    assert err == 0
    check_tree(c, out, lse)
    for _ in range(150):
        again, lse2, err = run_tree(kc, c)
        assert err == 0 and torch.equal(out, again) and torch.equal(lse, lse2)
