"""Tree attention on the GPU, where a wrong schedule or a lost value would show: shares of a single key
tile, repeated; NaN in keys that a row sees."""
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


@pytest.mark.parametrize("Hq,Hkv,D,context,n,window,key", [
    (16, 1, 128, 128, 2, 0, 128),      # the second key tile holds drafted keys alone
    (5, 1, 64, 384, 9, 0, 384),
    (1, 1, 128, 128, 64, 64, None),    # a row that sees no context inside its window: the first tile shows it nothing
    (24, 2, 64, 256, 30, 0, 261),      # three row tiles: a pair, and one alone
    (12, 2, 128, 640, 63, 0, 640),
    (8, 2, 128, 128, 5, 0, 128), (8, 2, 128, 192, 14, 100, 195), (8, 2, 128, 64, 30, 0, 64),
    (12, 12, 64, 128, 7, 0, 130), (12, 3, 64, 256, 16, 0, 256), (12, 4, 64, 64, 20, 64, 70)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_nan_keys_reach_the_rows_that_see_them(kc, Hq, Hkv, D, context, n, window, key, dt):
    """A NaN in a key makes every score against it NaN, and so the result and the lse of the rows that see
    it, of its kv head, however the keys are shared out; every other row keeps its bits."""
    rng = np.random.default_rng(n)
    masks = [1 << i if rng.random() < 0.5 else (2 << i) - 1 for i in range(n)]
    masks[0], masks[-1] = 1, (1 << n) - 1
    c = tree_case(71, [context], [n], Hq, Hkv, D, 16, dt, window, masks=masks)
    seen = R.seen_keys(c["masks"].view(np.uint64), n, context, window)
    keys = np.arange(context, context + n) if key is None else np.array([key])
    slots = c["table"][0, keys // 16].astype(np.int64) * 16 + keys % 16
    for head in range(0, Hkv, max(1, Hkv - 1)):
        p = dict(c, k=c["k"].clone())
        p["k"].view(-1, Hkv, D)[torch.from_numpy(slots).cuda(), head, 7] = float("nan")
        hit = np.zeros((n, Hq), bool)
        hit[:, head * (Hq // Hkv):(head + 1) * (Hq // Hkv)] = seen[:, keys].any(1)[:, None]
        assert hit.any()
        hit = torch.from_numpy(hit).cuda()
        for workers in (1, 0, 2, 3):
            out, lse, err = run_tree(kc, c, workers)
            out2, lse2, err2 = run_tree(kc, p, workers)
            assert err == 0 and err2 == 0
            assert torch.equal(torch.isnan(lse2), hit) and torch.equal(torch.isnan(out2), hit[..., None].expand_as(out2))
            assert torch.equal(out2[~hit], out[~hit]) and torch.equal(lse2[~hit], lse[~hit])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("drafts,Hq,Hkv,D", [([13, 64, 7, 30], 8, 2, 128), ([8, 7, 2, 5], 12, 3, 64), ([13, 16, 7, 11], 20, 5, 64),
                                             ([9, 11, 2, 8], 16, 1, 128), ([64, 20, 1, 40], 7, 1, 64)])
@pytest.mark.parametrize("window", [0, 70])
def test_nan_keys_of_trees_reach_the_rows_that_see_them(kc, dt, drafts, Hq, Hkv, D, window):
    contexts, bs = [150, 0, 128, 263], 16
    c = tree_case(72, contexts, drafts, Hq, Hkv, D, bs, dt, window)
    p = dict(c, k=c["k"].clone())
    touched = np.zeros(len(c["q"]), bool)
    for b, (ctx, n) in enumerate(zip(contexts, drafts)):
        t0 = int(c["qsl"][b])
        seen = R.seen_keys(c["masks"].view(np.uint64)[t0:t0 + n], n, ctx, window)
        some = np.flatnonzero(seen.any(0) & ~seen.all(0))
        for j in some[::max(1, len(some) // 3)]:
            touched[t0:t0 + n] |= seen[:, j]
            p["k"].view(-1, Hkv, D)[int(c["table"][b, j // bs]) * bs + j % bs, :, 3] = float("nan")
    assert touched.any()
    hit = torch.from_numpy(touched).cuda()
    for workers in (0, 1, 5):
        out, lse, _ = run_tree(kc, c, workers)
        out2, lse2, err = run_tree(kc, p, workers)
        assert err == 0 and torch.isnan(out2[hit]).all() and torch.isnan(lse2[hit]).all()
        assert torch.equal(out2[~hit], out[~hit]) and torch.equal(lse2[~hit], lse[~hit])
