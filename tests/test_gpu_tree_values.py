"""Tree attention on the GPU, where a wrong schedule or a lost value would show: shares of a single key
tile, repeated; NaN in keys that a row sees; weights far below the largest; values that say which key
they came from, over every grouping of heads and every split into shares."""
import numpy as np
import pytest
import torch

from . import step_reference as R
from .test_gpu_step import check_tree, f64, reference_tree, run_tree, tree_case

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


def tight_bounds(c, ref):
    """Bounds of the kernels' error, term by term (u: half a step of the 16-bit type).
    Weights, relative: scores are float32 sums of D exact products, each addition off by at most 2^-23 of
    the sum of magnitudes (twice: a weight and the normaliser), exp2 and the joins 2^-20; their rounding to
    16 bits u, in the product alone (the normaliser sums them before it).
    Weights, absolute: fp16 ones are rounded to multiples of 2^-24 at the finest, half of that off, 2^7 above
    their weight against a reference that no later maximum undercuts: L keys are off by at most L 2^-32 of
    the largest |v|, over a normaliser of at least 1.
    Sums: a product adds 16 keys a step to float32, each step off by at most 2^-22 of the weighted mean of |v|
    (16 truncated addends and the sum); 64 additions a lane and tile and one a tile in the normaliser.
    The result is rounded once."""
    out, lse, size, smax = ref
    u, L = R.HALF[c["dt"]], int(c["L"].max())
    e32 = c["D"] * 2.0 ** -23 * smax + 2.0 ** -20
    sums = L / 16 * 2.0 ** -22 + (64 + L / 64) * 2.0 ** -24
    low = L * 2.0 ** -32 * float(c["v"].abs().max()) if c["dt"] is torch.float16 else 0.0
    acc = (2 * e32[..., None] + u + sums) * size + low
    lse_tol = e32 + sums + np.abs(np.where(np.isfinite(lse), lse, 0)) * 2.0 ** -21
    return acc + u * (np.abs(out) + acc) + R.TINY[c["dt"]], lse_tol


def check_tight(c, out, lse, ref):
    tol, lse_tol = tight_bounds(c, ref)
    n = int(c["qsl"][-1])
    got, got_l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    off, off_l = np.abs(got - ref[0])[:n], np.abs(got_l - ref[1])[:n]
    assert (off <= tol[:n]).all(), (np.argwhere(~(off <= tol[:n]))[:4], (off / tol[:n]).max())
    assert (off_l <= lse_tol[:n]).all(), (np.argwhere(~(off_l <= lse_tol[:n]))[:4], (off_l / lse_tol[:n]).max())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("gap", [8.5, 16.5, 20.5, 25.5, 29.0])
@pytest.mark.parametrize("Hq,Hkv,D,n", [(4, 2, 64, 5), (4, 4, 64, 30), (2, 1, 64, 9), (8, 2, 128, 20), (32, 4, 128, 20)])
def test_weights_far_below_the_largest(kc, Hq, Hkv, D, n, gap, dt):
    """One key takes nearly all the weight and its value is zero (a first token that attention rests on), so
    that the result is what the others' weights, 2^-gap each, leave: in fp16 they are below the normal range
    from a gap of 14 on, and below half of its smallest value from 25."""
    L = 9000
    c = tree_case(73, [L - n], [n], Hq, Hkv, D, 16, dt, masks=[(2 << i) - 1 for i in range(n)])
    c["scale"] = 1.0
    for name, fill in (("q", 0), ("k", 0)):
        c[name].fill_(fill)
    c["q"][..., 0] = 1
    v = 1 + 0.25 * torch.rand(c["v"].shape, generator=torch.Generator().manual_seed(1))
    c["v"].copy_(v.to(dt))
    first = int(c["table"][0, 0]) * 16
    c["k"].view(-1, Hkv, D)[first, :, 0] = gap * float(np.log(2.0))
    c["v"].view(-1, Hkv, D)[first] = 0
    ref = reference_tree(c)
    for workers in (1, 0, 40):
        out, lse, err = run_tree(kc, c, workers)
        assert err == 0
        check_tight(c, out, lse, ref)


def needles(seed, context, n, Hq, Hkv, D, bs, dt, window):
    """A case whose weight lies on some twenty keys, at the edges of key tiles, blocks and the tree and in
    between, each with about the same share: a value taken from another key shows in every row."""
    rng = np.random.default_rng(seed)
    c = tree_case(seed, [context], [n], Hq, Hkv, D, bs, dt, window, pad=2)
    gen = torch.Generator().manual_seed(seed)
    u = torch.sign(torch.randn(Hkv, D, generator=gen)).cuda()
    c["q"].copy_((0.5 * u.repeat_interleave(Hq // Hkv, 0) + 0.02 * torch.randn(c["q"].shape, generator=gen).cuda()).to(dt))
    c["k"].mul_(0.5)
    c["scale"] = 3.0 * D ** -0.5
    lo = max(0, context - window) + n if window else 0
    at = [lo, context - 1, *(x for x in (63, 64, 127, 128, 255, 256, 1023) if lo <= x < context),
          *rng.integers(lo, context, 12)]
    at = np.unique(np.array(at))
    slots = c["table"][0, at // bs].astype(np.int64) * bs + at % bs
    c["k"].view(-1, Hkv, D)[torch.from_numpy(slots).cuda()] = u.to(dt)
    return c, slots


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hq,Hkv,D,n,bs,window", [
    (8, 2, 128, 7, 16, 0), (32, 8, 128, 64, 16, 0), (32, 8, 128, 7, 8, 0), (12, 12, 64, 24, 16, 0), (6, 1, 64, 40, 16, 0),
    (4, 1, 128, 64, 32, 0), (12, 3, 64, 11, 16, 5000), (7, 7, 64, 50, 16, 0), (16, 1, 128, 3, 16, 0), (24, 2, 128, 40, 32, 3000)])
def test_every_value_comes_from_its_own_key(kc, Hq, Hkv, D, n, bs, window, dt):
    context = 9000
    c, slots = needles(74, context, n, Hq, Hkv, D, bs, dt, window)
    ref = reference_tree(c)
    tol, _ = tight_bounds(c, ref)
    # the bound tells each of these values from another's: planted in the oracle's result, where taking b's
    # value for a's moves a row by its weight on a
    q, kf, vf = f64(c["q"])[:n], f64(c["k"]).reshape(-1, Hkv, D), f64(c["v"]).reshape(-1, Hkv, D)
    for a, b in zip(slots, np.roll(slots, 1)):
        k, dv = (x.repeat(Hq // Hkv, 0) for x in (kf[a], vf[b] - vf[a]))
        weight = np.exp((q * k).sum(-1) * c["scale"] - ref[1][:n])
        assert (np.abs(weight[..., None] * dv) > 2 * tol[:n]).any(-1).all()
    for workers in (0, 1, 33, 700):
        out, lse, err = run_tree(kc, c, workers)
        assert err == 0
        check_tight(c, out, lse, ref)
        assert (out[n:] == 7).all() and (lse[n:] == 7).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", [
    ([0, 127, 128, 129], [64, 1, 5, 64], 8, 2, 128, 16, 0), ([300, 0, 17, 1000, 64], [33, 0, 64, 2, 63], 4, 4, 64, 32, 0),
    ([513, 5, 255], [60, 3, 1], 64, 8, 128, 16, 0), ([200, 40, 0], [64, 31, 12], 16, 1, 128, 8, 0),
    ([900, 65, 0], [9, 16, 10], 28, 7, 128, 32, 200), ([500, 128, 2], [12, 9, 11], 15, 3, 64, 16, 0),
    ([2000, 128, 4096], [16, 16, 40], 32, 8, 128, 32, 1024)], ids=lambda c: f"{max(c[0])}+{max(c[1])}_g{c[2] // c[3]}_d{c[4]}")
def test_tree_within_the_tight_bound(kc, case, dt):
    c = tree_case(75, *case[:6], dt, case[6])
    ref = reference_tree(c)
    finite = np.where(np.isfinite(ref[1]), ref[1], 0)
    for workers in (0, 1, 7):
        out, lse, err = run_tree(kc, c, workers)
        assert err == 0 and np.array_equal(np.isfinite(ref[1]), torch.isfinite(lse).cpu().numpy())
        check_tight(c, out, torch.where(torch.isfinite(lse), lse, 0), (ref[0], finite, *ref[2:]))


def test_a_bound_of_no_rows_declares_an_empty_batch(kc):
    """max_query_len 0: rows, lse and the error word stay as they were, although sequences have rows; a
    bound of 1 already rejects the longer ones."""
    c = tree_case(76, [20, 5], [3, 1], 8, 2, 128, 16, torch.bfloat16)
    out, lse, err = run_tree(kc, c, max_query_len=0)
    assert err == 0 and (out == 7).all() and (lse == 7).all()
    out, lse, err = run_tree(kc, c, max_query_len=1)
    assert err == 16 and (out[:3] == 0).all() and torch.isneginf(lse[:3]).all()
    check_tree(c, out, lse, rows=np.array([3]))
