"""NaN and infinities in values that rows see, in the calls with a window and sinks: they reach their dim of the result
of every row that sees them, and of no other, however the keys are shared out."""
import numpy as np
import pytest
import torch

from tests.sinks_reference import BF16, F16, Inputs
from tests.test_gpu_prefill_sinks import prefill, verify as verify_prefill
from tests.test_gpu_sinks import decode, verify

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    from paged_kv_cache_block_gb300 import kvcache
    return kvcache


def odd_values(cache):
    return [np.nan] if cache == "e4m3" else [np.nan, np.inf, -np.inf]


@pytest.mark.parametrize("cache,dtype", [("same", BF16), ("same", F16), ("e4m3", BF16), ("e4m3", F16)])
@pytest.mark.parametrize("workers", [0, 1, 50])
@pytest.mark.parametrize("q_len,sinks", [(4, 4), (3, 64), (8, 5), (2, 2 ** 31 - 1)])
def test_decode_of_sequences_shorter_than_their_sinks(kv, cache, dtype, workers, q_len, sinks):
    """The rows' own tokens are sinks: each is in view of its row and the later ones."""
    ctx = [0, 1, 2, max(0, min(sinks, 70) - q_len), 62, 300]
    x = Inputs(40, ctx, [q_len] * len(ctx), 8, 2, window=16, sinks=sinks, cache=cache, dtype=dtype)
    bad = odd_values(cache)
    vc = x.v_cache.float().numpy()
    for b, c in enumerate(ctx):
        for i in range(q_len):  # a dim of its own for each token, in one of the heads
            vc[(*x.slot(b, c + i), i % 2, 3 * i + b)] = bad[i % len(bad)]
        vc[(*x.slot(b, c + q_len - 1), 1, 100)] = bad[0]
    x.v_cache = torch.from_numpy(vc).to(x.v_cache.dtype)
    verify(x, *decode(kv, x, num_workers=workers))
    out = x.reference()["out"]
    for b in range(len(ctx)):  # the last row sees what the one before it does not
        assert np.isnan(out[q_len * (b + 1) - 1, 4:, 100]).all() and np.isfinite(out[q_len * (b + 1) - 2, 4:, 100]).all()


def one_heavy_key(seed, ctx, new, D, cache, dtype, heavy):
    """Scores of 0 but for key `heavy`, 250 above the others: their weights are 0 in float32, and not in 64 bits."""
    x = Inputs(seed, ctx, new, 8, 2, D, window=4000, sinks=4, cache=cache, dtype=dtype)
    x.q = torch.ones_like(x.q)
    k = torch.zeros(x.k_cache.shape)
    for b in range(len(ctx)):
        k[x.slot(b, heavy)] = 250 / (D * x.scale * x.k_scale)
    x.k_cache = k.to(x.k_cache.dtype)
    return x


CASES = [("same", BF16, 128), ("same", F16, 128), ("same", F16, 64), ("e4m3", BF16, 128)]


@pytest.mark.parametrize("cache,dtype,D", CASES)
@pytest.mark.parametrize("workers", [0, 1, 3, 20, 300])
@pytest.mark.parametrize("ctx,q_len", [([3000], 1), ([3000], 4), ([3000], 3), ([700] * 12, 2)])
def test_decode_keeps_what_weighs_nothing(kv, cache, dtype, D, workers, ctx, q_len):
    """A NaN in the value of a key whose weight underflows reaches its dim in however many pieces the keys are taken."""
    for heavy in (0, 690):
        x = one_heavy_key(41, ctx, [q_len] * len(ctx), D, cache, dtype, heavy)
        vc = x.v_cache.float().numpy()
        for b, c in enumerate(ctx):
            for i, pos in enumerate((1, 140, c // 2, c - 20)):
                vc[(*x.slot(b, pos), i % 2, 7 * i + 1)] = np.nan
        x.v_cache = torch.from_numpy(vc).to(x.v_cache.dtype)
        out, lse, err = decode(kv, x, num_workers=workers)
        verify(x, out, lse, err)
        if cache == "same":  # an infinity: not in the result as a number, whether it comes out as itself or as NaN
            x.v_cache[x.v_cache.isnan()] = np.inf
            other = decode(kv, x, num_workers=workers)[0]
            assert torch.equal(other.isfinite(), out.isfinite())


@pytest.mark.parametrize("cache,dtype,D", CASES)
@pytest.mark.parametrize("workers", [0, 1, 3, 20, 300])
@pytest.mark.parametrize("ctx,new", [([3000], 1), ([3000], 40), ([3000], 90), ([700] * 12, 20)])
def test_prefill_keeps_what_weighs_nothing(kv, cache, dtype, D, workers, ctx, new):
    """The same, where the two chains of a row tile share its key tiles too."""
    for heavy in (0, 690):
        x = one_heavy_key(42, ctx, [new] * len(ctx), D, cache, dtype, heavy)
        vc = x.v_cache.float().numpy()
        for b, c in enumerate(ctx):
            for i, pos in enumerate((1, 140, c // 2, c - 20)):
                vc[(*x.slot(b, pos), i % 2, 7 * i + 1)] = np.nan
        x.v_cache = torch.from_numpy(vc).to(x.v_cache.dtype)
        out, lse, err = prefill(kv, x, num_workers=workers)
        verify_prefill(x, out, lse, err)
        if cache == "same":
            x.v_cache[x.v_cache.isnan()] = np.inf
            other = prefill(kv, x, num_workers=workers)[0]
            assert torch.equal(other.isfinite(), out.isfinite())
