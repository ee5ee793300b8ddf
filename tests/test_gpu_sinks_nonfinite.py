"""NaN and infinities in values that rows see, in the calls with a window and sinks: they reach their dim of the result
of every row that sees them, and of no other, however the keys are shared out."""
import numpy as np
import pytest
import torch

from tests.sinks_reference import BF16, F16, Inputs
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
