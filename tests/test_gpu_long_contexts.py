"""Attention over contexts of more than 2^28 keys, whose indexes times the eight 16-byte chunks of a key's 64 dims leave
32 bits.  The block table names the same few blocks over and over, so that the caches stay small and the softmax is one
over the distinct keys, each weighed by how often it is seen."""
import numpy as np
import pytest
import torch

from tests.sinks_reference import BF16, Inputs
from tests.step_reference import HALF, TINY

pytestmark = pytest.mark.gpu

BLOCKS, BS = 3, 32
CTX = 2 ** 28 + 100003


@pytest.fixture(scope="module")
def kv():
    from paged_kv_cache_block_gb300 import kvcache
    return kvcache


@pytest.fixture(scope="module")
def table():
    n = CTX // BS + 2
    yield torch.arange(n, dtype=torch.int32, device="cuda")[None] % BLOCKS
    torch.cuda.empty_cache()


def seen(lo, hi):
    """How often the keys lo .. hi hold each slot of the blocks."""
    period = BLOCKS * BS
    r = np.arange(period)
    return np.maximum(0, (hi - r) // period - (lo - 1 - r) // period)


def check(x, q, out, lse, counts):
    """counts [rows, slots].  The bounds are those of sinks_reference.bounds (no weight is far from the largest), and the
    float32 sums: a share is a 152th of the keys, its products are added 16 keys at a time, off by 2^-23 each, and its
    weights 128 or fewer at a time by 2^-24."""
    D = x.D
    k, v = (x.values(n).reshape(-1, D) for n in ("k", "v"))
    q = q.double().cpu().numpy()
    s = np.einsum("thd,kd->thk", q, k) * x.scale
    w = np.exp(s - s.max(-1, keepdims=True)) * counts[:, None]
    l = w.sum(-1, keepdims=True)
    want, size = w @ v / l, w @ np.abs(v) / l
    smax = (np.abs(q) @ np.abs(k).T).max(-1) * x.scale
    e = D * 2.0 ** -23 * smax + 2.0 ** -20
    vcoded = 0.0
    if x.cache == "int4":
        ks, vs = (np.repeat(t.numpy().astype(np.float64), x.group, 1) for t in (x.k_scales, x.v_scales))
        e = D * 2.0 ** -23 * (np.abs(q) * ks).sum(-1) * 15 * x.scale + 2.0 ** -20 + 2.0 ** -11 * smax
        vcoded = 15 * vs
    share = counts.sum(1).max() / 152
    u = HALF[x.dtype]
    acc = (2 * e[..., None] + 2 * u) * size + share / 16 * 2.0 ** -23 * np.maximum(size, vcoded)
    over = np.abs(out.double().cpu().numpy() - want) / (acc + u * (np.abs(want) + acc) + TINY[x.dtype])
    assert over.max() <= 1, f"out: {over.max():.3g} times its bound"
    lse_want = (s.max(-1, keepdims=True) + np.log(l))[..., 0]
    over = np.abs(lse.double().cpu().numpy() - lse_want) / (e + np.abs(lse_want) * 2.0 ** -21 + share * 2.0 ** -24 + u)
    assert over.max() <= 1, f"lse: {over.max():.3g} times its bound"


def inputs(seed, rows, cache):
    x = Inputs(seed, [BLOCKS * BS - rows], [rows], 4, 1, 128, BS, cache=cache, spare=0)
    order = torch.from_numpy(x.table[0, :BLOCKS].astype(np.int64))
    x.k_cache, x.v_cache = (c.view(torch.uint8)[order].contiguous().view(c.dtype) for c in (x.k_cache, x.v_cache))
    return x


@pytest.mark.parametrize("cache", ["same", "e4m3", "int4"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2 ** 28 + 77, 5), (40, 2 ** 28)])
@pytest.mark.parametrize("rows,decode", [(3, True), (3, False), (40, False)])
def test_windows_and_sinks(kv, table, cache, window, sinks, rows, decode):
    x = inputs(50, rows, cache)
    d = x.device()
    L = CTX + rows
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    lse, err = torch.empty(rows, 4, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    a = (d["q"], d["k_cache"], d["v_cache"], table, lens)
    a += (2 ** 31 - 1, rows, x.scale) if decode else (d["qsl"], 2 ** 31 - 1, rows, x.scale)
    name = "paged_attention_" + ("decode" if decode else "prefill") + "_sinks"
    if cache == "int4":
        out = getattr(kv, name + "_int4")(*a, d["k_scales"], d["v_scales"], window, sinks, lse_out=lse, d_err=err)
    else:
        out = getattr(kv, name)(*a, window, sinks, x.k_scale, x.v_scale, lse_out=lse, d_err=err)
    assert int(err) == 0
    counts = []
    for p in range(CTX, L):
        lo = max(0, p - window + 1) if window else 0
        counts.append(seen(lo, p) + seen(0, min(sinks, lo) - 1))
    check(x, d["q"], out, lse, np.stack(counts).astype(np.float64))


@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("window", [0, 2 ** 28 + 77])
def test_trees(kv, table, rows, window):
    x = inputs(51, rows, "same")
    d = x.device()
    lens = torch.tensor([CTX + rows], dtype=torch.int32, device="cuda")
    mask = torch.tensor([(1 << (i + 1)) - 1 for i in range(rows)], dtype=torch.int64, device="cuda")
    lse, err = torch.empty(rows, 4, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = kv.paged_attention_tree(d["q"], d["k_cache"], d["v_cache"], table, lens, d["qsl"], mask, 2 ** 31 - 1, rows, x.scale,
                                  window, lse_out=lse, d_err=err)
    assert int(err) == 0
    counts = np.stack([seen(max(0, p - window + 1) if window else 0, p) for p in range(CTX, CTX + rows)])
    check(x, d["q"], out, lse, counts.astype(np.float64))
