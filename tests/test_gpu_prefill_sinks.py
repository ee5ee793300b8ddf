"""Prefill attention with a sliding window and sinks, over 16-bit, E4M3 and INT4 caches, against the 64-bit
implementation."""
import numpy as np
import pytest
import torch

from tests.sinks_reference import BF16, F16, Inputs, check
from tests.step_reference import HALF, TINY

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    from paged_kv_cache_block_gb300 import kvcache
    return kvcache


def prefill(kv, x, d=None, **kw):
    """The library's call on the inputs x; returns out, lse, err."""
    d = x.device() if d is None else d
    lse = torch.full(x.q.shape[:2], 7.0, dtype=torch.float32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(lse_out=lse, d_err=err, **kw)
    max_len, max_new = kw.pop("max_seq_len", int(x.lens.max(initial=1))), kw.pop("max_query_len", int(x.new.max(initial=1)))
    head = (d["q"], d["k_cache"], d["v_cache"], d["table"], d["lens"], d["qsl"], max_len, max_new, x.scale)
    if x.cache == "int4":
        out = kv.paged_attention_prefill_sinks_int4(*head, d["k_scales"], d["v_scales"], x.window, x.sinks, **kw)
    else:
        out = kv.paged_attention_prefill_sinks(*head, x.window, x.sinks, x.k_scale, x.v_scale, **kw)
    torch.cuda.synchronize()
    return out, lse, int(err)


def verify(x, out, lse, err=0, want_err=0, rows=slice(None)):
    r = x.reference()
    tol, lse_tol = x.bounds(r, shift=7)
    assert err == want_err, f"error bits {err}"
    a = check(out[rows], r["out"][rows], tol[rows], "out")
    b = check(lse[rows], r["lse"][rows], np.broadcast_to(lse_tol, r["lse"].shape)[rows], "lse")
    return a, b


CACHES = [("same", BF16), ("same", F16), ("e4m3", BF16), ("e4m3", F16), ("int4", BF16), ("int4", F16)]


@pytest.mark.parametrize("cache,dtype", CACHES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5), (33, 40)])
def test_caches(kv, cache, dtype, window, sinks):
    x = Inputs(1, [0, 5, 300, 1000, 129], [1, 200, 70, 33, 0], 8, 2, window=window, sinks=sinks, cache=cache, dtype=dtype)
    verify(x, *prefill(kv, x))


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 8, 128), (28, 4, 128), (16, 1, 128), (128, 1, 128), (6, 2, 128), (12, 12, 64), (5, 1, 64),
                                      (40, 8, 64), (120, 2, 64)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_heads(kv, Hq, Hkv, D, dtype):
    x = Inputs(2, [0, 150, 40], [90, 1, 37], Hq, Hkv, D, window=64, sinks=3, dtype=dtype)
    verify(x, *prefill(kv, x))


@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("window,sinks", [(0, 9), (1, 0), (1, 1), (7, 4), (64, 31), (128, 128), (200, 1), (1000, 16), (48, 1000),
                                          (130, 300), (2 ** 31 - 1, 3), (20, 2 ** 31 - 1)])
def test_masks(kv, bs, window, sinks):
    x = Inputs(3, [0, 3, 64, 255, 700], [50, 65, 3, 40, 100], 8, 2, bs=bs, window=window, sinks=sinks)
    verify(x, *prefill(kv, x))


@pytest.mark.parametrize("cache", ["same", "e4m3", "int4"])
@pytest.mark.parametrize("workers", [1, 2, 7, 151, 400])
def test_shares(kv, cache, workers):
    """The same items whole, in two pieces and in one a key tile."""
    x = Inputs(4, [1500, 0, 600], [100, 300, 1], 8, 2, window=900, sinks=70, cache=cache)
    verify(x, *prefill(kv, x, num_workers=workers))


@pytest.mark.parametrize("workers", [0, 3])
@pytest.mark.parametrize("Hq", [4, 32])
def test_one_sequence_of_few_rows(kv, workers, Hq):
    """A row tile whose key tiles the two chains share, over every worker."""
    for new in (1, 2, 5):
        x = Inputs(5 + new, [9000], [new], Hq, 2, window=0 if new == 2 else 6000, sinks=4)
        verify(x, *prefill(kv, x, num_workers=workers))


@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("group", [8, 16, 64, 128])
def test_int4_groups(kv, bs, group):
    x = Inputs(6, [0, 100, 400], [40, 33, 128], bs=bs, window=130, sinks=20, cache="int4", group=group)
    verify(x, *prefill(kv, x))


@pytest.mark.parametrize("cache", ["int4", "e4m3"])
@pytest.mark.parametrize("size", [2.0 ** -40, 2.0 ** 15])
def test_queries_of_any_size(kv, cache, size):
    """Queries (and INT4 scales) far from fp16's range: each row brings its own power of two."""
    x = Inputs(7, [200, 30], [40, 20], window=100, sinks=4, cache=cache)
    x.q[::3] = (x.q[::3].float() * size).to(BF16)
    x.q[1] = 0
    if cache == "int4":
        x.k_scales *= 2.0 ** -30
        x.v_scales *= 2.0 ** -20
        x.scale *= 2.0 ** 30
    if size > 1:
        x.scale /= size
    verify(x, *prefill(kv, x))


@pytest.mark.parametrize("cache,dtype", [("same", BF16), ("same", F16), ("e4m3", BF16)])
@pytest.mark.parametrize("workers", [0, 1])
@pytest.mark.parametrize("Hq,new", [(16, 70), (4, 20), (2, 300)])
def test_nan_where_rows_do_not_see(kv, cache, dtype, workers, Hq, new):
    """Keys and values that some or all rows do not see: later rows' tokens, the window's edge, the gap behind the
    sinks.  The rows that see them get NaN and infinities, the others nothing."""
    window, sinks, ctx = 40, 3, 200
    x = Inputs(8, [ctx, ctx, 0, ctx], [new] * 4, Hq, 2, window=window, sinks=sinks, cache=cache, dtype=dtype, release=False)
    bad = [np.nan] if cache == "e4m3" else [np.nan, np.inf, -np.inf]
    kc, vc = x.k_cache.float().numpy(), x.v_cache.float().numpy()
    lo = ctx - window + 1
    for b, places in ((0, [ctx + new - 1, ctx + new - 2, ctx + 1]), (1, [lo, lo + 1, lo + 7, lo - 1, sinks, sinks + 1]), (2, [new - 1, 4])):
        for i, pos in enumerate(places):
            vc[(*x.slot(b, pos), i % 2, 5 + i)] = bad[i % len(bad)]
            vc[(*x.slot(b, pos), 0, 77)] = bad[0]
        kc[(*x.slot(b, places[0]), 1, 3)] = np.nan
    vc[(*x.slot(3, 1), 0, 9)] = bad[-1]   # a sink: every row
    x.k_cache, x.v_cache = (torch.from_numpy(t).to(x.k_cache.dtype) for t in (kc, vc))
    verify(x, *prefill(kv, x, num_workers=workers))
    r = x.reference()["out"]
    assert np.isnan(r).any() and np.isfinite(r[0, 2 if Hq > 2 else 1:]).any()


@pytest.mark.parametrize("cache,dtype", [("same", F16), ("same", BF16), ("e4m3", BF16), ("int4", BF16)])
def test_weights_beside_a_sink(kv, cache, dtype):
    """A sink whose score is far above the others' and whose value is zero: what the result is then made of are
    weights of 2^-23 of the largest."""
    x = Inputs(9, [4000], [3], 4, 1, window=3500, sinks=1, cache=cache, dtype=dtype)
    x.q = torch.ones_like(x.q)
    blk, off = x.slot(0, 0)
    x.scale = 16.0 / 128
    if cache == "int4":
        x.k_scales[:], x.v_scales[:] = 1.0, 1.0
        x.k_cache[:], x.v_cache[:] = 0x00, 0x33
        x.k_cache[blk, off], x.v_cache[blk, off] = 0x11, 0x00
    else:
        x.k_cache, x.v_cache = torch.zeros_like(x.k_cache), torch.full(x.v_cache.shape, 3.0).to(x.v_cache.dtype)
        x.k_cache[blk, off] = torch.ones(128).to(x.k_cache.dtype)
        x.v_cache[blk, off] = torch.zeros(128).to(x.v_cache.dtype)
        x.scale /= x.k_scale
    out, lse, err = prefill(kv, x)
    want = x.reference()["out"]
    assert err == 0
    # one rounding of each weight and of the result, whose terms are all of one sign; and float32
    u = 2.0 ** -8 if dtype is BF16 else 2.0 ** -11
    check(out, want, (2 * u + 2.0 ** -11) * np.abs(want), "out")


def test_rising_scores(kv):
    """A reference maximum that has to move at every tile, and one that never does again."""
    for sign in (1, -1):
        x = Inputs(10, [700], [40], 8, 2)
        x.scale = 1.0
        x.q = torch.full_like(x.q, 0.5)
        k = torch.zeros(x.k_cache.shape)
        for p in range(740):
            k[x.slot(0, p)] = sign * 0.01 * (p // 4) * 4
        x.k_cache = k.to(BF16)
        verify(x, *prefill(kv, x))


def test_scale_of_zero(kv):
    x = Inputs(11, [100], [20], 8, 2, window=30, sinks=2)
    x.scale = 0.0
    verify(x, *prefill(kv, x))


def test_rejected_lengths_bad_blocks_and_rows_behind(kv):
    x = Inputs(12, [30, 500, 80, 90, 10], [20, 30, 10, 40, 25], window=48, sinks=4)
    d = x.device()
    lens = d["lens"].clone()
    lens[0], lens[2] = 19, 4000            # fewer than its rows; past max_seq_len
    big = {**d, "lens": lens, "q": torch.cat([d["q"], d["q"][:7]])}   # seven rows of no sequence
    out = torch.full_like(big["q"], 5.0)
    lse = torch.full(out.shape[:2], 5.0, dtype=torch.float32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for workers in (0, 1):
        kv.paged_attention_prefill_sinks(big["q"], big["k_cache"], big["v_cache"], big["table"], big["lens"], big["qsl"], 3999, 40,
                                         x.scale, 48, 4, num_workers=workers, out=out, lse_out=lse, d_err=err)
        assert int(err) == kv.KV_DERR_BAD_LEN
        for rows in (slice(0, 20), slice(50, 60)):
            assert (out[rows] == 0).all() and torch.isneginf(lse[rows]).all()
        assert (out[125:] == 5).all() and (lse[125:] == 5).all()
        for rows in (slice(20, 50), slice(60, 125)):
            verify(x, out[:125], lse[:125], rows=rows)
    # a sequence of more rows than max_query_len
    out, lse, err = prefill(kv, x, max_query_len=39)
    assert err == kv.KV_DERR_BAD_LEN and (out[60:100] == 0).all()
    verify(x, out, lse, rows=slice(0, 60))
    verify(x, out, lse, rows=slice(100, 125))
    # a bad id: its keys read as zeros
    for bad in (-1, x.NB):
        table = x.table.copy()
        old = table[1, 30]
        table[1, 30] = bad
        out, lse, err = prefill(kv, x, {**d, "table": torch.from_numpy(table).cuda()})
        assert err == kv.KV_DERR_BAD_BLOCK
        y = Inputs(12, [30, 500, 80, 90, 10], [20, 30, 10, 40, 25], window=48, sinks=4)
        y.k_cache[old], y.v_cache[old] = 0, 0
        verify(y, out, lse)


def test_every_kind_of_batch_repeats_bit_for_bit(kv):
    for cache in ("same", "e4m3", "int4"):
        x = Inputs(13, [300, 0, 77], [90, 140, 1], 8, 2, window=100, sinks=9, cache=cache)
        d = x.device()
        a, la, _ = prefill(kv, x, d)
        for _ in range(3):
            b, lb, _ = prefill(kv, x, d)
            assert torch.equal(a, b) and torch.equal(la, lb)


def test_many_short_sequences(kv):
    rng = np.random.default_rng(14)
    x = Inputs(14, rng.integers(0, 40, 1000), rng.integers(0, 4, 1000), 4, 2, window=16, sinks=4)
    verify(x, *prefill(kv, x))


def test_empty(kv):
    x = Inputs(15, [20, 30], [0, 0], 4, 2)
    out, lse, err = prefill(kv, x, max_query_len=0)
    assert out.shape[0] == 0 and err == 0
    x = Inputs(15, [20, 30], [3, 0], 4, 2)
    d = x.device()
    out = torch.full_like(d["q"], 3.0)
    prefill(kv, x, d, max_query_len=0, out=out)
    assert (out == 3).all()


@pytest.mark.parametrize("cache", ["same", "e4m3", "int4"])
def test_chunks_of_a_prompt_are_the_prompt(kv, cache):
    """A prompt in chunks of several sizes, and its last tokens by the decode call."""
    total = 250
    whole = Inputs(16, [0], [total], 8, 2, window=90, sinks=6, cache=cache, release=False)
    d = whole.device()
    out, lse, err = prefill(kv, whole, d)
    r = whole.reference()
    tol = whole.bounds(r, shift=7, rounded_sum=True)[0]
    at = 0
    for n in (1, 63, 64, 100, 14, 8):
        qsl = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        lens = torch.tensor([at + n], dtype=torch.int32, device="cuda")
        q = d["q"][at:at + n].contiguous()
        head = (q, d["k_cache"], d["v_cache"], d["table"], lens)
        if cache == "int4":
            part = kv.paged_attention_prefill_sinks_int4(*head, qsl, 300, n, whole.scale, d["k_scales"], d["v_scales"], 90, 6)
        else:
            part = kv.paged_attention_prefill_sinks(*head, qsl, 300, n, whole.scale, 90, 6, whole.k_scale, whole.v_scale)
        check(part, r["out"][at:at + n], tol[at:at + n], "chunk")
        if n <= 8:
            if cache == "int4":
                part = kv.paged_attention_decode_sinks_int4(*head, 300, n, whole.scale, d["k_scales"], d["v_scales"], 90, 6)
            else:
                part = kv.paged_attention_decode_sinks(*head, 300, n, whole.scale, 90, 6, whole.k_scale, whole.v_scale)
            check(part, r["out"][at:at + n], tol[at:at + n], "decode")
        at += n


@pytest.mark.parametrize("cache", ["same", "int4"])
def test_graphs_share_a_workspace_and_streams(kv, cache):
    x = Inputs(17, [900, 30], [60, 100], window=500, sinks=4, cache=cache)
    y = Inputs(18, [70, 1500], [30, 3], window=500, sinks=4, cache=cache)
    both = [(z, z.device()) for z in (x, y)]
    code = kv.KV_INT4 if cache == "int4" else kv.KV_BF16
    ws = torch.empty(kv.paged_attention_prefill_sinks_workspace_size(2, 100, 8, 2, 128, code, 4096, 500, 4), dtype=torch.uint8,
                     device="cuda")
    graphs, outs = [], []
    side = torch.cuda.Stream()

    def call(z, d, out, stream=None):
        head = (d["q"], d["k_cache"], d["v_cache"], d["table"], d["lens"], d["qsl"], 4096, 100, z.scale)
        kw = dict(workspace=ws, out=out, stream=stream)
        if cache == "int4":
            kv.paged_attention_prefill_sinks_int4(*head, d["k_scales"], d["v_scales"], 500, 4, **kw)
        else:
            kv.paged_attention_prefill_sinks(*head, 500, 4, **kw)

    for z, d in both:
        out = torch.empty_like(d["q"])
        side.wait_stream(torch.cuda.current_stream())
        call(z, d, out, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(z, d, out)
        graphs.append(g)
        outs.append(out)
    for _ in range(3):
        for out in outs:
            out.fill_(9)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (z, _), out in zip(both, outs):
            r = z.reference()
            check(out, r["out"], z.bounds(r, shift=7)[0], "out")


@pytest.mark.parametrize("cache", ["same", "int4", "e4m3"])
def test_caches_past_32_bits(kv, cache):
    x = Inputs(19, [60, 40], [30, 70], 8, 8, window=24, sinks=2, cache=cache, spare=0)
    d = x.device()
    per = x.k_cache[0].numel()
    NB = (2 ** 31) // per + 500
    if cache == "same":
        x.v_cache[(*x.slot(0, 62), 1, 5)] = np.inf  # fetched again for the rows that see it
    big = []
    for t in (x.k_cache, x.v_cache):
        c = torch.empty((NB, *t.shape[1:]), dtype=t.dtype, device="cuda")
        c[NB - x.NB:] = t.cuda()
        big.append(c)
    d |= dict(k_cache=big[0], v_cache=big[1], table=torch.where(d["table"] >= 0, d["table"] + (NB - x.NB), -1))
    verify(x, *prefill(kv, x, d))


@pytest.mark.parametrize("cache,dtype", [("same", BF16), ("same", F16), ("e4m3", BF16)])
@pytest.mark.parametrize("Hq", [2, 16])
def test_one_key_comes_out_as_it_is(kv, cache, dtype, Hq):
    """A row that sees one key is that key's value, a bit copy over a 16-bit cache (E4M3: times v_scale, one rounding)."""
    x = Inputs(31, [0, 0, 40], [1, 90, 3], Hq, 2, window=1, sinks=0, cache=cache, dtype=dtype)
    out, lse, err = prefill(kv, x)
    verify(x, out, lse, err)
    got, v = out.float().cpu().numpy(), x.values("v")
    for b, (q0, n) in enumerate(zip(x.qsl, x.new)):
        for t in range(min(n, 64 - (x.lens[b] - n))):
            want = np.repeat(v[x.slot(b, x.lens[b] - n + t)], Hq // 2, 0)
            want = torch.from_numpy(want).to(dtype).float().numpy()
            if cache == "same":
                assert np.array_equal(got[q0 + t], want), (b, t)
            else:  # the sum's reciprocal, the product and the output are rounded
                step = np.abs(want) * (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -21)
                assert (np.abs(got[q0 + t] - want) <= step).all(), (b, t)


@pytest.mark.parametrize("cache", ["same", "int4"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (8, 8), (128, 1), (256, 2)])
def test_a_loose_bound_of_the_rows(kv, cache, Hq, Hkv):
    """Any max_query_len above the true one gives the tight one's bits: the items to merge are counted without it."""
    x = Inputs(32, [700, 0, 30], [5, 40, 1], Hq, Hkv, window=400, sinks=4, cache=cache)
    d = x.device()
    want = prefill(kv, x, d)
    verify(x, *want)
    # (of a tile of one token, 2^29 .. 2^30 + 2 made a product of 2^31 and more)
    for bound in (41, 4096, 2 ** 29, 2 ** 30 + 2, 2 ** 31 - 1):
        out, lse, err = prefill(kv, x, d, max_query_len=bound)
        assert err == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])


def one_rounding(x, out, want, acc=0.0):
    """out within acc (and float32's 2^-21) of want, rounded once (to a subnormal: half its step, which also
    keeps the quotient of the check defined where a value is 0)."""
    acc = acc + 2.0 ** -21 * np.abs(want)
    check(out, want, acc + HALF[x.dtype] * (np.abs(want) + acc) + TINY[x.dtype], "out")


@pytest.mark.parametrize("cache,dtype", CACHES)
@pytest.mark.parametrize("Hq,D", [(2, 128), (16, 128), (16, 64)])
def test_one_key_at_any_position(kv, cache, dtype, Hq, D):
    """A window of one key: each row is that key's value wherever it stands in the sequence."""
    if D == 64 and cache != "same":
        pytest.skip("128 dims alone")
    x = Inputs(33, [0, 100, 1000, 63], [200, 3, 150, 2], Hq, 2, D, window=1, sinks=0, cache=cache, dtype=dtype)
    out, lse, err = prefill(kv, x)
    verify(x, out, lse, err)
    v = x.values("v")
    rows = [v[x.slot(b, L - n + t)] for b, (L, n) in enumerate(zip(x.lens, x.new)) for t in range(n)]
    want = np.repeat(np.stack(rows), Hq // 2, 1)
    one_rounding(x, out, want)
    if cache == "same":
        assert np.array_equal(out.double().cpu().numpy(), want)


@pytest.mark.parametrize("cache,dtype", CACHES)
@pytest.mark.parametrize("workers", [0, 1, 40])
@pytest.mark.parametrize("new", [1, 5, 300])
@pytest.mark.parametrize("at", [0, 480])
def test_rows_of_one_heavy_key(kv, cache, dtype, workers, new, at):
    """A key that holds nearly all of every row's weight, a sink or one in the window: its value and one rounding."""
    x = Inputs(34, [500], [new], 8, 2, window=400, sinks=1, cache=cache, dtype=dtype)
    rng = np.random.default_rng(35)
    x.q = torch.from_numpy(1 + 0.25 * rng.standard_normal(x.q.shape)).to(dtype)
    blk, off = x.slot(0, at)
    # scores of about `heavy` and `others` in powers of 2, near the reference that the kernel begins with: a key far
    # above it has a weight of 1, which has no rounding
    heavy, others = (6.5, -25.0) if at == 0 else (14.5, -14.5)
    unit = x.scale * 128 / np.log(2)
    if cache == "int4":
        code = 2 if at == 0 else 7
        x.k_scales[:] = heavy / unit / code
        x.k_cache[:] = 0x88 if at == 0 else 0x99   # -8, -7
        x.k_cache[blk, off] = code * 0x11
    else:
        x.k_cache = torch.full(x.k_cache.shape, others / unit / x.k_scale).to(x.k_cache.dtype)
        x.k_cache[blk, off] = torch.full(x.k_cache.shape[2:], heavy / unit / x.k_scale).to(x.k_cache.dtype)
    r = x.reference()
    out, lse, err = prefill(kv, x, num_workers=workers)
    verify(x, out, lse, err)
    # (32 products of 16 keys or fewer: each addition to the heavy key's, of next to nothing, is off by 2^-23 at most)
    v = np.abs(x.values("v"))
    one_rounding(x, out, r["out"], 2.0 ** -18 * float(v[np.isfinite(v)].max()))
    value = np.repeat(x.values("v")[blk, off], 4, 0)
    assert np.abs(r["out"] - value).max() < 2.0 ** -17 * v[np.isfinite(v)].max(), "the inputs are what they claim"


@pytest.mark.parametrize("workers", [0, 1])
@pytest.mark.parametrize("new,Hq,D", [(3, 8, 128), (200, 8, 128), (60, 4, 64)])
def test_values_near_the_largest(kv, workers, new, Hq, D):
    """Values of 2^120 under scores that rise by powers of two: a weighted mean never leaves their range."""
    x = Inputs(36, [500], [new], Hq, 2, D, window=300, sinks=4)
    x.v_cache = (x.v_cache.float() * 2.0 ** 120).to(BF16)
    x.q = torch.ones_like(x.q)
    k = torch.zeros(x.k_cache.shape)
    unit = x.scale * D / np.log(2)
    for p in range(500 + new):
        if p < 4 or p > 200:  # from 2^-14 to 2^14
            k[x.slot(0, p)] = (28 * p / (500 + new) - 14) / unit
    x.k_cache = k.to(BF16)
    r = x.reference()
    assert np.isfinite(r["out"]).all() and np.abs(r["out"]).max() > 2.0 ** 116
    verify(x, *prefill(kv, x, num_workers=workers))


@pytest.mark.parametrize("cache", ["int4", "e4m3"])
@pytest.mark.parametrize("exponent", [-110, -60, 60, 118])
def test_queries_times_a_power_of_two(kv, cache, exponent):
    """Over E4M3 and INT4 caches each row brings its own power of two: queries larger or smaller by one under a scale that
    takes it off give the same bits, over all of bf16's exponents."""
    x = Inputs(37, [200, 30], [40, 20], window=100, sinks=4, cache=cache)
    x.q[x.q.abs() < 2.0 ** -8] = 0  # (so that no query leaves the normal numbers)
    want, lse, err = prefill(kv, x)
    verify(x, want, lse, err)
    x.q = (x.q.double() * 2.0 ** exponent).to(BF16)
    x.scale *= 2.0 ** -exponent
    out, lse2, err = prefill(kv, x)
    assert err == 0 and torch.equal(out, want) and torch.equal(lse2, lse)


@pytest.mark.parametrize("cache,dtype", CACHES)
@pytest.mark.parametrize("sinks", [2 ** 28 - 1, 2 ** 28 + 300, 2 ** 29, 2 ** 31 - 200, 2 ** 31 - 1])
@pytest.mark.parametrize("window", [1, 40, 2 ** 31 - 1])
def test_loose_bounds_and_sinks_past_any_length(kv, cache, dtype, sinks, window):
    """max_seq_len bounds nothing, and no sequence is as long as the sinks: every earlier key is seen."""
    x = Inputs(38, [118, 700, 0], [150, 1, 5], 8, 2, window=window, sinks=sinks, cache=cache, dtype=dtype)
    for workers in (0, 1000):
        verify(x, *prefill(kv, x, max_seq_len=2 ** 31 - 1, num_workers=workers))
