"""Decode attention with a sliding window and sinks against the 64-bit implementation."""
import numpy as np
import pytest
import torch

from tests.sinks_reference import BF16, F16, Inputs, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    from paged_kv_cache_block_gb300 import kvcache
    return kvcache


def decode(kv, x, d=None, **kw):
    """The library's call on the inputs x; returns out, lse, err."""
    d = x.device() if d is None else d
    lse = torch.full(x.q.shape[:2], 7.0, dtype=torch.float32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(lse_out=lse, d_err=err, **kw)
    q_len = int(x.new[0]) if len(x.new) else 1
    max_len = kw.pop("max_seq_len", int(x.lens.max(initial=1)))
    head = (d["q"], d["k_cache"], d["v_cache"], d["table"], d["lens"], max_len, q_len, x.scale)
    if x.cache == "int4":
        out = kv.paged_attention_decode_sinks_int4(*head, d["k_scales"], d["v_scales"], x.window, x.sinks, **kw)
    else:
        out = kv.paged_attention_decode_sinks(*head, x.window, x.sinks, x.k_scale, x.v_scale, **kw)
    torch.cuda.synchronize()
    return out, lse, int(err)


def verify(x, out, lse, err=0, want_err=0):
    r = x.reference()
    tol, lse_tol = x.bounds(r, rounded_sum=x.cache == "int4")
    assert err == want_err, f"error bits {err}"
    check(out, r["out"], tol, "out")
    check(lse, r["lse"], lse_tol, "lse")


HEADS = [(8, 2, 128), (8, 8, 128), (28, 4, 128), (32, 8, 128), (16, 1, 128), (12, 12, 64), (5, 1, 64)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_heads(kv, Hq, Hkv, D, dtype):
    x = Inputs(1, [0, 15, 40, 63, 64, 100, 500, 777], [1] * 8, Hq, Hkv, D, window=64, sinks=5, dtype=dtype)
    verify(x, *decode(kv, x))


@pytest.mark.parametrize("bs", [4, 8, 16, 32])
@pytest.mark.parametrize("window,sinks", [(0, 9), (1, 0), (1, 1), (7, 4), (33, 64), (64, 31), (100, 1), (1000, 16), (48, 1000),
                                          (2 ** 31 - 1, 3), (20, 2 ** 31 - 1)])
def test_masks(kv, bs, window, sinks):
    x = Inputs(2, [0, 3, 31, 64, 65, 200, 413], [1] * 7, bs=bs, window=window, sinks=sinks)
    verify(x, *decode(kv, x))


@pytest.mark.parametrize("cache,dtype", [("same", BF16), ("same", F16), ("e4m3", BF16), ("e4m3", F16), ("int4", BF16), ("int4", F16)])
@pytest.mark.parametrize("q_len,Hq", [(1, 8), (2, 8), (5, 8), (8, 16), (4, 2), (3, 12)])
def test_types_and_drafted_tokens(kv, cache, dtype, q_len, Hq):
    x = Inputs(3, [0, 7, 30, 61, 90, 300, 331], [q_len] * 7, Hq, 2, window=37, sinks=6, cache=cache, dtype=dtype)
    verify(x, *decode(kv, x))


@pytest.mark.parametrize("cache", ["same", "e4m3", "int4"])
@pytest.mark.parametrize("workers", [1, 7, 152, 1000])
def test_shares(kv, cache, workers):
    """One sequence in up to as many shares as it has stages, and many in one."""
    x = Inputs(4, [3000, 0, 900], [3] * 3, window=700, sinks=33, cache=cache)
    verify(x, *decode(kv, x, num_workers=workers))


@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("group", [8, 16, 64, 128])
def test_int4_groups(kv, bs, group):
    x = Inputs(5, [0, 100, 1000], [2] * 3, bs=bs, window=130, sinks=20, cache="int4", group=group)
    verify(x, *decode(kv, x))


def test_many_sequences(kv):
    """More lengths than the kernel keeps beside its ring, each in the same small cache."""
    rng = np.random.default_rng(6)
    x = Inputs(6, rng.integers(0, 60, 4000), np.full(4000, 1), 4, 2, window=16, sinks=4)
    verify(x, *decode(kv, x))


@pytest.mark.parametrize("cache", ["same", "e4m3", "int4"])
def test_sinks_zero_is_the_window(kv, cache):
    """Without sinks the call agrees with the windowed decode."""
    x = Inputs(7, [5, 100, 999], [2] * 3, window=80, sinks=0, cache=cache)
    d = x.device()
    out, lse, err = decode(kv, x, d)
    head = (d["q"], d["k_cache"], d["v_cache"], d["table"], d["lens"], int(x.lens.max()), 2, x.scale)
    if cache == "int4":
        other = kv.paged_attention_decode_int4(*head, d["k_scales"], d["v_scales"], window=80)
    else:
        other = kv.paged_attention_decode(*head, window=80, k_scale=x.k_scale, v_scale=x.v_scale)
    r = x.reference()
    tol, _ = x.bounds(r, rounded_sum=True)
    check(out, other.double().cpu().numpy(), 2 * tol, "out")


@pytest.mark.parametrize("cache,dtype", [("same", BF16), ("same", F16), ("e4m3", BF16)])
@pytest.mark.parametrize("workers", [0, 50])
def test_nan_where_rows_do_not_see(kv, cache, dtype, workers):
    """Keys and values that some or all rows of a sequence do not see: the later rows' own tokens, the window's
    edge, the gap behind the sinks.  The rows that see them get NaN and infinities, the others nothing."""
    q_len, window, sinks, ctx = 5, 40, 3, 200
    x = Inputs(8, [ctx, ctx, 10, ctx, ctx], [q_len] * 5, 16, 2, window=window, sinks=sinks, cache=cache, dtype=dtype,
               release=False)
    bad = [np.nan] if cache == "e4m3" else [np.nan, np.inf, -np.inf]
    kc, vc = x.k_cache.float().numpy(), x.v_cache.float().numpy()
    for b in (0, 1):  # sequence 0: a last token's value and key; 1: the window's lower edge and the gap
        last = ctx + q_len - 1
        lo = ctx - window + 1  # the first row's first key; row i sees from lo + i on
        for i, pos in enumerate([last, last - 1] if b == 0 else [lo, lo + 1, lo + 2, lo - 1, sinks, sinks + 1]):
            vc[(*x.slot(b, pos), i % 2, 5 + i)] = bad[i % len(bad)]
            vc[(*x.slot(b, pos), 0, 77)] = bad[0]
        kc[(*x.slot(b, last if b == 0 else lo), 1, 3)] = np.nan
    vc[(*x.slot(2, 12), 0, 1)] = bad[0]   # a short sequence: a token that three rows see
    vc[(*x.slot(3, 1), 0, 9)] = bad[-1]   # a sink: every row
    vc[(*x.slot(4, 190), 1, 9)] = bad[-1]  # a key in everyone's window
    x.k_cache, x.v_cache = (torch.from_numpy(t).to(x.k_cache.dtype) for t in (kc, vc))
    out, lse, err = decode(kv, x, num_workers=workers)
    verify(x, out, lse, err)
    assert np.isnan(x.reference()["out"]).any(), "the inputs reach some rows"


@pytest.mark.parametrize("cache,dtype", [("same", F16), ("same", BF16), ("e4m3", BF16), ("int4", BF16)])
def test_weights_beside_a_sink(kv, cache, dtype):
    """A sink whose score is far above the others' and whose value is zero: what the result is then made of are
    weights of about 2^-17 to 2^-27 of the largest."""
    x = Inputs(9, [4000], [1], 4, 1, window=3500, sinks=1, cache=cache, dtype=dtype)
    x.q = torch.ones_like(x.q)
    if cache == "int4":
        x.k_scales[:], x.v_scales[:] = 1.0, 1.0
        x.k_cache[:] = 0x00
        x.v_cache[:] = 0x33
        blk, off = x.slot(0, 0)
        x.k_cache[blk, off], x.v_cache[blk, off] = 0x11, 0x00
        x.scale = 16.0 / 128
    else:
        x.k_cache, x.v_cache = torch.zeros_like(x.k_cache), torch.full(x.v_cache.shape, 3.0).to(x.v_cache.dtype)
        blk, off = x.slot(0, 0)
        x.k_cache[blk, off] = torch.ones(128).to(x.k_cache.dtype)
        x.v_cache[blk, off] = torch.zeros(128).to(x.v_cache.dtype)
        x.scale = 16.0 / 128 / x.k_scale
    out, lse, err = decode(kv, x)
    want = x.reference()["out"]
    assert err == 0
    # one rounding of each weight and of the result, whose terms are all of one sign; the INT4 codes' offset
    # of 8 is taken out in float32, 8 * 2^-21 of the sink's weight of 1
    u = 2.0 ** -8 if dtype is BF16 else 2.0 ** -11
    tol = (2 * u + 2.0 ** -11) * np.abs(want) + (8 * 2.0 ** -20 if cache == "int4" else 0)
    check(out, want, tol, "out")


def test_rejected_lengths_and_blocks(kv):
    x = Inputs(10, [30, 500, 80, 90], [2] * 4, window=48, sinks=4)
    d = x.device()
    # a length below its rows, one past max_seq_len
    lens = d["lens"].clone()
    lens[0], lens[2] = 1, 400
    out, lse, err = decode(kv, x, {**d, "lens": lens}, max_seq_len=399)
    assert err == kv.KV_DERR_BAD_LEN
    r = x.reference()
    tol, _ = x.bounds(r)
    for b in (0, 1, 2):
        rows = slice(2 * b, 2 * b + 2)
        assert (out[rows] == 0).all() and torch.isneginf(lse[rows]).all()
    check(out[6:], r["out"][6:], tol[6:], "the other sequence")
    # bad ids: of the sinks' block and of one in the window; keys behind them are seen by no row
    for bad in (-1, x.NB):
        table = x.table.copy()
        table[1, 0], table[3, 5] = bad, bad
        out, lse, err = decode(kv, x, {**d, "table": torch.from_numpy(table).cuda()})
        assert err == kv.KV_DERR_BAD_BLOCK
        y = Inputs(10, [30, 500, 80, 90], [2] * 4, window=48, sinks=4)
        y.table = np.where(table == x.NB, -1, table)
        verify(y, out, lse)


def test_every_block_bad(kv):
    """Rows that see no key at all."""
    x = Inputs(11, [100, 40], [1] * 2, window=20, sinks=2)
    d = x.device()
    table = torch.full_like(d["table"], -1)
    for workers in (0, 1):
        out, lse, err = decode(kv, x, {**d, "table": table}, num_workers=workers)
        assert err == kv.KV_DERR_BAD_BLOCK and (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("cache", ["same", "int4"])
def test_graphs_share_a_workspace_and_streams(kv, cache):
    x = Inputs(12, [900, 30, 2000], [1] * 3, window=500, sinks=4, cache=cache)
    y = Inputs(13, [70, 1500, 333], [1] * 3, window=500, sinks=4, cache=cache)
    both = [(z, z.device()) for z in (x, y)]
    code = kv.KV_INT4 if cache == "int4" else kv.KV_BF16
    ws = torch.empty(kv.paged_attention_workspace_size(3, 1, 8, 2, 128, 16, code, 4096, 500), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    side = torch.cuda.Stream()

    def call(z, d, out, stream=None):
        head = (d["q"], d["k_cache"], d["v_cache"], d["table"], d["lens"], 4096, 1, z.scale)
        kw = dict(workspace=ws, out=out, stream=stream)
        if cache == "int4":
            kv.paged_attention_decode_sinks_int4(*head, d["k_scales"], d["v_scales"], 500, 4, **kw)
        else:
            kv.paged_attention_decode_sinks(*head, 500, 4, **kw)

    for z, d in both:
        out = torch.empty_like(d["q"])
        side.wait_stream(torch.cuda.current_stream())
        call(z, d, out, stream=side)  # warm-up, on a stream that is not the current one
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
            check(out, r["out"], z.bounds(r, rounded_sum=True)[0], "out")


def test_caches_past_32_bits(kv):
    """Blocks whose elements lie past 2^31: the value of a partly seen key among them is fetched again."""
    x = Inputs(14, [60, 40], [3] * 2, 8, 8, window=24, sinks=2, spare=0)
    NB = (2 ** 31) // (16 * 8 * 128) + 500
    d = x.device()
    x.v_cache[(*x.slot(0, 62), 1, 5)] = np.inf
    big = []
    for t in (x.k_cache, x.v_cache):
        c = torch.empty((NB, 16, 8, 128), dtype=BF16, device="cuda")
        c[NB - x.NB:] = t.cuda()
        big.append(c)
    d |= dict(k_cache=big[0], v_cache=big[1], table=torch.where(d["table"] >= 0, d["table"] + (NB - x.NB), -1))
    verify(x, *decode(kv, x, d))


def test_block_manager_and_a_step(kv):
    """Sequences grow by drafted steps over a manager whose window keeps the sinks: metadata, cache write and
    attention of every step, with the blocks that the manager has released given to others."""
    bs, window, sinks, Hq, Hkv, D, B, W = 8, 20, 5, 8, 2, 128, 3, 40
    bm = kv.BlockManager(3 * 6 + 1, bs, B, W, window=window, zero_fill=False, num_sinks=sinks)
    table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    caches = [torch.zeros((bm.num_blocks, bs, Hkv, D), dtype=BF16, device="cuda") for _ in range(2)]
    rng = np.random.default_rng(15)
    held = [[np.zeros((0, Hkv, D)) for _ in range(2)] for _ in range(B)]  # every sequence's K and V
    lens = np.zeros(B, np.int64)
    for step, n in enumerate([4, 8, 8, 8, 3, 1, 8, 8, 8, 8, 8, 1, 8, 8, 8, 8]):
        assert (bm.allocate_batch(np.arange(B), np.full(B, n)) == 0).all()
        ups, zero = bm.flush()
        kv.apply_block_updates(torch.from_numpy(ups.copy()).cuda(), table, torch.from_numpy(zero.copy()).cuda(), caches,
                               bm.num_blocks)
        rows = [torch.from_numpy(rng.standard_normal((B * n, h, D))).to(BF16) for h in (Hq, Hkv, Hkv)]
        q, k, v = (t.cuda() for t in rows)
        qsl = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
        pos = torch.from_numpy((lens[:, None] + np.arange(n)).reshape(-1).astype(np.int32)).cuda()
        lens += n
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        slots = kv.compute_slot_mapping(table, qsl, pos, bs, bm.num_blocks, d_err=err)
        kv.reshape_and_cache(k, v, slots, *caches, d_err=err)
        out = kv.paged_attention_decode_sinks(q, *caches, table, torch.from_numpy(lens.astype(np.int32)).cuda(), 400, n,
                                              D ** -0.5, window, sinks, d_err=err)
        assert int(err) == 0
        for b in range(B):
            for i in range(2):
                held[b][i] = np.concatenate([held[b][i], rows[1 + i][b * n:(b + 1) * n].double().numpy()])
            # the sequence in blocks of its own, nothing released
            x = Inputs(0, [lens[b] - n], [n], Hq, Hkv, D, bs, window, sinks, release=False, spare=0)
            x.q = rows[0][b * n:(b + 1) * n]
            order = x.table[0, :x.NB]
            for i, name in enumerate(("k_cache", "v_cache")):
                flat = np.zeros((x.NB * bs, Hkv, D))
                flat[:lens[b]] = held[b][i]
                c = np.empty((x.NB, bs, Hkv, D))
                c[order] = flat.reshape(x.NB, bs, Hkv, D)
                setattr(x, name, torch.from_numpy(c).to(BF16))
            r = x.reference()
            check(out[b * n:(b + 1) * n], r["out"], x.bounds(r)[0], f"step {step}, sequence {b}")
