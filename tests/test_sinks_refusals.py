"""Host-side refusals of the calls with sinks and of the INT4 append (kv_paged_attention_decode_sinks,
kv_paged_attention_prefill_sinks, both with _int4, kv_qk_norm_rope_int4), and the block manager whose windows keep
sinks: none of it needs a GPU.  Pointers are made-up aligned numbers: a refused call never looks at them."""
import numpy as np
import pytest
import torch

from tests.test_step_refusals import call, kc  # noqa: F401  (the library's fixture)

OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = range(5)
P = 1 << 20  # a made-up pointer; its neighbours are 1 MiB apart

DECODE = dict(q=P, q_dtype=1, num_seqs=2, q_len=4, q_heads=4, k_cache=3 * P, v_cache=4 * P, cache_dtype=1, kv_heads=1,
              head_dim=128, block_size=16, num_blocks=8, block_table=5 * P, bt_stride=8, max_blocks=8, seq_lens=6 * P,
              max_seq_len=100, scale=0.1, window=32, num_sinks=4, k_scale=1.0, v_scale=1.0, num_workers=0, workspace=None,
              workspace_bytes=0, out=8 * P, lse_out=None, d_err=None, stream=None)
DECODE4 = {}
for k_, v_ in DECODE.items():
    if k_ == "k_scale":
        DECODE4 |= dict(k_scales=9 * P, v_scales=10 * P, group_size=32)
    elif k_ not in ("v_scale", "cache_dtype"):
        DECODE4[k_] = v_
PREFILL = dict(q=P, q_dtype=1, query_start_loc=2 * P, num_seqs=2, num_tokens=8, max_query_len=4, q_heads=4, k_cache=3 * P,
               v_cache=4 * P, cache_dtype=1, kv_heads=1, head_dim=128, block_size=16, num_blocks=8, block_table=5 * P,
               bt_stride=8, max_blocks=8, seq_lens=6 * P, max_seq_len=100, scale=0.1, window=32, num_sinks=4, k_scale=1.0,
               v_scale=1.0, num_workers=0, workspace=None, workspace_bytes=0, out=8 * P, lse_out=None, d_err=None, stream=None)
PREFILL4 = {}
for k_, v_ in PREFILL.items():
    if k_ == "k_scale":
        PREFILL4 |= dict(k_scales=9 * P, v_scales=10 * P, group_size=32)
    elif k_ not in ("v_scale", "cache_dtype"):
        PREFILL4[k_] = v_
ROPE4 = dict(q=P, key=2 * P, value=3 * P, dtype=1, q_stride=512, key_stride=128, value_stride=128, num_tokens=4,
             q_heads=4, kv_heads=1, head_dim=128, q_weight=4 * P, k_weight=5 * P, eps=1e-6, positions=6 * P,
             cos_sin=7 * P, max_position=64, rotary_dim=128, interleaved=0, q_out=8 * P, q_out_stride=512, k_out=9 * P,
             k_out_stride=128, slot_mapping=10 * P, k_cache=11 * P, v_cache=12 * P, num_blocks=8, block_size=16,
             k_scales=13 * P, v_scales=14 * P, group_size=32, d_err=None, stream=None)

SIZES = [(dict(num_seqs=-1), INVALID), (dict(q_heads=0), INVALID), (dict(kv_heads=0), INVALID),
         (dict(q_heads=5, kv_heads=2), INVALID), (dict(window=-1), INVALID), (dict(num_sinks=-1), INVALID),
         (dict(num_workers=-1), INVALID), (dict(num_blocks=0), INVALID), (dict(bt_stride=7), INVALID),
         (dict(head_dim=96), UNSUPPORTED), (dict(q_dtype=2), UNSUPPORTED), (dict(q_dtype=3), UNSUPPORTED),
         (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=3e38), INVALID)]
POINTERS = [(dict([(k, None)]), INVALID) for k in ("q", "k_cache", "v_cache", "block_table", "seq_lens", "out")] + [
    (dict(q=P + 8), INVALID), (dict(out=8 * P + 4), INVALID), (dict(k_cache=3 * P + 8), INVALID), (dict(v_cache=4 * P + 2), INVALID),
    (dict(seq_lens=6 * P + 2), INVALID), (dict(block_table=5 * P + 1), INVALID), (dict(lse_out=9 * P + 2), INVALID),
    (dict(d_err=9 * P + 2), INVALID)]
# outputs over something: 8 tokens of 4 heads of 256 bytes; caches of 8 blocks of 4 KB (INT4: 1 KB)
OVERLAPS = [(dict(out=P), INVALID), (dict(out=P + 8176), INVALID), (dict(out=3 * P + 1024), INVALID), (dict(out=4 * P - 16), INVALID),
            (dict(lse_out=8 * P + 8188), INVALID), (dict(lse_out=6 * P), INVALID), (dict(lse_out=5 * P + 60), INVALID),
            (dict(workspace=8 * P, workspace_bytes=1 << 16), INVALID), (dict(workspace=P, workspace_bytes=1 << 16), INVALID),
            (dict(workspace=4 * P, workspace_bytes=1 << 62), INVALID)]


# (what the decode's launch plan refuses, it refuses once a device is there)
PLANNED = [dict(q_heads=5, kv_heads=2), dict(head_dim=96)]


@pytest.mark.parametrize("changes,status", [c for c in SIZES if c[0] not in PLANNED] + POINTERS + OVERLAPS + [
    (dict(q_len=0), INVALID), (dict(max_seq_len=0), INVALID), (dict(cache_dtype=0), UNSUPPORTED), (dict(cache_dtype=3), UNSUPPORTED),
    (dict(cache_dtype=2, k_scale=0.0), INVALID), (dict(cache_dtype=2, v_scale=float("inf")), INVALID)])
def test_decode_refuses(kc, changes, status):  # noqa: F811
    assert call(kc, "kv_paged_attention_decode_sinks", DECODE, **changes) == status
    assert kc.lib.kv_last_error()


@pytest.mark.parametrize("changes,status", [c for c in SIZES if c[0] != PLANNED[0]] + POINTERS + OVERLAPS + [
    (dict(group_size=4), UNSUPPORTED), (dict(group_size=24), UNSUPPORTED), (dict(group_size=256), UNSUPPORTED),
    (dict(head_dim=64), UNSUPPORTED), (dict(k_scales=None), INVALID), (dict(v_scales=10 * P + 2), INVALID),
    (dict(out=9 * P), INVALID), (dict(lse_out=10 * P + 12), INVALID)])
def test_decode_int4_refuses(kc, changes, status):  # noqa: F811
    assert call(kc, "kv_paged_attention_decode_sinks_int4", DECODE4, **changes) == status
    assert kc.lib.kv_last_error()


MORE = [(dict(num_tokens=-1), INVALID), (dict(max_query_len=-1), INVALID), (dict(max_seq_len=-1), INVALID),
        (dict(q_heads=129), UNSUPPORTED), (dict(block_size=4), UNSUPPORTED), (dict(block_size=64), UNSUPPORTED),
        (dict(num_workers=32768), UNSUPPORTED), (dict(scale=-0.1), INVALID), (dict(query_start_loc=None), INVALID),
        (dict(query_start_loc=2 * P + 2), INVALID), (dict(out=2 * P), INVALID)]


@pytest.mark.parametrize("changes,status", SIZES + POINTERS + OVERLAPS + MORE + [
    (dict(cache_dtype=0), UNSUPPORTED), (dict(cache_dtype=3), UNSUPPORTED), (dict(cache_dtype=2, head_dim=64), UNSUPPORTED),
    (dict(cache_dtype=2, k_scale=0.0), INVALID), (dict(cache_dtype=2, v_scale=float("nan")), INVALID)])
def test_prefill_refuses(kc, changes, status):  # noqa: F811
    assert call(kc, "kv_paged_attention_prefill_sinks", PREFILL, **changes) == status
    assert kc.lib.kv_last_error()


@pytest.mark.parametrize("changes,status", SIZES + POINTERS + OVERLAPS + MORE + [
    (dict(group_size=4), UNSUPPORTED), (dict(group_size=24), UNSUPPORTED), (dict(head_dim=64), UNSUPPORTED),
    (dict(k_scales=None), INVALID), (dict(v_scales=10 * P + 2), INVALID), (dict(out=9 * P), INVALID)])
def test_prefill_int4_refuses(kc, changes, status):  # noqa: F811
    assert call(kc, "kv_paged_attention_prefill_sinks_int4", PREFILL4, **changes) == status
    assert kc.lib.kv_last_error()


@pytest.mark.parametrize("changes,status", [
    (dict(num_tokens=-1), INVALID), (dict(head_dim=64), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED), (dict(group_size=4), UNSUPPORTED),
    (dict(group_size=48), UNSUPPORTED), (dict(rotary_dim=24), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
    (dict(eps=-1.0), INVALID), (dict(slot_mapping=None), INVALID), (dict(slot_mapping=None, k_cache=None, v_cache=None), INVALID),
    (dict(value=None), INVALID), (dict(k_cache=None), INVALID), (dict(k_scales=None), INVALID), (dict(v_scales=None), INVALID),
    (dict(k_scales=13 * P + 2), INVALID), (dict(q_stride=504), INVALID), (dict(block_size=0), INVALID), (dict(v_cache=12 * P + 8), INVALID),
    # outputs over something: scales of 16 bytes, caches of 8 blocks of 1 KB
    (dict(q_out=13 * P), INVALID), (dict(k_out=14 * P), INVALID), (dict(k_cache=13 * P - 8192 + 16), INVALID), (dict(v_cache=14 * P), INVALID),
    (dict(k_cache=12 * P - 8176), INVALID), (dict(q_out=11 * P + 8176), INVALID), (dict(q_out=2 * P), INVALID),
    (dict(k_cache=10 * P), INVALID)])
def test_append_refuses(kc, changes, status):  # noqa: F811
    assert call(kc, "kv_qk_norm_rope_int4", ROPE4, **changes) == status
    assert kc.lib.kv_last_error()


def test_neighbours_are_no_overlap(kc):  # noqa: F811
    """Buffers that touch: such calls pass every check up to the device's, which needs a machine without one (the
    pointers are made up)."""
    if torch.cuda.is_available():
        pytest.skip("made-up pointers stay off a device")
    assert call(kc, "kv_paged_attention_decode_sinks", DECODE, out=P + 8192, lse_out=P + 16384) == CUDA
    assert call(kc, "kv_paged_attention_decode_sinks_int4", DECODE4, out=3 * P + 8192) == CUDA
    assert call(kc, "kv_paged_attention_prefill_sinks", PREFILL, out=P + 8192, lse_out=P + 16384) == CUDA
    assert call(kc, "kv_paged_attention_prefill_sinks_int4", PREFILL4, out=3 * P + 8192) == CUDA
    assert call(kc, "kv_qk_norm_rope_int4", ROPE4, q_out=11 * P + 8192, k_scales=14 * P + 16) == CUDA


def test_nothing_to_do_needs_no_device(kc):  # noqa: F811
    assert call(kc, "kv_paged_attention_decode_sinks", DECODE, num_seqs=0, q=None) == OK
    assert call(kc, "kv_paged_attention_decode_sinks_int4", DECODE4, num_seqs=0, q=None) == OK
    for zero in (dict(num_seqs=0), dict(num_tokens=0), dict(max_query_len=0)):
        assert call(kc, "kv_paged_attention_prefill_sinks", PREFILL, **zero, q=None) == OK
        assert call(kc, "kv_paged_attention_prefill_sinks_int4", PREFILL4, **zero, q=None) == OK
    assert call(kc, "kv_qk_norm_rope_int4", ROPE4, num_tokens=0, q=None) == OK


def test_workspace_refusals(kc):  # noqa: F811
    for bad in ((-1, 4, 8, 2, 128, 1, 100), (1, -1, 8, 2, 128, 1, 100), (1, 4, 9, 2, 128, 1, 100), (1, 4, 8, 2, 80, 1, 100),
                (1, 4, 8, 2, 64, 3, 100), (1, 4, 8, 2, 64, 2, 100), (1, 4, 8, 2, 128, 1, 100, -1), (1, 4, 8, 2, 128, 1, 100, 0, -1),
                (1, 4, 8, 2, 128, 1, 100, 0, 0, -1)):
        with pytest.raises(kc.KVError):
            kc.paged_attention_prefill_sinks_workspace_size(*bad)


def test_binding_refuses_host_tensors_and_wrong_shapes(kc):  # noqa: F811
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    x = torch.zeros(3, 4, 128, dtype=torch.float16)
    c, c4 = torch.zeros(4, 16, 2, 128, dtype=torch.float16), torch.zeros(4, 16, 2, 64, dtype=torch.uint8)
    s = torch.ones(2, 4)
    with pytest.raises(kc.KVError, match="one CUDA device"):
        kc.paged_attention_decode_sinks(x, c, c, i32(3, 4), i32(3), 64, 1, 0.1, 16, 4)
    with pytest.raises(kc.KVError, match="one CUDA device"):
        kc.paged_attention_decode_sinks_int4(x, c4, c4, i32(3, 4), i32(3), 64, 1, 0.1, s, s, 16, 4)
    with pytest.raises(kc.KVError, match="scales are needed"):
        kc.paged_attention_decode_sinks_int4(x, c4, c4, i32(3, 4), i32(3), 64, 1, 0.1, None, s, 16, 4)
    with pytest.raises(kc.KVError, match="one CUDA device"):
        kc.paged_attention_prefill_sinks(x, c, c, i32(1, 4), i32(1), i32(2), 64, 3, 0.1, 16, 4)
    with pytest.raises(kc.KVError, match="scales are needed"):
        kc.paged_attention_prefill_sinks_int4(x, c4, c4, i32(1, 4), i32(1), i32(2), 64, 3, 0.1, s, None)
    with pytest.raises(kc.KVError, match="one CUDA device"):
        kc.qk_norm_rope_and_cache_int4(x, x[:, :2], x[:, :2], i32(3), torch.zeros(8, 128), torch.zeros(3, dtype=torch.int64), c4, c4, s, s)
    with pytest.raises(kc.KVError, match="scales are needed"):
        kc.qk_norm_rope_and_cache_int4(x, x[:, :2], x[:, :2], i32(3), torch.zeros(8, 128), torch.zeros(3, dtype=torch.int64), c4, c4, s, None)


# ---------------------------------------------------------------- the block manager

class Rows:
    """What a manager with sinks should hold, position by position."""

    def __init__(self, bs, window, sinks):
        self.bs, self.window, self.sinks, self.tokens, self.live = bs, window, sinks, 0, []

    def allocate(self, n):
        keep = -(-self.sinks // self.bs)
        for j in range(len(self.live)):
            if j >= keep and self.window and (j + 1) * self.bs - 1 <= self.tokens - self.window:
                self.live[j] = False
        self.tokens += n
        self.live += [True] * (-(-self.tokens // self.bs) - len(self.live))


@pytest.mark.parametrize("bs", [1, 4, 16])
@pytest.mark.parametrize("window,sinks", [(0, 5), (1, 0), (7, 0), (7, 1), (20, 4), (20, 33), (64, 16), (5, 10 ** 6)])
def test_manager_keeps_the_sinks(kc, bs, window, sinks):  # noqa: F811
    rng = np.random.default_rng(bs * 100 + window)
    bm = kc.BlockManager(4000, bs, 3, 1200, window=window, num_sinks=sinks)
    rows = [Rows(bs, window, sinks) for _ in range(3)]
    table = np.full((3, 1200), -7, np.int64)
    for _ in range(60):
        r, n = int(rng.integers(3)), int(rng.integers(0, 20))
        if rng.random() < 0.05:
            assert bm.free(r) == 0
            rows[r] = Rows(bs, window, sinks)
        else:
            assert bm.allocate(r, n) == 0
            rows[r].allocate(n)
        ups, _ = bm.flush()
        table[ups[:, 0], ups[:, 1]] = ups[:, 2]
        held = []
        for i, row in enumerate(rows):
            tokens, blocks = bm.row(i)
            assert tokens == row.tokens and [b >= 0 for b in blocks] == row.live
            assert table[i, :len(blocks)].tolist() == blocks
            held += [b for b in blocks if b >= 0]
        assert len(set(held)) == len(held) and bm.num_free_blocks() == 4000 - len(held)
        assert all(bm.ref_count(b) == 1 for b in held)
    for r in range(3):
        assert bm.free(r) == 0
    assert bm.num_free_blocks() == 4000


def test_manager_shares_sinks_after_the_window_has_moved(kc):  # noqa: F811
    bm = kc.BlockManager(64, 4, 3, 40, window=8, num_sinks=6)
    for _ in range(10):
        assert bm.allocate(0, 6) == 0
    blocks = bm.row(0)[1]
    assert blocks[0] >= 0 and blocks[1] >= 0 and blocks[2] == -1
    assert bm.share_prefix(1, 0, 3) == 1 and bm.share_prefix(1, 0, 2) == 0
    assert bm.row(1) == (8, blocks[:2]) and bm.ref_count(blocks[0]) == 2
    assert bm.free(0) == 0 and bm.ref_count(blocks[0]) == 1
    assert bm.allocate(1, 30) == 0 and bm.allocate(1, 4) == 0
    kept = bm.row(1)[1]
    assert kept[:2] == blocks[:2] and kept[2] == -1
    assert bm.free(1) == 0 and bm.num_free_blocks() == 64


def test_manager_refuses_negative_sinks(kc):  # noqa: F811
    with pytest.raises(kc.KVError):
        kc.BlockManager(64, 4, 3, 40, window=8, num_sinks=-1)


@pytest.mark.parametrize("dtype", [-1, 4, 5, 17, 2 ** 31 - 1])
@pytest.mark.parametrize("head_dim", [64, 128])
def test_workspace_of_no_cache_type(kc, dtype, head_dim):  # noqa: F811
    with pytest.raises(kc.KVError, match="cache dtype"):
        kc.paged_attention_prefill_sinks_workspace_size(1, 4, 8, 2, head_dim, dtype, 100)
    assert call(kc, "kv_paged_attention_prefill_sinks", PREFILL, cache_dtype=dtype, head_dim=head_dim) == UNSUPPORTED
