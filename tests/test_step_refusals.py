"""Host-side refusals of the step's calls (kv_build_batch, kv_qk_norm_rope,
kv_paged_attention_tree): every one answers before any device is touched, so these run without a
GPU.  Pointers are made-up aligned numbers: a refused call never looks at them."""
import ctypes

import pytest
import torch

OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = range(5)
P = 1 << 20  # a made-up pointer; its neighbours are 1 MiB apart


@pytest.fixture(scope="module")
def kc():
    from paged_kv_cache_block_gb300 import build
    build.build()
    from paged_kv_cache_block_gb300 import kvcache
    return kvcache


BATCH = dict(context_lens=P, new_lens=2 * P, held_blocks=3 * P, parents=None, num_seqs=4, num_tokens=16,
             block_table=4 * P, bt_stride=8, max_blocks=8, block_size=16, num_blocks=64, free_blocks=5 * P, num_free=9,
             free_start=None, query_start_loc=6 * P, seq_lens=7 * P, positions=8 * P, slot_mapping=9 * P,
             tree_mask=None, held_out=10 * P, free_next=11 * P, d_err=None, stream=None)
ROPE = dict(q=P, key=2 * P, value=3 * P, dtype=1, q_stride=512, key_stride=128, value_stride=128, num_tokens=4,
            q_heads=4, kv_heads=1, head_dim=128, q_weight=4 * P, k_weight=5 * P, eps=1e-6, positions=6 * P,
            cos_sin=7 * P, max_position=64, rotary_dim=128, interleaved=0, q_out=8 * P, q_out_stride=512, k_out=9 * P,
            k_out_stride=128, slot_mapping=10 * P, k_cache=11 * P, v_cache=12 * P, cache_dtype=1, num_blocks=8,
            block_size=16, k_scale=1.0, v_scale=1.0, d_err=None, stream=None)
TREE = dict(q=P, q_dtype=1, query_start_loc=2 * P, num_seqs=2, num_tokens=8, max_query_len=4, q_heads=4, k_cache=3 * P,
            v_cache=4 * P, cache_dtype=1, kv_heads=1, head_dim=128, block_size=16, num_blocks=8, block_table=5 * P,
            bt_stride=8, max_blocks=8, seq_lens=6 * P, max_seq_len=100, scale=0.1, window=0, tree_mask=7 * P,
            num_workers=0, workspace=None, workspace_bytes=0, out=8 * P, lse_out=None, d_err=None, stream=None)


def call(kc, fn, base, **changes):
    assert set(changes) <= set(base)
    return getattr(kc.lib, fn)(*{**base, **changes}.values())


@pytest.mark.parametrize("changes,status", [
    (dict(num_seqs=-1), INVALID), (dict(num_tokens=-1), INVALID), (dict(num_free=-2), INVALID),
    (dict(bt_stride=7), INVALID), (dict(block_size=12), UNSUPPORTED), (dict(block_size=64), UNSUPPORTED),
    (dict(max_blocks=1 << 30, bt_stride=1 << 30), UNSUPPORTED),
    (dict(context_lens=None), INVALID), (dict(new_lens=None), INVALID), (dict(block_table=None), INVALID),
    (dict(free_blocks=None), INVALID), (dict(query_start_loc=None), INVALID), (dict(positions=None), INVALID),
    (dict(slot_mapping=None), INVALID), (dict(held_out=None), INVALID), (dict(free_next=None), INVALID),
    (dict(seq_lens=None), INVALID),
    (dict(parents=12 * P), INVALID), (dict(tree_mask=12 * P), INVALID),          # one without the other
    (dict(parents=12 * P, tree_mask=12 * P), INVALID),                           # masks over the parents
    (dict(positions=8 * P + 2), INVALID), (dict(slot_mapping=9 * P + 4), INVALID),
    (dict(held_out=3 * P), INVALID),                                             # held blocks in place
    (dict(seq_lens=P), INVALID), (dict(seq_lens=P + 12), INVALID),               # lengths in place, or the last one
    (dict(free_start=11 * P), INVALID),                                          # the list's start in place
    (dict(query_start_loc=7 * P - 16), INVALID),                                 # two outputs: five words, then lens
    (dict(slot_mapping=8 * P), INVALID), (dict(free_next=4 * P + 4 * 31), INVALID),
    (dict(free_next=5 * P), INVALID), (dict(num_seqs=(1 << 24) + 1), UNSUPPORTED),
])
def test_build_batch_refuses(kc, changes, status):
    assert call(kc, "kv_build_batch", BATCH, **changes) == status
    assert kc.lib.kv_last_error()


@pytest.mark.parametrize("changes,status", [
    (dict(num_tokens=-1), INVALID), (dict(q_heads=0), INVALID), (dict(kv_heads=0), INVALID),
    (dict(head_dim=0), INVALID), (dict(head_dim=100), UNSUPPORTED), (dict(head_dim=264), UNSUPPORTED),
    (dict(rotary_dim=-16), INVALID), (dict(rotary_dim=24), UNSUPPORTED), (dict(rotary_dim=144), UNSUPPORTED),
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(cache_dtype=0), UNSUPPORTED),
    (dict(cache_dtype=3), UNSUPPORTED), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(q=None), INVALID), (dict(key=None), INVALID), (dict(q_out=None), INVALID),
    (dict(value=None), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID),
    (dict(slot_mapping=None), INVALID),                                          # caches without slots
    (dict(slot_mapping=None, k_cache=None, v_cache=None, k_out=None), INVALID),  # the keys go nowhere
    (dict(positions=None), INVALID), (dict(cos_sin=None), INVALID),
    (dict(q_stride=504), INVALID), (dict(q_stride=516), INVALID), (dict(key_stride=120), INVALID),
    (dict(value_stride=0), INVALID), (dict(k_out_stride=132), INVALID), (dict(q_out_stride=0), INVALID),
    (dict(q=P + 8), INVALID), (dict(k_weight=5 * P + 2), INVALID), (dict(cos_sin=7 * P + 4), INVALID),
    (dict(v_cache=12 * P + 8), INVALID), (dict(positions=6 * P + 1), INVALID),
    (dict(q_out=P, q_out_stride=1024), INVALID),                                 # in place, another stride
    (dict(cache_dtype=2, k_scale=0.0), INVALID), (dict(cache_dtype=2, v_scale=float("nan")), INVALID),
    (dict(block_size=0), INVALID), (dict(num_blocks=-1), INVALID),
    (dict(q_heads=65536, q_stride=1 << 23, q_out_stride=1 << 23), UNSUPPORTED), (dict(kv_heads=1 << 20), UNSUPPORTED),
    # outputs over something: 4 tokens, 4 query heads and one key head of 256 bytes
    (dict(q_out=2 * P), INVALID), (dict(k_out=3 * P), INVALID), (dict(q_out=P + 1024), INVALID),
    (dict(q_out=P - 16), INVALID), (dict(k_out=8 * P + 16), INVALID), (dict(k_out=2 * P + 16), INVALID),
    (dict(q_out=P, q_stride=512, key=P + 512, key_stride=512), INVALID),
    (dict(k_out=P + 1008, key=P + 1024, q_stride=640, key_stride=640, k_out_stride=640), INVALID),
    (dict(q_out=4 * P - 3840), INVALID), (dict(k_out=5 * P), INVALID), (dict(k_out=6 * P - 256), INVALID),
    (dict(q_out=7 * P), INVALID), (dict(k_out=10 * P + 16), INVALID),
    (dict(k_cache=12 * P), INVALID), (dict(k_cache=12 * P - 32752), INVALID), (dict(v_cache=3 * P - 16), INVALID),
    (dict(v_cache=8 * P), INVALID), (dict(k_cache=7 * P), INVALID), (dict(k_cache=10 * P), INVALID),
])
def test_qk_norm_rope_refuses(kc, changes, status):
    assert call(kc, "kv_qk_norm_rope", ROPE, **changes) == status
    assert kc.lib.kv_last_error()


@pytest.mark.parametrize("changes,status", [
    (dict(num_seqs=-1), INVALID), (dict(num_tokens=-1), INVALID), (dict(max_query_len=-1), INVALID),
    (dict(max_query_len=65), UNSUPPORTED), (dict(q_heads=0), INVALID), (dict(q_heads=5, kv_heads=2), INVALID),
    (dict(q_heads=129), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED),
    (dict(block_size=4), UNSUPPORTED), (dict(block_size=64), UNSUPPORTED), (dict(block_size=0), UNSUPPORTED),
    (dict(window=-1), INVALID), (dict(window=63), UNSUPPORTED), (dict(window=1), UNSUPPORTED),
    (dict(q_dtype=2), UNSUPPORTED), (dict(cache_dtype=0), UNSUPPORTED), (dict(cache_dtype=2), UNSUPPORTED),
    (dict(cache_dtype=3), UNSUPPORTED), (dict(num_blocks=0), INVALID), (dict(bt_stride=7), INVALID),
    (dict(scale=-0.1), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(num_workers=-1), INVALID), (dict(max_seq_len=-1), INVALID),
    (dict(q=None), INVALID), (dict(tree_mask=None), INVALID), (dict(query_start_loc=None), INVALID),
    (dict(block_table=None), INVALID), (dict(seq_lens=None), INVALID), (dict(out=None), INVALID),
    (dict(k_cache=None), INVALID), (dict(q=P + 8), INVALID), (dict(out=8 * P + 4), INVALID),
    (dict(tree_mask=7 * P + 4), INVALID), (dict(seq_lens=6 * P + 2), INVALID), (dict(lse_out=9 * P + 2), INVALID),
    (dict(scale=3e38), INVALID),
    (dict(out=P), INVALID), (dict(out=P + 8176), INVALID), (dict(out=7 * P), INVALID), (dict(out=3 * P), INVALID),
    (dict(lse_out=8 * P + 8188), INVALID), (dict(lse_out=6 * P), INVALID), (dict(lse_out=5 * P + 60), INVALID),
    (dict(workspace=8 * P, workspace_bytes=1 << 16), INVALID), (dict(workspace=P, workspace_bytes=1 << 16), INVALID),
    (dict(workspace=2 * P - 256, workspace_bytes=1 << 16), INVALID), (dict(workspace=4 * P, workspace_bytes=1 << 62), INVALID),
])
def test_tree_attention_refuses(kc, changes, status):
    assert call(kc, "kv_paged_attention_tree", TREE, **changes) == status
    assert kc.lib.kv_last_error()


def test_views_of_one_projection_are_not_an_overlap(kc):
    """Rows of one stride may lie between each other: such calls pass every check up to the device's, which
    needs a machine without one (the pointers are made up)."""
    if torch.cuda.is_available():
        pytest.skip("made-up pointers stay off a device")
    qkv = dict(q=P, key=P + 1024, value=P + 1280, q_stride=768, key_stride=768, value_stride=768)
    for out in (dict(), dict(q_out=P, q_out_stride=768), dict(k_out=P + 1024, k_out_stride=768),
                dict(q_out=P, q_out_stride=768, k_out=P + 1024, k_out_stride=768),
                dict(q_out=8 * P, k_out=8 * P + 1024, q_out_stride=640, k_out_stride=640)):
        assert call(kc, "kv_qk_norm_rope", ROPE, **qkv, **out) == CUDA
    assert call(kc, "kv_qk_norm_rope", ROPE, **qkv, q_out=P + 16, q_out_stride=768) == INVALID


def test_batch_buffers_follow_their_memory(kc):
    import copy
    a = kc.batch_buffers(5, 21, True, device="cpu")
    for b in (a, copy.deepcopy(a), copy.copy(a)):
        got = b._place(b._base.data_ptr())
        views = (b.query_start_loc, b.seq_lens, b.positions, b.slot_mapping, b.held_blocks, b.free_next, b.tree_mask)
        assert got == tuple(v.data_ptr() for v in views)
        assert [v.numel() for v in views] == [6, 5, 21, 21, 5, 1, 21]
        assert [v.dtype for v in views] == [torch.int32] * 3 + [torch.int64] + [torch.int32] * 2 + [torch.int64]
        assert all(v.data_ptr() % 16 == 0 for v in views)
        ends = sorted((v.data_ptr(), v.data_ptr() + v.numel() * v.element_size()) for v in views)
        assert all(x[1] <= y[0] for x, y in zip(ends, ends[1:])) and ends[-1][1] <= b._base.data_ptr() + 4 * b._base.numel()
    assert copy.deepcopy(a).positions.data_ptr() != a.positions.data_ptr()
    with pytest.raises(AttributeError):
        a.positions = torch.empty(21, dtype=torch.int32)
    plain = kc.batch_buffers(0, 0, device="cpu")
    assert plain.tree_mask is None and plain._place(plain._base.data_ptr())[6] is None
    with pytest.raises(kc.KVError):
        kc.batch_buffers(2, -1, device="cpu")
    a._base.untyped_storage().resize_(0)
    with pytest.raises(kc.KVError, match="released"):
        a._place(a._base.data_ptr())


def test_nothing_to_do_needs_no_device(kc):
    assert call(kc, "kv_qk_norm_rope", ROPE, num_tokens=0, q=None, key=None) == OK
    assert call(kc, "kv_paged_attention_tree", TREE, num_seqs=0, q=None) == OK
    assert call(kc, "kv_paged_attention_tree", TREE, max_query_len=0) == OK


def test_tree_workspace_refusals(kc):
    for bad in ((-1, 4, 8, 2, 128, 0), (1, 65, 8, 2, 128, 0), (1, 4, 9, 2, 128, 0), (1, 4, 8, 2, 80, 0),
                (1, 4, 8, 2, 128, -1)):
        with pytest.raises(kc.KVError):
            kc.paged_attention_tree_workspace_size(*bad)


def test_binding_refuses_host_tensors_and_wrong_shapes(kc):
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    with pytest.raises(kc.KVError, match="one CUDA device"):
        kc.build_batch(i32(2), i32(2), i32(8).view(2, 4), i32(3), 4, 16, 8)
    x = torch.zeros(3, 4, 64, dtype=torch.float16)
    with pytest.raises(kc.KVError, match="one CUDA device"):
        kc.qk_norm_rope(x, x, i32(3), torch.zeros(8, 64))
    c = torch.zeros(4, 16, 4, 64, dtype=torch.float16)
    with pytest.raises(kc.KVError, match="one CUDA device"):
        kc.paged_attention_tree(x, c, c, i32(4).view(1, 4), i32(1), i32(2), torch.zeros(3, dtype=torch.int64), 64, 3, 0.1)
    with pytest.raises(kc.KVError):
        kc.paged_attention_tree(x.transpose(0, 1), c, c, i32(4).view(1, 4), i32(1), i32(2),
                                torch.zeros(3, dtype=torch.int64), 64, 3, 0.1)


def test_python_constants_match_the_header(kc):
    import os
    import re
    text = open(os.path.join(os.path.dirname(__file__), "..", "include", "pagedkv_step.h")).read()
    values = dict(re.findall(r"#define (KV_[A-Z_]+)\s+(\d+)", text))
    assert {k: int(v) for k, v in values.items()} == {
        k: getattr(kc, k) for k in ("KV_DERR_BAD_POS", "KV_DERR_NO_BLOCKS", "KV_DERR_BAD_TREE", "KV_MAX_TREE")}
    assert ctypes.sizeof(ctypes.c_void_p) == 8
