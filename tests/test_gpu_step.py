"""The step's operators on the GPU against plain 64-bit implementations (tests/step_reference.py):
kv_build_batch exactly, kv_qk_norm_rope and kv_paged_attention_tree within bounds worked out from
the roundings (functions norm_rope_bound and tree_bounds), at the sizes and masks where they can go
wrong; then together, captured, and on several streams."""
import numpy as np
import pytest
import torch

from . import step_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kc():
    from paged_kv_cache_block_gb300 import kvcache
    return kvcache


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ batch metadata

def run_batch(kc, ctx, new, held, table, free, T, bs, NB, parents=None, start=None, width=None, stream=None):
    i32 = lambda a: None if a is None else dev(np.asarray(a, np.int32))  # noqa: E731
    tab = i32(table)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    b = kc.build_batch(i32(ctx), i32(new), tab, i32(free), T, bs, NB, held_blocks=i32(held), parents=i32(parents),
                       free_start=None if start is None else i32([start]), d_err=err, max_blocks_per_seq=width,
                       stream=stream)
    torch.cuda.synchronize()
    got = {k: (None if v is None else v.cpu().numpy()) for k, v in b._asdict().items()}
    got["block_table"] = tab.cpu().numpy()
    return got, int(err.item())


def check_batch(kc, ctx, new, held, table, free, T, bs, NB, parents=None, start=None, width=None):
    got, err = run_batch(kc, ctx, new, held, table, free, T, bs, NB, parents, start, width)
    want, want_err = R.build_batch(ctx, new, held, table, free, T, bs, NB, parents, start or 0, width)
    for k, v in want.items():
        assert (got[k] is None) == (v is None), k
        if v is not None:
            np.testing.assert_array_equal(got[k], v, err_msg=k)
    assert err == want_err
    return got, err


def batch_case(seed, B, max_ctx, max_new, bs, extra_held=0, pad=3, trees=False, free_cut=0):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, max_ctx + 1, B)
    new = rng.integers(0, max_new + 1, B)
    held = -(-ctx // bs) + rng.integers(0, extra_held + 1, B)
    total = -(-(ctx + new) // bs)
    need = np.where(new > 0, np.maximum(total - held, 0), 0)
    width = int(max(total.max(initial=1), held.max(initial=1))) + 1
    NB = int(held.sum() + need.sum()) + 5
    ids = rng.permutation(NB).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for r in range(B):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    free = ids[at:at + max(0, int(need.sum()) + 3 - free_cut)]
    T = int(new.sum()) + pad
    parents = None
    if trees:
        parents = np.full(T, -7, np.int32)  # what stands behind the last request is not looked at
        parents[:new.sum()] = np.concatenate([R.random_parents(rng, int(n)) for n in new] + [np.zeros(0, np.int64)])
    return ctx, new, held, table, free, T, bs, NB, parents


@pytest.mark.parametrize("B", [1, 2, 31, 511, 512, 513, 1500])
@pytest.mark.parametrize("bs", [4, 16])
def test_batch_decode(kc, B, bs):
    _, err = check_batch(kc, *batch_case(B + bs, B, 300, 1, bs, pad=B % 4))
    assert err == 0


@pytest.mark.parametrize("bs", [8, 32])
@pytest.mark.parametrize("B,max_new", [(1, 64), (3, 1), (40, 64), (600, 20)])
def test_batch_trees(kc, B, max_new, bs):
    _, err = check_batch(kc, *batch_case(B * 7 + max_new, B, 200, max_new, bs, extra_held=3, trees=True))
    assert err == 0


def test_batch_long_chunks(kc):
    _, err = check_batch(kc, *batch_case(3, 37, 5000, 9000, 16, extra_held=1))
    assert err == 0


def test_batch_chain_of_64_and_star(kc):
    chain = np.arange(-1, 63)
    star = np.concatenate([[-1], np.zeros(63, np.int64)])
    forest = np.full(64, -1)
    table = np.arange(3 * 8, dtype=np.int32).reshape(3, 8)
    got, err = check_batch(kc, [10, 0, 31], [64] * 3, [8] * 3, table, [], 192, 16, 24, np.concatenate([chain, star, forest]))
    assert err == 0 and got["tree_mask"][63] == -1 and got["positions"][63] == 73 and got["positions"][64 + 63] == 1


def test_batch_without_held_counts_takes_them_from_the_context(kc):
    ctx, new, held, table, free, T, bs, NB, _ = batch_case(9, 20, 90, 40, 16)
    check_batch(kc, ctx, new, None, table, free, T, bs, NB)


def test_batch_free_list_runs_out(kc):
    for cut in (4, 11, 200):  # one block short, several, none left
        case = batch_case(11, 30, 60, 50, 8, free_cut=cut)
        got, err = check_batch(kc, *case)
        assert err == 128 and (got["seq_lens"] == 0).any()


def test_batch_list_start(kc):
    ctx, new, held, table, free, T, bs, NB, _ = batch_case(12, 30, 60, 50, 8)
    free = np.concatenate([np.full(5, -1, np.int32), free])
    _, err = check_batch(kc, ctx, new, held, table, free, T, bs, NB, start=5)
    assert err == 0
    for start in (-1, len(free) + 1, len(free)):  # outside the list, or at its end: nothing to take
        got, err = check_batch(kc, ctx, new, held, table, free, T, bs, NB, start=start)
        assert err == 128 and got["free_next"][0] == start


def test_batch_bad_lengths_and_ids(kc):
    table = np.arange(6 * 5, dtype=np.int32).reshape(6, 5)
    # negative lengths, a request past its row, a held count past the row, one that fits
    _, err = check_batch(kc, [-1, 3, 70, 5, 4, 0], [2, -1, 11, 1, 1, 16], [1, 1, 5, 6, 1, 1], table, [90, 91], 40, 16, 99)
    assert err == 16
    # more than 64 drafted tokens are refused only as a tree
    t2 = np.arange(12, dtype=np.int32).reshape(1, 12)
    _, err = check_batch(kc, [3], [65], [6], t2, [], 65, 16, 12)
    assert err == 0
    _, err = check_batch(kc, [3], [65], [6], t2, [], 65, 16, 12, np.arange(-1, 64))
    assert err == 16
    # bad ids in the table and in the list
    t3 = np.array([[2, -5, -1, -1], [3, -1, -1, -1], [1, -1, -1, -1]], np.int32)
    _, err = check_batch(kc, [17, 16, 15], [3, 3, 20], [2, 1, 1], t3, [50, 4, 0], 26, 16, 5)
    assert err == 1


def test_batch_bad_parents(kc):
    table = np.arange(8, dtype=np.int32).reshape(1, 8)
    _, err = check_batch(kc, [5], [6], [8], table, [], 7, 16, 8, np.array([0, -2, 5, 1, 1000000, 4, -1]))
    assert err == 256


def test_batch_tokens_past_the_buffers(kc):
    ctx, new = [4, 4, 4, 4], [5, 6, 0, 3]
    table = np.arange(16, dtype=np.int32).reshape(4, 4)
    got, err = check_batch(kc, ctx, new, [1] * 4, table, [], 8, 16, 16)
    assert err == 16 and list(got["query_start_loc"]) == [0, 5, 8, 8, 8] and list(got["seq_lens"]) == [9, 0, 4, 0]


@pytest.mark.parametrize("B,T", [(0, 0), (0, 5), (3, 0)])
def test_batch_empty(kc, B, T):
    _, err = check_batch(kc, [7] * B, [0] * B, [1] * B, np.zeros((B, 2), np.int32), [], T, 16, 4)
    assert err == 0


def test_batch_strided_table_and_narrow_rows(kc):
    ctx, new, held, table, free, T, bs, NB, _ = batch_case(14, 25, 90, 40, 16)
    wide = torch.full((25, table.shape[1] + 6), -9, dtype=torch.int32, device="cuda")
    view = wide[:, 2:2 + table.shape[1]]
    view.copy_(dev(table))
    i32 = lambda a: dev(np.asarray(a, np.int32))  # noqa: E731
    b = kc.build_batch(i32(ctx), i32(new), view, i32(free), T, bs, NB, held_blocks=i32(held))
    want, _ = R.build_batch(ctx, new, held, table, free, T, bs, NB)
    np.testing.assert_array_equal(view.cpu().numpy(), want["block_table"])
    np.testing.assert_array_equal(b.slot_mapping.cpu().numpy(), want["slot_mapping"])
    assert (wide[:, :2] == -9).all() and (wide[:, 2 + table.shape[1]:] == -9).all()
    check_batch(kc, ctx, new, held, table, free, T, bs, NB, width=int(held.max()))


def test_batch_long_prompts_over_several_chunks_of_requests(kc):
    """More tokens than the grid has threads (four a thread) and more requests than a block has."""
    _, err = check_batch(kc, *batch_case(17, 1100, 40, 400, 16, extra_held=1, pad=2))
    assert err == 0
    ctx, new, held, table, free, T, bs, NB, _ = batch_case(18, 700, 300, 600, 8, pad=0)
    got, err = check_batch(kc, ctx, new, held, table, free[:len(free) // 2], T, bs, NB)
    assert err == 128


def test_batch_outputs_off_the_16_byte_boundary(kc):
    """The C call takes positions on 4 and slots on 8 bytes; the neighbours stay as they are."""
    ctx, new, held, table, free, T, bs, NB, _ = batch_case(19, 500, 40, 800, 16, pad=1)
    want, _ = R.build_batch(ctx, new, held, table, free, T, bs, NB)
    i32 = lambda a: dev(np.asarray(a, np.int32))  # noqa: E731
    B, tab, b = len(ctx), i32(table), kc.batch_buffers(len(ctx), T)
    ins = [i32(ctx), i32(new), i32(held), i32(free)]
    pos = torch.full((T + 8,), 77, dtype=torch.int32, device="cuda")
    slots = torch.full((T + 8,), 77, dtype=torch.int64, device="cuda")
    status = kc.lib.kv_build_batch(
        ins[0].data_ptr(), ins[1].data_ptr(), ins[2].data_ptr(), None, B, T, tab.data_ptr(), tab.shape[1], tab.shape[1], bs,
        NB, ins[3].data_ptr(), len(free), None, b.query_start_loc.data_ptr(), b.seq_lens.data_ptr(), pos.data_ptr() + 12,
        slots.data_ptr() + 24, None, b.held_blocks.data_ptr(), b.free_next.data_ptr(), None, None)
    torch.cuda.synchronize()
    assert status == 0
    np.testing.assert_array_equal(pos[3:3 + T].cpu().numpy(), want["positions"])
    np.testing.assert_array_equal(slots[3:3 + T].cpu().numpy(), want["slot_mapping"])
    for t in (pos, slots):
        assert (t[:3] == 77).all() and (t[3 + T:] == 77).all()


def test_batch_slots_agree_with_slot_mapping(kc):
    ctx, new, held, table, free, T, bs, NB, _ = batch_case(15, 60, 400, 90, 16, pad=0)
    i32 = lambda a: dev(np.asarray(a, np.int32))  # noqa: E731
    tab = i32(table)
    b = kc.build_batch(i32(ctx), i32(new), tab, i32(free), T, bs, NB, held_blocks=i32(held))
    slots = kc.compute_slot_mapping(tab, b.query_start_loc, b.positions, bs, NB)
    assert torch.equal(slots, b.slot_mapping)


def test_batch_matches_the_host_block_manager(kc):
    """The same requests through the host's allocator and through the device's list."""
    rng = np.random.default_rng(16)
    bs, rows, NB = 16, 24, 400
    bm = kc.BlockManager(NB, bs, rows, 64)
    ctx = rng.integers(1, 90, rows)
    for r in range(rows):
        bm.allocate(r, int(ctx[r]))
    bm.flush()
    table = np.full((rows, 64), -1, np.int32)
    held = np.zeros(rows, np.int32)
    for r in range(rows):
        tokens, blocks = bm.row(r)
        table[r, :len(blocks)] = blocks
        held[r] = len(blocks)
    taken = int(held.sum())
    new = rng.integers(0, 40, rows)
    got, err = check_batch(kc, ctx, new, held, table, np.arange(taken, NB), int(new.sum()), bs, NB)
    assert err == 0
    for r in range(rows):  # first in, first out: the manager hands out the same ids
        bm.allocate(r, int(new[r]))
        tokens, blocks = bm.row(r)
        assert tokens == got["seq_lens"][r] and list(got["block_table"][r, :len(blocks)]) == list(blocks)
    assert got["free_next"][0] == NB - bm.num_free_blocks() - taken


# ------------------------------------------------------------------ norm and rotation

def rope_table(max_pos, rot, seed=0):
    ang = np.arange(max_pos)[:, None] * 10000.0 ** (-np.arange(0, max(rot, 2), 2) / max(rot, 1))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)[:, :rot]


ROPE_CASES = [
    # T, Hq, Hkv, D, rot, interleaved, norm, cache, dtype
    (1, 32, 8, 128, 128, False, True, "same", torch.bfloat16),
    (1, 1, 1, 64, 64, True, True, "none", torch.float16),
    (5, 4, 2, 128, 64, False, True, "same", torch.float16),
    (37, 8, 2, 64, 32, True, True, "same", torch.bfloat16),
    (9, 7, 1, 128, 128, False, False, "e4m3", torch.bfloat16),
    (33, 3, 3, 128, 128, True, True, "e4m3", torch.float16),
    (130, 5, 5, 80, 80, False, True, "same", torch.bfloat16),
    (17, 6, 2, 96, 48, False, True, "none", torch.bfloat16),
    (11, 2, 1, 256, 256, False, True, "same", torch.float16),
    (11, 2, 2, 256, 64, True, True, "none", torch.bfloat16),
    (6, 9, 3, 16, 16, False, True, "same", torch.bfloat16),
    (4, 3, 1, 8, 0, False, True, "same", torch.float16),
    (21, 4, 4, 24, 16, True, True, "none", torch.float16),
    (40, 71, 1, 64, 64, False, True, "none", torch.bfloat16),
    (300, 12, 12, 64, 0, False, True, "same", torch.float16),
    (2100, 4, 1, 128, 128, False, True, "same", torch.bfloat16),
]


def rope_inputs(T, Hq, Hkv, D, rot, cache, dt, seed=0, max_pos=700):
    gen = torch.Generator().manual_seed(seed + T * 31 + D)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen).to(dt).cuda()
    q, k, v = (x.view(T, -1, D) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=gen)).to(dt).cuda() for _ in range(2))
    pos = torch.randint(0, max_pos, (T,), generator=gen, dtype=torch.int32)
    pos[0] = max_pos - 1
    s = dict(qkv=qkv, q=q, k=k, v=v, wq=wq, wk=wk, pos=pos.cuda(), cs=rope_table(max_pos, rot))
    if cache != "none":
        bs = 16
        NB = T // bs + 3
        s["slots"] = torch.randperm(NB * bs, generator=gen)[:T].cuda()
        cdt = dt if cache == "same" else torch.float8_e4m3fn
        raw = dt if cache == "same" else torch.uint8
        s["kc"] = torch.full((NB, bs, Hkv, D), 3, dtype=raw, device="cuda").view(cdt)
        s["vc"] = torch.full((NB, bs, Hkv, D), 5, dtype=raw, device="cuda").view(cdt)
    return s


def bits(t):
    return t.view(torch.uint8)


@pytest.mark.parametrize("case", ROPE_CASES, ids=lambda c: "x".join(str(v) for v in c[:5]) + f"_{c[5]}_{c[7]}_{str(c[8])[6:]}")
def test_norm_rope(kc, case):
    T, Hq, Hkv, D, rot, inter, norm, cache, dt = case
    s = rope_inputs(T, Hq, Hkv, D, rot, cache, dt)
    wq, wk = (s["wq"], s["wk"]) if norm else (None, None)
    cs = dev(s["cs"]) if rot else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = s["qkv"].clone()
    ks, vs = (0.02, 0.015) if cache == "e4m3" else (1.0, 1.0)
    if cache == "none":
        q_out, k_out = kc.qk_norm_rope(s["q"], s["k"], s["pos"], cs, wq, wk, 1e-5, inter, d_err=err)
    else:
        old = s["kc"].clone(), s["vc"].clone()
        k_out = torch.empty(T, Hkv, D, dtype=dt, device="cuda")
        q_out = kc.qk_norm_rope_and_cache(s["q"], s["k"], s["v"], s["pos"], cs, s["slots"], s["kc"], s["vc"], wq, wk,
                                          1e-5, inter, ks, vs, k_out=k_out, d_err=err)
    torch.cuda.synchronize()
    assert int(err) == 0 and torch.equal(before, s["qkv"])
    pos = s["pos"].cpu().numpy()
    keys = None
    for x, w, got in ((s["q"], wq, q_out), (s["k"], wk, k_out)):
        y, size = R.norm_rope(f64(x), None if w is None else f64(w), 1e-5, pos, s["cs"], rot, inter)
        bound = R.norm_rope_bound(y, size, D, dt)
        assert (np.abs(f64(got) - y) <= bound).all()
        keys = (y, size)
    if cache == "none":
        return
    # untouched slots keep their bytes; K and V land in their slots
    used = torch.zeros(s["kc"].shape[0] * 16, dtype=torch.bool, device="cuda")
    used[s["slots"]] = True
    for c, o in ((s["kc"], old[0]), (s["vc"], old[1])):
        flat, oflat = bits(c).reshape(len(used), -1), bits(o).reshape(len(used), -1)
        assert torch.equal(flat[~used], oflat[~used])
    kf, vf = (c.view(torch.uint8).view(len(used), Hkv, -1)[s["slots"]].view(c.dtype) for c in (s["kc"], s["vc"]))
    if cache == "same":
        assert torch.equal(bits(kf), bits(k_out)) and torch.equal(bits(vf), bits(s["v"].contiguous()))
    else:
        y, size = keys
        e32 = R.norm_rope_bound(y, size, D, torch.float8_e4m3fn) - R.HALF[torch.float8_e4m3fn] * np.abs(y) - R.TINY[torch.float8_e4m3fn]
        # e32 holds the float32 part (and its share of the rounding); the quotient adds half a unit
        z = np.clip(y / ks, -448, 448)
        bound = (e32 / ks) + 2.0 ** -4 * np.abs(z) + 2.0 ** -10 + np.abs(z) * 2.0 ** -23
        assert (np.abs(kf.float().double().cpu().numpy() - z) <= bound).all()
        # V is quantised as kv_reshape_and_cache does, bit for bit
        k2, v2 = torch.zeros_like(s["kc"].view(torch.uint8)), torch.zeros_like(s["vc"].view(torch.uint8))
        kc.reshape_and_cache(s["v"], s["v"], s["slots"], k2, v2, ks, vs)
        assert torch.equal(v2.view(len(used), Hkv, D)[s["slots"]].view(-1), bits(vf).reshape(-1))


@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_in_place(kc, inter):
    T, Hq, Hkv, D = 77, 6, 2, 64
    s = rope_inputs(T, Hq, Hkv, D, 64, "same", torch.bfloat16, seed=5)
    cs = dev(s["cs"])
    q, k = kc.qk_norm_rope(s["q"], s["k"], s["pos"], cs, s["wq"], s["wk"], 1e-6, inter)
    v = s["v"].clone()
    kc.qk_norm_rope_and_cache(s["q"], s["k"], s["v"], s["pos"], cs, s["slots"], s["kc"], s["vc"], s["wq"], s["wk"], 1e-6,
                              inter, q_out=s["q"], k_out=s["k"])
    assert torch.equal(s["q"], q) and torch.equal(s["k"], k) and torch.equal(s["v"], v)
    k2, v2 = torch.empty_like(s["kc"]), torch.empty_like(s["vc"])
    k2.copy_(s["kc"])
    v2.copy_(s["vc"])
    kc.reshape_and_cache(k, v.contiguous(), s["slots"], k2, v2)  # the two calls give the same cache
    assert torch.equal(k2, s["kc"]) and torch.equal(v2, s["vc"])


def test_norm_rope_padding_bad_positions_and_slots(kc):
    T, Hq, Hkv, D = 12, 4, 2, 128
    s = rope_inputs(T, Hq, Hkv, D, 128, "same", torch.float16, seed=6, max_pos=50)
    cs = dev(s["cs"])
    good_q, good_k = kc.qk_norm_rope(s["q"], s["k"], s["pos"], cs, s["wq"], s["wk"])
    pos, slots = s["pos"].clone(), s["slots"].clone()
    pos[3], pos[7] = -1, -100   # padding
    pos[5], pos[6] = 50, 2 ** 31 - 1  # past the table
    slots[1], slots[2] = -1, s["kc"].shape[0] * 16
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out, k_out = torch.full_like(good_q, 9), torch.full_like(good_k, 9)
    kc.qk_norm_rope_and_cache(s["q"], s["k"], s["v"], pos, cs, slots, s["kc"], s["vc"], s["wq"], s["wk"], q_out=q_out,
                              k_out=k_out, d_err=err)
    assert int(err) == 64 | 2
    skipped = [3, 5, 6, 7]
    kept = [t for t in range(T) if t not in skipped]
    assert (q_out[skipped] == 9).all() and (k_out[skipped] == 9).all()
    assert torch.equal(q_out[kept], good_q[kept]) and torch.equal(k_out[kept], good_k[kept])
    flat = s["kc"].view(-1, Hkv, D)
    written = [t for t in kept if t not in (1, 2)]
    assert torch.equal(flat[s["slots"][written]], good_k[written])
    assert (flat[s["slots"][skipped + [1, 2]]] == 3).all()
    assert int((flat != 3).any(2).any(1).sum()) == len(written)


def test_norm_rope_extreme_values(kc):
    """Rows of zeros (eps alone under the root), large values whose squares need float32, NaN in
    one head only."""
    T, Hq, Hkv, D = 4, 2, 1, 64
    s = rope_inputs(T, Hq, Hkv, D, 64, "none", torch.bfloat16, seed=7)
    s["q"][0] = 0
    s["q"][1] = 2.0 ** 60
    s["q"][2, 0, 5] = float("nan")
    cs = dev(s["cs"])
    q, k = kc.qk_norm_rope(s["q"], s["k"], s["pos"], cs, s["wq"], s["wk"], 1e-6)
    assert (q[0] == 0).all() and torch.isnan(q[2, 0]).all() and torch.isfinite(q[2, 1]).all() and torch.isfinite(k).all()
    y, size = R.norm_rope(f64(s["q"][1:2]), f64(s["wq"]), 1e-6, s["pos"][1:2].cpu().numpy(), s["cs"], 64, False)
    assert (np.abs(f64(q[1:2]) - y) <= R.norm_rope_bound(y, size, D, torch.bfloat16)).all()


# ------------------------------------------------------------------ tree attention

def tree_case(seed, contexts, drafts, Hq, Hkv, D, bs, dt, window=0, pad=0, masks=None):
    rng = np.random.default_rng(seed)
    L = np.array([c + n for c, n in zip(contexts, drafts)], np.int32)
    nblk = -(-L // bs)
    NB = int(nblk.sum()) + 5
    ids = rng.permutation(NB).astype(np.int32)
    table = np.full((len(L), int(nblk.max(initial=0)) + 2), -1, np.int32)
    o = 0
    for b in range(len(L)):
        table[b, :nblk[b]] = ids[o:o + nblk[b]]
        o += nblk[b]
        if window:  # blocks no row's window reaches may have gone back to the pool
            table[b, :max(0, contexts[b] - window) // bs] = -1
    qsl = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
    T = int(qsl[-1]) + pad
    if masks is None:
        masks = [w for n in drafts for w in R.masks_of(R.random_parents(rng, n))]
    masks = np.array(list(masks) + [0] * pad, np.uint64).view(np.int64)
    gen = torch.Generator().manual_seed(seed)
    q = torch.randn(T, Hq, D, generator=gen).to(dt).cuda()
    k = torch.randn(NB, bs, Hkv, D, generator=gen).to(dt).cuda()
    v = torch.randn(NB, bs, Hkv, D, generator=gen).to(dt).cuda()
    return dict(L=L, table=table, qsl=qsl, masks=masks, q=q, k=k, v=v, drafts=drafts, contexts=contexts, bs=bs,
                window=window, scale=D ** -0.5, dt=dt, D=D)


def run_tree(kc, c, workers=0, stream=None, fill=7.0, max_query_len=None):
    out = torch.full_like(c["q"], fill)
    lse = torch.full(c["q"].shape[:2], fill, dtype=torch.float32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc.paged_attention_tree(c["q"], c["k"], c["v"], dev(c["table"]), dev(c["L"]), dev(c["qsl"]), dev(c["masks"]),
                            max(1, int(c["L"].max(initial=1))),
                            max(list(c["drafts"]) + [1]) if max_query_len is None else max_query_len, c["scale"], c["window"],
                            num_workers=workers, out=out, lse_out=lse, d_err=err, stream=stream)
    torch.cuda.synchronize()
    return out, lse, int(err)


def reference_tree(c):
    return R.tree_attention(f64(c["q"]), f64(c["k"]), f64(c["v"]), c["table"], c["L"], c["qsl"], c["masks"], c["scale"],
                            c["window"])


def check_tree(c, out, lse, ref=None, rows=None):
    o, l, size, smax = reference_tree(c) if ref is None else ref
    tol, lse_tol = R.tree_bounds(o, l, size, smax, c["D"], c["dt"])
    T = int(c["qsl"][-1])
    rows = np.arange(T) if rows is None else rows
    got, got_l = f64(out), f64(lse)
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - o) <= tol)[rows]
        bad_l = ~((np.abs(got_l - l) <= lse_tol) | ((got_l == l) & ~np.isfinite(l)))[rows]
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(got - o)[rows][bad][:4], tol[rows][bad][:4])
    assert not bad_l.any(), (np.argwhere(bad_l)[:4], got_l[rows][bad_l][:4], l[rows][bad_l][:4])


TREE_CASES = [
    # contexts, drafts, Hq, Hkv, D, bs, dtype, window
    ([0], [1], 1, 1, 64, 8, torch.float16, 0),
    ([0], [1], 8, 2, 128, 16, torch.bfloat16, 0),
    ([100], [7], 32, 8, 128, 16, torch.bfloat16, 0),
    ([0, 127, 128, 129], [64, 1, 5, 64], 8, 2, 128, 16, torch.bfloat16, 0),
    ([300, 0, 17, 1000, 64], [33, 0, 64, 2, 63], 4, 4, 64, 32, torch.float16, 0),
    ([513, 5, 255], [60, 3, 1], 64, 8, 128, 16, torch.bfloat16, 0),           # several row tiles a head
    ([200, 40, 0], [64, 31, 12], 16, 1, 128, 8, torch.float16, 0),            # 16 heads a kv head
    ([200, 700], [40, 64], 28, 4, 128, 16, torch.bfloat16, 0),                # 7 heads a kv head
    ([77, 310], [64, 21], 10, 2, 64, 8, torch.bfloat16, 0),                   # 5 heads a kv head
    ([90], [9], 128, 1, 64, 16, torch.float16, 0),                            # one token a row tile
    ([90], [5], 100, 1, 128, 16, torch.bfloat16, 0),
    ([1500, 63, 64, 65, 200], [20, 64, 1, 30, 64], 8, 2, 128, 16, torch.bfloat16, 64),
    ([900, 300, 10], [64, 13, 64], 4, 4, 64, 8, torch.float16, 100),
    ([2000, 128, 4096], [16, 16, 40], 32, 8, 128, 32, torch.bfloat16, 1024),
    ([4000], [3], 8, 8, 64, 16, torch.float16, 0),                            # one long sequence, split
    ([1], [2], 2, 2, 128, 16, torch.float16, 4096),
    # groups of kv heads: 4 of up to 32 rows, 2 of up to 64 and 128, the last group not full
    ([130, 63, 700], [8, 3, 6], 12, 3, 128, 16, torch.bfloat16, 0),
    ([130, 64, 700], [32, 31, 1], 5, 5, 64, 8, torch.float16, 0),
    ([900, 65, 0], [9, 16, 10], 28, 7, 128, 32, torch.float16, 200),
    ([900, 127], [64, 33], 6, 6, 64, 16, torch.bfloat16, 0),
    ([500, 128, 2], [12, 9, 11], 15, 3, 64, 16, torch.bfloat16, 0),           # 60 rows, the group of 5
    ([1000, 257, 12], [32, 17, 31], 20, 5, 128, 16, torch.bfloat16, 0),       # 128 rows
    ([1000, 257, 12], [18, 16, 14], 21, 3, 128, 8, torch.float16, 300),       # 126 rows
    ([700, 40], [33, 64], 12, 6, 64, 32, torch.bfloat16, 0),                  # up to 128 rows of 64 dims
    ([700, 40, 300], [1, 1, 1], 64, 8, 128, 16, torch.bfloat16, 0),           # single tokens
    ([70] * 40, [2] * 40, 32, 8, 128, 16, torch.bfloat16, 64),
]


@pytest.mark.parametrize("case", TREE_CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}+{max(c[1])}_g{c[2] // c[3]}_d{c[4]}_bs{c[5]}_{str(c[6])[6:]}_w{c[7]}")
def test_tree(kc, case):
    c = tree_case(sum(case[0]) + sum(case[1]), *case)
    ref = reference_tree(c)
    for workers in (0, 1, 7):
        out, lse, err = run_tree(kc, c, workers)
        assert err == 0
        check_tree(c, out, lse, ref)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (6, 1, 64), (12, 6, 64)])
def test_tree_more_workers_than_sms_and_loose_bounds(kc, Hq, Hkv, D):
    """Shares of more CTAs than the GPU holds at once, and a max_query_len above every tree (which
    chooses the kernel): the same rows."""
    c = tree_case(31, [3000, 70, 1, 900], [3, 1, 20, 9], Hq, Hkv, D, 16, torch.bfloat16)
    ref = reference_tree(c)
    for workers, most in ((400, None), (1000, 64), (0, 64), (0, 40), (3, 21)):
        out, lse, err = run_tree(kc, c, workers, max_query_len=most)
        assert err == 0
        check_tree(c, out, lse, ref)


def test_step_in_a_cache_past_32_bit_offsets(kc):
    """Caches of more than 2^31 elements: slots and blocks at their end, written and read."""
    NB, bs, Hkv, Hq, D, dt = 140_000, 16, 8, 32, 128, torch.bfloat16
    kbig, vbig = (torch.empty(NB, bs, Hkv, D, dtype=dt, device="cuda") for _ in range(2))
    contexts, drafts = [300, 17], [9, 30]
    c = tree_case(32, contexts, drafts, Hq, Hkv, D, bs, dt)
    small = c["k"].shape[0]
    first = NB - small  # the small pool's blocks, at the end of the big one
    kbig[first:], vbig[first:] = c["k"], c["v"]
    # the drafted keys and values come through the norm, rotation and cache write
    gen = torch.Generator().manual_seed(32)
    T = int(c["qsl"][-1])
    q, k, v = (torch.randn(T, h, D, generator=gen).to(dt).cuda() for h in (Hq, Hkv, Hkv))
    table, slots, pos = c["table"].copy(), [], []
    for b, (ctx, n) in enumerate(zip(contexts, drafts)):
        at = np.arange(ctx, ctx + n)
        slots += (table[b, at // bs].astype(np.int64) * bs + at % bs).tolist()
        pos += at.tolist()
    cs = dev(rope_table(400, D))
    k_out = torch.empty_like(k)
    big_slots = dev(np.array(slots) + first * bs)
    assert int(big_slots.max()) * Hkv * D > 2 ** 31
    c["q"] = kc.qk_norm_rope_and_cache(q, k, v, dev(np.array(pos, np.int32)), cs, big_slots, kbig, vbig, k_out=k_out)
    for cache, rows in ((c["k"], k_out), (c["v"], v)):
        cache.view(-1, Hkv, D)[dev(np.array(slots))] = rows
    assert torch.equal(kbig[first:], c["k"]) and torch.equal(vbig[first:], c["v"])
    ref = reference_tree(c)
    big = dict(c, k=kbig, v=vbig, table=np.where(table >= 0, table + first, -1).astype(np.int32))
    for most in (None, 64):
        out, lse, err = run_tree(kc, big, max_query_len=most)
        assert err == 0
        check_tree(c, out, lse, ref)


def test_tree_masks_of_any_kind(kc):
    """Rows that see nothing (with and without a context), everything, only others, forward."""
    n = 9
    kinds = [0, (1 << n) - 1, ~0 & (2 ** 64 - 1), 1 << 8, (1 << 4) | (1 << 6), 1 << 63, 2, 1 << 6, 0]
    c = tree_case(1, [0, 200], [n, n], 8, 2, 128, 16, torch.bfloat16, masks=kinds + kinds[::-1])
    out, lse, err = run_tree(kc, c)
    assert err == 0
    check_tree(c, out, lse)
    for row in (0, 5, 8):  # no context and no bit below n
        assert (out[row] == 0).all() and torch.isneginf(lse[row]).all()


def check_unseen_keys(kc, dt, poison, window, drafts, Hq, Hkv, D=128, workers=0):
    """Poison in every slot no row sees: free blocks, the rest of the last block, keys before the
    window; and in drafted keys and window keys that only some rows see, whose other rows stay clean."""
    contexts, bs = [150, 0, 40, 263], 16
    # (row 0 of each tree sees itself alone of it, so that no drafted key is seen by all)
    c = tree_case(21, contexts, drafts, Hq, Hkv, D, bs, dt, window)
    clean = {k: c[k].clone() for k in ("k", "v")}
    seen_any = torch.zeros(c["k"].shape[0] * bs, dtype=torch.bool)
    touched = np.zeros(len(c["q"]), bool)
    masks = c["masks"].view(np.uint64)
    partly = []
    for b, (ctx, n) in enumerate(zip(contexts, drafts)):
        t0 = int(c["qsl"][b])
        seen = R.seen_keys(masks[t0:t0 + n], n, ctx, window)
        pos = np.arange(ctx + n)
        slots = np.maximum(c["table"][b, pos // bs], 0) * bs + pos % bs
        seen_any[slots[seen.any(0)]] = True
        some = np.flatnonzero(seen.any(0) & ~seen.all(0))
        for j in some[::max(1, len(some) // 3)]:
            partly.append(int(slots[j]))
            touched[t0:t0 + n] |= seen[:, j]
    for name in ("k", "v"):
        c[name].view(-1, Hkv, D)[~seen_any] = poison
    out, lse, err = run_tree(kc, c, workers)
    assert err == 0
    poisoned = dict(c)
    c_ref = {**c, **clean}
    ref = reference_tree(c_ref)
    check_tree(c_ref, out, lse, ref)
    # poison in values that some rows see: the other rows are untouched, bit for bit
    for name in ("v", "k"):
        p = {**poisoned, name: poisoned[name].clone()}
        p[name].view(-1, Hkv, D)[partly, :, 3] = poison
        out2, lse2, err = run_tree(kc, p, workers)
        rest = torch.from_numpy(~touched)
        assert touched.any() and (~touched).any() and torch.equal(out2[rest], out[rest]) and torch.equal(lse2[rest], lse[rest])
        if name == "v":  # and the rows that see it get it, in that dim alone
            hit = out2[torch.from_numpy(touched)]
            same = out[torch.from_numpy(touched)]
            dims = [d for d in range(D) if d != 3]
            assert torch.equal(hit[..., dims], same[..., dims]) and not torch.isfinite(hit[..., 3]).any()
            assert torch.equal(lse2, lse)
            if poison == poison:
                assert (hit[..., 3] == poison).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("drafts,Hq,Hkv", [([13, 64, 7, 30], 8, 2), ([8, 7, 2, 5], 12, 3), ([13, 16, 7, 11], 20, 5),
                                           ([13, 32, 7, 30], 12, 3), ([9, 11, 2, 8], 16, 1)],
                         ids=["pair", "four", "two", "two_wide", "one"])
def test_tree_unseen_keys_have_no_part(kc, dt, poison, window, drafts, Hq, Hkv):
    check_unseen_keys(kc, dt, poison, window, drafts, Hq, Hkv)


@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("drafts,Hq,Hkv,workers", [([8, 7, 2, 5], 12, 3, 0), ([13, 16, 7, 11], 20, 5, 5),
                                                   ([8, 7, 2, 16], 28, 7, 0), ([13, 64, 7, 30], 2, 2, 0)],
                         ids=["four", "four_in_two_tiles", "seven", "two"])
def test_tree_unseen_keys_of_64_dims_have_no_part(kc, poison, window, drafts, Hq, Hkv, workers):
    check_unseen_keys(kc, torch.bfloat16, poison, window, drafts, Hq, Hkv, 64, workers)


@pytest.mark.parametrize("Hq,Hkv,D,n,bs,window", [
    (8, 2, 128, 7, 16, 0), (32, 8, 128, 64, 16, 0), (32, 8, 128, 7, 8, 0), (12, 12, 64, 24, 16, 0), (6, 1, 64, 40, 16, 0),
    (4, 1, 128, 64, 32, 0), (12, 3, 64, 11, 16, 5000), (7, 7, 64, 50, 16, 0)])
def test_tree_one_sequence_over_every_worker(kc, Hq, Hkv, D, n, bs, window):
    """One sequence in many shares: few items of many pieces, which the warps of a CTA join together."""
    c = tree_case(35, [9000], [n], Hq, Hkv, D, bs, torch.bfloat16, window, pad=2)
    c["masks"][n // 2] = 0  # a row of the context alone
    ref = reference_tree(c)
    for workers in (0, 33, 700):
        out, lse, err = run_tree(kc, c, workers)
        assert err == 0
        check_tree(c, out, lse, ref)
        assert (out[n:] == 7).all() and (lse[n:] == 7).all()
    small = tree_case(36, [130], [n], Hq, Hkv, D, bs, torch.bfloat16, masks=[0] * (n - 1) + [1])  # few pieces of many
    out, lse, err = run_tree(kc, small)
    assert err == 0
    check_tree(small, out, lse)


def test_tree_seen_context_nan_reaches_every_row(kc):
    c = tree_case(22, [200], [5], 4, 2, 128, 16, torch.bfloat16)
    c["v"].view(-1, 2, 128)[c["table"][0, 3] * 16 + 2, 1, 9] = float("nan")
    out, lse, err = run_tree(kc, c)
    assert torch.isnan(out[:, 2:, 9]).all() and torch.isfinite(out[:, :2]).all() and torch.isfinite(lse).all()
    assert torch.isfinite(out[:, 2:, :9]).all()


def test_tree_rejected_sequences_rows_behind_and_bad_blocks(kc):
    c = tree_case(23, [40, 60, 90, 33], [10, 8, 6, 5], 8, 2, 128, 16, torch.bfloat16, pad=4)
    ref = reference_tree(c)
    good = c["L"].copy()
    c["L"][0], c["L"][2] = 9, 10 ** 6  # fewer than its drafted tokens; past max_seq_len and the table
    out = torch.full_like(c["q"], 7.0)
    lse = torch.full(c["q"].shape[:2], 7.0, dtype=torch.float32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc.paged_attention_tree(c["q"], c["k"], c["v"], dev(c["table"]), dev(c["L"]), dev(c["qsl"]), dev(c["masks"]),
                            int(good.max()), 10, c["scale"], out=out, lse_out=lse, d_err=err)
    assert int(err) == 16
    for r in list(range(0, 10)) + list(range(18, 24)):
        assert (out[r] == 0).all() and torch.isneginf(lse[r]).all()
    rows = np.array(list(range(10, 18)) + list(range(24, 29)))
    check_tree(c, out, lse, ref, rows)
    assert (out[29:] == 7).all() and (lse[29:] == 7).all()  # rows of no sequence
    # a sequence with more rows than max_query_len says
    out3, lse3 = torch.full_like(c["q"], 7.0), torch.full_like(lse, 7.0)
    c["L"] = good
    err.zero_()
    kc.paged_attention_tree(c["q"], c["k"], c["v"], dev(c["table"]), dev(c["L"]), dev(c["qsl"]), dev(c["masks"]),
                            int(good.max()), 8, c["scale"], out=out3, lse_out=lse3, d_err=err)
    assert int(err) == 16 and (out3[:10] == 0).all()
    check_tree(c, out3, lse3, ref, np.arange(10, 29))
    # block ids outside the pool read as zeros
    c["table"][1, 1], c["table"][3, 0] = -3, c["k"].shape[0]
    z = dict(c, table=c["table"].copy(), k=torch.cat([c["k"], torch.zeros_like(c["k"][:1])]),
             v=torch.cat([c["v"], torch.zeros_like(c["v"][:1])]))
    z["table"][1, 1] = z["table"][3, 0] = c["k"].shape[0]
    out4, lse4, e = run_tree(kc, c)
    assert e == 1
    check_tree(z, out4, lse4)


def test_tree_large_scores_and_scale_zero(kc):
    c = tree_case(24, [600, 3], [20, 64], 8, 2, 128, 16, torch.float16)
    c["q"] *= 30
    out, lse, err = run_tree(kc, c)
    check_tree(c, out, lse)
    c["scale"] = 0.0
    out, lse, err = run_tree(kc, c)
    check_tree(c, out, lse)


def test_tree_rising_scores(kc):
    """Scores that keep rising along the context, so that the running maximum moves in every tile."""
    c = tree_case(25, [1200], [12], 4, 1, 128, 16, torch.bfloat16)
    pos = np.arange(1212)
    slots = c["table"][0, pos // 16] * 16 + pos % 16
    u = torch.randn(128, generator=torch.Generator().manual_seed(1)).cuda()
    k = c["k"].view(-1, 1, 128)
    k[torch.from_numpy(slots).cuda().long(), 0] = (torch.arange(1212, device="cuda")[:, None] * 0.01 * u).to(torch.bfloat16)
    c["q"][:] = (u * 1.5).to(torch.bfloat16)
    out, lse, err = run_tree(kc, c)
    check_tree(c, out, lse)
    c["q"].neg_()
    out, lse, err = run_tree(kc, c)
    check_tree(c, out, lse)


def test_tree_chain_is_speculative_decode(kc):
    """A tree that is a chain: the speculative decode call and chunked prefill give the same rows."""
    n, contexts = 4, [130, 5, 700]
    masks = [(2 << i) - 1 for i in range(n)] * 3
    c = tree_case(26, contexts, [n] * 3, 8, 2, 128, 16, torch.bfloat16, masks=masks)
    ref = reference_tree(c)
    out, lse, err = run_tree(kc, c)
    check_tree(c, out, lse, ref)
    L = dev(c["L"])
    d = kc.paged_attention_decode(c["q"], c["k"], c["v"], dev(c["table"]), L, int(c["L"].max()), n, c["scale"])
    p = kc.paged_attention_prefill(c["q"], c["k"], c["v"], dev(c["table"]), L, dev(c["qsl"]), int(c["L"].max()), n, c["scale"])
    tol = 2 * torch.from_numpy(R.tree_bounds(*ref, 128, torch.bfloat16)[0]).cuda()
    assert ((out.double() - d.double()).abs() <= tol).all() and ((out.double() - p.double()).abs() <= tol).all()


def test_tree_repeats_bit_for_bit(kc):
    c = tree_case(27, [3000, 10, 900], [30, 64, 7], 32, 8, 128, 16, torch.bfloat16)
    first, l1, _ = run_tree(kc, c)
    for _ in range(3):
        again, l2, _ = run_tree(kc, c)
        assert torch.equal(first, again) and torch.equal(l1, l2)


def test_tree_many_short_sequences(kc):
    rng = np.random.default_rng(28)
    B = 700
    c = tree_case(28, rng.integers(0, 40, B).tolist(), rng.integers(0, 6, B).tolist(), 4, 2, 64, 8, torch.float16)
    out, lse, err = run_tree(kc, c)
    assert err == 0
    check_tree(c, out, lse)


def test_tree_workspace_grows_with_the_batch(kc):
    """A workspace made for the largest batch serves the smaller ones."""
    for Hq, Hkv, D in ((12, 12, 64), (32, 8, 64), (6, 3, 64), (4, 1, 64), (2, 2, 64), (32, 8, 128), (64, 8, 128), (8, 1, 128)):
        for workers in (0, 5, 600):
            sizes = np.array([[kc.paged_attention_tree_workspace_size(B, n, Hq, Hkv, D, workers) for n in range(1, 65)]
                              for B in (1, 2, 9, 13, 40, 500)])
            assert (np.diff(sizes, axis=0) >= 0).all() and (np.diff(sizes, axis=1) >= 0).all()


def test_tree_small_workspace_is_refused(kc):
    c = tree_case(29, [300], [20], 8, 2, 128, 16, torch.bfloat16)
    need = kc.paged_attention_tree_workspace_size(1, 20, 8, 2, 128)
    if need == 0:
        pytest.skip("no workspace needed")
    qsl, table, lens, masks = (dev(c[x]) for x in ("qsl", "table", "L", "masks"))
    args = (c["q"].data_ptr(), 1, qsl.data_ptr(), 1, 20, 20, 8, c["k"].data_ptr(), c["v"].data_ptr(), 1, 2, 128, 16,
            c["k"].shape[0], table.data_ptr(), table.shape[1], table.shape[1], lens.data_ptr(), 320, 0.1, 0,
            masks.data_ptr(), 0)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c["q"])
    f = kc.lib.kv_paged_attention_tree
    assert f(*args, None, 0, out.data_ptr(), None, None, None) == 4
    assert f(*args, ws.data_ptr(), need - 1, out.data_ptr(), None, None, None) == 4
    assert f(*args, ws.data_ptr() + 16, need, out.data_ptr(), None, None, None) == 1


# ------------------------------------------------------------------ together

class Step:
    """One speculative step of one layer: metadata, norm with rotation and cache write, attention."""

    def __init__(self, kc, seed=40, B=9, Hq=8, Hkv=2, D=128, bs=16, dt=torch.bfloat16, pad=3, max_new=29):
        rng = np.random.default_rng(seed)
        self.kc, self.D, self.bs, self.dt = kc, D, bs, dt
        self.ctx, self.new = rng.integers(0, 200, B), rng.integers(0, max_new + 1, B)
        self.new[0] = max_new
        self.held = -(-self.ctx // bs)
        need = -(-(self.ctx + self.new) // bs) - self.held
        self.NB = int(self.held.sum() + need.sum()) + 4
        ids = rng.permutation(self.NB).astype(np.int32)
        self.table = np.full((B, 300 // bs + 1), -1, np.int32)
        at = 0
        for r in range(B):
            self.table[r, :self.held[r]] = ids[at:at + self.held[r]]
            at += self.held[r]
        self.free = ids[at:]
        self.T = int(self.new.sum()) + pad
        self.parents = np.full(self.T, -1, np.int32)
        self.parents[:self.T - pad] = np.concatenate([R.random_parents(rng, int(n)) for n in self.new])
        gen = torch.Generator().manual_seed(seed)
        self.qkv = torch.randn(self.T, (Hq + 2 * Hkv) * D, generator=gen).to(dt).cuda()
        self.q, self.k, self.v = (x.view(self.T, -1, D) for x in self.qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
        self.wq, self.wk = ((1 + 0.3 * torch.randn(D, generator=gen)).to(dt).cuda() for _ in range(2))
        self.kc0 = torch.randn(self.NB, bs, Hkv, D, generator=gen).to(dt).cuda()
        self.vc0 = torch.randn(self.NB, bs, Hkv, D, generator=gen).to(dt).cuda()
        self.cs_np = rope_table(512, D)
        i32 = lambda a: dev(np.asarray(a, np.int32))  # noqa: E731
        self.d = dict(ctx=i32(self.ctx), new=i32(self.new), held=i32(self.held), free=i32(self.free), parents=i32(self.parents))
        self.cs = dev(self.cs_np)
        self.reset()
        self.batch = kc.batch_buffers(B, self.T, True)
        self.q_out = torch.empty(self.T, Hq, D, dtype=dt, device="cuda")
        self.out = torch.empty_like(self.q_out)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.max_len, self.max_new = int((self.ctx + self.new).max()), int(self.new.max())
        self.ws = torch.empty(max(256, kc.paged_attention_tree_workspace_size(B, self.max_new, Hq, Hkv, D)),
                              dtype=torch.uint8, device="cuda")

    def reset(self):
        self.d["table"] = dev(self.table)
        self.kcache, self.vcache = self.kc0.clone(), self.vc0.clone()

    def reset_in_place(self):
        """The state before a step again, in the tensors that a graph has captured."""
        self.d["table"].copy_(dev(self.table))
        self.kcache.copy_(self.kc0)
        self.vcache.copy_(self.vc0)

    def run(self, stream=None):
        kc, d = self.kc, self.d
        if stream is None:
            self.out.fill_(7.0)
        b = kc.build_batch(d["ctx"], d["new"], d["table"], d["free"], self.T, self.bs, self.NB, held_blocks=d["held"],
                           parents=d["parents"], out=self.batch, d_err=self.err, stream=stream)
        kc.qk_norm_rope_and_cache(self.q, self.k, self.v, b.positions, self.cs, b.slot_mapping, self.kcache, self.vcache,
                                  self.wq, self.wk, 1e-6, q_out=self.q_out, d_err=self.err, stream=stream)
        kc.paged_attention_tree(self.q_out, self.kcache, self.vcache, d["table"], b.seq_lens, b.query_start_loc,
                                b.tree_mask, self.max_len, self.max_new, self.D ** -0.5, workspace=self.ws, out=self.out,
                                d_err=self.err, stream=stream)

    def check(self):
        torch.cuda.synchronize()
        assert int(self.err) == 0
        want, e = R.build_batch(self.ctx, self.new, self.held, self.table, self.free, self.T, self.bs, self.NB, self.parents)
        assert e == 0
        for k, v in self.batch._asdict().items():
            np.testing.assert_array_equal(v.cpu().numpy(), want[k], err_msg=k)
        np.testing.assert_array_equal(self.d["table"].cpu().numpy(), want["block_table"])
        n = int(self.new.sum())
        pos = want["positions"][:n]
        yq, sq = R.norm_rope(f64(self.q[:n]), f64(self.wq), 1e-6, pos, self.cs_np, self.D, False)
        yk, sk = R.norm_rope(f64(self.k[:n]), f64(self.wk), 1e-6, pos, self.cs_np, self.D, False)
        assert (np.abs(f64(self.q_out[:n]) - yq) <= R.norm_rope_bound(yq, sq, self.D, self.dt)).all()
        # the caches: untouched but for the new slots
        kw, vw = f64(self.kc0), f64(self.vc0)
        flat_k, flat_v = (f64(c).reshape(self.NB * self.bs, -1, self.D) for c in (self.kcache, self.vcache))
        slots = want["slot_mapping"][:n]
        assert (np.abs(flat_k[slots] - yk) <= R.norm_rope_bound(yk, sk, self.D, self.dt)).all()
        vw.reshape(self.NB * self.bs, -1, self.D)[slots] = f64(self.v[:n])
        np.testing.assert_array_equal(flat_v, vw.reshape(flat_v.shape))
        kw.reshape(self.NB * self.bs, -1, self.D)[slots] = flat_k[slots]
        np.testing.assert_array_equal(flat_k, kw.reshape(flat_k.shape))
        # attention over what the cache now holds
        ref = R.tree_attention(f64(self.q_out), kw, vw, want["block_table"], want["seq_lens"], want["query_start_loc"],
                               want["tree_mask"], self.D ** -0.5)
        tol, _ = R.tree_bounds(*ref, self.D, self.dt)
        assert (np.abs(f64(self.out) - ref[0]) <= tol)[:n].all()
        assert (self.out[n:] == 7).all()


@pytest.mark.parametrize("Hq,Hkv,D,bs,dt,max_new", [
    (8, 2, 128, 16, torch.bfloat16, 29), (6, 3, 64, 8, torch.float16, 12), (4, 4, 128, 32, torch.bfloat16, 64),
    (16, 1, 64, 16, torch.float16, 40), (64, 8, 128, 16, torch.bfloat16, 50)])
def test_step_together(kc, Hq, Hkv, D, bs, dt, max_new):
    s = Step(kc, Hq=Hq, Hkv=Hkv, D=D, bs=bs, dt=dt, max_new=max_new)
    s.run()
    s.check()
    s.reset()  # again on fresh buffers
    s.run()
    s.check()


def test_step_captured_and_replayed(kc):
    """Two graphs that share one workspace, replayed one after the other with new contents."""
    a, b = Step(kc, 41), Step(kc, 42, B=5)
    ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    a.ws = b.ws = ws
    graphs = []
    for s in (a, b):
        s.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for s in (a, b):  # new contents in the captured buffers
        s.qkv.copy_(torch.randn(s.qkv.shape, generator=torch.Generator().manual_seed(7)).to(s.dt))
        s.kcache.copy_(s.kc0)
        s.vcache.copy_(s.vc0)
        s.d["table"].copy_(dev(s.table))
    for g in graphs + graphs:
        g.replay()
    a.check()
    b.check()


def test_steps_captured_behind_every_kind_of_work(kc):
    """The calls in one capture after a fill, a copy, a join of two streams, and on a forked stream."""
    a, b = Step(kc, 47), Step(kc, 48, B=20, bs=8)
    for s in (a, b):
        s.run()
    torch.cuda.synchronize()
    x = torch.zeros(1 << 20, device="cuda")
    y, host = torch.empty_like(x), torch.empty(1 << 20, pin_memory=True)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        x.zero_()
        y.copy_(x)
        a.run()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            b.run()          # first on a forked stream
            b.run()
        y.add_(1)
        main.wait_stream(side)
        a.run(stream=main)   # first after the join
        host.copy_(y, non_blocking=True)
        a.run()
    for _ in range(3):
        for s in (a, b):
            s.reset_in_place()
            s.out.fill_(7.0)
        graph.replay()
        a.check()
        b.check()
        assert (host == 1).all()


def test_steps_on_two_streams_at_once(kc):
    a, b = Step(kc, 43), Step(kc, 44, B=20)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                s.run()
    a.check()
    b.check()
    st = torch.cuda.Stream()
    a.reset()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        a.out.fill_(7.0)
    a.run(stream=st)  # an explicit stream that is not the current one
    st.synchronize()
    torch.cuda.synchronize()
    a.out[int(a.new.sum()):] = 7.0
    a.check()


def test_memory_of_a_call_on_another_stream(kc, monkeypatch):
    """The workspace that a call on a given stream makes for itself is that stream's: what the current
    stream allocates next, while the call may still run, lies elsewhere."""
    s = Step(kc, 46)
    s.run()
    torch.cuda.synchronize()
    seen = []
    real = kc.lib.kv_paged_attention_tree

    def call(*args):
        seen.append((args[23], args[24], args[25]))  # workspace, its bytes, out
        return real(*args)
    monkeypatch.setattr(kc.lib, "kv_paged_attention_tree", call)
    b, st = s.batch, torch.cuda.Stream()
    args = (s.q_out, s.kcache, s.vcache, s.d["table"], b.seq_lens, b.query_start_loc, b.tree_mask, s.max_len, s.max_new,
            s.D ** -0.5)
    s.out.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(3):
        kc.paged_attention_tree(*args, out=s.out, d_err=s.err, stream=st)
        at, size, _ = seen[-1]
        other = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
        assert all(x.data_ptr() + size <= at or at + size <= x.data_ptr() for x in other)
        del other
    s.check()
    out = kc.paged_attention_tree(*args, stream=st)
    st.synchronize()
    n = int(s.new.sum())
    assert torch.equal(out[:n], s.out[:n]) and seen[-1][2] == out.data_ptr()
    with torch.cuda.stream(st):
        assert torch.cuda.current_stream() == st
        q1 = kc.qk_norm_rope(s.q, s.k, b.positions, s.cs, s.wq, s.wk)[0]
    q2 = kc.qk_norm_rope(s.q, s.k, b.positions, s.cs, s.wq, s.wk, stream=st)[0]
    torch.cuda.synchronize()
    assert torch.equal(q1[:n], q2[:n])


def test_step_after_step(kc):
    """Three steps in a row without the host: accepted lengths go up, rejected tokens' blocks are
    used again, and the list's start moves on by itself."""
    rng = np.random.default_rng(45)
    B, bs, NB = 12, 8, 300
    ctx = rng.integers(1, 60, B)
    held = -(-ctx // bs)
    ids = rng.permutation(NB).astype(np.int32)
    table = np.full((B, 24), -1, np.int32)
    at = 0
    for r in range(B):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    free = ids[at:]
    i32 = lambda a: dev(np.asarray(a, np.int32))  # noqa: E731
    d_ctx, d_table, d_free = i32(ctx), i32(table), i32(free)
    sets = [kc.batch_buffers(B, 20 * B), kc.batch_buffers(B, 20 * B)]
    d_held, d_start, start = i32(held), None, 0
    for step in range(3):
        new = rng.integers(1, 20, B)
        accepted = np.minimum(new, rng.integers(1, 8, B))
        b = kc.build_batch(d_ctx, i32(new), d_table, d_free, 20 * B, bs, NB, held_blocks=d_held, free_start=d_start,
                           out=sets[step % 2])
        want, e = R.build_batch(ctx, new, held, table, free, 20 * B, bs, NB, start=start)
        assert e == 0
        for k, v in want.items():
            if v is not None and k != "block_table":
                np.testing.assert_array_equal(getattr(b, k).cpu().numpy(), v, err_msg=f"{k} of step {step}")
        np.testing.assert_array_equal(d_table.cpu().numpy(), want["block_table"])
        d_ctx = d_ctx + i32(accepted)
        ctx = ctx + accepted
        d_held, d_start = b.held_blocks, b.free_next
        held, table, start = want["held_blocks"], want["block_table"], int(want["free_next"][0])


def test_step_accepted_path_then_the_next_step(kc):
    """Drafted trees, acceptance of one path of each, its K/V moved to their final slots, and the next
    step over the accepted context: the cache then holds each sequence as if it had been written token
    by token, and the second step's attention is that of the definition over it."""
    rng = np.random.default_rng(60)
    B, Hq, Hkv, D, bs, NB, T, dt = 6, 8, 4, 128, 16, 200, 80, torch.bfloat16
    ctx = rng.integers(1, 90, B)
    held = -(-ctx // bs)
    ids = rng.permutation(NB).astype(np.int32)
    table = np.full((B, 16), -1, np.int32)
    at = 0
    for r in range(B):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    i32 = lambda a: dev(np.asarray(a, np.int32))  # noqa: E731
    gen = torch.Generator().manual_seed(60)
    kcache, vcache = (torch.randn(NB, bs, Hkv, D, generator=gen).to(dt).cuda() for _ in range(2))
    cs = dev(rope_table(300, D))
    w = torch.ones(D, dtype=dt, device="cuda")
    d_table, d_free = i32(table), i32(ids[at:])
    sets = [kc.batch_buffers(B, T, True), kc.batch_buffers(B, T, True)]
    d_held, d_start = i32(held), None
    tokens = [[(kcache.view(-1, Hkv, D)[s].clone(), vcache.view(-1, Hkv, D)[s].clone())
               for s in (int(table[r, p // bs]) * bs + p % bs for p in range(ctx[r]))] for r in range(B)]
    for step in range(3):
        new = rng.integers(1, 13, B)
        n = int(new.sum())
        parents = np.full(T, -1)
        trees = [R.random_parents(rng, int(k)) for k in new]
        parents[:n] = np.concatenate(trees)
        b = kc.build_batch(i32(ctx), i32(new), d_table, d_free, T, bs, NB, held_blocks=d_held, parents=i32(parents),
                           free_start=d_start, out=sets[step % 2])
        q, k, v = (torch.randn(T, h, D, generator=gen).to(dt).cuda() for h in (Hq, Hkv, Hkv))
        k_out = torch.zeros_like(k)
        q = kc.qk_norm_rope_and_cache(q, k, v, b.positions, cs, b.slot_mapping, kcache, vcache, w, w, k_out=k_out)
        out = kc.paged_attention_tree(q, kcache, vcache, d_table, b.seq_lens, b.query_start_loc, b.tree_mask,
                                      int((ctx + new).max()), int(new.max()), 0.09)
        # every row against its own path, token by token
        qsl = b.query_start_loc.cpu().numpy()
        for r in range(B):
            for i in range(new[r]):
                path = [i]
                while trees[r][path[-1]] >= 0:
                    path.append(int(trees[r][path[-1]]))
                rows = [qsl[r] + j for j in path]
                K = torch.stack([t[0] for t in tokens[r]] + [k_out[j] for j in rows]).double().cpu().numpy()
                V = torch.stack([t[1] for t in tokens[r]] + [v[j] for j in rows]).double().cpu().numpy()
                Q = f64(q[qsl[r] + i])
                for h in range(Hq):
                    kk, vv = K[:, h * Hkv // Hq], V[:, h * Hkv // Hq]
                    s = kk @ Q[h] * 0.09
                    p = np.exp(s - s.max())
                    o, size = p @ vv / p.sum(), p @ np.abs(vv) / p.sum()
                    smax = (np.abs(kk) @ np.abs(Q[h]) * 0.09).max()
                    tol, _ = R.tree_bounds(o, np.float64(0), size, np.float64(smax), D, dt)
                    assert (np.abs(f64(out[qsl[r] + i, h]) - o) <= tol).all()
        # accept the path to one token of each tree
        tab = d_table.cpu().numpy()
        move = np.full(T, -1, np.int64)
        accepted = np.zeros(B, np.int64)
        for r in range(B):
            path = [int(rng.integers(0, new[r]))]
            while trees[r][path[-1]] >= 0:
                path.append(int(trees[r][path[-1]]))
            for depth, j in enumerate(reversed(path)):
                p = ctx[r] + depth
                assert int(b.positions[qsl[r] + j]) == p
                move[qsl[r] + j] = tab[r, p // bs].astype(np.int64) * bs + p % bs
                tokens[r].append((k_out[qsl[r] + j].clone(), v[qsl[r] + j].clone()))
            accepted[r] = len(path)
        kc.reshape_and_cache(k_out, v, dev(move), kcache, vcache)
        ctx = ctx + accepted
        for r in range(B):
            p = np.arange(ctx[r])
            s = dev(tab[r, p // bs].astype(np.int64) * bs + p % bs)
            assert torch.equal(kcache.view(-1, Hkv, D)[s], torch.stack([t[0] for t in tokens[r]]))
            assert torch.equal(vcache.view(-1, Hkv, D)[s], torch.stack([t[1] for t in tokens[r]]))
        d_held, d_start = b.held_blocks, b.free_next
