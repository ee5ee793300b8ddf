"""Query/key norm with rotation and the write into INT4 caches (kv_qk_norm_rope_int4) against a 64-bit
implementation, and a step over such caches."""
import numpy as np
import pytest
import torch

from tests import step_reference as R
from tests.sinks_reference import BF16, F16, Inputs, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    from paged_kv_cache_block_gb300 import kvcache
    return kvcache


def f64(t):
    return t.double().cpu().numpy()


def codes(cache):
    x = cache.cpu().numpy().astype(np.int64)
    c = np.stack([x & 15, x >> 4], -1).reshape(*x.shape[:-1], -1)
    return np.where(c > 7, c - 16, c).reshape(-1, *c.shape[2:-1], c.shape[-1])


def inputs(seed, T, Hq, Hkv, dt, bs, group, rot, norm, spare=2):
    rng = np.random.default_rng(seed)
    D = 128
    qkv = torch.from_numpy(rng.standard_normal((T, (Hq + 2 * Hkv) * D))).to(dt).cuda()
    q, k, v = (t.view(T, -1, D) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    NB = -(-T // bs) + spare
    w = [torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).to(dt).cuda() if norm else None for _ in range(2)]
    angle = rng.uniform(-3, 3, (500, max(rot, 1) // 2))
    cs = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    scales = [torch.from_numpy(rng.uniform(0.05, 0.6, (Hkv, D // group)).astype(np.float32)).cuda() for _ in range(2)]
    caches = [torch.from_numpy(rng.integers(0, 256, (NB, bs, Hkv, D // 2), dtype=np.uint8)).cuda() for _ in range(2)]
    slots = rng.permutation(NB * bs)[:T].astype(np.int64)
    pos = rng.integers(0, 500, T).astype(np.int32)
    return dict(q=q, k=k, v=v, w=w, cs=cs, scales=scales, caches=caches, slots=slots, pos=pos)


def verify_codes(got, before, x, slots, scales, err):
    """got and before: codes [slots, H, D]; x [T, H, D] float64 written to slots >= 0; err: how far the kernel's
    value may be from x.  A code is the rounding of some value within err of x."""
    used = slots >= 0
    rest = np.ones(len(got), bool)
    rest[slots[used]] = False
    assert np.array_equal(got[rest], before[rest]), "other slots changed"
    step = np.repeat(scales.cpu().numpy().astype(np.float64), 128 // scales.shape[1], 1)
    e = np.broadcast_to(err, x.shape)[used] / step + np.abs(x[used] / step) * 2.0 ** -23  # and the division's rounding
    lo = np.clip(np.rint(x[used] / step - e), -8, 7)
    hi = np.clip(np.rint(x[used] / step + e), -8, 7)
    g = got[slots[used]]
    assert ((g >= lo) & (g <= hi)).all()
    return float((lo != hi).mean())


@pytest.mark.parametrize("T", [1, 2, 37, 700])
@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (8, 1), (7, 7), (64, 8)])
@pytest.mark.parametrize("dt,bs,group,rot,inter,norm", [
    (BF16, 16, 32, 128, False, True), (F16, 8, 8, 128, True, True), (BF16, 32, 128, 64, False, False),
    (F16, 16, 16, 32, True, True), (BF16, 4, 64, 16, False, True), (F16, 16, 32, 0, False, True)])
def test_append(kv, T, Hq, Hkv, dt, bs, group, rot, inter, norm):
    s = inputs(T + Hq, T, Hq, Hkv, dt, bs, group, rot, norm)
    slots = s["slots"].copy()
    slots[T // 2:T // 2 + T // 9] = -1
    before = [codes(c) for c in s["caches"]]
    pos, cs = torch.from_numpy(s["pos"]).cuda(), torch.from_numpy(s["cs"]).cuda() if rot else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k_out = torch.empty((T, Hkv, 128), dtype=dt, device="cuda")
    q = kv.qk_norm_rope_and_cache_int4(s["q"], s["k"], s["v"], pos, cs, torch.from_numpy(slots).cuda(), *s["caches"], *s["scales"],
                                       *s["w"], 1e-5, inter, k_out=k_out, d_err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    # queries and the 16-bit keys are those of the call without a cache
    q2, k2 = kv.qk_norm_rope(s["q"], s["k"], pos, cs, *s["w"], 1e-5, inter)
    assert torch.equal(q, q2) and torch.equal(k_out, k2)
    y, size = R.norm_rope(f64(s["k"]), None if s["w"][1] is None else f64(s["w"][1]), 1e-5, s["pos"], s["cs"], rot, inter)
    e32 = R.norm_rope_bound(y, size, 128, dt) - R.HALF[dt] * np.abs(y) - R.TINY[dt]
    near = verify_codes(codes(s["caches"][0]), before[0], y, slots, s["scales"][0], e32)
    assert near < 1e-3, "the bound leaves few codes open"
    verify_codes(codes(s["caches"][1]), before[1], f64(s["v"]), slots, s["scales"][1], 0.0)


def test_without_norm_and_rotation_it_is_the_cache_write(kv):
    s = inputs(3, 100, 8, 4, BF16, 16, 32, 0, False)
    slots = torch.from_numpy(s["slots"]).cuda()
    # values in the middle of two codes, infinities and NaN among them
    step = s["scales"][0].repeat_interleave(32, 1)
    half = (torch.arange(-20, 20, device="cuda").view(-1, 1, 1) + 0.5) * step
    s["k"][:40] = half.to(BF16)
    s["v"][3, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 3e38])
    s["k"][50, 1, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), -3e38])
    other = [c.clone() for c in s["caches"]]
    kv.reshape_and_cache_int4(s["k"], s["v"], slots, *other, *s["scales"])
    kv.qk_norm_rope_and_cache_int4(s["q"], s["k"], s["v"], None, None, slots, *s["caches"], *s["scales"])
    for a, b in zip(s["caches"], other):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("seed", [0, 1])
def test_codes_of_any_scale_are_those_of_the_cache_write(kv, dt, seed):
    """Without norm and rotation every code is that of the quotient's two roundings: scales of any size (0, the
    smallest and largest numbers, infinity, NaN, negative ones), values at and next to the middle of two codes."""
    rng = np.random.default_rng(seed)
    T, H, D, bs = 400, 16, 128, 16
    NB = T // bs
    with np.errstate(over="ignore"):
        scales = (rng.uniform(1, 2, (2, H, D // 8)) * 2.0 ** rng.integers(-149, 128, (2, H, D // 8))).astype(np.float32)
    scales[:, 8:] = rng.uniform(0.01, 2.0, (2, H - 8, D // 8))
    scales[:, 0, :8] = [0.0, -0.0, np.inf, np.nan, 1e-45, 3e38, -0.5, -1e-40]
    wide = np.repeat(scales.astype(np.float64), 8, 2)[:, None]
    with np.errstate(all="ignore"):
        x = np.where(rng.random((2, T, H, D)) < 0.7, rng.integers(-10, 10, (2, T, H, D)) + 0.5, rng.uniform(-10, 10, (2, T, H, D))) * wide
        x *= np.where(rng.random(x.shape) < 0.5, 1.0, 1 + rng.integers(-3, 4, x.shape) * 2.0 ** -8)
    x[:, 0] = [np.inf, -np.inf, np.nan, 0.0, -0.0, 6e-8, 65504.0, -65504.0] * 16
    k, v = (torch.from_numpy(y).to(dt).cuda() for y in x)
    sc = [torch.from_numpy(y).cuda() for y in scales]
    slots = torch.from_numpy(rng.permutation(T)).cuda()
    caches = [torch.zeros((NB, bs, H, D // 2), dtype=torch.uint8, device="cuda") for _ in range(4)]
    kv.reshape_and_cache_int4(k, v, slots, *caches[:2], *sc)
    kv.qk_norm_rope_and_cache_int4(k, k, v, None, None, slots, *caches[2:], *sc)
    for a, b in zip(caches[:2], caches[2:]):
        assert torch.equal(a, b)


def test_padding_bad_positions_and_slots(kv):
    s = inputs(4, 30, 8, 2, BF16, 16, 32, 128, True)
    pos, slots = s["pos"].copy(), s["slots"].copy()
    pos[3], pos[7] = -1, 500          # padding; past the table
    slots[5], slots[9] = -1, s["caches"][0].shape[0] * 16
    before = [codes(c) for c in s["caches"]]
    q_out = torch.full((30, 8, 128), 7.0, dtype=BF16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.qk_norm_rope_and_cache_int4(s["q"], s["k"], s["v"], torch.from_numpy(pos).cuda(), torch.from_numpy(s["cs"]).cuda(),
                                   torch.from_numpy(slots).cuda(), *s["caches"], *s["scales"], *s["w"], q_out=q_out, d_err=err)
    assert int(err) == kv.KV_DERR_BAD_POS | kv.KV_DERR_BAD_SLOT
    assert (q_out[[3, 7]] == 7).all() and not (q_out[[5, 9]] == 7).all(-1).any()
    skip = slots.copy()
    skip[[3, 5, 7, 9]] = -1
    y, size = R.norm_rope(f64(s["k"]), f64(s["w"][1]), 1e-6, np.clip(pos, 0, 499), s["cs"], 128, False)
    e32 = R.norm_rope_bound(y, size, 128, BF16) - R.HALF[BF16] * np.abs(y) - R.TINY[BF16]
    verify_codes(codes(s["caches"][0]), before[0], y, skip, s["scales"][0], e32)
    verify_codes(codes(s["caches"][1]), before[1], f64(s["v"]), skip, s["scales"][1], 0.0)


def test_no_tokens(kv):
    s = inputs(5, 1, 8, 2, BF16, 16, 32, 128, True)
    cut = {k: s[k][:0] for k in "qkv"}
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    q = kv.qk_norm_rope_and_cache_int4(cut["q"], cut["k"], cut["v"], empty, torch.from_numpy(s["cs"]).cuda(), empty.long(),
                                       *s["caches"], *s["scales"], *s["w"])
    assert q.shape == (0, 8, 128)


def test_steps_over_an_int4_cache(kv):
    """Append and decode with sinks, step after step, against attention over the codes that the appends left."""
    Hq, Hkv, D, bs, window, sinks, B = 8, 2, 128, 16, 40, 3, 4
    rng = np.random.default_rng(6)
    start = np.array([0, 17, 90, 130])
    x = Inputs(7, start, [16] * B, Hq, Hkv, D, bs, window, sinks, "int4", release=False)
    d = x.device()
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).to(BF16).cuda()
    angle = np.arange(200)[:, None] * 10000.0 ** (-np.arange(0, D, 2) / D)
    cs = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()
    lens = start.copy()
    for n in (1, 4, 1, 8, 2):
        qkv = torch.from_numpy(rng.standard_normal((B * n, (Hq + 2 * Hkv) * D))).to(BF16).cuda()
        q, k, v = (t.view(B * n, -1, D) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
        pos = torch.from_numpy((lens[:, None] + np.arange(n)).reshape(-1).astype(np.int32)).cuda()
        qsl = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
        lens = lens + n
        dl = torch.from_numpy(lens.astype(np.int32)).cuda()
        slots = kv.compute_slot_mapping(d["table"], qsl, pos, bs, x.NB)
        q = kv.qk_norm_rope_and_cache_int4(q, k, v, pos, cs, slots, d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"], w, w)
        out = kv.paged_attention_decode_sinks_int4(q, d["k_cache"], d["v_cache"], d["table"], dl, 256, n, D ** -0.5, d["k_scales"],
                                                   d["v_scales"], window, sinks)
        x.q, x.k_cache, x.v_cache = q.cpu(), d["k_cache"].cpu(), d["v_cache"].cpu()
        x.lens, x.qsl = lens.astype(np.int32), qsl.cpu().numpy()
        r = x.reference()
        check(out, r["out"], x.bounds(r, rounded_sum=True)[0], f"{n} tokens")
