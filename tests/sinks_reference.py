"""Plain 64-bit implementation of attention with a sliding window and sinks over a paged cache (16-bit,
E4M3 and INT4), the inputs its tests use, and the error bounds they hold the kernels to.  It shares no
code with the library."""
from __future__ import annotations

import numpy as np
import torch

from tests.step_reference import HALF, TINY

BF16, F16 = torch.bfloat16, torch.float16


def seen_keys(p, window, sinks):
    """The keys that the row at position p sees, in order."""
    j = np.arange(p + 1)
    return j if window == 0 else j[(j > p - window) | (j < sinks)]


def attention(q, K, V, table, lens, qsl, scale, window, sinks):
    """q [T, Hq, D], K and V [NB, bs, Hkv, D] float64, in the values that the codes stand for.  Returns out, lse,
    A = sum p |v|, smax = max over a row's keys of |q|.|k| scale, kmax = max |k| scale, n = number of keys."""
    T, Hq, D = q.shape
    NB, bs, Hkv, _ = K.shape
    g = Hq // Hkv
    out, size = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, smax, n = np.full((T, Hq), -np.inf), np.zeros((T, Hq)), np.zeros((T, 1))
    kf, vf = K.reshape(NB * bs, Hkv, D), V.reshape(NB * bs, Hkv, D)
    for b in range(len(lens)):
        t0, t1, L = int(qsl[b]), int(qsl[b + 1]), int(lens[b])
        for t in range(t0, t1):
            keys = seen_keys(L - (t1 - t), window, sinks)
            blocks = table[b, keys // bs].astype(np.int64)
            keys = keys[blocks >= 0]
            at = blocks[blocks >= 0] * bs + keys % bs
            n[t] = len(at)
            if len(at) == 0:
                continue
            for h in range(Hkv):
                k, v, Q, rows = kf[at, h], vf[at, h], q[t, h * g:(h + 1) * g], slice(h * g, (h + 1) * g)
                with np.errstate(invalid="ignore", over="ignore"):
                    s = Q @ k.T * scale
                    m = s.max(1, keepdims=True)
                    p = np.exp(s - m)
                    l = p.sum(1, keepdims=True)
                    out[t, rows] = p @ v / l
                    size[t, rows] = p @ np.abs(v) / l
                    lse[t, rows] = (m + np.log(l))[:, 0]
                    smax[t, rows] = (np.abs(Q) @ np.abs(k).T * abs(scale)).max(1)
    return dict(out=out, lse=lse, size=size, smax=smax, n=n)


def bounds(r, D, dtype, cache, scale, coded=0.0, vcoded=0.0, shift=14, rounded_sum=False):
    """Bounds of the kernel's error in out and lse.

    Scores are float32 sums of D exact products, each addition off by at most 2^-23 of the sum of the
    magnitudes; exp2, the sums and the merge of pieces add 2^-20 to a weight's relative error.  Over E4M3 and
    INT4 caches the products are fp16: queries are rounded to it (E4M3: exact but for the smallest, off by at most
    2^-25; INT4: q * scale, 2^-11 of each product), and INT4 codes are summed with an offset of 8 that is taken out
    again, so that float32 works on magnitudes of up to `coded` (scores) and `vcoded` (values).
    The weights are rounded for the second product: half a step of the weighted mean of |v|, as much again
    for a normaliser that sums the rounded ones, and below the fp16 range (2^-25 of 2^shift times a weight) an
    absolute one.  The result is rounded once."""
    wide = cache in ("e4m3", "int4")
    u = HALF[F16] if wide else HALF[dtype]
    smax = r["smax"]
    e = D * 2.0 ** -23 * np.maximum(smax, coded) + 2.0 ** -20
    if cache == "e4m3":
        e = e + D * 2.0 ** -25 * abs(scale) * 8
    if cache == "int4":
        e = e + 2.0 ** -11 * smax
    n = r["n"]
    lost = n * 2.0 ** (-25 - shift) if u == HALF[F16] else 0.0
    acc = (2 * e[..., None] + 2 * u + 2 * lost[..., None] if u == HALF[F16] else 2 * e[..., None] + 2 * u) * r["size"]
    if cache == "int4":
        acc = acc + (2.0 ** -19) * vcoded
    if u == HALF[F16]:  # a lost weight counts by its value, which may be far above the mean
        acc = acc + lost[..., None] * r.get("vmax", 0.0)
    lse = np.where(np.isfinite(r["lse"]), r["lse"], 0)
    lse_tol = e + np.abs(lse) * 2.0 ** -21 + (u if rounded_sum else 0.0)
    return acc + HALF[dtype] * (np.abs(r["out"]) + acc) + TINY[dtype], lse_tol


class Inputs:
    """A batch over a paged cache: sequences of `ctx` cached and `new` new tokens, blocks in a random order, and the
    blocks that no row sees released (-1), their contents and those of spare blocks NaN where the type has it."""

    def __init__(self, seed, ctx, new, Hq=8, Hkv=2, D=128, bs=16, window=0, sinks=0, cache="same", dtype=BF16, group=32,
                 release=True, spare=3):
        rng = np.random.default_rng(seed)
        self.Hq, self.Hkv, self.D, self.bs, self.window, self.sinks = Hq, Hkv, D, bs, window, sinks
        self.cache, self.dtype, self.group, self.scale = cache, dtype, group, D ** -0.5
        ctx, new = np.asarray(ctx), np.asarray(new)
        self.new, self.lens = new.astype(np.int32), (ctx + new).astype(np.int32)
        self.qsl = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        nblk = -(-self.lens // bs)
        logical = np.arange(int(nblk.max(initial=0)) + 1)[None]
        first = np.maximum(ctx - window + 1, 0) // bs if window else np.zeros_like(ctx)
        live = logical < nblk[:, None]
        if release:
            live &= (logical >= first[:, None]) | (logical * bs < sinks)
        self.NB = int(live.sum()) + spare
        self.table = np.full(live.shape, -1, np.int32)
        ids = rng.permutation(self.NB).astype(np.int32)
        self.table[live] = ids[:int(live.sum())]
        self.q = torch.from_numpy(rng.standard_normal((int(self.qsl[-1]), Hq, D))).to(dtype)
        shape = (self.NB, bs, Hkv, D)
        self.k_scale = self.v_scale = 1.0
        self.k_scales = self.v_scales = None
        self.vcoded = np.zeros((1, 1, 1))
        if cache == "int4":
            self.k_cache = torch.from_numpy(rng.integers(0, 256, (self.NB, bs, Hkv, D // 2), dtype=np.uint8))
            self.v_cache = torch.from_numpy(rng.integers(0, 256, (self.NB, bs, Hkv, D // 2), dtype=np.uint8))
            self.k_scales = torch.from_numpy(rng.uniform(0.1, 0.5, (Hkv, D // group)).astype(np.float32))
            self.v_scales = torch.from_numpy(rng.uniform(0.1, 0.5, (Hkv, D // group)).astype(np.float32))
        else:
            if cache == "e4m3":
                self.k_scale, self.v_scale = 0.75, 1.25
            k, v = rng.standard_normal(shape), rng.standard_normal(shape)
            k[ids[int(live.sum()):]] = v[ids[int(live.sum()):]] = np.nan  # spare blocks
            # what lies behind a sequence's end in its last block
            for b, L in enumerate(self.lens):
                if L % bs:
                    k[self.table[b, L // bs], L % bs:] = v[self.table[b, L // bs], L % bs:] = np.nan
            to = torch.float8_e4m3fn if cache == "e4m3" else dtype
            self.k_cache = torch.from_numpy(k).float().to(to)
            self.v_cache = torch.from_numpy(v).float().to(to)

    def slot(self, b, pos):
        """Where position pos of sequence b lies: (block, offset)."""
        return int(self.table[b, pos // self.bs]), pos % self.bs

    def values(self, which):
        """The cache as float64 values."""
        c = getattr(self, which + "_cache")
        if self.cache == "int4":
            x = c.numpy().astype(np.int64)
            code = np.stack([x & 15, x >> 4], -1).reshape(*x.shape[:-1], self.D)
            code = np.where(code > 7, code - 16, code)
            return code * np.repeat(getattr(self, which + "_scales").numpy().astype(np.float64), self.group, 1)
        return c.float().numpy().astype(np.float64) * getattr(self, which + "_scale")

    def reference(self):
        return attention(self.q.double().numpy(), self.values("k"), self.values("v"), self.table, self.lens, self.qsl,
                         self.scale, self.window, self.sinks)

    def bounds(self, r, shift=14, rounded_sum=False):
        coded = vcoded = 0.0
        if self.cache == "int4":
            g = self.Hq // self.Hkv
            ks = np.repeat(self.k_scales.numpy().astype(np.float64), self.group, 1)
            vs = np.repeat(self.v_scales.numpy().astype(np.float64), self.group, 1)
            coded = (np.abs(self.q.double().numpy()) * np.repeat(ks, g, 0)).sum(-1) * 15 * abs(self.scale)
            vcoded = 15 * np.repeat(vs, g, 0)[None]
        with np.errstate(invalid="ignore"):
            v = np.abs(self.values("v"))
            r["vmax"] = float(np.max(v[np.isfinite(v)], initial=0.0))
        return bounds(r, self.D, self.dtype, self.cache, self.scale, coded, vcoded, shift, rounded_sum)

    def device(self):
        """The tensors on the GPU, by the names of the calls' arguments."""
        d = {k: torch.from_numpy(getattr(self, k)).cuda() for k in ("table", "lens", "qsl")}
        for k in ("q", "k_cache", "v_cache", "k_scales", "v_scales"):
            t = getattr(self, k)
            d[k] = None if t is None else t.cuda()
        return d


def check(got, want, tol, what):
    """Every finite value within its bound, NaN and infinities in the same places."""
    got = got.double().cpu().numpy()
    for name, mask in (("NaN", np.isnan), ("infinities", np.isinf)):
        assert np.array_equal(mask(got), mask(want)), f"{what}: {name} elsewhere"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities of another sign"
    fine = np.isfinite(want)
    tol = np.broadcast_to(tol, want.shape)
    over = np.abs(got[fine] - want[fine]) / tol[fine]
    assert over.size == 0 or over.max() <= 1, f"{what}: {over.max():.3g} times its bound"
    return float(over.max(initial=0.0))
