"""Plain 64-bit implementations of the step's operators (batch metadata, query/key norm with
rotation, tree attention) and the error bounds the tests hold the kernels to.  They share no code
with the library."""
from __future__ import annotations

import numpy as np
import torch

# half a rounding step relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float8_e4m3fn: 2.0 ** -4}
# half the spacing of the smallest values (below the normal range)
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float8_e4m3fn: 2.0 ** -10}


# ------------------------------------------------------------------ batch metadata

def build_batch(ctx, new, held, table, free, num_tokens, bs, num_blocks, parents=None, start=0, width=None):
    """Request by request.  Returns a dict of the outputs and the error bits."""
    B = len(ctx)
    width = table.shape[1] if width is None else width
    table = table.copy()
    err = 0
    avail = len(free) - start if 0 <= start <= len(free) else 0
    qsl, lens, held_out = [0], [], []
    positions = np.full(num_tokens, -1, np.int32)
    slots = np.full(num_tokens, -1, np.int64)
    masks = [0] * num_tokens
    wanted = used = 0
    end = 0
    for r in range(B):
        c, n = int(ctx[r]), int(new[r])
        h = int(held[r]) if held is not None else -(-max(c, 0) // bs)
        total = -(-(c + n) // bs)
        t0 = end
        end += max(n, 0)
        ok = c >= 0 and n >= 0 and 0 <= h <= width and total <= width and not (parents is not None and n > 64)
        if n > 0 and end > num_tokens:
            ok = False
        if not ok:
            err |= 16
        need = max(0, total - h) if ok and n > 0 else 0
        wanted += need
        if ok and need and wanted > avail:
            ok, err = False, err | 128
        if ok:
            first = used
            for k in range(need):
                b = int(free[start + used])
                used += 1
                if 0 <= b < num_blocks:
                    table[r, h + k] = b
                else:
                    err |= 2 ** 0
            word, depth = [], []
            for i in range(n):
                lb = (c + i) // bs
                b = int(table[r, lb]) if lb < h else int(free[start + first + lb - h])
                if 0 <= b < num_blocks:
                    slots[t0 + i] = b * bs + (c + i) % bs
                else:
                    err |= 1
                p = -1
                if parents is not None:
                    p = int(parents[t0 + i])
                    if not -1 <= p < i:
                        p, err = -1, err | 256
                    word.append((1 << i) | (word[p] if p >= 0 else 0))
                    depth.append(depth[p] + 1 if p >= 0 else 0)
                    masks[t0 + i] = word[i]
                positions[t0 + i] = c + (i if parents is None else depth[i])
        qsl.append(min(end, num_tokens))
        lens.append(c + n if ok else 0)
        held_out.append(h + need if ok else h)
    return dict(query_start_loc=np.array(qsl, np.int32), seq_lens=np.array(lens, np.int32), positions=positions,
                slot_mapping=slots, held_blocks=np.array(held_out, np.int32), free_next=np.array([start + used], np.int32),
                tree_mask=None if parents is None else np.array(masks, np.uint64).view(np.int64), block_table=table), err


# ------------------------------------------------------------------ norm and rotation

def norm_rope(x, weight, eps, positions, cos_sin, rot, interleaved):
    """x [T, H, D] float64 -> (y, size): size bounds |a| + |b| of each dim's pair before the turn."""
    T, H, D = x.shape
    y = x.copy()
    if weight is not None:
        y = y / np.sqrt((y * y).sum(-1, keepdims=True) / D + eps) * weight
    size = np.abs(y)
    if rot:
        half = rot // 2
        cs = cos_sin[positions].astype(np.float64)
        cos, sin = cs[:, None, :half], cs[:, None, half:rot]
        ia = np.arange(0, rot, 2) if interleaved else np.arange(half)
        ib = ia + 1 if interleaved else ia + half
        a, b = y[..., ia].copy(), y[..., ib].copy()
        y[..., ia], y[..., ib] = a * cos - b * sin, b * cos + a * sin
        size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return y, size


def norm_rope_bound(y, size, D, dtype):
    """One rounding of the result, and float32 before it: the sum of D squares (relative error at
    most (D / 8 + 5) 2^-24 as eight chains of 8 joined by shuffles; taken as D 2^-24), halved by the
    root, the root itself (2 units), three products, two products and a sum of the turn."""
    e32 = (D / 2 + 10) * 2.0 ** -24
    err = e32 * size
    return err + HALF[dtype] * (np.abs(y) + err) + TINY[dtype]


# ------------------------------------------------------------------ tree attention

def seen_keys(mask, n, ctx, window):
    """bool [n, ctx + n]: the keys each row sees."""
    seen = np.zeros((n, ctx + n), bool)
    for i in range(n):
        bits = np.array([(int(mask[i]) >> j) & 1 for j in range(n)], bool)
        seen[i, ctx:] = bits
        lo = ctx - 1 + int(bits.sum()) - window + 1 if window else 0
        seen[i, max(0, lo):ctx] = True
    return seen


def tree_attention(q, k_cache, v_cache, table, lens, qsl, masks, scale, window=0):
    """q [T, Hq, D], caches [NB, bs, Hkv, D]: float64 arrays.  Returns out, lse, and the bounds'
    ingredients: A = sum p |v| (per output) and smax = max |q|.|k| scale over the row's keys."""
    T, Hq, D = q.shape
    NB, bs, Hkv, _ = k_cache.shape
    g = Hq // Hkv
    out = np.zeros((T, Hq, D))
    size = np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    smax = np.zeros((T, Hq))
    kf, vf = k_cache.reshape(NB * bs, Hkv, D), v_cache.reshape(NB * bs, Hkv, D)
    masks = np.asarray(masks).view(np.uint64)
    for b in range(len(lens)):
        t0, t1 = int(qsl[b]), int(qsl[b + 1])
        n, L = t1 - t0, int(lens[b])
        if n == 0:
            continue
        seen = seen_keys(masks[t0:t1], n, L - n, window)
        pos = np.arange(L)
        slots = np.maximum(table[b, pos // bs].astype(np.int64), 0) * bs + pos % bs
        for i in range(n):
            at = slots[seen[i]]
            if len(at) == 0:
                continue
            for h in range(Hkv):
                K, V = kf[at, h], vf[at, h]
                Q = q[t0 + i, h * g:(h + 1) * g]
                s = Q @ K.T * scale
                m = s.max(1, keepdims=True)
                p = np.exp(s - m)
                l = p.sum(1, keepdims=True)
                rows = slice(h * g, (h + 1) * g)
                out[t0 + i, rows] = p @ V / l
                size[t0 + i, rows] = p @ np.abs(V) / l
                lse[t0 + i, rows] = (m + np.log(l))[:, 0]
                smax[t0 + i, rows] = (np.abs(Q) @ np.abs(K).T * abs(scale)).max(1)
    return out, lse, size, smax


def tree_bounds(out, lse, size, smax, D, dtype):
    """Bounds of the kernel's error.  The scores are float32 sums of D exact products, each addition
    off by at most 2^-23 of the sum of magnitudes; exp2, the sums and the merge of pieces add about
    2^-20 to a weight's relative error.  The weights are rounded to the 16-bit type for the second
    product: half a step of the weighted mean of |v|, and as much again when the normaliser sums the
    rounded weights (the kernels' sums the weights before it).  The result is rounded once."""
    u = HALF[dtype]
    e32 = (D * 2.0 ** -23 * smax + 2.0 ** -20)
    acc = (2 * e32[..., None] + 2 * u) * size
    lse_tol = e32 + np.abs(np.where(np.isfinite(lse), lse, 0)) * 2.0 ** -21
    return acc + u * (np.abs(out) + acc) + TINY[dtype], lse_tol


# ------------------------------------------------------------------ trees

def random_parents(rng, n):
    p = np.full(n, -1, np.int64)
    for i in range(1, n):
        p[i] = rng.integers(-1, i) if rng.random() < 0.4 else i - 1
    return p


def masks_of(parents):
    words = []
    for i, p in enumerate(parents):
        words.append((1 << i) | (words[p] if p >= 0 else 0))
    return words
