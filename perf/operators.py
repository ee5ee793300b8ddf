"""Timed cases of the operators around one speculative decode step, with their plain forms.

  batch  block tables, slot maps, positions and tree masks of a step, from request lengths
  rope   RMS norm of every query and key head, rotary embedding, write into the paged cache
  tree   attention of a tree of drafted tokens over the paged cache

``run`` computes an operator in elementary torch operations, or (``own``) through the library.
``exact`` is the operator's definition in 64 bits, written apart from the plain form.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one request, one new token: what a single user waits for
        dict(name="batch_one", op="batch", seqs=1, kind="decode", ctx=1117, new=1, block=16, lens=1),
        # a decode step of the Llama-3-8B-shaped batch: 256 requests of up to 8192 tokens
        dict(name="batch_decode", op="batch", seqs=256, kind="decode", ctx=8192, new=1, block=16, lens=2),
        # drafted trees of up to 64 tokens for 128 requests
        dict(name="batch_trees", op="batch", seqs=128, kind="tree", ctx=4096, new=64, block=16, lens=3),
        # admission of 512 prompts of up to 2048 tokens (a long prefill step)
        dict(name="batch_prompts", op="batch", seqs=512, kind="chunk", ctx=0, new=2048, block=32, lens=4),
        # one token of the Llama-3-8B shape
        dict(name="rope_one", op="rope", tokens=1, q_heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, norm=True, cache="same", dtype="bf16", block=16),
        # a decode batch of the Llama-70B shape into an E4M3 cache
        dict(name="rope_decode_fp8", op="rope", tokens=256, q_heads=64, kv_heads=8, dim=128, rotary=128,
             interleaved=False, norm=True, cache="e4m3", dtype="bf16", block=16),
        # an odd-sized prompt of the OPT-125m shape, half of each head rotated in adjacent pairs
        dict(name="rope_prompt_d64", op="rope", tokens=4099, q_heads=12, kv_heads=12, dim=64, rotary=32,
             interleaved=True, norm=True, cache="none", dtype="f16", block=16),
        # 16 chunks of 1024 tokens of the Llama-70B shape
        dict(name="rope_prompts", op="rope", tokens=16384, q_heads=64, kv_heads=8, dim=128, rotary=128,
             interleaved=False, norm=True, cache="same", dtype="bf16", block=16),
        # one request's tree of 7 drafted tokens after 1117
        dict(name="tree_one", op="tree", seqs=1, ctx=1117, spread="fixed", new=7, q_heads=32, kv_heads=8,
             dim=128, block=16, window=0, dtype="bf16", lens=5),
        # 64 requests of the OPT-125m shape, ragged trees of up to 24 tokens
        dict(name="tree_opt125m", op="tree", seqs=64, ctx=2048, spread="uniform", new=24, q_heads=12,
             kv_heads=12, dim=64, block=16, window=0, dtype="f16", lens=6),
        # a sliding-window layer of the Mistral-shaped batch: log-normal lengths up to 32768
        dict(name="tree_window", op="tree", seqs=128, ctx=32768, spread="lognormal", new=16, q_heads=32,
             kv_heads=8, dim=128, block=16, window=4096, dtype="bf16", lens=7),
        # wide trees of the Llama-70B shape: up to 512 query rows a kv head over long contexts
        dict(name="tree_wide", op="tree", seqs=32, ctx=8192, spread="uniform", new=64, q_heads=64,
             kv_heads=8, dim=128, block=16, window=0, dtype="bf16", lens=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("batch", "rope", "tree", "tree"))
    if op == "batch":
        kind = rng.choice(("decode", "tree", "chunk"))
        seqs = _log(rng, 1, 512)
        new = {"decode": 1, "tree": rng.randint(1, 64), "chunk": _log(rng, 2, 1800)}[kind]
        return dict(op=op, seqs=seqs, kind=kind, ctx=0 if rng.random() < 0.1 else _log(rng, 1, 8000), new=new,
                    block=rng.choice((8, 16, 32)), lens=rng.randint(0, 1 << 20))
    if op == "rope":
        q_heads, kv_heads, dim = rng.choice(((32, 8, 128), (64, 8, 128), (12, 12, 64), (28, 4, 128), (8, 1, 256),
                                             (71, 1, 64), (40, 8, 96), (16, 16, 80)))
        tokens = _log(rng, 1, 12000)
        while tokens * (q_heads + 2 * kv_heads) * dim > 16384 * 80 * 128:
            tokens = tokens * 2 // 3
        # the attention over E4M3 caches takes 128 dims; any head size can be written in the 16-bit type
        cache = rng.choice(("none", "same", "e4m3") if dim == 128 else ("none", "same"))
        return dict(op=op, tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    rotary=rng.choice((dim, dim, 16 * max(1, dim // 32))), interleaved=rng.random() < 0.3,
                    norm=rng.random() < 0.8, cache=cache, dtype=rng.choice(("bf16", "f16")),
                    block=rng.choice((8, 16, 32)))
    q_heads, kv_heads, dim = rng.choice(((32, 8, 128), (64, 8, 128), (12, 12, 64), (28, 4, 128), (16, 1, 128),
                                         (8, 8, 128), (40, 8, 64), (5, 1, 64)))
    case = dict(op="tree", seqs=_log(rng, 1, 96), ctx=_log(rng, 1, 8100),
                spread=rng.choice(("fixed", "uniform")), new=rng.randint(1, 64), q_heads=q_heads,
                kv_heads=kv_heads, dim=dim, block=rng.choice((8, 16, 32)),
                window=rng.choice((0, 0, 0, 100, 1024, 4096)), dtype=rng.choice(("bf16", "f16")),
                lens=rng.randint(0, 1 << 20))
    while case["seqs"] * (case["ctx"] + case["new"]) * kv_heads > 32 * 5000 * 8:
        case["seqs"] = case["seqs"] * 2 // 3
    return case


# The lengths of a case go by the case alone (so that its work is known); a seed changes their order.

def _tree_lens(case):
    rng = np.random.default_rng(case["lens"])
    B, ctx = case["seqs"], case["ctx"]
    if case["spread"] == "uniform":
        c = rng.integers(max(0, ctx // 16), ctx + 1, B)
    elif case["spread"] == "lognormal":
        c = np.clip(np.exp(rng.normal(math.log(2048), 1.0, B)).astype(np.int64), 1, ctx)
    else:
        c = np.full(B, ctx)
    n = rng.integers(max(1, case["new"] // 2), case["new"] + 1, B) if B > 1 else np.full(1, case["new"])
    return c.astype(np.int64), n.astype(np.int64)


def _batch_lens(case):
    rng = np.random.default_rng(case["lens"])
    B = case["seqs"]
    c = rng.integers(case["ctx"] // 16, case["ctx"] + 1, B) if B > 1 else np.full(1, case["ctx"])
    n = np.full(B, case["new"]) if case["kind"] == "decode" or B == 1 else rng.integers(max(1, case["new"] // 16), case["new"] + 1, B)
    return c.astype(np.int64), n.astype(np.int64)


def _parents(rng, n):
    """A drafted tree of n tokens in the order they were drafted: mostly extends recent tokens."""
    p = np.full(n, -1, np.int64)
    for i in range(1, n):
        p[i] = i - 1 - min(i, int(rng.geometric(0.45)) - 1)
    return p


def _ancestors(p):
    masks = []
    for i, a in enumerate(p):
        masks.append((1 << i) | (masks[a] if a >= 0 else 0))
    return np.array(masks, np.uint64).view(np.int64)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    return {"batch": _prepare_batch, "rope": _prepare_rope, "tree": _prepare_tree}[case["op"]](case, seed)


def _prepare_batch(case, seed):
    rng = np.random.default_rng([seed, 11])
    bs = case["block"]
    ctx, new = _batch_lens(case)
    order = rng.permutation(len(ctx))
    ctx, new = ctx[order], new[order]
    held = -(-ctx // bs)
    if case["kind"] == "tree":  # blocks left over from the last tree's rejected tokens
        held = held + rng.integers(0, 3, len(ctx))
    total = -(-(ctx + new) // bs)
    need = np.maximum(total - held, 0)
    width = int(max(total.max(), held.max())) + 1
    num_blocks = int(held.sum() + need.sum()) + 9
    ids = rng.permutation(num_blocks).astype(np.int32)
    table = np.full((len(ctx), width), -1, np.int32)
    table[np.arange(width)[None, :] < held[:, None]] = ids[:held.sum()]
    free = ids[held.sum():]
    tokens = int(new.sum()) + 5  # a padded batch: five rows behind the last request
    s = dict(op="batch", block=bs, num_blocks=num_blocks, tokens=tokens, parents=None)
    for k, v in (("ctx", ctx), ("new", new), ("held", held), ("table", table), ("free", free)):
        s[k] = torch.from_numpy(v.astype(np.int32)).cuda()
    if case["kind"] == "tree":
        par = np.full(tokens, -1, np.int64)
        par[:new.sum()] = np.concatenate([_parents(rng, int(n)) for n in new])
        s["parents"] = torch.from_numpy(par.astype(np.int32)).cuda()
    if own:
        from paged_kv_cache_block_gb300 import kvcache as kv
        s["out"] = kv.batch_buffers(len(ctx), tokens, s["parents"] is not None)
    return s


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _prepare_rope(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    T, Hq, Hkv, D, rot, bs = (case[k] for k in ("tokens", "q_heads", "kv_heads", "dim", "rotary", "block"))
    dt = DTYPES[case["dtype"]]
    # the rows of one packed projection; query, key and value are views of it
    qkv = _normal(gen, (T, (Hq + 2 * Hkv) * D), dt)
    q, k, v = (x.view(T, -1, D) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1))
    s = dict(op="rope", q=q, k=k, v=v, rotary=rot, interleaved=case["interleaved"], eps=1e-6, wq=None, wk=None,
             cache=case["cache"], block=bs)
    if case["norm"]:
        s["wq"] = (1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dt)
        s["wk"] = (1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dt)
    max_pos = 32768
    s["positions"] = torch.randint(0, max_pos, (T,), generator=gen, device="cuda", dtype=torch.int32)
    inv = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    if case["cache"] != "none":
        NB = -(-T // bs) + 3
        s["slots"] = torch.randperm(NB * bs, generator=gen, device="cuda")[:T].to(torch.int64)
        s["slots"][T // 2:T // 2 + T // 50] = -1  # rows of padding
        cdt = dt if case["cache"] == "same" else torch.float8_e4m3fn
        s["k_cache"] = torch.zeros((NB, bs, Hkv, D), dtype=torch.uint8 if case["cache"] == "e4m3" else dt, device="cuda").view(cdt)
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        # calibrated: the largest normalised key of such a batch comes near 448 times its scale
        s["k_scale"], s["v_scale"] = (0.0175, 0.0131) if case["cache"] == "e4m3" else (1.0, 1.0)
    s["q_out"] = torch.empty((T, Hq, D), dtype=dt, device="cuda")
    s["k_out"] = torch.empty((T, Hkv, D), dtype=dt, device="cuda") if case["cache"] == "none" else None
    return s


def _prepare_tree(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    rng = np.random.default_rng([seed, 13])
    Hq, Hkv, D, bs = (case[k] for k in ("q_heads", "kv_heads", "dim", "block"))
    dt = DTYPES[case["dtype"]]
    ctx, new = _tree_lens(case)
    order = rng.permutation(len(ctx))
    ctx, new = ctx[order], new[order]
    L = ctx + new
    blocks = -(-L // bs)
    NB = int(blocks.sum()) + 3
    ids = rng.permutation(NB).astype(np.int32)
    table = np.full((len(L), int(blocks.max()) + 1), -1, np.int32)
    table[np.arange(table.shape[1])[None, :] < blocks[:, None]] = ids[:blocks.sum()]
    qsl = np.concatenate([[0], np.cumsum(new)])
    mask = np.concatenate([_ancestors(_parents(rng, int(n))) for n in new])
    s = dict(op="tree", block=bs, window=case["window"], scale=D ** -0.5, max_len=int(L.max()), max_new=int(new.max()))
    for k, v in (("table", table), ("lens", L.astype(np.int32)), ("qsl", qsl.astype(np.int32)), ("mask", mask)):
        s[k] = torch.from_numpy(v).cuda()
    s["q"] = _normal(gen, (int(qsl[-1]), Hq, D), dt)
    s["k_cache"] = _normal(gen, (NB, bs, Hkv, D), dt)
    s["v_cache"] = _normal(gen, (NB, bs, Hkv, D), dt)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    if own:
        from paged_kv_cache_block_gb300 import kvcache as kv
        n = kv.paged_attention_tree_workspace_size(len(L), s["max_new"], Hq, Hkv, D)
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return {"batch": _own_batch, "rope": _own_rope, "tree": _own_tree}[s["op"]](s)
    return {"batch": _plain_batch, "rope": _plain_rope, "tree": _plain_tree}[s["op"]](s)


def _own_batch(s):
    from paged_kv_cache_block_gb300 import kvcache as kv
    b = kv.build_batch(s["ctx"], s["new"], s["table"], s["free"], s["tokens"], s["block"], s["num_blocks"],
                       held_blocks=s["held"], parents=s["parents"], out=s["out"])
    return _batch_outputs(b.query_start_loc, b.seq_lens, b.positions, b.slot_mapping, b.held_blocks, b.free_next,
                          s["table"], b.tree_mask)


def _batch_outputs(qsl, lens, positions, slots, held, free_next, table, mask):
    out = dict(query_start_loc=qsl, seq_lens=lens, positions=positions, slot_mapping=slots, held_blocks=held,
               free_next=free_next, block_table=table)
    if mask is not None:
        out["tree_mask"] = mask
    return out


def _plain_batch(s):
    ctx, new, held, table, free = (s[k].long() for k in ("ctx", "new", "held", "table", "free"))
    B, bs, T, dev = len(ctx), s["block"], s["tokens"], s["ctx"].device
    end = new.cumsum(0)
    qsl = torch.cat([end.new_zeros(1), end])
    need = ((ctx + new + bs - 1) // bs - held).clamp(min=0) * (new > 0)
    taken = need.cumsum(0)
    granted = (need == 0) | (taken <= len(free))
    first = taken - need
    # table rows: columns held .. held + need - 1 take the next ids of the list
    col = torch.arange(table.shape[1], device=dev)[None, :]
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None]) & granted[:, None]
    source = (first[:, None] + col - held[:, None]).clamp(0, max(len(free) - 1, 0))
    table = torch.where(fresh, free[source], table)
    s["table"].copy_(table)
    # tokens: their request, index in it, position and slot
    t = torch.arange(T, device=dev)
    r = torch.searchsorted(end, t, right=True)
    live = r < B
    r = r.clamp(max=B - 1)
    i = t - qsl[r]
    live = live & granted[r]
    depth, mask = i, None
    if s["parents"] is not None:
        # ancestors of every token: powers of (identity + parent) over each tree's 64 places
        j = torch.arange(64, device=dev)
        at = qsl[:-1, None] + j
        inside = j < new[:, None]
        par = torch.where(inside, s["parents"].long()[at.clamp(max=T - 1)], -1)
        step = (par[:, :, None] == j) | torch.eye(64, dtype=torch.bool, device=dev)
        reach = torch.linalg.matrix_power(step.float(), 64) > 0
        word = (reach.long() << j).sum(2)
        depths = reach.sum(2) - 1
        inside_t = i.clamp(0, 63)
        depth = depths[r, inside_t]
        mask = torch.where(live, word[r, inside_t], 0)
    positions = torch.where(live, ctx[r] + depth, -1)
    index = torch.where(live, ctx[r] + i, 0)
    slots = torch.where(live, table[r, index // bs] * bs + index % bs, -1)
    held_out = torch.where(granted, held + need, held)
    free_next = torch.where(granted, taken, 0).amax().reshape(1)
    lens = torch.where(granted, ctx + new, 0)
    return _batch_outputs(qsl.int(), lens.int(), positions.int(), slots, held_out.int(), free_next.int(), s["table"], mask)


def _own_rope(s):
    from paged_kv_cache_block_gb300 import kvcache as kv
    if s["cache"] == "none":
        q, k = kv.qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], s["wq"], s["wk"], s["eps"],
                               s["interleaved"], q_out=s["q_out"], k_out=s["k_out"])
        return dict(q=q, k=k)
    q = kv.qk_norm_rope_and_cache(s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["slots"], s["k_cache"],
                                  s["v_cache"], s["wq"], s["wk"], s["eps"], s["interleaved"], s["k_scale"],
                                  s["v_scale"], q_out=s["q_out"])
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_rope(s):
    cs = s["cos_sin"][s["positions"].long()]
    cos, sin = (x[:, None, :] for x in cs.chunk(2, 1))
    rot = s["rotary"]

    def head(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
        y, rest = x[..., :rot], x[..., rot:]
        if s["interleaved"]:
            a, b = y[..., 0::2], y[..., 1::2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y.chunk(2, -1)
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, rest], -1)

    q, k = head(s["q"], s["wq"]), head(s["k"], s["wk"])
    dt = s["q"].dtype
    if s["cache"] == "none":
        return dict(q=q.to(dt), k=k.to(dt))
    slots, slots_of = s["slots"], s["k_cache"].shape[0] * s["block"]
    # rows without a slot go to one row behind the cache
    at = torch.where(slots >= 0, slots, slots_of)
    for name, x, scale in (("k_cache", k, s["k_scale"]), ("v_cache", s["v"].float(), s["v_scale"])):
        c = s[name]
        y = (x / scale).clamp(-448, 448).to(c.dtype) if s["cache"] == "e4m3" else x.to(c.dtype)
        raw = torch.uint8 if s["cache"] == "e4m3" else c.dtype
        flat = c.view(raw).view(slots_of, *c.shape[2:])
        flat.copy_(torch.cat([flat, flat[:1]]).index_put_((at,), y.view(raw))[:slots_of])
    return dict(q=q.to(dt), k_cache=s["k_cache"], v_cache=s["v_cache"])


def _own_tree(s):
    from paged_kv_cache_block_gb300 import kvcache as kv
    kv.paged_attention_tree(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["qsl"], s["mask"],
                            s["max_len"], s["max_new"], s["scale"], s["window"], workspace=s["workspace"],
                            out=s["out"], lse_out=s["lse"])
    return dict(out=s["out"], lse=s["lse"])


def _plain_tree(s):
    q, qsl, L, bs, window = s["q"], s["qsl"].long(), s["lens"].long(), s["block"], s["window"]
    Hq, D = q.shape[1:]
    NB, _, Hkv, _ = s["k_cache"].shape
    dev, B, g = q.device, len(L), Hq // Hkv
    N, new = s["max_new"], qsl[1:] - qsl[:-1]
    ctx = L - new
    span = min(s["max_len"], window + N) if window else s["max_len"]
    # the keys that some row may see, of every sequence: positions first .. first + span - 1
    first = (ctx - window).clamp(min=0) if window else torch.zeros_like(ctx)
    key = first[:, None] + torch.arange(span, device=dev)
    there = key < L[:, None]
    safe = torch.where(there, key, first[:, None])
    slot = s["table"].long().gather(1, safe // bs) * bs + safe % bs
    k, v = (c.view(NB * bs, Hkv, D)[slot].float() for c in (s["k_cache"], s["v_cache"]))
    # the rows, padded to N a sequence
    i = torch.arange(N, device=dev)
    row = (qsl[:-1, None] + i).clamp(max=len(q) - 1)
    qb = q[row].float().view(B, N, Hkv, g, D).permute(0, 2, 3, 1, 4)              # B Hkv g N D
    score = torch.matmul(qb.reshape(B, Hkv, g * N, D), k.permute(0, 2, 3, 1)) * s["scale"]
    word = s["mask"][row]                                                          # B N
    depth = ((word[:, :, None] >> torch.arange(64, device=dev)) & 1).sum(2) - 1
    j = key - ctx[:, None]                                                         # B span: index in the tree
    in_tree = ((word[:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1) == 1
    in_ctx = torch.ones_like(in_tree)
    if window:
        in_ctx = key[:, None, :] > (ctx[:, None] + depth - window)[:, :, None]
    seen = there[:, None, :] & torch.where(j[:, None, :] >= 0, in_tree, in_ctx)    # B N span
    seen = seen[:, None, None].expand(B, Hkv, g, N, span).reshape(B, Hkv, g * N, span)
    score = score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    score = score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score, v.permute(0, 2, 1, 3)) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    # back to the packed rows
    t = torch.arange(len(q), device=dev)
    b = torch.searchsorted(qsl[1:], t, right=True)
    n = t - qsl[b]
    o = o.view(B, Hkv, g, N, D).permute(0, 3, 1, 2, 4)[b, n].reshape(len(q), Hq, D)
    lse = lse.view(B, Hkv, g, N).permute(0, 3, 1, 2)[b, n].reshape(len(q), Hq)
    return dict(out=o.to(q.dtype), lse=lse)


# ------------------------------------------------------------------ work

def work(case):
    if case["op"] == "batch":
        ctx, new = _batch_lens(case)
        bs, tree = case["block"], case["kind"] == "tree"
        fresh = int((-(-(ctx + new) // bs) - -(-ctx // bs)).sum())
        per_token = 12 + (12 if tree else 0)  # position and slot; parent and mask
        return dict(bytes=24 * len(ctx) + per_token * int(new.sum()) + 8 * fresh, flops=0)
    if case["op"] == "rope":
        T, Hq, Hkv, D = (case[k] for k in ("tokens", "q_heads", "kv_heads", "dim"))
        out = {"none": 2 * Hkv, "same": 4 * Hkv, "e4m3": 2 * Hkv}[case["cache"]] + 2 * Hq
        heads = Hq + Hkv * (1 if case["cache"] == "none" else 2)
        return dict(bytes=T * (D * (2 * heads + out) + 4 * case["rotary"] + 4 + (8 if case["cache"] != "none" else 0)),
                    flops=T * (Hq + Hkv) * D * 7)
    ctx, new = _tree_lens(case)
    Hq, Hkv, D, W = (case[k] for k in ("q_heads", "kv_heads", "dim", "window"))
    keys = (np.minimum(ctx, W) if W else ctx) + new
    pairs = int(((np.minimum(ctx, W) if W else ctx) * new).sum() + (new * 6).sum())  # about six ancestors a token
    return dict(bytes=int(keys.sum()) * Hkv * D * 4 + int(new.sum()) * Hq * (D * 4 + 4) + int((keys / case["block"]).sum()) * 4,
                flops=4 * D * Hq * pairs)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    return {"batch": _exact_batch, "rope": _exact_rope, "tree": _exact_tree}[case["op"]](prepare(case, seed))


def _exact_batch(s):
    """Request by request on the host."""
    ctx, new, held, free = (s[k].cpu().tolist() for k in ("ctx", "new", "held", "free"))
    table = s["table"].cpu().numpy().copy()
    parents = None if s["parents"] is None else s["parents"].cpu().tolist()
    bs, T, B = s["block"], s["tokens"], len(ctx)
    qsl, lens, held_out = [0], [], []
    positions, slots, masks = np.full(T, -1, np.int32), np.full(T, -1, np.int64), np.zeros(T, np.int64)
    used, short = 0, False
    for r in range(B):
        c, n, h = ctx[r], new[r], held[r]
        want = max(0, -(-(c + n) // bs) - h) if n else 0
        short = short or used + want > len(free)
        ok = want == 0 or not short
        if ok:
            table[r, h:h + want] = free[used:used + want]
            used += want
            at = np.arange(c, c + n)
            slots[qsl[-1]:qsl[-1] + n] = table[r, at // bs].astype(np.int64) * bs + at % bs
            if parents is None:
                positions[qsl[-1]:qsl[-1] + n] = at
            else:
                word, deep = [], []
                for i in range(n):
                    p = parents[qsl[-1] + i]
                    word.append((1 << i) | (word[p] if p >= 0 else 0))
                    deep.append(deep[p] + 1 if p >= 0 else 0)
                positions[qsl[-1]:qsl[-1] + n] = c + np.array(deep)
                masks[qsl[-1]:qsl[-1] + n] = np.array(word, np.uint64).view(np.int64)
        qsl.append(qsl[-1] + n)
        lens.append(c + n if ok else 0)
        held_out.append(h + want if ok else h)
    as32 = lambda v: np.array(v, np.int32)  # noqa: E731
    return _batch_outputs(as32(qsl), as32(lens), positions, slots, as32(held_out), as32([used]), table,
                          None if parents is None else masks)


def _exact_rope(s):
    """Every pair as a complex number, turned by its angle's unit."""
    cs = s["cos_sin"].double()[s["positions"].long()]
    half = s["rotary"] // 2
    unit = torch.complex(cs[:, :half], cs[:, half:])[:, None]

    def head(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt() * w.double()
        x = x.clone()
        first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if s["interleaved"] else (slice(0, half), slice(half, 2 * half))
        z = torch.complex(x[..., first], x[..., second]) * unit
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q, k = head(s["q"], s["wq"]), head(s["k"], s["wk"])
    if s["cache"] == "none":
        return dict(q=q, k=k)
    out = dict(q=q)
    used = (s["slots"] >= 0).nonzero().squeeze(1)
    for name, x, scale in (("k_cache", k, s["k_scale"]), ("v_cache", s["v"].double(), s["v_scale"])):
        c = torch.zeros(s[name].shape, dtype=torch.float64, device="cuda")
        c.view(-1, *c.shape[2:])[s["slots"][used]] = x[used] / scale
        out[name] = c
    return out


def _exact_tree(s):
    """Sequence by sequence and kv head by kv head."""
    q, bs, W = s["q"], s["block"], s["window"]
    T, Hq, D = q.shape
    Hkv = s["k_cache"].shape[2]
    g = Hq // Hkv
    qsl, lens = s["qsl"].tolist(), s["lens"].tolist()
    masks = s["mask"].cpu().numpy().view(np.uint64)
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((T, Hq), dtype=torch.float64, device="cuda")
    for b in range(len(lens)):
        t0, t1, L = qsl[b], qsl[b + 1], lens[b]
        n, c = t1 - t0, L - (t1 - t0)
        lo = max(0, c - W) if W else 0
        hide = np.zeros((n, L - lo), bool)
        for i in range(n):
            bits = np.array([(int(masks[t0 + i]) >> j) & 1 for j in range(n)], bool)
            hide[i, c - lo:] = ~bits
            if W:
                hide[i, :c - lo] = np.arange(lo, c) <= c + bits.sum() - 1 - W
        hide = torch.from_numpy(hide).cuda()
        blocks = s["table"][b, lo // bs:-(-L // bs)].long()
        k, v = (x[blocks].reshape(-1, Hkv, D)[lo % bs:lo % bs + L - lo].double() for x in (s["k_cache"], s["v_cache"]))
        for h in range(Hkv):
            x = torch.einsum("nad,kd->ank", q[t0:t1, h * g:(h + 1) * g].double(), k[:, h]) * s["scale"]
            x = x.masked_fill(hide, -math.inf)
            out[t0:t1, h * g:(h + 1) * g] = torch.einsum("ank,kd->nad", torch.softmax(x, -1), v[:, h])
            lse[t0:t1, h * g:(h + 1) * g] = torch.logsumexp(x, -1).T
    return dict(out=out, lse=lse)
