"""Timed cases of attention with a sliding window and sinks, of attention over 4-bit caches, and of the
append that fills such caches, with their plain forms.

  decode   a few new tokens a sequence over a paged cache: each sees its window and the first tokens (sinks)
  prefill  chunks of new tokens with the same mask; window 0 is full attention
  append   RMS norm of every query and key head, rotary embedding, write into an INT4 paged cache

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
        # one request far into a long conversation: what a single user waits for at every token
        dict(name="decode_one", op="decode", seqs=1, ctx=30000, spread="fixed", q_len=1, q_heads=32, kv_heads=8,
             dim=128, block=16, window=4096, sinks=4, cache="same", group=0, dtype="bf16", lens=1),
        # the window layers of the Mistral-shaped step: log-normal lengths, 4 speculative tokens
        dict(name="decode_mistral", op="decode", seqs=128, ctx=32768, spread="lognormal", q_len=4, q_heads=32,
             kv_heads=8, dim=128, block=16, window=4096, sinks=4, cache="same", group=0, dtype="bf16", lens=2),
        # long conversations of the Llama-70B shape over an E4M3 cache
        dict(name="decode_long_fp8", op="decode", seqs=32, ctx=131072, spread="uniform", q_len=1, q_heads=64,
             kv_heads=8, dim=128, block=16, window=8192, sinks=64, cache="e4m3", group=0, dtype="bf16", lens=3),
        # the Llama-3-8B-shaped batch over an INT4 cache, a short window
        dict(name="decode_int4", op="decode", seqs=256, ctx=8192, spread="uniform", q_len=1, q_heads=32, kv_heads=8,
             dim=128, block=16, window=2048, sinks=16, cache="int4", group=32, dtype="bf16", lens=4),
        # the OPT-125m shape, one sink
        dict(name="decode_opt125m", op="decode", seqs=64, ctx=2048, spread="uniform", q_len=1, q_heads=12, kv_heads=12,
             dim=64, block=16, window=512, sinks=1, cache="same", group=0, dtype="f16", lens=5),
        # a short turn of one conversation: 100 tokens after 20000
        dict(name="prefill_one", op="prefill", seqs=1, new=100, ctx=20000, spread="fixed", q_heads=32, kv_heads=8,
             dim=128, block=16, window=4096, sinks=4, cache="same", group=0, dtype="bf16", lens=6),
        # 16 chunks of 1024 tokens of the Llama-3-8B shape in the middle of their prompts
        dict(name="prefill_chunks", op="prefill", seqs=16, new=1024, ctx=7168, spread="uniform", q_heads=32, kv_heads=8,
             dim=128, block=16, window=4096, sinks=4, cache="same", group=0, dtype="bf16", lens=7),
        # ragged whole prompts of the Llama-70B shape, a short window and many sinks
        dict(name="prefill_prompts", op="prefill", seqs=8, new=2048, ctx=0, spread="ragged", q_heads=64, kv_heads=8,
             dim=128, block=16, window=512, sinks=128, cache="same", group=0, dtype="f16", lens=8),
        # a question of 257 tokens about an 8000-token document that is held in INT4
        dict(name="prefill_int4_one", op="prefill", seqs=1, new=257, ctx=8000, spread="fixed", q_heads=32, kv_heads=8,
             dim=128, block=16, window=0, sinks=0, cache="int4", group=32, dtype="bf16", lens=9),
        # the 16 chunks over an INT4 cache, full attention
        dict(name="prefill_int4_chunks", op="prefill", seqs=16, new=1024, ctx=7168, spread="uniform", q_heads=32,
             kv_heads=8, dim=128, block=16, window=0, sinks=0, cache="int4", group=32, dtype="bf16", lens=10),
        # one token of the Llama-3-8B shape into an INT4 cache
        dict(name="append_one", op="append", tokens=1, q_heads=32, kv_heads=8, dim=128, rotary=128, interleaved=False,
             norm=True, group=32, dtype="bf16", block=16),
        # 16 chunks of 1024 tokens of the Llama-70B shape
        dict(name="append_prompts", op="append", tokens=16384, q_heads=64, kv_heads=8, dim=128, rotary=128,
             interleaved=False, norm=True, group=32, dtype="bf16", block=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("decode", "decode", "prefill", "prefill", "append"))
    if op == "append":
        q_heads, kv_heads = rng.choice(((32, 8), (64, 8), (28, 4), (8, 1), (8, 8), (16, 16)))
        tokens = _log(rng, 1, 14000)
        while tokens * (q_heads + 2 * kv_heads) > 16384 * 80:
            tokens = tokens * 2 // 3
        return dict(op=op, tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, dim=128, rotary=rng.choice((128, 128, 64)),
                    interleaved=rng.random() < 0.3, norm=rng.random() < 0.8, group=rng.choice((8, 16, 32, 64, 128)),
                    dtype=rng.choice(("bf16", "f16")), block=rng.choice((8, 16, 32)))
    cache = rng.choice(("same", "same", "e4m3", "int4"))
    case = dict(op=op, cache=cache, group=rng.choice((8, 16, 32, 64, 128)) if cache == "int4" else 0,
                dtype=rng.choice(("bf16", "f16")), block=rng.choice((8, 16, 32)),
                window=rng.choice((_log(rng, 64, 8192), _log(rng, 64, 8192), 4096)),
                sinks=rng.choice((0, 1, 4, 4, rng.randint(1, 200))), lens=rng.randint(0, 1 << 20))
    if op == "decode":
        q_heads, kv_heads, dim = rng.choice(((32, 8, 128), (64, 8, 128), (28, 4, 128), (8, 8, 128)) +
                                            (((12, 12, 64), (40, 8, 64)) if cache == "same" else ()))
        case |= dict(q_heads=q_heads, kv_heads=kv_heads, dim=dim, seqs=_log(rng, 1, 250), ctx=_log(rng, 1, 130000),
                     spread=rng.choice(("fixed", "uniform")), q_len=rng.choice((1, 1, 2, 3, 5)))
        while case["seqs"] * min(case["ctx"], case["window"]) * kv_heads * dim > 128 * 2600 * 8 * 128:
            case["seqs"] = case["seqs"] * 2 // 3
        return case
    q_heads, kv_heads, dim = rng.choice(((32, 8, 128), (64, 8, 128), (28, 4, 128), (8, 8, 128)) +
                                        (((12, 12, 64), (40, 8, 64)) if cache == "same" else ()))
    if rng.random() < 0.3:
        case |= dict(window=0, sinks=0)
    case |= dict(q_heads=q_heads, kv_heads=kv_heads, dim=dim, seqs=_log(rng, 1, 24), new=_log(rng, 1, 2000),
                 ctx=0 if rng.random() < 0.2 else _log(rng, 1, 7500 if case["window"] == 0 else 60000),
                 spread=rng.choice(("fixed", "uniform", "ragged")))
    # a drawn case costs no more than the 16 chunks
    while case["seqs"] * case["new"] * q_heads * (min(case["ctx"], case["window"] or case["ctx"]) + case["new"]) > 2 << 30:
        k = "seqs" if case["seqs"] > 1 else "new"
        case[k] = case[k] * 2 // 3
    return case


# The lengths of a case go by the case alone (so that its work is known); a seed changes their order.

def _lens(case):
    """Cached tokens and new tokens of every sequence."""
    rng = np.random.default_rng(case["lens"])
    B, ctx = case["seqs"], case["ctx"]
    if case["spread"] == "uniform":
        c = rng.integers(ctx // 16, ctx + 1, B)
    elif case["spread"] == "lognormal":
        c = np.clip(np.exp(rng.normal(math.log(2048), 1.0, B)).astype(np.int64), 1, ctx)
    else:
        c = np.full(B, ctx)
    if case["op"] == "decode":
        n = np.full(B, case["q_len"])
    elif case["spread"] == "ragged" and B > 1:
        n = rng.integers(max(1, case["new"] // 8), case["new"] + 1, B)
    else:
        n = np.full(B, case["new"])
    return c.astype(np.int64), n.astype(np.int64)


def _first(c, window):
    """The first key that a sequence's first new row sees through its window."""
    return np.maximum(c - window + 1, 0) if window else np.zeros_like(c)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    return _prepare_append(case, seed) if case["op"] == "append" else _prepare_attention(case, seed)


def _normal(gen, shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _int4_bytes(x, scales):
    """float32 [..., H, D] with scales [H, D / group] -> bytes, the even dim of a pair in the low nibble."""
    q = (x / scales.repeat_interleave(x.shape[-1] // scales.shape[-1], 1)).round_().clamp_(-8, 7).to(torch.uint8)
    return (q[..., 0::2] & 15) | ((q[..., 1::2] & 15) << 4)


def _group_scales(gen, heads, groups):
    # calibrated for values of about unit size: a step of near a third
    return 0.28 + 0.08 * torch.rand((heads, groups), generator=gen, device="cuda", dtype=torch.float32)


def _prepare_attention(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    rng = np.random.default_rng([seed, 17])
    Hq, Hkv, D, bs, W, S = (case[k] for k in ("q_heads", "kv_heads", "dim", "block", "window", "sinks"))
    dt = DTYPES[case["dtype"]]
    c, n = _lens(case)
    order = rng.permutation(len(c))
    c, n = c[order], n[order]
    L = c + n
    # the blocks that a row still sees; those between the sinks and the window have been released
    logical = np.arange(int(-(-L.max() // bs)) + 1)[None, :]
    live = (logical < -(-L // bs)[:, None]) & ((logical >= (_first(c, W) // bs)[:, None]) | (logical * bs < (S if W else 0)))
    NB = int(live.sum()) + 3
    table = np.full(live.shape, -1, np.int32)
    table[live] = rng.permutation(NB)[:int(live.sum())]
    qsl = np.concatenate([[0], np.cumsum(n)])
    s = dict(op=case["op"], block=bs, window=W, sinks=S, scale=D ** -0.5, max_len=int(L.max()), max_new=int(n.max()),
             q_len=case.get("q_len"), cache=case["cache"], k_scale=1.0, v_scale=1.0)
    for k, v in (("table", table), ("lens", L), ("qsl", qsl)):
        s[k] = torch.from_numpy(v.astype(np.int32)).cuda()
    # queries lean towards one direction a head, and so do the keys of the first tokens, whose values are
    # small: what makes such tokens sinks
    lean = 0.5 * _normal(gen, (Hkv, D))
    s["q"] = (_normal(gen, (int(qsl[-1]), Hkv, Hq // Hkv, D)) + lean[:, None]).view(-1, Hq, D).to(dt)
    first = table[table[:, 0] >= 0, 0]
    few = min(4, bs)
    for name in ("k_cache", "v_cache"):
        x = _normal(gen, (NB, bs, Hkv, D))
        at = torch.from_numpy(first).cuda().long()
        x[at, :few] = x[at, :few] + 2 * lean if name == "k_cache" else 0.1 * x[at, :few]
        if case["cache"] == "int4":
            s[name[0] + "_scales"] = _group_scales(gen, Hkv, D // case["group"])
            s[name] = _int4_bytes(x, s[name[0] + "_scales"])
        elif case["cache"] == "e4m3":
            s[name[0] + "_scale"] = 0.0131 if name == "v_cache" else 0.0175
            s[name] = (x / s[name[0] + "_scale"]).clamp_(-448, 448).to(torch.float8_e4m3fn)
        else:
            s[name] = x.to(dt)
        del x
    s["out"] = torch.empty_like(s["q"])
    # (the log-sum-exp is float32; the INT4 path rounds scaled queries to 16 bits, so that its digits end earlier)
    s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda") if case["cache"] != "int4" else None
    s["workspace"] = None
    if own:
        from paged_kv_cache_block_gb300 import kvcache as kv
        code = {"same": kv.dtype_code(dt), "e4m3": kv.KV_FP8_E4M3, "int4": kv.KV_INT4}[case["cache"]]
        if case["op"] == "decode":
            size = kv.paged_attention_workspace_size(len(c), s["q_len"], Hq, Hkv, D, bs, code, s["max_len"], W)
        else:
            size = kv.paged_attention_prefill_sinks_workspace_size(len(c), s["max_new"], Hq, Hkv, D, code, s["max_len"], W, S)
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


def _prepare_append(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    T, Hq, Hkv, D, rot, bs = (case[k] for k in ("tokens", "q_heads", "kv_heads", "dim", "rotary", "block"))
    dt = DTYPES[case["dtype"]]
    # the rows of one packed projection; query, key and value are views of it
    qkv = _normal(gen, (T, (Hq + 2 * Hkv) * D)).to(dt)
    q, k, v = (x.view(T, -1, D) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1))
    s = dict(op="append", q=q, k=k, v=v, rotary=rot, interleaved=case["interleaved"], eps=1e-6, wq=None, wk=None, block=bs)
    if case["norm"]:
        s["wq"] = (1 + 0.2 * _normal(gen, (D,))).to(dt)
        s["wk"] = (1 + 0.2 * _normal(gen, (D,))).to(dt)
    max_pos = 32768
    s["positions"] = torch.randint(0, max_pos, (T,), generator=gen, device="cuda", dtype=torch.int32)
    inv = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    NB = -(-T // bs) + 3
    s["slots"] = torch.randperm(NB * bs, generator=gen, device="cuda")[:T].to(torch.int64)
    s["slots"][T // 2:T // 2 + T // 50] = -1  # rows of padding
    # K and V of the layer, which hold earlier tokens; they are views of one allocation
    s["scales"] = torch.stack([_group_scales(gen, Hkv, D // case["group"]) for _ in range(2)])
    s["caches"] = torch.stack([_int4_bytes(_normal(gen, (NB, bs, Hkv, D)), x) for x in s["scales"]])
    s["q_out"] = torch.empty((T, Hq, D), dtype=dt, device="cuda")
    # what a byte stands for, to show the caches as values
    code = torch.arange(256, device="cuda")
    pair = torch.stack([code & 15, code >> 4], 1)
    s["pairs"] = torch.where(pair > 7, pair - 16, pair).to(torch.bfloat16)
    s["wide_scales"] = s["scales"].repeat_interleave(case["group"], 2)[:, None, None]
    s["values"] = torch.empty((2, NB, bs, Hkv, D), dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return {"decode": _own_decode, "prefill": _own_prefill, "append": _own_append}[s["op"]](s)
    return _plain_append(s) if s["op"] == "append" else _plain_attention(s)


def _attention_outputs(out, lse):
    return dict(out=out) if lse is None else dict(out=out, lse=lse)


def _own_decode(s):
    from paged_kv_cache_block_gb300 import kvcache as kv
    if s["cache"] == "int4":
        kv.paged_attention_decode_sinks_int4(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["max_len"],
                                             s["q_len"], s["scale"], s["k_scales"], s["v_scales"], s["window"], s["sinks"],
                                             workspace=s["workspace"], out=s["out"])
    else:
        kv.paged_attention_decode_sinks(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["max_len"], s["q_len"],
                                        s["scale"], s["window"], s["sinks"], s["k_scale"], s["v_scale"],
                                        workspace=s["workspace"], out=s["out"], lse_out=s["lse"])
    return _attention_outputs(s["out"], s["lse"])


def _own_prefill(s):
    from paged_kv_cache_block_gb300 import kvcache as kv
    if s["cache"] == "int4":
        kv.paged_attention_prefill_sinks_int4(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["qsl"],
                                              s["max_len"], s["max_new"], s["scale"], s["k_scales"], s["v_scales"],
                                              s["window"], s["sinks"], workspace=s["workspace"], out=s["out"])
    else:
        kv.paged_attention_prefill_sinks(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["qsl"], s["max_len"],
                                         s["max_new"], s["scale"], s["window"], s["sinks"], s["k_scale"], s["v_scale"],
                                         workspace=s["workspace"], out=s["out"], lse_out=s["lse"])
    return _attention_outputs(s["out"], s["lse"])


def _cache_rows(s, name, slot):
    """The rows [..., H, D] of the cache's slots, in float32."""
    c = s[name]
    c = c.view(torch.uint8).view(-1, *c.shape[2:]) if s["cache"] == "e4m3" else c.view(-1, *c.shape[2:])
    x = c[slot]
    if s["cache"] == "e4m3":
        return x.view(torch.float8_e4m3fn).float() * s[name[0] + "_scale"]
    if s["cache"] == "int4":
        code = torch.stack([x & 15, x >> 4], -1).flatten(-2).to(torch.int8)
        scales = s[name[0] + "_scales"]
        return ((code ^ 8) - 8).float() * scales.repeat_interleave(code.shape[-1] // scales.shape[-1], 1)
    return x.float()


def _plain_attention(s):
    q, qsl, L, bs, W, S = s["q"], s["qsl"].long(), s["lens"].long(), s["block"], s["window"], s["sinks"]
    Hq, D = q.shape[1:]
    dev, B = q.device, len(L)
    N, new = s["max_new"], qsl[1:] - qsl[:-1]
    ctx = L - new
    # the keys that some row sees: `few` sinks, then positions first .. L - 1
    first = (ctx - W + 1).clamp(min=0) if W else torch.zeros_like(ctx)
    few = first.clamp(max=S)
    span = min(s["max_len"], W + N - 1 + S) if W else s["max_len"]
    i = torch.arange(span, device=dev)
    key = torch.where(i < few[:, None], i, i - few[:, None] + first[:, None])
    there = key < L[:, None]
    safe = torch.where(there, key, first[:, None])
    slot = s["table"].long().gather(1, safe // bs) * bs + safe % bs
    k = _cache_rows(s, "k_cache", slot)
    Hkv = k.shape[2]
    g = Hq // Hkv
    # the rows, padded to N a sequence
    n = torch.arange(N, device=dev)
    row = (qsl[:-1, None] + n).clamp(max=len(q) - 1)
    qb = q[row].float().view(B, N, Hkv, g, D).permute(0, 2, 3, 1, 4)
    score = torch.matmul(qb.reshape(B, Hkv, g * N, D), k.permute(0, 2, 3, 1)).mul_(s["scale"])
    del k
    pos = ctx[:, None] + n
    seen = there[:, None, :] & (key[:, None, :] <= pos[:, :, None])
    if W:
        seen &= (key[:, None, :] > pos[:, :, None] - W) | (key[:, None, :] < S)
    score = score.view(B, Hkv, g, N, span).masked_fill_(~seen[:, None, None], -math.inf).view(B, Hkv, g * N, span)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    score = score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    v = _cache_rows(s, "v_cache", slot)
    o = torch.matmul(score, v.permute(0, 2, 1, 3)) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    # back to the packed rows
    t = torch.arange(len(q), device=dev)
    b = torch.searchsorted(qsl[1:], t, right=True)
    at = t - qsl[b]
    o = o.view(B, Hkv, g, N, D).permute(0, 3, 1, 2, 4)[b, at].reshape(len(q), Hq, D)
    lse = lse.view(B, Hkv, g, N).permute(0, 3, 1, 2)[b, at].reshape(len(q), Hq)
    return _attention_outputs(o.to(q.dtype), None if s["lse"] is None else lse)


def _append_outputs(s, q):
    """The queries, and the caches as the values they stand for."""
    pairs = torch.nn.functional.embedding(s["caches"].int(), s["pairs"])
    torch.mul(pairs.view(s["values"].shape), s["wide_scales"], out=s["values"])
    return dict(q=q, caches=s["values"])


def _own_append(s):
    from paged_kv_cache_block_gb300 import kvcache as kv
    q = kv.qk_norm_rope_and_cache_int4(s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["slots"], s["caches"][0],
                                       s["caches"][1], s["scales"][0], s["scales"][1], s["wq"], s["wk"], s["eps"],
                                       s["interleaved"], q_out=s["q_out"])
    return _append_outputs(s, q)


def _plain_append(s):
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
    caches = s["caches"]
    total = caches.shape[1] * s["block"]
    # rows without a slot go to one row behind the caches
    at = torch.where(s["slots"] >= 0, s["slots"], total)
    new = torch.stack([_int4_bytes(x, w) for x, w in ((k, s["scales"][0]), (s["v"].float(), s["scales"][1]))])
    flat = caches.view(2, total, *caches.shape[3:])
    flat.copy_(torch.cat([flat, flat[:, :1]], 1).index_copy_(1, at, new)[:, :total])
    return _append_outputs(s, q.to(s["q"].dtype))


# ------------------------------------------------------------------ work

def work(case):
    if case["op"] == "append":
        T, Hq, Hkv, D = (case[k] for k in ("tokens", "q_heads", "kv_heads", "dim"))
        return dict(bytes=T * (D * (4 * Hq + 4 * Hkv + Hkv) + 4 * case["rotary"] + 4 + 8), flops=T * (Hq + Hkv) * D * 7)
    c, n = _lens(case)
    Hq, Hkv, D, W, S = (case[k] for k in ("q_heads", "kv_heads", "dim", "window", "sinks"))
    first = _first(c, W)
    keys = int((c + n - first + np.minimum(first, S if W else 0)).sum())
    # rows of position p see min(p + 1, W) keys of their window and the sinks before it
    pairs = 0
    for a, m in zip(c.tolist(), n.tolist()):
        p = np.arange(a, a + m, dtype=np.int64)
        lo = np.maximum(p - W + 1, 0) if W else np.zeros_like(p)
        pairs += int((p + 1 - lo + np.minimum(lo, S)).sum())
    row = {"same": 2 * D, "e4m3": D, "int4": D // 2}[case["cache"]]
    return dict(bytes=keys * Hkv * row * 2 + int(n.sum()) * Hq * (4 * D + (4 if case["cache"] != "int4" else 0)) +
                keys // case["block"] * 4, flops=4 * D * Hq * pairs)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)


def _exact_append(s):
    """Every pair as a complex number, turned by its angle's unit; codes from the quotient in 64 bits."""
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

    used = (s["slots"] >= 0).nonzero().squeeze(1)
    values = []
    for x, held, scales in ((head(s["k"], s["wk"]), s["caches"][0], s["scales"][0]), (s["v"].double(), s["caches"][1], s["scales"][1])):
        step = scales.double().repeat_interleave(x.shape[-1] // scales.shape[-1], 1)
        code = torch.stack([held % 16, held // 16], -1).flatten(-2).double()
        code = code - 16 * (code >= 8)
        code.view(-1, *x.shape[1:])[s["slots"][used]] = torch.clamp(torch.round(x[used] / step), -8, 7)
        values.append(code * step)
    return dict(q=head(s["q"], s["wq"]), caches=torch.stack(values))


def _exact_attention(s):
    """Sequence by sequence and kv head by kv head."""
    q, bs, W, S = s["q"], s["block"], s["window"], s["sinks"]
    T, Hq, D = q.shape
    Hkv = s["k_cache"].shape[2]
    g = Hq // Hkv
    qsl, lens = s["qsl"].tolist(), s["lens"].tolist()
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((T, Hq), dtype=torch.float64, device="cuda")

    def rows(name, b, keys, h):
        c = s[name].view(torch.uint8) if s["cache"] == "e4m3" else s[name]
        x = c[s["table"][b, keys // bs].long(), keys % bs, h]
        if s["cache"] == "int4":
            x = torch.stack([x % 16, x // 16], -1).flatten(-2).double()
            step = s[name[0] + "_scales"][h].double()
            return (x - 16 * (x >= 8)) * step.repeat_interleave(D // len(step))
        return (x.view(torch.float8_e4m3fn) if s["cache"] == "e4m3" else x).double() * s[name[0] + "_scale"]

    for b in range(len(lens)):
        t0, t1, L = qsl[b], qsl[b + 1], lens[b]
        p = torch.arange(L - (t1 - t0), L, device="cuda")
        keys = torch.arange(L, device="cuda")
        if W:
            keys = keys[(keys > p[0] - W) | (keys < S)]
        hide = keys[None] > p[:, None]
        if W:
            hide |= (keys[None] <= p[:, None] - W) & (keys[None] >= S)
        for h in range(Hkv):
            x = torch.einsum("nad,kd->ank", q[t0:t1, h * g:(h + 1) * g].double(), rows("k_cache", b, keys, h)) * s["scale"]
            x = x.masked_fill(hide, -math.inf)
            lse[t0:t1, h * g:(h + 1) * g] = torch.logsumexp(x, -1).T
            out[t0:t1, h * g:(h + 1) * g] = torch.einsum("ank,kd->nad", torch.softmax(x, -1), rows("v_cache", b, keys, h))
    return dict(out=out) if s["cache"] == "int4" else dict(out=out, lse=lse)
