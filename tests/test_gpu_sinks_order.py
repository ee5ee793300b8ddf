"""The calls with sinks right behind a kernel that writes what they read: they are launched while it still runs, and
so are their merges behind the attention kernels."""
import numpy as np
import pytest
import torch

from tests.sinks_reference import BF16, F16, Inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    from paged_kv_cache_block_gb300 import kvcache
    return kvcache


NAMES = ("q", "k_cache", "v_cache", "table", "lens", "qsl", "k_scales", "v_scales")


@pytest.mark.parametrize("cache,dtype", [("same", BF16), ("e4m3", F16), ("int4", BF16)])
@pytest.mark.parametrize("decode,ctx,new", [
    (True, [900], [2]), (True, [40, 700, 300] * 8, [2] * 24), (False, [900], [2]), (False, [40, 700, 300] * 8, [2] * 24),
    (False, [900], [70]), (False, [40, 700, 300] * 4, [20, 130, 50] * 4)])
def test_inputs_written_by_the_kernel_before(kv, cache, dtype, decode, ctx, new):
    """Queries, caches, table, lengths and scales lie at the end of a long buffer that one kernel rewrites before
    each call; every call has to see the new ones."""
    window, sinks = 200, 5
    head = 1 << 25  # int32 words ahead of what the call reads
    xs = [Inputs(k, ctx if k == 0 else ctx[::-1], new if k == 0 else new[::-1], 16, 4, window=window, sinks=sinks, cache=cache,
                 dtype=dtype) for k in range(2)]
    parts = []
    for x in xs:
        t = {n: getattr(x, n) for n in NAMES}
        t = {n: torch.from_numpy(np.ascontiguousarray(v)) if isinstance(v, np.ndarray) else v for n, v in t.items() if v is not None}
        parts.append(t)
    at, end = {}, head
    for n, t in parts[0].items():
        assert parts[1][n].shape == t.shape
        size = t.numel() * t.element_size()
        at[n] = (end, size)
        end += -(-size // 256) * 64
    sets = []
    for t in parts:
        words = torch.zeros(end, dtype=torch.int32)
        for n, (start, size) in at.items():
            words.view(torch.uint8)[4 * start:4 * start + size] = t[n].contiguous().view(torch.uint8).flatten()
        sets.append(words.cuda())
    buf = torch.empty_like(sets[0])
    d = {n: buf.view(torch.uint8)[4 * s:4 * s + z].view(parts[0][n].dtype).view(parts[0][n].shape) for n, (s, z) in at.items()}
    x, B, T = xs[0], len(ctx), int(xs[0].qsl[-1])
    max_len, code = int(x.lens.max()), {"same": kv._code_of[dtype], "e4m3": kv._code_of[torch.float8_e4m3fn], "int4": kv.KV_INT4}[cache]
    size = kv.paged_attention_workspace_size(B, 2, 16, 4, 128, 16, code, max_len, window) if decode else \
        kv.paged_attention_prefill_sinks_workspace_size(B, max(new), 16, 4, 128, code, max_len, window, sinks)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    outs = [torch.empty(T, 16, 128, dtype=dtype, device="cuda") for _ in range(16)]

    def call(out):
        a = (d["q"], d["k_cache"], d["v_cache"], d["table"], d["lens"])
        a += (max_len, 2, x.scale) if decode else (d["qsl"], max_len, max(new), x.scale)
        name = "paged_attention_decode_sinks" if decode else "paged_attention_prefill_sinks"
        if cache == "int4":
            getattr(kv, name + "_int4")(*a, d["k_scales"], d["v_scales"], window, sinks, workspace=ws, out=out)
        else:
            getattr(kv, name)(*a, window, sinks, x.k_scale, x.v_scale, workspace=ws, out=out)

    want = []
    for words in sets:
        torch.bitwise_or(words, 0, out=buf)
        torch.cuda.synchronize()
        want.append(torch.empty_like(outs[0]))
        call(want[-1])
        torch.cuda.synchronize()
    assert not torch.equal(*want) and all(torch.isfinite(w).all() for w in want)
    for i, out in enumerate(outs):
        torch.bitwise_or(sets[i % 2], 0, out=buf)
        call(out)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, want[i % 2]), i
