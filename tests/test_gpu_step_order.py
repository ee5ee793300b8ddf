"""The step's calls right behind a kernel that writes what they read: they are launched while it still runs."""
import pytest
import torch

from .test_gpu_step import rope_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kc():
    from paged_kv_cache_block_gb300 import kvcache
    return kvcache


@pytest.mark.parametrize("T,D,inter", [(3, 128, False), (4000, 64, True), (4000, 128, False)])
def test_weights_and_angles_written_by_the_kernel_before(kc, T, D, inter):
    """Weights, table, positions and inputs lie at the end of a long buffer that one kernel rewrites before
    each call; every call has to see the new ones, whatever its CTAs' caches hold of the old."""
    Hq, Hkv, max_pos, dt = 8, 2, 700, torch.bfloat16
    gen = torch.Generator().manual_seed(D)
    head = 1 << 25  # float32 words ahead of what the call reads
    words = [D // 2, D // 2, max_pos * D, (T + 3) & ~3, T * (Hq + Hkv) * D // 2]
    sets = []
    for k in range(2):
        w = (1 + 0.3 * torch.randn(2 * D, generator=gen)).to(dt).view(torch.float32)
        cs = torch.from_numpy(rope_table(max_pos, D)).flatten() * (1 - 2 * k)  # the other half of the circle
        pos = torch.randint(0, max_pos, ((T + 3) & ~3,), generator=gen, dtype=torch.int32).view(torch.float32)
        x = torch.randn(T * (Hq + Hkv) * D, generator=gen).to(dt).view(torch.float32)
        sets.append(torch.cat([torch.zeros(head), w, cs, pos, x]).view(torch.int32).cuda())
    buf = torch.empty_like(sets[0])
    w1, w2, cs, pos, x = buf[head:].split(words)
    wq, wk = w1.view(dt), w2.view(dt)
    cs = cs.view(torch.float32).view(max_pos, D)
    qk = x.view(dt).view(T, -1)
    q, k = qk[:, :Hq * D].view(T, Hq, D), qk[:, Hq * D:].view(T, Hkv, D)
    outs = [(torch.empty(T, Hq, D, dtype=dt, device="cuda"), torch.empty(T, Hkv, D, dtype=dt, device="cuda")) for _ in range(24)]

    def call(i):
        torch.bitwise_or(sets[i % 2], 0, out=buf)
        kc.qk_norm_rope(q, k, pos[:T], cs, wq, wk, 1e-6, inter, q_out=outs[i][0], k_out=outs[i][1])
    want = []
    for i in range(2):
        torch.bitwise_or(sets[i], 0, out=buf)
        torch.cuda.synchronize()
        want.append([t.clone() for t in kc.qk_norm_rope(q, k, pos[:T], cs, wq, wk, 1e-6, inter)])
        torch.cuda.synchronize()
    assert not torch.equal(want[0][0], want[1][0]) and not torch.equal(want[0][1], want[1][1])
    for i in range(24):
        call(i)
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(outs):
        assert torch.equal(a, want[i % 2][0]) and torch.equal(b, want[i % 2][1]), i
