"""The operators as a serving loop uses them: a packed prompt is rotated, attended
to and put into a paged cache, its keys' weights are collected, tokens are decoded
with the weights carried on, the cache is cut down, and decoding goes on against
the smaller cache. Every step is compared with the same step in 64 bits, from the
bf16 values that the GPU's previous step left.

And the same calls at addresses past 32 bits of elements.

Tolerances: attention outputs within relative L2 2e-3 and LSE within 1e-3 (the
bar of the attention calls); weights within 1e-4 relative (scores of 128 products
in fp32 at |s| < 20, see test_key_mass_gpu.py: below 2e-5; a decayed sum of such
terms keeps the bound).
"""
import pytest
import torch

from test_evict_gpu import chosen
from test_rope_gpu import close, reference

pytestmark = pytest.mark.gpu

Hq, Hkv, D, PAGE, SECTIONS = 8, 2, 128, 64, (32, 16, 16)
SCALE = D ** -0.5


def attention(q, k, v):
    """q [n, Hq, D] at the end of k, v [m, Hkv, D], in 64 bits -> (o, lse [Hq, n], weights [Hkv, m])."""
    n, m = q.shape[0], k.shape[0]
    kk, vv = (x.double().repeat_interleave(Hq // Hkv, 1).permute(1, 0, 2) for x in (k, v))
    s = q.double().permute(1, 0, 2) @ kk.transpose(1, 2) * SCALE
    late = torch.arange(m, device="cuda")[None] > torch.arange(n, device="cuda")[:, None] + m - n
    s = s.masked_fill(late, float("-inf"))
    p = torch.softmax(s, -1)
    return (p @ vv).permute(1, 0, 2), torch.logsumexp(s, -1), p.sum(1).view(Hkv, -1, m).sum(1)


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def test_serving_loop(cuda_lib):
    mala = cuda_lib
    lens = [300, 129, 64]
    B, T, maxp = 3, sum(lens), 8
    g = torch.Generator(device="cuda").manual_seed(1)
    inv_freq = (10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)).float()
    pool = torch.full((B * maxp * 2, PAGE, Hkv, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    kp, vp = pool, pool.clone()
    ids = torch.randperm(B * maxp * 2, generator=g, device="cuda").to(torch.int32)
    table, small = ids[:B * maxp].view(B, maxp).contiguous(), ids[B * maxp:].view(B, maxp).contiguous()
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def rows_of(pages, tb, b, n):
        return pages[tb[b].long()].flatten(0, 1)[:n]

    # the prompt: rotate (contiguous q, k, v for the attention) and fill the pages
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.randint(0, 500, (3, T), generator=g, device="cuda", dtype=torch.int32)
    views = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    q, k, v = mala.rope(*views, pos, inv_freq, sections=SECTIONS)
    close(q, *reference(views[0].double(), pos, inv_freq, SECTIONS, False, False))
    mala.rope_append(None, views[1], views[2], pos, inv_freq, kp, vp, table, sl, cu_seqlens=cu, sections=SECTIONS)
    o, lse, _, _ = mala.forward_varlen(q, k, v, cu, cu, max(lens), max(lens), SCALE, 0.0)
    mass = torch.empty(B, Hkv, maxp * PAGE, device="cuda")
    mala.key_mass_varlen(q, k, lse, cu, cu, max(lens), max(lens), SCALE, out=mass)
    assert mala.mala_check_status() == 0
    want_mass = torch.zeros(B, Hkv, maxp * PAGE, device="cuda", dtype=torch.float64)
    for b, n in enumerate(lens):
        a = slice(int(cu[b]), int(cu[b + 1]))
        assert torch.equal(rows_of(kp, table, b, n), k[a]) and torch.equal(rows_of(vp, table, b, n), v[a])
        wo, wl, wm = attention(q[a], k[a], v[a])
        assert rel(o[a], wo) <= 2e-3 and float((lse[:, a].double() - wl).abs().max()) <= 1e-3
        want_mass[b, :, :n] = wm
    assert bool(((mass.double() - want_mass).abs() <= 1e-4 * want_mass + 1e-30).all())

    def step(tb, i):
        """One decoding step against the cache of table tb; the 64-bit weights follow."""
        nonlocal mass
        sl.add_(1)
        x = torch.randn(B, Hq + 2 * Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
        at = torch.randint(500, 600, (3, B), generator=g, device="cuda", dtype=torch.int32)
        qn = mala.rope_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], at, inv_freq, kp, vp, tb, sl,
                              sections=SECTIONS)
        o, lse, kept, _, _, mass = mala.decode_paged_mass(qn, kp, vp, tb, sl, SCALE, 0.0, mass=mass, decay=0.9, out=mass)
        assert mala.mala_check_status() == 0
        for b in range(B):
            n = int(sl[b])
            kk, vv = rows_of(kp, tb, b, n), rows_of(vp, tb, b, n)
            close(kk[-1:], *reference(x[b:b + 1, Hq:Hq + Hkv].double(), at[:, b:b + 1], inv_freq, SECTIONS, False,
                                      False))
            assert torch.equal(vv[-1], x[b, Hq + Hkv:])
            wo, wl, wm = attention(qn[b:b + 1], kk, vv)
            assert rel(o[b], wo[0]) <= 2e-3 and float((lse[b].double() - wl[:, 0]).abs().max()) <= 1e-3
            want_mass[b, :, :n - 1] *= 0.9
            want_mass[b, :, n - 1] = 0.0
            want_mass[b, :, :n] += wm
            assert int(kept[b * Hq]) == -(-n // PAGE)
        assert bool(((mass.double() - want_mass).abs() <= 1e-4 * want_mass + 1e-30).all())

    for i in range(3):
        step(table, i)

    # cut the caches down to 130 rows, and go on from the smaller ones
    old, k_old, v_old = sl.tolist(), kp.clone(), vp.clone()
    room = torch.full_like(mass, float("nan"))
    index, new, small_mass = mala.evict(mass, sl, 130, kp, vp, table, small, n_sink=4, n_recent=32, mass_out=room)
    assert mala.mala_check_status() == 0
    assert new.tolist() == [130, 130, 67]
    before = want_mass.clone()
    want_mass.zero_()
    for b in range(B):
        n = int(new[b])
        for h in range(Hkv):
            keep = chosen(mass[b, h].cpu().numpy(), old[b], 130, 4, 32)
            assert index[b, h, :n].tolist() == keep.tolist()
            i = torch.from_numpy(keep).cuda()
            assert torch.equal(rows_of(kp, small, b, n)[:, h], rows_of(k_old, table, b, old[b])[i, h])
            assert torch.equal(rows_of(vp, small, b, n)[:, h], rows_of(v_old, table, b, old[b])[i, h])
            want_mass[b, h, :n] = before[b, h, i]
    assert small_mass.data_ptr() == room.data_ptr()
    assert bool(((small_mass.double() - want_mass).abs() <= 1e-4 * want_mass).all())  # 0 past the rows that remain
    mass = small_mass
    sl.copy_(new)
    for i in range(3):
        step(small, 3 + i)


def test_addresses_past_32_bits(cuda_lib):
    """Pools of 2.4e9 values each (4.7 GB): the last pages are written, read and moved."""
    mala = cuda_lib
    n, page = 18000, 128
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    kp = torch.empty(n, page, 8, 128, device="cuda", dtype=torch.bfloat16)
    vp = torch.empty_like(kp)
    assert kp.numel() > 1 << 31
    last = list(range(n - 6, n))
    for p in last:
        kp[p].normal_()
        vp[p].normal_()
    table = torch.tensor([last[:3]], dtype=torch.int32, device="cuda")
    out_table = torch.tensor([last[3:5]], dtype=torch.int32, device="cuda")
    sl = torch.tensor([300], dtype=torch.int32, device="cuda")
    x = torch.randn(1, 48, 128, device="cuda").to(torch.bfloat16)
    inv_freq = (10000.0 ** (-torch.arange(0, 128, 2, device="cuda", dtype=torch.float64) / 128)).float()
    pos = torch.zeros(1, 1, device="cuda", dtype=torch.int32)  # turns by nothing
    q = mala.rope_append(x[:, :32], x[:, 32:40], x[:, 40:], pos, inv_freq, kp, vp, table, sl)
    assert torch.equal(kp[last[2], 43], x[0, 32:40]) and torch.equal(vp[last[2], 43], x[0, 40:])
    small_k, small_v = kp[last].clone(), vp[last].clone()
    o, lse, _, _, ns, mass = mala.decode_paged_mass(q, kp, vp, table, sl, SCALE, 0.0)
    tb = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")
    want = mala.decode_paged_mass(q, small_k, small_v, tb, sl, SCALE, 0.0, n_splits=ns)
    assert torch.equal(o, want[0]) and torch.equal(mass, want[5])
    index, new, _ = mala.evict(mass, sl, 200, kp, vp, table, out_table, n_sink=4, n_recent=20)
    index2, new2, _ = mala.evict(mass, sl, 200, small_k, small_v, tb,
                                 torch.tensor([[3, 4]], dtype=torch.int32, device="cuda"), n_sink=4, n_recent=20)
    assert mala.mala_check_status() == 0
    assert torch.equal(index, index2) and torch.equal(kp[last], small_k) and torch.equal(vp[last], small_v)
