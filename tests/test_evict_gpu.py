"""Eviction on the GPU (mala_evict_select, mala_evict_gather) against sorting on
the host: the rows that remain, their order, their masses and their K and V, all
exact (nothing is computed, only chosen and copied)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def chosen(mass, L, budget, n_sink, n_recent):
    """Rows that remain of one head's masses [ld] (fp32): the definition, by sorting."""
    if L <= budget:
        return np.arange(L)
    mid = np.arange(n_sink, L - n_recent)
    m = mass[mid].astype(np.float64)
    m[np.isnan(m)] = -np.inf
    order = mid[np.lexsort((mid, -m))]  # largest first, equal ones from the lowest row up
    keep = order[:budget - n_sink - n_recent]
    return np.sort(np.concatenate([np.arange(n_sink), keep, np.arange(L - n_recent, L)]))


def check_select(mala, mass, lens, budget, n_sink, n_recent):
    B, H, ld = mass.shape
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    index, new, out = mala.evict_select(mass, sl, budget, n_sink, n_recent)
    assert mala.mala_check_status() == 0
    index, new, out, m = index.cpu().numpy(), new.cpu().numpy(), out.cpu().numpy(), mass.cpu().numpy()
    for b in range(B):
        assert new[b] == min(lens[b], budget)
        for h in range(H):
            want = chosen(m[b, h], lens[b], budget, n_sink, n_recent)
            assert (index[b, h, :len(want)] == want).all(), (b, h)
            assert (index[b, h, len(want):] == -1).all()
            assert np.array_equal(out[b, h, :len(want)], m[b, h, want], equal_nan=True)
            assert (out[b, h, len(want):] == 0).all()
    return index, new


@pytest.mark.parametrize("lens,H,ld,budget,n_sink,n_recent", [
    ([1], 1, 1, 1, 0, 0),
    ([2], 1, 5, 1, 0, 0),
    ([5, 0, 3], 2, 7, 3, 1, 1),
    ([100, 64, 65, 1], 2, 128, 64, 4, 16),
    ([1000, 999], 3, 1024, 1000, 0, 0),      # one row goes, and none
    ([1000, 400], 3, 1001, 300, 0, 300),     # only the recent ones
    ([1000, 400], 3, 1001, 300, 300, 0),     # only the first
    ([1000], 3, 1000, 301, 100, 200),        # one by weight
    ([4100, 2049, 4000], 2, 4200, 700, 4, 64),
    ([40000, 20001], 2, 40000, 5000, 4, 512),   # a cluster of CTAs to a row
    ([131072], 8, 131072, 4096, 4, 1024),
    ([9000] * 40, 2, 9000, 123, 1, 7),          # more rows than a cluster each
])
def test_select(cuda_lib, lens, H, ld, budget, n_sink, n_recent):
    g = torch.Generator(device="cuda").manual_seed(sum(lens) + budget)
    u = torch.rand(len(lens), H, ld, generator=g, device="cuda")
    check_select(cuda_lib, 1.0 / (u + 1e-3), lens, budget, n_sink, n_recent)


@pytest.mark.parametrize("kind", ["equal", "few", "zeros", "negative", "nan", "inf", "denormal", "neighbours"])
@pytest.mark.parametrize("L", [700, 20000])
def test_select_orders(cuda_lib, kind, L):
    """Ties (taken from the lowest row up), both zeros, infinities, NaN, and values a bit apart."""
    g = torch.Generator(device="cuda").manual_seed(L)
    m = torch.rand(2, 2, L + 5, generator=g, device="cuda")
    if kind == "equal":
        m.fill_(0.25)
    elif kind == "few":
        m = (m * 4).floor()
    elif kind == "zeros":
        m = torch.where(m < 0.5, torch.zeros_like(m), -torch.zeros_like(m))
    elif kind == "negative":
        m = m - 0.7
    elif kind == "nan":
        m[m < 0.9] = float("nan")
        m[0, 0, 50:60] = -float("inf")
    elif kind == "inf":
        m = torch.where(m < 0.3, torch.full_like(m, float("inf")), m)
        m = torch.where(m > 0.8, torch.full_like(m, -float("inf")), m)
    elif kind == "denormal":
        m = m * 1e-42
    else:
        m = (m * 64).floor().to(torch.int32).add(0x3f800000).view(torch.float32)
    check_select(cuda_lib, m.contiguous(), [L, L - 1], L // 3, 4, 50)


def test_select_reports_bad_lengths(cuda_lib):
    m = torch.rand(3, 2, 100, device="cuda")
    for bad in (101, -1):
        sl = torch.tensor([80, bad, 30], dtype=torch.int32, device="cuda")
        index, new, out = cuda_lib.evict_select(m, sl, 40)
        assert cuda_lib.mala_check_status() == cuda_lib.MALA_ERR_INVALID_ARG
        assert new.tolist() == [40, 0, 30] and bool((index[1] == -1).all()) and bool((out[1] == 0).all())
        assert (index[0, 0].cpu().numpy() == chosen(m[0, 0].cpu().numpy(), 80, 40, 0, 0)).all()


def pools(n, page, H, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    bits = torch.randint(-32768, 32767, (2, n, page, H, d), generator=g, device="cuda", dtype=torch.int16)
    return bits.view(torch.bfloat16)[0], bits.view(torch.bfloat16)[1]  # any bit pattern, NaN among them


@pytest.mark.parametrize("lens,H,d,page,budget,n_sink,n_recent,same_pool", [
    ([300, 64, 1, 0, 129], 2, 128, 64, 100, 4, 10, False),
    ([300, 64, 1, 0, 129], 2, 128, 64, 100, 4, 10, True),
    ([1000], 1, 64, 128, 1, 0, 0, True),
    ([2000, 1999, 700], 3, 64, 128, 513, 0, 64, False),
    ([5000, 6000], 8, 128, 128, 2048, 4, 256, True),
])
def test_evict_moves_the_rows(cuda_lib, lens, H, d, page, budget, n_sink, n_recent, same_pool):
    B, mp, mo = len(lens), -(-max(lens) // page), -(-budget // page) + 1
    n = B * (mp + mo) + 2
    k, v = pools(n, page, H, d, seed=sum(lens))
    ids = torch.randperm(n, device="cuda").to(torch.int32)
    table, out_table = ids[:B * mp].view(B, mp).contiguous(), ids[B * mp:B * (mp + mo)].view(B, mo).contiguous()
    ko, vo = (k, v) if same_pool else pools(n, page, H, d, seed=77)
    k0, v0, ko0, vo0 = (x.clone() for x in (k, v, ko, vo))
    mass = torch.rand(B, H, mp * page, device="cuda")
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    index, new, _ = cuda_lib.evict(mass, sl, budget, k, v, table, out_table, n_sink=n_sink, n_recent=n_recent,
                                   k_out=None if same_pool else ko, v_out=None if same_pool else vo)
    assert cuda_lib.mala_check_status() == 0
    bits = lambda x: x.view(torch.int16)
    for src, dst, dst0 in ((k0, ko, ko0), (v0, vo, vo0)):
        want = bits(dst0).clone()
        for b in range(B):
            r = torch.arange(int(new[b]), device="cuda")
            to = out_table[b].long()[r // page]
            for h in range(H):
                i = index[b, h, :len(r)].long()
                want[to, r % page, h] = bits(src)[table[b].long()[i // page], i % page, h]
        assert torch.equal(bits(dst), want)  # the rows that remain, and every other row as it was
    if not same_pool:
        assert torch.equal(bits(k), bits(k0)) and torch.equal(bits(v), bits(v0))


def test_gather_reports_bad_rows(cuda_lib):
    """A page outside a pool, in either table, or an index past the table: reported, the row not copied."""
    k, v = pools(12, 64, 2, 64, seed=1)
    table = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")
    out_table = torch.tensor([[5, 6]], dtype=torch.int32, device="cuda")
    index = torch.arange(100, dtype=torch.int32, device="cuda").repeat(1, 2, 1)
    new = torch.tensor([100], dtype=torch.int32, device="cuda")
    ok_k, ok_v = k.clone(), v.clone()
    cuda_lib.evict_gather(index, new, ok_k, ok_v, table, out_table)
    assert cuda_lib.mala_check_status() == 0
    for what in ("table", "out", "index", "negative"):
        tb, ot, ix = table.clone(), out_table.clone(), index.clone()
        if what == "table":
            tb[0, 0] = 12
        elif what == "out":
            ot[0, 0] = -1
        elif what == "index":
            ix[0, :, :64] = 192
        else:
            ix[0, :, :64] = -5
        kc, vc = k.clone(), v.clone()
        cuda_lib.evict_gather(ix, new, kc, vc, tb, ot)
        assert cuda_lib.mala_check_status() == cuda_lib.MALA_ERR_INVALID_ARG
        for got, was, ok in ((kc, k, ok_k), (vc, v, ok_v)):
            got, was, ok = (x.view(torch.int16) for x in (got, was, ok))
            assert torch.equal(got[5], was[5])           # rows 0 .. 63 had the bad entry
            assert torch.equal(got[6], ok[6])            # the others are copied
    assert cuda_lib.mala_check_status() == 0


def test_select_is_the_same_in_a_graph_and_on_a_stream(cuda_lib):
    m = torch.rand(2, 4, 30000, device="cuda")
    sl = torch.tensor([30000, 25000], dtype=torch.int32, device="cuda")
    want = cuda_lib.evict_select(m, sl, 3000, 4, 100)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = cuda_lib.evict_select(m, sl, 3000, 4, 100, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b = cuda_lib.evict_select(m, sl, 3000, 4, 100)
    g.replay()
    for x, y, z in zip(want, a, b):
        assert torch.equal(x, y) and torch.equal(x, z)
    m.copy_(torch.rand_like(m))
    g.replay()
    for x, y in zip(cuda_lib.evict_select(m, sl, 3000, 4, 100), b):
        assert torch.equal(x, y)


def test_binding_checks(cuda_lib):
    m = torch.rand(2, 4, 100, device="cuda")
    sl = torch.ones(2, dtype=torch.int32, device="cuda")
    for args in ((m, sl, 0), (m.double(), sl, 5), (m[..., ::2], sl, 5), (m, sl.long(), 5), (m, sl[:1], 5)):
        with pytest.raises(ValueError):
            cuda_lib.evict_select(*args)
    with pytest.raises(cuda_lib.MalaError):
        cuda_lib.evict_select(m, sl, 5, n_sink=6)
    with pytest.raises(cuda_lib.MalaError):
        cuda_lib.evict_select(m, sl, 5, mass_out=torch.zeros(2, 4, 4, device="cuda"))
    with pytest.raises(ValueError):
        cuda_lib.evict_select(m, sl, 5, mass_out=torch.zeros(2, 3, 5, device="cuda"))
    index, new, _ = cuda_lib.evict_select(m, sl, 5)
    k, v = pools(4, 64, 4, 64, seed=1)
    t = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        cuda_lib.evict_gather(index, new, k, v[:3], t, t)
    with pytest.raises(ValueError):
        cuda_lib.evict_gather(index, new, k, v, t[:1], t)
    with pytest.raises(ValueError):
        cuda_lib.evict_gather(index[:, :2].contiguous(), new, k, v, t, t)


@pytest.mark.parametrize("kind", ["spread", "few", "equal", "nan"])
@pytest.mark.parametrize("n,ld", [(1, 1024), (3, 1025), (3, 3900), (2, 33000), (2, 200000), (20, 100000), (40, 60000),
                                  (80, 15000), (80, 32700), (80, 32800), (40, 66000)])
def test_select_at_every_length_of_a_thread(cuda_lib, kind, n, ld):
    """Rows that leave a thread one mass, a few, up to 32 and more, by one CTA and by clusters; lengths beside warps' ends."""
    g = torch.Generator(device="cuda").manual_seed(ld)
    m = torch.rand(n, 1, ld, generator=g, device="cuda")
    if kind == "spread":
        m = 1.0 / (m + 1e-4)
    elif kind == "few":
        m = (m * 3).floor() - 1.0
    elif kind == "equal":
        m.fill_(2.0)
    else:
        m[m < 0.99] = float("nan")
    lens = [ld, ld - 1, ld - 33][:n] + [ld - 31 * i for i in range(3, n)]
    check_select(cuda_lib, m, lens, ld // 5, 3, 40)


def test_gather_captured_behind_a_join(cuda_lib):
    """The copy alone in a captured graph, behind work of two streams that both write what it reads, and behind a copy."""
    k, v = pools(24, 64, 2, 64, seed=3)
    table = torch.randperm(24, device="cuda")[:8].to(torch.int32).view(2, 4)
    to = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    index = torch.zeros(2, 2, 150, dtype=torch.int32, device="cuda")
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    rows = torch.stack([torch.randperm(256, device="cuda")[:150].sort()[0] for _ in range(4)]).view(2, 2, 150)
    rows = rows.to(torch.int32)
    ko, vo = torch.zeros(2, 6, 64, 2, 64, dtype=torch.bfloat16, device="cuda").unbind()
    out = (torch.zeros_like(ko), torch.zeros_like(vo))
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            new.fill_(150)
        index.add_(rows)
        torch.cuda.current_stream().wait_stream(side)
        cuda_lib.evict_gather(index, new, k, v, table, to, ko, vo)
        out[0].copy_(ko)
        new.mul_(1)
        cuda_lib.evict_gather(index, new, k, v, table, to, ko, vo)
        out[1].copy_(vo)
        index.zero_()
        new.zero_()
    for _ in range(3):
        ko.zero_()
        vo.zero_()
        g.replay()
        torch.cuda.synchronize()
        for pool, got in ((k, out[0]), (v, out[1])):
            for b in range(2):
                old = pool[table[b].long()].flatten(0, 1)
                fresh = got[to[b].long()].flatten(0, 1)
                for h in range(2):
                    want = old[rows[b, h].long(), h]
                    assert torch.equal(fresh[:150, h].view(torch.int16), want.view(torch.int16))
    assert cuda_lib.mala_check_status() == 0
