"""Paged decode that collects each key's weight (mala_decode_paged_mass): behind a
gate its attention equals mala_decode_paged bit for bit; without one (another
kernel) it is held to 64 bits; its masses equal weights formed in 64 bits from its
own LSE.

Tolerance of a weight, relative: the score is an fp32 sum of d products (d 2^-24
scale sum_c |q_c k_c|), x = s log2e - LSE log2e rounds at its terms' size
(3 x 2^-24 (|s| + |LSE|) log2e), exp2 is good to 2^-21, the sums of at most eight
terms and the decayed mass to 8 x 2^-24. An output: rounded once to bf16 (2^-8 of
its value at most, 2^-9 on average), from probabilities held to 16 bits.
"""
import pytest
import torch

from test_rope_gpu import paged

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634


def reference(q, k, lse, scale, mass, decay, ld):
    """One sequence: q [Hq, d], k [n, Hkv, d], lse [Hq] -> (mass [Hkv, ld] in 64 bits, relative bound)."""
    n, Hkv, d = k.shape
    G = q.shape[0] // Hkv
    s = torch.einsum("hgd,nhd->hgn", q.double().view(Hkv, G, d), k.double()) * scale
    a = torch.einsum("hgd,nhd->hgn", q.double().abs().view(Hkv, G, d), k.double().abs())
    out = torch.zeros(Hkv, ld, device="cuda", dtype=torch.float64)
    if mass is not None and decay:
        out[:, :n - 1] = decay * mass[:, :n - 1].double()
    out[:, :n] += torch.exp(s - lse.double().view(Hkv, G, 1)).sum(1)
    rel = d * 2.0 ** -24 * scale * float(a.max()) + 3 * 2.0 ** -24 * LOG2E * float(s.abs().max() + lse.abs().max()) + \
        2.0 ** -21 + 8 * 2.0 ** -24
    return out, rel


def gathered(pages, table, n):
    return pages[table.long()].flatten(0, 1)[:n]


CASES = [
    # lens, Hq, Hkv, d, page, tau, n_splits
    ([1], 1, 1, 64, 64, 0.0, 0),
    ([300, 1, 64, 65], 8, 2, 128, 64, 0.0, 3),
    ([300, 1, 64, 65], 8, 2, 128, 64, 1.0, 3),
    ([5000, 128, 3333], 32, 8, 128, 128, 1.0, 0),
    ([5000, 128, 3333], 32, 8, 128, 128, 0.0, 7),
    ([1000, 999], 6, 2, 64, 128, 1.0, 2),     # groups of three
    ([700, 20], 16, 2, 64, 64, 4.0, 0),       # groups of eight
    ([700, 20], 16, 2, 128, 128, 0.0, 4),
    ([2100], 3, 3, 128, 64, 1.0, 40),         # more splits than tiles
    ([900, 130], 10, 2, 128, 128, 1.0, 2),    # groups of five
    ([64, 1, 700, 65, 64, 333, 2, 128] * 9, 8, 2, 128, 64, 0.0, 0),   # runs over many short sequences
    ([40000, 17], 8, 1, 64, 128, 0.0, 0),     # and over a part of one long one
    ([30001], 16, 2, 128, 128, 0.0, 0),
    ([129, 4000], 5, 1, 64, 64, 0.0, 0),
]


@pytest.mark.parametrize("lens,Hq,Hkv,d,page,tau,n_splits", CASES)
def test_decode_paged_mass(cuda_lib, lens, Hq, Hkv, d, page, tau, n_splits):
    B, scale = len(lens), d ** -0.5
    kp, vp, table = paged(B, max(lens), Hkv, d, page, seed=sum(lens) + d)
    g = torch.Generator(device="cuda").manual_seed(Hq)
    q = (2 * torch.randn(B, Hq, d, generator=g, device="cuda")).to(torch.bfloat16)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ld = table.shape[1] * page + 10
    mass = torch.rand(B, Hkv, ld, device="cuda")
    o, lse, kept, km, ns, got = cuda_lib.decode_paged_mass(q, kp, vp, table, sl, scale, tau, mass=mass, decay=0.9,
                                                           n_splits=n_splits, keep_map=True)
    o2, lse2, kept2, km2, _ = cuda_lib.decode_paged(q, kp, vp, table, sl, scale, tau, n_splits=ns, keep_map=True)
    assert cuda_lib.mala_check_status() == 0
    assert torch.equal(kept, kept2) and torch.equal(km, km2) and (ns > 0) == (tau > 0)
    if tau > 0:
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    alone = cuda_lib.decode_paged_mass(q, kp, vp, table, sl, scale, tau, n_splits=n_splits)[-1]
    for b, n in enumerate(lens):
        k = gathered(kp, table[b], n)
        want, rel = reference(q[b], k, lse[b], scale, mass[b], 0.9, ld)
        assert bool(((got[b].double() - want).abs() <= rel * want).all())
        want, rel = reference(q[b], k, lse[b], scale, None, 1.0, alone.shape[-1])
        assert bool(((alone[b].double() - want).abs() <= rel * want).all())
        if tau == 0:  # the whole row's weights, and the output, from 64 bits
            v = gathered(vp, table[b], n).double()
            s = torch.einsum("hgd,nhd->hgn", q[b].double().view(Hkv, -1, d), k.double()) * scale
            assert float((torch.logsumexp(s, -1).view(-1) - lse[b].double()).abs().max()) <= rel
            p = torch.softmax(s, -1)
            want_o = torch.einsum("hgn,nhd->hgd", p, v).view(Hq, d)
            size = torch.einsum("hgn,nhd->hgd", p, v.abs()).view(Hq, d)
            err = (o[b].double() - want_o).abs()
            assert bool((err <= 2.0 ** -8 * want_o.abs() + (2.0 ** -16 + 2 * rel) * size).all())


def test_in_place_and_not_read(cuda_lib):
    kp, vp, table = paged(2, 500, 2, 64, 64, seed=3)
    q = torch.randn(2, 8, 64, device="cuda").to(torch.bfloat16)
    sl = torch.tensor([500, 77], dtype=torch.int32, device="cuda")
    mass = torch.rand(2, 2, 512, device="cuda")
    want = cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.125, 0.0, mass=mass, decay=0.5)[-1]
    m = mass.clone()
    m[0, :, 499:] = float("nan")  # the newest key starts from 0; what lies behind is not read
    m[1, :, 76:] = float("nan")
    assert torch.equal(cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.125, 0.0, mass=m, decay=0.5, out=m)[-1], want)
    nan = torch.full_like(mass, float("nan"))
    none = cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.125, 0.0, mass=nan, decay=0.0)[-1]
    assert torch.equal(none, cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.125, 0.0)[-1])


@pytest.mark.parametrize("tau", [0.0, 1.0])
@pytest.mark.parametrize("d,page,G", [(128, 128, 4), (64, 64, 1), (128, 64, 8), (64, 128, 3)])
def test_what_lies_behind_the_keys_does_not_count(cuda_lib, d, page, G, tau):
    """The last page's other rows and every other page hold NaN and infinities; idle slots have length 0."""
    lens = [page * 3 + 5, 0, 1, page]
    kp, vp, table = paged(4, max(lens), 2, d, page, seed=d)
    q = torch.randn(4, 2 * G, d, device="cuda").to(torch.bfloat16)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    live = torch.zeros(kp.shape[:2], dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for j in range(n):
            live[int(table[b, j // page]), j % page] = True
    want = cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.1, tau, n_splits=2)
    kp[~live] = float("nan")
    vp[~live] = float("inf")
    got = cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.1, tau, n_splits=2)
    assert cuda_lib.mala_check_status() == 0  # the idle slot is no error
    for x, y in ((want[0], got[0]), (want[1], got[1]), (want[2], got[2]), (want[5], got[5])):
        assert torch.equal(x, y)
    assert bool((got[0][1] == 0).all()) and bool((got[1][1] == float("-inf")).all()) and bool((got[5][1] == 0).all())
    assert bool(torch.isfinite(got[0].float()).all())


def test_bad_tables_are_reported(cuda_lib):
    kp, vp, table = paged(2, 300, 2, 64, 64, seed=9)
    q = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    ok = torch.tensor([300, 200], dtype=torch.int32, device="cuda")
    want = cuda_lib.decode_paged_mass(q, kp, vp, table, ok, 0.125, 0.0, n_splits=2)
    for value in (table.shape[1] * 64 + 1, -2):
        sl = ok.clone()
        sl[1] = value
        got = cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.125, 0.0, n_splits=2)
        assert cuda_lib.mala_check_status() == cuda_lib.MALA_ERR_INVALID_ARG
        assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[5][0], want[5][0])
        assert bool((got[5][1] == 0).all())
    tb = table.clone()
    tb[1, 1] = kp.shape[0] + 3
    got = cuda_lib.decode_paged_mass(q, kp, vp, tb, ok, 0.125, 0.0, n_splits=2)
    assert cuda_lib.mala_check_status() == cuda_lib.MALA_ERR_INVALID_ARG
    assert torch.equal(got[5][0], want[5][0])
    cuda_lib.decode_paged_mass(q, kp, vp, table, ok, 0.125, 0.0, n_splits=2)
    assert cuda_lib.mala_check_status() == 0


@pytest.mark.parametrize("tau,tile,reached", [
    (1.0, 2, True), (0.0, 1, True), (0.0, 0, True),
    (0.0, 2, False),  # twenty tiles in runs of two: no run has a tile 2
])
def test_a_wait_that_runs_out_is_reported(cuda_lib, tau, tile, reached):
    kp, vp, table = paged(1, 600, 2, 64, 64, seed=9)
    q = torch.randn(1, 4, 64, device="cuda").to(torch.bfloat16)
    sl = torch.tensor([600], dtype=torch.int32, device="cuda")
    want = cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.125, tau, n_splits=1)
    cuda_lib.mala_test_hooks(20_000_000, tile, None)
    try:
        cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.125, tau, n_splits=1)
        assert cuda_lib.mala_check_status() == (cuda_lib.MALA_ERR_DEVICE_TIMEOUT if reached else 0)
    finally:
        cuda_lib.mala_test_hooks(0, -1, None)
    got = cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.125, tau, n_splits=1)
    assert cuda_lib.mala_check_status() == 0
    assert torch.equal(got[5], want[5])


def test_graph_and_stream(cuda_lib):
    """A captured step replayed after the cache grew by a token, and the same on another stream."""
    kp, vp, table = paged(3, 400, 2, 128, 128, seed=12)
    q = torch.randn(3, 8, 128, device="cuda").to(torch.bfloat16)
    sl = torch.tensor([400, 128, 7], dtype=torch.int32, device="cuda")
    mass = torch.rand(3, 2, table.shape[1] * 128, device="cuda")
    run = lambda **kw: cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.09, 1.0, mass=mass, decay=0.9, **kw)
    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b = run()
    g.replay()
    assert torch.equal(a[0], want[0]) and torch.equal(a[5], want[5])
    assert torch.equal(b[0], want[0]) and torch.equal(b[5], want[5])
    sl.add_(1)
    g.replay()
    want = run()
    assert torch.equal(b[0], want[0]) and torch.equal(b[5], want[5]) and torch.equal(b[2], want[2])


def test_binding_checks(cuda_lib):
    kp, vp, table = paged(2, 100, 2, 64, 64, seed=9)
    q = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    sl = torch.tensor([100, 50], dtype=torch.int32, device="cuda")
    for kw in (dict(q=q.float()), dict(v_pages=vp[:1]), dict(block_table=table[:1]), dict(seqlens_k=sl[:1]),
               dict(seqlens_k=sl.long()), dict(mass=torch.zeros(2, 1, 128, device="cuda")),
               dict(k_pages=kp.transpose(1, 2), v_pages=vp.transpose(1, 2))):
        a = dict(q=q, k_pages=kp, v_pages=vp, block_table=table, seqlens_k=sl, scale=0.1, tau=0.0)
        a.update(kw)
        with pytest.raises(ValueError):
            cuda_lib.decode_paged_mass(**a)
    with pytest.raises(cuda_lib.MalaError):
        cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.1, 0.0, mass=torch.zeros(2, 2, 127, device="cuda"))
