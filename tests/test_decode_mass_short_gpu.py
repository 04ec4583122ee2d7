"""Ungated decode with masses on both sides of its choice of kernel: short caches, each
taken by one cluster (every cluster size, every tile count, every group), and tables
with room for long ones, whose tiles are dealt over the whole GPU. Bounds are those
of test_decode_mass_gpu.
"""
import pytest
import torch

from test_decode_mass_gpu import gathered, reference, test_decode_paged_mass as check_case
from test_rope_gpu import paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,Hq,Hkv,d,page", [
    ([50, 64, 1, 33] * 35, 8, 2, 128, 64),         # one CTA, one tile
    ([500, 1, 65] * 40, 4, 2, 128, 64),            # one CTA, eight tiles
    ([900, 17] * 30, 6, 2, 64, 128),               # two CTAs
    ([2000, 511] * 18, 4, 2, 64, 64),              # four
    ([513, 1024], 1, 1, 64, 64),                   # eight, two tiles each
    ([4000, 63, 129], 24, 3, 128, 128),            # sixteen, groups of eight
    ([8192, 8129], 6, 2, 64, 128),                 # sixteen with eight tiles each, groups of three
    ([8000], 16, 2, 128, 64),                      # the same, one CTA to an SM
    ([8193, 12], 8, 2, 128, 64),                   # a tile too long
    ([500, 1, 65] * 60, 4, 2, 64, 128),            # too many clusters
    ([64, 1, 700, 65, 64, 333, 2, 128] * 9 + [9000], 8, 2, 128, 64),  # runs over many short sequences
])
def test_both_sides(cuda_lib, lens, Hq, Hkv, d, page):
    check_case(cuda_lib, lens, Hq, Hkv, d, page, 0.0, 0)


@pytest.mark.parametrize("room", [1, 9000])
@pytest.mark.parametrize("d,page,G", [(128, 128, 4), (64, 64, 1), (128, 64, 8), (64, 128, 3)])
def test_idle_slots_and_odd_ends(cuda_lib, d, page, G, room):
    """Lengths at and beside tile ends among idle slots; the last pages' other rows, and every other page, hold NaN."""
    lens = [0, 1, 63, 64, 0, 65, 127, 0]
    B = len(lens)
    kp, vp, table = paged(B, max(*lens, room), 2, d, page, seed=d + room)
    live = torch.zeros(kp.shape[:2], dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for j in range(n):
            live[int(table[b, j // page]), j % page] = True
    kp[~live] = float("nan")
    vp[~live] = float("nan")
    q = torch.randn(B, 2 * G, d, device="cuda").to(torch.bfloat16)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ld = table.shape[1] * page + 3
    mass = torch.rand(B, 2, ld, device="cuda")
    o, lse, kept, km, _, got = cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.1, 0.0, mass=mass, decay=0.5,
                                                          keep_map=True)
    assert cuda_lib.mala_check_status() == 0
    for b, n in enumerate(lens):
        pages = -(-n // page)
        assert kept.view(B, -1)[b].tolist() == [pages] * (2 * G)
        assert bool((km[b, :, :pages] == 1).all()) and bool((km[b, :, pages:] == 255).all())
        assert bool((got[b, :, n:] == 0).all())
        if n == 0:
            assert bool((o[b] == 0).all()) and bool((lse[b] == float("-inf")).all())
            continue
        k, v = gathered(kp, table[b], n), gathered(vp, table[b], n).double()
        want, rel = reference(q[b], k, lse[b], 0.1, mass[b], 0.5, ld)
        assert bool(((got[b].double() - want).abs() <= rel * want).all())
        s = torch.einsum("hgd,nhd->hgn", q[b].double().view(2, G, d), k.double()) * 0.1
        p = torch.softmax(s, -1)
        want_o = torch.einsum("hgn,nhd->hgd", p, v).reshape(2 * G, d)
        size = torch.einsum("hgn,nhd->hgd", p, v.abs()).reshape(2 * G, d)
        assert bool(((o[b].double() - want_o).abs() <= 2.0 ** -8 * want_o.abs() + (2.0 ** -16 + 2 * rel) * size).all())


@pytest.mark.parametrize("room", [300, 20000])
def test_bad_lengths_and_pages_are_reported(cuda_lib, room):
    kp, vp, table = paged(2, room, 2, 64, 64, seed=9)
    q = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    ok = torch.tensor([300, 200], dtype=torch.int32, device="cuda")
    want = cuda_lib.decode_paged_mass(q, kp, vp, table, ok, 0.125, 0.0)
    for value in (table.shape[1] * 64 + 1, -2):
        sl = ok.clone()
        sl[1] = value
        got = cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.125, 0.0)
        assert cuda_lib.mala_check_status() == cuda_lib.MALA_ERR_INVALID_ARG
        assert bool((got[0][1] == 0).all()) and bool((got[5][1] == 0).all())
        # the sound sequence: its runs may be cut elsewhere, so its LSE may differ in rounding
        torch.testing.assert_close(got[5][0], want[5][0], rtol=2.0 ** -19, atol=0)
    tb = table.clone()
    tb[1, 1] = -1
    got = cuda_lib.decode_paged_mass(q, kp, vp, tb, ok, 0.125, 0.0)
    assert cuda_lib.mala_check_status() == cuda_lib.MALA_ERR_INVALID_ARG
    assert torch.equal(got[5][0], want[5][0])


@pytest.mark.parametrize("room,tile,reached", [
    (4000, 0, True), (4000, 3, True), (4000, 4, False),  # 64 tiles over clusters of sixteen
    (9000, 1, True), (9000, 2, False),                   # 64 tiles a head in runs of two
])
def test_a_wait_that_runs_out_is_reported(cuda_lib, room, tile, reached):
    kp, vp, table = paged(1, room, 2, 64, 64, seed=9)
    q = torch.randn(1, 4, 64, device="cuda").to(torch.bfloat16)
    sl = torch.tensor([4000], dtype=torch.int32, device="cuda")
    want = cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.125, 0.0)
    cuda_lib.mala_test_hooks(20_000_000, tile, None)
    try:
        cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.125, 0.0)
        assert cuda_lib.mala_check_status() == (cuda_lib.MALA_ERR_DEVICE_TIMEOUT if reached else 0)
    finally:
        cuda_lib.mala_test_hooks(0, -1, None)
    got = cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.125, 0.0)
    assert cuda_lib.mala_check_status() == 0
    assert torch.equal(got[5], want[5])


def test_streams_and_graphs_at_once(cuda_lib):
    """Two steps of short caches on two streams, and a captured one between them."""
    kp, vp, table = paged(4, 2000, 2, 128, 64, seed=5)
    q = torch.randn(4, 8, 128, device="cuda").to(torch.bfloat16)
    sl = torch.tensor([2000, 1, 777, 1024], dtype=torch.int32, device="cuda")
    run = lambda **kw: cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 0.09, 0.0, **kw)
    want = run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = run()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        got += [run(stream=s) for s in side]
        g.replay()
    torch.cuda.synchronize()
    for x in got + [c]:
        assert torch.equal(x[0], want[0]) and torch.equal(x[1], want[1]) and torch.equal(x[5], want[5])
    assert cuda_lib.mala_check_status() == 0
