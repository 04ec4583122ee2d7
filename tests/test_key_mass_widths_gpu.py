"""Key mass of few rows at every width of the kernel that holds them: 64, 128, 192 and
256 columns in one block and 192 and 256 in two, head sizes both, with several key
tiles to a CTA and earlier masses. Bounds are those of test_key_mass_gpu.
"""
import pytest
import torch

from test_key_mass_gpu import close, inputs, lse_of, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,window,columns", [
    (2, 30, 64), (4, 64, 256), (3, 37, 120), (4, 40, 160), (3, 60, 192), (7, 35, 280), (4, 90, 384), (7, 48, 336), (2, 190, 384),
    (5, 80, 400), (8, 64, 512),
])
def test_width(cuda_lib, d, G, window, columns):
    assert (window + 7) // 8 * 8 * G == columns
    B, Hkv, Lk = 3, 8, 3001
    for Lq in (window, window + 300):
        q, k = inputs(B, G * Hkv, Hkv, Lq, Lk, d, seed=columns + d)
        scale = d ** -0.5
        lse = lse_of(q, k, scale)
        mass = torch.rand(B, Hkv, Lk + 9, device="cuda") * 20
        got = cuda_lib.key_mass(q, k, lse, scale, window=window, mass=mass, decay=0.75)
        assert cuda_lib.mala_check_status() == 0
        for b in range(B):
            want, rel = reference(q[b], k[b], lse[b], scale, window, mass[b], 0.75, Lk + 9)
            close(got[b], want, rel, G * Lq)


def test_width_of_a_packed_batch(cuda_lib):
    """336 columns, sequences shorter than the window among them: another sequence's rows lie behind theirs."""
    lens_q, lens_k, Hq, Hkv, d, window = [48, 7, 0, 300, 1], [48, 900, 500, 4000, 2000], 14, 2, 128, 48
    S, tq, tk = len(lens_q), sum(lens_q), sum(lens_k)
    q, k = (x[0] for x in inputs(1, Hq, Hkv, tq, tk, d, seed=5))
    cq = torch.tensor([0] + lens_q, device="cuda").cumsum(0).to(torch.int32)
    ck = torch.tensor([0] + lens_k, device="cuda").cumsum(0).to(torch.int32)
    lse = torch.zeros(Hq, tq, device="cuda")
    for s in range(S):
        a, b = slice(int(cq[s]), int(cq[s + 1])), slice(int(ck[s]), int(ck[s + 1]))
        if lens_q[s]:
            lse[:, a] = lse_of(q[None, a], k[None, b], 0.1)[0]
    ld = max(lens_k)
    mass = torch.rand(S, Hkv, ld, device="cuda")
    got = cuda_lib.key_mass_varlen(q, k, lse, cq, ck, max(lens_q), ld, 0.1, window=window, mass=mass, decay=1.5)
    assert cuda_lib.mala_check_status() == 0
    for s in range(S):
        a, b = slice(int(cq[s]), int(cq[s + 1])), slice(int(ck[s]), int(ck[s + 1]))
        want, rel = reference(q[a], k[b], lse[:, a], 0.1, window, mass[s], 1.5, ld)
        # (a sequence without queries has no other bound than that of decay * mass, one rounding)
        close(got[s], want, rel + 2.0 ** -24, 7 * max(1, lens_q[s]))
