"""Key mass on the GPU at scores that the tensor cores sum without an error, so that the
rest of the arithmetic shows.

Every row and key are alike and every product and partial sum is a small multiple of
1/2, exact in the accumulator whatever its order and however it drops bits. The LSE is
the fp32 value, among those next to the score, whose product with the log2(e) that the
fp32 scale carries lies closest to an fp32 value (within 2^-6 of a step, of at most
2^-18 at 64: 6e-8), so that its rounding does not show either. What is left is exp2
(ex2.approx and the polynomial are both good to 2^-22) and the sums of equal terms
(64 of them in fp32, at most 8 additions deep, and the compensated sum): 2^-21 in all.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

SHAPES = [(2000, 2000, 0), (700, 1500, 0), (64, 3000, 0), (1200, 4000, 100)]  # walks, cut walks, few rows, a window


def quiet_lse(s, scale):
    """An fp32 LSE beside s whose product with fl(scale log2 e) / scale is next to an fp32 value."""
    ratio = float(np.float32(scale * 1.4426950408889634)) / scale
    near = np.float32(s) + np.arange(-200, 201, dtype=np.float32) * np.spacing(np.float32(s))
    x = near.astype(np.float64) * ratio
    off = np.abs(x - x.astype(np.float32).astype(np.float64))
    best = int(off.argmin())
    assert off[best] <= 2.0 ** -6 * np.spacing(np.float32(x[best]))
    return float(near[best])


def alike(Lq, Lk, d, where, Hq=4, Hkv=2):
    """q, k with every score's sum 352, its products in one block of 16 channels or in all of them."""
    qv = torch.zeros(d)
    kv = torch.zeros(d)
    if where == "all":
        qv[:64], kv[:64] = 2.75, 2.0
        if d == 128:
            qv[:], kv[:] = 2.75, 1.0
    else:
        at = slice(0, 16) if where == "first" else slice(d - 16, d)
        qv[at], kv[at] = 5.5, 4.0
    assert float((qv.double() * kv.double()).sum()) == 352.0
    q = qv.to("cuda", torch.bfloat16).expand(1, Lq, Hq, d).contiguous()
    k = kv.to("cuda", torch.bfloat16).expand(1, Lk, Hkv, d).contiguous()
    return q, k


@pytest.mark.parametrize("where", ["first", "last", "all"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq,Lk,window", SHAPES)
def test_weights_of_exact_scores(cuda_lib, Lq, Lk, window, d, where):
    q, k = alike(Lq, Lk, d, where)
    scale = 0.125
    lse = quiet_lse(352 * scale, scale)
    got = cuda_lib.key_mass(q, k, torch.full((1, 4, Lq), lse, device="cuda"), scale, window=window).double()
    assert cuda_lib.mala_check_status() == 0
    pos = torch.arange(Lk - (window or Lq), Lk, device="cuda")
    rows = (pos[None] >= torch.arange(Lk, device="cuda")[:, None]).sum(1)  # that see key j
    want = 2 * rows * np.exp(352 * scale - lse)
    err = ((got[0] - want).abs() / want).max()
    assert float(err) <= 2.0 ** -21, float(err)


@pytest.mark.parametrize("Lq,Lk,window", SHAPES)
def test_a_row_with_an_infinite_lse_adds_exactly_nothing(cuda_lib, Lq, Lk, window):
    q, k = alike(Lq, Lk, 64, "all")
    lse = torch.full((1, 4, Lq), float("inf"), device="cuda")
    got = cuda_lib.key_mass(q, k, lse, 0.125, window=window)
    assert cuda_lib.mala_check_status() == 0
    assert bool((got == 0).all()), float(got.max())


@pytest.mark.parametrize("what", ["nan query", "nan lse", "overflow"])
@pytest.mark.parametrize("Lq,Lk,window", SHAPES)
def test_a_broken_row_shows_in_every_key_that_it_sees(cuda_lib, Lq, Lk, window, what):
    """Wherever the row stands among 16 and among the strips: all of its keys' masses are not finite, and no other's."""
    q, k = alike(Lq, Lk, 64, "all")
    base = torch.full((1, 4, Lq), 44.0, device="cuda")
    first = Lq - (window or Lq)
    for r in list(range(first, min(first + 18, Lq))) + list(range(Lq - 18, Lq)):
        q2, lse = q.clone(), base.clone()
        if what == "nan query":
            q2[0, r, 1] = float("nan")
        elif what == "nan lse":
            lse[0, 1, r] = float("nan")
        else:
            lse[0, 1, r] = -100.0  # the weight is e^144
        got = cuda_lib.key_mass(q2, k, lse, 0.125, window=window)
        seen = torch.arange(Lk, device="cuda") <= r + Lk - Lq
        assert bool((~got[0, 0].isfinite() == seen).all()), r
        assert bool(got[0, 1].isfinite().all())
    assert cuda_lib.mala_check_status() == 0
