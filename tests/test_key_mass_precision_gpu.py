"""How exact key mass is on inputs whose products the tensor cores cannot sum exactly, from
an exact LSE: diffuse attention, concentrated attention, large scores, long rows, by both
kernels.

The accumulator drops bits of every partial sum toward zero, about half a step: 4.3e-8 of
the partial sum on average (a step is 2^-23 to 2^-24 of a number, 0.72 x 2^-23 on
average). With -LSE added after 5 of 8 sixteenths of the channels (3 of 4), and the
channels alike, what is dropped before and after has opposite signs. For a score near the
LSE the two leave 1.1 (d = 64: 1.25) times 4.3e-8 of the LSE, for one near 0 they leave 3
(1), where LSEs taken off at the end leave 3.5 (1.5) of a large score. So the masses'
relative L2 error is held to 1.25 x 4.3e-8 of the largest LSE where few keys hold a row's
weight (prompts, large scores), else to 3 x that, and 2^-22 for exp2 and the sums.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


def inputs(kind, Lq, Lk, Hq, Hkv, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    q, k = r(Lq, Hq, d), r(Lk, Hkv, d)
    if kind == "prompt":  # chunks of keys like their queries
        z = r(-(-Lk // 32), Hkv, d).repeat_interleave(32, 0)[:Lk]
        k = 0.8 * z + 0.6 * k
        q = 1.0 * z[Lk - Lq:].repeat_interleave(Hq // Hkv, 1) + q
    elif kind == "offset":  # every score large, none above the others
        u = r(d)
        q, k = q + 8 * u / u.norm(), k + 8 * u / u.norm()
    elif kind == "large":
        q = 4 * q
    return q.to(torch.bfloat16), k.to(torch.bfloat16)


@pytest.mark.parametrize("kind", ["diffuse", "prompt", "offset", "large"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq,Lk", [(3000, 3000), (50, 9000)])
def test_relative_error(cuda_lib, Lq, Lk, d, kind):
    Hq, Hkv, scale = 4, 2, d ** -0.5
    q, k = inputs(kind, Lq, Lk, Hq, Hkv, d, seed=Lq + d)
    want = torch.zeros(Hkv, Lk, dtype=torch.float64, device="cuda")
    lse = torch.empty(Hq, Lq, device="cuda")
    late = torch.arange(Lk, device="cuda")[None] > torch.arange(Lk - Lq, Lk, device="cuda")[:, None]
    for h in range(Hq):
        s = (q[:, h].double() @ k[:, h // 2].double().T) * scale
        s.masked_fill_(late, -float("inf"))
        lse[h] = torch.logsumexp(s, -1).float()
        want[h // 2] += torch.exp(s - lse[h].double()[:, None]).sum(0)
    got = cuda_lib.key_mass(q[None], k[None], lse[None], scale)[0].double()
    assert cuda_lib.mala_check_status() == 0
    top = float(lse.max())
    bound = (1.25 if kind in ("prompt", "large") else 3.0) * 4.3e-8 * top + 2.0 ** -22
    rel = float((got - want).norm() / want.norm())
    assert rel <= bound, (rel, bound, top)
