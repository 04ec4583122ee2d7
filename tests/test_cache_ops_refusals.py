"""More of what the host refuses of the operators beside attention (no call here reaches CUDA)."""
import pytest

import mass_gated_causal_b200 as mala
from test_cache_ops_abi import P, mass, select, vmass


@pytest.mark.parametrize("kw", [
    # 2 x 2 rows of 1000 masses from P on: the last byte of them, the first row's end, all of them within
    dict(mass_out=P + 4 * 4000 - 16), dict(mass_out=P + 4 * 1000), dict(mass=1 << 20, mass_out=(1 << 20) - 16),
    dict(mass=1 << 20, mass_out=(1 << 20) - 4 * 4 * 200 + 16),  # 2 x 2 x 200 masses out, their last four
    dict(mass=1 << 20, mass_out=1 << 24, new_seqlens=4 * P, seqlens_k=4 * P + 4),
    dict(mass=1 << 20, mass_out=1 << 24, new_seqlens=4 * P + 4, seqlens_k=4 * P),
])
def test_evict_select_rejects_overlaps(kw):
    a = dict(mass=P, mass_out=1 << 24, index=1 << 22, new_seqlens=1 << 23, seqlens_k=(1 << 23) + 8)
    a.update(kw)
    assert select(**a) == 1


def test_workspace_of_heads_that_do_not_group_is_0():
    assert mala.mala_decode_mass_workspace_size(4, 8, 2, 128, 128, 40, 0) > 0
    assert mala.mala_decode_mass_workspace_size(4, 8, 3, 128, 128, 40, 0) == 0
    assert mala.mala_decode_mass_workspace_size(4, 2, 8, 128, 128, 40, 4) == 0


@pytest.mark.parametrize("scale,code", [(2.0 ** -65, 2), (1e-42, 2), (2.0 ** 65, 2)])
def test_key_mass_rejects_scales_that_leave_the_range(scale, code):
    assert mass(scale=scale) == code and vmass(scale=scale) == code
    assert mass(scale=2.0 ** -64, workspace=None) == 3 and vmass(scale=2.0 ** 64, workspace=None) == 3
