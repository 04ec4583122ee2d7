"""An eviction that is refused leaves everything as it was, also where only its second half
(the copy into other pages) cannot be done."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def setting():
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(12, 64, 2, 64, generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn(12, 64, 2, 64, generator=g, device="cuda").to(torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    return dict(mass=torch.rand(1, 2, 256, generator=g, device="cuda"), seqlens_k=i32(200), budget=100, k_pages=k,
                v_pages=v, block_table=i32([0, 1, 2, 3]), out_table=i32([6, 7]))


@pytest.mark.parametrize("kw,error", [
    (dict(out_table=lambda a: a["out_table"][:, :1].contiguous()), "MalaError"),    # 64 rows of room for 100
    (dict(out_table=lambda a: a["out_table"].long()), "ValueError"),
    (dict(out_table=lambda a: a["out_table"].repeat(2, 1)), "ValueError"),
    (dict(v_pages=lambda a: a["v_pages"][:11]), "ValueError"),
    (dict(k_out=lambda a: a["k_pages"][:, :, :1].contiguous()), "ValueError"),
    (dict(k_out=lambda a: torch.empty(12 * 64 * 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(12, 64, 2, 64)),
     "MalaError"),  # not 16-byte aligned
    (dict(block_table=lambda a: a["block_table"].cpu()), "ValueError"),
    (dict(budget=lambda a: 0), "ValueError"),
    (dict(n_sink=lambda a: 101), "MalaError"),
])
def test_a_refused_eviction_writes_nothing(cuda_lib, kw, error):
    a = setting()
    changed = {n: f(a) for n, f in kw.items()}
    a.update(changed)
    out = torch.full((1, 2, 128), 7.0, device="cuda")
    was = {n: x.clone() for n, x in a.items() if isinstance(x, torch.Tensor)}
    with pytest.raises(cuda_lib.MalaError if error == "MalaError" else ValueError):
        cuda_lib.evict(**a, mass_out=out)
    torch.cuda.synchronize()
    assert cuda_lib.mala_check_status() == 0
    assert bool((out == 7.0).all())
    bits = lambda x: x.view(torch.int16) if x.dtype == torch.bfloat16 else x  # (uninitialised memory may hold NaN)
    for n, x in was.items():
        assert torch.equal(bits(a[n]), bits(x)), n
