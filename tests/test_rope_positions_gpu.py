"""Positions of several axes are [n_axes, ...tokens]; a tensor of as many values laid out
otherwise (a token's axes side by side) is refused, not read as something else."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_positions_laid_out_by_token_are_refused(cuda_lib):
    T, d = 6, 64
    q = torch.randn(T, 4, d, device="cuda").to(torch.bfloat16)
    k = torch.randn(T, 2, d, device="cuda").to(torch.bfloat16)
    f = torch.rand(d // 2, device="cuda")
    pos = torch.randint(0, 50, (3, T), dtype=torch.int32, device="cuda")
    sec = (16, 8, 8)
    want = cuda_lib.rope(q, k, k, pos, f, sections=sec)
    for same in (pos.view(3, 2, 3), pos.view(3, T, 1), pos.flatten()):
        got = cuda_lib.rope(q, k, k, same, f, sections=sec)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    kp = torch.zeros(2, 64, 2, d, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    sl = torch.tensor([T], dtype=torch.int32, device="cuda")
    by_token = pos.T.contiguous()
    for call in (lambda p: cuda_lib.rope(q, k, k, p, f, sections=sec),
                 lambda p: cuda_lib.rope_backward(q, k, k, p, f, sections=sec),
                 lambda p: cuda_lib.rope_append(q, k, k, p, f, kp, kp.clone(), table, sl, sections=sec)):
        with pytest.raises(ValueError):
            call(by_token)
        with pytest.raises(ValueError):
            call(by_token.view(2, 3, 3))
    assert torch.equal(cuda_lib.rope(q, k, k, pos[0].view(2, 3), f)[0], cuda_lib.rope(q, k, k, pos[:1], f)[0])
