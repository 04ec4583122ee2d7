"""Rotary positions on the GPU (mala_rope, mala_rope_append) against a 64-bit
rotation, the gradient against the formula's and against differences, and the
cache rows that an append writes and leaves.

Tolerance, per value: the kernel rounds once to bf16 (half a step, 2^-8 of the
value), after fp32 arithmetic on y1 = x1 c - x2 s: the angle as a fraction of a
turn is rounded to fp32 (2^-25 of a half turn, 1e-7 rad), sincospif is good to
2 ulp, and a product and an FMA round: together below 1e-6 (|x1| + |x2|).
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def axis_of_pair(sections, cyclic):
    if not cyclic:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    n = len(sections)
    return [i % n if i < n * sections[i % n] else 0 for i in range(sum(sections))]


def reference(x, positions, inv_freq, sections, adjacent, cyclic, sign=1.0):
    """x [T, H, d] fp64 -> (rotated, |x1| + |x2| per value)."""
    ax = axis_of_pair(sections, cyclic)
    th = sign * torch.stack([positions[a].double() * inv_freq[i].double() for i, a in enumerate(ax)], -1)[:, None]
    n = len(ax)
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if adjacent else (x[..., :n], x[..., n:2 * n])
    ya, yb = a * th.cos() - b * th.sin(), b * th.cos() + a * th.sin()
    y, size = x.clone(), x.abs()
    if adjacent:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = ya, yb
        size[..., 0:2 * n:2] = size[..., 1:2 * n:2] = a.abs() + b.abs()
    else:
        y[..., :n], y[..., n:2 * n] = ya, yb
        size[..., :n] = size[..., n:2 * n] = a.abs() + b.abs()
    return y, size


def close(got, want, size):
    err = (got.double() - want).abs()
    assert bool((err <= want.abs() * 2.0 ** -8 + 1e-6 * size + 1e-37).all()), float(err.max())


def inputs(T, Hq, Hkv, d, rot, axes, seed, far=100000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g, device="cuda", dtype=torch.bfloat16)
    pos = torch.randint(-50, far, (axes, T), generator=g, device="cuda", dtype=torch.int32)
    f = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)).float()
    n = rot // 2
    per = n // axes // 2 * 2 if axes > 1 else 0
    return qkv, pos, f, (n - per * (axes - 1),) + (per,) * (axes - 1)


CASES = [
    # T, Hq, Hkv, d, rotary, axes, adjacent, cyclic
    (1, 8, 2, 128, 128, 1, False, False),
    (1, 1, 1, 64, 16, 1, True, False),
    (7, 32, 8, 128, 128, 3, False, False),
    (7, 32, 8, 128, 128, 3, False, True),
    (333, 12, 4, 64, 64, 2, True, True),
    (1000, 5, 5, 128, 96, 4, False, True),
    (1000, 28, 4, 128, 64, 3, True, False),
    (5000, 3, 1, 64, 48, 2, False, False),
    (9001, 16, 16, 128, 112, 1, True, False),
]


@pytest.mark.parametrize("T,Hq,Hkv,d,rot,axes,adjacent,cyclic", CASES)
def test_rope_splits_and_rotates(cuda_lib, T, Hq, Hkv, d, rot, axes, adjacent, cyclic):
    qkv, pos, f, sec = inputs(T, Hq, Hkv, d, rot, axes, seed=T + d)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    before = qkv.clone()
    qo, ko, vo = cuda_lib.rope(q, k, v, pos, f, sections=sec, adjacent=adjacent, cyclic=cyclic)
    assert qo.is_contiguous() and ko.is_contiguous() and torch.equal(vo, v) and torch.equal(qkv, before)
    for got, x in ((qo, q), (ko, k)):
        close(got, *reference(x.double(), pos, f, sec, adjacent, cyclic))


@pytest.mark.parametrize("T,Hq,Hkv,d,rot,axes,adjacent,cyclic", CASES)
def test_rope_backward_is_the_transpose(cuda_lib, T, Hq, Hkv, d, rot, axes, adjacent, cyclic):
    """Into the views of a fused gradient; and <y, R x> = <R^T y, x> in 64 bits for the reference used."""
    qkv, pos, f, sec = inputs(T, Hq, Hkv, d, rot, axes, seed=2 * T + d)
    dq, dk, dv = (qkv[:, a:b].contiguous() for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    grad = torch.full((T, Hq + 2 * Hkv + 1, d), 7.0, device="cuda", dtype=torch.bfloat16)
    cuda_lib.rope_backward(dq, dk, dv, pos, f, sections=sec, adjacent=adjacent, cyclic=cyclic,
                           out=(grad[:, :Hq], grad[:, Hq:Hq + Hkv], grad[:, Hq + Hkv:-1]))
    for got, x in ((grad[:, :Hq], dq), (grad[:, Hq:Hq + Hkv], dk)):
        close(got, *reference(x.double(), pos, f, sec, adjacent, cyclic, sign=-1.0))
    assert torch.equal(grad[:, Hq + Hkv:-1], dv)
    assert bool((grad[:, -1] == 7.0).all())  # what lies between the rows is left alone
    x, y = torch.randn_like(dq, dtype=torch.float64), torch.randn_like(dq, dtype=torch.float64)
    lhs = (y * reference(x, pos, f, sec, adjacent, cyclic)[0]).sum()
    rhs = (reference(y, pos, f, sec, adjacent, cyclic, sign=-1.0)[0] * x).sum()
    assert abs(float(lhs - rhs)) <= 1e-9 * float(lhs.abs() + x.norm() * y.norm())


def test_rope_backward_matches_differences(cuda_lib):
    """d/dx of sum(w . rope(x)) by differences of the rotation itself: the rotation is linear, so a
    difference over a step of 1 is exact up to the roundings (each output 2^-8 of its value, twice)."""
    qkv, pos, f, sec = inputs(3, 2, 1, 64, 32, 2, seed=5)
    q = qkv[:, :2].contiguous()
    w = torch.randn(3, 2, 64, device="cuda", dtype=torch.bfloat16)
    grad = cuda_lib.rope_backward(w, None, None, pos, f, sections=sec)[0].double()
    base = cuda_lib.rope(q, None, None, pos, f, sections=sec)[0].double()
    for t, h, c in ((0, 0, 0), (1, 1, 17), (2, 0, 15), (2, 1, 40)):
        x = q.clone()
        x[t, h, c] += 1.0
        step = float(x[t, h, c].double() - q[t, h, c].double())  # bf16 may not hold exactly 1 more
        moved = cuda_lib.rope(x, None, None, pos, f, sections=sec)[0].double()
        diff = float(((moved - base) * w.double()).sum()) / step
        tol = float((w.double().abs() * (moved.abs() + base.abs()))[t, h].sum()) * 2.0 ** -8 / abs(step) + \
            abs(float(grad[t, h, c])) * 2.0 ** -8 + 1e-5
        assert abs(diff - float(grad[t, h, c])) <= tol


def test_rope_layouts(cuda_lib):
    """Heads before tokens, batches, one tensor alone, in place, and a stream of its own."""
    qkv, pos, f, sec = inputs(60, 4, 2, 128, 128, 3, seed=9)
    q, k = qkv[:, :4], qkv[:, 4:6]
    want = cuda_lib.rope(q, k, None, pos, f, sections=sec)
    hq = q.transpose(0, 1).contiguous().transpose(0, 1)  # [T, H, d] stored as [H, T, d]
    out = torch.empty(4, 60, 128, device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    cuda_lib.rope(hq, None, None, pos, f, sections=sec, out=(out, None, None))
    assert torch.equal(out, want[0])
    batched = cuda_lib.rope(q.reshape(3, 20, 4, 128), k.reshape(3, 20, 2, 128), None, pos, f, sections=sec)
    assert torch.equal(batched[0].view(60, 4, 128), want[0]) and torch.equal(batched[1].view(60, 2, 128), want[1])
    x = qkv.clone()
    cuda_lib.rope(x[:, :4], x[:, 4:6], x[:, 6:], pos, f, sections=sec, out=(x[:, :4], x[:, 4:6], x[:, 6:]))
    assert torch.equal(x[:, :4], want[0]) and torch.equal(x[:, 4:6], want[1]) and torch.equal(x[:, 6:], qkv[:, 6:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = cuda_lib.rope(q, k, None, pos, f, sections=sec, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(on_side[0], want[0])
    by_handle = cuda_lib.rope(q, k, None, pos, f, sections=sec, stream=0)  # the legacy default stream
    torch.cuda.synchronize()
    assert torch.equal(by_handle[0], want[0])
    empty = cuda_lib.rope(q[:0], k[:0], None, pos[:, :0].contiguous(), f, sections=sec)
    assert empty[0].shape == (0, 4, 128)


def test_rope_far_positions(cuda_lib):
    """Positions whose fp32 angle would be off by radians."""
    qkv, _, f, _ = inputs(64, 2, 1, 128, 128, 1, seed=3)
    pos = (torch.arange(64, device="cuda", dtype=torch.int32) * 33554393 - (1 << 30)).view(1, 64)
    q = qkv[:, :2].contiguous()
    close(cuda_lib.rope(q, None, None, pos, f)[0], *reference(q.double(), pos, f, (64,), False, False))


def test_rope_gradient_path_captured_beside_an_eager_one(cuda_lib):
    """The rotation and its gradient captured into one graph, replayed on new inputs."""
    qkv, pos, f, sec = inputs(40, 4, 2, 64, 64, 2, seed=11)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    eager = cuda_lib.rope(q, k, v, pos, f, sections=sec)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = cuda_lib.rope(q, k, v, pos, f, sections=sec)
        x = cuda_lib.rope_backward(*y, pos, f, sections=sec)
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(y, eager))
    qkv.mul_(-2.0)
    g.replay()
    assert all(torch.equal(a, b * -2) for a, b in zip(y, eager))
    back = cuda_lib.rope_backward(*y, pos, f, sections=sec)
    assert all(torch.equal(a, b) for a, b in zip(x, back))


# ------------------------------------------------------------------ into a paged cache
def paged(B, rows, Hkv, d, page, seed, fill=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mp = -(-rows // page)
    shape = (B * mp + 3, page, Hkv, d)
    k = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    table = torch.randperm(B * mp + 3, generator=g, device="cuda")[:B * mp].to(torch.int32).view(B, mp)
    return k, v, table


def expect_append(k_pages, v_pages, table, lens, news, k, v):
    """The pools after the append of the rotated k and v, sequence by sequence."""
    kp, vp, page = k_pages.clone(), v_pages.clone(), k_pages.shape[1]
    t = 0
    for b, (n, L) in enumerate(zip(news, lens)):
        for i in range(n):
            if L >= n:
                row = L - n + i
                pg = int(table[b, row // page])
                kp[pg, row % page], vp[pg, row % page] = k[t], v[t]
            t += 1
    return kp, vp


@pytest.mark.parametrize("news,lens,Hq,Hkv,d,page,rot,adjacent", [
    ([1, 1, 1, 1], [1, 64, 65, 300], 8, 2, 128, 64, 128, False),   # a decoding step, on and off page borders
    ([1], [128], 1, 1, 64, 128, 32, True),
    ([130, 0, 1, 64, 200], [130, 50, 70, 64, 383], 12, 4, 64, 64, 64, False),  # ragged, one without tokens
    ([3, 500], [3, 900], 32, 8, 128, 128, 64, True),
])
def test_rope_append(cuda_lib, news, lens, Hq, Hkv, d, page, rot, adjacent):
    T, B = sum(news), len(news)
    qkv, pos, f, sec = inputs(T, Hq, Hkv, d, rot, 3, seed=T + B)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    kp, vp, table = paged(B, max(lens), Hkv, d, page, seed=T)
    want_q, want_k, _ = cuda_lib.rope(q, k, None, pos, f, sections=sec, adjacent=adjacent)
    want = expect_append(kp, vp, table, lens, news, want_k, v)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = None if set(news) == {1} else torch.tensor(np.cumsum([0] + news), dtype=torch.int32, device="cuda")
    got_q = cuda_lib.rope_append(q, k, v, pos, f, kp, vp, table, sl, cu_seqlens=cu, sections=sec, adjacent=adjacent)
    assert cuda_lib.mala_check_status() == 0
    assert torch.equal(got_q, want_q)  # the same rotation as mala_rope, which is held to 64 bits above
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


def test_rope_append_padding_and_idle_slots(cuda_lib):
    """Tokens behind the last sequence and slots of length 0 are left alone, queries included."""
    qkv, pos, f, sec = inputs(10, 4, 2, 64, 64, 1, seed=21)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    kp, vp, table = paged(3, 100, 2, 64, 64, seed=4)
    lens, news = [40, 0, 30], [3, 2, 2]
    want_q, want_k, _ = cuda_lib.rope(q, k, None, pos, f, sections=sec)
    want = expect_append(kp, vp, table, [40, -1, 30], news, want_k, v)
    out = torch.full((10, 4, 64), 5.0, device="cuda", dtype=torch.bfloat16)
    cu = torch.tensor([0, 3, 5, 7], dtype=torch.int32, device="cuda")
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cuda_lib.rope_append(q, k, v, pos, f, kp, vp, table, sl, cu_seqlens=cu, sections=sec, out=out)
    assert cuda_lib.mala_check_status() == 0
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    live = [0, 1, 2, 5, 6]
    assert torch.equal(out[live], want_q[live])
    assert bool((out[[3, 4, 7, 8, 9]] == 5.0).all())


def test_rope_append_reports_bad_tables(cuda_lib):
    """A length shorter than the new tokens, one past the table, a page outside the pool: reported, and nothing
    but the queries is written for that token."""
    qkv, pos, f, sec = inputs(3, 4, 2, 64, 64, 1, seed=22)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    kp, vp, table = paged(3, 128, 2, 64, 64, seed=6)
    want_q, want_k, _ = cuda_lib.rope(q, k, None, pos, f, sections=sec)
    good = [50, 60, 70]
    for b, value, where in ((1, -3, "lens"), (1, 129, "lens"), (1, kp.shape[0], "table"), (1, -1, "table")):
        lens, tb = list(good), table.clone()
        if where == "lens":
            lens[b] = value
        else:
            tb[b, lens[b] // 64] = tb[b, 0] = value
        kc, vc = kp.clone(), vp.clone()
        want = expect_append(kc, vc, table, [x if i != b else -1 for i, x in enumerate(good)], [1, 1, 1], want_k, v)
        sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        got = cuda_lib.rope_append(q, k, v, pos, f, kc, vc, tb, sl, sections=sec)
        assert cuda_lib.mala_check_status() == cuda_lib.MALA_ERR_INVALID_ARG
        assert torch.equal(got, want_q) and torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    assert cuda_lib.mala_check_status() == 0


def test_binding_checks(cuda_lib):
    qkv, pos, f, sec = inputs(8, 4, 2, 64, 64, 1, seed=30)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    bad = [
        (q.float(), k, v, pos, f), (q, k[:4], v, pos, f), (q, k, v[:, :1], pos, f), (q, k, v, pos.long(), f),
        (q, k, v, pos[:, :4].contiguous(), f), (q, k, v, pos, f.double()), (q, k, v, pos.cpu(), f),
        (q.transpose(1, 2), k, v, pos, f),
    ]
    for args in bad:
        with pytest.raises(ValueError):
            cuda_lib.rope(*args)
    with pytest.raises(cuda_lib.MalaError):
        cuda_lib.rope(q, k, v, pos, f, sections=(16,))
    with pytest.raises(ValueError):
        cuda_lib.rope(q, k, v, pos, f, out=(q, k, None))
    kp, vp, table = paged(8, 64, 2, 64, 64, seed=6)
    sl = torch.ones(8, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        cuda_lib.rope_append(q, k, v, pos, f, kp, vp[:2], table, sl)
    with pytest.raises(ValueError):
        cuda_lib.rope_append(q, k, v, pos, f, kp, vp, table[:4], sl)
    with pytest.raises(ValueError):
        cuda_lib.rope_append(q, k, v, pos, f, kp.transpose(1, 2), vp, table, sl)
