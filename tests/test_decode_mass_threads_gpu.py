"""Decodes of short caches from several host threads at once, each with its own stream,
buffers and shape: the C calls hold no lock, and a launch must not depend on what
another thread sets up between."""
import threading

import pytest
import torch

from test_rope_gpu import paged

pytestmark = pytest.mark.gpu

N = 20000


def job(mala, lens, Hq, Hkv, d, seed):
    page = 64
    B = len(lens)
    kp, vp, table = paged(B, max(lens), Hkv, d, page, seed=seed)
    q = torch.randn(B, Hq, d, device="cuda").to(torch.bfloat16)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    mp = table.shape[1]
    size = mala.mala_decode_mass_workspace_size(B, Hq, Hkv, d, page, mp, 0)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    o = torch.zeros(B, Hq, d, dtype=torch.bfloat16, device="cuda")
    lse, kept = torch.zeros(B, Hq, device="cuda"), torch.zeros(B * Hq, dtype=torch.int32, device="cuda")
    mass = torch.zeros(B, Hkv, mp * page, device="cuda")
    stream = torch.cuda.Stream()

    def call():
        return mala.mala_decode_paged_mass(q, kp, vp, table, sl, o, lse, None, mass, B, Hq, Hkv, kp.shape[0], page, mp,
                                           d, d ** -0.5, 0.0, 1.0, mp * page, 0, ws, size, kept, None,
                                           stream.cuda_stream)
    return call, (q, kp, vp, table, sl), (o, lse, mass)


def test_threads_with_shapes_of_their_own(cuda_lib):
    # from one head and one tile to a CTA to groups of eight with eight tiles
    shapes = [([60], 1, 1), ([8000], 16, 2), ([700, 500], 4, 2), ([8192], 8, 1)]
    jobs = [job(cuda_lib, lens, Hq, Hkv, 128, i) for i, (lens, Hq, Hkv) in enumerate(shapes)]
    want = []
    for call, (q, kp, vp, table, sl), _ in jobs:
        r = cuda_lib.decode_paged_mass(q, kp, vp, table, sl, 128 ** -0.5, 0.0)
        want.append((r[0], r[1], r[5]))
    torch.cuda.synchronize()
    codes = [{} for _ in jobs]
    start = threading.Barrier(len(jobs))

    def work(i):
        torch.cuda.set_device(0)
        start.wait()
        for _ in range(N):
            rc = jobs[i][0]()
            codes[i][rc] = codes[i].get(rc, 0) + 1

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert cuda_lib.mala_check_status() == 0
    assert codes == [{0: N}] * len(jobs)
    for (_, _, got), w in zip(jobs, want):
        for x, y in zip(got, w):
            assert torch.equal(x, y)
