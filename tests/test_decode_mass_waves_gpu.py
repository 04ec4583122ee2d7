"""Short caches of as many heads as clusters of sixteen no longer hold at once (14 of a whole
B200's, two CTAs to an SM; 7 with one), on both sides of that. Bounds are those of
test_decode_mass_gpu.
"""
import os
import subprocess
import sys

import pytest

from test_decode_mass_gpu import test_decode_paged_mass as check_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,Hq,Hkv,d,page", [
    ([2000] * 13 + [1], 4, 1, 128, 64),        # fourteen
    ([2000, 1999, 65], 10, 5, 128, 128),       # fifteen
    ([4096, 100], 16, 8, 128, 64),             # sixteen
    ([8192, 4000], 8, 8, 128, 128),            # sixteen, too long for eight CTAs
    ([3000, 3000, 17, 129], 16, 4, 64, 64),    # sixteen, d = 64
    ([8000], 64, 8, 128, 64),                  # eight of one CTA to an SM
    ([1100] * 17, 6, 2, 128, 64),              # 34: four CTAs each
])
def test_one_wave(cuda_lib, lens, Hq, Hkv, d, page):
    check_case(cuda_lib, lens, Hq, Hkv, d, page, 0.0, 0)


SCRIPT = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import mass_gated_causal_b200 as mala
from test_rope_gpu import paged
kp, vp, table = paged(2, 2000, 8, 128, 64, seed=5)
q = torch.randn(2, 16, 128, device="cuda").to(torch.bfloat16)
sl = torch.tensor([2000, 777], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    c = mala.decode_paged_mass(q, kp, vp, table, sl, 0.09, 0.0)
g.replay()
want = mala.decode_paged_mass(q, kp, vp, table, sl, 0.09, 0.0)
torch.cuda.synchronize()
assert mala.mala_check_status() == 0
assert all(torch.equal(c[i], want[i]) for i in (0, 1, 5))
print("ok")
"""


def test_the_first_call_of_a_process_captured(cuda_lib):
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=os.path.dirname(here), tests=here)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
