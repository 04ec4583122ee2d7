"""Key mass on the GPU (mala_key_mass, mala_key_mass_varlen) against column sums
of the softmax matrix in 64 bits, from the same q, k and LSE.

Tolerance, relative, per key (every term is positive, so a bound on each term's
relative error bounds the sum's): the score is an fp32 sum of d products, off by
at most 2 d 2^-24 scale sum_c |q_c k_c| (the 2 for an accumulator that drops bits
instead of rounding them), x = s log2e - LSE log2e rounds at its terms' size
(3 x 2^-24 (|s| + |LSE|) log2e), exp2 is good to 2^-21, and the sums (64 terms
in fp32 before the compensated sum, its 8 partials) to 16 x 2^-24. Weights below
2^-126 count as 2^-126.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634


def inputs(B, Hq, Hkv, Lq, Lk, d, seed, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32)
    u = r(d)
    k = r(B, Lk, Hkv, d) * spread
    k[:, :3] += 2.0 * u / u.norm()
    q = r(B, Lq, Hq, d) + 1.5 * u / u.norm()
    return q.to(torch.bfloat16), k.to(torch.bfloat16)


def weights(q, k, scale):
    """fp64 scores [Hq, Lq, Lk] of one sequence, -inf where a row does not see a key, and
    sum_c |q_c k_c|'s maximum."""
    Lq, Hq, _ = q.shape
    Lk, Hkv, _ = k.shape
    kk = k.double().repeat_interleave(Hq // Hkv, dim=1).permute(1, 2, 0)
    s = torch.matmul(q.double().permute(1, 0, 2), kk) * scale
    late = torch.arange(Lk, device="cuda")[None] > torch.arange(Lq, device="cuda")[:, None] + (Lk - Lq)
    a = torch.matmul(q.double().abs().permute(1, 0, 2), kk.abs()).amax() if Lq and Lk else torch.zeros(())
    return s.masked_fill(late, float("-inf")), float(a)


def reference(q, k, lse, scale, window, mass, decay, ld):
    """One sequence in 64 bits -> (mass [Hkv, ld], relative bound)."""
    Lq, Hq, d = q.shape
    Lk, Hkv, _ = k.shape
    out = torch.zeros(Hkv, ld, device="cuda", dtype=torch.float64)
    if mass is not None and decay:
        out[:, :Lk - Lq] = decay * mass[:, :Lk - Lq].double()
    if Lq == 0:
        return out, 0.0
    s, a = weights(q, k, scale)
    first = Lq - window if 0 < window < Lq else 0
    w = torch.exp(s[:, first:] - lse[:, first:].double()[..., None]).sum(1)  # [Hq, Lk]
    out[:, :Lk] += w.view(Hkv, Hq // Hkv, Lk).sum(1)
    top = float(s[s > float("-inf")].abs().max())
    fin = lse[torch.isfinite(lse)].abs()
    rel = 2 * d * 2.0 ** -24 * scale * a + 3 * 2.0 ** -24 * LOG2E * (top + float(fin.max()) if fin.numel() else top) + \
        2.0 ** -21 + 16 * 2.0 ** -24
    return out, rel


def close(got, want, rel, terms):
    err = (got.double() - want).abs()
    assert bool((err <= rel * want + terms * 2.0 ** -126).all()), float((err / want.clamp_min(1e-30)).max())


def lse_of(q, k, scale):
    return torch.stack([torch.logsumexp(weights(q[b], k[b], scale)[0], -1).float() for b in range(q.shape[0])])


CASES = [
    # B, Hq, Hkv, Lq, Lk, d, window
    (1, 1, 1, 1, 1, 64, 0),
    (1, 8, 1, 1, 5, 128, 0),
    (2, 4, 2, 64, 64, 128, 0),        # few rows: the keys stream past them
    (2, 6, 2, 37, 500, 64, 0),
    (1, 7, 1, 50, 131, 128, 0),
    (3, 16, 2, 300, 1000, 128, 64),   # 512 columns: two blocks of them
    (1, 4, 4, 257, 700, 64, 256),
    (1, 2, 1, 500, 513, 128, 1),
    (1, 4, 1, 128, 4000, 64, 100),
    (1, 8, 8, 300, 300, 128, 0),      # walks over the query tiles
    (2, 4, 2, 1000, 1000, 64, 0),
    (1, 6, 3, 700, 1500, 128, 513),
    (1, 3, 1, 1500, 1501, 128, 0),
    (1, 16, 2, 900, 2900, 64, 0),
    (1, 32, 8, 2049, 2049, 128, 0),
    (4, 32, 16, 1100, 1100, 128, 0),
]


@pytest.mark.parametrize("B,Hq,Hkv,Lq,Lk,d,window", CASES)
def test_key_mass(cuda_lib, B, Hq, Hkv, Lq, Lk, d, window):
    q, k = inputs(B, Hq, Hkv, Lq, Lk, d, seed=Lq + Lk)
    scale = d ** -0.5
    lse = lse_of(q, k, scale)
    ld = Lk + 70
    mass = torch.rand(B, Hkv, ld, device="cuda") * 50
    got = cuda_lib.key_mass(q, k, lse, scale, window=window, mass=mass, decay=0.75)
    alone = cuda_lib.key_mass(q, k, lse, scale, window=window)
    assert cuda_lib.mala_check_status() == 0
    assert got.shape == (B, Hkv, ld) and alone.shape == (B, Hkv, Lk)
    terms = Hq // Hkv * Lq
    for b in range(B):
        want, rel = reference(q[b], k[b], lse[b], scale, window, mass[b], 0.75, ld)
        close(got[b], want, rel, terms)
        want, rel = reference(q[b], k[b], lse[b], scale, window, None, 1.0, Lk)
        close(alone[b], want, rel, terms)
    rows = window if 0 < window < Lq else Lq
    total = alone.double().sum()  # every row's weights sum to 1
    assert abs(float(total) - B * Hq * rows) <= 1e-4 * B * Hq * rows


def test_in_place_decay_zero_and_repeatable(cuda_lib):
    for shape in ((1, 8, 2, 600, 900, 128, 0), (1, 8, 2, 60, 900, 64, 0)):
        B, Hq, Hkv, Lq, Lk, d, window = shape
        q, k = inputs(B, Hq, Hkv, Lq, Lk, d, seed=2)
        lse = lse_of(q, k, 0.1)
        mass = torch.rand(B, Hkv, Lk, device="cuda")
        a = cuda_lib.key_mass(q, k, lse, 0.1, mass=mass, decay=0.5)
        b = cuda_lib.key_mass(q, k, lse, 0.1, mass=mass, decay=0.5)
        assert torch.equal(a, b)  # the same bits every time
        nan = torch.full_like(mass, float("nan"))
        c = cuda_lib.key_mass(q, k, lse, 0.1, mass=nan, decay=0.0)  # not read
        assert torch.equal(c, cuda_lib.key_mass(q, k, lse, 0.1))
        own = mass.clone()
        own[..., Lk - Lq:] = float("nan")  # the queries' own tokens start from 0
        assert torch.equal(cuda_lib.key_mass(q, k, lse, 0.1, mass=own, decay=0.5, out=own), a)


@pytest.mark.parametrize("Lq,Lk", [(500, 800), (40, 800)])
def test_rows_that_add_nothing(cuda_lib, Lq, Lk):
    """A row whose LSE is +infinity; keys no row sees; a mask is a selection, not a product."""
    q, k = inputs(1, 4, 2, Lq, Lk, 64, seed=8)
    lse = lse_of(q, k, 0.125)
    lse[0, 1, ::3] = float("inf")
    got = cuda_lib.key_mass(q, k, lse, 0.125)
    want, rel = reference(q[0], k[0], lse[0], 0.125, 0, None, 1.0, Lk)
    close(got[0], want, rel, 2 * Lq)


PACKED = [
    # lens_q, lens_k, Hq, Hkv, d, window
    ([5, 1, 64], [5, 1, 64], 4, 2, 64, 0),
    ([300, 0, 129, 1], [300, 40, 700, 1], 8, 2, 128, 0),
    ([300, 0, 129, 1], [300, 40, 700, 1], 8, 2, 128, 32),
    ([1200, 457, 700], [1200, 457, 1111], 4, 4, 128, 0),
    ([64, 64, 64], [2000, 900, 64], 16, 4, 128, 64),
    ([900, 33], [900, 2000], 6, 1, 64, 0),
]


@pytest.mark.parametrize("lens_q,lens_k,Hq,Hkv,d,window", PACKED)
def test_key_mass_varlen(cuda_lib, lens_q, lens_k, Hq, Hkv, d, window):
    """Sequences end to end, and NaN in the rows behind the last one: no sequence sees another's rows."""
    scale = d ** -0.5
    S, tq, tk = len(lens_q), sum(lens_q) + 9, sum(lens_k) + 11
    q, k = (x[0] for x in inputs(1, Hq, Hkv, tq, tk, d, seed=sum(lens_q)))
    cq = torch.tensor([0] + lens_q, device="cuda").cumsum(0).to(torch.int32)
    ck = torch.tensor([0] + lens_k, device="cuda").cumsum(0).to(torch.int32)
    q[int(cq[-1]):] = float("nan")
    k[int(ck[-1]):] = float("nan")
    lse = torch.full((Hq, tq), float("nan"), device="cuda")
    for s in range(S):
        a, b = slice(int(cq[s]), int(cq[s + 1])), slice(int(ck[s]), int(ck[s + 1]))
        if lens_q[s]:
            lse[:, a] = torch.logsumexp(weights(q[a], k[b], scale)[0], -1).float()
    ld = max(lens_k) + 5
    mass = torch.rand(S, Hkv, ld, device="cuda")
    got = cuda_lib.key_mass_varlen(q, k, lse, cq, ck, max(lens_q), max(lens_k), scale, window=window, mass=mass,
                                   decay=2.0)
    loose = cuda_lib.key_mass_varlen(q, k, lse, cq, ck, tq, tk, scale, window=window, mass=None,
                                     out=torch.empty(S, Hkv, tk, device="cuda"))
    assert cuda_lib.mala_check_status() == 0
    for s in range(S):
        a, b = slice(int(cq[s]), int(cq[s + 1])), slice(int(ck[s]), int(ck[s + 1]))
        want, rel = reference(q[a], k[b], lse[:, a], scale, window, mass[s], 2.0, ld)
        close(got[s], want, rel, Hq // Hkv * max(1, lens_q[s]))
        want, rel = reference(q[a], k[b], lse[:, a], scale, window, None, 1.0, tk)
        close(loose[s], want, rel, Hq // Hkv * max(1, lens_q[s]))


@pytest.mark.parametrize("window", [0, 16])
def test_varlen_reports_bad_tables(cuda_lib, window):
    q, k = (x[0] for x in inputs(1, 4, 2, 600, 600, 64, seed=1))
    lse = torch.zeros(4, 600, device="cuda")
    ok = [0, 250, 600]
    for bad in ([0, 250, 601], [0, -1, 600], [0, 601, 600]):
        out = torch.full((2, 2, 600), 3.0, device="cuda")
        cq = torch.tensor(bad, dtype=torch.int32, device="cuda")
        ck = torch.tensor(ok, dtype=torch.int32, device="cuda")
        cuda_lib.key_mass_varlen(q, k, lse, cq, ck, 600, 600, 0.1, window=window, out=out)
        assert cuda_lib.mala_check_status() == cuda_lib.MALA_ERR_INVALID_ARG
        bad_seqs = [s for s in range(2) if not (0 <= bad[s] <= bad[s + 1] <= 600 and bad[s + 1] - bad[s] <= ok[s + 1] - ok[s])]
        assert bad_seqs
        for s in bad_seqs:
            assert bool((out[s] == 3.0).all())
    assert cuda_lib.mala_check_status() == 0


@pytest.mark.parametrize("Lq,item,reached", [
    (600, 1, True), (600, 0, True), (40, 0, True),
    (40, 1, False),  # eight key tiles, one to a CTA: no walk has an item 1, and nothing stalls
])
def test_a_wait_that_runs_out_is_reported(cuda_lib, Lq, item, reached):
    q, k = inputs(1, 4, 2, Lq, 900, 64, seed=1)
    lse = lse_of(q, k, 0.1)
    want = cuda_lib.key_mass(q, k, lse, 0.1)
    cuda_lib.mala_test_hooks(20_000_000, item, None)
    try:
        cuda_lib.key_mass(q, k, lse, 0.1)
        assert cuda_lib.mala_check_status() == (cuda_lib.MALA_ERR_DEVICE_TIMEOUT if reached else 0)
    finally:
        cuda_lib.mala_test_hooks(0, -1, None)
    assert torch.equal(cuda_lib.key_mass(q, k, lse, 0.1), want)
    assert cuda_lib.mala_check_status() == 0


def test_graph_and_stream(cuda_lib):
    q, k = inputs(1, 8, 2, 700, 700, 128, seed=4)
    lse = lse_of(q, k, 0.09)
    want = cuda_lib.key_mass(q, k, lse, 0.09)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = cuda_lib.key_mass(q, k, lse, 0.09, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b = cuda_lib.key_mass(q, k, lse, 0.09)
    g.replay()
    assert torch.equal(a, want) and torch.equal(b, want)


def test_of_the_forward_with_a_gate(cuda_lib):
    """From mala_forward's own LSE at tau = 1: the skipped tiles' keys count with their weights too."""
    q, k = inputs(1, 4, 2, 1000, 1000, 128, seed=6)
    v = torch.randn_like(k)
    scale = 128 ** -0.5
    for tau in (0.0, 1.0):
        _, lse, _, _ = cuda_lib.forward(q, k, v, scale, tau)
        got = cuda_lib.key_mass(q, k, lse, scale)
        assert cuda_lib.mala_check_status() == 0
        want, rel = reference(q[0], k[0], lse[0], scale, 0, None, 1.0, 1000)
        close(got[0], want, rel, 2000)


def test_binding_checks(cuda_lib):
    q, k = inputs(1, 4, 2, 20, 30, 64, seed=6)
    lse = torch.zeros(1, 4, 20, device="cuda")
    m = torch.zeros(1, 2, 30, device="cuda")
    for kw in (dict(q=q.float()), dict(k=k[:, :, :1].contiguous().half()), dict(lse=lse[:, :2].contiguous()), dict(mass=m.double()),
               dict(mass=m[:, :1].contiguous()), dict(out=m[..., ::2]), dict(k=k.transpose(1, 2)),
               dict(mass=m, out=torch.zeros(1, 2, 40, device="cuda"))):
        a = dict(q=q, k=k, lse=lse, scale=0.1)
        a.update(kw)
        with pytest.raises(ValueError):
            cuda_lib.key_mass(**a)
    with pytest.raises(cuda_lib.MalaError):
        cuda_lib.key_mass(q, k, lse, 0.1, out=torch.zeros(1, 2, 29, device="cuda"))


@pytest.mark.parametrize("Lq,tile,reached", [(100, 0, True), (100, 1, True), (60, 1, True), (100, 2000, False)])
def test_teams_that_wait_in_vain_end(cuda_lib, Lq, tile, reached):
    """Few rows, the keys streaming past them: two blocks of columns (416) and one (256), a team of warps each."""
    q, k = inputs(1, 4, 1, Lq, 9000, 64, seed=1)
    lse = lse_of(q, k, 0.1)
    want = cuda_lib.key_mass(q, k, lse, 0.1, mass=torch.ones(1, 1, 9000, device="cuda"), decay=0.5)
    cuda_lib.mala_test_hooks(20_000_000, tile, None)
    try:
        cuda_lib.key_mass(q, k, lse, 0.1)
        # 71 key tiles go to a CTA each; of eight heads, several to a CTA
        q2, k2 = (x.repeat(1, 1, 8, 1) for x in (q, k))
        cuda_lib.key_mass(q2, k2, lse.repeat(1, 8, 1), 0.1)
        assert cuda_lib.mala_check_status() == (cuda_lib.MALA_ERR_DEVICE_TIMEOUT if reached else 0)
    finally:
        cuda_lib.mala_test_hooks(0, -1, None)
    got = cuda_lib.key_mass(q, k, lse, 0.1, mass=torch.ones(1, 1, 9000, device="cuda"), decay=0.5)
    assert cuda_lib.mala_check_status() == 0 and torch.equal(got, want)
    many = cuda_lib.key_mass(q2, k2, lse.repeat(1, 8, 1), 0.1)
    for h in range(8):
        torch.testing.assert_close(many[:, h], cuda_lib.key_mass(q, k, lse, 0.1)[:, 0], rtol=2.0 ** -20, atol=0)
