"""The operators beside attention on a machine without a GPU: every refusal that
the host makes (no call here reaches CUDA), workspace sizes, and the binding's
checks of its tensors."""
import pytest
import torch

import mass_gated_causal_b200 as mala

P = 256  # a fake, 256-byte aligned "device pointer": never dereferenced by the rejected calls
S = 0


def rope(**kw):
    a = dict(q=P, k=P, v=P, q_out=P, k_out=P, v_out=P, strides=[1536, 128, 1536, 128, 1536, 128, 1024, 128, 256, 128,
                                                               256, 128],
             positions=P, inv_freq=P, T=10, Hq=8, Hkv=2, d=128, rotary_dim=128, sections=[32, 16, 16], n_axes=3,
             flags=0, stream=S)
    a.update(kw)
    return mala.mala_rope(**a)


def strides(i, value):
    s = [1536, 128, 1536, 128, 1536, 128, 1024, 128, 256, 128, 256, 128]
    s[i] = value
    return s


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(k_out=None), 1), (dict(q=None, k=None, v=None, q_out=None, k_out=None, v_out=None), 1),
    (dict(positions=None), 1), (dict(inv_freq=None), 1), (dict(strides=None), 1), (dict(sections=None), 1),
    (dict(T=-1), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(flags=8), 1),
    (dict(n_axes=0, sections=[]), 1), (dict(n_axes=5, sections=[16, 16, 16, 8, 8]), 1),
    (dict(sections=[32, 16, 15]), 1), (dict(sections=[80, -8, -8]), 1), (dict(sections=[32, 16, 24]), 1),
    (dict(sections=[16, 32, 16], flags=2), 1),  # more pairs than the turns of an axis
    (dict(strides=strides(6, 120)), 1), (dict(strides=strides(7, 64)), 1), (dict(strides=strides(6, 1016)), 1),
    (dict(strides=strides(7, 1024)), 1), (dict(strides=strides(11, 1 << 62)), 2), (dict(strides=strides(6, 128)), 1), (dict(strides=strides(0, -1536)), 1),
    (dict(d=96), 2), (dict(d=256), 2), (dict(rotary_dim=120), 2), (dict(rotary_dim=0), 2), (dict(rotary_dim=144), 2),
    (dict(q=P + 8), 2), (dict(v_out=P + 2), 2), (dict(strides=strides(1, 132)), 2), (dict(strides=strides(8, 260)), 2),
])
def test_rope_rejects(kw, code):
    assert rope(**kw) == code


def test_rope_of_no_tokens_does_nothing():
    assert rope(T=0, positions=None, q=None, q_out=None) == 0


def append(**kw):
    a = dict(q=P, k=P, v=P, q_out=P, strides=[1536, 128, 1536, 128, 1536, 128, 1024, 128], positions=P, inv_freq=P,
             k_pages=P, v_pages=P, block_table=P, seqlens_k=P, cu_seqlens=P, num_seqs=3, T=10, Hq=8, Hkv=2,
             num_pages=50, page_size=128, max_pages_per_seq=8, d=128, rotary_dim=64, sections=[32], n_axes=1, flags=0,
             stream=S)
    a.update(kw)
    return mala.mala_rope_append(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(q=None), 1), (dict(q_out=None), 1), (dict(k_pages=None), 1),
    (dict(block_table=None), 1), (dict(seqlens_k=None), 1), (dict(positions=None), 1), (dict(strides=None), 1),
    (dict(num_seqs=0), 1), (dict(num_pages=0), 1), (dict(max_pages_per_seq=0), 1), (dict(T=-1), 1),
    (dict(cu_seqlens=None), 1),  # 10 tokens, 3 sequences
    (dict(flags=4), 1), (dict(sections=[31]), 1),
    (dict(page_size=32), 2), (dict(page_size=96), 2), (dict(d=80), 2), (dict(rotary_dim=40), 2),
    (dict(max_pages_per_seq=1 << 24), 2), (dict(num_pages=1 << 25), 2), (dict(k_pages=P + 8), 2), (dict(k=P + 4), 2),
    (dict(strides=[1536, 128, 1540, 128, 1536, 128, 1024, 128]), 2),
])
def test_rope_append_rejects(kw, code):
    assert append(**kw) == code


def mass(**kw):
    a = dict(q=P, k=P, lse=P, mass_in=P, mass_out=P, B=1, Hq=8, Hkv=2, Lq=1000, Lk=2000, d=128, scale=0.1, window=0,
             decay=1.0, ld_mass=2000, workspace=P, workspace_bytes=1 << 40, stream=S)
    a.update(kw)
    return mala.mala_key_mass(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(lse=None), 1), (dict(mass_out=None), 1), (dict(B=0), 1),
    (dict(Lq=0), 1), (dict(Lk=999), 1), (dict(Hq=7), 1), (dict(scale=0.0), 1), (dict(scale=float("inf")), 1),
    (dict(window=-1), 1), (dict(decay=-0.5), 1), (dict(decay=float("nan")), 1), (dict(ld_mass=1999), 1),
    (dict(d=32), 2), (dict(lse=P + 4), 2), (dict(mass_out=P + 8), 2), (dict(mass_in=P + 4), 2), (dict(Hkv=1 << 16,
                                                                                                   Hq=1 << 16), 2),
    (dict(workspace=None), 3), (dict(workspace_bytes=100), 3), (dict(workspace=P + 16), 3),
])
def test_key_mass_rejects(kw, code):
    assert mala.mala_key_mass_workspace_size(1, 8, 2, 1000, 2000, 0) > 100  # the workspace refusals below are real
    assert mass(**kw) == code


def vmass(**kw):
    a = dict(q=P, k=P, lse=P, cu_seqlens_q=P, cu_seqlens_k=P, mass_in=P, mass_out=P, num_seqs=3, max_seqlen_q=600,
             max_seqlen_k=900, total_q=1000, total_k=2000, Hq=8, Hkv=2, d=64, scale=0.1, window=0, decay=1.0,
             ld_mass=900, workspace=P, workspace_bytes=1 << 40, stream=S)
    a.update(kw)
    return mala.mala_key_mass_varlen(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(cu_seqlens_q=None), 1), (dict(cu_seqlens_k=None), 1), (dict(num_seqs=0), 1), (dict(total_q=0), 1),
    (dict(max_seqlen_q=1001), 1), (dict(max_seqlen_k=2001), 1), (dict(max_seqlen_q=0), 1), (dict(ld_mass=899), 1),
    (dict(Hq=9), 1), (dict(d=96), 2), (dict(q=P + 8), 2), (dict(workspace=None), 3),
])
def test_key_mass_varlen_rejects(kw, code):
    assert vmass(**kw) == code


def test_key_mass_workspace_sizes():
    ws = mala.mala_key_mass_workspace_size
    assert ws(0, 8, 2, 100, 100, 0) == 0 and ws(1, 8, 3, 100, 100, 0) == 0 and ws(1, 8, 2, 200, 100, 0) == 0
    assert ws(1, 32, 8, 32768, 32768, 0) == 0  # the key tiles fill the GPU: whole walks
    assert ws(2, 32, 8, 2000, 32000, 64) == 0  # few query rows: the keys stream past them
    one = ws(1, 8, 2, 1000, 2000, 0)
    assert one > 0 and one % 256 == 0
    # partials of whole key blocks (128 or 256 keys) for every (b, KV head)
    assert one % (2 * 2048 * 4) == 0
    # a packed batch: room for every sequence's longest walk
    assert mala.mala_key_mass_varlen_workspace_size(3, 8, 2, 1000, 2000, 1000, 0) % (3 * 2 * 2048 * 4) == 0


def decode(**kw):
    a = dict(q=P, k_pages=P, v_pages=P, block_table=P, seqlens_k=P, o=P, lse=P, mass_in=P, mass_out=P, B=4, Hq=8,
             Hkv=2, num_pages=100, page_size=128, max_pages_per_seq=40, d=128, scale=0.1, tau=1.0, decay=1.0,
             ld_mass=40 * 128, n_splits=4, workspace=P, workspace_bytes=1 << 40, kept_tiles=P, keep_map=None, stream=S)
    a.update(kw)
    return mala.mala_decode_paged_mass(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(mass_out=None), 1), (dict(block_table=None), 1), (dict(seqlens_k=None), 1),
    (dict(kept_tiles=None), 1), (dict(num_pages=0), 1), (dict(Hq=6, Hkv=4), 1), (dict(n_splits=-1), 1),
    (dict(tau=-1.0), 1), (dict(decay=-1.0), 1), (dict(decay=float("inf")), 1), (dict(ld_mass=40 * 128 - 1), 1),
    (dict(page_size=256), 2), (dict(d=96), 2), (dict(Hq=64, Hkv=2), 2), (dict(max_pages_per_seq=1 << 24), 2),
    (dict(k_pages=P + 8), 2), (dict(mass_out=P + 4), 2), (dict(n_splits=70000, ld_mass=1 << 20), 2),
    (dict(ld_mass=(1 << 30) + 1), 2), (dict(ld_mass=(1 << 31) - 1), 2),
    (dict(workspace=None), 3), (dict(workspace_bytes=1000), 3), (dict(workspace=P + 64), 3),
])
def test_decode_paged_mass_rejects(kw, code):
    assert decode(**kw) == code


def test_decode_mass_workspace_size():
    a256 = lambda x: (x + 255) // 256 * 256
    ws = mala.mala_decode_mass_workspace_size
    scores, plan = a256(4 * 8 * 40 * 128 * 4), a256(5 * 4)
    # behind a gate: a partial for each split
    assert ws(4, 8, 2, 128, 128, 40, 5) == scores + mala.mala_decode_workspace_size(4, 8, 128, 5) + plan
    # without: 80 tiles in runs of at least two, and one run more that begins before them
    assert ws(4, 8, 2, 128, 128, 40, 0) == scores + mala.mala_decode_workspace_size(4, 8, 128, 41) + plan
    for bad in ((4, 8, 2, 96, 128, 40, 5), (4, 8, 2, 128, 100, 40, 5), (4, 8, 2, 128, 128, 40, -1), (4, 8, 0, 128, 128, 40, 5)):
        assert ws(*bad) == 0


def select(**kw):
    a = dict(mass=P, seqlens_k=2 * P, index=P, new_seqlens=P, mass_out=3 * P, B=2, Hkv=2, ld_mass=1000, budget=200,
             n_sink=4, n_recent=50, ld_mass_out=200, stream=S)
    a.update(kw)
    return mala.mala_evict_select(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(mass=None), 1), (dict(seqlens_k=None), 1), (dict(index=None), 1), (dict(new_seqlens=None), 1),
    (dict(B=0), 1), (dict(Hkv=0), 1), (dict(ld_mass=0), 1), (dict(budget=0), 1), (dict(n_sink=-1), 1),
    (dict(n_recent=-1), 1), (dict(n_sink=151), 1), (dict(ld_mass_out=199), 1), (dict(mass_out=P), 1),
    (dict(new_seqlens=2 * P), 1),  # the old lengths' array
    (dict(n_sink=(1 << 31) - 1, n_recent=(1 << 31) - 1), 1),
    (dict(mass=P + 8), 2), (dict(index=P + 4), 2), (dict(ld_mass=(1 << 30) + 1), 2),
    (dict(budget=(1 << 30) + 1, mass_out=None), 2), (dict(ld_mass_out=(1 << 30) + 1), 2),
])
def test_evict_select_rejects(kw, code):
    assert select(**kw) == code


def gather(**kw):
    a = dict(k_pages=P, v_pages=P, block_table=P, index=P, new_seqlens=P, k_out_pages=P, v_out_pages=P, out_table=P,
             B=2, Hkv=2, budget=200, num_pages=40, num_out_pages=40, page_size=64, max_pages_per_seq=16,
             max_out_pages_per_seq=4, d=128, stream=S)
    a.update(kw)
    return mala.mala_evict_gather(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(k_pages=None), 1), (dict(v_out_pages=None), 1), (dict(out_table=None), 1), (dict(index=None), 1),
    (dict(B=0), 1), (dict(budget=0), 1), (dict(num_pages=0), 1), (dict(max_out_pages_per_seq=3), 1),
    (dict(page_size=48), 2), (dict(d=32), 2), (dict(k_pages=P + 8), 2), (dict(v_out_pages=P + 4), 2),
    (dict(B=70000), 2), (dict(num_out_pages=1 << 26), 2),
])
def test_evict_gather_rejects(kw, code):
    assert gather(**kw) == code


def test_binding_refuses_cpu_tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    pos, f, pool = i32(1, 4), torch.zeros(64), bf(8, 64, 2, 128)
    with pytest.raises(ValueError):
        mala.rope(bf(4, 8, 128), bf(4, 2, 128), bf(4, 2, 128), pos, f)
    with pytest.raises(ValueError):
        mala.rope(None, None, None, pos, f)
    with pytest.raises(ValueError):
        mala.rope_append(bf(4, 8, 128), bf(4, 2, 128), bf(4, 2, 128), pos, f, pool, pool.clone(), i32(4, 2), i32(4))
    with pytest.raises(ValueError):
        mala.key_mass(bf(1, 4, 8, 128), bf(1, 4, 2, 128), torch.zeros(1, 8, 4), 0.1)
    with pytest.raises(ValueError):
        mala.key_mass_varlen(bf(4, 8, 128), bf(4, 2, 128), torch.zeros(8, 4), i32(2), i32(2), 4, 4, 0.1)
    with pytest.raises(ValueError):
        mala.decode_paged_mass(bf(4, 8, 128), pool, pool, i32(4, 2), i32(4), 0.1, 0.0)
    with pytest.raises(ValueError):
        mala.evict_select(torch.zeros(1, 2, 100), i32(1), 10)
    with pytest.raises(ValueError):
        mala.evict_gather(i32(1, 2, 10), i32(1), pool, pool, i32(1, 2), i32(1, 1))


@pytest.mark.parametrize("make,want", [
    (lambda x: x.view(4, 6, 128), (4, 6, 128, 768, 128)),
    (lambda x: x.view(2, 2, 6, 128)[:, :, :4], (4, 4, 128, 768, 128)),
    (lambda x: x.view(4, 1, 6, 128)[:, :, 2:3], (4, 1, 128, 768, 0)),
    (lambda x: x.view(6, 4, 128).transpose(0, 1), (4, 6, 128, 128, 512)),
    (lambda x: x.view(1, 1, 24, 128), (1, 24, 128, 0, 128)),
])
def test_rows_of_a_strided_tensor(make, want):
    assert mala._load_native().rows(make(torch.zeros(4 * 6 * 128))) == want


def test_rows_refuses_tokens_at_two_strides():
    x = torch.zeros(4, 3, 6, 128)[:, :2]
    with pytest.raises(ValueError):
        mala._load_native().rows(x)
    with pytest.raises(ValueError):
        mala._load_native().rows(torch.zeros(4, 128, 6).transpose(1, 2))
