"""What a bounded key-value cache needs beside attention: rotary positions with several axes
(training, and written straight into a paged cache when serving), the attention weight that
each cached key has collected, and the eviction of the keys that collected least.

`run` computes each operator in its plain form, or with the package's calls where `own` is set.

Layouts: bf16 queries [.., Hq, d], keys and values [.., Hkv, d]; page pools
[num_pages, page, Hkv, d] with an int32 block table [B, max_pages] and lengths [B];
collected weight ("mass") fp32 [B, Hkv, ld], row j of a sequence's cache at index j.
"""
import math

import numpy as np
import torch

own = False

BF = torch.bfloat16


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoding step of a small batch: eight new tokens rotated and put into the cache (latency)
        dict(name="append_step_b8", op="append", lens="step", B=8, T=8, rows=1024, Hq=32, Hkv=8, d=128, rot=128,
             axes=1, adjacent=False, page=128),
        # a packed prompt of nine ragged sequences (32K tokens) rotated and put into the cache
        dict(name="append_packed_32k", op="append", lens="ragged", B=9, T=32768, rows=16384, Hq=32, Hkv=8, d=128,
             rot=128, axes=3, adjacent=False, page=128),
        # training on 32K tokens of video: a fused projection's output split and rotated on three axes
        dict(name="rope_32k_3axes", op="rope", back=False, T=32768, Hq=32, Hkv=8, d=128, rot=128, axes=3,
             cyclic=True, adjacent=False),
        # the gradient of the same kind of split, 8K tokens, half of each head rotated, neighbouring pairs
        dict(name="rope_back_8k_partial", op="rope", back=True, T=8192, Hq=16, Hkv=16, d=128, rot=64, axes=2,
             cyclic=False, adjacent=True),
        # the weight that every key of a short prompt collected (a ragged length)
        dict(name="mass_1000_d64", op="mass", B=2, Hq=4, Hkv=2, Lq=1000, Lk=1000, d=64, window=0),
        # an 8K prompt with a head of keys for each head of queries
        dict(name="mass_8k_h16", op="mass", B=1, Hq=16, Hkv=16, Lq=8192, Lk=8192, d=128, window=0),
        # a 32K prompt, four query heads to a key head
        dict(name="mass_32k_gqa", op="mass", B=1, Hq=32, Hkv=8, Lq=32768, Lk=32768, d=128, window=0),
        # what the last 64 queries of a prompt chunk gave to a long cache
        dict(name="mass_window_64", op="mass", B=2, Hq=32, Hkv=8, Lq=2000, Lk=32000, d=128, window=64),
        # decoding one token for two short sequences, the weights collected on the way (latency)
        dict(name="decode_2k_b2", op="decode", B=2, Hq=8, Hkv=2, rows=2048, d=128, page=64),
        # decoding for eight sequences of up to 128K keys
        dict(name="decode_128k_b8", op="decode", B=8, Hq=32, Hkv=8, rows=131072, d=128, page=128),
        # a small cache cut down to a quarter
        dict(name="evict_1000_b2", op="evict", B=2, Hkv=2, rows=1024, d=64, page=64, budget=256, sinks=4, recent=64),
        # eight caches of up to 32K keys cut down to 4K each
        dict(name="evict_32k_b8", op="evict", B=8, Hkv=8, rows=32768, d=128, page=128, budget=4096, sinks=4,
             recent=512),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "mass", "decode", "evict"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 4, 8] if op == "decode" else [1, 2, 3, 4, 7, 8])
    page = rng.choice([64, 128])
    if op in ("rope", "append"):
        rot = rng.choice([r for r in (32, 64, 96, 128) if r <= d])
        axes = rng.choice([1, 2, 3])
        G = min(G, 32 // Hkv)
        if op == "rope":
            return dict(op=op, back=rng.random() < 0.5, T=_spread(rng, 1, 30000), Hq=Hkv * G, Hkv=Hkv, d=d, rot=rot,
                        axes=axes, cyclic=rng.random() < 0.5, adjacent=rng.random() < 0.5)
        lens = rng.choice(["step", "ragged"])
        B = _spread(rng, 1, 64)
        T = B if lens == "step" else _spread(rng, B, 20000)
        rows = min(T + page if lens == "ragged" else _spread(rng, 64, 2048), 262144 // B)
        return dict(op=op, lens=lens, B=B, T=T if lens == "step" else min(T, rows), rows=rows, Hq=Hkv * G, Hkv=Hkv,
                    d=d, rot=rot, axes=axes, adjacent=rng.random() < 0.5, page=page)
    if op == "mass":
        Lk = _spread(rng, 1, 16000)
        Lq = Lk if rng.random() < 0.5 else _spread(rng, 1, Lk)
        window = 0 if rng.random() < 0.5 else _spread(rng, 1, Lq)
        B = rng.choice([1, 2, 3]) if Lk < 6000 else 1
        return dict(op=op, B=B, Hq=Hkv * min(G, 32 // Hkv), Hkv=Hkv, Lq=Lq, Lk=Lk, d=d, window=window)
    if op == "decode":
        B = _spread(rng, 1, 16)
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, rows=_spread(rng, 1, 500000 // B), d=d, page=page)
    B = _spread(rng, 1, 16)
    rows = _spread(rng, 16, 260000 // B)
    budget = _spread(rng, 4, rows)
    sinks = rng.choice([0, 1, 4])
    return dict(op=op, B=B, Hkv=Hkv, rows=rows, d=d, page=page, budget=budget, sinks=sinks,
                recent=rng.randint(0, min(budget - sinks, 600)))


# ------------------------------------------------------------------ the inputs
def _lengths(case, gen):
    """One length for each sequence of a cache with room for `rows`: the first is full, the others
    lie anywhere from half of it up, on and off the borders of pages."""
    B, rows = case["B"], case["rows"]
    frac = torch.rand(B, generator=gen, device="cuda", dtype=torch.float64)
    lens = (rows * (0.5 + 0.5 * frac)).long().clamp(1, rows)
    lens[0] = rows
    return lens.to(torch.int32)


def _ragged(B, T, gen):
    """T tokens cut into B sequences of at least one token, at random places: offsets [B + 1]."""
    cuts = torch.randperm(T - 1, generator=gen, device="cuda")[:B - 1].sort().values + 1 if T > 1 else \
        torch.empty(0, dtype=torch.long, device="cuda")
    ends = torch.tensor([T], device="cuda")
    return torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), cuts, ends]).to(torch.int32)


def _pools(case, gen):
    """K and V pools with their pages in random order, and the block table of `rows` rows a sequence."""
    B, page = case["B"], case["page"]
    mp = -(-case["rows"] // page)
    shape = (B * mp, page, case["Hkv"], case["d"])
    k = torch.randn(shape, generator=gen, device="cuda", dtype=BF)
    v = torch.randn(shape, generator=gen, device="cuda", dtype=BF)
    table = torch.randperm(B * mp, generator=gen, device="cuda").to(torch.int32).view(B, mp)
    return k, v, table


def _sections(rot, axes):
    """Pairs for each axis: the first (time) gets what the others leave."""
    pairs = rot // 2
    per = (pairs // axes) // 2 * 2 if axes > 1 else 0
    return (pairs - per * (axes - 1),) + (per,) * (axes - 1)


def _positions(axes, T, gen):
    """Token positions: time runs on to tens of thousands, height and width are small."""
    t = torch.arange(T, device="cuda", dtype=torch.int32) + torch.randint(0, 100000, (1,), generator=gen,
                                                                          device="cuda", dtype=torch.int32)
    if axes == 1:
        return t.view(1, T)
    small = torch.randint(0, 80, (axes - 1, T), generator=gen, device="cuda", dtype=torch.int32)
    return torch.cat([t.view(1, T), small])


def _collected(case, gen):
    """Mass as a cache holds it after many steps: a few keys hold most of it."""
    B, Hkv = case["B"], case["Hkv"]
    ld = -(-case["rows"] // case["page"]) * case["page"]
    u = torch.rand(B, Hkv, ld, generator=gen, device="cuda")
    return (1.0 / (u + 1e-3) - 0.9).contiguous()


def _prompt(case, gen):
    """Queries and keys with local attention and sinks, and the log-normalisers that the attention
    call left behind."""
    B, Hq, Hkv, Lq, Lk, d = (case[x] for x in ("B", "Hq", "Hkv", "Lq", "Lk", "d"))
    G = Hq // Hkv
    coarse = torch.randn(B, -(-Lk // 32), Hkv, d, generator=gen, device="cuda")
    z = coarse.repeat_interleave(32, dim=1)[:, :Lk]
    u = torch.randn(d, generator=gen, device="cuda")
    u = u / u.norm()
    k = 0.8 * z + 0.6 * torch.randn(B, Lk, Hkv, d, generator=gen, device="cuda")
    k[:, :4] += 3.0 * u
    q = 0.8 * z[:, Lk - Lq:].repeat_interleave(G, dim=2) + 1.5 * u
    q += 0.6 * torch.randn(B, Lq, Hq, d, generator=gen, device="cuda")
    q, k = q.to(BF), k.to(BF)
    scale = d ** -0.5
    lse = torch.zeros(B, Hq, Lq, device="cuda")
    col = torch.arange(Lk, device="cuda")
    step = max(1, (1 << 28) // Lk)
    first = Lq - (case["window"] or Lq)
    for b in range(B):
        for h in range(Hq):
            for i in range(first, Lq, step):
                s = (q[b, i:i + step, h] @ k[b, :, h // G].T).float().mul_(scale)
                row = torch.arange(i, min(i + step, Lq), device="cuda") + (Lk - Lq)
                s.masked_fill_(col[None, :] > row[:, None], -math.inf)
                lse[b, h, i:i + step] = torch.logsumexp(s, dim=-1)
    return q, k, lse, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    if op in ("rope", "append"):
        T, Hq = case["T"], case["Hq"]
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) /
                                     case["rot"])).float()
        s["sections"] = _sections(case["rot"], case["axes"])
        s["positions"] = _positions(case["axes"], T, gen)
        if op == "rope" and case["back"]:
            for x, h in (("dq", Hq), ("dk", Hkv), ("dv", Hkv)):
                s[x] = torch.randn(T, h, d, generator=gen, device="cuda", dtype=BF)
        else:
            s["qkv"] = torch.randn(T, (Hq + 2 * Hkv) * d, generator=gen, device="cuda", dtype=BF)
        if op == "append":
            s["k_pages"], s["v_pages"], s["table"] = _pools(case, gen)
            if case["lens"] == "step":
                s["cu"], s["lens"] = None, _lengths(case, gen)
            else:
                s["cu"] = _ragged(case["B"], T, gen)
                new = s["cu"][1:] - s["cu"][:-1]
                old = torch.randint(0, 65, (case["B"],), generator=gen, device="cuda", dtype=torch.int32)
                s["lens"] = torch.minimum(new + old, torch.full_like(new, case["rows"]))
    elif op == "mass":
        s["q"], s["k"], s["lse"], s["scale"] = _prompt(case, gen)
        s["mass"] = torch.rand(case["B"], Hkv, case["Lk"], generator=gen, device="cuda")
    elif op == "decode":
        s["k_pages"], s["v_pages"], s["table"] = _pools(case, gen)
        s["lens"] = _lengths(case, gen)
        s["q"] = 2.0 * torch.randn(case["B"], case["Hq"], d, generator=gen, device="cuda")
        s["q"] = s["q"].to(BF)
        s["mass"] = _collected(case, gen)
        s["scale"] = d ** -0.5
    else:
        s["k_pages"], s["v_pages"], s["table"] = _pools(case, gen)
        s["lens"] = _lengths(case, gen)
        s["mass"] = _collected(case, gen)
        mp = -(-case["budget"] // case["page"])
        shape = (case["B"] * mp, case["page"], Hkv, d)
        s["k_out"] = torch.zeros(shape, device="cuda", dtype=BF)
        s["v_out"] = torch.zeros(shape, device="cuda", dtype=BF)
        s["out_table"] = torch.randperm(case["B"] * mp, generator=gen, device="cuda").to(torch.int32).view(-1, mp)
    return s


def _split(s):
    """q, k and v as views of the fused projection's output."""
    Hq, Hkv, d = s["Hq"], s["Hkv"], s["d"]
    qkv = s["qkv"].view(-1, Hq + 2 * Hkv, d)
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]


# ------------------------------------------------------------------ plain forms
def _axis_of_pair(sections, cyclic):
    n = len(sections)
    i = torch.arange(sum(sections), device="cuda")
    if cyclic:  # pair i belongs to axis i mod n while that axis has pairs left, else to the first
        a = i % n
        return torch.where(i < n * torch.tensor(sections, device="cuda")[a], a, torch.zeros_like(a))
    return torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(sections, device="cuda"))


def _angles(s, dtype):
    axis = _axis_of_pair(s["sections"], s.get("cyclic", False))
    ang = s["positions"][axis].T.double() * s["inv_freq"].double()  # [T, pairs]
    return torch.cos(ang).to(dtype), torch.sin(ang).to(dtype)


def _rotated(x, cos, sin, rot, adjacent):
    """x [T, H, d] with its first `rot` values of each head turned pair by pair."""
    x = x.float()
    c, n = cos[:, None, :], sin[:, None, :]
    if adjacent:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * c - b * n, b * c + a * n], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1).to(BF)


def _rope_plain(s):
    cos, sin = _angles(s, torch.float32)
    if s["back"]:  # the transposed rotation, laid out as the fused projection's gradient
        dq, dk = (_rotated(s[x], cos, -sin, s["rot"], s["adjacent"]) for x in ("dq", "dk"))
        return torch.cat([dq, dk, s["dv"]], dim=1).flatten(1)
    q, k, v = _split(s)
    return (_rotated(q, cos, sin, s["rot"], s["adjacent"]), _rotated(k, cos, sin, s["rot"], s["adjacent"]),
            v.contiguous())


def _append_plain(s):
    q, k, v = _split(s)
    cos, sin = _angles(s, torch.float32)
    T, page = s["T"], s["page"]
    token = torch.arange(T, device="cuda")
    if s["cu"] is None:
        seq, row = token, s["lens"].long() - 1
    else:
        cu = s["cu"].long()
        seq = torch.searchsorted(cu[1:], token, right=True)
        row = s["lens"].long()[seq] - cu[seq + 1] + token
    at = s["table"].long()[seq, row // page]
    s["k_pages"][at, row % page] = _rotated(k, cos, sin, s["rot"], s["adjacent"])
    s["v_pages"][at, row % page] = v
    return _rotated(q, cos, sin, s["rot"], s["adjacent"]), s["k_pages"], s["v_pages"]


DECAY = 0.9


def _mass_plain(s):
    B, Hq, Hkv, Lq, Lk = (s[x] for x in ("B", "Hq", "Hkv", "Lq", "Lk"))
    G, first = Hq // Hkv, Lq - (s["window"] or Lq)
    out = DECAY * s["mass"]
    out[..., Lk - Lq:] = 0  # the keys of the call's own tokens start from nothing
    row = torch.arange(first, Lq, device="cuda") + (Lk - Lq)
    late = torch.arange(Lk, device="cuda")[None, :] > row[:, None]
    for b in range(B):  # one head's [Lq, Lk] weights at a time: all of them do not fit
        for h in range(Hq):
            w = s["q"][b, first:, h].float() @ s["k"][b, :, h // G].float().T
            w = w.mul_(s["scale"]).sub_(s["lse"][b, h, first:, None]).exp_().masked_fill_(late, 0.0)
            out[b, h // G] += w.sum(0)
    return out


def _decode_plain(s):
    B, Hq, Hkv, d, page = (s[x] for x in ("B", "Hq", "Hkv", "d", "page"))
    o = torch.empty(B, Hq, d, device="cuda")
    lse = torch.empty(B, Hq, device="cuda")
    out = torch.zeros_like(s["mass"])
    lens = s["lens"].tolist()
    for b in range(B):  # sequences of different lengths
        n = lens[b]
        pages = s["table"][b].long()
        k = s["k_pages"][pages].flatten(0, 1)[:n].float()  # [n, Hkv, d]
        v = s["v_pages"][pages].flatten(0, 1)[:n].float()
        q = s["q"][b].float().view(Hkv, Hq // Hkv, d)
        sc = torch.matmul(q, k.permute(1, 2, 0)) * s["scale"]  # [Hkv, G, n]
        top = sc.amax(-1, keepdim=True)
        e = torch.exp(sc - top)
        z = e.sum(-1, keepdim=True)
        lse[b] = (top + torch.log(z)).view(Hq)
        p = e / z
        o[b] = torch.matmul(p, v.permute(1, 0, 2)).view(Hq, d)
        out[b, :, :n - 1] = DECAY * s["mass"][b, :, :n - 1]  # the newest key is the query's own
        out[b, :, :n] += p.sum(1)
    kept = (s["lens"] + page - 1) // page  # every tile is kept
    return o.to(BF), lse, kept.repeat_interleave(Hq), out


def _evict_plain(s):
    B, Hkv, page, budget = (s[x] for x in ("B", "Hkv", "page", "budget"))
    ld = s["mass"].shape[-1]
    lens = s["lens"].long()
    row = torch.arange(ld, device="cuda")
    there = (row[None] < lens[:, None])[:, None]  # [B, 1, ld]
    forced = ((row[None] < s["sinks"]) | (row[None] >= lens[:, None] - s["recent"]))[:, None] & there
    # by rank (forced, then present, then the rest) and inside a rank by mass; equal ones in the order of rows
    order = s["mass"].sort(dim=-1, descending=True, stable=True).indices
    rank = (forced.int() + there.int()).expand_as(s["mass"]).gather(-1, order)
    order = order.gather(-1, rank.sort(dim=-1, descending=True, stable=True).indices)
    new = torch.minimum(lens, torch.full_like(lens, budget))
    slot = torch.arange(budget, device="cuda")
    live = (slot[None] < new[:, None])[:, None].expand(B, Hkv, budget)
    order = order[..., :budget]
    if order.shape[-1] < budget:
        order = torch.nn.functional.pad(order, (0, budget - order.shape[-1]))
    kept = torch.where(live, order, ld).sort(dim=-1).values  # ascending rows, the empty slots last
    index = torch.where(live, kept, -1)
    b, h, r = live.nonzero(as_tuple=True)
    src = index[b, h, r]
    mass = torch.zeros(B, Hkv, budget, device="cuda")
    mass[b, h, r] = s["mass"][b, h, src]
    frm, to = s["table"].long()[b, src // page], s["out_table"].long()[b, r // page]
    for x, y in (("k_pages", "k_out"), ("v_pages", "v_out")):
        s[y][to, r % page, h] = s[x][frm, src % page, h]
    return index.to(torch.int32), new.to(torch.int32), mass, s["k_out"], s["v_out"]


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    if not own:
        return {"rope": _rope_plain, "append": _append_plain, "mass": _mass_plain, "decode": _decode_plain,
                "evict": _evict_plain}[s["op"]](s)
    import mass_gated_causal_b200 as mala
    if s["op"] == "rope":
        how = dict(sections=s["sections"], cyclic=s["cyclic"], adjacent=s["adjacent"])
        if s["back"]:
            Hq, Hkv, d = s["Hq"], s["Hkv"], s["d"]
            grad = torch.empty(s["T"], Hq + 2 * Hkv, d, device="cuda", dtype=BF)
            mala.rope_backward(s["dq"], s["dk"], s["dv"], s["positions"], s["inv_freq"], **how,
                               out=(grad[:, :Hq], grad[:, Hq:Hq + Hkv], grad[:, Hq + Hkv:]))
            return grad.flatten(1)
        q, k, v = _split(s)
        return mala.rope(q, k, v, s["positions"], s["inv_freq"], **how)
    if s["op"] == "append":
        q, k, v = _split(s)
        q = mala.rope_append(q, k, v, s["positions"], s["inv_freq"], s["k_pages"], s["v_pages"], s["table"],
                             s["lens"], cu_seqlens=s["cu"], sections=s["sections"], adjacent=s["adjacent"])
        return q, s["k_pages"], s["v_pages"]
    if s["op"] == "mass":
        return mala.key_mass(s["q"], s["k"], s["lse"], s["scale"], window=s["window"], mass=s["mass"], decay=DECAY)
    if s["op"] == "decode":
        o, lse, kept, _, _, mass = mala.decode_paged_mass(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                                          s["scale"], 0.0, mass=s["mass"], decay=DECAY)
        return o, lse, kept, mass
    index, new, mass = mala.evict(s["mass"], s["lens"], s["budget"], s["k_pages"], s["v_pages"], s["table"],
                                  s["out_table"], n_sink=s["sinks"], n_recent=s["recent"], k_out=s["k_out"],
                                  v_out=s["v_out"])
    return index, new, mass, s["k_out"], s["v_out"]


# ------------------------------------------------------------------ the work
def work(case):
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    if op in ("rope", "append"):
        rows = case["T"] * (case["Hq"] + 2 * Hkv)  # heads read once and written once
        turned = case["T"] * (case["Hq"] + Hkv) * case["rot"] // 2
        return {"bytes": 2 * rows * d * 2 + 4 * case["axes"] * case["T"], "flops": 6 * turned}
    if op == "mass":
        B, Hq, Lq, Lk = (case[x] for x in ("B", "Hq", "Lq", "Lk"))
        w = case["window"] or Lq
        pairs = w * (Lk - w) + w * (w + 1) // 2  # (query, key) pairs that a query sees
        return {"bytes": B * (2 * d * (w * Hq + Lk * Hkv) + 4 * w * Hq + 4 * Hkv * (2 * Lk - Lq)),
                "flops": B * Hq * pairs * (2 * d + 3)}
    if op == "decode":
        keys = case["B"] * case["rows"] * 0.75 * Hkv  # lengths lie between half of the room and all of it
        G = case["Hq"] // Hkv
        return {"bytes": keys * (4 * d + 8) + case["B"] * case["Hq"] * (4 * d + 4), "flops": keys * G * (4 * d + 3)}
    kept = case["B"] * min(case["budget"], case["rows"]) * Hkv
    return {"bytes": 4 * case["B"] * Hkv * case["rows"] * 0.75 + kept * (8 * d + 8), "flops": 0}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The operators from their definitions, in 64 bits."""
    s = prepare(case, seed)
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    f8 = torch.float64
    if op in ("rope", "append"):
        rot, n = case["rot"], case["rot"] // 2
        owner = torch.zeros(n, dtype=torch.long)
        sec = s["sections"]
        if s.get("cyclic", False):
            for a in range(1, len(sec)):
                owner[a:len(sec) * sec[a]:len(sec)] = a
        else:
            for a in range(len(sec)):
                owner[sum(sec[:a]):sum(sec[:a + 1])] = a
        theta = torch.stack([s["positions"][int(owner[i])].to(f8) * s["inv_freq"][i].to(f8) for i in range(n)], 1)
        back = case.get("back", False)
        turn = torch.polar(torch.ones_like(theta), -theta if back else theta)[:, None, :]  # e^(i theta)

        def turned(x):
            x = x.to(f8)
            if case["adjacent"]:
                z = torch.view_as_complex(x[..., :rot].unflatten(-1, (n, 2)).contiguous()) * turn
                y = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(x[..., :n], x[..., n:rot]) * turn
                y = torch.cat([z.real, z.imag], -1)
            return torch.cat([y, x[..., rot:]], -1)

        if back:
            return torch.cat([turned(s["dq"]), turned(s["dk"]), s["dv"].to(f8)], 1).flatten(1)
        q, k, v = _split(s)
        if op == "rope":
            return turned(q), turned(k), v.to(f8)
        kp, vp, tk = s["k_pages"].to(f8), s["v_pages"].to(f8), turned(k)
        ends = list(range(1, case["B"] + 1)) if s["cu"] is None else s["cu"].tolist()[1:]
        begin = 0
        for b, end in enumerate(ends):
            rows = torch.arange(int(s["lens"][b]) - (end - begin), int(s["lens"][b]), device="cuda")
            flat = s["table"][b].long()[rows // case["page"]] * case["page"] + rows % case["page"]
            kp.view(-1, Hkv, d)[flat] = tk[begin:end]
            vp.view(-1, Hkv, d)[flat] = v[begin:end].to(f8)
            begin = end
        return turned(q), kp, vp
    if op == "mass":
        B, Hq, Lq, Lk = (case[x] for x in ("B", "Hq", "Lq", "Lk"))
        old = Lk - Lq
        out = torch.zeros(B, Hkv, Lk, device="cuda", dtype=f8)
        out[..., :old] = DECAY * s["mass"][..., :old].to(f8)
        step = 4096
        for b in range(B):
            for h in range(Hq):
                key = s["k"][b, :, h * Hkv // Hq].to(f8)
                for i in range(Lq - (case["window"] or Lq), Lq, step):
                    e = min(i + step, Lq)
                    t = s["q"][b, i:e, h].to(f8) @ key[:old + e].T * s["scale"] - s["lse"][b, h, i:e].to(f8)[:, None]
                    out[b, h * Hkv // Hq, :old + e] += torch.exp(t).tril(old + i).sum(0)
        return out
    if op == "decode":
        B, Hq, page = case["B"], case["Hq"], case["page"]
        o = torch.zeros(B, Hq, d, device="cuda", dtype=f8)
        lse = torch.zeros(B, Hq, device="cuda", dtype=f8)
        out = torch.zeros_like(s["mass"], dtype=f8)
        for b in range(B):
            n = int(s["lens"][b])
            flat = (s["table"][b].long()[:, None] * page + torch.arange(page, device="cuda")).flatten()[:n]
            for h in range(Hq):
                g = h * Hkv // Hq
                t = s["k_pages"].view(-1, Hkv, d)[flat, g].to(f8) @ s["q"][b, h].to(f8) * s["scale"]
                lse[b, h] = torch.logsumexp(t, 0)
                w = torch.softmax(t, 0)
                o[b, h] = w @ s["v_pages"].view(-1, Hkv, d)[flat, g].to(f8)
                out[b, g, :n] += w
            out[b, :, :n - 1] += DECAY * s["mass"][b, :, :n - 1].to(f8)
        return o, lse, ((s["lens"] + page - 1) // page).repeat_interleave(Hq), out
    B, page, budget = case["B"], case["page"], case["budget"]
    lens, mass_in = s["lens"].tolist(), s["mass"].double().cpu().numpy()
    index = torch.full((B, Hkv, budget), -1, dtype=torch.int32)
    mass = torch.zeros(B, Hkv, budget, device="cuda", dtype=f8)
    pools = [s[x].to(f8) for x in ("k_out", "v_out")]
    for b in range(B):
        n = lens[b]
        new = min(n, budget)
        lo, hi = min(case["sinks"], n), max(min(case["sinks"], n), n - case["recent"])
        ends = np.concatenate([np.arange(lo), np.arange(hi, n)])
        to = s["out_table"][b].long()[torch.arange(new, device="cuda") // page] * page
        to = to + torch.arange(new, device="cuda") % page
        for h in range(Hkv):
            middle = np.arange(lo, hi)
            heavy = middle[np.lexsort((middle, -mass_in[b, h, lo:hi]))][:new - len(ends)]
            rows = torch.from_numpy(np.sort(np.concatenate([ends, heavy])))
            index[b, h, :new] = rows.int()
            rows = rows.cuda()
            mass[b, h, :new] = s["mass"][b, h, rows].to(f8)
            frm = s["table"][b].long()[rows // page] * page + rows % page
            for pool, x in zip(pools, ("k_pages", "v_pages")):
                pool.view(-1, Hkv, d)[to, h] = s[x].view(-1, Hkv, d)[frm, h].to(f8)
    return index.cuda(), torch.tensor([min(n, budget) for n in lens], dtype=torch.int32).cuda(), mass, *pools
