"""Cases for timing the serving operators of a chunk of new tokens over the
page-size-1 pool: the rows' preparation (per-head norm, rotation, append), the
chunk's attention, the attention mass its entries receive, and eviction by
that mass.

A case names its operator ("op") and sizes; lengths of a batch are drawn from
the case's own numbers, inputs from the seed.  ``run`` computes the plain form
in elementary torch operations, or, with ``own``, calls the library.
"""
import math
import random

import torch

own = False

D = 64
BASE = 10000.0
EPS = 1e-6
DEV = "cuda"


def listed():
    return [
        # one decode step of 14 agents: their 14 new rows (GQA 64/8)
        dict(name="append 14", op="append", n=14, Hq=64, Hkv=8, dtype="bf16", pad=0, fused=0),
        # a prefill chunk of many tool responses, q, k and v as column blocks of one projection
        dict(name="append 16384", op="append", n=16384, Hq=64, Hkv=8, dtype="bf16", pad=0, fused=1),
        # an odd batch padded to a captured size: one row in 16 is padding
        dict(name="append 4999 f32", op="append", n=4999, Hq=16, Hkv=4, dtype="f32", pad=16, fused=0),
        # single tokens of 14 agents over 20k-90k active entries each
        dict(name="chunk decode", op="chunk", B=14, q_lo=1, q_hi=1, kv_lo=20000, kv_hi=90000, Hq=64, Hkv=8,
             dtype="bf16", lengths=4),
        # short tool responses and single tokens in one batch, three KV heads
        dict(name="chunk mixed", op="chunk", B=9, q_lo=1, q_hi=700, kv_lo=701, kv_hi=12000, Hq=24, Hkv=3,
             dtype="bf16", lengths=2),
        # two agents' long pasted documents over their caches
        dict(name="chunk long", op="chunk", B=2, q_lo=4096, q_hi=4096, kv_lo=50000, kv_hi=70000, Hq=64, Hkv=8,
             dtype="bf16", lengths=3),
        # single precision, as the library's parity workloads use
        dict(name="chunk f32", op="chunk", B=3, q_lo=100, q_hi=301, kv_lo=500, kv_hi=4000, Hq=16, Hkv=4,
             dtype="f32", lengths=1),
        # the weight a decode step's tokens give to 20k-90k entries each
        dict(name="mass decode", op="mass", B=14, q_lo=1, q_hi=1, kv_lo=20000, kv_hi=90000, Hq=64, Hkv=8,
             dtype="bf16", lengths=4),
        # the weight that two tool responses give to their caches
        dict(name="mass chunk", op="mass", B=2, q_lo=1100, q_hi=1500, kv_lo=40000, kv_hi=56000, Hq=64, Hkv=8,
             dtype="bf16", lengths=5),
        dict(name="mass f32", op="mass", B=3, q_lo=1, q_hi=201, kv_lo=500, kv_hi=4000, Hq=16, Hkv=4,
             dtype="f32", lengths=6),
        # 14 agents' caches cut to half
        dict(name="evict 14", op="evict", B=14, kv_lo=20000, kv_hi=90000, keep=32768, lengths=4),
        # one cache of a million and a half entries cut to 256k
        dict(name="evict long", op="evict", B=1, kv_lo=1500000, kv_hi=1500000, keep=262144, lengths=7),
    ]


HEADS = [(64, 8), (16, 4), (8, 2), (24, 3), (32, 16), (2, 2)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "chunk", "chunk", "mass", "mass", "evict"])
    if op == "evict":
        B = _log(rng, 1, 14)
        hi = _log(rng, 16, 1500000 // B)
        return dict(op=op, B=B, kv_lo=rng.randint(0, hi), kv_hi=hi, keep=_log(rng, 1, hi),
                    lengths=rng.randrange(1 << 20))
    Hq, Hkv = rng.choice(HEADS)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "append":
        return dict(op=op, n=_log(rng, 1, 16384 if dtype == "bf16" else 8192), Hq=Hq, Hkv=Hkv,
                    dtype=dtype, pad=rng.choice([0, 0, 7, 16]), fused=rng.randint(0, 1))
    B = _log(rng, 1, 14)
    q = _log(rng, 1, 4096 if dtype == "bf16" else 512)
    kv = _log(rng, max(q, 16), 90000 if dtype == "bf16" else 8000)
    room = 2 * 1300 * 48000 * 64 if op == "mass" else 2 * 4096 * 60000 * 64
    if dtype == "f32":
        room //= 32
    while B > 1 and B * q * kv * Hq > room:
        B -= 1
    if B * q * kv * Hq > room:
        q = max(1, room // (B * kv * Hq))
    return dict(op=op, B=B, q_lo=rng.randint(1, q), q_hi=q, kv_lo=max(q, kv // 3), kv_hi=kv, Hq=Hq, Hkv=Hkv,
                dtype=dtype, lengths=rng.randrange(1 << 20))


def _lengths(case):
    """Chunk and cache lengths of the batch: the longest of each first."""
    rng = random.Random(case["lengths"])
    more = range(case["B"] - 1)
    kv = [case["kv_hi"]] + [rng.randint(case["kv_lo"], case["kv_hi"]) for _ in more]
    if case["op"] == "evict":
        return None, kv
    return [case["q_hi"]] + [rng.randint(case["q_lo"], case["q_hi"]) for _ in more], kv


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _csr(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case=case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    if case["op"] == "append":
        n, Hq, Hkv, t = case["n"], case["Hq"], case["Hkv"], _type(case)
        if case["fused"]:  # column blocks of one [n, (Hq + 2 Hkv) D] projection
            x = randn(n, Hq + 2 * Hkv, D).to(t)
            s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            s["q"], s["k"], s["v"] = (randn(n, h, D).to(t) for h in (Hq, Hkv, Hkv))
        s["qw"], s["kw"] = 1 + 0.2 * randn(D), 1 + 0.2 * randn(D)
        S = n + max(64, n // 8)
        slot = torch.randperm(S, generator=g, device=DEV)[:n].to(torch.int32)
        if case["pad"]:
            slot[torch.arange(n, device=DEV) % case["pad"] == case["pad"] - 1] = -1
        s["slot"] = slot
        s["pos"] = torch.randint(0, 131072, (n,), generator=g, device=DEV, dtype=torch.int32)
        s["k_pool"], s["v_pool"] = randn(S, Hkv, D).to(t), randn(S, Hkv, D).to(t)
        s["q_out"] = torch.zeros(n, Hq, D, dtype=t, device=DEV)
        return s

    qn, kv = _lengths(case)
    nnz, S = sum(kv), sum(kv) + max(64, sum(kv) // 10)
    s["kv"], s["kv_ptr"] = kv, _csr(kv)
    s["kv_indptr"] = _i32(s["kv_ptr"])
    s["kv_indices"] = torch.randperm(S, generator=g, device=DEV)[:nnz].to(torch.int32)
    if case["op"] == "evict":
        B, wide = case["B"], max(1, max(kv))
        # heavy tails, and one entry in eight that got nothing at all
        mass = torch.exp(2 * randn(B, wide))
        mass[torch.rand(B, wide, generator=g, device=DEV) < 0.125] = 0
        s["mass"] = mass
        s["kv_pos"] = torch.randint(0, 131072, (nnz,), generator=g, device=DEV, dtype=torch.int32)
        s["keep"] = _i32([case["keep"]] * B)
        kept = [min(n, case["keep"]) for n in kv]
        s["n_kept"], s["n_dropped"] = sum(kept), nnz - sum(kept)
        s["out_indptr"], s["dropped_indptr"] = (torch.zeros(B + 1, dtype=torch.int32, device=DEV)
                                                for _ in range(2))
        s["out_indices"], s["out_pos"] = (torch.zeros(s["n_kept"], dtype=torch.int32, device=DEV)
                                          for _ in range(2))
        s["out_mass"] = torch.zeros(B, wide, device=DEV)
        s["dropped"] = torch.zeros(s["n_dropped"], dtype=torch.int32, device=DEV)
        return s

    t, Hq, Hkv = _type(case), case["Hq"], case["Hkv"]
    s["qn"], s["q_ptr"] = qn, _csr(qn)
    s["q_indptr"] = _i32(s["q_ptr"])
    # normalised rows (scores of standard deviation 2), keys of uneven length
    s["q"] = (2 * randn(sum(qn), Hq, D)).to(t)
    s["k_pool"] = (randn(S, Hkv, D) * torch.exp(0.3 * randn(S, 1, 1))).to(t)
    if case["op"] == "chunk":
        s["v_pool"] = randn(S, Hkv, D).to(t)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(sum(qn), Hq, device=DEV)
    else:
        s["lse"] = _attend(s, None)[1]
        s["mass_in"] = torch.rand(case["B"], max(kv), generator=g, device=DEV)
        s["mass_out"] = torch.zeros(case["B"], max(kv), device=DEV)
    return s


def _norm_rope(x, w, pos):
    """Rows normalised per head and rotated at their positions, in 32 bits."""
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    th = BASE ** (-2.0 * torch.arange(D // 2, device=DEV, dtype=torch.float64) / D)
    a = pos.double()[:, None, None] * th
    c, sn = torch.cos(a).float(), torch.sin(a).float()
    y1, y2 = y[..., :D // 2], y[..., D // 2:]
    return torch.cat([y1 * c - y2 * sn, y1 * sn + y2 * c], -1)


def _append(s):
    ok = s["slot"] >= 0
    # a padding row's slot is the pool's last row plus one: a row that is cut off again
    S = s["k_pool"].shape[0]
    slot = torch.where(ok, s["slot"], S).long()
    q = _norm_rope(s["q"], s["qw"], s["pos"]).to(s["q"].dtype)
    k = _norm_rope(s["k"], s["kw"], s["pos"]).to(s["k"].dtype)
    q_out = torch.where(ok[:, None, None], q, s["q_out"])
    if s["case"]["pad"]:
        k_pool, v_pool = (torch.cat([p, p[:1]]) for p in (s["k_pool"], s["v_pool"]))
        k_pool[slot], v_pool[slot] = k, s["v"]
        return q_out, k_pool[:S], v_pool[:S]
    s["k_pool"][slot], s["v_pool"][slot] = k, s["v"]
    return q_out, s["k_pool"], s["v_pool"]


def _blocks(s):
    """(request, its first list entry, rows [i0, i1) of its chunk) in blocks
    whose scores take about 2 GB at most."""
    Hq = s["case"]["Hq"]
    for b, (m, n) in enumerate(zip(s["qn"], s["kv"])):
        step = max(1, (1 << 29) // max(1, Hq * n))
        for i0 in range(0, m, step):
            yield b, m, n, i0, min(m, i0 + step)


def _scores(s, K, b, m, n, i0, i1):
    """[Hkv, G, rows, n] scores of rows i0..i1-1 of request b, -inf where hidden."""
    Hkv, G = s["case"]["Hkv"], s["case"]["Hq"] // s["case"]["Hkv"]
    q = s["q"][s["q_ptr"][b] + i0:s["q_ptr"][b] + i1].float().view(-1, Hkv, G, D).permute(1, 2, 0, 3)
    x = (q.reshape(Hkv, -1, D) @ K.transpose(1, 2)).view(Hkv, G, i1 - i0, n) * 0.125
    if i0 + 1 < m or n < m:  # else every row sees the whole list
        seen = n - m + 1 + torch.arange(i0, i1, device=DEV)
        x = torch.where(torch.arange(n, device=DEV) < seen[:, None], x, -math.inf)
    return x


def _cached(s, pool, b):
    """[Hkv, n, D] in 32 bits: request b's listed rows."""
    return s[pool][s["kv_indices"][s["kv_ptr"][b]:s["kv_ptr"][b + 1]].long()].float().transpose(0, 1)


def _attend(s, v_pool):
    Hq = s["case"]["Hq"]
    out = torch.empty(s["q"].shape, device=DEV) if v_pool else None
    lse = torch.empty(s["q"].shape[0], Hq, device=DEV)
    at = None
    for b, m, n, i0, i1 in _blocks(s):
        if at != b:
            at, K = b, _cached(s, "k_pool", b)
            V = _cached(s, v_pool, b) if v_pool else None
        x = _scores(s, K, b, m, n, i0, i1)
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top)
        tot = p.sum(-1, keepdim=True)
        r = slice(s["q_ptr"][b] + i0, s["q_ptr"][b] + i1)
        lse[r] = (top + torch.log(tot)).permute(2, 0, 1, 3).reshape(i1 - i0, Hq)
        if v_pool:
            o = (p.flatten(1, 2) @ V).view(p.shape[:3] + (D,)) / tot
            out[r] = o.permute(2, 0, 1, 3).reshape(i1 - i0, Hq, D)
    return out, lse


DECAY = 0.875


def _mass(s):
    case = s["case"]
    Hkv, G = case["Hkv"], case["Hq"] // case["Hkv"]
    out = s["mass_out"].clone()
    at = None
    for b, m, n, i0, i1 in _blocks(s):
        if at != b:
            at, K = b, _cached(s, "k_pool", b)
            # entries older than the chunk carry their decayed mass; the chunk's own start at zero
            out[b, :n] = torch.where(torch.arange(n, device=DEV) < n - m, DECAY * s["mass_in"][b, :n], 0.0)
        x = _scores(s, K, b, m, n, i0, i1)
        r = slice(s["q_ptr"][b] + i0, s["q_ptr"][b] + i1)
        lse = s["lse"][r].view(i1 - i0, Hkv, G).permute(1, 2, 0)
        out[b, :n] += torch.exp(x - lse[..., None]).sum((0, 1, 2))
    return out


FIRST, RECENT = 4, 64


def _evict(s):
    n = s["kv_indptr"][1:] - s["kv_indptr"][:-1]
    j = torch.arange(s["mass"].shape[1], device=DEV)
    there = j < n[:, None]
    fixed = there & ((j < FIRST) | (j >= n[:, None] - RECENT))
    key = torch.where(fixed, math.inf, torch.where(torch.isnan(s["mass"]), -math.inf, s["mass"]))
    key = torch.where(there, key, -math.inf)
    order = torch.argsort(key, dim=1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(1, order, j.expand_as(order))
    kept = there & (rank < torch.minimum(n, s["keep"])[:, None])
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    outs = []
    for mask, size in ((kept, s["n_kept"]), (there & ~kept, s["n_dropped"])):
        count = mask.sum(1, dtype=torch.int32)
        ptr = torch.cat([zero, torch.cumsum(count, 0, dtype=torch.int32)])
        at = torch.where(mask, torch.cumsum(mask, 1) - 1, 0)
        # what is not in the list goes to one place behind it
        to = torch.where(mask, at + ptr[:-1, None], size)
        entry = (s["kv_indptr"][:-1, None] + j).clamp(max=s["kv_indices"].numel() - 1).long()
        row = torch.where(mask, at, s["mass"].shape[1])
        outs.append((ptr, to, entry, row, size))
    ptr, to, entry, row, size = outs[0]
    put = lambda to, x, size: torch.zeros(size + 1, dtype=x.dtype, device=DEV).scatter_(  # noqa: E731
        0, to.flatten(), x.flatten())[:size]
    mass = torch.cat([s["out_mass"], s["out_mass"][:, :1]], 1).scatter(1, row, s["mass"])[:, :-1]
    dptr, dto, dentry, _, dsize = outs[1]
    return (ptr, put(to, s["kv_indices"][entry], size), put(to, s["kv_pos"][entry], size), mass,
            dptr, put(dto, s["kv_indices"][dentry], dsize))


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        if op == "append":
            return _append(s)
        if op == "chunk":
            out, lse = _attend(s, "v_pool")
            return out.to(s["q"].dtype), lse
        return _mass(s) if op == "mass" else _evict(s)
    import kv_cache_drop_gb300 as akv
    if op == "evict":
        akv.akv_evict_by_mass(case["B"], s["kv_indptr"], s["kv_indices"], s["kv_pos"], s["mass"].shape[1],
                              s["mass"], s["keep"], FIRST, RECENT, s["out_indptr"], s["out_indices"],
                              s["out_pos"], s["out_mass"], s["dropped_indptr"], s["dropped"])
        return (s["out_indptr"], s["out_indices"], s["out_pos"], s["out_mass"], s["dropped_indptr"],
                s["dropped"])
    if "shape" not in s:
        s["shape"] = akv.shape(case["Hq"], case["Hkv"], D, case["dtype"], BASE)
    if op == "append":
        akv.akv_qk_norm_append(s["shape"], case["n"], s["q"], s["k"], s["v"], s["pos"], s["slot"],
                               s["k_pool"], s["v_pool"], s["q_out"], q_weight=s["qw"], k_weight=s["kw"],
                               eps=EPS)
        return s["q_out"], s["k_pool"], s["v_pool"]
    max_q, max_kv = max(s["qn"]), max(s["kv"])
    if "ws" not in s:  # sized once, kept with the batch's buffers
        size = akv.akv_chunk_workspace if op == "chunk" else akv.akv_attention_mass_workspace
        s["ws"] = torch.empty(size(s["shape"], case["B"], s["q"].shape[0], max_q, max_kv),
                              dtype=torch.uint8, device=DEV)
    if op == "chunk":
        akv.akv_chunk_attention(s["shape"], case["B"], s["q_indptr"], s["q"], s["k_pool"], s["v_pool"],
                                s["kv_indptr"], s["kv_indices"], max_q, max_kv, s["out"], s["lse"], s["ws"])
        return s["out"], s["lse"]
    akv.akv_attention_mass(s["shape"], case["B"], s["q_indptr"], s["q"], s["k_pool"], s["kv_indptr"],
                           s["kv_indices"], max_q, max_kv, s["lse"], DECAY, s["mass_in"], s["mass_out"],
                           s["ws"])
    return s["mass_out"]


def work(case):
    if case["op"] == "append":
        n, Hq, Hkv = case["n"], case["Hq"], case["Hkv"]
        real = n - n // case["pad"] if case["pad"] else n
        e = 2 if case["dtype"] == "bf16" else 4
        return dict(bytes=8 * n + 2 * real * (Hq + 2 * Hkv) * D * e + 8 * D,
                    flops=8 * real * (Hq + Hkv) * D)
    qn, kv = _lengths(case)
    if case["op"] == "evict":
        kept = sum(min(n, case["keep"]) for n in kv)
        return dict(bytes=12 * sum(kv) + 12 * kept + 4 * (sum(kv) - kept), flops=sum(kv))
    Hq, Hkv = case["Hq"], case["Hkv"]
    e = 2 if case["dtype"] == "bf16" else 4
    pairs = sum(sum(max(0, n - m + 1 + i) for i in range(m)) for m, n in zip(qn, kv))
    rows = sum(qn)
    if case["op"] == "chunk":
        return dict(bytes=2 * rows * Hq * D * e + 4 * rows * Hq + sum(kv) * (2 * Hkv * D * e + 4),
                    flops=4 * D * Hq * pairs)
    return dict(bytes=rows * Hq * (D * e + 4) + sum(kv) * (Hkv * D * e + 12), flops=2 * D * Hq * pairs)


def exact(case, seed):
    """The definitions in 64 bits, entry by entry of the lists."""
    if work(case)["flops"] > 1e13:
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op == "append":
        angle = s["pos"].double()[:, None] * torch.pow(
            torch.tensor(BASE, dtype=torch.float64, device=DEV),
            -torch.arange(0, D, 2, dtype=torch.float64, device=DEV) / D)
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]

        def row(x, w):
            x = x.double()
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + EPS) * w.double()
            z = torch.complex(x[..., :D // 2], x[..., D // 2:]) * turn
            return torch.cat([z.real, z.imag], -1)

        real = torch.nonzero(s["slot"] >= 0).flatten()
        to = s["slot"][real].long()
        q, k, v = s["q_out"].double(), s["k_pool"].double(), s["v_pool"].double()
        q[real] = row(s["q"], s["qw"])[real]
        k[to] = row(s["k"], s["kw"])[real]
        v[to] = s["v"].double()[real]
        return q, k, v
    if op == "evict":
        return (None,) * 3 + (_exact_kept_mass(s),) + (None,) * 2
    Hq, G = case["Hq"], case["Hq"] // case["Hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    mass = s["mass_out"].double() if op == "mass" else None
    for b, (m, n) in enumerate(zip(s["qn"], s["kv"])):
        at = s["kv_indices"][s["kv_ptr"][b]:s["kv_ptr"][b + 1]].long()
        if op == "mass":
            mass[b, :n - m] = DECAY * s["mass_in"][b, :n - m].double()
            mass[b, n - m:n] = 0
        step = max(1, (1 << 28) // (n * G))
        for h in range(0, Hq, G):
            K = s["k_pool"][at, h // G].double()
            V = s["v_pool"][at, h // G].double() if op == "chunk" else None
            for i in range(0, m, step):
                rows = torch.arange(s["q_ptr"][b] + i, s["q_ptr"][b] + min(m, i + step), device=DEV)
                last = n - m + (rows - s["q_ptr"][b])
                x = torch.einsum("rhd,kd->rhk", s["q"][rows, h:h + G].double() / math.sqrt(D), K)
                x.masked_fill_((torch.arange(n, device=DEV) > last[:, None])[:, None], -math.inf)
                if op == "mass":
                    mass[b, :n] += torch.exp(x - s["lse"][rows, h:h + G].double()[..., None]).sum((0, 1))
                    continue
                lse[rows, h:h + G] = torch.logsumexp(x, -1)
                out[rows, h:h + G] = torch.einsum("rhk,kd->rhd", torch.softmax(x, -1), V)
    return mass if op == "mass" else (out, lse)


def _exact_kept_mass(s):
    """The kept entries' masses, request by request, chosen one by one in 64 bits."""
    out = s["out_mass"].double()
    for b, n in enumerate(s["kv"]):
        value = s["mass"][b, :n].double()
        value[:FIRST] = math.inf
        value[max(0, n - RECENT):] = math.inf
        best = torch.sort(value, descending=True, stable=True).indices[:s["case"]["keep"]]
        best = torch.sort(best).values
        out[b, :len(best)] = s["mass"][b, best].double()
    return out
