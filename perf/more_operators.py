"""Cases for timing the operators of a cache held in 8 bits and of a shared
prefix: rows quantised as they are written, read back, decoded with rotation on
read, and attention of a batch whose requests share a long prefix.

An 8-bit row is 64 e4m3 values and one power of two: the smallest 2^s with
max |x| <= 448 * 2^s (s held to -127 .. 127; -127 for a row of zeros).

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
DEV = "cuda"
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def listed():
    return [
        # one decode step of 14 agents: their 14 new rows (8 KV heads)
        dict(name="write 14", op="write", n=14, Hkv=8, dtype="bf16", pad=0, fused=0),
        # a prefill chunk of many tool responses, k and v as column blocks of one projection
        dict(name="write 16384", op="write", n=16384, Hkv=8, dtype="bf16", pad=0, fused=1),
        # an odd batch padded to a captured size: one row in 16 is padding
        dict(name="write 4999 f32", op="write", n=4999, Hkv=4, dtype="f32", pad=16, fused=0),
        # the survivors of a 128k trajectory taken into a bf16 pool, keys rotated to 0 .. r-1
        dict(name="read 26081", op="read", n=26081, Hkv=8, dtype="bf16", turn=1),
        # a short message read back as it was written, three KV heads, single precision
        dict(name="read 701 f32", op="read", n=701, Hkv=3, dtype="f32", turn=0),
        # single tokens of 14 agents over 20k-90k active entries each, their rows appended in the call
        dict(name="decode 14", op="decode", B=14, kv_lo=20000, kv_hi=90000, Hq=64, Hkv=8, dtype="bf16",
             new=1, lengths=4),
        # short and long caches in one batch, three KV heads
        dict(name="decode mixed", op="decode", B=9, kv_lo=1, kv_hi=12000, Hq=24, Hkv=3, dtype="bf16",
             new=0, lengths=2),
        # single precision, as the library's parity workloads use
        dict(name="decode f32", op="decode", B=3, kv_lo=500, kv_hi=4000, Hq=16, Hkv=4, dtype="f32", new=1,
             lengths=1),
        # one token of each of 32 requests over a prefix of 8,192 and up to 24,576 entries of their own
        dict(name="prefix 32", op="prefix", G=1, B=32, q_lo=1, q_hi=1, p_lo=8192, p_hi=8192, kv_lo=1,
             kv_hi=24576, Hq=16, Hkv=4, dtype="bf16", lengths=5),
        # 14 agents that share a long document, a short history of each behind it
        dict(name="prefix 14 long", op="prefix", G=1, B=14, q_lo=1, q_hi=1, p_lo=50000, p_hi=50000, kv_lo=64,
             kv_hi=4096, Hq=64, Hkv=8, dtype="bf16", lengths=3),
        # two groups of requests, tool responses and single tokens mixed
        dict(name="prefix chunks", op="prefix", G=2, B=9, q_lo=1, q_hi=300, p_lo=1000, p_hi=8192, kv_lo=300,
             kv_hi=4000, Hq=24, Hkv=3, dtype="bf16", lengths=2),
        dict(name="prefix f32", op="prefix", G=2, B=5, q_lo=1, q_hi=20, p_lo=300, p_hi=2049, kv_lo=20,
             kv_hi=1000, Hq=16, Hkv=4, dtype="f32", lengths=6),
    ]


HEADS = [(64, 8), (16, 4), (8, 2), (24, 3), (32, 16), (2, 2)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "prefix", "prefix"])
    Hq, Hkv = rng.choice(HEADS)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    wide = Hkv * (1 if dtype == "bf16" else 2)  # of a token, beside a bf16 KV head
    if op == "write":
        return dict(op=op, n=_log(rng, 1, min(16384, 131072 // wide)), Hkv=Hkv, dtype=dtype,
                    pad=rng.choice([0, 0, 7, 16]), fused=rng.randint(0, 1))
    if op == "read":
        return dict(op=op, n=_log(rng, 1, min(26081, 208648 // wide)), Hkv=Hkv, dtype=dtype,
                    turn=rng.randint(0, 1))
    B = _log(rng, 1, 14 if op == "decode" else 32)
    if op == "decode":
        # 5.6 million (entry, KV head) pairs at most; in single precision 100,000
        most = (5600000 if dtype == "bf16" else 100000) // (B * Hkv)
        hi = _log(rng, 16, min(90000 if dtype == "bf16" else 8000, most))
        return dict(op=op, B=B, kv_lo=rng.randint(1, hi), kv_hi=hi, Hq=Hq, Hkv=Hkv, dtype=dtype,
                    new=rng.randint(0, 1), lengths=rng.randrange(1 << 20))
    G = rng.choice([1, 1, 2, 3])
    B = max(B, G)
    q = _log(rng, 1, 300 if dtype == "bf16" else 64)
    p = _log(rng, 16, 50000 if dtype == "bf16" else 4000)
    kv = _log(rng, max(q, 16), min(24576, 2400000 // (B * Hkv)) if dtype == "bf16" else 4000)
    # scores of the plain form: 2^27 over each of the two lists at most, or 2^24
    room = 1 << (24 if dtype == "f32" else 27)
    q = max(1, min(q, room // (B * Hq * max(p, kv))))
    return dict(op=op, G=G, B=B, q_lo=rng.randint(1, q), q_hi=q, p_lo=rng.randint(1, p), p_hi=p,
                kv_lo=rng.randint(q, kv), kv_hi=kv, Hq=Hq, Hkv=Hkv, dtype=dtype,
                lengths=rng.randrange(1 << 20))


def _lengths(case):
    """(chunks, own lists, groups' first requests, prefixes) of a batch, the
    longest of each first."""
    rng = random.Random(case["lengths"])
    B = case["B"]

    def some(lo, hi, n):
        return [hi] + [rng.randint(lo, hi) for _ in range(n - 1)]

    kv = some(case["kv_lo"], case["kv_hi"], B)
    if case["op"] == "decode":
        return [1] * B, kv, None, None
    qn = some(case["q_lo"], case["q_hi"], B)
    G = case["G"]
    cut = [0] + sorted(rng.sample(range(1, B), G - 1)) + [B]
    return qn, kv, cut, some(case["p_lo"], case["p_hi"], G)


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _csr(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _power(s):
    """2^s for whole s in -127 .. 127, exactly, in 32 bits."""
    return torch.exp2(s.double()).float()


def _quantise(x):
    """Rows [..., D] as e4m3 values and their powers of two."""
    x = x.float()
    top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    m, e = torch.frexp(top)  # top = m 2^e, 1/2 <= m < 1, and 448 = 0.875 * 2^9
    s = torch.where(top > 0, e - 9 + (m > 0.875), -127).clamp(-127, 127)
    codes = (x * _power(-s)[..., None]).to(F8)
    return codes, (s + 127).to(torch.uint8).view(E8)


def _values(codes, scale):
    """What they stand for, in 32 bits."""
    return codes.float() * _power(scale.view(torch.uint8).int() - 127)[..., None]


def _rotated(x, pos):
    """x [..., heads, D] turned to pos [...]: angles in 64 bits, the rest in 32."""
    th = BASE ** (-2.0 * torch.arange(D // 2, device=DEV, dtype=torch.float64) / D)
    a = pos.double()[..., None, None] * th
    c, sn = torch.cos(a).float(), torch.sin(a).float()
    x1, x2 = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([x1 * c - x2 * sn, x1 * sn + x2 * c], -1)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case=case)
    op, Hkv, t = case["op"], case["Hkv"], _type(case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def rows(n, spread):  # rows of uneven length, as projections give
        return (randn(n, Hkv, D) * torch.exp(spread * randn(n, 1, 1))).to(t)

    def pools(S):
        s["k_pool"], s["k_scale"] = _quantise(rows(S, 0.3))
        s["v_pool"], s["v_scale"] = _quantise(rows(S, 0.7))

    if op == "write":
        n = case["n"]
        S = n + max(64, n // 8)
        if case["fused"]:  # column blocks of one [n, 2 Hkv D] projection
            x = torch.cat([rows(n, 0.3), rows(n, 0.7)], 1)
            s["k"], s["v"] = x[:, :Hkv], x[:, Hkv:]
        else:
            s["k"], s["v"] = rows(n, 0.3), rows(n, 0.7)
        slot = torch.randperm(S, generator=g, device=DEV)[:n].to(torch.int32)
        if case["pad"]:
            slot[torch.arange(n, device=DEV) % case["pad"] == case["pad"] - 1] = -1
        s["slot"] = slot
        pools(S)
        return s
    if op == "read":
        n = case["n"]
        S = n + max(64, n // 8)
        pools(S)
        s["src"], s["dst"] = (torch.randperm(S, generator=g, device=DEV)[:n].to(torch.int32) for _ in range(2))
        s["pos"] = torch.arange(n, dtype=torch.int32, device=DEV) if case["turn"] else None
        s["k_out"], s["v_out"] = rows(S, 0.3), rows(S, 0.7)
        return s

    Hq = case["Hq"]
    qn, kv, cut, pre = _lengths(case)
    nnz = sum(kv) + sum(pre or [])
    S = nnz + max(64, nnz // 10)
    free = torch.randperm(S, generator=g, device=DEV).to(torch.int32)
    s["kv"], s["kv_ptr"] = kv, _csr(kv)
    s["kv_indptr"], s["kv_indices"] = _i32(s["kv_ptr"]), free[:sum(kv)].contiguous()
    # normalised rows (scores of standard deviation 2)
    s["q"] = (2 * randn(sum(qn), Hq, D)).to(t)
    s["out"] = torch.zeros_like(s["q"])
    if op == "decode":
        pools(S)
        # logical order with whole messages dropped, or renumbered 0 .. n-1
        j = torch.arange(sum(kv), device=DEV) - torch.repeat_interleave(
            s["kv_indptr"][:-1], (s["kv_indptr"][1:] - s["kv_indptr"][:-1]).long())
        gap = torch.repeat_interleave(_i32([(b % 3) * 331 for b in range(case["B"])]),
                                      (s["kv_indptr"][1:] - s["kv_indptr"][:-1]).long())
        s["kv_pos"] = (j + gap * (j // 701)).to(torch.int32)
        last = s["kv_indptr"][1:].long() - 1
        s["q_pos"] = s["kv_pos"][last].contiguous()
        s["k_new"], s["v_new"], s["new_slot"] = None, None, None
        if case["new"]:  # each list ends with its new token's slot
            s["k_new"], s["v_new"] = rows(case["B"], 0.3), rows(case["B"], 0.7)
            s["new_slot"] = s["kv_indices"][last].contiguous()
        return s
    s["qn"], s["q_ptr"] = qn, _csr(qn)
    s["q_indptr"] = _i32(s["q_ptr"])
    s["pre"], s["pre_ptr"] = pre, _csr(pre)
    s["prefix_indptr"], s["prefix_indices"] = _i32(s["pre_ptr"]), free[sum(kv):nnz].contiguous()
    # rows of group g: those of its requests
    s["group_ptr"] = [s["q_ptr"][b] for b in cut]
    s["group_indptr"] = _i32(s["group_ptr"])
    s["max_rows"] = max(b - a for a, b in zip(s["group_ptr"], s["group_ptr"][1:]))
    s["k_pool"], s["v_pool"] = rows(S, 0.3), rows(S, 0.3)
    s["lse"] = torch.zeros(sum(qn), Hq, device=DEV)
    return s


def _write(s):
    S = s["k_pool"].shape[0]
    # a padding row's slot is the pool's last row plus one: a row that is cut off again
    slot = torch.where(s["slot"] >= 0, s["slot"], S).long()
    outs = []
    for x, pool, scale in ((s["k"], "k_pool", "k_scale"), (s["v"], "v_pool", "v_scale")):
        codes, power = _quantise(x)
        for old, new, t in ((s[pool], codes, F8), (s[scale], power, E8)):
            old, new = old.view(torch.uint8), new.view(torch.uint8)
            if s["case"]["pad"]:
                old = torch.cat([old, old[:1]])
            old[slot] = new
            outs.append(old[:S].view(t))
    return outs


def _read(s):
    src, dst = s["src"].long(), s["dst"].long()
    for pool, scale, out in (("k_pool", "k_scale", "k_out"), ("v_pool", "v_scale", "v_out")):
        x = _values(s[pool].view(torch.uint8)[src].view(F8), s[scale].view(torch.uint8)[src].view(E8))
        if out == "k_out" and s["pos"] is not None:
            x = _rotated(x, s["pos"])
        s[out][dst] = x.to(s[out].dtype)
    return s["k_out"], s["v_out"]


def _padded(ptr, wide, total):
    """[lists, wide] places of the entries of lists, and which of them there are."""
    j = torch.arange(wide, device=DEV)
    at = ptr[:-1, None] + j
    return at.clamp(max=total - 1).long(), at < ptr[1:, None]


def _decode(s):
    case = s["case"]
    B, Hkv, G = case["B"], case["Hkv"], case["Hq"] // case["Hkv"]
    if case["new"]:
        at = s["new_slot"].long()
        for x, pool, scale in ((s["k_new"], "k_pool", "k_scale"), (s["v_new"], "v_pool", "v_scale")):
            codes, power = _quantise(x)
            s[pool].view(torch.uint8)[at] = codes.view(torch.uint8)
            s[scale].view(torch.uint8)[at] = power.view(torch.uint8)
    e, there = _padded(s["kv_indptr"], max(s["kv"]), s["kv_indices"].numel())
    slot = s["kv_indices"][e].long()

    def cached(pool, scale):  # [B, n, Hkv, D]
        return _values(s[pool].view(torch.uint8)[slot].view(F8), s[scale].view(torch.uint8)[slot].view(E8))

    q = _rotated(s["q"].float(), s["q_pos"]).view(B, Hkv, G, D)
    k = _rotated(cached("k_pool", "k_scale"), s["kv_pos"][e])
    x = (q @ k.permute(0, 2, 3, 1)) * 0.125
    x = torch.where(there[:, None, None], x, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = (p @ cached("v_pool", "v_scale").transpose(1, 2)) / p.sum(-1, keepdim=True)
    out = o.reshape(B, case["Hq"], D).to(s["q"].dtype)
    return (out, s["k_pool"], s["k_scale"], s["v_pool"], s["v_scale"]) if case["new"] else out


def _part(s, row_ptr, most, list_ptr, indices, wide, causal):
    """Attention of packed rows over the lists of their requests (or groups):
    unnormalised outputs [rows, Hq, D], maxima and sums [rows, Hq]."""
    case = s["case"]
    Hkv, G = case["Hkv"], case["Hq"] // case["Hkv"]
    r, row = _padded(row_ptr, most, s["q"].shape[0])
    e, there = _padded(list_ptr, wide, indices.numel())
    slot = indices[e].long()
    k, v = (s[n][slot].float().permute(0, 2, 1, 3) for n in ("k_pool", "v_pool"))  # [L, Hkv, n, D]
    q = s["q"][r].float().view(-1, most, Hkv, G, D).permute(0, 2, 1, 3, 4)  # [L, Hkv, rows, G, D]
    x = (q.reshape(q.shape[0], Hkv, most * G, D) @ k.transpose(2, 3)).view(-1, Hkv, most, G, wide) * 0.125
    see = there[:, None].expand(-1, most, -1)
    if causal:
        n, m = (p[1:] - p[:-1] for p in (list_ptr, row_ptr))
        i = torch.arange(most, device=DEV)
        see = see & (torch.arange(wide, device=DEV) <= ((n - m)[:, None] + i)[..., None])
    x = torch.where(see[:, None, :, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    o = (p.view(-1, Hkv, most * G, wide) @ v).view(-1, Hkv, most, G, D)
    pack = lambda y: y.permute(0, 2, 1, 3, 4).reshape(y.shape[0], most, case["Hq"], -1)[row]  # noqa: E731
    return pack(o), pack(top), pack(p.sum(-1, keepdim=True))


def _prefix(s):
    parts = [_part(s, s["group_indptr"], s["max_rows"], s["prefix_indptr"], s["prefix_indices"],
                   max(s["pre"]), False),
             _part(s, s["q_indptr"], max(s["qn"]), s["kv_indptr"], s["kv_indices"], max(s["kv"]), True)]
    top = torch.maximum(parts[0][1], parts[1][1])
    f = [torch.exp(m - top) for _, m, _ in parts]
    tot = f[0] * parts[0][2] + f[1] * parts[1][2]
    out = (f[0] * parts[0][0] + f[1] * parts[1][0]) / tot
    return out.to(s["q"].dtype), (top + torch.log(tot))[..., 0]


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return dict(write=_write, read=_read, decode=_decode, prefix=_prefix)[op](s)
    import kv_cache_drop_gb300 as akv
    if "shape" not in s:
        s["shape"] = akv.shape(case.get("Hq", case["Hkv"]), case["Hkv"], D, case["dtype"], BASE)
    if op == "write":
        akv.akv_append_kv_q8(s["shape"], case["n"], s["k"], s["v"], s["slot"], s["k_pool"], s["v_pool"],
                             s["k_scale"], s["v_scale"])
        return [s["k_pool"], s["k_scale"], s["v_pool"], s["v_scale"]]
    if op == "read":
        akv.akv_read_kv_q8(s["shape"], case["n"], s["src"], s["pos"], s["dst"], s["k_pool"], s["v_pool"],
                           s["k_scale"], s["v_scale"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    max_kv = max(s["kv"])
    if op == "decode":
        if "ws" not in s:  # sized once, kept with the batch's buffers
            s["ws"] = torch.empty(akv.akv_decode_q8_workspace(s["shape"], case["B"], max_kv),
                                  dtype=torch.uint8, device=DEV)
        akv.akv_decode_attention_q8(s["shape"], case["B"], s["q"], s["q_pos"], s["k_new"], s["v_new"],
                                    s["new_slot"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"],
                                    s["kv_indptr"], s["kv_indices"], s["kv_pos"], max_kv, s["out"], s["ws"])
        if case["new"]:
            return s["out"], s["k_pool"], s["k_scale"], s["v_pool"], s["v_scale"]
        return s["out"]
    sizes = dict(max_rows=s["max_rows"], max_prefix=max(s["pre"]), max_q=max(s["qn"]), max_kv=max_kv)
    if "ws" not in s:
        s["ws"] = torch.empty(akv.akv_prefix_workspace(s["shape"], case["G"], case["B"], s["q"].shape[0],
                                                       **sizes), dtype=torch.uint8, device=DEV)
    akv.akv_prefix_attention(s["shape"], case["G"], s["group_indptr"], s["prefix_indptr"],
                             s["prefix_indices"], case["B"], s["q_indptr"], s["q"], s["k_pool"],
                             s["v_pool"], s["kv_indptr"], s["kv_indices"], out=s["out"], lse=s["lse"],
                             workspace=s["ws"], **sizes)
    return s["out"], s["lse"]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, Hkv = case["op"], case["Hkv"]
    if op == "write":
        n = case["n"]
        real = n - n // case["pad"] if case["pad"] else n
        return dict(bytes=4 * n + 2 * real * Hkv * (D * e + D + 1), flops=3 * 2 * real * Hkv * D)
    if op == "read":
        n = case["n"]
        return dict(bytes=(8 + 4 * case["turn"]) * n + 2 * n * Hkv * (D + 1 + D * e), flops=6 * n * Hkv * D)
    Hq = case["Hq"]
    qn, kv, cut, pre = _lengths(case)
    if op == "decode":
        B = case["B"]
        new = 2 * B * Hkv * (D * e + D + 1) if case["new"] else 0
        return dict(bytes=2 * B * Hq * D * e + sum(kv) * (2 * Hkv * (D + 1) + 8) + new,
                    flops=sum(kv) * (4 * D * Hq + 4 * D * Hkv))
    rows = sum(qn)
    pairs = sum(sum(qn[a:b]) * n for a, b, n in zip(cut, cut[1:], pre))
    pairs += sum(sum(max(0, n - m + 1 + i) for i in range(m)) for m, n in zip(qn, kv))
    return dict(bytes=2 * rows * Hq * D * e + 4 * rows * Hq + (sum(kv) + sum(pre)) * (2 * Hkv * D * e + 4),
                flops=4 * D * Hq * pairs)


def _exact_rows(x):
    """Rows in 64 bits to the nearest e4m3 value (ties to even) and their powers of two."""
    x = x.double()
    two = torch.tensor([2.0 ** s for s in range(-127, 128)], dtype=torch.float64, device=DEV)
    s = (x.abs().amax(-1)[..., None] > 448 * two[:-1]).sum(-1)  # steps to the first that holds the row
    y = x / two[s][..., None]
    place = (y.abs()[..., None] >= two[127 - 6:127 + 9]).sum(-1).clamp(min=1) - 1  # exponent + 6
    step = two[127 - 9:][place]
    return torch.round(y / step) * step, two[s]


def _exact_turn(x, pos):
    a = pos.double()[:, None] * torch.pow(torch.tensor(BASE, dtype=torch.float64, device=DEV),
                                          -torch.arange(0, D, 2, dtype=torch.float64, device=DEV) / D)
    z = torch.complex(x[..., :D // 2], x[..., D // 2:]) * torch.polar(torch.ones_like(a), a)[:, None]
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    """The definitions in 64 bits, list by list."""
    if work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    op = case["op"]

    def held(pool, scale, at):  # what the rows `at` of an 8-bit pool stand for
        p = s[scale].view(torch.uint8)[at].view(E8).double()
        return s[pool].view(torch.uint8)[at].view(F8).double() * p[..., None]

    def written(x, pool, scale, at):  # an 8-bit pool's values after rows x went to `at`
        v, p = _exact_rows(x)
        codes, power = s[pool].double(), s[scale].double()
        codes[at], power[at] = v, p
        return codes, power

    if op == "write":
        real = torch.nonzero(s["slot"] >= 0).flatten()
        at = s["slot"][real].long()
        return [x for a, b, c in (("k", "k_pool", "k_scale"), ("v", "v_pool", "v_scale"))
                for x in written(s[a][real], b, c, at)]
    if op == "read":
        src, dst = s["src"].long(), s["dst"].long()
        k, v = s["k_out"].double(), s["v_out"].double()
        x = held("k_pool", "k_scale", src)
        k[dst] = x if s["pos"] is None else _exact_turn(x, s["pos"])
        v[dst] = held("v_pool", "v_scale", src)
        return k, v
    Hq, G = case["Hq"], case["Hq"] // case["Hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    if op == "decode":
        state = []
        if case["new"]:
            at = s["new_slot"].long()
            for a, b, c in (("k_new", "k_pool", "k_scale"), ("v_new", "v_pool", "v_scale")):
                codes, power = written(s[a], b, c, at)
                state += [codes, power]
                s[b].view(torch.uint8)[at] = codes[at].to(F8).view(torch.uint8)
                s[c].view(torch.uint8)[at] = (torch.frexp(power[at])[1] + 126).to(torch.uint8)
        q = _exact_turn(s["q"].double(), s["q_pos"]) / math.sqrt(D)
        for b in range(case["B"]):
            one = slice(s["kv_ptr"][b], s["kv_ptr"][b + 1])
            at = s["kv_indices"][one].long()
            k = _exact_turn(held("k_pool", "k_scale", at), s["kv_pos"][one])
            v = held("v_pool", "v_scale", at)
            for h in range(Hq):
                w = torch.softmax(k[:, h // G] @ q[b, h], 0)
                out[b, h] = w @ v[:, h // G]
        return (out, *state) if case["new"] else out
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    for b, (m, n) in enumerate(zip(s["qn"], s["kv"])):
        r0, r1 = s["q_ptr"][b], s["q_ptr"][b + 1]
        g = max(i for i in range(case["G"]) if s["group_ptr"][i] <= r0)
        at = torch.cat([s["prefix_indices"][s["pre_ptr"][g]:s["pre_ptr"][g + 1]],
                        s["kv_indices"][s["kv_ptr"][b]:s["kv_ptr"][b + 1]]]).long()
        j = torch.arange(len(at), device=DEV) - s["pre"][g]  # below 0: the prefix
        hidden = j > (n - m + torch.arange(m, device=DEV))[:, None]
        for h in range(Hq):
            x = (s["q"][r0:r1, h].double() / math.sqrt(D)) @ s["k_pool"][at, h // G].double().T
            x.masked_fill_(hidden, -math.inf)
            lse[r0:r1, h] = torch.logsumexp(x, -1)
            out[r0:r1, h] = torch.softmax(x, -1) @ s["v_pool"][at, h // G].double()
    return out, lse
