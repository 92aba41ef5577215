"""The measured calls of the 4-bit cache and of eviction: writing K/V rows to 4-bit pages and
reading them back, verify attention over such pages, adding up the attention weight of each
cached position, and evicting the positions of least weight.

``own`` False computes every operator in plain torch operations; ``own`` True calls the
library. ``exact`` computes the same outputs in 64 bits, sequence by sequence.
"""
import math
import random

import torch

own = False

GOLDEN = 0.6180339887498949


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], spread evenly and out of order (the ragged lengths of a
    batch; the same for every seed, so that a case has one amount of work)."""
    return [lo + int(((i + 1) * GOLDEN) % 1.0 * (hi - lo + 1)) for i in range(n)]


def _ceil(a, b):
    return -(-a // b)


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # the windows of one decoding step are written, and read back as the rounded values
        # that the step's own attention uses: a small batch, all launch latency
        dict(name="write windows", op="write", B=8, Hkv=8, d=128, start=1000, count=9, block=16),
        # prompts of a ragged prefill batch, rounded and read back for the prefill's attention
        dict(name="write prompts", op="write", B=8, Hkv=8, d=128, start=0, count=8192, block=16),
        # one sequence's context is read back to be moved to another cache
        dict(name="read context", op="read", B=1, Hkv=8, d=128, start=0, count=4001, block=16),
        # contexts of a batch, read back for a chunk of prefill over them
        dict(name="read contexts", op="read", B=16, Hkv=8, d=128, start=0, count=16384, block=64),
        # a small model's only sequence: launch latency is all there is
        dict(name="attn small", op="attn", B=1, Hq=4, Hkv=1, d=64, D=3, T=256, ragged=False, block=16),
        # plain decoding of a ragged batch: single tokens
        dict(name="attn single tokens", op="attn", B=64, Hq=32, Hkv=8, d=128, D=0, T=8192, ragged=True,
             block=16),
        # full draft windows, 128 query rows a KV head
        dict(name="attn windows", op="attn", B=16, Hq=32, Hkv=8, d=128, D=31, T=8192, ragged=False,
             block=16),
        # long contexts of a larger model
        dict(name="attn long", op="attn", B=8, Hq=64, Hkv=8, d=128, D=15, T=32768, ragged=False, block=64),
        # after acceptance, the accepted rows' weights over a 4-bit cache, log-sums from the attention call
        dict(name="mass 4 bits", op="mass", kv="kv4", lse=True, B=16, Hq=32, Hkv=8, d=128, D=8, T=8192,
             ragged=True, block=16),
        # the same over a bf16 cache whose attention call gave no log-sums
        dict(name="mass bf16", op="mass", kv="bf16", lse=False, B=32, Hq=32, Hkv=4, d=128, D=7, T=16384,
             ragged=True, block=16),
        # two short conversations are cut to a small budget
        dict(name="evict short", op="evict", kv="bf16", B=2, Hkv=2, d=64, T=600, keep=256, first=4, last=32,
             block=16),
        # long contexts of a batch are cut to a quarter, 8-bit cache
        dict(name="evict long", op="evict", kv="e4m3", B=32, Hkv=4, d=128, T=16384, keep=4096, first=64,
             last=256, block=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "attn", "mass", "mass", "evict"])
    block = rng.choice([8, 16, 32, 64, 128])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([2, 4, 8])
    while True:
        if op in ("write", "read"):
            c = dict(op=op, B=_log(rng, 1, 64), Hkv=Hkv, d=d, start=rng.choice([0, _log(rng, 1, 2000)]),
                     count=_log(rng, 1, 16384), block=block)
            if sum(_counts(c)) * Hkv * d <= (1 << 26):
                return c
        elif op == "attn":
            c = dict(op=op, B=_log(rng, 1, 64), Hq=Hkv * rng.choice([1, 2, 4, 7, 8]), Hkv=Hkv, d=d,
                     D=rng.choice([0, 0, 1, 3, 5, 8, 15, 31]), T=_log(rng, 1, 32768),
                     ragged=rng.random() < 0.5, block=block)
        elif op == "mass":
            c = dict(op=op, kv=rng.choice(["bf16", "e4m3", "kv4", "kv4"]), lse=rng.random() < 0.5,
                     B=_log(rng, 1, 32), Hq=Hkv * rng.choice([1, 2, 4, 7, 8]), Hkv=Hkv, d=d,
                     D=rng.choice([0, 1, 3, 5, 8, 15]), T=_log(rng, 1, 16384), ragged=rng.random() < 0.5,
                     block=block)
        else:
            T = _log(rng, 64, 16384)
            keep = _log(rng, 8, T)
            c = dict(op=op, kv=rng.choice(["bf16", "e4m3"]), B=_log(rng, 1, 32), Hkv=Hkv, d=d, T=T, keep=keep,
                     first=rng.randint(0, keep // 4), last=rng.randint(0, keep // 2), block=block)
        w = work(c)
        if w["flops"] < 5e10 and w["bytes"] < 3e8:
            return c


# -------------------------------------------------------------- what a case's sizes are

def _counts(c):
    """Rows of each sequence of a write or read case: ragged above a window's length."""
    return _spread(c["B"], max(1, c["count"] // 2) if c["count"] > 64 else 1, c["count"])


def _lens(c):
    """(T, D) of each sequence of an attention or mass case."""
    T = _spread(c["B"], 0, c["T"]) if c["ragged"] else [c["T"]] * c["B"]
    D = _spread(c["B"], 0, c["D"]) if c["ragged"] else [c["D"]] * c["B"]
    return T, D


def _accepted(c):
    """Accepted rows of each window."""
    return [1 + (7 * b + 3) % (1 + n) for b, n in enumerate(_lens(c)[1])]


def _evict_lens(c):
    """Lengths of the rows of an evict case: some are within the budget already."""
    return _spread(c["B"], max(1, c["T"] * 3 // 4), c["T"])


def _evict_new(c):
    return [min(c["keep"], n) for n in _evict_lens(c)]


def _row_bytes(c):
    """Bytes of one (position, KV head) of K."""
    return {"kv4": c["d"] // 2 + c["d"] // 16, "e4m3": c["d"], "bf16": 2 * c["d"]}[c.get("kv", "kv4")]


def work(c):
    if c["op"] in ("write", "read"):
        n = sum(_counts(c)) * c["Hkv"] * 2
        both = n * (2 * c["d"] + _row_bytes(c))
        return {"bytes": both * (2 if c["op"] == "write" else 1), "flops": 0}
    if c["op"] == "evict":
        n, m = sum(_evict_lens(c)), sum(_evict_new(c))
        # kept positions: the first stay, of the others the share that the heaviest are moves
        moved = sum(max(0, k - c["first"]) for k, t in zip(_evict_new(c), _evict_lens(c)) if k < t)
        return {"bytes": 4 * c["Hkv"] * (2 * n + m) + 4 * moved * c["Hkv"] * _row_bytes(c), "flops": 0}
    T, D = _lens(c)
    rows, keys = sum(D) + c["B"], sum(T) + sum(D) + c["B"]
    if c["op"] == "attn":
        flops = sum((t + i + 1) * 4 * c["Hq"] * c["d"] for t, n in zip(T, D) for i in range(1 + n))
        return {"bytes": 4 * rows * c["Hq"] * c["d"] + 4 * rows * c["Hq"] + 2 * keys * c["Hkv"] * _row_bytes(c),
                "flops": flops}
    A = _accepted(c)
    flops = sum((t + i + 1) * 2 * c["Hq"] * c["d"] for t, n in zip(T, A) for i in range(n))
    keys = sum(t + n for t, n in zip(T, A))
    return {"bytes": sum(A) * c["Hq"] * (2 * c["d"] + 4) + keys * c["Hkv"] * (_row_bytes(c) + 8), "flops": flops}


# ------------------------------------------------------------------------------ the format

def _e4m3_round(a):
    """a >= 0 in 64 bits to the nearest E4M3 value, ties to even, 448 at most."""
    step = torch.exp2((torch.frexp(a).exponent - 1).clamp(min=-6).double() - 3)
    return (torch.round(a / step) * step).clamp(max=448.0)


def _e2m1_code(y):
    """y in 64 bits to E2M1 codes, ties to even, saturating."""
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
            + (a > 5.0))
    return code + 8 * (y < 0).to(torch.uint8)


def _quantise(x, head_scale):
    """x [..., Hkv, d] -> (codes uint8 [..., Hkv, d / 2], block scales [..., Hkv, d / 16] as
    uint8 E4M3 codes). The quotients are taken in 64 bits: a value next to the middle of two
    codes goes where the real quotient does."""
    b = x.double().unflatten(-1, (-1, 16))
    hs = head_scale.double()[:, None]
    c = _e4m3_round(b.abs().amax(-1) / (6 * hs))
    unit = (c * hs)[..., None]
    code = _e2m1_code(torch.where(unit > 0, b / torch.where(unit > 0, unit, 1.0), 0.0)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), c.to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes, scales, head_scale, dtype=torch.float32):
    """What codes [..., Hkv, d / 2] with block scales [..., Hkv, d / 16] stand for, [..., Hkv, d]."""
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=dtype, device=codes.device)
    lut = torch.cat([lut, -lut])
    e = lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]
    u = scales.view(torch.float8_e4m3fn).to(dtype) * head_scale.to(dtype)[:, None]
    return (e.unflatten(-1, (-1, 16)) * u[..., None]).flatten(-2)


# ------------------------------------------------------------------------------ inputs

def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _table(lens, bs, gen, dev, spare=5):
    """A block table for rows of these lengths, their pages placed at random; (table, blocks)."""
    pages = [_ceil(n, bs) for n in lens]
    stride, blocks = max(pages) + 1, sum(pages) + spare
    place = torch.randperm(blocks, generator=gen, device=dev).to(torch.int32)
    first = torch.tensor(pages).cumsum(0) - torch.tensor(pages)
    j = torch.arange(stride)
    have = (j < torch.tensor(pages)[:, None]).to(dev)
    at = (first[:, None] + j).clamp(max=blocks - 1).to(dev)
    return torch.where(have, place[at], -1).contiguous(), blocks


def _normal(gen, dev, *shape):
    return torch.empty(*shape, dtype=torch.bfloat16, device=dev).normal_(generator=gen)


def _pages4(c, blocks, gen, dev, v=True):
    """Pages of a 4-bit cache that hold rounded normal values: (k codes, v codes, scales, kv_scale)."""
    shape = (blocks, c["block"], c["Hkv"])
    hs = torch.rand(2, c["Hkv"], generator=gen, device=dev) * 0.002 + 0.001
    scales = torch.empty(*shape, 2, c["d"] // 16, dtype=torch.uint8, device=dev)
    codes = [torch.empty(*shape, c["d"] // 2, dtype=torch.uint8, device=dev) for _ in range(1 + v)]
    some = max(1, (1 << 24) // (c["block"] * c["Hkv"] * c["d"]))
    for i in range(1 + v):
        for p in range(0, blocks, some):  # a part of the pool at a time, in 64 bits
            n = min(some, blocks - p)
            codes[i][p:p + n], scales[p:p + n, :, :, i] = _quantise(_normal(gen, dev, n, *shape[1:], c["d"]), hs[i])
    return codes[0], codes[-1], scales, hs


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    c, bs = case, case["block"]
    s = dict(c=c)
    if c["op"] in ("write", "read"):
        n = _counts(c)
        s["table"], blocks = _table([c["start"] + k for k in n], bs, gen, dev)
        s["start"], s["count"], s["rows"] = _i32([c["start"]] * c["B"], dev), _i32(n, dev), sum(n)
        s["kc"], s["vc"], s["scales"], s["hs"] = _pages4(c, blocks, gen, dev)
        if c["op"] == "write":
            s["k"], s["v"] = (_normal(gen, dev, s["rows"], c["Hkv"], c["d"]) for _ in "kv")
        s["kout"], s["vout"] = (torch.zeros(s["rows"], c["Hkv"], c["d"], dtype=torch.bfloat16, device=dev)
                                for _ in "kv")
    elif c["op"] in ("attn", "mass"):
        T, D = _lens(c)
        s["table"], blocks = _table([t + 1 + n for t, n in zip(T, D)], bs, gen, dev)
        s.update(T=_i32(T, dev), D=_i32(D, dev), max_T=max(T), max_D=max(D))
        s["q"] = _normal(gen, dev, sum(D) + c["B"], c["Hq"], c["d"])
        if c["op"] == "attn":
            s["kc"], s["vc"], s["scales"], s["hs"] = _pages4(c, blocks, gen, dev)
            s["out"] = torch.zeros_like(s["q"])
            s["lse"] = torch.zeros(s["q"].shape[:2], dtype=torch.float32, device=dev)
        else:
            _mass_inputs(c, s, blocks, gen, dev)
    else:
        _evict_inputs(c, s, gen, dev)
    if own:
        _own_plan(s)
    return s


def _mass_inputs(c, s, blocks, gen, dev):
    s["scales"] = s["hs"] = None
    if c["kv"] == "kv4":
        s["kc"], _, s["scales"], s["hs"] = _pages4(c, blocks, gen, dev, v=False)
        s["scales"][..., 1, :] = s["scales"][..., 0, :]
    else:
        s["kc"] = _normal(gen, dev, blocks, c["block"], c["Hkv"], c["d"])
        if c["kv"] == "e4m3":
            s["hs"] = (s["kc"].abs().amax(dim=(0, 1, 3)).float() / 448).expand(2, -1).contiguous()
            s["kc"] = (s["kc"].float() / s["hs"][0][:, None]).to(torch.float8_e4m3fn)
    s["accepted"] = _i32(_accepted(c), dev)
    s["width"] = s["max_T"] + 1 + s["max_D"]
    # what earlier steps added: most positions little, a few much
    s["mass"] = torch.empty(c["B"], c["Hkv"], s["width"], device=dev).exponential_(100, generator=gen)
    s["lse"] = _scores(s)[1] if c["lse"] else None


def _evict_inputs(c, s, gen, dev):
    n = _evict_lens(c)
    s["table"], blocks = _table(n, c["block"], gen, dev)
    s["ref"] = torch.zeros(blocks, dtype=torch.int32, device=dev)
    s["ref"][s["table"][s["table"] >= 0].long()] = 1
    s["lens"], s["new_len"], s["first"] = _i32(n, dev), _i32(_evict_new(c), dev), _i32([c["first"]] * c["B"], dev)
    s["row"] = torch.randperm(c["B"], generator=gen, device=dev).to(torch.int32)
    s["new_len"] = s["new_len"][s["row"].long()].contiguous()
    # the weights that decoding adds up: heavy-tailed, and zero for some positions
    m = torch.empty(c["B"], c["Hkv"], max(n), device=dev).normal_(generator=gen)
    s["mass0"] = (2 * m).exp_() * (m > -1)
    s["mass"] = s["mass0"].clone()
    kv = _normal(gen, dev, 2, blocks, c["block"], c["Hkv"], c["d"])
    s["kv"] = (kv * 32).to(torch.float8_e4m3fn) if c["kv"] == "e4m3" else kv
    s["kept"] = torch.zeros(c["B"], c["Hkv"], max(_evict_new(c)), dtype=torch.int32, device=dev)


def _own_plan(s):
    """The workspaces, and the handle of the pools, that a program of the library's keeps
    between its calls."""
    import speculative_decoding_verification_gqa_gb300 as sv
    c, dev = s["c"], s["table"].device
    if c["op"] in ("attn", "mass"):
        desc = sv.paged_attn_desc(s["q"], s["kc"], c["B"], s["max_D"], s["max_T"], kv4=s["scales"] is not None)
        n = (sv.verify_kv4_workspace_bytes if c["op"] == "attn" else sv.mass_workspace_bytes)(desc)
    elif c["op"] == "evict":
        s["data"] = sv.page_pools(list(s["kv"].unbind(0)))
        n = sv.evict_workspace_bytes(c["B"], c["Hkv"], s["mass"].shape[2])
    else:
        n = sv.kv4_workspace_bytes(c["B"])
    s["ws"] = sv.new_workspace(n, dev)


# ---------------------------------------------------------------------------- the passes

def run(s):
    return (_own if own else _plain)[s["c"]["op"]](s)


def _write_own(s):
    import speculative_decoding_verification_gqa_gb300 as sv
    sv.spec_kv4_write(s["k"], s["v"], s["kc"], s["vc"], s["scales"], s["hs"], s["table"], s["start"], s["count"],
                      workspace=s["ws"])
    return _read_own(s)


def _read_own(s):
    import speculative_decoding_verification_gqa_gb300 as sv
    sv.spec_kv4_read(s["kc"], s["vc"], s["scales"], s["hs"], s["table"], s["start"], s["count"], k_out=s["kout"],
                     v_out=s["vout"], workspace=s["ws"])
    return dict(k=s["kout"], v=s["vout"])


def _attn_own(s):
    import speculative_decoding_verification_gqa_gb300 as sv
    sv.spec_verify_attn_kv4(s["q"], s["kc"], s["vc"], s["scales"], s["hs"], s["table"], s["T"], s["D"],
                            max_draft_len=s["max_D"], max_seq_len=s["max_T"], out=s["out"], lse=s["lse"],
                            workspace=s["ws"])
    return dict(out=s["out"], lse=s["lse"])


def _mass_own(s):
    import speculative_decoding_verification_gqa_gb300 as sv
    return sv.spec_attn_mass(s["q"], s["kc"], s["table"], s["T"], s["D"], s["mass"], max_draft_len=s["max_D"],
                             max_seq_len=s["max_T"], kv_scale=s["hs"], scales=s["scales"], lse=s["lse"],
                             row_count=s["accepted"], workspace=s["ws"])


def _evict_own(s):
    import speculative_decoding_verification_gqa_gb300 as sv
    s["mass"].copy_(s["mass0"])  # a pass changes the weights in place: start from the same ones
    sv.spec_kv_evict(s["ref"], s["table"], s["lens"], s["row"], s["new_len"], s["mass"], block_size=s["c"]["block"],
                     pools=s["data"], keep_first=s["first"], keep_last=s["c"]["last"], kept=s["kept"],
                     workspace=s["ws"])
    return dict(kept=s["kept"], mass=s["mass"], kv=s["kv"])


def _written(s):
    """(page, position in it) of each packed row of a write or read."""
    bs, rows, dev = s["c"]["block"], s["rows"], s["table"].device
    ends = s["count"].long().cumsum(0)
    r = torch.arange(rows, device=dev)
    seq = torch.searchsorted(ends, r, right=True)
    pos = r - (ends - s["count"])[seq] + s["start"][seq]
    return s["table"][seq, pos // bs].long(), pos % bs


def _write_plain(s):
    at = _written(s)
    s["kc"][at], ks = _quantise(s["k"], s["hs"][0])
    s["vc"][at], vs = _quantise(s["v"], s["hs"][1])
    s["scales"][at] = torch.stack([ks, vs], -2)
    return _read_plain(s)


def _read_plain(s):
    at = _written(s)
    u = s["scales"][at]
    s["kout"].copy_(_values(s["kc"][at], u[:, :, 0], s["hs"][0]))
    s["vout"].copy_(_values(s["vc"][at], u[:, :, 1], s["hs"][1]))
    return dict(k=s["kout"], v=s["vout"])


def _cached(s, pages, pos):
    """The rows of `pages` at positions `pos` [m] of every sequence, [B, m, ...]."""
    bs = s["c"]["block"]
    page = s["table"][:, (pos // bs).clamp(max=s["table"].shape[1] - 1)].long().clamp(min=0)
    return pages[page, pos % bs]


def _scores(s):
    """Every window row's scores in natural units, masked ones -inf, [B, Hkv, W * G, keys]; the
    log-sum-exp of the packed rows [rows, Hq]; the (sequence, row) of each packed row."""
    c, dev = s["c"], s["q"].device
    B, Hkv, d, G = c["B"], c["Hkv"], c["d"], c["Hq"] // c["Hkv"]
    T, D = s["T"].long(), s["D"].long()
    W, n = s["max_D"] + 1, s["max_T"] + 1 + s["max_D"]
    pos = torch.arange(n, device=dev)
    K = _cached(s, s["kc"], pos)
    if s["scales"] is not None:
        K = _values(K, _cached(s, s["scales"], pos)[:, :, :, 0], s["hs"][0])
    else:
        K = K.float() * (s["hs"][0][:, None] if s["hs"] is not None else 1.0)
    off = (1 + D).cumsum(0) - (1 + D)
    i = torch.arange(W, device=dev)
    q = s["q"][(off[:, None] + i).clamp(max=s["q"].shape[0] - 1)].float()
    q = q.view(B, W, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, W * G, d)
    S = torch.matmul(q * d ** -0.5, K.permute(0, 2, 3, 1))
    see = (pos <= (T[:, None] + i)[:, :, None]) & (i <= D[:, None])[:, :, None]
    S.view(B, Hkv, W, G, n).masked_fill_(~see[:, None, :, None, :], -math.inf)
    r = torch.arange(s["q"].shape[0], device=dev)
    seq = torch.searchsorted(off, r, right=True) - 1
    at = (seq, r - off[seq])
    lse = torch.logsumexp(S, -1).view(B, Hkv, W, G).permute(0, 2, 1, 3)[at].reshape(-1, c["Hq"])
    return S, lse, at


def _attn_plain(s):
    c = s["c"]
    S, lse, at = _scores(s)
    pos = torch.arange(S.shape[-1], device=S.device)
    V = _values(_cached(s, s["vc"], pos), _cached(s, s["scales"], pos)[:, :, :, 1], s["hs"][1])
    W, G = s["max_D"] + 1, c["Hq"] // c["Hkv"]
    S.sub_(S.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    O = torch.matmul(S, V.permute(0, 2, 1, 3)) / S.sum(-1, keepdim=True)
    O = O.view(c["B"], c["Hkv"], W, G, c["d"]).permute(0, 2, 1, 3, 4)[at]
    s["out"].copy_(O.reshape(-1, c["Hq"], c["d"]))
    s["lse"].copy_(lse)
    return dict(out=s["out"], lse=s["lse"])


def _mass_plain(s):
    c = s["c"]
    S, lse, at = _scores(s)
    lse = lse if s["lse"] is None else s["lse"]
    W, G = s["max_D"] + 1, c["Hq"] // c["Hkv"]
    full = torch.zeros(c["B"], W, c["Hq"], device=S.device)
    full[at] = lse
    full = full.view(c["B"], W, c["Hkv"], G).permute(0, 2, 1, 3)[..., None]
    w = torch.exp(S.view(c["B"], c["Hkv"], W, G, -1) - full)
    count = torch.arange(W, device=S.device) < s["accepted"][:, None]
    s["mass"].add_(w.mul_(count[:, None, :, None, None]).sum((2, 3)))
    return s["mass"]


def _evict_plain(s):
    c, dev = s["c"], s["mass"].device
    bs, B, Hkv = c["block"], c["B"], c["Hkv"]
    s["mass"].copy_(s["mass0"])
    row, m = s["row"].long(), s["new_len"].long()
    n = s["lens"].long()[row]
    mass = s["mass"][row]
    j = torch.arange(mass.shape[2], device=dev)
    key = torch.where((j < s["first"][:, None]) | (j >= (n - c["last"])[:, None]), math.inf, 0.0)[:, None] + mass
    key = torch.where((j < n[:, None])[:, None], key, -math.inf)
    rank = torch.empty_like(key, dtype=torch.long)
    rank.scatter_(2, key.sort(dim=-1, descending=True, stable=True).indices, j.expand_as(key).contiguous())
    keep = (rank < m[:, None, None]) & (m < n)[:, None, None] | (j < n[:, None])[:, None] & (m >= n)[:, None, None]
    new = torch.where(keep, keep.cumsum(-1) - 1, mass.shape[2])
    k = s["kept"].shape[2]
    src = torch.zeros(B, Hkv, mass.shape[2] + 1, dtype=torch.long, device=dev)
    src.scatter_(2, new, j.expand_as(new).contiguous())
    src = src[:, :, :k]
    live = (torch.arange(k, device=dev) < m[:, None])[:, None].expand(B, Hkv, k)
    s["kept"].copy_(torch.where(live, src, s["kept"].long()))
    moved = torch.zeros_like(mass)
    moved[:, :, :k] = torch.where(live, mass.gather(2, src), 0.0)
    s["mass"][row] = torch.where((j < n[:, None])[:, None], moved, mass)
    i, h, to = live.nonzero(as_tuple=True)
    frm = src[i, h, to]
    page = lambda p: s["table"][row[i], p // bs].long()  # noqa: E731
    kv = s["kv"].view(torch.uint8) if c["kv"] == "e4m3" else s["kv"]
    kv[:, page(to), to % bs, h] = kv[:, page(frm), frm % bs, h]
    return dict(kept=s["kept"], mass=s["mass"], kv=s["kv"])


_own = dict(write=_write_own, read=_read_own, attn=_attn_own, mass=_mass_own, evict=_evict_own)
_plain = dict(write=_write_plain, read=_read_plain, attn=_attn_plain, mass=_mass_plain, evict=_evict_plain)


# ---------------------------------------------------------------------- in 64 bits, apart

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("write", "read"):
        return _rows_exact(s)
    return _evict_exact(s) if case["op"] == "evict" else _attention_exact(s)


def _nearest(x, grid):
    """The entry of `grid` (ascending, its even places the even codes) nearest to each x >= 0."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    down, up = x - grid[lo], grid[hi] - x
    return grid[torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)]


def _round_exact(x, hs):
    """x [n, d] of one head in 64 bits to the values that its 4-bit form stands for."""
    dev = x.device
    e4m3 = torch.arange(127, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn).double()
    b = x.view(x.shape[0], -1, 16)
    c = _nearest(b.abs().amax(-1) / (6 * hs), e4m3) * hs
    y = torch.where(c[..., None] > 0, b.abs() / c[..., None], torch.zeros_like(b))
    e = _nearest(y, torch.tensor(_E2M1, dtype=torch.float64, device=dev))
    return (e * b.sign() * c[..., None]).view_as(x)


def _decode_exact(codes, u, hs):
    """codes [n, d / 2] of one head with block scales u [n, d / 16] to values."""
    lut = torch.tensor(_E2M1 + [-x for x in _E2M1], dtype=torch.float64, device=codes.device)
    e = torch.stack([lut[(codes % 16).long()], lut[(codes // 16).long()]], 2).view(codes.shape[0], -1, 16)
    return (e * u.view(torch.float8_e4m3fn).double()[:, :, None] * hs.double()).view(codes.shape[0], -1)


def _rows_exact(s):
    c, bs = s["c"], s["c"]["block"]
    table = s["table"].cpu()
    k, v, r = [], [], 0
    for b, n in enumerate(_counts(c)):
        p = torch.arange(c["start"], c["start"] + n)
        page, at = table[b, p // bs].long().to(s["kc"].device), (p % bs).to(s["kc"].device)
        for i, out in enumerate((k, v)):
            heads = []
            for h in range(c["Hkv"]):
                hs = s["hs"][i, h].double()
                if c["op"] == "write":
                    heads.append(_round_exact((s["k"], s["v"])[i][r:r + n, h].double(), hs))
                else:
                    heads.append(_decode_exact((s["kc"], s["vc"])[i][page, at, h], s["scales"][page, at, h, i], hs))
            out.append(torch.stack(heads, 1))
        r += n
    return dict(k=torch.cat(k), v=torch.cat(v))


def _key_rows(s, b, n, which):
    """K (which 0) or V (1) of the first n positions of sequence b in 64 bits, [Hkv, n, d]."""
    bs = s["c"]["block"]
    pages = s["table"][b, :_ceil(n, bs)].long()
    x = (s["kc"], s.get("vc"))[which][pages].flatten(0, 1)[:n]
    if s["scales"] is None:
        x = x.double().transpose(0, 1)
        return x if s["hs"] is None else x * s["hs"][0].double()[:, None, None]
    u = s["scales"][pages].flatten(0, 1)[:n, :, which]
    return torch.stack([_decode_exact(x[:, h].contiguous(), u[:, h].contiguous(), s["hs"][which, h])
                        for h in range(s["c"]["Hkv"])])


def _attention_exact(s):
    c = s["c"]
    T, D = _lens(c)
    A = _accepted(c) if c["op"] == "mass" else None
    Hkv, G, d = c["Hkv"], c["Hq"] // c["Hkv"], c["d"]
    out, lse, mass, r = [], [], s["mass"].double() if A else None, 0
    for b in range(c["B"]):
        w, n = 1 + D[b], T[b] + 1 + D[b]
        K = _key_rows(s, b, n, 0)
        Q = s["q"][r:r + w].double().view(w, Hkv, G, d).permute(1, 0, 2, 3).reshape(Hkv, w * G, d)
        S = (Q @ K.transpose(1, 2) / math.sqrt(d)).view(Hkv, w, G, n)
        late = torch.arange(n, device=S.device) > T[b] + torch.arange(w, device=S.device)[:, None]
        S = S.masked_fill(late[None, :, None, :], -math.inf)
        L = S.logsumexp(-1, keepdim=True)
        if A:
            L = L if s["lse"] is None else s["lse"][r:r + w].double().view(w, Hkv, G).permute(1, 0, 2)[..., None]
            mass[b, :, :n] += (S - L).exp()[:, :A[b]].sum((1, 2))
        else:
            O = (S - L).exp().view(Hkv, w * G, n) @ _key_rows(s, b, n, 1)
            out.append(O.view(Hkv, w, G, d).permute(1, 0, 2, 3).reshape(w, c["Hq"], d))
            lse.append(L[..., 0].permute(1, 0, 2).reshape(w, c["Hq"]))
        r += w
    return mass if A else dict(out=torch.cat(out), lse=torch.cat(lse))


def _evict_exact(s):
    c, bs = s["c"], s["c"]["block"]
    mass, kept, table = s["mass"].cpu(), s["kept"].cpu(), s["table"].cpu()
    kv = s["kv"].double()
    for i, (r, m) in enumerate(zip(s["row"].tolist(), s["new_len"].tolist())):
        n = _evict_lens(c)[r]
        for h in range(c["Hkv"]):
            w = mass[r, h].tolist()
            sure = set(range(n)) if m >= n else set(range(c["first"])) | set(range(n - c["last"], n))
            rest = sorted((j for j in range(n) if j not in sure), key=lambda j: (-w[j], j))
            src = torch.tensor(sorted(sure | set(rest[:m - len(sure)])))
            kept[i, h, :m] = src.int()
            mass[r, h, :m] = mass[r, h, src]
            mass[r, h, m:n] = 0
            to = torch.arange(m)
            kv[:, table[r, to // bs].long(), to % bs, h] = kv[:, table[r, src // bs].long(), src % bs, h]
    dev = s["mass"].device
    return dict(kept=kept.to(dev), mass=mass.double().to(dev), kv=kv)
