"""The measured calls of the paged-cache operators: verify attention over a shared prefix,
and forking, extending, trimming and compacting the pages of a cache.

``own`` False computes every operator in plain torch operations in 32 bits; ``own`` True
calls the library. ``exact`` computes the same outputs in 64 bits, sequence by sequence.
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
        # two samples of one short prompt on a small model: launch latency is all there is
        dict(name="attn two samples", op="attn", B=2, groups=1, Hq=4, Hkv=1, d=64, D=3, prefix=256,
             own_len=64, block=16, kv="bf16"),
        # a serving batch under one system prompt, ragged drafts and conversations
        dict(name="attn system prompt", op="attn", B=64, groups=1, Hq=32, Hkv=8, d=128, D=8,
             prefix=8192, own_len=1024, block=16, kv="bf16"),
        # sampled completions of two long documents, 8-bit cache, full draft windows
        dict(name="attn documents e4m3", op="attn", B=32, groups=2, Hq=64, Hkv=8, d=128, D=15,
             prefix=32768, own_len=2048, block=16, kv="e4m3"),
        # several agents' batches, each under its own prompt, long private histories
        dict(name="attn agents", op="attn", B=128, groups=4, Hq=32, Hkv=4, d=128, D=7,
             prefix=16385, own_len=4096, block=32, kv="bf16"),
        # a prompt is forked for a few samples
        dict(name="fork samples", op="fork", parents=2, children=3, len=1000, block=16, part=False),
        # a wide tree search forks long contexts, each child up to its own branching point
        dict(name="fork tree", op="fork", parents=32, children=31, len=32768, block=16, part=True),
        # the next window of a small batch: samples of one prompt part from their shared page
        dict(name="extend window", op="extend", rows=8, family=4, len=1001, window=4, block=16,
             Hkv=8, d=128, pools=2),
        # the same for a large batch of forked samples, eight pools (four layers' K and V)
        dict(name="extend forked batch", op="extend", rows=256, family=8, len=2056, window=9, block=16,
             Hkv=4, d=128, pools=8),
        # rejected drafts are rolled back after a step: a page or none for each sequence
        dict(name="trim rejected drafts", op="trim", rows=64, family=1, len=4096, drop=16, block=16),
        # half of a large batch of samples has finished
        dict(name="trim finished", op="trim", rows=1024, family=8, len=16000, drop=16000, block=16),
        # a small pool, half of it free in scattered pages
        dict(name="compact small pool", op="compact", blocks=512, live=0.5, rows=16, block=16, Hkv=8, d=64,
             pools=2),
        # a large pool before it is handed back in part
        dict(name="compact large pool", op="compact", blocks=12288, live=0.6, rows=256, block=16, Hkv=8,
             d=128, pools=2),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "fork", "extend", "trim", "compact"])
    block = rng.choice([8, 16, 32, 64, 128])
    if op == "attn":
        while True:
            B = _log(rng, 1, 128)
            Hkv = rng.choice([1, 2, 4, 8])
            c = dict(op=op, B=B, groups=_log(rng, 1, min(B, 8)), Hq=Hkv * rng.choice([1, 2, 4, 7, 8]), Hkv=Hkv,
                     d=rng.choice([64, 128, 128]), D=rng.choice([0, 1, 3, 5, 8, 15]),
                     prefix=_log(rng, 16, 32768), own_len=_log(rng, 1, 4096), block=block,
                     kv=rng.choice(["bf16", "bf16", "e4m3"]))
            w = work(c)
            if w["flops"] < 5e11 and w["bytes"] < 2e9:
                return c
    if op == "fork":
        return dict(op=op, parents=_log(rng, 1, 32), children=_log(rng, 1, 31), len=_log(rng, 1, 32768),
                    block=block, part=rng.random() < 0.5)
    if op == "extend":
        family = _log(rng, 1, 8)
        return dict(op=op, rows=family * _log(rng, 1, 32), family=family, len=_log(rng, 1, 2056),
                    window=rng.randint(1, 16), block=rng.choice([8, 16, 32]), Hkv=rng.choice([1, 2, 4]),
                    d=rng.choice([64, 128]), pools=2 * rng.randint(1, 4))
    if op == "trim":
        family = _log(rng, 1, 8)
        n = _log(rng, 1, 16000)
        return dict(op=op, rows=family * _log(rng, 1, 128), family=family, len=n, drop=_log(rng, 1, n),
                    block=block)
    blocks = _log(rng, 64, 4096)
    return dict(op=op, blocks=blocks, live=round(rng.uniform(0.1, 0.95), 2), rows=_log(rng, 1, 256), block=16,
                Hkv=rng.choice([2, 4, 8]), d=rng.choice([64, 128]), pools=2 * rng.randint(1, 2))


# -------------------------------------------------------------- what a case's sizes are

def _attn_shape(c):
    """(group starts, prefix lengths, T, D) of a case, as lists."""
    B, NG = c["B"], c["groups"]
    gb = [B * n // NG for n in range(NG + 1)]
    P = [max(1, c["prefix"] - 37 * n * (c["prefix"] > 64 * NG)) for n in range(NG)]
    T = _spread(B, 0, c["own_len"])
    for n in range(NG):
        for b in range(gb[n], gb[n + 1]):
            T[b] += P[n]
    D = [c["D"]] * B if c["D"] in (3, 7, 15) else _spread(B, 0, c["D"])
    return gb, P, T, D


def _fork_len(c):
    n = c["parents"] * c["children"]
    return _spread(n, max(1, c["len"] // 2), c["len"]) if c["part"] else [c["len"]] * n


def _trim_len(c):
    """What each row keeps: under a drop of its whole length every other row goes wholly."""
    n = c["rows"]
    if c["drop"] == c["len"]:
        return [0 if i % 2 else c["len"] for i in range(n)]
    return [c["len"] - k for k in _spread(n, 0, c["drop"])]


def _cows(c):
    """Rows of an extend case that part from a shared page: all of a family but the last."""
    return c["rows"] // c["family"] * (c["family"] - 1) if c["len"] % c["block"] else 0


def work(c):
    bs = c["block"]
    if c["op"] == "attn":
        gb, P, T, D = _attn_shape(c)
        es = 1 if c["kv"] == "e4m3" else 2
        rows = sum(D) + c["B"]
        keys = sum(P)
        flops = 0
        for n in range(c["groups"]):
            for b in range(gb[n], gb[n + 1]):
                keys += T[b] + 1 + D[b] - P[n]
                flops += sum(T[b] + i + 1 for i in range(1 + D[b])) * 4 * c["Hq"] * c["d"]
        return {"bytes": 4 * rows * c["Hq"] * c["d"] + 2 * es * keys * c["Hkv"] * c["d"], "flops": flops}
    if c["op"] == "fork":
        pages = [_ceil(n, bs) for n in _fork_len(c)]
        # parents' entries and their counts once, the children's entries written
        uniq = c["parents"] * _ceil(c["len"], bs)
        return {"bytes": 4 * (3 * uniq + sum(pages)), "flops": 0}
    if c["op"] == "extend":
        per = c["len"] % bs
        new = c["rows"] * (_ceil(c["len"] + c["window"], bs) - _ceil(c["len"], bs)) + _cows(c)
        moved = _cows(c) * per * c["Hkv"] * c["d"] * 2 * c["pools"]
        return {"bytes": 2 * moved + 8 * new + 16 * c["rows"] + 4 * _extend_blocks(c), "flops": 0}
    if c["op"] == "trim":
        dropped = sum(_ceil(c["len"], bs) - _ceil(k, bs) for k in _trim_len(c))
        return {"bytes": 16 * dropped + 16 * c["rows"], "flops": 0}
    L = int(c["blocks"] * c["live"])
    moves = L * (1 - c["live"])  # live pages lie evenly: this share of them is above the L-th
    page = bs * c["Hkv"] * c["d"] * 2 * c["pools"]
    return {"bytes": 2 * moves * page + 8 * L + 12 * c["blocks"], "flops": 0}


def _extend_blocks(c):
    bs = c["block"]
    return c["rows"] // c["family"] * _ceil(c["len"], bs) + c["rows"] * (2 + _ceil(c["window"], bs)) + 7


# ------------------------------------------------------------------------------ inputs

def _control(device, ref, lens, table):
    """Reference counts, cached lengths and block table in one buffer: a first state and
    the working copy that a pass changes."""
    n, R, S = ref.numel(), lens.numel(), table.shape[1]
    a, b = _ceil(n, 4) * 4, _ceil(R, 4) * 4
    ctl = torch.zeros(a + b + _ceil(R * S + 1, 4) * 4, dtype=torch.int32, device=device)

    def views(t):
        return dict(ref=t[:n], lens=t[a:a + R], table=t[a + b:a + b + R * S].view(R, S), flat=t[a + b:])

    v = views(ctl)
    v["ref"].copy_(ref)
    v["lens"].copy_(lens)
    v["table"].copy_(table)
    now = ctl.clone()
    return dict(first=ctl, now=now, **views(now))


def _families(gen, dev, rows, family, length, bs, extra):
    """A pool in which each `family` rows share all pages of `length` positions, pages
    placed at random; extra free pages beside them."""
    nb = _ceil(length, bs)
    fams = rows // family
    total = fams * nb + extra
    stride = nb + 4
    ids = torch.randperm(total, generator=gen, device=dev)[:fams * nb].to(torch.int32).view(fams, nb)
    table = torch.full((rows, stride), -1, dtype=torch.int32, device=dev)
    table[:, :nb] = ids.repeat_interleave(family, 0)
    ref = torch.zeros(total, dtype=torch.int32, device=dev)
    ref[ids.flatten().long()] = family
    return ref, torch.full((rows,), length, dtype=torch.int32, device=dev), table


def _pool(gen, dev, pools, blocks, bs, Hkv, d):
    kv = torch.empty(pools, blocks, bs, Hkv, d, dtype=torch.bfloat16, device=dev)
    return kv.normal_(generator=gen)


def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    c, bs = case, case["block"]
    s = dict(c=c)
    if c["op"] == "attn":
        s.update(_attn_inputs(c, gen, dev))
    elif c["op"] == "fork":
        n = c["parents"] * c["children"]
        R, nb = c["parents"] + n, _ceil(c["len"], bs)
        ref, lens, table = _families(gen, dev, c["parents"], 1, c["len"], bs, 3)
        full = torch.full((R, table.shape[1]), -1, dtype=torch.int32, device=dev)
        # rows in use and empty rows lie mixed, as in a running server
        order = torch.randperm(R, generator=gen, device=dev).to(torch.int32)
        par, child = order[:c["parents"]], order[c["parents"]:].contiguous()
        full[par.long()] = table
        alllens = torch.zeros(R, dtype=torch.int32, device=dev)
        alllens[par.long()] = lens
        s["ctl"] = _control(dev, ref, alllens, full)
        s["parents"] = par.repeat_interleave(c["children"]).contiguous()
        s["children"] = child
        s["fork_len"] = _i32(_fork_len(c), dev)
        s["rows"] = R
    elif c["op"] in ("extend", "trim"):
        extra = 3 if c["op"] == "trim" else _extend_blocks(c) - c["rows"] // c["family"] * _ceil(c["len"], bs)
        ref, lens, table = _families(gen, dev, c["rows"], c["family"], c["len"], bs, extra)
        s["ctl"] = _control(dev, ref, lens, table)
        s["row"] = torch.randperm(c["rows"], generator=gen, device=dev).to(torch.int32)
        if c["op"] == "trim":
            s["new_len"] = _i32(_trim_len(c), dev)
        else:
            s["new_len"] = torch.full_like(s["row"], c["len"] + c["window"])
            s["kv"] = _pool(gen, dev, c["pools"], ref.numel(), bs, c["Hkv"], c["d"])
    else:
        nb = c["blocks"]
        L = max(1, int(nb * c["live"]))
        ids = torch.randperm(nb, generator=gen, device=dev)[:L].to(torch.int32)
        R = min(c["rows"], L)
        ends = torch.tensor([L * (i + 1) // R for i in range(R)], device=dev)
        begin = torch.cat([ends.new_zeros(1), ends[:-1]])
        stride = int(_ceil(L, R)) + 1
        j = torch.arange(stride, device=dev)
        have = j < (ends - begin)[:, None]
        table = torch.where(have, ids[(begin[:, None] + j).clamp(max=L - 1)], -1).to(torch.int32)
        ref = torch.zeros(nb, dtype=torch.int32, device=dev)
        ref[ids.long()] = 1
        s["ctl"] = _control(dev, ref, ((ends - begin) * bs - 3).to(torch.int32), table)
        s["kv"] = _pool(gen, dev, c["pools"], nb, bs, c["Hkv"], c["d"])
        s["remap"] = torch.empty(nb, dtype=torch.int32, device=dev)
        s["num_live"] = torch.empty(1, dtype=torch.int32, device=dev)
    if "kv" in s:
        s["pools"] = list(s["kv"].unbind(0))
    if own:
        _own_plan(s)
    return s


def _attn_inputs(c, gen, dev):
    gb, P, T, D = _attn_shape(c)
    bs, B, NG = c["block"], c["B"], c["groups"]
    stride = max(_ceil(T[b] + 1 + D[b], bs) for b in range(B))
    # pages: a group's whole prefix pages once, every other page per sequence
    table = torch.full((B, stride), -1, dtype=torch.int64)
    used = 0
    for n in range(NG):
        whole = P[n] // bs
        first = torch.arange(used, used + whole)
        used += whole
        for b in range(gb[n], gb[n + 1]):
            k = _ceil(T[b] + 1 + D[b], bs)
            table[b, :whole] = first
            table[b, whole:k] = torch.arange(used, used + k - whole)
            used += k - whole
    blocks = used + 5
    place = torch.randperm(blocks, generator=gen, device=dev).to(torch.int32)
    table = table.to(dev)
    table = torch.where(table >= 0, place[table.clamp(min=0)], -1).to(torch.int32)
    q = torch.empty(sum(D) + B, c["Hq"], c["d"], dtype=torch.bfloat16, device=dev).normal_(generator=gen)
    k = torch.empty(blocks, bs, c["Hkv"], c["d"], dtype=torch.bfloat16, device=dev).normal_(generator=gen)
    v = torch.empty_like(k).normal_(generator=gen)
    # the shared partial page of a group: every sequence's own copy holds the same positions
    for n in range(NG):
        whole, rest = P[n] // bs, P[n] % bs
        if rest:
            pages = table[gb[n]:gb[n + 1], whole].long()
            k[pages, :rest] = k[pages[0], :rest].clone()
            v[pages, :rest] = v[pages[0], :rest].clone()
    scale = None
    if c["kv"] == "e4m3":
        scale = torch.stack([x.abs().amax(dim=(0, 1, 3)).float() / 448 for x in (k, v)]).contiguous()
        k, v = ((x.float() / scale[i][:, None]).to(torch.float8_e4m3fn) for i, x in enumerate((k, v)))
    return dict(q=q, k=k, v=v, scale=scale, table=table, T=_i32(T, dev), D=_i32(D, dev), gb=_i32(gb, dev),
                P=_i32(P, dev), max_T=max(T), max_D=max(D), max_P=max(P),
                max_own=max(T[b] + 1 + D[b] - P[n] for n in range(NG) for b in range(gb[n], gb[n + 1])),
                max_rows=max(sum(D[gb[n]:gb[n + 1]]) + gb[n + 1] - gb[n] for n in range(NG)),
                out=torch.zeros_like(q))


def _own_plan(s):
    """The workspace, and the handle of the pools, that a program of the library's keeps
    between its calls."""
    import speculative_decoding_verification_gqa_gb300 as sv
    c = s["c"]
    if "kv" in s:
        s["data"] = sv.page_pools(s["pools"])
    if c["op"] == "attn":
        desc = sv.api.attn_desc(s["q"], s["k"].view(-1, c["Hkv"], c["d"]), c["B"], s["max_D"], s["max_T"])
        n = sv.shared_workspace_bytes(desc, c["groups"])
    else:
        n = sv.pages_workspace_bytes(s["ctl"]["ref"].numel(), s["ctl"]["lens"].numel())
    s["ws"] = sv.new_workspace(n, s["q"].device if c["op"] == "attn" else s["ctl"]["ref"].device)


# ---------------------------------------------------------------------------- the passes

def run(s):
    c = s["c"]
    if c["op"] == "attn":
        return _attn_own(s) if own else _attn_plain(s)
    t = s["ctl"]
    t["now"].copy_(t["first"])  # a pass changes the pool's state in place: start from the same one
    if c["op"] == "fork":
        (_fork_own if own else _fork_plain)(s, t)
        return dict(ref=t["ref"], lens=t["lens"], table=t["table"])
    if c["op"] == "trim":
        (_trim_own if own else _trim_plain)(s, t)
        return dict(ref=t["ref"], lens=t["lens"], table=t["table"])
    if c["op"] == "extend":
        (_extend_own if own else _extend_plain)(s, t)
        return dict(ref=t["ref"], lens=t["lens"], table=t["table"], pools=s["kv"])
    (_compact_own if own else _compact_plain)(s, t)
    return dict(ref=t["ref"], table=t["table"], pools=s["kv"], remap=s["remap"], num_live=s["num_live"])


def _attn_own(s):
    import speculative_decoding_verification_gqa_gb300 as sv
    return sv.spec_verify_attn_shared(
        s["q"], s["k"], s["v"], s["table"], s["T"], s["D"], s["gb"], s["P"], max_draft_len=s["max_D"],
        max_seq_len=s["max_T"], kv_scale=s["scale"], out=s["out"], workspace=s["ws"])


def _fork_own(s, t):
    import speculative_decoding_verification_gqa_gb300 as sv
    sv.spec_pages_fork(t["ref"], t["table"], t["lens"], s["parents"], s["children"], fork_len=s["fork_len"],
                       block_size=s["c"]["block"], workspace=s["ws"])


def _extend_own(s, t):
    import speculative_decoding_verification_gqa_gb300 as sv
    sv.spec_pages_extend(t["ref"], t["table"], t["lens"], s["row"], s["new_len"], pools=s["data"],
                         block_size=s["c"]["block"], workspace=s["ws"])


def _trim_own(s, t):
    import speculative_decoding_verification_gqa_gb300 as sv
    sv.spec_pages_trim(t["ref"], t["table"], t["lens"], s["row"], s["new_len"], block_size=s["c"]["block"],
                       workspace=s["ws"])


def _compact_own(s, t):
    import speculative_decoding_verification_gqa_gb300 as sv
    sv.spec_pages_compact(t["ref"], t["table"], t["lens"], pools=s["data"], remap=s["remap"],
                          num_live=s["num_live"], block_size=s["c"]["block"], workspace=s["ws"])


def _rows(pages, table, pos, bs):
    """Cache rows of positions `pos` [n, m] through the table rows `table` [n, stride]."""
    at = table.gather(1, (pos // bs).clamp(max=table.shape[1] - 1)).long().clamp(min=0)
    return pages.reshape(-1, *pages.shape[2:])[at * bs + pos % bs].float()


def _attn_plain(s):
    c = s["c"]
    bs, Hkv, d, G = c["block"], c["Hkv"], c["d"], c["Hq"] // c["Hkv"]
    q, dev = s["q"], s["q"].device
    T, D, gb, P = (s[n].long() for n in ("T", "D", "gb", "P"))
    B, NG, rows = c["B"], c["groups"], q.shape[0]
    W = 1 + D
    q_off = W.cumsum(0) - W
    group = torch.searchsorted(gb, torch.arange(B, device=dev), right=True) - 1
    seq = torch.searchsorted(q_off, torch.arange(rows, device=dev), right=True) - 1
    i_row = torch.arange(rows, device=dev) - q_off[seq]
    qf = q.float().view(rows, Hkv, G, d) * (1 / math.sqrt(d))
    ks, vs = (s["scale"][0][:, None], s["scale"][1][:, None]) if s["scale"] is not None else (1.0, 1.0)

    def part(qp, K, V, see):
        """(m, l, O) of query rows qp [n, Hkv, r, d] over K, V [n, k, Hkv, d], see [n, 1, r, k]"""
        S = torch.matmul(qp, (K * ks).permute(0, 2, 3, 1))
        S.masked_fill_(~see, -math.inf)
        m = S.amax(-1, keepdim=True)
        S.sub_(m.clamp(min=-3e38)).exp_()
        return m, S.sum(-1, keepdim=True), torch.matmul(S, (V * vs).permute(0, 2, 1, 3))

    # the prefix: every row of a group at once
    r0 = q_off[gb[:-1]]
    r1 = torch.cat([q_off, W.sum()[None]])[gb[1:]]
    Rm = s["max_rows"]
    ridx = (r0[:, None] + torch.arange(Rm, device=dev)).clamp(max=rows - 1)
    pos = torch.arange(s["max_P"], device=dev).expand(NG, -1)
    first = s["table"][gb[:-1]]
    see = (pos < P[:, None])[:, None, None, :]
    qp = qf[ridx].permute(0, 2, 1, 3, 4).reshape(NG, Hkv, Rm * G, d)
    shared = part(qp, _rows(s["k"], first, pos, bs), _rows(s["v"], first, pos, bs), see)
    at = (group[seq], torch.arange(rows, device=dev) - r0[group[seq]])
    m1, l1, o1 = (x.view(NG, Hkv, Rm, G, -1).permute(0, 2, 1, 3, 4)[at] for x in shared)
    # the sequences' own positions
    Wm = s["max_D"] + 1
    ridx = (q_off[:, None] + torch.arange(Wm, device=dev)).clamp(max=rows - 1)
    j = torch.arange(s["max_own"], device=dev)
    pos = P[group][:, None] + j
    last = T[:, None] + torch.arange(Wm, device=dev)
    see = (pos[:, None, :] <= last[:, :, None])[:, None, :, None, :].expand(B, 1, Wm, G, -1).reshape(B, 1, Wm * G, -1)
    keep = (pos <= (T + D)[:, None])[:, :, None, None]
    qp = qf[ridx].permute(0, 2, 1, 3, 4).reshape(B, Hkv, Wm * G, d)
    mine = part(qp, _rows(s["k"], s["table"], pos, bs) * keep, _rows(s["v"], s["table"], pos, bs) * keep, see)
    at = (seq, i_row)
    m2, l2, o2 = (x.view(B, Hkv, Wm, G, -1).permute(0, 2, 1, 3, 4)[at] for x in mine)
    m = torch.maximum(m1, m2)
    a1, a2 = (m1 - m).exp(), (m2 - m).exp()
    return ((a1 * o1 + a2 * o2) / (a1 * l1 + a2 * l2)).reshape(rows, c["Hq"], d).to(q.dtype)


def _fork_plain(s, t):
    bs = s["c"]["block"]
    par, child, n = s["parents"].long(), s["children"].long(), s["fork_len"]
    have = torch.arange(t["table"].shape[1], device=n.device) < ((n + bs - 1) // bs)[:, None]
    ent = t["table"][par]
    t["table"][child] = torch.where(have, ent, t["table"][child])
    t["ref"].scatter_add_(0, ent.clamp(min=0).flatten().long(), have.to(torch.int32).flatten())
    t["lens"][child] = n


def _trim_plain(s, t):
    bs = s["c"]["block"]
    row, new = s["row"].long(), s["new_len"]
    old = t["lens"][row]
    j = torch.arange(t["table"].shape[1], device=new.device)
    drop = (j >= ((new + bs - 1) // bs)[:, None]) & (j < ((old + bs - 1) // bs)[:, None])
    ent = t["table"][row]
    t["table"][row] = torch.where(drop, -1, ent)
    t["ref"].scatter_add_(0, ent.clamp(min=0).flatten().long(), -drop.to(torch.int32).flatten())
    t["lens"][row] = new


def _extend_plain(s, t):
    c, bs = s["c"], s["c"]["block"]
    row, new = s["row"].long(), s["new_len"].long()
    ref, stride = t["ref"], t["table"].shape[1]
    dev, n, nb = ref.device, row.numel(), ref.numel()
    old = t["lens"][row].long()
    i = torch.arange(n, device=dev)
    fill = old % bs
    part = (fill != 0) & (new > old)
    page = t["table"][row, (old - 1) // bs].long()
    count = torch.zeros(nb, dtype=torch.int32, device=dev).scatter_add_(0, page, part.to(torch.int32))
    last = torch.full((nb,), -1, device=dev).scatter_reduce_(0, page, torch.where(part, i, -1), "amax")
    cow = part & (ref[page] > 1) & ~((count[page] == ref[page]) & (last[page] == i))
    have = (old + bs - 1) // bs
    need = cow.long() + (new + bs - 1) // bs - have
    start = need.cumsum(0) - need
    # the free pages, lowest first
    free = ref == 0
    rank = torch.where(free, free.cumsum(0) - 1, nb)
    fresh = torch.zeros(nb + 1, dtype=torch.long, device=dev).scatter_(0, rank, torch.arange(nb, device=dev))
    k = torch.arange(2 + c["window"] // bs + 1, device=dev)
    take = k < need[:, None]
    got = fresh[(start[:, None] + k).clamp(max=nb)]
    cell = row[:, None] * stride + (have - cow.long())[:, None] + k
    dump = t["flat"].numel() - 1
    t["flat"].scatter_(0, torch.where(take, cell, dump).flatten(), got.to(torch.int32).flatten())
    ref.scatter_add_(0, page, -cow.to(torch.int32))
    ref.scatter_add_(0, torch.where(take, got, 0).flatten(), take.to(torch.int32).flatten())
    t["lens"][row] = s["new_len"]
    # the filled positions of a page that a row parts from
    dst = torch.where(cow, got[:, 0], page)
    move = (torch.arange(bs, device=dev) < fill[:, None]) & cow[:, None]
    kv = s["kv"]
    kv[:, dst] = torch.where(move[None, :, :, None, None], kv[:, page], kv[:, dst])


def _compact_plain(s, t):
    bs = s["c"]["block"]
    ref = t["ref"]
    nb, dev = ref.numel(), ref.device
    ids = torch.arange(nb, device=dev)
    live = ref > 0
    L = live.sum()
    src = (live & (ids >= L)).nonzero().flatten()
    dst = (~live & (ids < L)).nonzero().flatten()
    remap = torch.where(live, ids, -1)
    remap[src] = dst
    have = torch.arange(t["table"].shape[1], device=dev) < ((t["lens"] + bs - 1) // bs)[:, None]
    t["table"].copy_(torch.where(have, remap[t["table"].clamp(min=0).long()], t["table"].long()))
    ref[dst] = ref[src]
    ref[src] = 0
    s["kv"][:, dst] = s["kv"][:, src]
    s["remap"].copy_(remap)
    s["num_live"].copy_(L)


# ---------------------------------------------------------------------- in 64 bits, apart

def exact(case, seed):
    s = prepare(case, seed)
    return _attn_exact(s) if case["op"] == "attn" else _pages_exact(s)


def _attn_exact(s):
    c = s["c"]
    gb, P, T, D = _attn_shape(c)
    bs, Hkv, G, d = c["block"], c["Hkv"], c["Hq"] // c["Hkv"], c["d"]
    table = s["table"].cpu().tolist()
    out, r = [], 0
    for b in range(c["B"]):
        n, w = T[b] + 1 + D[b], 1 + D[b]
        pages = torch.tensor(table[b][:_ceil(n, bs)], device=s["q"].device)
        K = s["k"][pages].double().flatten(0, 1)[:n].transpose(0, 1)
        V = s["v"][pages].double().flatten(0, 1)[:n].transpose(0, 1)
        if s["scale"] is not None:
            K, V = K * s["scale"][0].double()[:, None, None], V * s["scale"][1].double()[:, None, None]
        Q = s["q"][r:r + w].double().view(w, Hkv, G, d).transpose(0, 1).reshape(Hkv, w * G, d)
        S = Q @ K.transpose(1, 2) * d ** -0.5
        late = torch.arange(n, device=S.device)[None, :] > T[b] + torch.arange(w, device=S.device)[:, None]
        S = S.view(Hkv, w, G, n).masked_fill(late[None, :, None, :], -math.inf)
        O = torch.softmax(S, -1).view(Hkv, w * G, n) @ V
        out.append(O.view(Hkv, w, G, d).transpose(0, 1).reshape(w, c["Hq"], d))
        r += w
    return torch.cat(out)


def _pages_exact(s):
    """The page operators one row and one page after another, on the host."""
    c, bs, t = s["c"], s["c"]["block"], s["ctl"]
    dev = t["ref"].device
    ref, lens, table = t["ref"].tolist(), t["lens"].tolist(), t["table"].tolist()
    got, moves = {}, []
    if c["op"] == "fork":
        for p, ch, n in zip(s["parents"].tolist(), s["children"].tolist(), s["fork_len"].tolist()):
            for j in range(_ceil(n, bs)):
                table[ch][j] = table[p][j]
                ref[table[p][j]] += 1
            lens[ch] = n
    elif c["op"] == "trim":
        for r, n in zip(s["row"].tolist(), s["new_len"].tolist()):
            for j in range(_ceil(n, bs), _ceil(lens[r], bs)):
                ref[table[r][j]] -= 1
                table[r][j] = -1
            lens[r] = n
    elif c["op"] == "extend":
        free = iter([p for p in range(len(ref)) if ref[p] == 0])
        for r, n in zip(s["row"].tolist(), s["new_len"].tolist()):
            j = lens[r] // bs
            if lens[r] % bs and n > lens[r] and ref[table[r][j]] > 1:
                p = next(free)
                moves.append((table[r][j], p, lens[r] % bs))
                ref[table[r][j]] -= 1
                table[r][j] = p
                ref[p] = 1
            for j in range(_ceil(lens[r], bs), _ceil(n, bs)):
                table[r][j] = next(free)
                ref[table[r][j]] = 1
            lens[r] = n
    else:
        L = sum(1 for x in ref if x)
        holes = iter([p for p in range(L) if not ref[p]])
        remap = [p if ref[p] else -1 for p in range(len(ref))]
        for p in range(L, len(ref)):
            if ref[p]:
                h = next(holes)
                remap[p], ref[h], ref[p] = h, ref[p], 0
                moves.append((p, h, bs))
        for r in range(len(lens)):
            for j in range(_ceil(lens[r], bs)):
                table[r][j] = remap[table[r][j]]
        got.update(remap=_i32(remap, dev), num_live=_i32([L], dev))
    if "kv" in s:
        kv = s["kv"]
        if moves:
            src, dst, n = (torch.tensor(x, device=dev) for x in zip(*moves))
            part = (torch.arange(bs, device=dev) < n[:, None])[:, :, None, None]
            for p in s["pools"]:
                p[dst] = torch.where(part, p[src], p[dst])
        got["pools"] = kv.double()
    got.update(ref=_i32(ref, dev), table=_i32(table, dev))
    if c["op"] != "compact":
        got["lens"] = _i32(lens, dev)
    return got
