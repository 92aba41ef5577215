"""Accumulated attention weight and eviction by it on the GPU, against plain models in 64 bits,
and the operators of a 4-bit cache in a run together."""
import random

import pytest
import torch

import speculative_decoding_verification_gqa_gb300 as sv
from speculative_decoding_verification_gqa_gb300 import api

from gpu_util import ensure_built
from kv4_util import Cache, DEV, attention, block_table, evict, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def make_q(rows, Hq, d, seed):
    return torch.randn(rows, Hq, d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)


def mass_call(c, q, T, D, mass, n=None, lse=None, **kw):
    return sv.spec_attn_mass(q, c.k, c.table, i32(T), i32(D), mass, max_draft_len=kw.pop("max_draft", max(D)),
                             max_seq_len=max(T), kv_scale=c.hs, scales=c.scales, lse=lse,
                             row_count=None if n is None else i32(n), **kw)


def check_mass(kind, T, D, Hq, Hkv, d, bs, n=None, given=False, seed=0, scale=0.0):
    """A weight's relative error is its score's and its log-sum's: 2^-17 of scale * sum |q k|
    each (products exact, eight accumulating MMA steps, scaling), and 2^-19 for the exponent
    and the log-sum's own arithmetic; the sum over rows in fp32 adds 2^-16 (some hundred
    additions), the addition to mass 2^-23 of the total."""
    c = Cache(kind, [t + 1 + k for t, k in zip(T, D)], Hkv, d, bs, seed + 5)
    rows = sum(D) + len(D)
    q = make_q(rows + 1, Hq, d, seed)
    gen = torch.Generator().manual_seed(seed + 1)
    mass = torch.rand(len(T), Hkv, max(T) + 1 + max(D) + 5, generator=gen).to(DEV)
    before = mass.clone()
    G, off, refs = Hq // Hkv, 0, []
    lse = torch.full((rows + 1, Hq), 7.0, device=DEV)
    for b, (t, k) in enumerate(zip(T, D)):
        refs.append(attention(q[off:off + 1 + k], c.dense(b, t + 1 + k, 0), None, t, k, G, scale or d ** -0.5))
        lse[off:off + 1 + k] = refs[-1][1].float()
        off += 1 + k
    got = mass_call(c, q, T, D, mass, n, lse if given else None, softmax_scale=scale)
    assert got is mass
    for b, (t, k) in enumerate(zip(T, D)):
        P, L, _, size, _ = refs[b]
        m = 1 + k if n is None else n[b]
        add = P[:, :m].sum((1, 2))
        worst = float(size.max()) if m else 0.0
        tol = add * (2.5 * worst * 2 ** -17 + 2 ** -15 + float(L.abs().max()) * 2 ** -22) + mass[b].abs().amax() * 2 ** -23 + 1e-30
        err = (mass[b, :, :t + 1 + k].double() - before[b, :, :t + 1 + k].double() - add).abs()
        assert (err <= tol).all(), float((err / tol).max())
        assert torch.equal(mass[b, :, t + m:], before[b, :, t + m:])


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "kv4"])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("T,D,Hq,Hkv,d,bs,n", [
    ([0], [0], 1, 1, 64, 8, None),
    ([0, 30, 31, 255, 256, 257], [0, 1, 2, 0, 3, 1], 8, 2, 128, 16, None),
    ([100, 700, 5], [7, 3, 0], 14, 2, 64, 16, [3, 4, 1]),
    ([100, 700, 5], [7, 3, 0], 14, 2, 128, 16, [0, 4, 0]),    # sequences without a counted row
    ([500, 90], [31, 8], 32, 4, 128, 32, [32, 5]),            # 256 rows: two blocks of rows
    ([5000], [15], 64, 8, 128, 64, None),
    ([20000, 3], [2, 0], 4, 4, 64, 128, [1, 1]),
])
def test_mass(kind, given, T, D, Hq, Hkv, d, bs, n):
    check_mass(kind, T, D, Hq, Hkv, d, bs, n, given, seed=T[0])


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
def test_many_sequences(kind):
    rng = random.Random(1)
    T = [rng.choice([0, 3, 50, 300, 900]) for _ in range(300)]
    D = [rng.choice([0, 1, 4]) for _ in range(300)]
    check_mass(kind, T, D, 8, 2, 64, 16, [rng.randint(0, 1 + k) for k in D])


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("kind", ["e4m3", "kv4"])
def test_more_sequences_than_threads(kind, given):
    T = [(7 * b) % 41 for b in range(800)] + [1500]
    D = [b % 2 for b in range(801)]
    check_mass(kind, T, D, 4, 2, 64, 16, [b % (2 + k) if b % 5 else 0 for b, k in enumerate(D)], given)


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
def test_scores_that_rise(kind):
    """Scores that grow along the keys by some hundred binary digits in steps: a row's first
    maximum lies far below its last."""
    T, D, Hq, Hkv, d = [2000, 300], [3, 0], 8, 2, 64
    c = Cache(kind, [t + 1 + k for t, k in zip(T, D)], Hkv, d, 16, 9)
    q = make_q(5, Hq, d, 4).abs()
    for b, t in enumerate(T):
        n = t + 1 + D[b]
        at = c.rows(b, n).to(DEV)
        if kind == "bf16":
            k = c.k.view(-1, Hkv, d)
            k[at] = ((torch.arange(n, device=DEV) // 100)[:, None, None] * 2.0).expand(n, Hkv, d).to(torch.bfloat16)
        else:
            c.k.view(-1, Hkv, d // 2)[at] = 0x22  # ones
            s = c.scales.view(-1, Hkv, 2, d // 16)
            s[at, :, 0] = (8 + 4 * (torch.arange(n, device=DEV) // 100))[:, None, None].to(torch.uint8)
    if kind == "kv4":
        c.hs[0] = 40.0
    before = torch.zeros(2, Hkv, 2010, device=DEV)
    got = mass_call(c, q, T, D, before.clone())
    off = 0
    for b, (t, k) in enumerate(zip(T, D)):
        P, L, _, size, _ = attention(q[off:off + 1 + k], c.dense(b, t + 1 + k, 0), None, t, k, Hq // Hkv, d ** -0.5)
        off += 1 + k
        add = P.sum((1, 2))
        tol = add * (2.5 * float(size.max()) * 2 ** -17 + 2 ** -15 + float(L.abs().max()) * 2 ** -22) + 1e-30
        assert b == 1 or float(L.max()) > 139  # 2 x 100 binary digits above the first scores
        assert ((got[b, :, :t + 1 + k].double() - add).abs() <= tol).all()


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
@pytest.mark.parametrize("given", [False, True])
def test_a_row_without_numbers_reaches_its_own_keys_only(kind, given):
    """An infinity in the second row of a window: NaN for the keys that it sees, the others'
    weights after them."""
    T, D = [140], [3]
    c = Cache(kind, [144], 1, 64, 16, 3)
    q = make_q(4, 2, 64, 1)
    _, L, _, _, _ = attention(q, c.dense(0, 144, 0), None, 140, 3, 2, 64 ** -0.5)
    lse = L.float()
    q[1, 0, 5] = float("inf")
    lse[1, 0] = float("nan")
    got = mass_call(c, q, T, D, torch.zeros(1, 1, 144, device=DEV), lse=lse if given else None)[0, 0]
    assert torch.isnan(got[:142]).all()
    assert torch.isfinite(got[142:]).all() and (got[142:] > 0).all()


def test_no_row_counted():
    """Nothing is added, whatever the log-sums hold, by either form of the call."""
    T, D = [100, 3], [3, 0]
    c = Cache("kv4", [104, 4], 2, 64, 16, 3)
    q, mass = make_q(5, 4, 64, 1), torch.rand(2, 2, 104, device=DEV)
    was = mass.clone()
    mass_call(c, q, T, D, mass, n=[0, 0])
    mass_call(c, q, T, D, mass, n=[0, 0], lse=torch.full((5, 4), float("nan"), device=DEV))
    assert torch.equal(mass, was)


@pytest.mark.parametrize("given", [False, True])
def test_sharp_weights(given):
    """A scale at which all weight goes to a few keys."""
    check_mass("bf16", [600], [3], 8, 2, 128, 16, None, given, scale=2.0)


def test_weights_add_up():
    """Calls add; with every row counted a call's weights add up to the number of rows."""
    T, D, Hq, Hkv = [1000, 20], [3, 0], 8, 2
    c = Cache("kv4", [1004, 21], Hkv, 128, 16, 3)
    q = make_q(5, Hq, 128, 1)
    mass = torch.zeros(2, Hkv, 1010, device=DEV)
    for k in range(1, 4):
        mass_call(c, q, T, D, mass)
        total = mass.double().sum(-1) / (Hq // Hkv)
        want = k * torch.tensor([[4.0, 4.0], [1.0, 1.0]], device=DEV).double()
        assert ((total - want).abs() < 1e-4 * k).all()


def test_log_sums_of_the_attention_call():
    """The 4-bit attention call's log-sums give what the call's own do."""
    T, D, Hq, Hkv = [900, 33], [7, 2], 16, 2
    c = Cache("kv4", [908, 36], Hkv, 128, 16, 3)
    q = make_q(11, Hq, 128, 1)
    lse = torch.empty(11, Hq, device=DEV)
    sv.spec_verify_attn_kv4(q, c.k, c.v, c.scales, c.hs, c.table, i32(T), i32(D), max_draft_len=7, max_seq_len=900,
                            lse=lse)
    a, b = (mass_call(c, q, T, D, torch.zeros(2, Hkv, 908, device=DEV), lse=x) for x in (lse, None))
    assert torch.allclose(a, b, rtol=1e-4, atol=0)


def test_same_bits_again_and_captured():
    T, D, Hq, Hkv = [3000, 700], [7, 7], 32, 4
    c = Cache("bf16", [3008, 708], Hkv, 128, 16, 3)
    q = make_q(16, Hq, 128, 1)
    desc = sv.paged_attn_desc(q, c.k, 2, 7, 3000)
    ws = sv.new_workspace(sv.mass_workspace_bytes(desc))
    first = mass_call(c, q, T, D, torch.zeros(2, Hkv, 3008, device=DEV), workspace=ws)
    again = mass_call(c, q, T, D, torch.zeros(2, Hkv, 3008, device=DEV), workspace=ws)
    assert torch.equal(first, again)
    mass = torch.zeros(2, Hkv, 3008, device=DEV)
    Ti, Di = i32(T), i32(D)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_attn_mass(q, c.k, c.table, Ti, Di, mass, max_draft_len=7, max_seq_len=3000, workspace=ws)
    for _ in range(2):
        mass.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(mass, first)


@pytest.mark.parametrize("T,D,n", [([-1, 5], [0, 0], None), ([5, 101], [0, 0], None), ([5, 5], [0, 4], None),
                                   ([5, 5], [0, 0], [1, 2]), ([5, 5], [0, 0], [1, -1]), ([5, 95], [0, 1], None)])
@pytest.mark.parametrize("given", [False, True])
def test_lengths_out_of_range_leave_mass(T, D, n, given):
    """At most 100 positions and 3 drafts; rows of the table, and of mass, that hold 96."""
    c = Cache("bf16", [96, 96], 2, 64, 16, 1)
    c.table = c.table[:, :6].contiguous()
    q = make_q(8, 4, 64, 1)
    mass = torch.ones(2, 2, 96, device=DEV)
    desc = sv.paged_attn_desc(q, c.k, 2, 3, 100)
    ws = sv.new_workspace(sv.mass_workspace_bytes(desc))
    lse = torch.ones(8, 4, device=DEV) if given else None
    call = lambda T, D, n: sv.spec_attn_mass(  # noqa: E731
        q, c.k, c.table, i32(T), i32(D), mass, max_draft_len=3, max_seq_len=100, workspace=ws, lse=lse,
        row_count=None if n is None else i32(n))
    call(T, D, n)
    assert sv.workspace_status(ws, clear=True) == 8 and (mass == 1).all()
    call([92, 0], [3, 3], None)
    assert sv.workspace_status(ws) == 0 and not (mass == 1).all()


def test_mass_with_a_table_entry_outside_the_pool():
    c = Cache("kv4", [100], 2, 128, 16, 1)
    c.table[0, 2] = c.blocks + 3
    q = make_q(1, 8, 128, 1)
    desc = sv.paged_attn_desc(q, c.k, 1, 0, 99, kv4=True)
    ws = sv.new_workspace(sv.mass_workspace_bytes(desc))
    mass = mass_call(c, q, [99], [0], torch.zeros(1, 2, 100, device=DEV), workspace=ws)
    assert sv.workspace_status(ws) == 8 and torch.isfinite(mass).all()


# --------------------------------------------------------------------------- eviction

class Rows:
    """A table of rows with pools of random bytes and weights."""

    def __init__(self, lens, Hkv, bs, widths, seed, positions=None, ties=False):
        gen = torch.Generator().manual_seed(seed)
        table, blocks = block_table(lens, bs, gen)
        self.lens, self.bs, self.Hkv = lens, bs, Hkv
        self.table, self.host = table.to(DEV), table
        self.ref = torch.zeros(blocks, dtype=torch.int32, device=DEV)
        self.ref[self.table[self.table >= 0].long()] = 1
        self.len = i32(lens)
        self.pools = [torch.randint(0, 256, (blocks, bs, Hkv, w), generator=gen, dtype=torch.uint8).to(DEV)
                      for w in widths]
        self.mass = torch.randn(len(lens), Hkv, positions or max(lens) + 3, generator=gen)
        if ties:
            self.mass = (self.mass * 2).round() / 2
        self.mass = self.mass.to(DEV)

    def at(self, r, pos):
        return self.host[r, pos // self.bs].long() * self.bs + pos % self.bs

    def call(self, rows, new, first=None, last=0, kept=None, **kw):
        sv.spec_kv_evict(self.ref, self.table, self.len, None if rows is None else i32(rows), i32(new), self.mass,
                         block_size=self.bs, pools=self.pools, keep_first=None if first is None else i32(first),
                         keep_last=last, kept=kept, **kw)


def check_evict(s, rows, new, first=None, last=0):
    pools, mass = [p.clone() for p in s.pools], s.mass.cpu().clone()
    kept = torch.full((len(new), s.Hkv, max(new + [1]) + 2), -5, dtype=torch.int32, device=DEV)
    ws = sv.new_workspace(sv.evict_workspace_bytes(len(new), s.Hkv, s.mass.shape[2]))
    s.call(rows, new, first, last, kept, workspace=ws)
    assert sv.workspace_status(ws) == 0
    want_mass, got_kept = mass.clone(), kept.cpu()
    for i, m in enumerate(new):
        r = i if rows is None else rows[i]
        n = s.lens[r]
        for g in range(s.Hkv):
            src = torch.tensor(evict(mass[r, g].tolist()[:n], n, m, first[i] if first else 0, last), dtype=torch.long)
            assert got_kept[i, g, :m].tolist() == src.tolist()
            assert (got_kept[i, g, m:] == -5).all()
            want_mass[r, g, :m] = mass[r, g, src]
            if m < n:
                want_mass[r, g, m:n] = 0
            to, frm = s.at(r, torch.arange(m)).to(DEV), s.at(r, src).to(DEV)
            for p, old in zip(pools, [p.clone() for p in pools]):
                p.flatten(0, 1)[to, g] = old.flatten(0, 1)[frm, g]
    assert torch.equal(s.mass.cpu().view(torch.int32), want_mass.view(torch.int32))
    for got, want in zip(s.pools, pools):
        assert torch.equal(got, want)


@pytest.mark.parametrize("lens,rows,new,first,last,Hkv,bs,widths", [
    ([40], None, [16], None, 0, 2, 8, (128,)),
    ([1], None, [0], None, 0, 2, 8, (64,)),                       # everything
    ([100, 7, 333], [2, 0], [64, 100], [5, 0], 9, 2, 16, (256, 256)),  # a row within its budget
    ([1000, 999], None, [500, 998], [0, 17], 100, 4, 16, (64, 64, 16)),  # a 4-bit layer's pools
    ([1000, 4097], [1, 0], [1, 1], None, 1, 2, 32, (32, 32, 8)),  # d 64: scales of 8 bytes
    ([5000], None, [300], [300], 0, 2, 64, (48, 520)),            # the first only; odd widths
    ([9000, 20000, 64], [1, 2, 0], [4096, 40, 8191], [4, 4, 4], 32, 3, 128, (128, 16)),
    ([260] * 40, None, [200] * 40, None, 20, 2, 8, (64,)),
])
@pytest.mark.parametrize("ties", [False, True])
def test_evict(lens, rows, new, first, last, Hkv, bs, widths, ties):
    check_evict(Rows(lens, Hkv, bs, widths, len(lens) + Hkv, ties=ties), rows, new, first, last)


def test_pools_on_16_bytes_only():
    """Page data that begins on 16 bytes but not on 32."""
    s = Rows([700, 90], 2, 16, (128, 64), 5)
    for i, p in enumerate(s.pools):
        flat = torch.empty(p.numel() + 16, dtype=torch.uint8, device=DEV)
        s.pools[i] = flat[16:].view(p.shape).copy_(p)
        assert s.pools[i].data_ptr() % 32 == 16
    check_evict(s, None, [300, 60], [4, 4], 16)


def test_weights_of_every_kind():
    """Equal weights, zeros of either sign, infinities, subnormals and NaN (least of all)."""
    s = Rows([64, 64, 64], 2, 16, (64,), 3)
    s.mass[0] = 0.25
    s.mass[1, :, ::2] = 0.0
    s.mass[1, :, 1::2] = -0.0
    x = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), 1e-40, -1e-40, 3.4e38], device=DEV)
    s.mass[2, :, :64] = x.repeat(8)
    check_evict(s, None, [20, 33, 49], None, 0)


def test_evict_twice_and_with_other_sizes_on_one_workspace():
    s = Rows([500, 300], 2, 16, (64, 16), 4)
    ws = sv.new_workspace(sv.evict_workspace_bytes(2, 2, s.mass.shape[2]))
    for new in ([400, 300], [100, 250], [50, 0]):
        s.call(None, new, None, 3 if min(new) else 0, workspace=ws)
        s.lens = new
        s.len = i32(new)
    assert sv.workspace_status(ws) == 0
    s = Rows([40], 1, 8, (64,), 4)
    s.call(None, [30], workspace=ws)
    assert sv.workspace_status(ws) == 0


@pytest.mark.parametrize("why", ["row", "twice", "longer", "negative", "first", "last", "page", "shared", "shared part",
                                 "kept", "mass"])
def test_refused_on_the_device(why):
    """A call that fails a check changes neither pools nor mass, nor any other row's."""
    s = Rows([100, 100, 100], 2, 16, (64,), 6)
    rows, new, first, last, kept = [0, 1, 2], [50, 50, 50], [20, 20, 20], 4, None
    if why == "row":
        rows[1] = 3
    elif why == "twice":
        rows[2] = 0
    elif why == "longer":
        new[1] = 101
    elif why == "negative":
        new[1] = -1
    elif why == "first":
        first[2] = -1
    elif why == "last":
        first[2] = 47
    elif why == "page":
        s.table[1, 6] = s.ref.numel()
    elif why == "shared":
        s.ref[s.table[2, 2]] = 2
    elif why == "shared part":
        s.ref[s.table[2, 1]] = 2  # positions 16 .. 31: the first 20 stay, the rest would move
    elif why == "kept":
        kept = torch.zeros(3, 2, 49, dtype=torch.int32, device=DEV)
    elif why == "mass":
        s.mass = s.mass[:, :, :99].contiguous()
    pools, mass = [p.clone() for p in s.pools], s.mass.clone()
    ws = sv.new_workspace(sv.evict_workspace_bytes(3, 2, s.mass.shape[2]))
    s.call(rows, new, first, last, kept, workspace=ws)
    assert sv.workspace_status(ws, clear=True) == 8
    assert all(torch.equal(a, b) for a, b in zip(s.pools, pools)) and torch.equal(s.mass, mass)
    if why not in ("page", "mass"):
        s.ref.fill_(1)
        s.call([0, 1, 2], [50, 50, 50], [20, 20, 20], 4, workspace=ws)
        assert sv.workspace_status(ws) == 0


def test_a_pool_without_whole_16_bytes_a_position_is_refused():
    s = Rows([100], 1, 16, (520,), 6)
    with pytest.raises(sv.SpecVerifyError) as e:
        s.call(None, [50])
    assert e.value.status == 2


def test_shared_pages_before_the_kept_beginning():
    """Pages that other rows share are no obstacle where nothing moves within them."""
    s = Rows([100, 100], 2, 16, (64,), 6)
    s.ref[s.table[0, 0].long()] = 5
    s.ref[s.table[0, 6].long()] = 5  # past the budget: read only
    check_evict(s, None, [50, 100], [16, 0], 4)


def test_evict_captured_and_on_another_stream():
    ref = Rows([3000, 500], 4, 16, (64, 64, 16), 9)
    want = Rows([3000, 500], 4, 16, (64, 64, 16), 9)
    check_evict(want, None, [1000, 500], [4, 0], 32)
    for graph in (False, True):
        s = Rows([3000, 500], 4, 16, (64, 64, 16), 9)
        new, first = i32([1000, 500]), i32([4, 0])
        ws = sv.new_workspace(sv.evict_workspace_bytes(2, 4, s.mass.shape[2]))
        data = sv.page_pools(s.pools)
        args = (s.ref, s.table, s.len, None, new, s.mass)
        kw = dict(block_size=16, pools=data, keep_first=first, keep_last=32, workspace=ws)
        torch.cuda.synchronize()
        if graph:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                sv.spec_kv_evict(*args, **kw)
            assert torch.equal(s.mass, ref.mass)
            g.replay()
        else:
            side = torch.cuda.Stream()
            sv.spec_kv_evict(*args, **kw, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(s.mass, want.mass) and all(torch.equal(a, b) for a, b in zip(s.pools, want.pools))


def test_launch_failures():
    s = Rows([100], 2, 16, (64,), 6)
    c = Cache("bf16", [100], 2, 64, 16, 1)
    q = make_q(1, 4, 64, 1)
    for after in range(2):
        api.inject_launch_failure(after)
        with pytest.raises(sv.SpecVerifyError):
            s.call(None, [50])
    for after in range(2):
        api.inject_launch_failure(after)
        with pytest.raises(sv.SpecVerifyError):
            mass_call(c, q, [99], [0], torch.zeros(1, 2, 100, device=DEV))
    assert api.inject_launch_failure(-1) == -1


# --------------------------------------------------------------------- a run together

def test_a_decoding_loop_on_an_evicted_4_bit_cache():
    """Prompts are written, windows verified, accepted rows counted, rows cut to a budget and
    verified again: after every step the cache holds, for each head, what a plain list of the
    kept positions says, and attention and mass are those of the values there."""
    B, Hq, Hkv, d, bs, D, budget = 3, 8, 2, 128, 16, 3, 96
    rng, gen = random.Random(0), torch.Generator().manual_seed(0)
    nb, stride = 64, 16
    ref = torch.zeros(nb, dtype=torch.int32, device=DEV)
    table = torch.full((B, stride), -1, dtype=torch.int32, device=DEV)
    length = i32([0] * B)
    kc, vc = (torch.zeros(nb, bs, Hkv, d // 2, dtype=torch.uint8, device=DEV) for _ in "kv")
    sc = torch.full((nb, bs, Hkv, 2, d // 16), 0x7f, dtype=torch.uint8, device=DEV)
    hs = torch.full((2, Hkv), 0.0013, device=DEV)
    pools = sv.page_pools([kc, vc, sc])
    mass = torch.zeros(B, Hkv, stride * bs, device=DEV)
    kw = dict(block_size=bs, workspace=sv.new_workspace(sv.pages_workspace_bytes(nb, B)))
    ews = sv.new_workspace(sv.evict_workspace_bytes(B, Hkv, stride * bs))
    held = [[[] for _ in range(Hkv)] for _ in range(B)]  # (k row, v row) of each position
    lens = [0] * B

    def write(count):
        rows = sum(count)
        k, v = (torch.randn(rows, Hkv, d, generator=gen).to(torch.bfloat16).to(DEV) for _ in "kv")
        sv.spec_pages_extend(ref, table, length, None, i32([n + c for n, c in zip(lens, count)]), pools=pools, **kw)
        sv.spec_kv4_write(k, v, kc, vc, sc, hs, table, i32(lens), i32(count))
        rk, rv = sv.spec_kv4_read(kc, vc, sc, hs, table, i32(lens), i32(count), rows=rows)
        r = 0
        for b in range(B):
            for _ in range(count[b]):
                for g in range(Hkv):
                    held[b][g].append((rk[r, g].double(), rv[r, g].double()))
                r += 1

    def trim(new):
        sv.spec_pages_trim(ref, table, length, None, i32(new), **kw)
        lens[:] = new

    write([70, 41, 101])
    lens[:] = [70, 41, 101]
    for step in range(6):
        Ds = [D, rng.randint(0, D), D]
        write([1 + n for n in Ds])
        q = torch.randn(sum(Ds) + B, Hq, d, generator=gen).to(torch.bfloat16).to(DEV)
        lse = torch.zeros(q.shape[:2], device=DEV)
        out = sv.spec_verify_attn_kv4(q, kc, vc, sc, hs, table, i32(lens), i32(Ds), max_draft_len=D,
                                      max_seq_len=max(lens), lse=lse)
        accepted = [rng.randint(1, 1 + n) for n in Ds]
        was = mass.clone()
        sv.spec_attn_mass(q, kc, table, i32(lens), i32(Ds), mass, max_draft_len=D, max_seq_len=max(lens), kv_scale=hs,
                          scales=sc, lse=lse, row_count=i32(accepted))
        r = 0
        for b in range(B):
            n = lens[b] + 1 + Ds[b]
            K, V = (torch.stack([torch.stack([held[b][g][j][i] for g in range(Hkv)]) for j in range(n)])
                    for i in range(2))
            P, L, want, size, spread = attention(q[r:r + 1 + Ds[b]], K, V, lens[b], Ds[b], Hq // Hkv, d ** -0.5)
            # K and V here are the read values, rounded to bf16: 2^-8 of each on top
            slack = size[..., None] * 2 ** -7
            tol = want.abs() * 2 ** -8 + spread * (2 ** -8 + 2 ** -11 + slack)
            assert ((out[r:r + 1 + Ds[b]].double() - want).abs() <= tol).all()
            add = P[:, :accepted[b]].sum((1, 2))
            assert ((mass[b, :, :n] - was[b, :, :n]).double() - add).abs().max() <= float(size.max()) * 2 ** -7 * add.max() + 1e-5
            r += 1 + Ds[b]
        trim([n + a for n, a in zip(lens, accepted)])
        for b in range(B):
            for g in range(Hkv):
                del held[b][g][lens[b]:]
        new = [min(n, budget) for n in lens]
        kept = torch.zeros(B, Hkv, budget, dtype=torch.int32, device=DEV)
        sv.spec_kv_evict(ref, table, length, None, i32(new), mass, block_size=bs, pools=pools, keep_first=i32([4] * B),
                         keep_last=16, kept=kept, workspace=ews)
        trim(new)
        kept = kept.cpu()
        for b in range(B):
            for g in range(Hkv):
                held[b][g] = [held[b][g][j] for j in kept[b, g, :new[b]].tolist()]
        got = sv.spec_kv4_read(kc, vc, sc, hs, table, i32([0] * B), i32(lens), rows=sum(lens))
        r = 0
        for b in range(B):
            for g in range(Hkv):
                for i in range(2):
                    assert torch.equal(got[i][r:r + lens[b], g].double(), torch.stack([x[i] for x in held[b][g]]))
            r += lens[b]
        assert (mass[0, :, lens[0]:] == 0).all()
    assert max(lens) == budget and sv.workspace_status(kw["workspace"]) == 0 and sv.workspace_status(ews) == 0
    assert int(ref.sum()) == sum(-(-n // bs) for n in lens)


# ------------------------------------------------- state between a call's two launches

MASS_JOBS = [("bf16", [3000, 40, 700], [2, 0, 3], 32, 4), ("kv4", [900, 1700], [7, 3], 8, 2),
             ("e4m3", [5000], [1], 16, 2)]


def mass_jobs():
    """(q, cache, T, D, keyword arguments, zeros for mass, what it becomes) without log-sums: the
    second launch reads what the first left in the workspace."""
    jobs = []
    for k, (kind, T, D, Hq, Hkv) in enumerate(MASS_JOBS):
        c = Cache(kind, [t + 1 + n for t, n in zip(T, D)], Hkv, 128, 16, 50 + k)
        q = make_q(sum(D) + len(D), Hq, 128, k)
        mass = torch.zeros(len(T), Hkv, max(T) + 10, device=DEV)
        want = mass_call(c, q, T, D, mass.clone())
        kw = dict(max_draft_len=max(D), max_seq_len=max(T), kv_scale=c.hs, scales=c.scales)
        jobs.append((q, c, i32(T), i32(D), kw, mass, want))
    torch.cuda.synchronize()
    return jobs


def mass_workspace(jobs):
    n = max(sv.mass_workspace_bytes(sv.paged_attn_desc(q, c.k, len(T), kw["max_draft_len"], kw["max_seq_len"],
                                                       kv4=c.scales is not None)) for q, c, T, D, kw, _, _ in jobs)
    return sv.new_workspace(n)


def capture(call):
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    return g


def test_graphs_of_weights_on_one_workspace():
    """Replayed one after another, in any order and often."""
    jobs = mass_jobs()
    ws = mass_workspace(jobs)
    graphs = [capture(lambda: sv.spec_attn_mass(q, c.k, c.table, T, D, m, workspace=ws, **kw))
              for q, c, T, D, kw, m, _ in jobs]
    for order in ([0, 1, 2], [2, 0, 1, 1, 0, 2], [1, 0]):
        for k in order:
            jobs[k][5].zero_()
            graphs[k].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(jobs[k][5], jobs[k][6]) for k in order)
    assert sv.workspace_status(ws) == 0


def test_weights_of_calls_in_flight():
    """A stream and a workspace each."""
    jobs = mass_jobs()
    lanes = [(torch.cuda.Stream(), mass_workspace([j])) for j in jobs]
    out = [[j[5].clone() for _ in range(15)] for j in jobs]
    torch.cuda.synchronize()
    for i in range(15):
        for (q, c, T, D, kw, _, _), (s, ws), o in zip(jobs, lanes, out):
            sv.spec_attn_mass(q, c.k, c.table, T, D, o[i], workspace=ws, stream=s, **kw)
    torch.cuda.synchronize()
    for j, o in zip(jobs, out):
        assert all(torch.equal(m, j[6]) for m in o)
    assert all(sv.workspace_status(ws) == 0 for _, ws in lanes)


EVICT_JOBS = [dict(lens=[3000, 500], new=[1000, 500], last=32), dict(lens=[90, 2000, 700], new=[64, 9, 699], last=4)]


def evict_jobs():
    """(state, new_len, last, what to put back before a call, what it then becomes)."""
    jobs = []
    for k, j in enumerate(EVICT_JOBS):
        done = Rows(j["lens"], 4, 16, (64, 64, 16), 60 + k)
        check_evict(done, None, j["new"], None, j["last"])
        s = Rows(j["lens"], 4, 16, (64, 64, 16), 60 + k)
        jobs.append((s, i32(j["new"]), j["last"], [t.clone() for t in (*s.pools, s.mass)], (*done.pools, done.mass)))
    torch.cuda.synchronize()
    return jobs


def evict_again(job, ws, stream=None):
    """The state as it was, and the call, on one stream."""
    s, new, last, old, _ = job
    with torch.cuda.stream(stream or torch.cuda.current_stream()):
        for t, o in zip((*s.pools, s.mass), old):
            t.copy_(o)
        sv.spec_kv_evict(s.ref, s.table, s.len, None, new, s.mass, block_size=16, pools=sv.page_pools(s.pools),
                         keep_last=last, workspace=ws, stream=stream)


def evicted(job):
    return all(torch.equal(t, w) for t, w in zip((*job[0].pools, job[0].mass), job[4]))


def test_graphs_of_evictions_on_one_workspace():
    jobs = evict_jobs()
    ws = sv.new_workspace(max(sv.evict_workspace_bytes(len(j[1]), 4, j[0].mass.shape[2]) for j in jobs))
    graphs = [capture(lambda: evict_again(j, ws)) for j in jobs]
    for order in ([0, 1], [1, 0, 0, 1], [1]):
        for k in order:
            graphs[k].replay()
        torch.cuda.synchronize()
        assert all(evicted(jobs[k]) for k in order)
    assert sv.workspace_status(ws) == 0


def test_evictions_in_flight():
    """A stream and a workspace each."""
    jobs = evict_jobs()
    lanes = [(torch.cuda.Stream(), sv.new_workspace(sv.evict_workspace_bytes(len(j[1]), 4, j[0].mass.shape[2])))
             for j in jobs]
    torch.cuda.synchronize()
    for _ in range(15):
        for j, (s, ws) in zip(jobs, lanes):
            evict_again(j, ws, s)
    torch.cuda.synchronize()
    assert all(evicted(j) for j in jobs) and all(sv.workspace_status(ws) == 0 for _, ws in lanes)
