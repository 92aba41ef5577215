"""The 4-bit cache on the GPU: rows written and read, and verify attention over them, against
plain models in 64 bits."""
import math

import pytest
import torch

import speculative_decoding_verification_gqa_gb300 as sv
from speculative_decoding_verification_gqa_gb300 import api

from gpu_util import ensure_built
from kv4_util import (Cache, DEV, attention, block_table, e4m3_values, i32, quantise,
                      values)

pytestmark = pytest.mark.gpu

CANARY = 0xA5


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def empty_pages(blocks, bs, Hkv, d, fill=CANARY):
    return [torch.full((blocks, bs, Hkv, *s), fill, dtype=torch.uint8, device=DEV)
            for s in ((d // 2,), (d // 2,), (2, d // 16))]


def places(table, bs, start, count):
    """Flat cache rows of a call's packed rows."""
    out = []
    for b, (s, n) in enumerate(zip(start, count)):
        j = torch.arange(s, s + n)
        out.append(table[b, j // bs].long() * bs + j % bs)
    return torch.cat(out)


def written(pages, at):
    return [p.flatten(0, 1)[at.to(DEV)] for p in pages]


def expect_rows(k, v, hs):
    ks, vs = (quantise(x, hs[i][:, None]) for i, x in enumerate((k, v)))
    return ks[0], vs[0], torch.stack([ks[1], vs[1]], -2)


@pytest.mark.parametrize("d,Hkv,bs,start,count", [
    (128, 8, 16, [0, 5, 31], [3, 0, 17]),        # a short batch, an empty sequence
    (64, 1, 8, [7], [1]),                        # one row
    (128, 3, 32, [0] * 5, [1, 2, 1, 9, 4]),      # heads that are no power of two
    (64, 2, 16, [1000, 0], [33, 1]),
    (128, 8, 128, [0, 100, 4000], [700, 1, 1300]),   # four items a thread
    (128, 40, 16, [3, 0], [2, 5]),               # a row of more items than a CTA has threads
    (64, 5, 64, list(range(300)), [b % 3 for b in range(300)]),  # more sequences than threads
])
@pytest.mark.parametrize("strided", [False, True])
def test_written_rows_are_the_nearest_codes(d, Hkv, bs, start, count, strided):
    gen = torch.Generator().manual_seed(7 * d + Hkv)
    table, blocks = block_table([s + n for s, n in zip(start, count)], bs, gen)
    rows = sum(count)
    fused = torch.randn(rows + 2, 3, Hkv, d, generator=gen).to(torch.bfloat16).to(DEV)
    k, v = fused[:rows, 1], fused[:rows, 2]
    if not strided:
        k, v = k.contiguous(), v.contiguous()
    hs = ((torch.rand(2, Hkv, generator=gen) + 0.1) * 0.003).to(DEV)
    pages = empty_pages(blocks, bs, Hkv, d)
    before = [p.clone() for p in pages]
    ws = sv.new_workspace(sv.kv4_workspace_bytes(len(count)))
    args = (*pages, hs, table.to(DEV), i32(start), i32(count))
    sv.spec_kv4_write(k, v, *args, workspace=ws)
    at = places(table, bs, start, count)
    for got, want, full, old in zip(written(pages, at), expect_rows(k, v, hs), pages, before):
        assert torch.equal(got, want)
        full.flatten(0, 1)[at.to(DEV)] = CANARY  # every other byte as it was
        assert torch.equal(full, old)
    assert sv.workspace_status(ws) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_read_rows_are_the_values(d):
    Hkv, bs, start, count = 4, 16, [3, 0, 40], [20, 1, 900]
    c = Cache("kv4", [s + n for s, n in zip(start, count)], Hkv, d, bs, d)
    rows, tail = sum(count), 3
    outs = [torch.full((rows + tail, Hkv, d), 9.0, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    ws = sv.new_workspace(sv.kv4_workspace_bytes(3))
    args = (c.k, c.v, c.scales, c.hs, c.table, i32(start), i32(count))
    got = sv.spec_kv4_read(*args, k_out=outs[0], v_out=outs[1], workspace=ws)
    at = places(c.host_table, bs, start, count).to(DEV)
    for i, (x, codes) in enumerate(zip(got, (c.k, c.v))):
        want = values(codes.flatten(0, 1)[at], c.scales.flatten(0, 1)[at][:, :, i], c.hs[i][:, None])
        # two roundings: to fp32 (2^-24), to bf16 (2^-8)
        err = (x[:rows].double() - want).abs()
        assert (err <= want.abs() * (2 ** -8 + 2 ** -23)).all()
        assert (x[rows:] == 9.0).all()
    fresh = sv.spec_kv4_read(*args, rows=rows)
    assert torch.equal(fresh[0], got[0][:rows]) and torch.equal(fresh[1], got[1][:rows])
    assert sv.workspace_status(ws) == 0


@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("count", [3, 2000])
def test_rows_on_16_bytes_only(which, count):
    """Arrays and row strides that are multiples of 16 bytes but not of 32: the same as others."""
    Hkv, d, bs, pad = 3, 64, 16, 8  # rows of Hkv d + 8 elements
    gen = torch.Generator().manual_seed(count)
    table, blocks = block_table([count], bs, gen)
    x = [torch.randn(count, Hkv, d, generator=gen).to(torch.bfloat16).to(DEV) for _ in "kv"]
    hs = torch.full((2, Hkv), 0.002, device=DEV)
    args = (hs, table.to(DEV), i32([0]), i32([count]))
    want, got = (empty_pages(blocks, bs, Hkv, d, 0) for _ in range(2))
    odd = []
    for name, t in zip("kv", x):
        flat = torch.zeros(count * (Hkv * d + pad) + pad, dtype=torch.bfloat16, device=DEV)
        o = flat[pad:].view(count, Hkv * d + pad)[:, :Hkv * d].view(count, Hkv, d)
        o.copy_(t)
        odd.append(o if which in (name, "both") else t)
    sv.spec_kv4_write(*x, *want, *args)
    sv.spec_kv4_write(*odd, *got, *args)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [torch.full((count * Hkv * d + pad,), 9.0, dtype=torch.bfloat16, device=DEV)[pad:].view(count, Hkv, d)
            if which in (name, "both") else torch.zeros(count, Hkv, d, dtype=torch.bfloat16, device=DEV) for name in "kv"]
    assert which == "v" or outs[0].data_ptr() % 32 == 16
    sv.spec_kv4_read(*want, *args, k_out=outs[0], v_out=outs[1])
    assert all(torch.equal(a, b) for a, b in zip(outs, sv.spec_kv4_read(*want, *args, rows=count)))


def _near_middles(hs, gen):
    """bf16 blocks whose elements lie next to the middles of two codes, and whose largest lies
    next to the middle of two block scales."""
    grid = e4m3_values()
    top = (0.5 * (grid[1:] + grid[:-1]))[torch.randint(8, 120, (4096,), generator=gen)] * 6 * hs
    b = torch.zeros(4096, 16, dtype=torch.float64)
    b[:, 0] = top
    # the scale that this block gets decides its middles
    c = quantise(b.to(torch.bfloat16), torch.tensor([hs]))[1][:, 0].long()
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    pick = mids[torch.randint(0, 7, (4096, 15), generator=gen)]
    b[:, 1:] = pick * (grid[c] * hs)[:, None] * (torch.randint(0, 2, (4096, 15), generator=gen) * 2 - 1)
    return b.to(torch.bfloat16)


@pytest.mark.parametrize("hs", [1.0, 0.25, 2.0 ** -90, 2.0 ** 90, 1 / 3, 0.001171875, 0.7310585975646973])
def test_values_next_to_the_middle_of_two_codes(hs):
    """Quotients on a middle (scales that are powers of two: many) go to the even code, others
    where the real quotient goes."""
    hs = float(torch.tensor(hs, dtype=torch.float32))
    gen = torch.Generator().manual_seed(3)
    b = _near_middles(hs, gen)
    # the neighbours of each value too
    bits = b.view(torch.int16)
    x = torch.cat([b, (bits + 1).view(torch.bfloat16), (bits - 1).view(torch.bfloat16)])
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).view(-1, 1, 64).to(DEV)
    rows, bs = x.shape[0], 64
    nb = -(-rows // bs)
    pages = empty_pages(nb, bs, 1, 64)
    scale = torch.full((2, 1), hs, dtype=torch.float32, device=DEV)
    table = torch.arange(nb, dtype=torch.int32, device=DEV).view(1, -1)
    sv.spec_kv4_write(x, x, *pages, scale, table, i32([0]), i32([rows]))
    want = expect_rows(x, x, scale)
    at = torch.arange(rows)
    for got, w in zip(written(pages, at), want):
        assert torch.equal(got, w)


def test_special_blocks():
    """Zeros, blocks too small for a scale, too large for one, infinities and NaN."""
    x = torch.zeros(8, 2, 64, dtype=torch.float32)
    x[1] = 1e-6                      # max / (6 s) under half of the least E4M3 value: zeros
    x[2] = -3e38                     # saturates
    x[3, 0, 20] = math.inf
    x[3, 1, 63] = -math.inf
    x[4, 0, 0] = math.nan
    x[5, :, ::2] = 1.0
    x[6] = -(2.0 ** -9) * 3          # the least scale
    x[7] = -0.0
    x = x.to(torch.bfloat16).to(DEV)
    hs = torch.ones(2, 2, device=DEV)
    pages = empty_pages(1, 8, 2, 64)
    args = (*pages, hs, i32([[0]]), i32([0]), i32([8]))
    sv.spec_kv4_write(x, x, *args)
    for got, want in zip(written(pages, torch.arange(8)), expect_rows(x, x, hs)):
        assert torch.equal(got, want)
    k, v = sv.spec_kv4_read(*args, rows=8)
    assert torch.equal(k.isnan(), v.isnan())
    nan = torch.zeros(8, 2, 4, dtype=torch.bool, device=DEV)
    nan[3, 0, 1] = nan[3, 1, 3] = nan[4, 0, 0] = True
    assert torch.equal(k.isnan(), nan.repeat_interleave(16, -1))
    assert (k[2] == -6 * 448).all() and (k[1] == 0).all() and (k[0] == 0).all()


@pytest.mark.parametrize("start,count", [([-1, 0], [1, 1]), ([0, 0], [1, -1]), ([0, 30], [1, 3]),
                                         ([0, 0], [4, 5]), ([2 ** 31 - 1, 0], [2 ** 31 - 1, 0])])
@pytest.mark.parametrize("which", ["write", "read"])
def test_lengths_out_of_range_change_nothing(which, start, count):
    """8 packed rows, rows of the table that hold 32 positions."""
    pages = empty_pages(4, 16, 2, 64)
    before = [p.clone() for p in pages]
    ws = sv.new_workspace(sv.kv4_workspace_bytes(2))
    x = torch.ones(8, 2, 64, dtype=torch.bfloat16, device=DEV)
    out = [x.clone(), x.clone()]
    args = (*pages, torch.ones(2, 2, device=DEV), i32([[0, 1], [2, 3]]), i32(start), i32(count))
    if which == "write":
        sv.spec_kv4_write(x, x, *args, workspace=ws)
    else:
        sv.spec_kv4_read(*args, k_out=out[0], v_out=out[1], workspace=ws)
    assert sv.workspace_status(ws, clear=True) == 8
    assert all(torch.equal(p, b) for p, b in zip(pages, before)) and all((o == 1).all() for o in out)
    # the workspace serves the next call
    args = (*pages, torch.ones(2, 2, device=DEV), i32([[0, 1], [2, 3]]), i32([0, 0]), i32([4, 4]))
    sv.spec_kv4_write(x, x, *args, workspace=ws)
    assert sv.workspace_status(ws) == 0


def test_table_entries_outside_the_pool():
    """A row whose entry names no page is skipped (written) or reads as zeros, and reported."""
    pages = empty_pages(4, 8, 2, 64)
    ws = sv.new_workspace(sv.kv4_workspace_bytes(1))
    x = torch.full((24, 2, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    args = (*pages, torch.ones(2, 2, device=DEV), i32([[2, 4, -1]]), i32([0]), i32([24]))
    sv.spec_kv4_write(x, x, *args, workspace=ws)
    assert sv.workspace_status(ws, clear=True) == 8
    for i in (0, 1, 3):
        assert all((p[i] == CANARY).all() for p in pages)
    k, v = sv.spec_kv4_read(*args, k_out=x.clone(), v_out=x.clone(), workspace=ws)
    assert sv.workspace_status(ws) == 8
    assert (k[:8] == 3).all() and (k[8:] == 0).all() and (v[8:] == 0).all()


def test_a_pool_past_32_bit_offsets():
    """Codes of more than 2^32 bytes: the last page's rows are written, read and attended."""
    bs, Hkv, d = 64, 8, 128
    nb = 2 ** 32 // (bs * Hkv * d // 2) + 7
    k = torch.zeros(nb, bs, Hkv, d // 2, dtype=torch.uint8, device=DEV)
    v = torch.zeros_like(k)
    s = torch.zeros(nb, bs, Hkv, 2, d // 16, dtype=torch.uint8, device=DEV)
    hs = torch.full((2, Hkv), 0.001, device=DEV)
    x = torch.randn(70, Hkv, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    table, start, count = i32([[nb - 1, nb - 3]]), i32([0]), i32([70])
    sv.spec_kv4_write(x, x * 2, k, v, s, hs, table, start, count)
    got = sv.spec_kv4_read(k, v, s, hs, table, start, count, rows=70)
    at = places(table.cpu(), bs, [0], [70]).to(DEV)
    dense = [values(p.flatten(0, 1)[at], s.flatten(0, 1)[at][:, :, i], hs[i][:, None])
             for i, p in enumerate((k, v))]
    for g, w in zip(got, dense):
        assert ((g.double() - w).abs() <= w.abs() * (2 ** -8 + 2 ** -23)).all()
    q = torch.randn(1, 16, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    out = sv.spec_verify_attn_kv4(q, k, v, s, hs, table, i32([69]), i32([0]), max_draft_len=0,
                                  max_seq_len=69)
    mass = sv.spec_attn_mass(q, k, table, i32([69]), i32([0]), torch.zeros(1, Hkv, 70, device=DEV),
                             max_draft_len=0, max_seq_len=69, kv_scale=hs, scales=s)
    P, L, want, size, spread = attention(q, *dense, 69, 0, 2, d ** -0.5)
    check_out(out, None, want, L, size, spread)
    assert torch.allclose(mass[0].double(), P[:, 0].sum(1), rtol=1e-4, atol=1e-6)
    assert int(k.view(nb, -1).any(1).sum()) == 2


# ------------------------------------------------------------------------- attention

def bounds(want, size, spread):
    """Errors of out and lse. A score's: products are exact, eight accumulating steps of the
    MMA round (2^-21 of the terms' sum each at most), scaling and the exponent's argument two
    more: 2^-17 of scale * sum |q k| in all. A weight of relative error 2 e (its score's and its
    normaliser's) is rounded to 11 bits (2^-11) for P V; the parts are joined in fp32 (2^-20);
    the output is rounded to bf16 (2^-8)."""
    e = size * 2 ** -17 + 2 ** -20
    return want.abs() * 2 ** -8 + spread * (2 ** -11 + 2.5 * e[..., None]), e + 2 ** -19


def check_out(out, lse, want, L, size, spread):
    tol, tol_l = bounds(want, size, spread)
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all()
    worst = float((err / tol.clamp(min=1e-300)).max())
    assert (err <= tol).all(), "worst error over its bound: %.3g" % worst
    if lse is not None:
        tol_l = tol_l + L.abs() * 2 ** -22
        assert ((lse.double() - L).abs() <= tol_l).all()


@pytest.fixture(params=[1, 2], ids=["mma", "tcgen05"])
def kernel(request):
    """Both attention kernels, whatever the call's rows."""
    prev = sv.set_attn_kernel(request.param)
    yield request.param
    sv.set_attn_kernel(prev)


def run_attn(c, q, T, D, window=0, scale=0.0, max_seq=None, **kw):
    out = torch.full_like(q, 5.0)
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    ws = kw.pop("workspace", None)
    if ws is None:
        desc = sv.paged_attn_desc(q, c.k, len(T), max(D), max(T) if max_seq is None else max_seq, kv4=True)
        ws = sv.new_workspace(sv.verify_kv4_workspace_bytes(desc))
    sv.spec_verify_attn_kv4(q, c.k, c.v, c.scales, c.hs, c.table, i32(T), i32(D), max_draft_len=max(D),
                            max_seq_len=max(T) if max_seq is None else max_seq, out=out, lse=lse,
                            workspace=ws, sliding_window=window, softmax_scale=scale, **kw)
    return out, lse, ws


def make_q(rows, Hq, d, seed):
    return torch.randn(rows, Hq, d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)


def check_attn(T, D, Hq, Hkv, d, bs, window=0, scale=0.0, seed=0, tail=2):
    c = Cache("kv4", [t + 1 + n for t, n in zip(T, D)], Hkv, d, bs, seed + 11)
    rows = sum(D) + len(D)
    q = make_q(rows + tail, Hq, d, seed)
    out, lse, ws = run_attn(c, q, T, D, window, scale)
    r = 0
    for b, (t, n) in enumerate(zip(T, D)):
        K, V = (c.dense(b, t + 1 + n, i) for i in range(2))
        _, L, want, size, spread = attention(q[r:r + 1 + n], K, V, t, n, Hq // Hkv,
                                             scale or d ** -0.5, window)
        check_out(out[r:r + 1 + n], lse[r:r + 1 + n], want, L, size, spread)
        r += 1 + n
    assert (out[rows:] == 5).all() and (lse[rows:] == 5).all()
    assert sv.workspace_status(ws) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (14, 2), (8, 1), (32, 4)])
@pytest.mark.parametrize("T,D", [
    ([0], [0]),                          # one key
    ([0, 1, 30, 31, 32, 33], [0] * 6),   # chunk edges
    ([127, 128, 129], [1, 0, 3]),        # tile edges
    ([500, 3, 0, 257], [3, 7, 2, 0]),    # windows across edges
])
def test_small_batches(kernel, d, Hq, Hkv, T, D):
    check_attn(T, D, Hq, Hkv, d, 16)


@pytest.mark.parametrize("T,D,Hq,Hkv,d,bs", [
    ([4000, 1], [0, 0], 8, 1, 128, 8),
    ([9001], [0], 64, 8, 128, 64),           # a unit's keys over many CTAs
    ([700, 2000, 64], [31, 15, 0], 32, 8, 128, 16),   # 128 rows
    ([300, 90], [31, 20], 56, 8, 128, 32),   # 224 rows: two row tiles, the second not full
    ([1000], [255], 2, 1, 64, 16),           # the longest window
    ([40000], [2], 16, 4, 64, 128),
    ([100] * 70, [b % 4 for b in range(70)], 28, 4, 128, 16),
    ([513, 2, 1025], [7, 8, 3], 32, 4, 128, 1024),
])
def test_larger_batches(kernel, T, D, Hq, Hkv, d, bs):
    check_attn(T, D, Hq, Hkv, d, bs, seed=T[0])


@pytest.mark.parametrize("T,D,Hq,Hkv,d,bs", [
    ([b % 37 for b in range(599)] + [1900], [0] * 600, 4, 2, 64, 8),  # more sequences than threads, one split
    ([b % 37 for b in range(600)], [b % 3 for b in range(600)], 4, 2, 64, 8),    # short: pairs of heads
    ([9 * b for b in range(130)] + [1500], [2] * 131, 16, 4, 128, 32),           # long: pairs of heads
    ([2000 + 8 * b for b in range(8)], [0] * 8, 16, 8, 64, 16),   # seven parts a unit: a warp joins a row
    ([30, 1000, 16, 2000], [3, 2, 3, 1], 9, 3, 128, 16),          # heads that do not pair
    ([1023, 600, 1000], [0, 0, 0], 16, 2, 128, 16),               # at the longest of the short
])
def test_batches_of_every_layout(kernel, T, D, Hq, Hkv, d, bs):
    check_attn(T, D, Hq, Hkv, d, bs, seed=len(T))


def test_many_units_a_cta_again_and_again():
    """Six units a CTA of the tcgen05 kernel and full rows: the same bits every time, and right."""
    T, D, Hkv, G = [(311 * b) % 1101 for b in range(150)], [7 - b % 3 for b in range(150)], 6, 16
    prev = sv.set_attn_kernel(2)
    try:
        check_attn(T, D, G * Hkv, Hkv, 128, 64, seed=3)
        c = Cache("kv4", [t + 1 + n for t, n in zip(T, D)], Hkv, 128, 64, 14)
        q = make_q(sum(D) + len(D), G * Hkv, 128, 4)
        first = run_attn(c, q, T, D)
        for _ in range(40):
            again = run_attn(c, q, T, D, workspace=first[2])
            assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    finally:
        sv.set_attn_kernel(prev)


@pytest.mark.parametrize("B,T,G,D", [(1, 300, 8, 15), (70, 2000, 8, 3), (70, 2000, 8, 4), (3, 900, 16, 15)])
def test_the_kernel_the_rules_choose(B, T, G, D):
    check_attn([T - 7 * b for b in range(B)], [D] * B, 2 * G, 2, 64, 16)


@pytest.mark.parametrize("window", [1, 5, 32, 100, 129, 1000, 100000])
@pytest.mark.parametrize("D", [0, 3, 17])
def test_sliding_windows(kernel, window, D):
    check_attn([0, 70, 700], [D, D, D // 2], 8, 2, 128, 16, window=window)


@pytest.mark.parametrize("scale", [0.01, 1.0, 3.0])
def test_scales(kernel, scale):
    """3.0: scores of some hundreds, weights that are zero but for a few keys."""
    check_attn([333, 50], [2, 0], 8, 2, 128, 16, scale=scale)


def test_rising_scores_move_the_reference(kernel):
    """Keys in ascending order of score: the reference maximum moves all the way."""
    c = Cache("kv4", [3001], 1, 128, 16, 5)
    q = make_q(1, 4, 128, 9)
    rows = c.rows(0, 3001).to(DEV)
    flat = c.k.flatten(0, 1)
    flat[rows] = flat[rows][:1]  # one key's codes everywhere, its scales growing
    s = c.scales.flatten(0, 1)
    s[rows, :, 0] = (8 + torch.arange(3001, device=DEV) * 100 // 3001).to(torch.uint8)[:, None, None]
    for sign in (1, -1):
        x = (q.float() * sign).to(torch.bfloat16)
        out, lse, _ = run_attn(c, x, [3000], [0])
        _, L, want, size, spread = attention(x, c.dense(0, 3001, 0), c.dense(0, 3001, 1), 3000, 0, 4, 128 ** -0.5)
        check_out(out, lse, want, L, size, spread)


@pytest.mark.parametrize("big", [1e30, 1e-30, 3e38])
def test_queries_of_any_magnitude(kernel, big):
    """Rows of large and of tiny elements: the softmax scale takes the magnitude back."""
    c = Cache("kv4", [200], 2, 128, 16, 3)
    q = make_q(1, 8, 128, 4)
    x = (q.float() * (big / float(q.float().abs().max()))).to(torch.bfloat16)
    scale = 0.3 / big
    if scale < 1e-37:
        scale = 1e-37
    out, lse, _ = run_attn(c, x, [199], [0], scale=float(scale))
    f32 = float(torch.tensor(scale, dtype=torch.float32))
    _, L, want, size, spread = attention(x, c.dense(0, 200, 0), c.dense(0, 200, 1), 199, 0, 4, f32)
    check_out(out, lse, want, L, size, spread)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_query_row_with_an_infinity_is_nan_and_alone(kernel, bad):
    c = Cache("kv4", [300], 2, 128, 16, 3)
    q = make_q(1, 8, 128, 4)
    good, lse0, _ = run_attn(c, q, [299], [0])
    x = q.clone()
    x[0, 3, 7] = bad
    out, lse, _ = run_attn(c, x, [299], [0])
    assert out[0, 3].isnan().all() and lse[0, 3].isnan()
    others = [h for h in range(8) if h != 3]
    assert torch.equal(out[0, others], good[0, others]) and torch.equal(lse[0, others], lse0[0, others])


@pytest.mark.parametrize("D", [0, 7, 31])
def test_nan_rows_reach_their_head_only(kernel, D):
    """A NaN block of K at a position: the rows that see it; of V: all rows of the sequence and
    head may; other heads and sequences not."""
    T, Hkv, G = [400, 90], 2, 4
    c = Cache("kv4", [t + 1 + D for t in T], Hkv, 128, 16, 8)
    q = make_q(2 * (1 + D), Hkv * G, 128, 5)
    good, _, _ = run_attn(c, q, T, [D, D])
    at = c.rows(0, 401)[37]
    c.scales.flatten(0, 1)[at, 1, 0, 2] = 0x7f
    out, lse, _ = run_attn(c, q, T, [D, D])
    assert out[:1 + D, G:].isnan().all() and lse[:1 + D, G:].isnan().all()
    assert torch.equal(out[:1 + D, :G], good[:1 + D, :G]) and torch.equal(out[1 + D:], good[1 + D:])
    # at the last window position, that only the last row sees
    c = Cache("kv4", [t + 1 + D for t in T], Hkv, 128, 16, 8)
    at = c.rows(0, 401 + D)[400 + D]
    c.scales.flatten(0, 1)[at, 0, 0, 0] = 0x7f
    out, _, _ = run_attn(c, q, T, [D, D])
    assert out[D, :G].isnan().all()
    assert torch.equal(out[:D], good[:D]) and torch.equal(out[D, G:], good[D, G:])


def test_zero_head_scales(kernel):
    """A K scale of 0: even weights; a V scale of 0: zeros."""
    c = Cache("kv4", [100], 2, 128, 16, 3)
    c.hs[0, 0] = 0
    c.hs[1, 1] = 0
    q = make_q(1, 4, 128, 4)
    out, lse, _ = run_attn(c, q, [99], [0])
    V = c.dense(0, 100, 1)
    want = V[:, 0].mean(0).expand(2, -1)
    tol = want.abs() * 2 ** -8 + V[:, 0].abs().mean(0) * 2 ** -10
    assert ((out[0, :2].double() - want).abs() <= tol).all()
    assert (out[0, 2:] == 0).all()
    assert ((lse[0, :2].double() - math.log(100)).abs() < 1e-5).all()


@pytest.mark.parametrize("T,D", [([-1, 5], [0, 0]), ([5, 101], [0, 0]), ([5, 5], [0, 4]), ([5, 5], [0, -1]),
                                 ([5, 95], [0, 1])])
def test_lengths_out_of_range_leave_the_outputs(kernel, T, D):
    """At most 100 positions and 3 drafts; rows of the table that hold 96 positions."""
    c = Cache("kv4", [96, 96], 2, 64, 16, 1)
    table = c.table[:, :6].contiguous()
    q = make_q(8, 4, 64, 1)
    out, lse = torch.full_like(q, 5.0), torch.full((8, 4), 5.0, device=DEV)
    desc = sv.paged_attn_desc(q, c.k, 2, 3, 100, kv4=True)
    ws = sv.new_workspace(sv.verify_kv4_workspace_bytes(desc))
    call = lambda T, D: sv.spec_verify_attn_kv4(  # noqa: E731
        q, c.k, c.v, c.scales, c.hs, table, i32(T), i32(D), max_draft_len=3, max_seq_len=100, out=out, lse=lse,
        workspace=ws)
    call(T, D)
    assert sv.workspace_status(ws, clear=True) == 8
    assert (out == 5).all() and (lse == 5).all()
    call([92, 0], [3, 3])
    assert sv.workspace_status(ws) == 0 and torch.isfinite(out).all() and not (out == 5).all()


def test_attention_with_a_table_entry_outside_the_pool(kernel):
    c = Cache("kv4", [100, 40], 2, 128, 16, 1)
    c.table[0, 2] = c.blocks
    c.table[0, 4] = -7
    q = make_q(2, 8, 128, 1)
    out, lse, ws = run_attn(c, q, [99, 39], [0, 0])
    assert sv.workspace_status(ws) == 8
    assert torch.isfinite(out).all()
    _, L, want, size, spread = attention(q[1:], c.dense(1, 40, 0), c.dense(1, 40, 1), 39, 0, 4, 128 ** -0.5)
    check_out(out[1:], lse[1:], want, L, size, spread)


def test_empty_batch():
    c = Cache("kv4", [10], 1, 64, 16, 1)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    table = torch.empty(0, 3, dtype=torch.int32, device=DEV)
    out = sv.spec_verify_attn_kv4(q, c.k, c.v, c.scales, c.hs, table, none, none, max_draft_len=3, max_seq_len=9)
    assert out.shape == q.shape
    x = torch.empty(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    sv.spec_kv4_write(x, x, c.k, c.v, c.scales, c.hs, table, none, none)
    assert sv.spec_kv4_read(c.k, c.v, c.scales, c.hs, table, none, none, rows=0)[0].shape == (0, 1, 64)


@pytest.mark.parametrize("T,D,Hq", [([3000, 17], [0, 0], 8), ([2000, 900], [7, 3], 32)])
def test_same_bits_again_captured_and_on_another_stream(kernel, T, D, Hq):
    Hkv = 2
    c = Cache("kv4", [t + 1 + n for t, n in zip(T, D)], Hkv, 128, 16, 2)
    q = make_q(sum(D) + 2, Hq, 128, 3)
    out, lse, ws = run_attn(c, q, T, D)
    for _ in range(3):
        again = run_attn(c, q, T, D, workspace=ws)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2 = sv.spec_verify_attn_kv4(q, c.k, c.v, c.scales, c.hs, c.table, i32(T), i32(D), max_draft_len=max(D),
                                 max_seq_len=max(T), stream=side)
    side.synchronize()
    assert torch.equal(o2, out)
    Ti, Di = i32(T), i32(D)
    o3, l3 = torch.zeros_like(out), torch.zeros_like(lse)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        sv.spec_verify_attn_kv4(q, c.k, c.v, c.scales, c.hs, c.table, Ti, Di, max_draft_len=max(D),
                                max_seq_len=max(T), out=o3, lse=l3, workspace=ws)
    for _ in range(2):
        o3.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o3, out) and torch.equal(l3, lse)


def test_two_graphs_on_one_workspace(kernel):
    """Replayed one after another, in either order and often."""
    jobs, ws = [], sv.new_workspace(sv.verify_kv4_workspace_bytes(
        sv.paged_attn_desc(make_q(40, 8, 128, 0), torch.empty(999, 16, 2, 64, dtype=torch.uint8, device=DEV), 3, 15,
                           4000, kv4=True)))
    for k, (T, D) in enumerate((([3000, 40, 7], [2, 0, 3]), ([900, 1700], [15, 3]))):
        c = Cache("kv4", [t + 1 + n for t, n in zip(T, D)], 2, 128, 16, 30 + k)
        q = make_q(sum(D) + len(D), 8, 128, k)
        want = run_attn(c, q, T, D)[0]
        out, Ti, Di = torch.zeros_like(q), i32(T), i32(D)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sv.spec_verify_attn_kv4(q, c.k, c.v, c.scales, c.hs, c.table, Ti, Di, max_draft_len=max(D),
                                    max_seq_len=max(T), out=out, workspace=ws)
        jobs.append((g, out, want, c, q, Ti, Di))
    for order in ([0, 1, 0, 0, 1, 1], [1, 0]):
        for _, out, *_ in jobs:
            out.zero_()
        for k in order:
            jobs[k][0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(j[1], j[2]) for j in jobs)


def test_two_calls_in_flight(kernel):
    """Two streams, a workspace each."""
    jobs = []
    for k in range(2):
        T, D = [2000 + 500 * k, 300], [3, 0]
        c = Cache("kv4", [t + 1 + n for t, n in zip(T, D)], 2, 128, 16, 20 + k)
        q = make_q(5, 8, 128, k)
        out, _, ws = run_attn(c, q, T, D)
        jobs.append((c, q, i32(T), i32(D), max(T), out, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for k, (c, q, T, D, mt, _, ws, s) in enumerate(jobs):
            outs[k].append(sv.spec_verify_attn_kv4(q, c.k, c.v, c.scales, c.hs, c.table, T, D, max_draft_len=3,
                                                   max_seq_len=mt, workspace=ws, stream=s))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(o, jobs[k][5]) for o in outs[k])


def test_launch_failures_leave_the_workspace_usable(kernel):
    T, D = [900], [0]
    c = Cache("kv4", [901], 2, 128, 16, 2)
    q = make_q(1, 8, 128, 3)
    out, lse, ws = run_attn(c, q, T, D)
    for after in range(2):
        api.inject_launch_failure(after)
        with pytest.raises(sv.SpecVerifyError):
            run_attn(c, q, T, D, workspace=ws)
        again = run_attn(c, q, T, D, workspace=ws)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    assert api.inject_launch_failure(-1) == -1


@pytest.mark.parametrize("T,D", [([900, 5, 300], [7, 0, 3]), ([40], [1])])
def test_a_wait_that_runs_out_is_reported(T, D):
    """With a short limit and every CTA's first tile withheld the waits for it run out: the
    kernel returns well before the default limit of about 2 s, the workspace says so, and the
    next call is right."""
    import time
    prev = sv.set_attn_kernel(2)
    try:
        c = Cache("kv4", [t + 1 + n for t, n in zip(T, D)], 2, 128, 16, 2)
        q = make_q(sum(D) + len(D), 8, 128, 3)
        out, lse, ws = run_attn(c, q, T, D)
        torch.cuda.synchronize()
        assert api.inject_wait_timeout(100000) == 0
        t0 = time.perf_counter()
        run_attn(c, q, T, D, workspace=ws)
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 0.5
        assert sv.workspace_status(ws, clear=True) == 7  # SV_ERR_TIMEOUT
        assert api.inject_wait_timeout(0) == 0           # used once
        again = run_attn(c, q, T, D, workspace=ws)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
        assert sv.workspace_status(ws) == 0
    finally:
        api.inject_wait_timeout(0)
        sv.set_attn_kernel(prev)


def test_one_workspace_serves_both_kernels():
    """Calls of few rows and of many, and either kernel, one after another on one workspace."""
    jobs = [([700, 30], [0, 0]), ([600, 500], [15, 7]), ([40, 2], [1, 0])]
    c = Cache("kv4", [800, 600], 2, 128, 16, 2)
    ws = None
    desc = sv.paged_attn_desc(make_q(32, 16, 128, 0), c.k, 2, 31, 1000, kv4=True)
    ws = sv.new_workspace(sv.verify_kv4_workspace_bytes(desc))
    for which in (0, 2, 1, 0):
        prev = sv.set_attn_kernel(which)
        for T, D in jobs:
            q = make_q(sum(D) + 2, 16, 128, T[0])
            out, lse, _ = run_attn(c, q, T, D, workspace=ws)
            r = 0
            for b, (t, n) in enumerate(zip(T, D)):
                _, L, want, size, spread = attention(q[r:r + 1 + n], c.dense(b, t + 1 + n, 0), c.dense(b, t + 1 + n, 1),
                                                     t, n, 8, 128 ** -0.5)
                check_out(out[r:r + 1 + n], lse[r:r + 1 + n], want, L, size, spread)
                r += 1 + n
        sv.set_attn_kernel(prev)
    assert sv.workspace_status(ws) == 0


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("Hq,D", [(4, 0), (32, 7)])
def test_lengths_that_the_kernel_before_has_changed(kernel, captured, Hq, D):
    """spec_pages_trim sets the lengths directly before the call, whose few units are split over
    CTAs: both of its grids go by the new ones, every time."""
    Hkv, bs, full = 2, 16, [3000, 1500]
    c = Cache("kv4", [n + 1 + D for n in full], Hkv, 128, bs, 2)
    q = make_q(2 * (1 + D), Hq, 128, 3)
    cuts = [[2003, 77], [311, 1499], [2999, 1], [45, 1003]]
    want = [run_attn(c, q, n, [D, D], max_seq=3000)[:2] for n in cuts]
    ref0 = torch.ones(c.blocks, dtype=torch.int32, device=DEV)
    ref, table, length = ref0.clone(), c.table.clone(), i32([0, 0])
    grown, new, Di = i32([n + 1 + D for n in full]), [i32(n) for n in cuts], i32([D, D])
    pages_ws = sv.new_workspace(sv.pages_workspace_bytes(c.blocks, 2))
    ws = sv.new_workspace(sv.verify_kv4_workspace_bytes(sv.paged_attn_desc(q, c.k, 2, D, 3000, kv4=True)))
    outs = [(torch.full_like(q, 5.0), torch.full(q.shape[:2], 5.0, device=DEV)) for _ in cuts]

    def step(n, out, lse):
        ref.copy_(ref0)
        table.copy_(c.table)
        length.copy_(grown)
        sv.spec_pages_trim(ref, table, length, None, n, block_size=bs, workspace=pages_ws)
        # (the rows of the pages are all there still: the call goes by a table that was not cut)
        sv.spec_verify_attn_kv4(q, c.k, c.v, c.scales, c.hs, c.table, length, Di, max_draft_len=D, max_seq_len=3000,
                                out=out, lse=lse, workspace=ws)

    def run():
        for n, (out, lse) in zip(new, outs):
            step(n, out, lse)

    if captured:
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
    for _ in range(25):
        for out, lse in outs:
            out.fill_(5.0)
            lse.fill_(5.0)
        if captured:
            g.replay()
        else:
            run()
        for (out, lse), (o, l) in zip(outs, want):
            assert torch.equal(out, o) and torch.equal(lse, l)
    assert sv.workspace_status(ws) == 0 and sv.workspace_status(pages_ws) == 0


@pytest.mark.parametrize("count", [3, 3000])
def test_rows_that_the_kernel_before_has_made(count):
    """Two sequences read into one buffer, one after the other, and each written from it to
    another cache directly after: the rows of its own read, every time."""
    Hkv, d, bs = 4, 128, 16
    src = [Cache("kv4", [count], Hkv, d, bs, 40 + k) for k in range(2)]
    start, n = i32([0]), i32([count])
    ws = sv.new_workspace(sv.kv4_workspace_bytes(1))
    hs = torch.full((2, Hkv), 0.004, device=DEV)

    def move(k, buf, to):
        c = src[k]
        sv.spec_kv4_read(c.k, c.v, c.scales, c.hs, c.table, start, n, k_out=buf[0], v_out=buf[1], workspace=ws)
        sv.spec_kv4_write(*buf, *to, hs, c.table, start, n, workspace=ws)

    want, got = ([empty_pages(src[0].blocks, bs, Hkv, d) for _ in range(2)] for _ in range(2))
    for k in range(2):
        move(k, [torch.zeros(count, Hkv, d, dtype=torch.bfloat16, device=DEV) for _ in "kv"], want[k])
        torch.cuda.synchronize()
    buf = [torch.zeros(count, Hkv, d, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    assert buf[0].data_ptr() % 32 == 0
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        for _ in range(3):
            for k in range(2):
                move(k, buf, got[k])
    for _ in range(20):
        for p in got[0] + got[1]:
            p.fill_(CANARY)
        g.replay()
        for k in range(2):
            assert all(torch.equal(a, b) for a, b in zip(got[k], want[k]))
    assert sv.workspace_status(ws) == 0


@pytest.mark.parametrize("which", ["write", "read"])
@pytest.mark.parametrize("start,count", [([0, 0], [0, 0]), ([0, 0], [1, 0]), ([-1, 0], [0, -1])])
def test_a_call_without_rows_looks_at_nothing(which, start, count):
    """rows = 0: the lengths, whatever they are, are not read and not reported."""
    pages = empty_pages(4, 16, 2, 64)
    x = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    ws = sv.new_workspace(sv.kv4_workspace_bytes(2))
    args = (*pages, torch.ones(2, 2, device=DEV), i32([[0, 1], [2, 3]]), i32(start), i32(count))
    if which == "write":
        sv.spec_kv4_write(x, x, *args, workspace=ws)
    else:
        assert sv.spec_kv4_read(*args, rows=0, workspace=ws)[0].shape == (0, 2, 64)
    assert sv.workspace_status(ws) == 0 and all((p == CANARY).all() for p in pages)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("strided", [False, True])
def test_a_head_scale_of_zero(kernel, d, strided):
    """What the largest magnitude / (6 * 448) gives for a head of zeros: the head is written as
    zeros, whatever finite it holds, and is read, attended and weighted as such."""
    Hkv, G, bs, n = 3, 2, 16, 70
    gen = torch.Generator().manual_seed(d)
    fused = torch.randn(n, 3, Hkv, d, generator=gen).to(torch.bfloat16).to(DEV)
    fused[:, 0, 1] = 0  # K of head 1 is zeros, V of head 2 has no scale
    k, v = fused[:, 0], fused[:, 1]
    if not strided:
        k, v = k.contiguous(), v.contiguous()
    hs = torch.stack([t.float().abs().amax((0, 2)) for t in (k, v)]) / (6 * 448)
    hs[1, 2] = 0
    assert hs[0, 1] == 0
    table, blocks = block_table([n], bs, gen)
    pages = empty_pages(blocks, bs, Hkv, d)
    args = (*pages, hs, table.to(DEV), i32([0]), i32([n]))
    sv.spec_kv4_write(k, v, *args)
    kc, vc, sc = written(pages, places(table, bs, [0], [n]))
    zeroed = [k.clone(), v.clone()]
    zeroed[1][:, 2] = 0
    for got, want in zip((kc, vc, sc), expect_rows(*zeroed, torch.where(hs == 0, torch.ones_like(hs), hs))):
        assert torch.equal(got, want)
    rk, rv = sv.spec_kv4_read(*args, rows=n)
    assert (rk[:, 1] == 0).all() and (rv[:, 2] == 0).all() and rk.isfinite().all() and rv.isfinite().all()
    q = make_q(1, Hkv * G, d, 7)
    lse = torch.zeros(1, Hkv * G, device=DEV)
    out = sv.spec_verify_attn_kv4(q, *pages, hs, table.to(DEV), i32([n - 1]), i32([0]), max_draft_len=0,
                                  max_seq_len=n - 1, lse=lse)
    mass = sv.spec_attn_mass(q, pages[0], table.to(DEV), i32([n - 1]), i32([0]), torch.zeros(1, Hkv, n, device=DEV),
                             max_draft_len=0, max_seq_len=n - 1, kv_scale=hs, scales=pages[2], lse=lse)
    assert out.isfinite().all() and (out[0, 2 * G:] == 0).all()
    # ln n and even weights, to the arithmetic of the log-sum and the exponent (2^-19 and 2^-15)
    assert ((lse[0, G:2 * G] - math.log(n)).abs() <= 2 ** -17).all()
    assert ((mass[0, 1] * n - G).abs() <= G * 2 ** -14).all()
    k[3, 1, 5] = math.inf  # and what is not finite is NaN still
    sv.spec_kv4_write(k, v, *args)
    assert sv.spec_kv4_read(*args, rows=n)[0][3, 1, :16].isnan().all()


@pytest.mark.parametrize("d,D,which", [(64, 5, 1), (64, 7, 2), (128, 3, 1), (128, 5, 2)])
def test_the_rule_takes_the_kernel_that_measures_faster(d, D, which):
    """64 sequences of up to 4000 positions, 4 KV heads of 8 query heads: the bits are those of
    the kernel whose time beside the rule is the smaller."""
    B, Hkv, G = 64, 4, 8
    T = [4000 - 37 * b for b in range(B)]
    c = Cache("kv4", [t + 1 + D for t in T], Hkv, d, 16, d)
    q = make_q(B * (1 + D), G * Hkv, d, D)
    prev = sv.set_attn_kernel(0)
    try:
        got = run_attn(c, q, T, [D] * B)
        for k in (1, 2):
            sv.set_attn_kernel(k)
            out = run_attn(c, q, T, [D] * B)
            assert (torch.equal(out[0], got[0]) and torch.equal(out[1], got[1])) == (k == which)
    finally:
        sv.set_attn_kernel(prev)


@pytest.mark.parametrize("d,bs,window", [(64, 64, 0), (64, 8, 0), (128, 8, 0), (128, 16, 0), (128, 16, 150),
                                         (64, 16, 150), (128, 64, 150)])
def test_every_layout_with_many_units_a_cta_again_and_again(d, bs, window):
    """Boxes of a whole tile and of 8 rows, both head dimensions, units that begin at a window:
    the same bits every time, and right."""
    T, D, Hkv, G = [(311 * b) % 1101 for b in range(150)], [7 - b % 3 for b in range(150)], 6, 16
    prev = sv.set_attn_kernel(2)
    try:
        check_attn(T, D, G * Hkv, Hkv, d, bs, window=window, seed=3)
        c = Cache("kv4", [t + 1 + n for t, n in zip(T, D)], Hkv, d, bs, 14)
        q = make_q(sum(D) + len(D), G * Hkv, d, 4)
        first = run_attn(c, q, T, D, window=window)
        for _ in range(30):
            again = run_attn(c, q, T, D, window=window, workspace=first[2])
            assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    finally:
        sv.set_attn_kernel(prev)
