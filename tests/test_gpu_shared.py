"""GPU tests of spec_verify_attn_shared (groups of sequences with a common prefix, attended
once per group) against the fp64 oracle, with NaN in everything that must not be read."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_gqa_gb300 as sv

from gpu_util import bf16_to_f64, ensure_built
from shared_util import assert_within, inputs, pages, run, to_device

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[1, 2], ids=["mma", "tcgen05"])
def kernel(request):
    ensure_built()
    lib = sv.api.load_library()
    prev = lib.sv_set_attn_kernel(request.param)
    if prev < 0:
        pytest.skip("kernel not built")
    yield request.param
    lib.sv_set_attn_kernel(prev)


TWO = [(300, [(300, 3), (301, 0), (455, 7), (700, 2)]), (129, [(129, 1), (1000, 5)])]


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 64, 128, 512])
def test_two_groups_ragged(kernel, bs, d, kv):
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=d, kv=kv, seed=bs + d)
    assert_within(run(x, pages(x, gb, P, bs, seed=bs), gb, P), w, x)


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("P", [1, 7, 8, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000])
def test_prefix_lengths_around_tiles_and_pages(kernel, P, kv):
    """Own parts of no cached position (T = P), one, and more than a tile."""
    w, x, gb, p = inputs([(P, [(P, 0), (P + 1, 3), (P + 140, 1)])], Hq=4, Hkv=2, d=128, kv=kv, seed=P)
    assert_within(run(x, pages(x, gb, p, 16, seed=P), gb, p), w, x)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 1), (28, 4), (3, 3), (64, 8), (48, 1)])
def test_head_layouts(kernel, Hq, Hkv):
    w, x, gb, P = inputs([(200, [(210, 2), (200, 4), (300, 0)])], Hq=Hq, Hkv=Hkv, d=128, seed=Hq)
    assert_within(run(x, pages(x, gb, P, 16, seed=1), gb, P), w, x)


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("n,D", [(1, 0), (2, 31), (8, 15), (17, 7), (33, 3), (64, 4)])
def test_many_rows_of_a_group(kernel, n, D, kv):
    """Groups of under one to many 128-row tiles, whole and ragged."""
    seqs = [(257 + (5 * b) % 40, (D + b) % (D + 1)) for b in range(n)]
    w, x, gb, P = inputs([(257, seqs)], Hq=16, Hkv=2, d=128, kv=kv, seed=n)
    assert_within(run(x, pages(x, gb, P, 32, seed=2), gb, P), w, x)


def test_groups_without_prefix_without_sequences_and_of_one(kernel):
    groups = [(0, [(90, 2), (0, 0), (400, 1)]), (77, []), (500, [(640, 3)]), (0, []),
              (40, [(40, 0), (1500, 2)])]
    w, x, gb, P = inputs(groups, Hq=8, Hkv=2, d=128, seed=6)
    assert_within(run(x, pages(x, gb, P, 16, seed=3), gb, P), w, x)


def test_nothing_shared_is_the_paged_call(kernel):
    w, x, gb, P = inputs([(0, [(300, 3), (41, 0), (700, 2)])], Hq=8, Hkv=2, d=128, seed=8)
    pg = pages(x, gb, P, 16, seed=3)
    got = run(x, pg, gb, P)
    assert_within(got, w, x)


@pytest.mark.parametrize("junk", [-1, 1 << 30])
def test_entries_before_the_prefix_end_are_not_read(kernel, junk):
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=128, seed=9)
    ws = sv.new_workspace(1 << 27)
    assert_within(run(x, pages(x, gb, P, 16, seed=4, junk=junk), gb, P, workspace=ws), w, x)
    assert sv.workspace_status(ws) == 0


@pytest.mark.parametrize("scale", [0.0, 0.02, 1.5])
def test_softmax_scale(kernel, scale):
    import oracle
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=64, seed=10)
    got = bf16_to_f64(run(x, pages(x, gb, P, 16, seed=4), gb, P, softmax_scale=scale))
    ref = oracle.verify_attn(x["q"], x["k"], x["v"], x["seq_lens"], x["draft_len"], Hq=w.Hq,
                             Hkv=w.Hkv, d=w.d, scale=scale if scale else 64 ** -0.5)
    mag = oracle.verify_attn(x["q"], x["k"], x["v"] & 0x7FFF, x["seq_lens"], x["draft_len"], Hq=w.Hq,
                             Hkv=w.Hkv, d=w.d, scale=scale if scale else 64 ** -0.5)
    # the bound of assert_within; under a scale 12 times the default's the scores' rounding
    # changes a probability by 12 times as much: 12 * 2^-11 < 2^-7
    assert (np.abs(got - ref) <= np.abs(ref) * 2.0 ** -8 + mag * (2.0 ** -8 + 2.0 ** -6)).all()


def test_prefix_that_dominates_or_is_dominated(kernel):
    """Scores hundreds of units apart on the two sides of the border: the join neither
    overflows nor loses the larger part."""
    for sign in (1, -1):
        w, x, gb, P = inputs([(200, [(260, 3), (333, 1)])], Hq=4, Hkv=2, d=128, seed=11)
        off = np.cumsum([0] + [int(t + n + 1) for t, n in zip(x["seq_lens"], x["draft_len"])])
        k = bf16_to_f64(x["k"])
        for b in range(2):
            k[off[b]:off[b] + 200] *= 16.0 if sign > 0 else 1 / 16.0
            k[off[b] + 200:off[b + 1]] *= 1 / 16.0 if sign > 0 else 16.0
        x["k"] = (k.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
        assert np.array_equal(bf16_to_f64(x["k"]), k)  # powers of two: exact
        got = bf16_to_f64(run(x, pages(x, gb, P, 16, seed=4), gb, P))
        from shared_util import reference
        ref, mag = reference(w, x)
        # scores 16 times as large: their rounding counts 16 * 2^-11 = 2^-7 (both ways 2^-6)
        assert (np.abs(got - ref) <= np.abs(ref) * 2.0 ** -8 + mag * (2.0 ** -8 + 2.0 ** -6)).all()


def test_infinite_and_nan_queries_stay_in_their_rows(kernel):
    """A row of q that holds NaN or infinity spoils its own output only."""
    w, x, gb, P = inputs([(150, [(160, 1), (150, 2)])], Hq=4, Hkv=2, d=128, seed=12)
    pg = pages(x, gb, P, 16, seed=4)
    clean = run(x, pg, gb, P)
    x["q"][1, 2, 5] = 0x7F80
    x["q"][3, 0, 7] = 0x7FC0
    got = run(x, pg, gb, P)
    spoilt = np.zeros(got.shape[:2], dtype=bool)
    spoilt[1, 2] = spoilt[3, 0] = True
    assert np.array_equal(got[~spoilt], clean[~spoilt])


def test_rows_behind_the_batch_are_left(kernel):
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=128, seed=13)
    pg = pages(x, gb, P, 16, seed=4)
    n = x["q"].shape[0]
    x["q"] = np.concatenate([x["q"], np.full((5, 8, 128), 0x7FC0, dtype=np.uint16)])
    out = torch.full((n + 5, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    got = run(x, pg, gb, P, out=out)
    assert (bf16_to_f64(got[n:]) == 7.0).all()
    x["q"] = x["q"][:n]
    assert_within(got, w, x)


def test_same_bits_every_time_and_on_a_used_workspace(kernel):
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=128, seed=14)
    pg = pages(x, gb, P, 16, seed=4)
    ws = sv.new_workspace(1 << 27)
    first = run(x, pg, gb, P, workspace=ws)
    ws[256:] = 0xFF  # NaN in all but the flags: nothing stale is read
    assert np.array_equal(run(x, pg, gb, P, workspace=ws), first)
    assert np.array_equal(run(x, pg, gb, P, workspace=ws), first)


@pytest.mark.parametrize("field,at,value", [
    ("gb", 0, 1), ("gb", 1, 7), ("gb", 2, 5), ("gb", 1, -1), ("P", 0, 301), ("P", 1, 130),
    ("P", 0, -1), ("P", 0, 1 << 30), ("T", 0, 1001), ("T", 1, -1), ("D", 2, 8), ("D", 0, -1)])
def test_lengths_out_of_range_are_reported(kernel, field, at, value):
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=128, seed=15)
    pg = pages(x, gb, P, 16, seed=4)
    ws = sv.new_workspace(1 << 27)
    out = torch.full(x["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    bad = dict(gb=gb.copy(), P=P.copy(), T=x["seq_lens"].copy(), D=x["draft_len"].copy())
    bad[field][at] = value
    y = dict(x, seq_lens=bad["T"], draft_len=bad["D"])
    got = run(y, pg, bad["gb"], bad["P"], workspace=ws, out=out, max_draft=7, max_seq=1000)
    assert sv.workspace_status(ws, clear=True) == 8
    assert (bf16_to_f64(got) == 7.0).all()
    assert_within(run(x, pg, gb, P, workspace=ws), w, x)
    assert sv.workspace_status(ws) == 0


def test_more_rows_than_q_holds_and_narrow_tables(kernel):
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=128, seed=16)
    pg = pages(x, gb, P, 16, seed=4)
    ws = sv.new_workspace(1 << 27)
    run(dict(x, q=x["q"][:-1]), pg, gb, P, workspace=ws)
    assert sv.workspace_status(ws, clear=True) == 8
    narrow = dict(pg, block_table=np.ascontiguousarray(pg["block_table"][:, :20]))
    run(x, narrow, gb, P, workspace=ws)
    assert sv.workspace_status(ws, clear=True) == 8


def test_table_entry_outside_the_pool_is_reported(kernel):
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=128, seed=17)
    ws = sv.new_workspace(1 << 27)
    for row, col in ((0, 3), (1, 18), (5, 20)):  # a prefix's, and two own entries
        pg = pages(x, gb, P, 16, seed=4)
        assert pg["block_table"][row, col] >= 0
        pg["block_table"][row, col] = 1 << 29
        run(x, pg, gb, P, workspace=ws)
        assert sv.workspace_status(ws, clear=True) == 8


def test_graph_replay_follows_new_lengths(kernel):
    """One captured call, replayed with other lengths, groups and queries in place."""
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=128, seed=18)
    pg = pages(x, gb, P, 16, seed=4)
    q, k, v, bt, T, D, _ = to_device(x, pg)
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    g_, p_ = i32(gb), i32(P)
    out = torch.empty_like(q)
    ws = sv.new_workspace(1 << 27)
    call = lambda: sv.spec_verify_attn_shared(q, k, v, bt, T, D, g_, p_, max_draft_len=7,  # noqa: E731
                                              max_seq_len=1000, out=out, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    torch.cuda.synchronize()
    assert_within(out.view(torch.int16).cpu().numpy().view(np.uint16), w, x)
    # the prefixes shortened: the same attention (all of it in the pool's first rows)
    p_.copy_(i32([288, 128]))
    pg2 = pages(x, gb, np.array([288, 128]), 16, seed=4)
    _, k2, v2, bt2, _, _, _ = to_device(x, pg2)
    k.copy_(k2), v.copy_(v2), bt.copy_(bt2)
    graph.replay()
    torch.cuda.synchronize()
    assert_within(out.view(torch.int16).cpu().numpy().view(np.uint16), w, x)
    assert sv.workspace_status(ws) == 0


def test_positions_past_32_bits_of_bytes(kernel):
    """A pool whose far pages lie past 2^32 bytes; the prefix and own pages among them."""
    w, x, gb, P = inputs([(100, [(130, 2), (100, 0)])], Hq=8, Hkv=8, d=128, seed=19)
    pg = pages(x, gb, P, 64, seed=4)
    q, k, v, bt, T, D, _ = to_device(x, pg)
    far = 40000  # pages of 128 KiB: 5.2 GB
    K = torch.zeros(far + k.shape[0], 64, 8, 128, dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    K[far:], V[far:] = k, v
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    out = sv.spec_verify_attn_shared(q, K, V, torch.where(bt >= 0, bt + far, bt), T, D, i32(gb), i32(P),
                                     max_draft_len=2, max_seq_len=130)
    torch.cuda.synchronize()
    assert_within(out.view(torch.int16).cpu().numpy().view(np.uint16), w, x)


# plan, sequences, prefixes, join; or, for a small call, plan, attention, join
@pytest.mark.parametrize("after,max_seq", [(0, 2000), (1, 2000), (2, 2000), (3, 2000), (0, 1000), (1, 1000), (2, 1000)])
def test_failed_launch_is_reported_and_the_workspace_serves_on(after, max_seq):
    ensure_built()
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=128, seed=20)
    pg = pages(x, gb, P, 16, seed=4)
    ws = sv.new_workspace(1 << 27)
    sv.api.inject_launch_failure(after)
    with pytest.raises(sv.SpecVerifyError) as e:
        run(x, pg, gb, P, workspace=ws, max_seq=max_seq)
    assert e.value.status == 6
    assert_within(run(x, pg, gb, P, workspace=ws, max_seq=max_seq), w, x)
    assert sv.workspace_status(ws) == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_bounded_wait_runs_out_and_the_call_returns(kv):
    ensure_built()
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=128, kv=kv, seed=21)
    pg = pages(x, gb, P, 16, seed=4)
    ws = sv.new_workspace(1 << 27)
    sv.api.inject_wait_timeout(100000)
    run(x, pg, gb, P, workspace=ws, max_seq=2000)
    assert sv.workspace_status(ws, clear=True) == 7
    assert sv.api.inject_wait_timeout(0) == 0  # taken by that call
    assert_within(run(x, pg, gb, P, workspace=ws, max_seq=2000), w, x)
    assert sv.workspace_status(ws) == 0


def test_fork_extend_attend_trim_compact_together(kernel):
    """A prompt is forked, the samples extend their windows (parting from the shared page),
    write K/V, attend under the shared prefix, roll back and are compacted; the attention
    over the moved pages gives the same bits."""
    bs, Hkv, Hq, d, P = 16, 2, 8, 128, 200
    w, x, gb, Pl = inputs([(P, [(P, 3), (P, 1), (P, 2)])], Hq=Hq, Hkv=Hkv, d=d, seed=22)
    nb, stride = 64, 20
    ref = torch.zeros(nb, dtype=torch.int32, device="cuda")
    lens = torch.zeros(4, dtype=torch.int32, device="cuda")
    table = torch.full((4, stride), -1, dtype=torch.int32, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    k = torch.full((nb, bs, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, float("nan"))
    pools = sv.page_pools([k, v])
    ws = sv.new_workspace(sv.pages_workspace_bytes(nb, 4))
    kw = dict(block_size=bs, workspace=ws)
    bits = lambda a: torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda()  # noqa: E731
    packed = (bits(x["k"]), bits(x["v"]))
    off = np.cumsum([0] + [int(P + n + 1) for n in x["draft_len"]])

    def write(r, b, lo, hi):
        at = torch.arange(lo, hi, device="cuda")
        page = table[r, at // bs].long()
        for pool, src in zip((k, v), packed):
            pool[page, at % bs] = src[off[b] + lo:off[b] + hi]

    # scattered on purpose: row 3 takes pages first and hands them back later
    sv.spec_pages_extend(ref, table, lens, i32([3]), i32([100]), pools=pools, **kw)
    sv.spec_pages_extend(ref, table, lens, i32([0]), i32([P]), pools=pools, **kw)
    write(0, 0, 0, P)
    sv.spec_pages_fork(ref, table, lens, i32([0, 0]), i32([1, 2]), **kw)
    T = lens[:3].clone()
    D = i32(x["draft_len"].tolist())
    sv.spec_pages_extend(ref, table, lens, None, (T + 1 + D).contiguous(), pools=pools, **kw)
    for b in range(3):
        write(b, b, P, P + 1 + int(x["draft_len"][b]))
    q = bits(x["q"])

    def attend():
        o = sv.spec_verify_attn_shared(q, k, v, table[:3], T, D, i32(gb.tolist()), i32([P]),
                                       max_draft_len=3, max_seq_len=P)
        p = sv.spec_verify_attn_paged(q, k, v, table[:3], T, D, max_draft_len=3, max_seq_len=P)
        torch.cuda.synchronize()
        return o.view(torch.int16).cpu().numpy().view(np.uint16), p.view(torch.int16).cpu().numpy().view(np.uint16)

    shared, paged = attend()
    assert_within(shared, w, x)
    assert_within(paged, w, x)
    sv.spec_pages_trim(ref, table, lens, i32([3]), i32([0]), **kw)
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.spec_pages_compact(ref, table, lens, pools=pools, num_live=live, **kw)
    assert int(live) == 12 + 3 * 1  # whole prefix pages once, one last page each
    assert int(table[:3].max()) < int(live)
    again, _ = attend()
    assert np.array_equal(again, shared)
    al, _ = sv.spec_accept(torch.randn(9, 50, device="cuda"), i32([0] * 6), D, max_draft_len=3)
    sv.spec_pages_trim(ref, table, lens, None, (T + al).contiguous(), **kw)
    assert lens[:3].tolist() == (T + al).tolist()
    assert sv.workspace_status(ws) == 0


@pytest.mark.parametrize("B,NG", [(1100, 3), (1100, 1100), (700, 350)])
def test_batches_beyond_the_plans_tables(kernel, B, NG):
    """More sequences and groups than the plan keeps on chip, more units than it does, and
    groups of one."""
    gb = [B * n // NG for n in range(NG + 1)]
    groups = [(17 + n % 9, [(17 + n % 9 + (7 * b) % 30, b % 3) for b in range(gb[n], gb[n + 1])])
              for n in range(NG)]
    w, x, gbeg, P = inputs(groups, Hq=4, Hkv=2, d=64, seed=B + NG)
    assert_within(run(x, pages(x, gbeg, P, 16, seed=5), gbeg, P), w, x)


def test_groups_of_very_different_sizes(kernel):
    """So many groups beside a large one that the plan lays its units out group by group."""
    groups = [(20, [(21 + b % 5, 3) for b in range(260)])] + [(9, [(12, 0)])] * 9000
    w, x, gbeg, P = inputs(groups, Hq=16, Hkv=1, d=64, seed=3)
    assert_within(run(x, pages(x, gbeg, P, 8, seed=5), gbeg, P), w, x)


def test_two_streams_at_once_and_a_given_stream(kernel):
    """Calls on two streams with a workspace each, in flight together, and one on a stream
    passed by argument: the bits of calls alone."""
    cases = []
    for seed, groups in ((30, TWO), (31, [(500, [(510 + 9 * b, b % 4) for b in range(12)])])):
        w, x, gb, P = inputs(groups, Hq=8, Hkv=2, d=128, seed=seed)
        pg = pages(x, gb, P, 16, seed=seed)
        alone = run(x, pg, gb, P)
        i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
        t = to_device(x, pg)
        cases.append((t, i32(gb), i32(P), x, alone, sv.new_workspace(1 << 27), torch.empty_like(t[0]),
                      torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for (q, k, v, bt, T, D, _), g_, p_, x, _, ws, out, s in cases:
            sv.spec_verify_attn_shared(q, k, v, bt, T, D, g_, p_, out=out, workspace=ws, stream=s,
                                       max_draft_len=int(x["draft_len"].max()),
                                       max_seq_len=int(x["seq_lens"].max()))
    torch.cuda.synchronize()
    for _, _, _, _, alone, ws, out, _ in cases:
        assert np.array_equal(out.view(torch.int16).cpu().numpy().view(np.uint16), alone)
        assert sv.workspace_status(ws) == 0


def test_calls_follow_each_other_without_a_wait(kernel):
    """Calls of this and other kinds in one stream, each reading what the one before wrote:
    the second's queries are the first's output, and the paged call's the second's."""
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=128, seed=32)
    pg = pages(x, gb, P, 16, seed=4, junk=-1)
    full = pages(x, gb, np.zeros_like(P), 16, seed=4)  # (the paged call reads every own entry)
    q, k, v, bt, T, D, _ = to_device(x, pg)
    _, k2, v2, bt2, _, _, _ = to_device(x, full)
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    kw = dict(max_draft_len=7, max_seq_len=1000)
    ws, ws2 = sv.new_workspace(1 << 27), sv.new_workspace(1 << 27)

    def chain(wait):
        a = sv.spec_verify_attn_shared(q, k, v, bt, T, D, i32(gb), i32(P), workspace=ws, **kw)
        wait()
        b = sv.spec_verify_attn_shared(a, k, v, bt, T, D, i32(gb), i32(P), workspace=ws, **kw)
        wait()
        c = sv.spec_verify_attn_paged(b, k2, v2, bt2, T, D, workspace=ws2, **kw)
        wait()
        d = sv.spec_verify_attn_shared(c, k, v, bt, T, D, i32(gb), i32(P), workspace=ws, **kw)
        torch.cuda.synchronize()
        return [t.clone() for t in (a, b, c, d)]

    slow = chain(torch.cuda.synchronize)
    for _ in range(10):
        for s, f in zip(slow, chain(lambda: None)):
            assert torch.equal(s, f)


def test_nothing_in_the_batch():
    ensure_built()
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
    o = sv.spec_verify_attn_shared(q, k, k, torch.zeros(0, 3, dtype=torch.int32, device="cuda"), z[:0], z[:0],
                                   torch.zeros(2, dtype=torch.int32, device="cuda"), z, max_draft_len=3,
                                   max_seq_len=30)
    assert o.shape == (0, 8, 128)


def test_binding_refuses():
    ensure_built()
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=128, seed=33)
    q, k, v, bt, T, D, _ = to_device(x, pages(x, gb, P, 16, seed=4))
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    kw = dict(max_draft_len=7, max_seq_len=1000)
    ok = (q, k, v, bt, T, D, i32(gb), i32(P))

    def bad(err, i, t, **more):
        a = list(ok)
        a[i] = t
        with pytest.raises(err):
            sv.spec_verify_attn_shared(*a, **{**kw, **more})

    bad(TypeError, 0, q.float())
    bad(TypeError, 4, T.long())
    bad(TypeError, 6, i32(gb).cpu())
    bad(TypeError, 7, None)
    bad(ValueError, 0, q[:, :, :64].contiguous())
    bad(ValueError, 1, k.transpose(0, 1))
    bad(ValueError, 3, bt[:2])
    bad(ValueError, 6, i32(gb)[:2])
    bad(ValueError, 0, q, out=torch.empty_like(q)[:2])
    bad(ValueError, 0, q, kv_scale=torch.ones(2, 3, device="cuda"))
    bad(sv.SpecVerifyError, 0, q, workspace=sv.new_workspace(1024))


def test_memory_of_a_call_is_made_on_its_stream(kernel):
    """A call on a stream passed by argument, without out and workspace, while the current
    stream is busy."""
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=128, seed=41)
    pg = pages(x, gb, P, 16, seed=41)
    alone = run(x, pg, gb, P)
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    q, k, v, bt, T, D, _ = to_device(x, pg)
    g_, p_, s = i32(gb), i32(P), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    out = sv.spec_verify_attn_shared(q, k, v, bt, T, D, g_, p_, stream=s,
                                     max_draft_len=int(x["draft_len"].max()),
                                     max_seq_len=int(x["seq_lens"].max()))
    s.synchronize()
    assert not torch.cuda.current_stream().query()  # that is still asleep
    torch.cuda.synchronize()
    assert np.array_equal(out.view(torch.int16).cpu().numpy().view(np.uint16), alone)


@pytest.mark.parametrize("B,Hkv,max_seq,small", [
    (2, 2, 1024, True), (2, 2, 1025, False), (20, 2, 512, True), (20, 2, 513, False)])
def test_small_calls_take_the_mma_kernel(B, Hkv, max_seq, small):
    """The automatic choice is by the descriptor: 1024 positions, and 20480 times units."""
    ensure_built()
    w, x, gb, P = inputs([(200, [(201 + 15 * b, b % 4) for b in range(B)])], Hq=4 * Hkv, Hkv=Hkv, d=128,
                         seed=B)
    pg = pages(x, gb, P, 16, seed=B)
    got = run(x, pg, gb, P, max_seq=max_seq)
    assert_within(got, w, x)
    lib = sv.api.load_library()
    same = []
    for k in (1, 2):
        prev = lib.sv_set_attn_kernel(k)
        same.append(np.array_equal(run(x, pg, gb, P, max_seq=max_seq), got))
        lib.sv_set_attn_kernel(prev)
    assert same == [small, not small]


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_longest_windows(kernel, kv):
    """255 drafts, many row tiles a sequence, beside windows of one row."""
    w, x, gb, P = inputs([(70, [(100, 255), (70, 0), (333, 254)]), (0, [(0, 255)])], Hq=8, Hkv=2, d=128,
                         kv=kv, seed=50)
    assert_within(run(x, pages(x, gb, P, 32, seed=1), gb, P), w, x)


def test_largest_pages(kernel):
    w, x, gb, P = inputs([(300, [(300, 3), (640, 1)]), (90, [(95, 2)])], Hq=8, Hkv=2, d=128, seed=51)
    assert_within(run(x, pages(x, gb, P, 65536, seed=1), gb, P), w, x)


def test_graphs_that_share_a_workspace(kernel):
    """Two captured calls of different shapes on one workspace, replayed in turn."""
    cases = []
    ws = sv.new_workspace(1 << 27)
    for seed, groups, Hkv in ((60, TWO, 2), (61, [(500, [(510 + 9 * b, b % 4) for b in range(12)])], 1)):
        w, x, gb, P = inputs(groups, Hq=8, Hkv=Hkv, d=128, seed=seed)
        pg = pages(x, gb, P, 16, seed=seed)
        alone = run(x, pg, gb, P)
        q, k, v, bt, T, D, _ = to_device(x, pg)
        i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
        args = (q, k, v, bt, T, D, i32(gb), i32(P))
        kw = dict(max_draft_len=int(x["draft_len"].max()), max_seq_len=int(x["seq_lens"].max()),
                  out=torch.empty_like(q), workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sv.spec_verify_attn_shared(*args, **kw)
        cases.append((graph, kw["out"], alone, args))
    for _ in range(5):
        for graph, out, _, _ in cases:
            out.zero_()
            graph.replay()
    torch.cuda.synchronize()
    for _, out, alone, _ in cases:
        assert np.array_equal(out.view(torch.int16).cpu().numpy().view(np.uint16), alone)
    assert sv.workspace_status(ws) == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_prefixes_take_their_inputs_over_from_the_sequences_grid(kv):
    """The prefixes' grid runs beside the sequences' and waits for neither the plan nor what
    came before it. Each of its CTAs takes a ticket (a counter at byte 132 of the workspace)
    and acquires a permit (byte 128) that the sequences' grid, which does wait, releases in the
    same call: one per SM a call, also after a call whose prefixes' kernel was not launched."""
    ensure_built()
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=128, kv=kv, seed=70)
    pg = pages(x, gb, P, 16, seed=4)
    ws = sv.new_workspace(1 << 27)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    counters = lambda: ws[128:136].view(torch.int32).tolist()  # noqa: E731
    for call in range(1, 4):
        assert_within(run(x, pg, gb, P, workspace=ws, max_seq=2000), w, x)
        assert counters() == [call * sms] * 2
    sv.api.inject_launch_failure(2)  # plan, sequences, prefixes
    with pytest.raises(sv.SpecVerifyError):
        run(x, pg, gb, P, workspace=ws, max_seq=2000)
    torch.cuda.synchronize()
    assert counters() == [4 * sms, 3 * sms]
    assert_within(run(x, pg, gb, P, workspace=ws, max_seq=2000), w, x)
    assert counters() == [5 * sms] * 2
    ws[128:136].view(torch.int32).fill_(-(sms // 2))  # they wrap in the next call
    assert_within(run(x, pg, gb, P, workspace=ws, max_seq=2000), w, x)
    assert counters() == [sms - sms // 2] * 2
    assert sv.workspace_status(ws) == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e", [-80, -30, 20, 100])
def test_queries_of_any_finite_magnitude(kernel, e, d, kv):
    """q times 2^e under a softmax scale times 2^-e: every product and sum is the same number
    times a power of two, so the bits are the same, far outside f16's range too."""
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=d, kv=kv, seed=71)
    pg = pages(x, gb, P, 16, seed=4)
    scale = 2.0 ** -4
    want = run(x, pg, gb, P, softmax_scale=scale)
    q = bf16_to_f64(x["q"])
    assert np.abs(q).max() * 2.0 ** 20 > 65504 and np.abs(q).max() < 2 ** 20
    big = q * 2.0 ** e
    y = dict(x, q=(big.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16))
    assert np.array_equal(bf16_to_f64(y["q"]), big)  # powers of two: exact
    got = run(y, pg, gb, P, softmax_scale=scale * 2.0 ** -e)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_very_different_magnitudes(kernel, d, kv):
    """Rows 2^24 times as large and as small as their neighbours, in one tile, each within the
    bound: the softmax scale is that of the largest, so the others' weights are nearly even."""
    import oracle
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=d, kv=kv, seed=72)
    q = bf16_to_f64(x["q"])
    q[0::3] *= 2.0 ** 24
    q[1::3] *= 2.0 ** -24
    x["q"] = (q.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    assert np.array_equal(bf16_to_f64(x["q"]), q)
    scale = 2.0 ** -28
    got = bf16_to_f64(run(x, pages(x, gb, P, 16, seed=4), gb, P, softmax_scale=scale))
    kw = dict(Hq=w.Hq, Hkv=w.Hkv, d=w.d, scale=scale, kv_scale=x["kv_scale"])
    mag = x["v"] & (0x7F if x["v"].dtype == np.uint8 else 0x7FFF)
    ref = oracle.verify_attn(x["q"], x["k"], x["v"], x["seq_lens"], x["draft_len"], **kw)
    mag = oracle.verify_attn(x["q"], x["k"], mag.astype(x["v"].dtype), x["seq_lens"], x["draft_len"], **kw)
    assert np.isfinite(got).all()
    # the bound of assert_within: a scale of 2^-4 for the large rows is that of d = 256
    assert (np.abs(got - ref) <= np.abs(ref) * 2.0 ** -8 + mag * (2.0 ** -8 + 2.0 ** -10)).all()


@pytest.mark.parametrize("kv", ["bf16", "bf16 K of 0", "fp8_e4m3", "fp8_e4m3 K of 0"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_infinite_and_nan_queries_become_nan(kernel, d, kv):
    """Scores of an infinity are infinite or NaN, whichever the key: no finite output may come
    of them, with 8-bit keys too (E4M3 has no infinity). All other rows keep their bits."""
    w, x, gb, P = inputs([(150, [(160, 1), (150, 2), (400, 3)])], Hq=4, Hkv=2, d=d, kv=kv.split()[0],
                         seed=74)
    if kv.endswith("0"):  # where q is infinite
        x["k"][:, :, 5:] = 0
    pg = pages(x, gb, P, 16, seed=4)
    full = pages(x, gb, np.zeros_like(P), 16, seed=4)  # (the paged call reads every own entry)

    def both():
        q, k, v, bt, T, D, sc = to_device(x, full)
        o = sv.spec_verify_attn_paged(q, k, v, bt, T, D, max_draft_len=3, max_seq_len=400, kv_scale=sc)
        return run(x, pg, gb, P), o.view(torch.int16).cpu().numpy().view(np.uint16)

    clean = both()
    spoilt = np.zeros(x["q"].shape[:2], dtype=bool)
    for r, h, bits in ((1, 2, [0x7F80]), (3, 0, [0xFF80]), (4, 3, [0x7FC0]), (5, 1, [0x7F80, 0xFF80]),
                       (8, 0, [0x7F80] * (d - 5))):
        x["q"][r, h, 5:5 + len(bits)] = bits
        spoilt[r, h] = True
    for got, want in zip(both(), clean):
        assert np.isnan(bf16_to_f64(got[spoilt])).all()
        assert np.array_equal(got[~spoilt], want[~spoilt])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [0.0, 1e-44, 1e-30])
def test_heads_of_zeros_and_of_tiny_keys(kernel, scale, d):
    """A K scale of 0 (a head whose keys are all zero), one below the normal numbers and one
    next to nothing: even weights over the visible keys, masked tiles and split parts among
    them; the paged call's too. The other heads keep their bits."""
    w, x, gb, P = inputs(TWO, Hq=8, Hkv=2, d=d, kv="fp8_e4m3", seed=76)
    pg = pages(x, gb, P, 16, seed=4)
    full = pages(x, gb, np.zeros_like(P), 16, seed=4)  # (the paged call reads every own entry)

    def both():
        q, k, v, bt, T, D, sc = to_device(x, full)
        o = sv.spec_verify_attn_paged(q, k, v, bt, T, D, max_draft_len=7, max_seq_len=1000, kv_scale=sc)
        return run(x, pg, gb, P), o.view(torch.int16).cpu().numpy().view(np.uint16)

    clean = both()
    x["kv_scale"][0, 1] = scale
    for got, want in zip(both(), clean):
        assert_within(got, w, x)
        assert np.array_equal(got[:, :4], want[:, :4])
