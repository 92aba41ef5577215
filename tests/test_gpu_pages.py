"""GPU tests of the page operators (fork, extend with copy on write, trim, compact) against
the plain model: whole numbers and moved bits, so everything is compared for equality."""
import random
import threading

import pytest
import torch

import speculative_decoding_verification_gqa_gb300 as sv

from gpu_util import ensure_built
from page_model import Pages, pages_of

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Device:
    """The model's state on the device; the data of page position (p, j) is a number that
    stands in every pool (with the pool's index added)."""

    def __init__(self, m, pools=2, width=8, dtype=torch.int32):
        ensure_built()
        self.m, nb, bs = m, len(m.ref), m.bs
        self.ref = torch.tensor(m.ref, dtype=torch.int32, device=DEV)
        self.lens = torch.tensor(m.lens, dtype=torch.int32, device=DEV)
        self.table = torch.tensor(m.table, dtype=torch.int32, device=DEV)
        ident = torch.arange(nb * bs, dtype=torch.int32, device=DEV).view(nb, bs, 1)
        self.pools = [(ident + 1000000 * k).expand(nb, bs, width).contiguous().to(dtype)
                      for k in range(pools)]
        m.data = [[p * bs + j for j in range(bs)] for p in range(nb)]
        self.handle = sv.page_pools(self.pools)
        self.ws = sv.new_workspace(sv.pages_workspace_bytes(nb, len(m.lens)))

    def i32(self, v):
        return None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)

    def fork(self, p, c, n=None):
        sv.spec_pages_fork(self.ref, self.table, self.lens, self.i32(p), self.i32(c),
                           fork_len=self.i32(n), block_size=self.m.bs, workspace=self.ws)

    def extend(self, rows, n):
        sv.spec_pages_extend(self.ref, self.table, self.lens, self.i32(rows), self.i32(n),
                             block_size=self.m.bs, pools=self.handle, workspace=self.ws)

    def trim(self, rows, n):
        sv.spec_pages_trim(self.ref, self.table, self.lens, self.i32(rows), self.i32(n),
                           block_size=self.m.bs, workspace=self.ws)

    def compact(self):
        remap = torch.full_like(self.ref, -7)
        live = torch.full((1,), -7, dtype=torch.int32, device=DEV)
        sv.spec_pages_compact(self.ref, self.table, self.lens, block_size=self.m.bs,
                              pools=self.handle, remap=remap, num_live=live, workspace=self.ws)
        return remap.tolist(), int(live)

    def status(self):
        return sv.workspace_status(self.ws, clear=True)

    def same(self, data=True):
        m = self.m
        assert self.ref.tolist() == m.ref
        assert self.lens.tolist() == m.lens
        assert self.table.tolist() == m.table
        if data:
            want = torch.tensor(m.data, dtype=torch.int64)
            for k, p in enumerate(self.pools):
                assert bool((p.cpu().long() == (want + 1000000 * k)[..., None]).all()), "pool %d" % k


def filled(rows, blocks, bs, lens, max_blocks=None, seed=0):
    """A state in which row r holds lens[r] positions on pages placed at random."""
    m = Pages(blocks, rows, max_blocks or max(1, max(pages_of(n, bs) for n in lens) + 2), bs)
    ids = list(range(blocks))
    random.Random(seed).shuffle(ids)
    for r, n in enumerate(lens):
        for j in range(pages_of(n, bs)):
            p = ids.pop()
            m.table[r][j], m.ref[p] = p, 1
        m.lens[r] = n
    return m


@pytest.mark.parametrize("bs", [8, 16, 64])
@pytest.mark.parametrize("seed", range(4))
def test_random_life_of_a_pool(bs, seed):
    """A hundred calls of all four operators on ragged batches, each compared with the model:
    state, page data, and the too-few-pages answer."""
    rng = random.Random(100 * bs + seed)
    R, nb, mb = 12, 60, 9
    m = Pages(nb, R, mb, bs)
    d = Device(m, pools=3)
    full = 0
    for _ in range(100):
        op = rng.choice(["fork", "extend", "extend", "extend", "trim", "compact"])
        if op == "fork":
            empty = [r for r in range(R) if m.lens[r] == 0]
            par = [r for r in range(R) if m.lens[r] > 0]
            ch = rng.sample(empty, rng.randint(0, len(empty)))
            if not par or not ch:
                continue
            ps = [rng.choice(par) for _ in ch]
            n = None if rng.random() < 0.4 else [rng.randint(0, m.lens[p]) for p in ps]
            d.fork(ps, ch, n)
            m.fork(ps, ch, n)
            assert d.status() == 0
        elif op == "compact":
            assert d.compact() == m.compact()
            assert d.status() == 0
        else:
            rows = rng.sample(range(R), rng.randint(1, R))
            if rng.random() < 0.3:
                rows = list(range(len(rows)))
            as_null = rows == list(range(len(rows)))
            if op == "extend":
                n = [rng.choice([m.lens[r], min(mb * bs, m.lens[r] + rng.randint(0, 3 * bs))]) for r in rows]
                d.extend(None if as_null else rows, n)
                ok = m.extend(rows, n)
                assert d.status() == (0 if ok else 9)
                full += not ok
            else:
                n = [rng.choice([m.lens[r], rng.randint(0, m.lens[r]), 0]) for r in rows]
                d.trim(None if as_null else rows, n)
                m.trim(rows, n)
                assert d.status() == 0
        m.check()
        d.same()


@pytest.mark.parametrize("family,share_outside", [(2, 0), (5, 0), (5, 1)])
def test_copy_on_write_leaves_the_last_holder_in_place(family, share_outside):
    """All holders of a partial page in one call: every row but the last of the call takes a
    copy; with a holder outside the call all rows of the call take one."""
    bs, n = 16, 37
    m = filled(family + share_outside, 40, bs, [n] + [0] * (family + share_outside - 1))
    kids = list(range(1, family + share_outside))
    d = Device(m)
    d.fork([0] * len(kids), kids)
    m.fork([0] * len(kids), kids)
    rows = list(range(family))[::-1]
    d.extend(rows, [n + 1 + r for r in rows])
    assert m.extend(rows, [n + 1 + r for r in rows])
    d.same()
    shared = m.table[0][2]
    assert (shared in [m.table[r][2] for r in range(1, family)]) is False
    assert m.ref[shared] == 1
    if share_outside:
        assert m.table[family][2] != shared


def test_many_rows_and_pages_span_chunks():
    """More rows than one block of the planning kernel has threads, and a pool of several
    counting chunks with pages taken and moved across their borders."""
    bs, R, nb = 8, 2500, 13001
    lens = [(7 * r) % 33 for r in range(R)]
    m = filled(R, nb, bs, lens, max_blocks=9, seed=4)
    d = Device(m, pools=1, width=4)
    rows = list(range(R))
    random.Random(1).shuffle(rows)
    to = [lens[r] + (r % 17) for r in rows]
    d.extend(rows, to)
    assert m.extend(rows, to)
    d.same()
    rows = rows[:2100]
    to = [m.lens[r] // 2 for r in rows]
    d.trim(rows, to)
    m.trim(rows, to)
    assert d.compact() == m.compact()
    assert d.status() == 0
    d.same()


@pytest.mark.parametrize("children", [1, 7, 8, 9, 31])
def test_fork_many_children_across_table_segments(children):
    bs, n = 8, 8 * 1100 + 3
    m = filled(2 + 2 * children, 2300, bs, [n, n - 900] + [0] * (2 * children), seed=2)
    d = Device(m, pools=1, width=4)
    kids = list(range(2, 2 + 2 * children))
    par = [k % 2 for k in kids] if children % 2 else [k >= 2 + children for k in kids]
    par = [int(p) for p in par]
    length = [(313 * k) % (m.lens[p] + 1) for k, p in zip(kids, par)]
    d.fork(par, kids, length)
    m.fork(par, kids, length)
    assert d.status() == 0
    d.same(data=False)


@pytest.mark.parametrize("page_bytes_per_pos", [16, 48, 4096])
def test_page_sizes(page_bytes_per_pos):
    """Pages below, above and off the copying granule."""
    bs = 32
    m = filled(4, 64, bs, [100, 0, 33, 64], seed=9)
    d = Device(m, pools=2, width=page_bytes_per_pos // 4)
    d.fork([0], [1])
    m.fork([0], [1])
    d.extend([1, 0, 2], [101, 130, 34])
    assert m.extend([1, 0, 2], [101, 130, 34])
    d.same()
    assert d.compact() == m.compact()
    d.same()


def test_pool_used_up_exactly_and_by_one_page_too_many():
    bs = 8
    m = filled(3, 10, bs, [8, 5, 0], max_blocks=12, seed=1)
    d = Device(m)
    d.extend([2, 0], [bs * 6, bs * 4])  # nine pages: one too many
    assert d.status() == 9
    d.same()
    d.extend([2, 0], [bs * 5, bs * 4])  # the eight that are free
    assert m.extend([2, 0], [bs * 5, bs * 4])
    assert d.status() == 0
    d.same()
    d.extend(None, m.lens)  # nothing to take from an empty pool
    assert d.status() == 0
    d.extend([1], [9])
    assert d.status() == 9
    d.same()
    assert d.compact() == (list(range(10)), 10)
    d.same()


def test_empty_pool_and_rows():
    m = Pages(9, 2, 3, 8)
    d = Device(m)
    assert d.compact() == ([-1] * 9, 0)
    d.trim([1], [0])
    d.fork([0], [1])
    d.extend([0, 1], [0, 0])
    assert d.status() == 0
    d.same()


@pytest.mark.parametrize("bad", ["twice", "below", "above", "short", "long"])
@pytest.mark.parametrize("op", ["extend", "trim"])
def test_bad_rows_change_nothing(op, bad):
    bs = 8
    m = filled(4, 30, bs, [20, 9, 0, 16], max_blocks=6, seed=3)
    d = Device(m)
    rows, n = [0, 3, 1], ([25, 16, 10] if op == "extend" else [4, 16, 0])
    if bad == "twice":
        rows[2] = 0
        n[2] = n[0]
    elif bad == "below":
        rows[1] = -1
    elif bad == "above":
        rows[1] = 4
    elif bad == "short":
        n[0] = 19 if op == "extend" else -1
    else:
        n[0] = 6 * bs + 1 if op == "extend" else 21
    getattr(d, op)(rows, n)
    assert d.status() == 8
    d.same()


@pytest.mark.parametrize("p,c,n", [
    ([0, 1], [2, 2], None), ([0], [1], None), ([0, 2], [2, 3], None), ([0], [4], None),
    ([-1], [2], None), ([0], [2], [21]), ([0], [2], [-1])])
def test_bad_forks_change_nothing(p, c, n):
    m = filled(4, 30, 8, [20, 9, 0, 0], max_blocks=6, seed=3)
    d = Device(m)
    d.fork(p, c, n)
    assert d.status() == 8
    d.same()


@pytest.mark.parametrize("entry", [-1, 30, 1 << 30])
def test_damaged_tables_touch_nothing_else(entry):
    """An entry in use that names no page: reported; compact changes nothing, extend neither
    where it needs the entry; trim and fork leave every count of other pages right."""
    m = filled(4, 30, 8, [20, 9, 0, 16], max_blocks=6, seed=3)
    m.table[0][2] = entry
    d = Device(m)
    d.compact()
    assert d.status() == 8
    d.same()
    d.extend([0], [21])
    assert d.status() == 8
    d.same()
    d.fork([0], [2])
    assert d.status() == 8
    want = list(m.ref)
    for j in (0, 1):
        want[m.table[0][j]] += 1
    assert d.ref.tolist() == want
    d.trim([2, 0], [0, 0])
    assert d.status() == 8
    for j in (0, 1):
        want[m.table[0][j]] -= 2
    assert d.ref.tolist() == want and min(want) >= 0


def test_free_page_named_by_a_row():
    m = filled(2, 20, 8, [20, 9], seed=5)
    d = Device(m)
    d.ref[m.table[0][1]] = 0
    before = d.ref.tolist()
    d.compact()
    assert d.status() == 8 and d.ref.tolist() == before
    d.trim([0], [0])
    assert d.status() == 8 and min(d.ref.tolist()) == 0


@pytest.mark.parametrize("count", [0, 1, 2])
def test_rows_that_drop_a_page_more_often_than_it_is_counted(count):
    """Three rows of a call name one page: the count ends at 0, and the call says so."""
    m = filled(4, 20, 8, [20, 9, 5, 8], seed=6)
    d = Device(m)
    p = m.table[0][0]
    for r in (1, 2):
        d.ref[m.table[r][0]] = 0
        d.table[r, 0] = p
    d.ref[p] = count
    d.trim([0, 1, 2, 3], [0, 0, 0, 0])
    assert d.status() == 8
    assert d.ref.tolist() == [0] * 20
    assert d.lens.tolist() == [0] * 4 and bool((d.table == -1).all())


@pytest.mark.parametrize("n", [7, 8, 9, 40])
def test_rows_that_share_parts_of_their_pages_are_trimmed(n):
    """Runs of rows that share some pages and not others, in call orders that keep and break
    the runs, trimmed to different lengths."""
    rng = random.Random(n)
    m = Pages(400, 64, 40, 8)
    assert m.extend([0, 1], [300, 130])
    m.fork([rng.choice([0, 0, 1]) for _ in range(n)], list(range(2, 2 + n)),
           [rng.randint(60, 130) for _ in range(n)])
    assert m.extend(list(range(2, 2 + n)), [m.lens[r] + rng.randint(0, 12) for r in range(2, 2 + n)])
    d = Device(m)
    for rows in (list(range(2 + n)), rng.sample(range(2 + n), n)):
        to = [rng.randint(0, m.lens[r]) for r in rows]
        d.trim(rows, to)
        m.trim(rows, to)
        assert d.status() == 0
        d.same(data=False)


def test_graph_replays_a_step_on_its_own_stream():
    """fork, extend, trim and compact in one captured graph, replayed: the state at the start
    of every replay is put back, and the results are those of eager calls."""
    bs = 16
    m = filled(6, 50, bs, [40, 0, 0, 33, 16, 0], max_blocks=5, seed=7)
    d = Device(m)
    first = [t.clone() for t in (d.ref, d.lens, d.table)]
    par, kids, rows, to, back = d.i32([0, 3]), d.i32([1, 5]), d.i32([1, 0, 5]), d.i32([44, 47, 50]), d.i32([41, 41, 33])
    live = torch.zeros(1, dtype=torch.int32, device=DEV)

    def step():
        for t, f in zip((d.ref, d.lens, d.table), first):
            t.copy_(f)
        sv.spec_pages_fork(d.ref, d.table, d.lens, par, kids, block_size=bs, workspace=d.ws)
        sv.spec_pages_extend(d.ref, d.table, d.lens, rows, to, block_size=bs, pools=d.handle, workspace=d.ws)
        sv.spec_pages_trim(d.ref, d.table, d.lens, rows, back, block_size=bs, workspace=d.ws)
        sv.spec_pages_compact(d.ref, d.table, d.lens, block_size=bs, pools=d.handle, num_live=live, workspace=d.ws)

    m.fork([0, 3], [1, 5])
    assert m.extend([1, 0, 5], [44, 47, 50])
    m.trim([1, 0, 5], [41, 41, 33])
    _, L = m.compact()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        d.same(data=False)
        assert int(live) == L
    assert d.status() == 0


@pytest.mark.parametrize("op,launches", [("fork", 1), ("extend", 2), ("trim", 1), ("compact", 2)])
def test_failed_launch_is_reported_and_the_workspace_serves_on(op, launches):
    for k in range(launches):
        m = filled(4, 30, 8, [20, 9, 0, 16], max_blocks=6, seed=3)
        d = Device(m)
        args = dict(fork=([0], [2]), extend=([0], [25]), trim=([0], [3]), compact=())[op]
        sv.api.inject_launch_failure(k)
        with pytest.raises(sv.SpecVerifyError) as e:
            getattr(d, op)(*args)
        assert e.value.status == 6
        d.same()  # the state changes in the last kernel only
        getattr(d, op)(*args)
        getattr(m, op)(*args)
        assert d.status() == 0
        d.same()


def test_binding_refuses():
    m = filled(4, 30, 8, [20, 9, 0, 16], max_blocks=6, seed=3)
    d = Device(m)
    one = d.i32([0])
    kw = dict(block_size=8, workspace=d.ws)
    with pytest.raises(TypeError):
        sv.spec_pages_trim(d.ref.long(), d.table, d.lens, one, one, **kw)
    with pytest.raises(ValueError):
        sv.spec_pages_trim(d.ref, d.table[:, ::2], d.lens, one, one, **kw)
    with pytest.raises(ValueError):
        sv.spec_pages_trim(d.ref, d.table, d.lens, one, d.i32([0, 1]), **kw)
    with pytest.raises(ValueError):
        sv.spec_pages_extend(d.ref, d.table, d.lens, one, one, pools=[d.pools[0][:5].contiguous()], **kw)
    with pytest.raises(ValueError):
        sv.page_pools([d.pools[0], d.pools[0]])
    with pytest.raises(ValueError):
        sv.spec_pages_compact(d.ref, d.table, d.lens, remap=one, **kw)
    with pytest.raises(sv.SpecVerifyError) as e:
        sv.spec_pages_trim(d.ref, d.table, d.lens, one, one, block_size=8, workspace=d.ws[:256])
    assert e.value.status == 5
    d.same()


def test_more_than_a_thousand_rows_part_from_shared_pages():
    """Beyond the rows that the plan counts on chip: families of a partial page, some with a
    holder outside the call, in one call of 1500 rows."""
    bs, fam, R = 8, 6, 1800
    lens = [13 if r % fam == 0 else 0 for r in range(R)]
    m = filled(R, 6000, bs, lens, max_blocks=4, seed=8)
    d = Device(m, pools=1, width=4)
    kids = [r for r in range(R) if r % fam]
    d.fork([r // fam * fam for r in kids], kids)
    m.fork([r // fam * fam for r in kids], kids)
    rows = random.Random(2).sample(range(R), 1500)
    to = [13 + r % 12 for r in rows]
    d.extend(rows, to)
    assert m.extend(rows, to)
    assert d.status() == 0
    d.same()


@pytest.mark.parametrize("nb", [4096, 4097, 4096 * 11 - 3])
def test_pools_of_many_chunks(nb):
    """Around the pool size above which the ranks have a kernel of their own."""
    bs, R = 8, 120
    m = filled(R, nb, bs, [(37 * r) % 500 for r in range(R)], max_blocks=70, seed=nb)
    d = Device(m, pools=1, width=4)
    rows = list(range(0, R, 2))
    d.trim(rows, [m.lens[r] // 3 for r in rows])
    m.trim(rows, [m.lens[r] // 3 for r in rows])
    assert d.compact() == m.compact()
    assert d.status() == 0
    d.same()


def test_a_table_of_very_many_rows():
    bs, R = 8, 300000
    m = filled(R, 64, bs, [9, 4] + [0] * (R - 2), max_blocks=2, seed=8)
    d = Device(m, pools=1, width=4)
    d.fork([0, 1], [R - 1, 7])
    m.fork([0, 1], [R - 1, 7])
    d.extend([R - 1, 0], [16, 10])
    assert m.extend([R - 1, 0], [16, 10])
    d.trim([R - 1, 7], [3, 0])
    m.trim([R - 1, 7], [3, 0])
    d.trim([5, 5], [0, 0])
    assert d.status() == 8
    assert d.compact() == m.compact()
    d.same()


@pytest.mark.parametrize("op", ["fork", "extend", "trim", "compact"])
def test_rows_of_very_many_entries(op):
    """A table row may have any number of entries; a few of them are in use."""
    bs = 8
    m = Pages(64, 2, 9, bs)
    for j in range(8):
        m.table[0][j], m.ref[3 * j] = 3 * j, 1
    m.lens[0] = 60
    d = Device(m)
    wide = (1 << 31) - 1
    big = torch.empty(2 * wide, dtype=torch.int32, device=DEV).view(2, wide)
    big[:, :9] = d.table
    d.table = big
    if op == "fork":
        d.fork([0], [1], [50])
        m.fork([0], [1], [50])
    elif op == "extend":
        d.extend([0, 1], [66, 20])
        assert m.extend([0, 1], [66, 20])
    elif op == "trim":
        d.trim([0], [9])
        m.trim([0], [9])
    else:
        d.compact()
        m.compact()
    assert d.status() == 0
    d.table = big[:, :9].contiguous()
    d.same(data=op == "compact")


@pytest.mark.parametrize("as_number", [False, True])
def test_workspace_is_made_on_the_stream_of_the_call(as_number):
    """A call on a stream passed by argument, without a workspace, while the current stream is
    busy: its zeros come before it, although the memory held other bits before."""
    m = filled(2, 64, 16, [100, 0], max_blocks=9)
    d = Device(m)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):  # what the allocator will hand out again
        junk = torch.full((sv.pages_workspace_bytes(64, 2),), 255, dtype=torch.uint8, device=DEV)
    ps, ch = d.i32([0]), d.i32([1])
    del junk
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    sv.spec_pages_fork(d.ref, d.table, d.lens, ps, ch, block_size=16,
                       stream=s.cuda_stream if as_number else s)
    s.synchronize()
    assert not torch.cuda.current_stream().query()  # that is still asleep
    torch.cuda.synchronize()
    m.fork([0], [1])
    d.same()


@pytest.mark.parametrize("op", ["fork", "extend", "trim"])
def test_host_threads_with_tables_of_different_sizes(op):
    """Two host threads, each with a state, a stream and a workspace of its own; both tables have
    more rows than a launch has room for unasked, one three times as many as the other."""
    ensure_built()
    bs, calls, bad = 8, 3000, []
    start = threading.Barrier(2)

    def work(R):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            ref = torch.zeros(64, dtype=torch.int32, device=DEV)
            lens = torch.zeros(R, dtype=torch.int32, device=DEV)
            table = torch.full((R, 2), -1, dtype=torch.int32, device=DEV)
            a, b = (torch.tensor([r], dtype=torch.int32, device=DEV) for r in (R - 2, R - 1))
            zero = torch.zeros(1, dtype=torch.int32, device=DEV)
            ws = sv.new_workspace(sv.pages_workspace_bytes(64, R))
            s.synchronize()
            start.wait()
            try:
                for _ in range(calls):  # calls that leave an empty state as it is
                    if op == "fork":
                        sv.spec_pages_fork(ref, table, lens, a, b, block_size=bs, workspace=ws)
                    elif op == "extend":
                        sv.spec_pages_extend(ref, table, lens, a, zero, block_size=bs, workspace=ws)
                    else:
                        sv.spec_pages_trim(ref, table, lens, a, zero, block_size=bs, workspace=ws)
            except sv.SpecVerifyError as e:
                bad.append((R, e.status))
            s.synchronize()
            if sv.workspace_status(ws, stream=s) != 0 or int(lens.sum()) or int(ref.sum()):
                bad.append((R, "state"))

    threads = [threading.Thread(target=work, args=(R,)) for R in (300_000, 1 << 20)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert bad == []


@pytest.mark.parametrize("kids", [1, 7, 8, 9, 31])
@pytest.mark.parametrize("col", [0, 1, 600])
def test_fork_of_a_row_that_names_a_free_page(kids, col):
    """Damaged before the call, so the call says so, whichever item of the work meets the page,
    and for children of one parent or of two that both name the page."""
    bs, n = 8, 8 * 601 + 3
    for parents in ([0], [0, 1]):
        m = filled(3 + kids, 1400, bs, [n, n] + [0] * (1 + kids), seed=kids)
        d = Device(m, pools=1, width=4)
        p = m.table[0][col]
        d.ref[p] = 0
        if len(parents) == 2:
            d.ref[m.table[1][col]] = 0
            d.table[1, col] = p
        d.fork([parents[k % len(parents)] for k in range(kids)], list(range(3, 3 + kids)))
        assert d.status() == 8
        d.trim([2], [0])  # a row that is sound
        assert d.status() == 0


def test_fork_beside_a_free_page_is_not_reported():
    """An entry past the forked length, or of a row that is no parent, is not met."""
    bs = 8
    m = filled(4, 30, bs, [20, 9, 0, 0], seed=3)
    d = Device(m)
    d.ref[m.table[0][2]] = 0
    d.ref[m.table[1][0]] = 0
    d.fork([0, 0], [2, 3], [16, 9])
    assert d.status() == 0


def test_calls_of_very_many_rows():
    """A call of 2^18 rows of a table of 2^18 + 2^17: every row of it extends, half of them
    from shared partial pages; the others are forked, and all are trimmed. Against the same on
    tensors, as the model takes rows one by one."""
    ensure_built()
    bs, n, kids = 8, 1 << 18, 1 << 17
    R, nb, mb = n + kids, 3 * (1 << 18), 3
    i32 = lambda t: t.to(torch.int32)  # noqa: E731
    rows = torch.randperm(R, device=DEV, generator=torch.Generator(DEV).manual_seed(5))
    par, child = rows[:kids], rows[n:]  # every child has a parent of its own
    ref = torch.zeros(nb, dtype=torch.int32, device=DEV)
    lens = torch.zeros(R, dtype=torch.int32, device=DEV)
    table = torch.full((R, mb), -1, dtype=torch.int32, device=DEV)
    pool = torch.arange(nb * bs, dtype=torch.int32, device=DEV).view(nb, bs, 1).expand(nb, bs, 4).contiguous()
    first = pool.clone()
    kw = dict(block_size=bs, workspace=sv.new_workspace(sv.pages_workspace_bytes(nb, R)))
    status = lambda: sv.workspace_status(kw["workspace"], clear=True)  # noqa: E731
    # 2^18 rows take a page of 5 positions each, in call order
    sv.spec_pages_extend(ref, table, lens, i32(rows[:n]), torch.full((n,), 5, dtype=torch.int32, device=DEV),
                         pools=[pool], **kw)
    assert status() == 0
    assert torch.equal(table[rows[:n], 0], torch.arange(n, dtype=torch.int32, device=DEV))
    sv.spec_pages_fork(ref, table, lens, i32(par), i32(child), **kw)
    assert status() == 0
    assert torch.equal(table[child, 0], table[par, 0]) and bool((lens[child] == 5).all())
    assert bool((ref[:kids] == 2).all()) and bool((ref[kids:n] == 1).all())
    # the children, then half of the other rows: each child takes a copy, the others a second page
    call = torch.cat([child, rows[kids:n]])
    to = torch.where(torch.arange(n, device=DEV) < kids, 6, 9)
    sv.spec_pages_extend(ref, table, lens, i32(call), i32(to), pools=[pool], **kw)
    assert status() == 0
    fresh = torch.arange(n, n + n, dtype=torch.int32, device=DEV)
    assert torch.equal(table[child, 0], fresh[:kids]) and torch.equal(table[rows[kids:n], 1], fresh[kids:])
    assert bool((ref[:2 * n] == 1).all()) and bool((ref[2 * n:] == 0).all())
    assert torch.equal(pool[n:n + kids, :5], first[:kids, :5]) and torch.equal(pool[n:n + kids, 5:], first[n:n + kids, 5:])
    assert torch.equal(pool[:n], first[:n]) and torch.equal(pool[n + kids:], first[n + kids:])
    sv.spec_pages_trim(ref, table, lens, i32(rows[torch.randperm(R, device=DEV)]),
                       torch.zeros(R, dtype=torch.int32, device=DEV), **kw)
    assert status() == 0
    assert bool((ref == 0).all()) and bool((lens == 0).all()) and bool((table == -1).all())
