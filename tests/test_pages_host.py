"""Host-side checks of the page operators (C ABI and Python binding), and the plain model
that their GPU tests compare with. CPU only."""
import ctypes
import random

import pytest
import torch

from speculative_decoding_verification_gqa_gb300 import api, build

from page_model import Pages

FAKE = 0x10000  # never dereferenced: checks fail before any launch
ODD = 0x10002


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load_library()


def table(**kw):
    d = dict(num_blocks=64, block_size=16, table_rows=4, max_blocks_per_seq=8, ref_count=FAKE,
             block_table=FAKE, cached_len=FAKE)
    d.update(kw)
    return api.PageTable(**d)


def call(lib, which, t, n=2, lists=(FAKE, FAKE), pools=((FAKE, 4096),), ws=FAKE, ws_bytes=1 << 20,
         num_pools=None):
    arr = (api.PageData * max(1, len(pools)))(*[api.PageData(*p) for p in pools])
    t = None if t is None else ctypes.byref(t)
    np_ = len(pools) if num_pools is None else num_pools
    parr = arr if pools else None
    if which == "fork":
        return lib.spec_pages_fork(t, n, lists[0], lists[1], None, ws, ws_bytes, None)
    if which == "trim":
        return lib.spec_pages_trim(t, n, lists[0], lists[1], ws, ws_bytes, None)
    if which == "extend":
        return lib.spec_pages_extend(t, n, lists[0], lists[1], np_, parr, ws, ws_bytes, None)
    return lib.spec_pages_compact(t, np_, parr, None, None, ws, ws_bytes, None)


ALL = ["fork", "extend", "trim", "compact"]


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("bad,status", [
    (dict(num_blocks=0), 2), (dict(num_blocks=1 << 28), 2), (dict(block_size=12), 2),
    (dict(block_size=4), 2), (dict(block_size=1 << 17), 2), (dict(table_rows=-1), 2), (dict(table_rows=(1 << 20) + 1), 2),
    (dict(max_blocks_per_seq=0), 2), (dict(ref_count=None), 1), (dict(block_table=None), 1),
    (dict(cached_len=None), 1), (dict(ref_count=FAKE + 4), 4), (dict(block_table=ODD), 4),
    (dict(cached_len=ODD), 4)])
def test_bad_state_is_refused(lib, which, bad, status):
    assert call(lib, which, table(**bad)) == status


@pytest.mark.parametrize("which", ALL)
def test_bad_workspace_is_refused(lib, which):
    assert call(lib, which, None) == 1
    assert call(lib, which, table(), ws=None) == 1
    assert call(lib, which, table(), ws=FAKE + 16) == 4
    need = lib.spec_pages_workspace_size(64, 4)
    assert call(lib, which, table(), ws_bytes=need - 1) == 5


@pytest.mark.parametrize("which", ["fork", "extend", "trim"])
def test_bad_lists_are_refused(lib, which):
    assert call(lib, which, table(), n=-1) == 2
    assert call(lib, which, table(), n=5) == 2  # more rows than the table has
    assert call(lib, which, table(), lists=(FAKE, None)) == 1
    assert call(lib, which, table(), lists=(ODD, FAKE)) == 4
    assert call(lib, which, table(), lists=(FAKE, ODD)) == 4
    assert call(lib, which, table(), n=0, lists=(None, None)) == 0  # nothing to do
    if which == "fork":
        assert call(lib, which, table(), lists=(None, FAKE)) == 1


@pytest.mark.parametrize("which", ["extend", "compact"])
@pytest.mark.parametrize("pools,status", [
    (((None, 4096),), 1), (((FAKE + 8, 4096),), 4), (((FAKE, 0),), 2), (((FAKE, 128),), 2),
    (((FAKE, 4096 + 16),), 2), (((FAKE, (1 << 30) + 256),), 2), (((FAKE, 4096),) * 257, 2)])
def test_bad_pools_are_refused(lib, which, pools, status):
    assert call(lib, which, table(), pools=pools) == status


SPREAD = dict(ref_count=1 << 30, block_table=2 << 30, cached_len=3 << 30)  # apart
WS = 4 << 30


@pytest.mark.parametrize("which", ALL)
@pytest.mark.parametrize("a,b", [("ref_count", "block_table"), ("ref_count", "cached_len"),
                                 ("block_table", "cached_len")])
def test_state_arrays_that_overlap_are_refused(lib, which, a, b):
    lists = (5 << 30, 6 << 30)
    nbytes = dict(ref_count=64 * 4, block_table=4 * 8 * 4, cached_len=4 * 4)
    for at in (SPREAD[b], SPREAD[b] + nbytes[b] // 16 * 16 - 16):
        t = table(**{**SPREAD, a: at})
        assert call(lib, which, t, lists=lists, pools=((7 << 30, 4096),), ws=WS) == 2
    assert call(lib, which, table(**{**SPREAD, a: WS + 512}), lists=lists, ws=WS) == 2  # workspace


@pytest.mark.parametrize("which", ["fork", "extend", "trim"])
@pytest.mark.parametrize("name", [*SPREAD, "workspace"])
@pytest.mark.parametrize("k", [0, 1])
def test_lists_inside_what_the_call_changes_are_refused(lib, which, name, k):
    """extend with new_len = cached_len itself, say."""
    lists = [5 << 30, 6 << 30]
    lists[k] = WS + 4 if name == "workspace" else SPREAD[name] + 4
    assert call(lib, which, table(**SPREAD), lists=lists, pools=((7 << 30, 4096),), ws=WS) == 2


@pytest.mark.parametrize("which", ["extend", "compact"])
@pytest.mark.parametrize("name", [*SPREAD, "workspace"])
def test_pools_over_the_state_are_refused(lib, which, name):
    at = WS if name == "workspace" else SPREAD[name]
    pools = ((7 << 30, 4096), (at - 63 * 4096, 4096))  # its last page
    assert call(lib, which, table(**SPREAD), lists=(5 << 30, 6 << 30), pools=pools, ws=WS) == 2


def test_outputs_of_compact_over_the_state_are_refused(lib):
    t = table(**SPREAD)
    for remap, live in ((SPREAD["ref_count"], None), (None, SPREAD["cached_len"] + 12),
                        (5 << 30, (5 << 30) + 252), (WS - 4, None)):
        assert lib.spec_pages_compact(ctypes.byref(t), 0, None, remap, live, WS, 1 << 20, None) == 2


def test_null_pool_list_is_refused(lib):
    assert call(lib, "compact", table(), pools=(), num_pools=1) == 1
    assert call(lib, "compact", table(), num_pools=-1) == 2


def test_workspace_size(lib):
    assert lib.spec_pages_workspace_size(0, 4) == 0
    assert lib.spec_pages_workspace_size(64, -1) == 0
    a, b = (lib.spec_pages_workspace_size(n, 16) for n in (64, 1 << 20))
    assert 0 < a < b


def test_binding_refuses_host_tensors():
    z = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(TypeError):
        api.spec_pages_trim(z, z.view(2, 4), z[:2], None, z[:2], block_size=16)
    with pytest.raises(TypeError):
        api.page_pools([torch.zeros(8, 16, 4)])
    with pytest.raises(ValueError):
        api.page_pools([None] * (api.MAX_PAGE_POOLS + 1))


def test_model_keeps_contents_and_counts():
    """Whatever the operators do to pages, each row holds what was written to it."""
    rng = random.Random(3)
    m, rows = Pages(96, 6, 12, 8), {r: [] for r in range(6)}
    for step in range(400):
        r = rng.randrange(6)
        what = rng.choice(["fork", "extend", "extend", "trim", "compact"])
        if what == "fork" and not rows[r]:
            p = rng.randrange(6)
            if p != r:
                n = rng.randint(0, len(rows[p]))
                m.fork([p], [r], [n])
                rows[r] = rows[p][:n]
        elif what == "extend":
            n = min(96, len(rows[r]) + rng.randint(0, 20))
            if m.extend([r], [n]):
                for pos in range(len(rows[r]), n):
                    m.data[m.table[r][pos // 8]][pos % 8] = (step, pos)
                    rows[r] = rows[r] + [(step, pos)]
        elif what == "trim":
            n = rng.randint(0, len(rows[r]))
            m.trim([r], [n])
            rows[r] = rows[r][:n]
        else:
            m.compact()
            used = sum(1 for x in m.ref if x)
            assert all(x for x in m.ref[:used])
        m.check()
        for k, v in rows.items():
            assert m.content(k) == v
