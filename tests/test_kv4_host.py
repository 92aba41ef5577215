"""Host-side checks of the 4-bit cache's calls, of spec_attn_mass and of spec_kv_evict (C ABI
and Python binding), and the plain model of the 4-bit format. CPU only."""
import ctypes
import math

import pytest
import torch

from speculative_decoding_verification_gqa_gb300 import api, build

from kv4_util import E2M1, e4m3_values, evict, quantise, values

FAKE = 0x10000  # never dereferenced: checks fail before any launch
KV4 = 3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load_library()


def pages(**kw):
    d = dict(num_blocks=64, block_size=16, num_kv_heads=2, head_dim=128, k_codes=1 << 30, v_codes=2 << 30,
             scales=3 << 30, kv_scale=4 << 30)
    d.update(kw)
    return api.Kv4Pages(**d)


def desc(**kw):
    d = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, max_draft_len=3, max_seq_len=100, q_rows=8,
             kv_rows=0, kv_dtype=KV4, softmax_scale=0.0)
    d.update(kw)
    return api.AttnDesc(**d)


def ref(x):
    return None if x is None else ctypes.byref(x)


def rows_call(lib, which, p, **kw):
    a = dict(n=2, bt=FAKE, mb=8, start=FAKE, count=FAKE, rows=8, k=5 << 30, v=6 << 30, ks=256, vs=256, ws=FAKE,
             bytes=256)
    a.update(kw)
    head = (ref(p), a["n"], a["bt"], a["mb"], a["start"], a["count"], a["rows"])
    if which == "write":
        return lib.spec_kv4_write(*head, a["k"], a["ks"], a["v"], a["vs"], a["ws"], a["bytes"], None)
    return lib.spec_kv4_read(*head, a["k"], a["v"], a["ws"], a["bytes"], None)


def attn_call(lib, d, p, **kw):
    a = dict(q=FAKE, bt=FAKE, mb=8, T=FAKE, D=FAKE, out=FAKE, lse=None, ws=FAKE, bytes=1 << 40)
    a.update(kw)
    return lib.spec_verify_attn_kv4(ref(d), a["q"], ref(p), a["bt"], a["mb"], a["T"], a["D"], a["out"], a["lse"],
                                    a["ws"], a["bytes"], None)


def mass_call(lib, d, **kw):
    a = dict(q=FAKE, k=FAKE, sc=FAKE, hs=FAKE, nb=64, bs=16, bt=FAKE, mb=8, T=FAKE, D=FAKE, n=None, lse=None,
             mass=FAKE, stride=104, ws=FAKE, bytes=1 << 40)
    a.update(kw)
    return lib.spec_attn_mass(ref(d), a["q"], a["k"], a["sc"], a["hs"], a["nb"], a["bs"], a["bt"], a["mb"], a["T"],
                              a["D"], a["n"], a["lse"], a["mass"], a["stride"], a["ws"], a["bytes"], None)


STATE = dict(ref_count=1 << 30, block_table=2 << 30, cached_len=3 << 30)


def evict_call(lib, **kw):
    t = dict(num_blocks=64, block_size=16, table_rows=4, max_blocks_per_seq=8, **STATE)
    t.update({k: kw.pop(k) for k in list(kw) if k in t})
    a = dict(n=2, rows=None, new=4 << 30, first=None, last=0, heads=2, mass=5 << 30, stride=128, kept=None, ks=0,
             pools=((6 << 30, 2048),), ws=7 << 30, bytes=1 << 30, num=None)
    a.update(kw)
    arr = (api.PageData * max(1, len(a["pools"])))(*[api.PageData(*p) for p in a["pools"]])
    return lib.spec_kv_evict(ctypes.byref(api.PageTable(**t)), a["n"], a["rows"], a["new"], a["first"], a["last"],
                             a["heads"], a["mass"], a["stride"], a["kept"], a["ks"],
                             len(a["pools"]) if a["num"] is None else a["num"], arr, a["ws"], a["bytes"], None)


def test_layout_of_the_structure():
    assert ctypes.sizeof(api.Kv4Pages) == 56
    assert [getattr(api.Kv4Pages, n).offset for n, _ in api.Kv4Pages._fields_] == [0, 8, 12, 16, 24, 32, 40, 48]


def test_packed_descriptors_are_the_structures():
    d = desc(softmax_scale=0.25, sliding_window=7, q_rows=1 << 40, kv_rows=5)
    fields = [getattr(d, n) for n, _ in api.AttnDesc._fields_]
    assert api._ATTN_DESC.pack(*fields) == bytes(d)
    p = pages(num_blocks=1 << 33)
    assert api._KV4_PAGES.pack(*[getattr(p, n) for n, _ in api.Kv4Pages._fields_]) == bytes(p)


@pytest.mark.parametrize("bad", [dict(max_seq_len=1 << 31), dict(max_draft_len=-1 << 40), dict(window=1 << 31),
                                 dict(scale="1"), dict(max_seq_len=2.5)])
def test_arguments_that_the_descriptor_cannot_hold(bad):
    a = dict(B=1, Hq=4, hkv=1, d=64, max_draft_len=0, max_seq_len=9, q_rows=3, dtype=0, scale=0.0, window=0)
    with pytest.raises(ValueError):
        api._packed_desc(**{**a, **bad})


BAD_PAGES = [
    (dict(num_blocks=0), 2), (dict(num_blocks=1 << 31), 2), (dict(num_blocks=1 << 28), 2), (dict(block_size=12), 2),
    (dict(block_size=4), 2), (dict(block_size=1 << 17), 2), (dict(num_kv_heads=0), 2), (dict(num_kv_heads=4097), 2),
    (dict(head_dim=96), 2), (dict(head_dim=256), 2), (dict(k_codes=None), 1), (dict(v_codes=None), 1),
    (dict(scales=None), 1), (dict(kv_scale=None), 1), (dict(k_codes=FAKE + 8), 4), (dict(v_codes=FAKE + 8), 4),
    (dict(scales=FAKE + 8), 4), (dict(kv_scale=FAKE + 2), 4)]


@pytest.mark.parametrize("which", ["write", "read", "attn"])
@pytest.mark.parametrize("bad,status", BAD_PAGES)
def test_bad_pages(lib, which, bad, status):
    if which == "attn":
        assert attn_call(lib, desc(), pages(**bad)) == status
        assert attn_call(lib, desc(), None) == 1
    else:
        assert rows_call(lib, which, pages(**bad)) == status
        assert rows_call(lib, which, None) == 1


@pytest.mark.parametrize("which", ["write", "read"])
@pytest.mark.parametrize("bad,status", [
    (dict(n=-1), 2), (dict(mb=0), 2), (dict(rows=-1), 2), (dict(rows=1 << 31), 2), (dict(bt=None), 1),
    (dict(start=None), 1), (dict(count=None), 1), (dict(ws=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(bt=FAKE + 2), 4), (dict(start=FAKE + 1), 4), (dict(count=FAKE + 2), 4), (dict(k=(5 << 30) + 8), 4),
    (dict(v=(6 << 30) + 2), 4), (dict(ws=FAKE + 128), 4), (dict(bytes=255), 5),
    (dict(k=1 << 30), 2), (dict(v=(2 << 30) + 64), 2), (dict(v=(3 << 30) - 16), 2),  # inside the pages
    (dict(n=0, bt=None, k=None), 0), (dict(rows=0, k=None, v=None), 0)])  # nothing to do
def test_bad_row_calls(lib, which, bad, status):
    assert rows_call(lib, which, pages(), **bad) == status


@pytest.mark.parametrize("name", ["ks", "vs"])
@pytest.mark.parametrize("stride", [0, 255, 248, 260, (1 << 30) + 8])
def test_bad_row_strides(lib, name, stride):
    assert rows_call(lib, "write", pages(), **{name: stride}) == 2


def test_outputs_that_overlap(lib):
    assert rows_call(lib, "read", pages(), k=6 << 30) == 2
    assert rows_call(lib, "read", pages(), k=(6 << 30) + 8 * 2 * 128 * 2 - 16) == 2


@pytest.mark.parametrize("bad,status", [
    (dict(sliding_window=-1), 2), (dict(head_dim=96), 2), (dict(num_q_heads=7), 2), (dict(max_draft_len=256), 2),
    (dict(batch=-1), 2), (dict(kv_dtype=0), 3), (dict(kv_dtype=1), 3), (dict(kv_dtype=2), 3), (dict(kv_dtype=4), 3),
    (dict(softmax_scale=math.nan), 2), (dict(softmax_scale=-1.0), 2), (dict(num_kv_heads=4), 2), (dict(head_dim=64), 2),
    (dict(q_rows=1 << 29), 2)])
def test_bad_descriptors(lib, bad, status):
    assert attn_call(lib, desc(**bad), pages()) == status
    if "num_kv_heads" not in bad and bad.get("head_dim") != 64 and "q_rows" not in bad:  # (against the pages)
        assert lib.spec_verify_attn_kv4_workspace_size(ctypes.byref(desc(**bad))) == 0
    assert attn_call(lib, None, pages()) == 1


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), 1), (dict(bt=None), 1), (dict(T=None), 1), (dict(D=None), 1), (dict(out=None), 1),
    (dict(ws=None), 1), (dict(mb=0), 2), (dict(q=FAKE + 8), 4), (dict(out=FAKE + 8), 4), (dict(lse=FAKE + 2), 4),
    (dict(T=FAKE + 2), 4), (dict(D=FAKE + 1), 4), (dict(bt=FAKE + 2), 4), (dict(ws=FAKE + 16), 4)])
def test_bad_attention_calls(lib, bad, status):
    assert attn_call(lib, desc(), pages(), **bad) == status


def test_empty_batches(lib):
    assert attn_call(lib, desc(batch=0), pages(), q=None, out=None) == 0
    assert mass_call(lib, desc(batch=0), q=None, mass=None) == 0
    assert evict_call(lib, n=0, new=None, mass=None) == 0


def test_the_other_calls_take_no_4_bit_pages(lib):
    d = desc()
    assert lib.spec_verify_attn_paged(ref(d), FAKE, FAKE, FAKE, 64, 16, FAKE, 8, FAKE, FAKE, FAKE, FAKE, FAKE,
                                      1 << 40, None) == 3
    assert lib.spec_verify_attn_workspace_size(ref(d)) == 0


@pytest.mark.parametrize("kw,bad,status", [
    (dict(sliding_window=8), {}, 2), (dict(kv_dtype=2), {}, 3), ({}, dict(nb=0), 2), ({}, dict(bs=12), 2),
    ({}, dict(nb=1 << 28), 2), ({}, dict(mb=0), 2), ({}, dict(stride=0), 2), ({}, dict(stride=1 << 41), 2),
    ({}, dict(q=None), 1), ({}, dict(k=None), 1), ({}, dict(mass=None), 1), ({}, dict(T=None), 1),
    ({}, dict(sc=None), 1), ({}, dict(hs=None), 1), (dict(kv_dtype=1), dict(sc=None, hs=None), 1),
    (dict(kv_dtype=1), {}, 2), (dict(kv_dtype=0), dict(sc=None), 2), (dict(kv_dtype=0), dict(hs=None), 2),
    ({}, dict(sc=FAKE + 8), 4), ({}, dict(k=FAKE + 8), 4), ({}, dict(n=FAKE + 2), 4), ({}, dict(lse=FAKE + 2), 4),
    ({}, dict(mass=FAKE + 2), 4), ({}, dict(ws=FAKE + 16), 4)])
def test_bad_mass_calls(lib, kw, bad, status):
    assert mass_call(lib, desc(**kw), **bad) == status
    assert mass_call(lib, None) == 1


@pytest.mark.parametrize("bad,status", [
    (dict(num_blocks=0), 2), (dict(block_size=12), 2), (dict(ref_count=None), 1), (dict(n=5), 2), (dict(n=-1), 2),
    (dict(last=-1), 2), (dict(heads=0), 2), (dict(heads=4097), 2), (dict(stride=0), 2), (dict(stride=(1 << 30) + 1), 2),
    (dict(kept=FAKE, ks=-1), 2), (dict(kept=FAKE, ks=(1 << 30) + 1), 2), (dict(new=None), 1), (dict(mass=None), 1),
    (dict(new=FAKE + 2), 4), (dict(rows=FAKE + 2), 4), (dict(first=FAKE + 1), 4), (dict(mass=(5 << 30) + 2), 4),
    (dict(kept=FAKE + 2, ks=9), 4), (dict(ws=None), 1), (dict(ws=(7 << 30) + 16), 4), (dict(bytes=1024), 5),
    (dict(pools=((6 << 30, 2048 + 16),)), 2), (dict(pools=((6 << 30, 256),), heads=4), 2),  # 4 bytes a head
    (dict(pools=((None, 2048),)), 1), (dict(pools=(), num=-1), 2)])
def test_bad_eviction_calls(lib, bad, status):
    assert evict_call(lib, **bad) == status


@pytest.mark.parametrize("bad", [
    dict(mass=STATE["ref_count"]), dict(mass=STATE["cached_len"] + 4), dict(ws=5 << 30), dict(rows=5 << 30),
    dict(new=(5 << 30) + 4092), dict(kept=5 << 30, ks=128), dict(kept=4 << 30, ks=128), dict(first=7 << 30),
    dict(pools=((5 << 30, 2048),)), dict(pools=((6 << 30, 2048), ((6 << 30) + 4096, 2048))),
    dict(pools=((STATE["block_table"], 2048),))])
def test_eviction_arrays_that_overlap(lib, bad):
    assert evict_call(lib, **bad) == 2


def test_workspace_sizes(lib):
    assert lib.spec_kv4_workspace_size(-1) == 0 and lib.spec_kv4_workspace_size(1 << 20) > 0
    size = lib.spec_kv_evict_workspace_size
    assert size(-1, 2, 100) == 0 and size(2, 0, 100) == 0 and size(2, 4097, 100) == 0 and size(2, 2, 0) == 0
    assert size((1 << 16) + 1, 2, 100) == 0 and size(2, 2, (1 << 30) + 1) == 0 < size(2, 2, 1 << 30)
    assert 0 < size(0, 2, 100) <= size(1, 2, 100) < size(2, 2, 1000) < size(9, 3, 1000)


def test_binding_refuses():
    u8 = torch.zeros(4, 16, 2, 32, dtype=torch.uint8)
    hs, sc = torch.ones(2, 2), torch.zeros(4, 16, 2, 2, 4, dtype=torch.uint8)
    kv, one = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    bt = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(TypeError):  # host tensors
        api.spec_kv4_write(kv, kv, u8, u8, sc, hs, bt, one, one)
    with pytest.raises(TypeError):
        api.spec_kv4_read(u8, u8, sc, hs, bt, one, one, rows=3)
    with pytest.raises(TypeError):
        api.spec_verify_attn_kv4(kv, u8, u8, sc, hs, bt, one, one, max_draft_len=0, max_seq_len=9)
    with pytest.raises(TypeError):
        api.spec_attn_mass(kv, u8, bt, one, one, torch.zeros(1, 2, 9), max_draft_len=0, max_seq_len=9, kv_scale=hs,
                           scales=sc)
    with pytest.raises(TypeError):
        api.spec_kv_evict(one, bt, one, None, one, torch.zeros(1, 2, 9), block_size=16, pools=[])


def test_the_model_rounds_to_the_nearest():
    """Every code's values against a search over all pairs of scales and codes."""
    gen = torch.Generator().manual_seed(1)
    x = (torch.randn(40, 16, generator=gen) * 10.0 ** torch.randint(-3, 4, (40, 1), generator=gen)).to(torch.bfloat16)
    hs = torch.tensor(0.37)
    codes, scales = quantise(x, hs)
    got = values(codes, scales, hs)
    grid = e4m3_values()
    for i in range(40):
        want = x[i].double().abs().max() / (6 * float(hs))
        c = grid[(grid - want).abs().argmin()]
        assert abs(float(scales[i, 0].view(torch.float8_e4m3fn).double()) - float(c)) <= 1e-12
        if c > 0:
            mags = torch.tensor(E2M1, dtype=torch.float64)
            near = (x[i].double().abs()[:, None] / (float(hs) * c) - mags).abs().min(1).values
            assert torch.allclose((got[i] / (float(hs) * c)).sub(x[i].double() / (float(hs) * c)).abs(), near, atol=1e-9)


def test_the_model_keeps_the_heaviest():
    assert evict([0.0, 5.0, 1.0, 5.0, math.nan, 2.0], 6, 3, 1, 1) == [0, 1, 5]
    assert evict([1.0, 1.0, 1.0, 1.0], 4, 2, 0, 0) == [0, 1]


@pytest.mark.parametrize("last", [(1 << 32) + 5, -(1 << 32), 1 << 31])
def test_a_keep_last_that_32_bits_cannot_hold(last):
    """Refused: its low 32 bits are another number of positions."""
    one, bt = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="keep_last"):
        api.spec_kv_evict(one, bt, one, None, one, torch.zeros(1, 2, 9), block_size=16, pools=[], keep_last=last)
