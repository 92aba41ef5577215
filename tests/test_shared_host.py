"""Host-side checks of spec_verify_attn_shared. CPU only."""
import ctypes

import pytest

from speculative_decoding_verification_gqa_gb300 import api, build

FAKE = 0x10000  # never dereferenced: checks fail before any launch


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load_library()


def desc(**kw):
    d = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, max_draft_len=3, max_seq_len=100,
             q_rows=8, kv_rows=0, kv_dtype=0, softmax_scale=0.0)
    d.update(kw)
    return api.AttnDesc(**d)


def call(lib, d, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, nb=32, bs=16, bt=FAKE, mb=8, T=FAKE, D=FAKE, ng=1, gb=FAKE, P=FAKE,
             sc=None, out=FAKE, ws=FAKE, bytes=1 << 40)
    a.update(kw)
    return lib.spec_verify_attn_shared(
        None if d is None else ctypes.byref(d), a["q"], a["k"], a["v"], a["nb"], a["bs"], a["bt"], a["mb"],
        a["T"], a["D"], a["ng"], a["gb"], a["P"], a["sc"], a["out"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(sliding_window=5), 2), (dict(head_dim=96), 2), (dict(num_q_heads=6, num_kv_heads=4), 2),
    (dict(max_draft_len=256), 2), (dict(batch=-1), 2), (dict(kv_dtype=3), 3)])
def test_bad_descriptors(lib, kw, status):
    assert call(lib, desc(**kw)) == status
    assert lib.spec_verify_attn_shared_workspace_size(ctypes.byref(desc(**kw)), 1) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(bs=12), 2), (dict(bs=4), 2), (dict(nb=0), 2), (dict(nb=1 << 28), 2), (dict(mb=0), 2),
    (dict(ng=0), 2), (dict(ng=3), 2), (dict(ng=-1), 2), (dict(gb=None), 1), (dict(P=None), 1),
    (dict(bt=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(sc=FAKE), 2),
    (dict(q=FAKE + 2), 4), (dict(P=FAKE + 1), 4), (dict(gb=FAKE + 2), 4), (dict(ws=FAKE + 16), 4)])
def test_bad_arguments(lib, kw, status):
    assert call(lib, desc(), **kw) == status


def test_null_descriptor_and_missing_scales(lib):
    assert call(lib, None) == 1
    assert call(lib, desc(kv_dtype=1)) == 1
    assert call(lib, desc(batch=0)) == 0  # nothing to do


def test_too_many_units_are_refused(lib):
    d = desc(batch=1 << 16, num_q_heads=4096, num_kv_heads=1, max_draft_len=255, q_rows=1 << 24)
    assert call(lib, d, ng=1) == 2
