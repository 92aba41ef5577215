"""E4M3 attention with several units a CTA and full rings, again and again: the stages of raw V
codes that the decoding warps give back to TMA hold the same bits in every call."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_verification_gqa_gb300 as sv
from speculative_decoding_verification_gqa_gb300 import synth

from gpu_util import assert_close, dev_attn, ensure_built
from shared_util import inputs, pages, to_device

pytestmark = pytest.mark.gpu

AGAIN = 40


@pytest.fixture(autouse=True)
def tcgen05():
    ensure_built()
    prev = sv.set_attn_kernel(2)
    yield
    sv.set_attn_kernel(prev)


def _batch(seed):
    """120 sequences of 4 KV heads and up to 128 rows a head: more than 3 units for each SM."""
    T, D = [(311 * b) % 701 for b in range(120)], [7 - b % 3 for b in range(120)]
    w = synth.Workload("rep", B=len(T), Hq=64, Hkv=4, d=128, D=0, T=0, V=8, p=0.5, kv_dtype="fp8_e4m3",
                       outlier_prob=0.001)
    return w, synth.attn_inputs(w, seed, seq_lens=np.array(T), draft_len=np.array(D))


@pytest.mark.parametrize("bs,window", [(0, 0), (0, 200), (16, 0), (64, 0), (64, 200)])
def test_e4m3_the_same_bits_every_time(bs, window):
    """Packed rows (bs 0) and pages, whose boxes outside a sequence TMA fills with zeros."""
    w, x = _batch(bs + window)
    q, k, v, sc, T, D = dev_attn(x)
    kw = dict(max_draft_len=int(x["draft_len"].max()), max_seq_len=int(x["seq_lens"].max()), kv_scale=sc,
              sliding_window=window)
    if bs:
        pg = synth.paged_layout(x, bs, seed=3, spare_blocks=5)
        k, v, table = (torch.from_numpy(pg[n]).cuda() for n in ("k_pages", "v_pages", "block_table"))
        call = lambda ws: sv.spec_verify_attn_paged(q, k, v, table, T, D, workspace=ws, **kw)  # noqa: E731
    else:
        call = lambda ws: sv.spec_verify_attn(q, k, v, T, D, workspace=ws, **kw)  # noqa: E731
    ws = sv.new_workspace(1 << 28)
    prev = sv.set_unit_ctas(0)  # the split line: ranges of several units
    try:
        first = call(ws)
        assert all(torch.equal(call(ws), first) for _ in range(AGAIN))
    finally:
        sv.set_unit_ctas(prev)
    assert sv.workspace_status(ws) == 0
    ref = oracle.verify_attn(x["q"], x["k"], x["v"], x["seq_lens"], x["draft_len"], Hq=w.Hq, Hkv=w.Hkv, d=w.d,
                             kv_scale=x["kv_scale"], window=window,
                             units=[(b, (5 * b) % 4) for b in range(0, 120, 7)])
    assert_close(first.view(torch.int16).cpu().numpy().view(np.uint16), ref)


@pytest.mark.parametrize("bs", [16, 64])
def test_e4m3_shared_prefixes_the_same_bits_every_time(bs):
    """24 groups of 5 sequences of up to 128 rows a KV head: more than 3 units of the sequences
    and nearly 2 of the prefixes for each SM."""
    groups = [((311 * g) % 701, [((311 * g) % 701 + (211 * (5 * g + b)) % 500, 7 - b % 3) for b in range(5)])
              for g in range(24)]
    w, x, gb, P = inputs(groups, Hq=64, Hkv=4, d=128, kv="fp8_e4m3", seed=bs)
    q, k, v, table, T, D, sc = to_device(x, pages(x, gb, P, bs, seed=bs))
    gb, P = torch.from_numpy(gb).cuda(), torch.from_numpy(P).cuda()
    ws = sv.new_workspace(1 << 28)

    def call():
        return sv.spec_verify_attn_shared(q, k, v, table, T, D, gb, P, max_draft_len=7, kv_scale=sc, workspace=ws,
                                          max_seq_len=int(x["seq_lens"].max()))

    first = call()
    assert all(torch.equal(call(), first) for _ in range(AGAIN))
    assert sv.workspace_status(ws) == 0
    ref = oracle.verify_attn(x["q"], x["k"], x["v"], x["seq_lens"], x["draft_len"], Hq=w.Hq, Hkv=w.Hkv, d=w.d,
                             kv_scale=x["kv_scale"], units=[(b, (5 * b) % 4) for b in range(0, 120, 7)])
    assert_close(first.view(torch.int16).cpu().numpy().view(np.uint16), ref)
