"""Inputs and bounds of the shared-prefix attention tests."""
import numpy as np
import torch

import oracle
import speculative_decoding_verification_gqa_gb300 as sv
from speculative_decoding_verification_gqa_gb300 import synth

from gpu_util import bf16_to_f64


def inputs(groups, *, Hq, Hkv, d, kv="bf16", seed=0):
    """groups: a list of (P, [(T, D), ...]). Packed inputs in which the sequences of a group
    hold the first one's K/V at positions before P. Returns (workload, x, group_begin, P)."""
    T = [t for _, seqs in groups for t, _ in seqs]
    D = [n for _, seqs in groups for _, n in seqs]
    w = synth.Workload("sh", B=len(T), Hq=Hq, Hkv=Hkv, d=d, D=0, T=0, V=8, p=0.5, kv_dtype=kv,
                       outlier_prob=0.001 if kv != "bf16" else 0.0)
    x = synth.attn_inputs(w, seed, seq_lens=np.array(T), draft_len=np.array(D))
    gb = np.cumsum([0] + [len(s) for _, s in groups]).astype(np.int32)
    P = np.array([p for p, _ in groups], dtype=np.int32)
    off = np.cumsum([0] + [t + n + 1 for t, n in zip(T, D)])
    for n, p in enumerate(P):
        for b in range(gb[n] + 1, gb[n + 1]):
            for a in (x["k"], x["v"]):
                a[off[b]:off[b] + p] = a[off[gb[n]]:off[gb[n]] + p]
    return w, x, gb, P


def pages(x, gb, P, bs, seed, junk=-1):
    """The paged layout, with what must not be read spoilt: the entries of all but a group's
    first sequence for blocks wholly before P are `junk`, those blocks hold NaN, and so do
    the positions before P of the block that P falls into (in the others' own copies)."""
    pg = synth.paged_layout(x, bs, seed=seed, spare_blocks=3)
    nan = 0x7F if x["k"].dtype == np.uint8 else 0x7FC0
    for n, p in enumerate(P):
        for b in range(gb[n] + 1, gb[n + 1]):
            row = pg["block_table"][b]
            for a in (pg["k_pages"], pg["v_pages"]):
                a[row[:p // bs]] = nan
                if p % bs:
                    a[row[p // bs], :p % bs] = nan
            row[:p // bs] = junk
    return pg


def to_device(x, pg):
    q = torch.from_numpy(x["q"].view(np.int16)).view(torch.bfloat16).cuda()
    if x["k"].dtype == np.uint8:
        k, v = (torch.from_numpy(pg[n]).cuda() for n in ("k_pages", "v_pages"))
        sc = torch.from_numpy(x["kv_scale"]).cuda()
    else:
        k, v = (torch.from_numpy(pg[n].view(np.int16)).view(torch.bfloat16).cuda()
                for n in ("k_pages", "v_pages"))
        sc = None
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    return q, k, v, i32(pg["block_table"]), i32(x["seq_lens"]), i32(x["draft_len"]), sc


def run(x, pg, gb, P, *, workspace=None, out=None, max_draft=None, max_seq=None, **kw):
    q, k, v, bt, T, D, sc = to_device(x, pg)
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    o = sv.spec_verify_attn_shared(
        q, k, v, bt, T, D, i32(gb), i32(P), kv_scale=sc, workspace=workspace, out=out,
        max_draft_len=int(x["draft_len"].max()) if max_draft is None else max_draft,
        max_seq_len=int(x["seq_lens"].max()) if max_seq is None else max_seq, **kw)
    torch.cuda.synchronize()
    return o.view(torch.int16).cpu().numpy().view(np.uint16)


def reference(w, x):
    """(out, spread): the fp64 result, and the same softmax over |V|, which bounds what
    rounding the probabilities can change."""
    kw = dict(Hq=w.Hq, Hkv=w.Hkv, d=w.d, kv_scale=x["kv_scale"])
    mag = x["v"] & (0x7F if x["v"].dtype == np.uint8 else 0x7FFF)
    return (oracle.verify_attn(x["q"], x["k"], x["v"], x["seq_lens"], x["draft_len"], **kw),
            oracle.verify_attn(x["q"], x["k"], mag.astype(x["v"].dtype), x["seq_lens"], x["draft_len"], **kw))


def assert_within(bits, w, x, what=""):
    """|got - ref| <= 2^-8 |ref| + (2^-8 + 2^-10) A, with A = sum p |v|. The output is rounded
    once to bf16 (half a step: 2^-8 of the value), each probability once to bf16 or f16 (at
    most 2^-8 of it: 2^-8 A); the sums and the joins are fp32, and the scores' fp32 sums over
    d <= 128 products of N(0, 1) (sum |q k| about 100, scaled by 1/8 or less) and, for E4M3,
    Q held to 2^-17 of its row's maximum, change a probability by less than 2^-11 of it; the
    sum that divides changes by as much: 2^-10 A."""
    ref, mag = reference(w, x)
    got = bf16_to_f64(bits[:ref.shape[0]])
    assert np.isfinite(got).all(), what
    bound = np.abs(ref) * 2.0 ** -8 + mag * (2.0 ** -8 + 2.0 ** -10)
    over = np.abs(got - ref) / bound
    print("%s worst error over bound %.3f" % (what, over.max()))
    assert over.max() <= 1.0, "%s: %.3f of the bound at %s" % (
        what, over.max(), np.unravel_index(over.argmax(), over.shape))
