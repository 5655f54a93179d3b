"""Refusals of the paged-cache operators: the C ABI rejects bad arguments before anything is
enqueued, and the Python binding rejects operands that do not match before a pointer is taken.
Runs on the CPU."""
from __future__ import annotations

import ctypes

import pytest
import torch

import linear_attention_token_b200 as gdn
from linear_attention_token_b200 import build as gdn_build
from linear_attention_token_b200._binding import _PagedKVStruct

A = 0x7f0000000000                     # device-looking, never dereferenced
P = ctypes.c_void_p
BAD, UNSUPPORTED = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def L():
    gdn_build.build()
    return gdn.lib()


def paged(**over):
    a = dict(k=A, v=A + (1 << 30), page_table=A + (1 << 31), num_pages=8, max_pages=4, page_size=16,
             H_kv=2, d=128, dtype=1)
    a.update({n: over.pop(n) for n in list(over) if n in a})
    return ctypes.byref(_PagedKVStruct(*a.values())), over


PAGED = [(dict(dtype=5), BAD), (dict(num_pages=-1), BAD), (dict(max_pages=-1), BAD),
         (dict(H_kv=0), BAD), (dict(d=96), UNSUPPORTED), (dict(d=0), BAD),
         (dict(page_size=24), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
         (dict(page_size=2048), UNSUPPORTED), (dict(k=None), BAD), (dict(v=A + 8), BAD),
         (dict(page_table=None), BAD), (dict(page_table=A + 2), BAD),
         (dict(num_pages=1 << 28), UNSUPPORTED), (dict(max_pages=1 << 28), UNSUPPORTED),
         (dict(num_seqs=-1), BAD)]


def append(L, **over):
    kv, over = paged(**over)
    a = dict(tk=A, tv=A, q=A, q_out=A, ks=256, vs=256, qs=512, cu=None, pos0=None, num_seqs=2, T=64,
             H_q=4, inv_freq=A, rope=64, rope_pos=None, sections=None, axes=1, flags=0)
    a.update(over)
    sec = (ctypes.c_int32 * 3)(*a["sections"]) if a["sections"] else None
    return L.gdn_kv_append(kv, P(a["tk"]), P(a["tv"]), P(a["q"]), P(a["q_out"]), a["ks"], a["vs"],
                           a["qs"], P(a["cu"]), P(a["pos0"]), a["num_seqs"], a["T"], a["H_q"],
                           P(a["inv_freq"]), a["rope"], P(a["rope_pos"]), sec, a["axes"],
                           a["flags"], None)


@pytest.mark.parametrize("over,expect", PAGED + [
    (dict(T=-1), BAD), (dict(T=1 << 31), BAD), (dict(T=65), BAD),        # 65 tokens, 2 sequences
    (dict(num_seqs=0), BAD), (dict(flags=2), BAD), (dict(rope=144), BAD), (dict(rope=24), BAD),
    (dict(rope=-16), BAD), (dict(inv_freq=None), BAD), (dict(axes=0), BAD), (dict(axes=4), BAD),
    (dict(axes=3), BAD), (dict(axes=3, rope_pos=A), BAD),
    (dict(axes=3, rope_pos=A, sections=(16, 8, 7)), BAD),
    (dict(axes=3, rope_pos=A, sections=(40, -4, -4)), BAD),
    (dict(tk=None), BAD), (dict(q_out=None), BAD), (dict(q=None), BAD), (dict(H_q=0), BAD),
    (dict(ks=260), BAD), (dict(qs=511), BAD), (dict(tv=A + 4), BAD), (dict(cu=A + 2), BAD),
    (dict(pos0=A + 1), BAD), (dict(H_q=1 << 20), UNSUPPORTED)])
def test_append_rejects(L, over, expect):
    assert append(L, **over) == expect


def test_append_nothing_to_do(L):
    assert append(L, T=0, tk=None, tv=None, q=None, q_out=None) == gdn.GDN_OK
    assert append(L, T=0, num_seqs=0) == gdn.GDN_OK


def decode(L, listed=False, **over):
    kv, over = paged(**over)
    a = dict(q=A, q_pos=A, out=A, lse=A, num_seqs=3, T=1, H_q=4, scale=1.0, cap=0.0, window=0,
             ws=A, ws_bytes=1 << 40, list=A, list_len=64, recent=4)
    a.update(over)
    if listed:
        return L.gdn_qsa_attn_decode(P(a["q"]), P(a["q_pos"]), kv, P(a["list"]), a["list_len"],
                                     a["recent"], P(a["out"]), P(a["lse"]), a["num_seqs"], a["T"],
                                     a["H_q"], a["scale"], a["cap"], P(a["ws"]), a["ws_bytes"], None)
    return L.gdn_attn_decode(P(a["q"]), P(a["q_pos"]), kv, P(a["out"]), P(a["lse"]), a["num_seqs"],
                             a["T"], a["H_q"], a["scale"], a["cap"], a["window"], P(a["ws"]),
                             a["ws_bytes"], None)


DECODE = PAGED + [
    (dict(T=0), UNSUPPORTED), (dict(T=9), UNSUPPORTED), (dict(H_q=3), BAD), (dict(H_q=0), BAD),
    (dict(H_q=8192), UNSUPPORTED), (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD),
    (dict(cap=-1.0), BAD), (dict(cap=float("nan")), BAD), (dict(cap=1e-5), BAD), (dict(cap=1e7), BAD),
    (dict(q=None), BAD), (dict(q=A + 2), BAD),
    (dict(q_pos=None), BAD), (dict(q_pos=A + 2), BAD), (dict(out=None), BAD), (dict(lse=A + 2), BAD),
    (dict(ws=None), BAD), (dict(ws=A + 8), BAD), (dict(ws_bytes=1024), BAD)]


@pytest.mark.parametrize("over,expect", DECODE + [(dict(window=-1), BAD)])
def test_decode_rejects(L, over, expect):
    assert decode(L, **over) == expect


@pytest.mark.parametrize("over,expect", DECODE + [
    (dict(list=None), BAD), (dict(list=A + 1), BAD), (dict(list_len=-1), BAD),
    (dict(list_len=16385), UNSUPPORTED), (dict(recent=-1), BAD), (dict(recent=65537), UNSUPPORTED)])
def test_listed_rejects(L, over, expect):
    assert decode(L, listed=True, **over) == expect


def test_decode_of_no_sequences_is_a_no_op(L):
    assert decode(L, num_seqs=0) == gdn.GDN_OK
    assert decode(L, listed=True, num_seqs=0) == gdn.GDN_OK


def test_decode_workspace_size(L):
    # per CTA (two per SM): a 16-byte record and two parts of `block` rows of d + 2 floats
    # (from 33 rows on, 64 KB more)
    for rows, block in ((1, 16), (16, 16), (17, 32), (33, 64), (64, 64), (500, 64)):
        n = gdn.gdn_attn_decode_workspace_size(1, rows, 1, 128) - (65536 if rows > 32 else 0)
        assert n > 0 and n % (2 * (16 + 2 * block * 130 * 4)) == 0
    assert gdn.gdn_attn_decode_workspace_size(9, 4, 2, 128) == 0
    assert gdn.gdn_attn_decode_workspace_size(1, 3, 2, 128) == 0
    assert gdn.gdn_attn_decode_workspace_size(1, 4, 2, 96) == 0


def prefill(L, **over):
    kv, over = paged(**over)
    a = dict(q=A, cu=None, pos0=None, prefix=None, out=A, lse=None, num_seqs=2, T=64, H_q=4, scale=1.0,
             cap=0.0, window=0, ws=None, ws_bytes=0)
    a.update(over)
    return L.gdn_attn_prefill(P(a["q"]), kv, P(a["cu"]), P(a["pos0"]), P(a["prefix"]), P(a["out"]),
                              P(a["lse"]), a["num_seqs"], a["T"], a["H_q"], a["scale"], a["cap"],
                              a["window"], P(a["ws"]), a["ws_bytes"], None)


@pytest.mark.parametrize("over,expect", PAGED + [
    (dict(T=-1), BAD), (dict(T=1 << 31), BAD), (dict(T=65), BAD), (dict(num_seqs=0), BAD),
    (dict(H_q=3), BAD), (dict(H_q=0), BAD), (dict(H_q=8192), UNSUPPORTED),
    (dict(scale=float("nan")), BAD), (dict(cap=-1.0), BAD), (dict(cap=float("inf")), BAD),
    (dict(window=-1), BAD), (dict(window=8, prefix=A), UNSUPPORTED), (dict(q=None), BAD),
    (dict(q=A + 2), BAD), (dict(out=None), BAD), (dict(cu=A + 2), BAD), (dict(pos0=A + 2), BAD),
    (dict(prefix=A + 2), BAD), (dict(lse=A + 2), BAD), (dict(ws=A, ws_bytes=8), BAD),
    (dict(ws=A + 8, ws_bytes=64), BAD)])
def test_prefill_rejects(L, over, expect):
    assert prefill(L, **over) == expect


def test_prefill_nothing_to_do(L):
    assert prefill(L, T=0, q=None, out=None) == gdn.GDN_OK
    assert prefill(L, T=0, num_seqs=0) == gdn.GDN_OK


# --------------------------------------------------------------------------- the binding
def _kv(dtype=torch.bfloat16, N=2):
    k = torch.zeros(4, 16, 2, 64, dtype=dtype)
    return gdn.PagedKV(k, k.clone(), torch.zeros(N, 2, dtype=torch.int32))


def test_cache_refusals():
    k, t = torch.zeros(4, 16, 2, 64), torch.zeros(2, 2, dtype=torch.int32)
    for bad, exc in (((k[0], k[0], t), ValueError), ((k, k[:2], t), ValueError),
                     ((k, k.bfloat16(), t), TypeError), ((k.half(), k.half(), t), TypeError),
                     ((k, k, t.long()), TypeError), ((k, k, t[0]), ValueError),
                     ((k.transpose(1, 2), k.transpose(1, 2), t), ValueError),
                     ((k, k.to("meta"), t), ValueError), ((k, k, t[:, ::2]), ValueError)):
        with pytest.raises(exc):
            gdn.PagedKV(*bad)


def test_append_binding_refusals():
    kv, i32 = _kv(), torch.int32
    k = torch.zeros(6, 2, 64, dtype=torch.bfloat16)
    cu, freq = torch.tensor([0, 2, 6], dtype=i32), torch.ones(32)
    ok = dict(cu_seqlens=cu, q=torch.zeros(6, 4, 64, dtype=torch.bfloat16), inv_freq=freq)
    for over, exc, match in (
            (dict(cu_seqlens=cu.long()), TypeError, "int32"),
            (dict(cu_seqlens=torch.zeros(4, dtype=i32)), ValueError, "page_table has 2 rows"),
            (dict(pos0=torch.zeros(3, dtype=i32)), ValueError, "pos0"),
            (dict(q=torch.zeros(5, 4, 64, dtype=torch.bfloat16)), ValueError, "q has shape"),
            (dict(q=torch.zeros(6, 4, 64)), TypeError, "q must have the cache's dtype"),
            (dict(q=torch.zeros(6, 64, 4, dtype=torch.bfloat16).transpose(1, 2)), ValueError, "contig"),
            (dict(q=None, q_out=k), ValueError, "q_out needs q"),
            (dict(inv_freq=None, rope_pos=cu), ValueError, "need inv_freq"),
            (dict(rope_sections=(16, 8, 8)), ValueError, "need rope_pos"),
            (dict(rope_sections=(8, 8, 8, 8), rope_pos=cu), ValueError, "1 to 3"),
            (dict(), ValueError, "no CPU path")):
        with pytest.raises(exc, match=match):
            gdn.gdn_kv_append(k, k, kv, **{**ok, **over})
    with pytest.raises(ValueError, match="v has shape"):
        gdn.gdn_kv_append(k, k[:5], kv, cu)
    with pytest.raises(ValueError, match="evenly spaced"):
        x = torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16)[:, :3]
        gdn.gdn_kv_append(x, x, kv)


def test_decode_binding_refusals():
    kv, i32, bf = _kv(), torch.int32, torch.bfloat16
    q, pos = torch.zeros(2, 1, 4, 64, dtype=bf), torch.zeros(2, dtype=i32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="no CPU path"):
        gdn.gdn_attn_decode(q, pos, kv, workspace=ws)
    for args, exc, match in (((q[0], pos, kv), ValueError, "n_queries"),
                             ((q.float(), pos, kv), TypeError, "q must be"),
                             ((torch.zeros(3, 1, 4, 64, dtype=bf), pos, kv), ValueError, "rows for 3")):
        with pytest.raises(exc, match=match):
            gdn.gdn_attn_decode(*args, workspace=ws)


def test_prefill_binding_refusals():
    kv, i32, bf = _kv(), torch.int32, torch.bfloat16
    q, cu = torch.zeros(6, 4, 64, dtype=bf), torch.tensor([0, 2, 6], dtype=i32)
    for over, exc, match in (
            (dict(), ValueError, "no CPU path"), (dict(cu_seqlens=cu.long()), TypeError, "int32"),
            (dict(cu_seqlens=torch.zeros(4, dtype=i32)), ValueError, "page_table has 2 rows"),
            (dict(pos0=torch.zeros(3, dtype=i32)), ValueError, "pos0"),
            (dict(prefix_len=torch.zeros(2)), TypeError, "prefix_len"),
            (dict(out=torch.zeros(6, 4, 64)), TypeError, "out"),
            (dict(lse=torch.zeros(6, 3)), ValueError, "lse"),
            (dict(workspace=torch.zeros(64, device="meta")), ValueError, "workspace")):
        with pytest.raises(exc, match=match):
            gdn.gdn_attn_prefill(q, kv, **{**dict(cu_seqlens=cu), **over})
    with pytest.raises(ValueError, match="head dim"):
        gdn.gdn_attn_prefill(q[..., :32].contiguous(), kv, cu)
    with pytest.raises(ValueError, match="contiguous"):
        gdn.gdn_attn_prefill(q.transpose(0, 1).contiguous().transpose(0, 1), kv, cu)
