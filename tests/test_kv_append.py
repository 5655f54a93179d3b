"""gdn_kv_append against its definition in 64 bits.

A rotated element y = a cos - b sin is off by at most (|a| + |b|) times: the angle's rounding
to fp32 (2^-24 pi), the sine and cosine (two units, 2^-23), a product, and a sum (2^-24 each),
all below 2^-20; plus the rounding to the cache's type, eps / 2 of y.  Values and dims that are
not rotated are copied bit for bit, and no other row of the cache or of q_out changes.
"""
from __future__ import annotations

import pytest
import torch

import linear_attention_token_b200 as gdn

from attn_ref import cache, normal

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rotated(x, angle, half):
    """x [T, H, d], angle [T, half] double -> (y, tolerance before the final rounding)."""
    x = x.double()
    y, tol = x.clone(), torch.zeros_like(x)
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = x[..., :half], x[..., half:2 * half]
    y[..., :half] = a * c - b * s
    y[..., half:2 * half] = b * c + a * s
    tol[..., :half] = tol[..., half:2 * half] = 2.0 ** -20 * (a.abs() + b.abs())
    return y, tol


def axis_of(i, sections, interleaved):
    n = len(sections)
    if interleaved:
        return i % n if i < n * sections[i % n] else 0
    run = 0
    for a, s in enumerate(sections):
        run += s
        if i < run:
            return a


def close(got, want, tol, dtype):
    half_step = torch.finfo(dtype).eps / 2
    return bool(((got.double() - want).abs() <= tol * (1 + half_step) + half_step * want.abs()).all())


CASES = [
    # lens, pos0, H_q, H_kv, d, page, rope, sections, interleaved, dtype
    ([1], [0], 2, 1, 64, 16, 64, None, False, torch.bfloat16),
    ([1] * 37, list(range(0, 370, 10)), 8, 2, 128, 16, 64, None, False, torch.bfloat16),
    ([5, 0, 33, 1], [15, 3, 0, 127], 4, 4, 128, 32, 128, None, False, torch.float32),
    ([700, 801, 900], [0, 64, 1_000_000], 6, 2, 128, 64, 64, None, False, torch.bfloat16),
    ([2049], [7], 0, 3, 64, 16, 32, None, False, torch.float32),
    ([9, 40], [1, 2], 4, 2, 128, 16, 128, (24, 20, 20), False, torch.bfloat16),
    ([9, 40], [1, 2], 4, 2, 64, 16, 64, (12, 10, 10), True, torch.float32),
    ([9, 40], [1, 2], 4, 2, 64, 16, 32, (10, 6), False, torch.float32),
    ([17, 3], [0, 5], 2, 2, 128, 1024, 0, None, False, torch.bfloat16),
    ([17, 3], [0, 5], 2, 2, 64, 16, 16, None, False, torch.bfloat16),
]


@pytest.mark.parametrize("lens,pos0,H_q,H_kv,d,page,rope,sections,interleaved,dtype", CASES)
def test_matches_definition(lens, pos0, H_q, H_kv, d, page, rope, sections, interleaved, dtype):
    N, T = len(lens), sum(lens)
    base = [p // page * page for p in pos0]                # pages below are not there
    kc, vc, table = cache(N, max(p - b + L for p, b, L in zip(pos0, base, lens)), H_kv, d, page,
                          dtype, 5, dead=3.0)
    wide = torch.full((N, max(b // page for b in base) + table.shape[1]), -1, dtype=torch.int32,
                      device=DEV)
    for n in range(N):
        wide[n, base[n] // page: base[n] // page + table.shape[1]] = table[n]
    kv = gdn.PagedKV(kc, vc, wide)
    tail = 3                                               # rows behind the last sequence
    k, v = normal((T + tail, H_kv, d), dtype, 1), normal((T + tail, H_kv, d), dtype, 2)
    q = normal((T + tail, H_q, d), dtype, 3) if H_q else None
    q_out = torch.full_like(q, 7.0) if H_q else None
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    freq = gdn.rope_inv_freq(rope) if rope else None
    pos = torch.cat([torch.arange(p, p + L) for p, L in zip(pos0, lens)]).to(DEV)
    rp = None
    if sections:
        g = torch.Generator().manual_seed(4)
        rp = torch.randint(0, 5000, (len(sections), T + tail), generator=g).to(torch.int32).to(DEV)
    want_k, want_v = kc.double(), vc.double()
    tol_k = torch.zeros_like(want_k)
    half = rope // 2
    angle = torch.zeros(T, half, dtype=torch.float64, device=DEV)
    for i in range(half):
        at = rp[axis_of(i, sections, interleaved), :T] if sections else pos
        angle[:, i] = at.double() * freq[i].double()
    yk, tk = rotated(k[:T], angle, half)
    seq = torch.repeat_interleave(torch.arange(N), torch.tensor(lens)).to(DEV)
    rows = wide.long()[seq, pos // page], pos % page
    want_k[rows], want_v[rows], tol_k[rows] = yk, v[:T].double(), tk
    gdn.gdn_kv_append(k, v, kv, cu, torch.tensor(pos0, dtype=torch.int32, device=DEV), q=q,
                      q_out=q_out, inv_freq=freq, rope_pos=rp, rope_sections=sections,
                      interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(vc.double(), want_v)
    assert close(kc, want_k, tol_k, dtype)
    untouched = torch.ones(kc.shape[:2], dtype=torch.bool, device=DEV)
    untouched[rows] = False
    assert bool((kc[untouched] == 3.0).all())
    if rope < d:
        assert torch.equal(kc[rows][..., rope:], k[:T, :, rope:])
    if H_q:
        yq, tq = rotated(q[:T], angle, half)
        assert close(q_out[:T], yq, tq, dtype)
        assert bool((q_out[T:] == 7.0).all())


def test_far_positions():
    """Angles of millions of radians: positions up to 2^31 - 1 on one axis."""
    d, half = 64, 32
    pos = torch.tensor([[1 << 20, 123_456_789, (1 << 31) - 1]], dtype=torch.int32, device=DEV)
    kc, vc, table = cache(1, 3, 1, d, 16, torch.float32, 0)
    kv = gdn.PagedKV(kc, vc, table)
    k = normal((3, 1, d), torch.float32, 1)
    freq = gdn.rope_inv_freq(d)
    gdn.gdn_kv_append(k, k, kv, q=k, inv_freq=freq, rope_pos=pos)
    # 31 + 24 bits of position x frequency are rounded to 53: 2^-53 2^31 more on the angle
    want, tol = rotated(k, pos[0].double()[:, None] * freq.double(), half)
    got = kc.view(-1, 1, d)[table[0, 0].long() * 16 + torch.arange(3, device=DEV)]
    assert close(got, want, tol + 2.0 ** -21 * tol.amax() * 2.0 ** 20, torch.float32)


def test_positions_past_32_bits():
    """Tokens behind the last 32-bit position are not in the cache; their queries are rotated there all
    the same, and not at a position that wrapped."""
    d, half, T = 64, 32, 5
    kc, vc, table = cache(1, 16, 1, d, 16, torch.float32, 0)
    kv = gdn.PagedKV(kc, vc, table)
    q = normal((T, 1, d), torch.float32, 1)
    # frequencies of few bits, so that position x frequency is exact in 64 bits
    freq = (2.0 ** -torch.arange(half, dtype=torch.float64)).float().to(DEV)
    start = (1 << 31) - 3
    out = gdn.gdn_kv_append(q, q, kv, None, torch.tensor([start], dtype=torch.int32, device=DEV), q=q,
                            inv_freq=freq)
    at = start + torch.arange(T, device=DEV).double()
    want, tol = rotated(q, at[:, None] * freq.double(), half)
    assert close(out, want, tol, torch.float32)
    assert bool(torch.isnan(kc).all()) and bool(torch.isnan(vc).all())


def test_strided_projection_and_in_place():
    """q, k, v as slices of one fused projection; q rotated in place where it is contiguous."""
    H_q, H_kv, d, T = 4, 2, 128, 50
    fused = normal((T, (H_q + 2 * H_kv) * d), torch.bfloat16, 1)
    q = fused[:, :H_q * d].view(T, H_q, d)
    k = fused[:, H_q * d:(H_q + H_kv) * d].view(T, H_kv, d)
    v = fused[:, (H_q + H_kv) * d:].view(T, H_kv, d)
    freq = gdn.rope_inv_freq(64)
    outs = []
    for split in (False, True):
        kc, vc, table = cache(1, T, H_kv, d, 16, torch.bfloat16, 0, dead=0.0)
        kv = gdn.PagedKV(kc, vc, table)
        if split:
            qc = q.contiguous()
            r = gdn.gdn_kv_append(k.contiguous(), v.contiguous(), kv, q=qc, q_out=qc, inv_freq=freq)
            assert r is qc
        else:
            r = gdn.gdn_kv_append(k, v, kv, q=q, inv_freq=freq)
        outs.append((r, kc, vc))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_absent_pages_and_negative_positions_are_not_written():
    kc, vc, table = cache(2, 64, 1, 64, 16, torch.bfloat16, 0, dead=3.0)
    table[0, 1], table[1, 2] = -1, kc.shape[0]             # out of range on both sides
    kv = gdn.PagedKV(kc, vc, table)
    k = normal((2, 80, 1, 64), torch.bfloat16, 1)          # 80 tokens: 16 past the table
    pos0 = torch.tensor([0, -8], dtype=torch.int32, device=DEV)
    gdn.gdn_kv_append(k, k, kv, None, pos0)
    want = torch.full_like(vc, 3.0)
    for n in range(2):
        for i in range(80):
            t = i + int(pos0[n])
            page = int(table[n, t // 16]) if 0 <= t < 64 else -1
            if 0 <= page < kc.shape[0]:
                want[page, t % 16] = k[n, i]
    assert torch.equal(vc, want)


def test_dense_batch_equals_packed():
    k, v = normal((3, 21, 2, 64), torch.bfloat16, 1), normal((3, 21, 2, 64), torch.bfloat16, 2)
    freq = gdn.rope_inv_freq(64)
    pos0 = torch.tensor([0, 3, 9], dtype=torch.int32, device=DEV)
    got = []
    for dense in (True, False):
        kc, vc, table = cache(3, 40, 2, 64, 16, torch.bfloat16, 0, dead=0.0)
        kv = gdn.PagedKV(kc, vc, table)
        if dense:
            gdn.gdn_kv_append(k, v, kv, None, pos0, inv_freq=freq)
        else:
            cu = torch.tensor([0, 21, 42, 63], dtype=torch.int32, device=DEV)
            gdn.gdn_kv_append(k.view(63, 2, 64), v.view(63, 2, 64), kv, cu, pos0, inv_freq=freq)
        got.append((kc, vc))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_many_sequences_offsets():
    """More sequences than one probe of the offsets covers, many of them empty."""
    g = torch.Generator().manual_seed(0)
    lens = torch.randint(0, 3, (1500,), generator=g).tolist()
    T = sum(lens)
    kc, vc, table = cache(1500, 16, 1, 64, 16, torch.float32, 0, dead=0.0)
    kv = gdn.PagedKV(kc, vc, table)
    k = normal((T, 1, 64), torch.float32, 1)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    gdn.gdn_kv_append(k, k, kv, cu)
    seq = torch.repeat_interleave(torch.arange(1500), torch.tensor(lens)).to(DEV)
    slot = torch.arange(T, device=DEV) - cu.long()[seq]
    assert torch.equal(kc[table.long()[seq, 0], slot], k)
    assert int((kc != 0).any(-1).sum()) == T


def test_row_offsets_past_32_bits():
    """A cache of more than 2^32 bytes per tensor: the last page is written where it is."""
    pages = (1 << 32) // (1024 * 8 * 128 * 2) + 2
    kc = torch.zeros(pages, 1024, 8, 128, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device=DEV)
    k = normal((40, 8, 128), torch.bfloat16, 1)
    gdn.gdn_kv_append(k, k, gdn.PagedKV(kc, vc, table))
    assert torch.equal(kc[-1, :40], k) and torch.equal(vc[-1, :40], k)
    assert not bool(kc[:-1].any()) and not bool(vc[-1, 40:].any())
