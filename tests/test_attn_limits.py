"""The paged attention at the ends of what its arguments allow: caps and scales that leave little of
fp32's range, positions at the end of 32 bits, one workspace for every call, and parts of a long
sequence that each have to arrive.  Inputs are chosen so that the exact answer is known well below a
kernel's rounding; each tolerance stands beside the roundings it counts (u = 2^-24, half a step of fp32;
bf16: 2^-8)."""
from __future__ import annotations

import math

import pytest
import torch

import linear_attention_token_b200 as gdn

from attn_ref import attend, cache, check, fill, normal

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def one_hot(dots, heads, d, dtype, seed=0):
    """A cache of len(dots) tokens (one key head) whose key t has dots[t] in dim 0 and noise elsewhere, and
    the values; a query with a power of two in dim 0 and zeros elsewhere then has an exact dot product."""
    g = torch.Generator().manual_seed(seed)
    n, page = len(dots), 64
    pages = -(-n // page)
    k = torch.zeros(pages, page, 1, d, dtype=dtype, device=DEV)
    k.view(-1, d)[:n] = torch.randn(n, d, generator=g).to(dtype).to(DEV)
    k.view(-1, d)[:n, 0] = torch.as_tensor(dots).to(dtype).to(DEV)
    v = torch.zeros_like(k)
    v.view(-1, d)[:n] = torch.randn(n, d, generator=g).to(dtype).to(DEV)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    return gdn.PagedKV(k, v, table), k.view(-1, d)[:n, 0].double(), v.view(-1, d)[:n].double()


def capped_softmax(dot, seen, v, scale, cap):
    """The definition in 64 bits: dot [n] or [R, n], seen [R, n] -> out [R, d], lse [R], sum w |v|."""
    x = (cap * torch.tanh(dot * scale / cap)).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(x, -1)
    w = torch.exp(x - lse[:, None])
    return w @ v, lse, w @ v.abs()


def close(got, want, tol, what):
    e = (got.double() - want).abs()
    assert bool((e <= tol).all()), f"{what}: off by {float((e / tol).max()):.3g} of its tolerance"


# ------------------------------------------------------------------------- the end of 32 bits
@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_last_positions(page, dtype):
    """A table up to the last 32-bit position that pages reach, its first pages freed, and queries at its
    end (some behind it) with a window: what a tile covers would not fit 32 bits."""
    H_q, H_kv, d, L, window = 4, 2, 64, 90, 150
    per = (2 ** 31 - 1) // page
    end = per * page                                         # the table holds tokens 0 .. end - 1
    used = -(-512 // page)
    kc, vc, small = cache(1, used * page, H_kv, d, page, dtype, 1)
    table = torch.full((1, per), -1, dtype=torch.int32, device=DEV)
    table[0, per - used:] = small[0]
    kv = gdn.PagedKV(kc, vc, table)
    first = end - used * page                                # the oldest token the cache holds
    ks, vs = fill(kc, vc, small, [used * page], 3)
    k, v, t = ks[0], vs[0], torch.arange(used * page, device=DEV) + first
    q = normal((L, H_q, d), dtype, 5)
    for start in (end - L, end - 60, end - L - 100):
        at = torch.arange(start, start + L, device=DEV)[:, None]
        out, lse = gdn.gdn_attn_prefill(q, kv, ints(0, L), ints(start), window=window)
        small_out, small_lse = gdn.gdn_attn_prefill(q, kv, ints(0, L), ints(start), window=window,
                                                    workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))
        for h in range(H_q):
            want = attend(q[:, h], k[:, h // 2], v[:, h // 2], (t <= at) & (t > at - window), d ** -0.5, 0.0, dtype == BF)
            check(out[:, h], lse[:, h], want, f"start {start - end} head {h}")
            check(small_out[:, h], small_lse[:, h], want, f"in one piece: start {start - end} head {h}")
    for T, G in ((1, 2), (4, 2), (8, 32)):                   # (8 x 32 rows run on the prompt kernel in bf16)
        N = 4
        wide = gdn.PagedKV(kc, vc, table.expand(N, per).contiguous()) if page > 16 and G > 2 else kv
        n = wide.page_table.shape[0]
        q = normal((n, T, G * H_kv, d), dtype, 6)
        for start in (end - T, end - 1):
            out, lse = gdn.gdn_attn_decode(q, torch.full((n,), start, dtype=torch.int32, device=DEV), wide, window=window)
            at = torch.arange(start, start + T, device=DEV)[:, None]
            for h in range(G * H_kv):
                want = attend(q[0, :, h], k[:, h // G], v[:, h // G], (t <= at) & (t > at - window), d ** -0.5, 0.0, dtype == BF)
                check(out[0, :, h], lse[0, :, h], want, f"decode {T} x {G}: start {start - end} head {h}")


# ------------------------------------------------------------------------------ caps and scales
@pytest.mark.parametrize("scale,cap", [(1e9, 1e6), (-1e9, 1e6), (2e8, 2e5), (6e9, 1e6), (1e9, 1e5), (30.0, 30.0),
                                       (1e-3, 20.0), (3e13, 1e6)])
@pytest.mark.parametrize("d", [64, 128])
def test_caps_beside_large_scales(scale, cap, d):
    """Scores on both sides of half the cap, in whole tiles, with scales that no model has.  A score is off
    by 2^-20 of itself (the cap's polynomials and roundings), and equal dot products of a whole and of a
    masked tile go through different polynomials, so
      out  a weight beside another is off by a factor e^dx, dx = 2 2^-20 cap; it is rounded to bf16 for
           the product (2^-8), the sum takes it unrounded, and out is rounded (2^-8); n u for sums;
      lse  2^-20 of the largest score, n u of the sum."""
    n, R, H = 450, 150, 4
    levels = torch.tensor([0.25, 0.5, 0.625, 0.75, 0.875, 1.0])
    g = torch.Generator().manual_seed(int(d))
    dots = levels[torch.randint(0, 6, (n,), generator=g)] * (torch.randint(0, 2, (n,), generator=g) * 2 - 1)
    dots[::7] = 0.125
    kv, k0, v = one_hot(dots, H, d, BF)
    q0 = 2.0 ** math.floor(math.log2(cap / abs(scale)))      # largest |score| 0.5 .. 1 of the cap
    q = torch.zeros(R, H, d, dtype=BF, device=DEV)
    q[:, :, 0] = torch.tensor([q0, q0 / 2, -q0, q0 / 4], device=DEV)
    t = torch.arange(n, device=DEV)
    seen = t <= torch.arange(n - R, n, device=DEV)[:, None]
    dx = 2 * 2.0 ** -20 * cap
    out, lse = gdn.gdn_attn_prefill(q, kv, ints(0, R), ints(n - R), scale=scale, softcap=cap)
    for h in range(H):
        o, l, mag = capped_softmax(k0 * float(q[0, h, 0]), seen, v, scale, cap)
        close(out[:, h], o, (2.0 ** -8 + n * U + math.expm1(dx)) * mag + 2.0 ** -8 * o.abs() + 1e-30, f"out {h}")
        close(lse[:, h], l, 2.0 ** -20 * (cap + l.abs()) + n * U, f"lse {h}")
    last, lse1 = gdn.gdn_attn_decode(q[-1:, None].contiguous().view(1, 1, H, d), ints(n - 1), kv, scale=scale, softcap=cap)
    for h in range(H):
        o, l, mag = capped_softmax(k0 * float(q[0, h, 0]), seen[-1:], v, scale, cap)
        close(last[0, :, h], o, (2.0 ** -8 + n * U + math.expm1(dx)) * mag + 2.0 ** -8 * o.abs() + 1e-30, f"decode out {h}")
        close(lse1[0, :, h], l, 2.0 ** -20 * (cap + l.abs()) + n * U, f"decode lse {h}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale,cap", [(1e35, 1e-4), (-3e38, 1e-4), (3e38, 1.0)])
def test_zero_scores_beside_quotients_past_fp32(scale, cap, dtype):
    """scale / cap does not fit fp32: a score is 0 where the dot product is, and the cap with its sign
    elsewhere.  out: weights and result rounded (bf16 2^-8, fp32 8 u: exponential 4 u, sums n u); lse the
    same beside a score of at most 1."""
    n, H, d = 300, 2, 64
    dots = torch.tensor([0.0, 1.0, -1.0, 0.5, 0.0])[torch.arange(n) % 5]
    kv, k0, v = one_hot(dots, H, d, dtype)
    q = torch.zeros(2, H, d, dtype=dtype, device=DEV)
    q[:, 1, 0] = 2.0                                         # head 0: every dot product is 0
    seen = torch.arange(n, device=DEV) <= torch.tensor([[n - 2], [n - 1]], device=DEV)
    half = 2.0 ** -8 if dtype == BF else U
    got = [gdn.gdn_attn_prefill(q, kv, ints(0, 2), ints(n - 2), scale=scale, softcap=cap),
           [x[0] for x in gdn.gdn_attn_decode(q[None], ints(n - 2), kv, scale=scale, softcap=cap)]]
    for out, lse in got:
        for h in range(H):
            o, l, mag = capped_softmax(k0 * 2.0 * h, seen, v, scale, cap)
            close(out[:, h], o, (half + (n + 40) * U) * mag + half * o.abs() + 1e-30, f"out {h}")
            close(lse[:, h], l, (n + 40) * U + 4 * U * l.abs(), f"lse {h}")


@pytest.mark.parametrize("rows", [1, 4, 8])
@pytest.mark.parametrize("most", [1.0, 3.0])
def test_cap_in_fp32(most, rows):
    """One token a sequence, so lse is its capped score.  The dot product and its quotient with a cap of 32
    are exact; then cap2 = 32 log2 e (u), y R(y^2) by the polynomial (4.3 u: y^2 .3, the outermost sum 1,
    the inner ones .6, coefficients .7, fit .1, the product 1, and the one with cap2 1 more) or
    1 - 2 / (1 + e^2y) beyond 1 (4.8 u: 2y log2 e, ex2, the sum and the quotient make 3.8 u of the
    result, the last sum 1), and ln 2 and its product (2 u): 8 u of the score."""
    N, d, cap = 512, 64, 32.0
    kv, k0, v = one_hot(torch.ones(64 * N), rows, d, F32)
    kv = gdn.PagedKV(kv.k, kv.v, torch.arange(N, dtype=torch.int32, device=DEV)[:, None].contiguous())
    q = torch.zeros(N, 1, rows, d, device=DEV)
    g = torch.Generator().manual_seed(rows)
    q[..., 0] = ((torch.rand(N, 1, rows, generator=g) * 2 - 1) * most * cap).to(DEV)
    want = cap * torch.tanh(q[..., 0].double() / cap)
    _, lse = gdn.gdn_attn_decode(q, torch.zeros(N, dtype=torch.int32, device=DEV), kv, scale=1.0, softcap=cap)
    close(lse, want, 8 * U * want.abs() + 1e-30, "decode")
    _, lse = gdn.gdn_attn_prefill(q, kv, None, None, scale=1.0, softcap=cap)
    close(lse, want, 8 * U * want.abs() + 1e-30, "prompt")


# ----------------------------------------------------------------------------------- one workspace
def zeros_cache(N, H_kv, d, tokens, dtype=BF):
    k = torch.zeros(4, 64, H_kv, d, dtype=dtype, device=DEV)
    table = (torch.arange(N * (tokens // 64), dtype=torch.int32, device=DEV) % 4).view(N, -1)
    return gdn.PagedKV(k, torch.zeros_like(k), table)


def test_decode_leaves_the_error_word_alone():
    """One zeroed workspace: an even split of more units than CTAs, then drafts on the prompt kernel with
    no polls allowed, then both again.  Only the call that gave up is reported, and is."""
    many = zeros_cache(700, 1, 64, 512), torch.zeros(700, 1, 4, 64, dtype=BF, device=DEV)
    wide = zeros_cache(8, 1, 64, 512), torch.zeros(8, 8, 16, 64, dtype=BF, device=DEV)
    n = max(gdn.gdn_attn_decode_workspace_size(q.shape[1], q.shape[2], 1, 64) for _, q in (many, wide))
    ws = gdn.attn_decode_workspace(8, 16, 1, 64)             # the larger of the two
    assert ws.numel() == n

    def call(kv, q):
        at = torch.full((q.shape[0],), 512 - q.shape[1], dtype=torch.int32, device=DEV)
        gdn.gdn_attn_decode(q, at, kv, workspace=ws)
        return gdn.gdn_get_device_error(ws)

    assert call(*many) == gdn.GDN_OK
    assert call(*wide) == gdn.GDN_OK
    old = gdn.gdn_set_wait_budget(0)
    try:
        assert call(*wide) == gdn.GDN_ERR_TIMEOUT
    finally:
        gdn.gdn_set_wait_budget(old)
    assert call(*many) == gdn.GDN_OK
    assert call(*wide) == gdn.GDN_OK
    kv, q = wide                                             # and a prompt on the same scratch
    call(*many)
    gdn.gdn_attn_prefill(q, kv, None, None, workspace=ws)
    assert gdn.gdn_get_device_error(ws) == gdn.GDN_OK


@pytest.mark.parametrize("T,G", [(4, 16), (8, 16)])
def test_wide_tables_keep_the_even_split(T, G):
    """Drafts of many rows run on the prompt kernel only where no sequence can be far longer than the rest:
    its waits (none allowed here) give up, the even split has none.  One long sequence among short ones is
    right either way."""
    N, H_kv, d = 8, 1, 64
    q = torch.zeros(N, T, G * H_kv, d, dtype=BF, device=DEV)
    at = torch.full((N,), 500 - T, dtype=torch.int32, device=DEV)
    narrow = zeros_cache(N, H_kv, d, 512)
    wide = gdn.PagedKV(narrow.k, narrow.v, torch.zeros(N, 1 << 15, dtype=torch.int32, device=DEV))
    ws = gdn.attn_decode_workspace(T, G * H_kv, H_kv, d)
    old = gdn.gdn_set_wait_budget(0)
    try:
        for kv, window, want in ((narrow, 0, gdn.GDN_ERR_TIMEOUT), (wide, 0, gdn.GDN_OK),
                                 (wide, 1000, gdn.GDN_ERR_TIMEOUT)):
            gdn.gdn_attn_decode(q, at, kv, window=window, workspace=ws)
            assert gdn.gdn_get_device_error(ws) == want
    finally:
        gdn.gdn_set_wait_budget(old)
    kv, dots, v = one_hot(torch.tensor([0.0, 1.0, -1.0, 0.5])[torch.arange(20_000) % 4], G, d, BF)
    table = torch.full((N, 1 << 15), -1, dtype=torch.int32, device=DEV)
    table[:, :kv.page_table.shape[1]] = kv.page_table
    lens = [20_000] + [30 + n for n in range(N - 1)]
    q[..., 0] = 1.0
    out, lse = gdn.gdn_attn_decode(q, ints(*lens) - T, gdn.PagedKV(kv.k, kv.v, table), scale=1.0)
    for n, L in enumerate(lens):
        for j in range(T):
            x = dots[:L - T + j + 1]
            want = torch.exp(x - torch.logsumexp(x, 0)) @ v[:len(x)]
            mag = torch.exp(x - torch.logsumexp(x, 0)) @ v[:len(x)].abs()
            # weights and result rounded to bf16; exponentials 4 u and the sums n u
            close(out[n, j], want.expand(G, d), (2.0 ** -8 + (len(x) + 8) * U) * mag + 2.0 ** -8 * want.abs(), f"{n} {j}")
            close(lse[n, j], torch.logsumexp(x, 0).expand(G), (len(x) + 16) * U, f"lse {n} {j}")


# --------------------------------------------------------------------------------- parts of a join
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("levels", [1, 5])
@pytest.mark.parametrize("N,H_kv,L", [(1, 1, 120_000), (40, 4, 3000), (400, 1, 1500), (3, 2, 2048)])
def test_every_step_arrives(N, H_kv, L, levels, dtype):
    """Every step of 64 keys has a place of its own in out and a weight of 2^-j (j < levels) in the sum, so
    that a step lost or joined twice shows in both: 1 sequence over every SM, units joined by warps, units
    recorded by CTA, and clusters.

    Weights are within 4 j ln 2 u + 4 u of 2^-j (scale, log2 e, their product and the one with the dot
    product; the exponential), a part's weight within 4 u; a sum goes through at most 100 roundings (48 of a
    lane, its row's lanes and the teams; 37 parts of a warp, the warps): 120 u < 2^-17 in all.  In lse also
    log2 and ln 2, 4 u of it; in out the weights' and its own rounding to its type."""
    d, steps = 128, -(-L // 64)
    j = torch.arange(steps) * 7 % levels                     # exponent of a step
    t = torch.arange(L)
    G = 2
    pages = -(-L // 64)
    k = torch.zeros(pages, 64, H_kv, d, dtype=dtype, device=DEV)
    v = torch.zeros_like(k)
    k.view(-1, H_kv, d)[:L, :, 0] = -j[t // 64].to(dtype).to(DEV)[:, None]
    rows = torch.arange(L, device=DEV)
    v.view(-1, H_kv, d)[rows, :, (rows // 64) % d] = 1.0
    kv = gdn.PagedKV(k, v, torch.arange(pages, dtype=torch.int32, device=DEV).expand(N, pages).contiguous())
    q = torch.zeros(N, 1, G * H_kv, d, dtype=dtype, device=DEV)
    q[..., 0] = 1.0
    at = torch.full((N,), L - 1, dtype=torch.int32, device=DEV)
    out, lse = gdn.gdn_attn_decode(q, at, kv, scale=math.log(2.0))
    share = torch.tensor([min(64, L - 64 * s) for s in range(steps)], dtype=torch.float64) * 2.0 ** -j.double()
    total = share.sum()
    want = torch.zeros(d, dtype=torch.float64).index_add_(0, torch.arange(steps) % d, share) / total
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    tol, tol_lse = (2 * half + 2.0 ** -17) * want, 2.0 ** -17 + 2.0 ** -22 * math.log(float(total))
    # the oracle without one step, or with one twice, is out of tolerance, whichever it is
    for sign in (-1.0, 1.0):
        other = total + sign * share
        assert bool(((other.log() - total.log()).abs() > 2 * tol_lse).all())
    close(lse, total.log().to(DEV).expand_as(lse), tol_lse, "lse")
    close(out, want.to(DEV).expand_as(out), tol.to(DEV) + 1e-30, "out")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("levels", [1, 5])
def test_every_tile_arrives_in_split_prompts(levels, dtype):
    """The same for a prompt that is split over the context: every query sees every token (a prefix), a tile of
    128 tokens has a place and a share of its own.  A sum goes through at most 140 roundings (fp32: 4 keys of
    a tile a lane, 25 tiles of 64 a part; bf16: 32 pairs of a tile, 32 tiles a part; lanes, parts): with the
    weights' 20 u, 160 u < 2^-16."""
    d, L, R, G = 128, 100_000, 40, 2
    steps = -(-L // 128)
    j = torch.arange(steps) * 7 % levels
    rows = torch.arange(L, device=DEV)
    pages = -(-L // 64)
    k = torch.zeros(pages, 64, 1, d, dtype=dtype, device=DEV)
    v = torch.zeros_like(k)
    k.view(-1, d)[:L, 0] = -j.to(dtype).to(DEV)[rows // 128]
    v.view(-1, d)[rows, (rows // 128) % d] = 1.0
    kv = gdn.PagedKV(k, v, torch.arange(pages, dtype=torch.int32, device=DEV)[None])
    q = torch.zeros(R, G, d, dtype=dtype, device=DEV)
    q[..., 0] = 1.0
    assert gdn.gdn_attn_prefill_workspace_size(kv, 1, R, G) > 256          # split
    out, lse = gdn.gdn_attn_prefill(q, kv, ints(0, R), ints(L - R), prefix_len=ints(L), scale=math.log(2.0))
    share = torch.tensor([min(128, L - 128 * s) for s in range(steps)], dtype=torch.float64) * 2.0 ** -j.double()
    total = share.sum()
    want = torch.zeros(d, dtype=torch.float64).index_add_(0, torch.arange(steps) % d, share) / total
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    tol, tol_lse = (2 * half + 2.0 ** -16) * want, 2.0 ** -16 + 2.0 ** -22 * math.log(float(total))
    for sign in (-1.0, 1.0):
        other = total + sign * share
        assert bool(((other.log() - total.log()).abs() > 2 * tol_lse).all())
    close(lse, total.log().to(DEV).expand_as(lse), tol_lse, "lse")
    close(out, want.to(DEV).expand_as(out), tol.to(DEV) + 1e-30, "out")
