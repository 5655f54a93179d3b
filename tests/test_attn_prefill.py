"""gdn_attn_prefill against the definition in 64 bits (attn_ref.py holds the tolerances and where
they come from).  Every cache row that holds no live token is NaN."""
from __future__ import annotations

import pytest
import torch

import linear_attention_token_b200 as gdn

from attn_ref import attend, cache, check, fill, normal

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def make(lens, past, H_q, H_kv, d, page, dtype, seed=0, by=1.5, tail=0):
    N = len(lens)
    ends = [p + L for p, L in zip(past, lens)]
    kc, vc, table = cache(N, max(ends + [1]), H_kv, d, page, dtype, seed)
    ks, vs = fill(kc, vc, table, ends, seed + 10)
    q = normal((sum(lens) + tail, H_q, d), dtype, seed + 5, by)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    pos0 = torch.tensor(past, dtype=torch.int32, device=DEV)
    return q, gdn.PagedKV(kc, vc, table), cu, pos0, ks, vs


def seen_by(L, p, window=0, prefix=0, hidden=()):
    t, at = torch.arange(p + L, device=DEV), torch.arange(p, p + L, device=DEV)[:, None]
    seen = t <= at
    if window:
        seen = seen & (t > at - window)
    seen = seen | (t < prefix)
    for a, b in hidden:
        seen = seen & ~((t >= a) & (t < b))
    return seen


def verify(out, lse, q, ks, vs, lens, past, scale, softcap, seen_of):
    G = q.shape[1] // ks[0].shape[1]
    first = 0
    for n, L in enumerate(lens):
        seen = seen_of(n)
        for h in range(q.shape[1]):
            rows = slice(first, first + L)
            want = attend(q[rows, h], ks[n][:, h // G], vs[n][:, h // G], seen, scale, softcap,
                          q.dtype == BF)
            check(out[rows, h], lse[rows, h], want, f"n={n} h={h}")
        first += L


CASES = [
    # lens, past, H_q, H_kv, d, page, softcap, window, prefix, dtype
    ([1], [0], 1, 1, 128, 16, 0.0, 0, None, BF),
    ([128], [0], 2, 1, 128, 128, 0.0, 0, None, BF),
    ([300], [0], 8, 1, 128, 64, 0.0, 0, None, BF),
    ([333, 0, 1, 65], [0, 5, 0, 0], 4, 2, 128, 16, 0.0, 0, None, BF),
    ([700, 129], [0, 0], 3, 3, 128, 32, 0.0, 0, None, BF),              # one head per tile row block
    ([200, 77], [100, 513], 6, 1, 128, 64, 0.0, 0, None, BF),           # 6 heads: three packs of 2
    ([50, 2, 90], [1000, 129, 0], 16, 1, 128, 256, 0.0, 0, None, BF),
    ([400, 150], [0, 300], 4, 2, 128, 16, 0.0, 100, None, BF),
    ([600, 20], [30, 900], 2, 2, 128, 16, 20.0, 1, None, BF),
    ([400, 150, 30], [0, 300, 7], 4, 2, 128, 16, 0.0, 0, [250, 420, 0], BF),
    ([500, 64], [77, 0], 8, 2, 128, 1024, 30.0, 0, [577, 3], BF),
    ([333, 1, 130], [0, 40, 64], 8, 2, 64, 16, 0.0, 0, None, BF),
    ([260, 31], [500, 3], 2, 1, 64, 128, 25.0, 0, [100, 9], BF),
    ([513], [0], 32, 1, 64, 64, 0.0, 200, None, BF),
    ([1, 64, 65, 0], [0, 0, 9, 4], 2, 1, 64, 16, 0.0, 0, None, F32),
    ([150, 77], [33, 200], 6, 2, 128, 32, 0.0, 0, None, F32),
    ([150, 77], [33, 200], 4, 4, 128, 16, 15.0, 50, None, F32),
    ([150, 77], [33, 0], 3, 1, 64, 64, 0.0, 0, [170, 500], F32),
]


@pytest.mark.parametrize("lens,past,H_q,H_kv,d,page,softcap,window,prefix,dtype", CASES)
def test_matches_definition(lens, past, H_q, H_kv, d, page, softcap, window, prefix, dtype):
    tail = 5                                                # rows behind the last sequence
    q, kv, cu, pos0, ks, vs = make(lens, past, H_q, H_kv, d, page, dtype, tail=tail)
    q[sum(lens):] = float("nan")
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    pre = None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    gdn.gdn_attn_prefill(q, kv, cu, pos0, prefix_len=pre, softcap=softcap, window=window, out=out,
                         lse=lse, workspace=ws)
    assert gdn.gdn_get_device_error(ws) == gdn.GDN_OK
    verify(out, lse, q, ks, vs, lens, past, d ** -0.5, softcap,
           lambda n: seen_by(lens[n], past[n], window, prefix[n] if prefix else 0))
    assert bool((out[sum(lens):] == 7.0).all()) and bool((lse[sum(lens):] == 7.0).all())
    again, lse2 = gdn.gdn_attn_prefill(q, kv, cu, pos0, prefix_len=pre, softcap=softcap,
                                       window=window, workspace=ws)
    assert torch.equal(again[:sum(lens)], out[:sum(lens)])  # same order of sums
    assert torch.equal(lse2[:sum(lens)], lse[:sum(lens)])


SPLIT_CASES = [
    # lens, past, H_q, H_kv, d, page, softcap, window, prefix, dtype
    ([64], [5000], 16, 2, 128, 64, 0.0, 0, None, BF),
    ([3, 40, 1, 0], [9000, 100, 2500, 3], 8, 1, 128, 16, 0.0, 0, None, BF),
    ([70], [9000], 3, 1, 64, 128, 20.0, 0, None, BF),
    ([40, 9], [9000, 4000], 8, 2, 128, 16, 0.0, 3000, None, BF),
    ([33, 9], [3000, 6000], 4, 1, 128, 64, 0.0, 0, [3020, 10], BF),
    ([100], [4000], 8, 2, 128, 64, 0.0, 0, None, F32),
    ([9, 0, 50], [4000, 9, 600], 6, 1, 64, 16, 10.0, 0, None, F32),
    ([9, 50], [4000, 3000], 2, 2, 64, 16, 0.0, 2000, None, F32),
]


@pytest.mark.parametrize("lens,past,H_q,H_kv,d,page,softcap,window,prefix,dtype", SPLIT_CASES)
def test_few_rows_behind_a_long_context(lens, past, H_q, H_kv, d, page, softcap, window, prefix, dtype):
    """Calls that are split over the context's length, and the same in one piece."""
    q, kv, cu, pos0, ks, vs = make(lens, past, H_q, H_kv, d, page, dtype, tail=2)
    total = sum(lens)
    pre = None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device=DEV)
    n = gdn.gdn_attn_prefill_workspace_size(kv, len(lens), total + 2, H_q)
    assert n > 256                                          # it would be split
    opts = dict(prefix_len=pre, softcap=softcap, window=window)
    first = None
    for ws in (torch.zeros(n, dtype=torch.uint8, device=DEV), None,
               torch.full((n - 1,), 0, dtype=torch.uint8, device=DEV)):
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=DEV)
        gdn.gdn_attn_prefill(q, kv, cu, pos0, out=out, lse=lse, workspace=ws, **opts)
        if ws is not None:
            assert gdn.gdn_get_device_error(ws) == gdn.GDN_OK
        verify(out, lse, q, ks, vs, lens, past, d ** -0.5, softcap,
               lambda i: seen_by(lens[i], past[i], window, prefix[i] if prefix else 0))
        assert bool((out[total:] == 7.0).all()) and bool((lse[total:] == 7.0).all())
        if first is None:
            first = out
        elif ws is None:
            assert torch.equal(out, first)                  # split the same way, same order of sums


def test_wide_table_short_context():
    """A table that could hold a long context, and sequences that do not: nothing is split."""
    q, kv, cu, pos0, ks, vs = make([70, 12], [30, 0], 8, 2, 128, 16, BF)
    wide = torch.full((2, 4096), -1, dtype=torch.int32, device=DEV)
    wide[:, :kv.page_table.shape[1]] = kv.page_table
    big = gdn.PagedKV(kv.k, kv.v, wide)
    assert gdn.gdn_attn_prefill_workspace_size(big, 2, 82, 8) > 256
    out, lse = gdn.gdn_attn_prefill(q, big, cu, pos0)
    verify(out, lse, q, ks, vs, [70, 12], [30, 0], 128 ** -0.5, 0.0,
           lambda n: seen_by([70, 12][n], [30, 0][n]))
    small, _ = gdn.gdn_attn_prefill(q, kv, cu, pos0)
    assert torch.equal(small, out)


def test_dense_batch_equals_packed():
    q, kv, cu, pos0, ks, vs = make([140, 140, 140], [0, 3, 50], 8, 2, 128, 16, BF)
    a, la = gdn.gdn_attn_prefill(q, kv, cu, pos0)
    b, lb = gdn.gdn_attn_prefill(q.view(3, 140, 8, 128), kv, None, pos0)
    assert torch.equal(a, b.view_as(a)) and torch.equal(la, lb.view_as(la))


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.0])
@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_scale_of_any_sign(scale, softcap):
    q, kv, cu, pos0, ks, vs = make([150], [20], 4, 2, 128, 16, BF)
    out, lse = gdn.gdn_attn_prefill(q, kv, cu, pos0, scale=scale, softcap=softcap)
    verify(out, lse, q, ks, vs, [150], [20], scale, softcap, lambda n: seen_by(150, 20))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("softcap,far", [(1e3, 1.0), (1e6, 1.0), (2e4, 3e4), (1e6, 2e6), (12.0, 1.0), (5e3, 1e3)])
def test_large_caps(softcap, far, dtype):
    """A large cap changes small scores by nothing, also beside a head whose scores pass it."""
    q, kv, cu, pos0, ks, vs = make([150], [300], 4, 2, 64, 16, dtype)
    q[:, 1] *= far
    out, lse = gdn.gdn_attn_prefill(q, kv, cu, pos0, softcap=softcap)
    verify(out, lse, q, ks, vs, [150], [300], 0.125, softcap, lambda n: seen_by(150, 300))


def test_growing_maxima():
    """Scores that rise by hundreds along the sequence: O is rescaled again and again; and scores
    that fall, where it never is."""
    L, d = 1500, 128
    for sign in (1.0, -1.0):
        q, kv, cu, pos0, ks, vs = make([L], [0], 4, 1, d, 64, BF)
        ramp = torch.linspace(0, 40, L, device=DEV)[:, None, None] * sign
        k = (ks[0] * 0.5 + ramp).to(BF)
        page = kv.page_table[0].long()[torch.arange(L, device=DEV) // 64]
        kv.k[page, torch.arange(L, device=DEV) % 64] = k
        q.abs_()
        out, lse = gdn.gdn_attn_prefill(q, kv, cu, pos0)
        verify(out, lse, q, [k], vs, [L], [0], d ** -0.5, 0.0, lambda n: seen_by(L, 0))


@pytest.mark.parametrize("dtype,page", [(BF, 16), (BF, 64), (BF, 256), (F32, 16)])
def test_absent_pages_are_not_seen(dtype, page):
    lens, past = [300, 280], [0, 40]
    q, kv, cu, pos0, ks, vs = make(lens, past, 4, 2, 128, page, dtype)
    kv.page_table[0, 0] = -1
    kv.page_table[1, 1] = kv.k.shape[0]
    gone = [(0, page), (page, 2 * page)]
    out, lse = gdn.gdn_attn_prefill(q, kv, cu, pos0)
    verify(out, lse, q, ks, vs, lens, past, 128 ** -0.5, 0.0,
           lambda n: seen_by(lens[n], past[n], hidden=[gone[n]]))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_freed_pages_before_the_window(dtype):
    """Pages that only tokens before the window used may be gone, or hold NaN."""
    L, p, w = 60, 400, 33
    q, kv, cu, pos0, ks, vs = make([L], [p], 4, 2, 128, 16, dtype)
    first = (p - w + 1) // 16
    kv.page_table[0, :first - 2] = -1
    for i in range(first - 2, first):
        kv.k[kv.page_table[0, i]] = float("nan")
        kv.v[kv.page_table[0, i]] = float("nan")
    out, lse = gdn.gdn_attn_prefill(q, kv, cu, pos0, window=w)
    old = (p - w + 1) // 16 * 16
    vs[0][:old], ks[0][:old] = 0, 0
    verify(out, lse, q, ks, vs, [L], [p], 128 ** -0.5, 0.0, lambda n: seen_by(L, p, w))
    qd = q[:1, None].contiguous()                           # the same for a decode step
    out, lse = gdn.gdn_attn_decode(qd, pos0, kv, window=w)
    want = [attend(qd[0, 0, 2 * h:2 * h + 2], ks[0][:p + 1, h], vs[0][:p + 1, h],
                   seen_by(1, p, w).expand(2, -1), 128 ** -0.5, 0.0, dtype == BF) for h in range(2)]
    for h in range(2):
        check(out[0, 0, 2 * h:2 * h + 2], lse[0, 0, 2 * h:2 * h + 2], want[h])


def test_tokens_past_the_table():
    """Tokens that did not fit the table do not exist; queries behind it see what did."""
    q, kv, cu, pos0, ks, vs = make([200], [0], 4, 2, 128, 16, BF)
    short = gdn.PagedKV(kv.k, kv.v, kv.page_table[:, :5].contiguous())
    out, lse = gdn.gdn_attn_prefill(q, short, cu, pos0)
    seen = seen_by(200, 0)[:, :80]
    verify(out, lse, q, [ks[0][:80]], [vs[0][:80]], [200], [0], 128 ** -0.5, 0.0, lambda n: seen)


def test_many_short_sequences():
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 20, (900,), generator=g).tolist()
    past = torch.randint(0, 40, (900,), generator=g).tolist()
    for dtype, heads in ((BF, 8), (F32, 4)):
        q, kv, cu, pos0, ks, vs = make(lens, past, heads, 1, 64, 16, dtype)
        out, lse = gdn.gdn_attn_prefill(q, kv, cu, pos0)
        verify(out, lse, q, ks, vs, lens, past, 0.125, 0.0, lambda n: seen_by(lens[n], past[n]))


def test_prefill_continues_into_decode():
    """A prompt in one call, in two calls, and its last tokens as decode steps agree."""
    H_q, H_kv, d, L = 8, 2, 128, 300
    q, kv, cu, pos0, ks, vs = make([L], [0], H_q, H_kv, d, 16, BF)
    out, lse = gdn.gdn_attn_prefill(q, kv, cu, pos0)
    i32 = dict(dtype=torch.int32, device=DEV)
    a = gdn.gdn_attn_prefill(q[:170].contiguous(), kv, torch.tensor([0, 170], **i32), pos0)
    b = gdn.gdn_attn_prefill(q[170:].contiguous(), kv, torch.tensor([0, 130], **i32), pos0 + 170)
    c = gdn.gdn_attn_decode(q[None, 292:].contiguous(), torch.tensor([292], **i32), kv)
    for o, l in ((torch.cat([a[0], b[0]]), torch.cat([a[1], b[1]])),):
        verify(o, l, q, ks, vs, [L], [0], d ** -0.5, 0.0, lambda n: seen_by(L, 0))
    G = H_q // H_kv
    for h in range(H_q):
        want = attend(q[292:, h], ks[0][:, h // G], vs[0][:, h // G], seen_by(8, 292), d ** -0.5, 0.0, True)
        check(c[0][0, :, h], c[1][0, :, h], want)


def test_row_offsets_past_32_bits():
    pages = (1 << 32) // (1024 * 8 * 128 * 2) + 2
    kc = torch.full((pages, 1024, 8, 128), float("nan"), dtype=BF, device=DEV)
    vc = torch.full_like(kc, float("nan"))
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device=DEV)
    ks, vs = fill(kc, vc, table, [1100], 3)
    q = normal((150, 16, 128), BF, 1)
    i32 = dict(dtype=torch.int32, device=DEV)
    out, lse = gdn.gdn_attn_prefill(q, gdn.PagedKV(kc, vc, table), torch.tensor([0, 150], **i32),
                                    torch.tensor([950], **i32))
    verify(out, lse, q, ks, vs, [150], [950], 128 ** -0.5, 0.0, lambda n: seen_by(150, 950))


def test_timeout_is_reported():
    """With no polls allowed every wait gives up: the error is reported, the context lives, and the
    next call is right."""
    q, kv, cu, pos0, ks, vs = make([700, 90], [0, 300], 8, 2, 128, 16, BF)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    old = gdn.gdn_set_wait_budget(0)
    try:
        gdn.gdn_attn_prefill(q, kv, cu, pos0, workspace=ws)
        assert gdn.gdn_get_device_error(ws) == gdn.GDN_ERR_TIMEOUT
    finally:
        gdn.gdn_set_wait_budget(old)
    out, lse = gdn.gdn_attn_prefill(q, kv, cu, pos0, workspace=ws)
    assert gdn.gdn_get_device_error(ws) == gdn.GDN_OK
    verify(out, lse, q, ks, vs, [700, 90], [0, 300], 128 ** -0.5, 0.0,
           lambda n: seen_by([700, 90][n], [0, 300][n]))


@pytest.mark.parametrize("budget", [1, 8, 65, 68, 72, 80])
def test_waits_that_run_out_midway(budget):
    """With few polls allowed some waits give up and others do not: the call is right or reports the
    timeout, and the next one is right."""
    q, kv, cu, pos0, ks, vs = make([700, 90], [0, 300], 8, 2, 128, 16, BF)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    old = gdn.gdn_set_wait_budget(budget)
    try:
        results = [gdn.gdn_attn_prefill(q, kv, cu, pos0, workspace=ws)]
        status = gdn.gdn_get_device_error(ws)
    finally:
        gdn.gdn_set_wait_budget(old)
    assert status in (gdn.GDN_OK, gdn.GDN_ERR_TIMEOUT)
    if status == gdn.GDN_ERR_TIMEOUT:
        results.clear()
    results.append(gdn.gdn_attn_prefill(q, kv, cu, pos0, workspace=ws))
    assert gdn.gdn_get_device_error(ws) == gdn.GDN_OK
    for out, lse in results:
        verify(out, lse, q, ks, vs, [700, 90], [0, 300], 128 ** -0.5, 0.0,
               lambda n: seen_by([700, 90][n], [0, 300][n]))


def test_graph_replay_and_streams():
    q, kv, cu, pos0, ks, vs = make([500, 130], [0, 64], 8, 2, 128, 16, BF)
    want, want_lse = gdn.gdn_attn_prefill(q, kv, cu, pos0)
    out, lse = torch.empty_like(q), torch.empty_like(want_lse)

    def call():
        gdn.gdn_attn_prefill(q, kv, cu, pos0, out=out, lse=lse)

    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [gdn.gdn_attn_prefill(q, kv, cu, pos0, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want) and torch.equal(l, want_lse)
