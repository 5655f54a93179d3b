"""gdn_attn_decode and gdn_qsa_attn_decode against the definition in 64 bits (attn_ref.py holds
the tolerances and where they come from).  Every cache row that holds no live token is NaN."""
from __future__ import annotations

import pytest
import torch

import linear_attention_token_b200 as gdn

from attn_ref import attend, cache, check, fill, normal

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(lens, T, H_q, H_kv, d, page, dtype, seed=0, by=1.5):
    N = len(lens)
    kc, vc, table = cache(N, max(lens + [1]), H_kv, d, page, dtype, seed)
    ks, vs = fill(kc, vc, table, lens, seed + 10)
    q = normal((N, T, H_q, d), dtype, seed + 5, by)
    pos = torch.tensor([L - T for L in lens], dtype=torch.int32, device=DEV)
    return q, pos, gdn.PagedKV(kc, vc, table), ks, vs


def dense_seen(L, T, window):
    t = torch.arange(L, device=DEV)
    at = torch.arange(L - T, L, device=DEV)[:, None]
    seen = t <= at
    return seen & (t > at - window) if window else seen


def verify(out, lse, q, ks, vs, seen_of, scale, softcap, dtype, where=""):
    """seen_of(n, j): positions into ks[n], vs[n] (with repeats) that query j sees."""
    N, T, H_q, d = q.shape
    G = H_q // ks[0].shape[1]
    for n in range(N):
        for j in range(T):
            idx = seen_of(n, j)
            for h in range(H_q // G):
                k, v = ks[n][idx, h], vs[n][idx, h]
                rows = slice(h * G, (h + 1) * G)
                seen = torch.ones(G, len(idx), dtype=torch.bool, device=DEV)
                want = attend(q[n, j, rows], k, v, seen, scale, softcap, dtype == torch.bfloat16)
                check(out[n, j, rows], lse[n, j, rows], want, f"{where} n={n} j={j} h={h}")


CASES = [
    # lens, T, H_q, H_kv, d, page, softcap, window, dtype
    ([1], 1, 1, 1, 64, 16, 0.0, 0, torch.bfloat16),
    ([1, 2, 15, 16, 17], 1, 4, 2, 128, 16, 0.0, 0, torch.bfloat16),
    ([63, 64, 65, 0, 129, 1000], 1, 16, 2, 128, 64, 0.0, 0, torch.bfloat16),
    ([500, 3, 77], 3, 8, 8, 64, 32, 0.0, 0, torch.bfloat16),
    ([500, 8, 300], 8, 8, 2, 128, 16, 0.0, 0, torch.bfloat16),        # 32 rows per key head
    ([333, 90], 5, 24, 2, 128, 128, 20.0, 0, torch.bfloat16),         # 60 rows
    ([150, 40], 8, 32, 2, 64, 16, 0.0, 0, torch.bfloat16),            # 128 rows: two blocks
    ([700, 260, 5], 2, 8, 2, 128, 16, 0.0, 100, torch.bfloat16),
    ([700, 260, 5], 4, 8, 2, 128, 16, 30.0, 1, torch.bfloat16),
    ([5000], 1, 6, 3, 128, 1024, 0.0, 0, torch.bfloat16),
    ([500, 9, 130, 0, 1500], 4, 32, 2, 128, 16, 0.0, 0, torch.bfloat16),   # 64 rows, 10 units
    ([700, 40, 300, 5], 8, 16, 2, 64, 64, 20.0, 0, torch.bfloat16),
    ([4000] + [30] * 9, 3, 16, 1, 128, 16, 0.0, 900, torch.bfloat16),
    ([1, 2, 15, 16, 17, 0], 1, 4, 2, 128, 16, 0.0, 0, torch.float32),
    ([63, 1000], 1, 2, 2, 64, 16, 0.0, 0, torch.float32),
    ([500, 3, 77], 3, 8, 2, 64, 32, 15.0, 0, torch.float32),          # 12 rows: two blocks
    ([500, 80], 2, 6, 3, 128, 32, 0.0, 33, torch.float32),
]


@pytest.mark.parametrize("lens,T,H_q,H_kv,d,page,softcap,window,dtype", CASES)
def test_decode_matches_definition(lens, T, H_q, H_kv, d, page, softcap, window, dtype):
    q, pos, kv, ks, vs = make(lens, T, H_q, H_kv, d, page, dtype)
    out, lse = gdn.gdn_attn_decode(q, pos, kv, softcap=softcap, window=window)
    torch.cuda.synchronize()

    def seen(n, j):
        at = lens[n] - T + j
        lo = max(0, at - window + 1) if window else 0
        return torch.arange(lo, max(lo, at + 1), device=DEV)

    verify(out, lse, q, ks, vs, seen, d ** -0.5, softcap, dtype)


LIST_CASES = [
    # lens, T, H_q, H_kv, d, page, list_len, recent, softcap, dtype
    ([200, 9, 64, 0], 1, 16, 2, 128, 16, 32, 4, 0.0, torch.bfloat16),
    ([3000, 1500], 4, 16, 2, 128, 64, 2048, 65, 0.0, torch.bfloat16),
    ([3000, 40], 2, 40, 2, 128, 16, 260, 0, 25.0, torch.bfloat16),    # 20 rows
    ([3000], 1, 80, 1, 64, 16, 100, 7, 0.0, torch.bfloat16),          # 80 rows: two blocks
    ([500, 17], 1, 4, 4, 64, 16, 0, 20, 0.0, torch.bfloat16),         # newest tokens only
    ([500, 17], 2, 4, 4, 128, 16, 64, 0, 0.0, torch.float32),
    ([900, 30], 3, 10, 2, 64, 32, 128, 12, 10.0, torch.float32),
]


def lists(lens, T, list_len, recent, seed):
    """Distinct tokens in random order, some of them among the newest or later than the query,
    -1 at random places."""
    g = torch.Generator().manual_seed(seed)
    idx = torch.full((len(lens), T, list_len), -1, dtype=torch.int32)
    for n, L in enumerate(lens):
        for j in range(T):
            m = min(list_len, L)
            put = torch.randperm(list_len, generator=g)[:m]
            idx[n, j, put] = torch.randperm(L, generator=g)[:m].to(torch.int32)
            if list_len > 4 and L > 0:
                idx[n, j, :2] = torch.tensor([L + 5, -7], dtype=torch.int32)
    return idx.to(DEV)


@pytest.mark.parametrize("lens,T,H_q,H_kv,d,page,list_len,recent,softcap,dtype", LIST_CASES)
def test_listed_matches_definition(lens, T, H_q, H_kv, d, page, list_len, recent, softcap, dtype):
    q, pos, kv, ks, vs = make(lens, T, H_q, H_kv, d, page, dtype)
    idx = lists(lens, T, list_len, recent, 3)
    out, lse = gdn.gdn_qsa_attn_decode(q, pos, kv, idx, recent=recent, softcap=softcap)
    torch.cuda.synchronize()

    def seen(n, j):
        at = lens[n] - T + j
        x = idx[n, j].long()
        x = x[(x >= 0) & (x <= at - recent)]
        return torch.cat([x, torch.arange(max(0, at - recent + 1), at + 1, device=DEV)
                          if at >= 0 and recent else x[:0]])

    verify(out, lse, q, ks, vs, seen, d ** -0.5, softcap, dtype)


def test_token_listed_twice_counts_twice():
    q, pos, kv, ks, vs = make([100], 1, 4, 2, 64, 16, torch.bfloat16)
    idx = torch.tensor([[5, 9, 5, -1, 5, 40]], dtype=torch.int32, device=DEV)
    out, lse = gdn.gdn_qsa_attn_decode(q, pos, kv, idx)
    verify(out, lse, q, ks, vs, lambda n, j: idx[0][idx[0] >= 0].long(), 0.125, 0.0, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,H_kv,most", [(1, 1, 4096), (2, 4, 1000), (3, 2, 2048), (30, 1, 1024), (60, 1, 500),
                                         (60, 2, 500)])
def test_short_calls_of_few_units(N, H_kv, most, dtype):
    """Every number of CTAs to a unit, with lengths down to none: some CTAs of a unit have no key."""
    lens = [most - 37 * n if n % 3 else n for n in range(N)]
    lens = [max(0, L) for L in lens]
    T, G = 1, 3
    q, pos, kv, ks, vs = make(lens, T, G * H_kv, H_kv, 64, 16, dtype)
    out, lse = gdn.gdn_attn_decode(q, pos, kv)
    verify(out, lse, q, ks, vs, lambda n, j: torch.arange(lens[n], device=DEV), 0.125, 0.0, dtype)
    again, _ = gdn.gdn_attn_decode(q, pos, kv)
    assert torch.equal(again, out)


def test_many_ragged_sequences():
    """Units that end anywhere inside a CTA's stretch, idle slots among them."""
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 300, (300,), generator=g).tolist()
    lens[7] = lens[150] = 0
    lens[200] = 4000
    for dtype in (torch.bfloat16, torch.float32):
        q, pos, kv, ks, vs = make(lens, 1, 4, 2, 64, 16, dtype)
        out, lse = gdn.gdn_attn_decode(q, pos, kv)
        verify(out, lse, q, ks, vs, lambda n, j: torch.arange(lens[n], device=DEV), 0.125, 0.0,
               dtype)


def test_long_sequence_every_sm_joins():
    L = 120_000
    q, pos, kv, ks, vs = make([L], 1, 8, 1, 128, 64, torch.bfloat16)
    out, lse = gdn.gdn_attn_decode(q, pos, kv)
    verify(out, lse, q, ks, vs, lambda n, j: torch.arange(L, device=DEV), 128 ** -0.5, 0.0,
           torch.bfloat16)
    again, lse2 = gdn.gdn_attn_decode(q, pos, kv)
    assert torch.equal(out, again) and torch.equal(lse, lse2)       # same order of sums


def test_workspace_of_any_contents():
    """One workspace for calls of different shapes in turn, whatever it holds."""
    calls = []
    for lens, T, H_q, H_kv in (([120_000], 1, 8, 1), ([700, 30], 4, 16, 2), ([9000] * 5, 1, 4, 4)):
        q, pos, kv, _, _ = make(lens, T, H_q, H_kv, 128, 64, torch.bfloat16)
        calls.append((q, pos, kv, gdn.gdn_attn_decode(q, pos, kv)))
    n = max(gdn.gdn_attn_decode_workspace_size(q.shape[1], q.shape[2], kv.H_kv, 128)
            for q, _, kv, _ in calls)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        for q, pos, kv, (out, lse) in calls:
            o, l = gdn.gdn_attn_decode(q, pos, kv, workspace=ws)
            assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale,softcap", [(-0.1, 0.0), (0.0, 0.0), (2.0, 5.0), (-1.0, 1.0), (0.0, 3.0)])
def test_scale_of_any_sign_and_far_caps(scale, softcap, dtype):
    """Scores on both sides of the cap, where the cap's two forms meet."""
    q, pos, kv, ks, vs = make([300, 20], 2, 4, 2, 64, 16, dtype)
    out, lse = gdn.gdn_attn_decode(q, pos, kv, scale=scale, softcap=softcap)
    verify(out, lse, q, ks, vs, lambda n, j: torch.arange([300, 20][n] - 1 + j, device=DEV), scale,
           softcap, dtype)
    again, none = gdn.gdn_attn_decode(q, pos, kv, scale=scale, softcap=softcap, want_lse=False)
    assert none is None and torch.equal(again, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("softcap,far", [(1e3, 1.0), (1e6, 1.0), (2e4, 3e4), (1e6, 2e6)])
def test_large_caps(softcap, far, dtype):
    """A large cap changes small scores by nothing, also beside a head whose scores pass it."""
    q, pos, kv, ks, vs = make([300, 20], 2, 4, 2, 64, 16, dtype)
    q[:, :, 1] *= far
    out, lse = gdn.gdn_attn_decode(q, pos, kv, softcap=softcap)
    verify(out, lse, q, ks, vs, lambda n, j: torch.arange([300, 20][n] - 1 + j, device=DEV), 0.125,
           softcap, dtype)


def test_peaked_scores():
    """Scores of hundreds, of both signs: one key decides, and the running maximum jumps."""
    q, pos, kv, ks, vs = make([2000], 1, 8, 2, 128, 16, torch.bfloat16, by=60.0)
    out, lse = gdn.gdn_attn_decode(q, pos, kv)
    verify(out, lse, q, ks, vs, lambda n, j: torch.arange(2000, device=DEV), 128 ** -0.5, 0.0,
           torch.bfloat16)


def test_absent_pages_are_not_seen():
    """Entries out of range hide their tokens; with a window, freed pages before it may be -1."""
    lens = [100, 100]
    q, pos, kv, ks, vs = make(lens, 1, 4, 2, 64, 16, torch.bfloat16)
    kv.page_table[0, 2] = -1
    kv.page_table[1, 0] = kv.k.shape[0]
    out, lse = gdn.gdn_attn_decode(q, pos, kv)
    gone = [set(range(32, 48)), set(range(16))]
    live = [torch.tensor([t for t in range(100) if t not in gone[n]], device=DEV) for n in range(2)]
    verify(out, lse, q, ks, vs, lambda n, j: live[n], 0.125, 0.0, torch.bfloat16)
    kv.page_table[:, :4] = -1
    out, lse = gdn.gdn_attn_decode(q, pos, kv, window=36)
    verify(out, lse, q, ks, vs, lambda n, j: torch.arange(64, 100, device=DEV), 0.125, 0.0,
           torch.bfloat16)


def test_positions_past_the_table():
    """Only the table's tokens exist for a query that sits past them."""
    q, pos, kv, ks, vs = make([64], 1, 4, 2, 64, 16, torch.bfloat16)
    for at in (64, 1000, 2**31 - 1):
        pos.fill_(at)
        out, lse = gdn.gdn_attn_decode(q, pos, kv)
        verify(out, lse, q, ks, vs, lambda n, j: torch.arange(64, device=DEV), 0.125, 0.0,
               torch.bfloat16)
    pos.fill_(-(2**31))
    out, lse = gdn.gdn_attn_decode(q, pos, kv)
    assert not out.any() and bool((lse == -float("inf")).all())


def test_row_offsets_past_32_bits():
    pages = (1 << 32) // (1024 * 8 * 128 * 2) + 2
    kc = torch.full((pages, 1024, 8, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    vc = torch.full_like(kc, float("nan"))
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device=DEV)
    ks, vs = fill(kc, vc, table, [300], 3)
    q = normal((1, 1, 16, 128), torch.bfloat16, 1)
    pos = torch.tensor([299], dtype=torch.int32, device=DEV)
    kv = gdn.PagedKV(kc, vc, table)
    out, lse = gdn.gdn_attn_decode(q, pos, kv)
    verify(out, lse, q, ks, vs, lambda n, j: torch.arange(300, device=DEV), 128 ** -0.5, 0.0,
           torch.bfloat16)
    idx = torch.arange(256, dtype=torch.int32, device=DEV)[None]
    out, lse = gdn.gdn_qsa_attn_decode(q, pos, kv, idx, recent=40)
    seen = torch.cat([torch.arange(256), torch.arange(260, 300)]).to(DEV)
    verify(out, lse, q, ks, vs, lambda n, j: seen, 128 ** -0.5, 0.0, torch.bfloat16)


def test_graph_replay_as_sequences_grow():
    """A captured append and decode step replayed while positions advance equals eager calls."""
    N, H_q, H_kv, d, steps = 3, 8, 2, 128, 20
    lens = [60, 1, 130]
    q, pos, kv, ks, vs = make([L + steps for L in lens], 1, H_q, H_kv, d, 16, torch.bfloat16)
    kv.k.fill_(0), kv.v.fill_(0)
    ws = gdn.attn_decode_workspace(1, H_q, H_kv, d)
    k, v = normal((N, 1, H_kv, d), torch.bfloat16, 1), normal((N, 1, H_kv, d), torch.bfloat16, 2)
    q1, out = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty(N, 1, H_q, device=DEV)
    freq = gdn.rope_inv_freq(64)

    def step():
        gdn.gdn_kv_append(k, v, kv, None, pos, q=q, q_out=q1, inv_freq=freq)
        gdn.gdn_attn_decode(q1, pos, kv, out=out, lse=lse, workspace=ws)

    def run(fn):
        pos.copy_(torch.tensor(lens))
        kv.k.fill_(0), kv.v.fill_(0)
        got = []
        for s in range(steps):
            k.copy_(normal((N, 1, H_kv, d), torch.bfloat16, 100 + s))
            fn()
            got.append((out.clone(), lse.clone()))
            pos.add_(1)
        torch.cuda.synchronize()
        return got

    want = run(step)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for (a, b), (x, y) in zip(run(g.replay), want):
        assert torch.equal(a, x) and torch.equal(b, y)


def test_other_stream():
    q, pos, kv, ks, vs = make([4000, 2000], 1, 8, 2, 128, 16, torch.bfloat16)
    want, want_lse = gdn.gdn_attn_decode(q, pos, kv)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [gdn.gdn_attn_decode(q, pos, kv, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for o, l in outs:
        assert torch.equal(o, want) and torch.equal(l, want_lse)


def test_calls_at_once():
    """Calls of every form side by side on four streams, each with its own workspace."""
    kinds = [make([900, 30, 512], 1, 8, 2, 128, 16, torch.bfloat16), make([9000, 700], 2, 8, 2, 128, 16, torch.bfloat16),
             make([300] * 9, 4, 16, 1, 128, 16, torch.bfloat16), make([1000, 5], 1, 4, 2, 64, 16, torch.float32)]
    want = [gdn.gdn_attn_decode(q, pos, kv) for q, pos, kv, _, _ in kinds]
    streams = [torch.cuda.Stream() for _ in kinds]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for i, (q, pos, kv, _, _) in enumerate(kinds):
            got.append((i, gdn.gdn_attn_decode(q, pos, kv, stream=streams[i])))
    torch.cuda.synchronize()
    for i, (out, lse) in got:
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1]), i
