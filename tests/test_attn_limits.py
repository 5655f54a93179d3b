"""The paged attention at the ends of what its arguments allow."""
from __future__ import annotations

import pytest
import torch

import linear_attention_token_b200 as gdn

from attn_ref import attend, cache, check, fill, normal

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


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
