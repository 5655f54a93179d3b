"""What the paged attention calls refuse at the ends of their arguments' ranges, and what they take.
Runs on the CPU: calls that pass the checks have no sequence or token to work on."""
from __future__ import annotations

import pytest

import linear_attention_token_b200 as gdn

from test_attn_checks import BAD, L, decode, prefill  # noqa: F401  (L: the library, built)


@pytest.mark.parametrize("scale,cap,status", [
    (2.3e38, 0.0, gdn.GDN_OK), (-2.3e38, 0.0, gdn.GDN_OK), (2.4e38, 0.0, BAD), (-3e38, 0.0, BAD),
    (3e38, 1.0, gdn.GDN_OK), (-3e38, 1e-4, gdn.GDN_OK), (1e-45, 1e6, gdn.GDN_OK),
    (float("inf"), 1.0, BAD), (float("nan"), 1.0, BAD)])
def test_scales(L, scale, cap, status):
    """Without a cap the scale times log2 e has to be a number of fp32; with one any finite scale serves."""
    assert decode(L, num_seqs=0, scale=scale, cap=cap) == status
    assert decode(L, listed=True, num_seqs=0, scale=scale, cap=cap) == status
    assert prefill(L, T=0, scale=scale, cap=cap) == status
