"""Attention over a paged cache from its definition, in 64 bits, with the error each step of
the kernels may add.  Shared by the tests of the paged-cache operators.

Tolerances.  eps(t) / 2 is the most a rounding to type t is off, relative to the value (bf16
2^-8, fp32 2^-24).
  scores    a dot of d products summed in fp32 is off by at most (d + 2) 2^-24 sum |q_i k_i|;
            times scale, plus 2^-20 absolute for the cap and the base-2 exponential, whose
            argument is rounded too (2^-24 of it).
  weights   so each e^x is off by a relative eta = 2 (score error) + 2^-20 (the difference to the
            maximum counts twice), plus the rounding of the weights to bf16 for the product.
  sums      n terms summed in fp32 add at most n 2^-24 of the sum of their magnitudes.
  out       |error| <= (2 eta + n 2^-24 + [bf16] 2^-8) sum w |v| + eps/2 |out|
  lse       |error| <= 2 eta + n 2^-24 + 2^-23 |lse|
"""
from __future__ import annotations

import math

import torch

DEV = "cuda"


def cache(N, max_tokens, H_kv, d, page, dtype, seed, *, dead=float("nan"), extra_pages=2, dev=DEV):
    """A cache whose pages are dealt out in random order, every row `dead` until written, and
    the page table with entries past each sequence's need out of range."""
    g = torch.Generator().manual_seed(seed)
    per = max(1, -(-max_tokens // page))
    pages = N * per + extra_pages
    order = torch.randperm(pages, generator=g)[:N * per].reshape(N, per).to(torch.int32)
    k = torch.full((pages, page, H_kv, d), dead, dtype=dtype, device=dev)
    v = torch.full_like(k, dead)
    return k, v, order.to(dev)


def normal(shape, dtype, seed, by=1.0, dev=DEV):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * by).to(dtype).to(dev)


def fill(k_cache, v_cache, table, lens, seed, by=1.0):
    """Write keys and values for tokens 0 .. lens[n] - 1; returns them as lists [len, H_kv, d]."""
    page, H, d = k_cache.shape[1:]
    ks, vs = [], []
    for n, L in enumerate(lens):
        k = normal((L, H, d), k_cache.dtype, seed + 2 * n, by, k_cache.device)
        v = normal((L, H, d), k_cache.dtype, seed + 2 * n + 1, 1.0, k_cache.device)
        t = torch.arange(L, device=k.device)
        rows = table[n].long()[t // page] * page + t % page
        k_cache.view(-1, H, d)[rows] = k
        v_cache.view(-1, H, d)[rows] = v
        ks.append(k)
        vs.append(v)
    return ks, vs


def attend(q, k, v, seen, scale, softcap, bf16):
    """q [R, d], k, v [n, d], seen [R, n] bool -> (out, lse, tol_out, tol_lse), all double."""
    d, n = q.shape[1], k.shape[0]
    q, k, v = q.double(), k.double(), v.double()
    R = q.shape[0]
    out = torch.zeros(R, d, dtype=torch.float64, device=q.device)
    lse = torch.full((R,), -math.inf, dtype=torch.float64, device=q.device)
    if n == 0:
        return out, lse, out.clone(), torch.zeros_like(lse)
    x = q @ k.T * scale
    mag = q.abs() @ k.abs().T * abs(scale)
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    x = x.masked_fill(~seen, -math.inf)
    some = seen.any(1)
    lse[some] = torch.logsumexp(x[some], 1)
    w = torch.where(some[:, None], torch.exp(x - torch.where(some, lse, 0.0)[:, None]), 0.0)
    out = w @ v
    dx = (d + 4) * 2.0 ** -24 * mag + 2.0 ** -20
    eta = 2 * torch.where(seen, dx, 0.0).amax(1) + 2.0 ** -20
    rel = 2 * eta + n * 2.0 ** -24 + (2.0 ** -8 if bf16 else 0.0)
    tol = rel[:, None] * (w @ v.abs()) + (2.0 ** -8 if bf16 else 2.0 ** -24) * out.abs() + 1e-30
    tol_lse = 2 * eta + n * 2.0 ** -24 + 2.0 ** -23 * lse.nan_to_num(neginf=0.0).abs()
    return out, lse, tol, tol_lse


def check(out, lse, want, where=""):
    o, l, tol, tol_l = want
    e = (out.double() - o).abs()
    assert bool((e <= tol).all()), f"{where}: out off by {float((e / tol).max()):.2f} of its tolerance"
    if lse is not None:
        fin = torch.isfinite(l)
        assert torch.equal(fin, torch.isfinite(lse)), where
        assert bool((lse[~fin] == -math.inf).all()), where
        e = (lse.double() - l)[fin].abs()
        assert bool((e <= tol_l[fin]).all()), f"{where}: lse off by {e.max().item()}"
