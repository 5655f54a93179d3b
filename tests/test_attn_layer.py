"""An attention layer's serving run on the paged cache, its operators together as a model calls
them: a packed batch of prompts (queries, keys and values sliced out of one projection) is appended
and attended, its indexer keys are compressed, and then tokens are decoded one by one: append, index,
attention over the listed tokens and the newest ones; the last tokens again as drafts.  Every output
is checked against the definition in 64 bits, with what the cache holds and what the indexer listed.
"""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

import linear_attention_token_b200 as gdn

from attn_ref import attend, check, normal

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16
H_Q, H_KV, D, PAGE, BUDGET, RECENT = 8, 2, 128, 16, 16, 8
I32 = dict(dtype=torch.int32, device=DEV)


class Layer:
    """The layer's state: cache, page table, indexer block cache; and what the test knows of it."""

    def __init__(self, lens, room):
        self.N, self.lens = len(lens), list(lens)
        self.most = max(lens) + room
        per = -(-self.most // PAGE)
        g = torch.Generator().manual_seed(0)
        order = torch.randperm(self.N * per, generator=g)
        shape = (self.N * per, PAGE, H_KV, D)
        self.kv = gdn.PagedKV(torch.full(shape, float("nan"), dtype=BF, device=DEV),
                              torch.full(shape, float("nan"), dtype=BF, device=DEV),
                              order.view(self.N, per).to(**I32))
        self.freq = gdn.rope_inv_freq(64)
        self.blocks = self.most // 4
        self.cu_blocks = torch.arange(self.N + 1, **I32) * self.blocks
        self.k_hat = torch.zeros(self.N * self.blocks, 128, dtype=BF, device=DEV)
        self.index_keys = [torch.empty(0, 128, dtype=BF, device=DEV) for _ in lens]

    def held(self, n, tokens):
        """Keys and values of sequence n's tokens, as the cache holds them."""
        row = self.kv.page_table[n].long()[tokens // PAGE], tokens % PAGE
        return self.kv.k[row], self.kv.v[row]

    def compress(self):
        """Every whole block's key (a serving loop does this for the new blocks alone)."""
        cu = torch.tensor([0] + [len(k) for k in self.index_keys]).cumsum(0).to(**I32)
        gdn.gdn_qsa_compress(torch.cat(self.index_keys), cu, self.cu_blocks, k_hat=self.k_hat)

    def expect(self, q, n, tokens):
        k, v = self.held(n, tokens)
        G = H_Q // H_KV
        parts = [attend(q[h * G:(h + 1) * G], k[:, h], v[:, h],
                        torch.ones(G, len(tokens), dtype=torch.bool, device=DEV), D ** -0.5, 0.0, True)
                 for h in range(H_KV)]
        return tuple(torch.cat(x) for x in zip(*parts))


def projection(T, seed):
    fused = normal((T, (H_Q + 2 * H_KV) * D), BF, seed)
    q, k, v = fused.split([H_Q * D, H_KV * D, H_KV * D], dim=1)
    return q.view(T, H_Q, D), k.view(T, H_KV, D), v.view(T, H_KV, D)


def test_prompts_then_listed_decode_then_drafts():
    lens, steps = [150, 9, 64, 301], 6
    layer = Layer(lens, steps)
    cu = torch.tensor([0] + lens).cumsum(0).to(**I32)
    q, k, v = projection(sum(lens), 1)
    qr = gdn.gdn_kv_append(k, v, layer.kv, cu, q=q, inv_freq=layer.freq)
    out, lse = gdn.gdn_attn_prefill(qr, layer.kv, cu)
    for n, L in enumerate(lens):
        for i in (0, L // 2, L - 1):
            t = int(cu[n]) + i
            check(out[t], lse[t], layer.expect(qr[t], n, torch.arange(i + 1, device=DEV)), f"prompt {n} {i}")
        layer.index_keys[n] = normal((L, 128), BF, 20 + n)
    ws = gdn.attn_decode_workspace(1, H_Q, H_KV, D)
    queries = []
    for s in range(steps):
        pos = torch.tensor(layer.lens, **I32)
        q, k, v = projection(layer.N, 100 + s)
        qr = gdn.gdn_kv_append(k[:, None], v[:, None], layer.kv, None, pos, q=q[:, None], inv_freq=layer.freq)
        queries.append(qr)
        for n in range(layer.N):
            layer.index_keys[n] = torch.cat([layer.index_keys[n], normal((1, 128), BF, 1000 + 10 * s + n)])
        layer.compress()
        iq = normal((layer.N, 4, 128), BF, 500 + s)
        _, _, listed = gdn.gdn_qsa_index_decode(iq, pos, layer.k_hat, layer.cu_blocks, BUDGET)
        out, lse = gdn.gdn_qsa_attn_decode(qr, pos, layer.kv, listed, recent=RECENT, workspace=ws)
        for n, L in enumerate(layer.lens):
            x = listed[n].long()
            near = torch.arange(max(0, L - RECENT + 1), L + 1, device=DEV)
            far = x[(x >= 0) & (x <= L - RECENT)]
            assert len(far) <= 4 * BUDGET and len(set(far.tolist())) == len(far)
            check(out[n, 0], lse[n, 0], layer.expect(qr[n, 0], n, torch.cat([far, near])), f"step {s} {n}")
        layer.lens = [L + 1 for L in layer.lens]
    # the same tokens as one call of drafts over the whole cache
    drafts = torch.cat(queries[-4:], dim=1).contiguous()
    pos = torch.tensor([L - 4 for L in layer.lens], **I32)
    out, lse = gdn.gdn_attn_decode(drafts, pos, layer.kv)
    for n in range(layer.N):
        for j in range(4):
            seen = torch.arange(layer.lens[n] - 3 + j, device=DEV)
            check(out[n, j], lse[n, j], layer.expect(drafts[n, j], n, seen), f"draft {n} {j}")


def test_decode_step_replayed_as_one_graph():
    """Append, index and listed attention captured once; positions, inputs and block cache change
    between replays."""
    lens, steps = [130, 40, 77], 5
    layer = Layer(lens, steps + 1)
    cu = torch.tensor([0] + lens).cumsum(0).to(**I32)
    q, k, v = projection(sum(lens), 1)
    gdn.gdn_kv_append(k, v, layer.kv, cu, inv_freq=layer.freq)
    layer.index_keys = [normal((L + steps, 128), BF, 20 + n) for n, L in enumerate(lens)]
    layer.compress()
    fused = [x.clone() for x in projection(layer.N, 2)]
    iq, pos = normal((layer.N, 4, 128), BF, 3), torch.tensor(lens, **I32)
    ws, iws = gdn.attn_decode_workspace(1, H_Q, H_KV, D), gdn.qsa_index_workspace(layer.N, layer.k_hat.shape[0])
    qr = torch.empty(layer.N, 1, H_Q, D, dtype=BF, device=DEV)
    out, lse = torch.empty_like(qr), torch.empty(layer.N, 1, H_Q, device=DEV)

    def step():
        q, k, v = (x[:, None] for x in fused)
        gdn.gdn_kv_append(k, v, layer.kv, None, pos, q=q, q_out=qr, inv_freq=layer.freq)
        _, _, listed = gdn.gdn_qsa_index_decode(iq, pos, layer.k_hat, layer.cu_blocks, BUDGET, workspace=iws)
        gdn.gdn_qsa_attn_decode(qr, pos, layer.kv, listed, recent=RECENT, out=out, lse=lse, workspace=ws)
        return listed

    def run(call):
        got = []
        pos.copy_(torch.tensor(lens))
        for s in range(steps):
            for x, y in zip(fused, projection(layer.N, 50 + s)):
                x.copy_(y)
            iq.copy_(normal(iq.shape, BF, 70 + s))
            call()
            got.append((out.clone(), lse.clone()))
            pos.add_(1)
        torch.cuda.synchronize()
        return got

    want = run(step)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for (a, b), (x, y) in zip(run(graph.replay), want):
        assert torch.equal(a, x) and torch.equal(b, y)


FIRST_CALLS = """
import torch, linear_attention_token_b200 as gdn
i32 = dict(dtype=torch.int32, device="cuda")
B, H_q, H_kv, d = 3, 8, 2, 128
k = torch.randn(40, 16, H_kv, d, dtype=torch.bfloat16, device="cuda")
kv = gdn.PagedKV(k, torch.randn_like(k), torch.arange(30, **i32).reshape(B, 10))
new = torch.randn(B, 1, H_kv, d, dtype=torch.bfloat16, device="cuda")
q = torch.randn(B, 1, H_q, d, dtype=torch.bfloat16, device="cuda")
prompt = torch.randn(B, 100, H_q, d, dtype=torch.bfloat16, device="cuda")
pos, idx = torch.tensor([120, 7, 90], **i32), torch.arange(60, **i32).expand(B, 60).contiguous()
freq = gdn.rope_inv_freq(d)

def step():
    turned = gdn.gdn_kv_append(new, new, kv, None, pos, q=q, inv_freq=freq)
    return (turned, *gdn.gdn_attn_decode(turned, pos, kv), *gdn.gdn_qsa_attn_decode(turned, pos, kv, idx, recent=4),
            *gdn.gdn_attn_prefill(prompt, kv))

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = step()
graph.replay()
torch.cuda.synchronize()
for a, b in zip(captured, step()):
    assert torch.equal(a, b)
print("same")
"""


def test_first_calls_inside_a_capture():
    """A process whose first calls are captured: what a first call sets up does not break the capture."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
