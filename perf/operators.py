"""What the attention operators over a paged key-value cache are measured on.

Four operators that belong together: appending keys and values to the cache with the
rotation applied on the way, attention of the newest tokens over the whole cache, the same
over the token lists that the QSA indexer returns, and attention of a prompt.

`own` false: the plain forms below (elementary torch operations in 32 bits, angles in 64).
`own` true: the calls of linear_attention_token_b200.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SCRATCH = 64 << 20                       # bytes of scratch a serving program keeps


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a batch: 64 sequences, one token each, at different positions
        dict(name="append step", op="append", n=64, tokens=64, past=4096, hq=32, hkv=8, d=128,
             page=64, rope=64, axes=1, dtype="bf16", mix=1),
        # prompts with image and video spans: positions on three axes; 32-bit cache, small heads
        dict(name="append axes", op="append", n=5, tokens=4099, past=1000, hq=8, hkv=4, d=64,
             page=16, rope=64, axes=3, dtype="f32", mix=2),
        # one long prompt's worth of tokens
        dict(name="append prompt", op="append", n=2, tokens=65536, past=0, hq=16, hkv=2, d=128,
             page=64, rope=128, axes=1, dtype="bf16", mix=3),
        # a handful of short chats: latency
        dict(name="decode short", op="decode", n=4, t=1, ctx=1024, hq=16, hkv=2, d=128, page=64,
             softcap=0.0, window=0, dtype="bf16", mix=4),
        # a ragged batch with one idle slot, two drafted tokens each, capped scores
        dict(name="decode ragged", op="decode", n=64, t=2, ctx=16384, hq=32, hkv=8, d=128, page=16,
             softcap=30.0, window=0, dtype="bf16", mix=5),
        # the native context length, few sequences
        dict(name="decode long", op="decode", n=8, t=1, ctx=262144, hq=16, hkv=2, d=128, page=64,
             softcap=0.0, window=0, dtype="bf16", mix=6),
        # the indexer's budget (512 blocks of 4 tokens) out of the native context length
        dict(name="listed few", op="listed", n=8, t=1, ctx=262144, budget=512, recent=4, hq=16,
             hkv=2, d=128, page=64, softcap=0.0, dtype="bf16", mix=7),
        # a serving batch whose four drafted tokens each have a list of their own
        dict(name="listed drafts", op="listed", n=32, t=4, ctx=32768, budget=512, recent=64, hq=16,
             hkv=2, d=128, page=64, softcap=0.0, dtype="bf16", mix=8),
        # one short prompt of odd length
        dict(name="prompt short", op="prompt", n=1, tokens=333, past=0, hq=16, hkv=2, d=128, page=64,
             softcap=0.0, window=0, prefix=0, dtype="bf16", mix=9),
        # two prompts of 4096 tokens, 16 heads
        dict(name="prompt mid", op="prompt", n=2, tokens=8192, past=0, hq=16, hkv=2, d=128, page=64,
             softcap=0.0, window=0, prefix=0, even=True, dtype="bf16", mix=10),
        # packed ragged prompts continuing cached ones, capped scores, prefixes seen both ways
        dict(name="prompt ragged", op="prompt", n=6, tokens=8191, past=4096, hq=16, hkv=4, d=128,
             page=16, softcap=30.0, window=0, prefix=1500, dtype="bf16", mix=11),
        # one long prompt
        dict(name="prompt long", op="prompt", n=1, tokens=16384, past=0, hq=16, hkv=2, d=128, page=64,
             softcap=0.0, window=0, prefix=0, dtype="bf16", mix=12),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["append", "decode", "listed", "prompt"])
    c = dict(op=op, hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128, 128]),
             page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]),
             mix=rng.randrange(1, 1 << 20))
    c["hq"] = c["hkv"] * rng.choice([1, 2, 4, 8])
    if op != "append":
        c["softcap"] = rng.choice([0.0, 0.0, 30.0])
    row = c["hkv"] * c["d"] * (2 if c["dtype"] == "bf16" else 4)
    if op == "append":
        c["n"] = _log(rng, 1, 256)
        c["tokens"] = max(c["n"], _log(rng, 64, 65536))
        while c["tokens"] * (2 * c["hkv"] + c["hq"]) * c["d"] * (2 if c["dtype"] == "bf16" else 4) > 330e6:
            c["tokens"] = max(1, c["tokens"] // 2)
        c["n"] = min(c["n"], c["tokens"])
        c["past"] = _log(rng, 1, 4096)
        c["rope"] = rng.choice([c["d"] // 2, c["d"]])
        c["axes"] = rng.choice([1, 1, 3])
    elif op in ("decode", "listed"):
        c["n"] = _log(rng, 1, 128)
        c["t"] = rng.choice([1, 1, 2, 3, 4])
        c["ctx"] = _log(rng, 16, 262144)
        while c["n"] * c["ctx"] * row > 1.0e9:
            c["ctx"] = max(1, c["ctx"] // 2)
        if op == "decode":
            c["window"] = rng.choice([0, 0, _log(rng, 16, 8192)])
        else:
            c["budget"] = _log(rng, 16, 512)
            c["recent"] = rng.choice([4, rng.randrange(1, 300)])
    else:
        c["n"] = _log(rng, 1, 8)
        c["tokens"] = max(c["n"], _log(rng, 64, 6000 if c["dtype"] == "bf16" else 1500))
        c["past"] = rng.choice([0, _log(rng, 16, 4096)])
        c["window"] = rng.choice([0, 0, _log(rng, 64, 2048)])
        c["prefix"] = 0 if c["window"] else rng.choice([0, 0, _log(rng, 16, 1024)])
    return c


def _lengths(case):
    """Tokens of this call and tokens cached before it, for each sequence."""
    rng, n = random.Random(case["mix"]), case["n"]
    if case["op"] in ("append", "prompt"):
        total = case["tokens"]
        if case.get("even") or n == 1 or total < 2 * n:
            new = [total // n + (i < total % n) for i in range(n)]
        else:
            cuts = sorted(rng.sample(range(1, total), n - 1))
            new = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        past = [rng.randrange(case["past"] // 2, case["past"] + 1) for _ in range(n)]
        return new, past
    # the last of the t newest tokens is at the context's end; a large batch has an idle slot
    ctx = case["ctx"] if n <= 8 else None
    past = [(ctx or rng.randrange(max(1, case["ctx"] // 8), case["ctx"] + 1)) - case["t"] for _ in range(n)]
    if n > 8:
        past[n // 2] = -case["t"]
    return [case["t"]] * n, past


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    new, past = _lengths(case)
    n, hq, hkv, d, page = case["n"], case["hq"], case["hkv"], case["d"], case["page"]
    ints = dict(dtype=torch.int32, device="cuda")

    def normal(*shape, by=1.0):
        x = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
        return x.mul_(by) if by != 1.0 else x

    most = max(1, max(max(p, 0) + t for p, t in zip(past, new)))
    per_seq = (most + page - 1) // page
    pages = n * per_seq + 3                          # a cache has free pages too
    order = torch.randperm(pages, generator=g, device="cuda")
    s = dict(case=case, dtype=dt, most=most,
             k_cache=normal(pages, page, hkv, d), v_cache=normal(pages, page, hkv, d),
             table=order[:n * per_seq].reshape(n, per_seq).to(torch.int32).contiguous(),
             pos0=torch.tensor(past, **ints), new=torch.tensor(new, device="cuda"),
             scratch=torch.zeros(SCRATCH, dtype=torch.uint8, device="cuda"), longest=max(new))
    if case["op"] in ("append", "prompt"):
        s["cu"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
        total = sum(new)
        # queries come as their projection leaves them: scores of a few units
        s["q"] = normal(total, hq, d, by=1.5)
        s["out"] = torch.empty_like(s["q"])
    if case["op"] == "append":
        s["k"], s["v"] = normal(total, hkv, d), normal(total, hkv, d)
        half = case["rope"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
        s["sections"] = None
        if case["axes"] == 3:
            # time runs on, height and width stay inside a frame
            at = torch.arange(total, device="cuda")
            s["rope_pos"] = torch.stack([at // 64, at % 64 // 8, at % 8]).to(torch.int32).contiguous()
            s["sections"] = (half - 2 * (half // 3), half // 3, half // 3)
    elif case["op"] == "prompt":
        s["prefix"] = None
        if case["prefix"]:
            rng = random.Random(case["mix"] + 1)
            s["prefix"] = torch.tensor([rng.randrange(0, case["prefix"] + 1) for _ in range(n)], **ints)
    else:
        s["q"] = normal(n, case["t"], hq, d, by=1.5)
        s["out"] = torch.empty_like(s["q"])
    if case["op"] == "listed":
        # the indexer's lists: whole blocks of 4 tokens at or before the query, in order, then -1
        t, budget, blocks = case["t"], case["budget"], max(1, (most + 3) // 4)
        at = s["pos0"][:, None] + torch.arange(t, device="cuda")[None]
        may = torch.arange(blocks, device="cuda")[None, None] * 4 + 3 <= at[..., None]
        score = torch.rand(n, t, blocks, generator=g, device="cuda").masked_fill_(~may, -1.0)
        k = min(budget, blocks)
        best, which = score.topk(k, dim=-1)
        which = which.masked_fill(best < 0, blocks).sort(dim=-1).values
        tok = which[..., None] * 4 + torch.arange(4, device="cuda")
        tok = tok.masked_fill((which == blocks)[..., None], -1).reshape(n, t, 4 * k)
        idx = torch.full((n, t, 4 * budget), -1, device="cuda")
        idx[..., :4 * k] = tok
        s["tokens"] = idx.to(torch.int32).contiguous()
    if own:                                          # the handle that a program keeps with its cache
        import linear_attention_token_b200 as gdn
        s["gdn"], s["kv"] = gdn, gdn.PagedKV(s["k_cache"], s["v_cache"], s["table"])
    return s


# ------------------------------------------------------------------------------ passes
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    c, gdn = s["case"], s["gdn"]
    if c["op"] == "append":
        gdn.gdn_kv_append(s["k"], s["v"], s["kv"], s["cu"], s["pos0"], q=s["q"], q_out=s["out"],
                          inv_freq=s["inv_freq"], rope_pos=s.get("rope_pos"),
                          rope_sections=s["sections"])
        return s["out"], s["k_cache"], s["v_cache"]
    if c["op"] == "decode":
        return gdn.gdn_attn_decode(s["q"], s["pos0"], s["kv"], scale=c["d"] ** -0.5,
                                   softcap=c["softcap"], window=c["window"], out=s["out"],
                                   workspace=s["scratch"])
    if c["op"] == "listed":
        return gdn.gdn_qsa_attn_decode(s["q"], s["pos0"], s["kv"], s["tokens"], recent=c["recent"],
                                       scale=c["d"] ** -0.5, softcap=c["softcap"], out=s["out"],
                                       workspace=s["scratch"])
    return gdn.gdn_attn_prefill(s["q"], s["kv"], s["cu"], s["pos0"], prefix_len=s["prefix"],
                                scale=c["d"] ** -0.5, softcap=c["softcap"], window=c["window"],
                                out=s["out"], workspace=s["scratch"])


def _slots(s, tokens):
    """Rows of the cache that hold tokens [n, m] of the n sequences."""
    page = s["case"]["page"]
    return torch.gather(s["table"].long(), 1, tokens // page) * page + tokens % page


def _softmax_pv(x, seen, v, softcap):
    """x scores [..., r, m], seen broadcastable to it, v [..., m, d]: output and log-sum."""
    if softcap:
        x = x.div_(softcap).tanh_().mul_(softcap)
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out = (x @ v) / torch.where(total == 0, torch.ones_like(total), total)
    return out, (total.log() + top).squeeze(-1)


def _plain(s):
    c = s["case"]
    hq, hkv, d, n = c["hq"], c["hkv"], c["d"], c["n"]
    group, scale = hq // hkv, c["d"] ** -0.5
    if c["op"] == "append":
        return _plain_append(s)
    kc, vc = s["k_cache"].view(-1, hkv, d), s["v_cache"].view(-1, hkv, d)
    pos0 = s["pos0"].long()
    every = torch.arange(s["most"], device="cuda")
    if c["op"] == "decode":
        at = (pos0[:, None] + torch.arange(c["t"], device="cuda"))[:, None, :, None, None]
        tok = every[None].expand(n, -1)
        slots = _slots(s, tok)
        k = kc[slots].permute(0, 2, 3, 1).float()                 # [n, hkv, d, m]
        v = vc[slots].permute(0, 2, 1, 3).float()
        q = s["q"].float().view(n, c["t"], hkv, group, d).transpose(1, 2).reshape(n, hkv, c["t"] * group, d)
        seen = every <= at
        if c["window"]:
            seen = seen & (every > at - c["window"])
        seen = seen.expand(n, 1, c["t"], group, -1).reshape(n, 1, c["t"] * group, -1)
        out, lse = _softmax_pv((q * scale) @ k, seen, v, c["softcap"])
        out = out.view(n, hkv, c["t"], group, d).transpose(1, 2).reshape(n, c["t"], hq, d)
        lse = lse.view(n, hkv, c["t"], group).transpose(1, 2).reshape(n, c["t"], hq)
        return out.to(s["dtype"]), lse
    if c["op"] == "listed":
        at = pos0[:, None] + torch.arange(c["t"], device="cuda")              # [n, t]
        newest = at[..., None] - torch.arange(c["recent"], device="cuda")     # the newest tokens
        lst = s["tokens"].long()
        tok = torch.cat([lst, newest], -1)
        seen = torch.cat([(lst >= 0) & (lst <= at[..., None] - c["recent"]), newest >= 0], -1)
        slots = _slots(s, tok.clamp(0, s["most"] - 1).view(n, -1)).view(tok.shape)
        k = kc[slots].permute(0, 1, 3, 4, 2).float()                          # [n, t, hkv, d, m]
        v = vc[slots].permute(0, 1, 3, 2, 4).float()
        q = s["q"].float().view(n, c["t"], hkv, group, d)
        out, lse = _softmax_pv((q * scale) @ k, seen[:, :, None, None], v, c["softcap"])
        return out.reshape(n, c["t"], hq, d).to(s["dtype"]), lse.reshape(n, c["t"], hq)
    # prompt: pad the packed queries to [n, longest]
    cu, step = s["cu"].long(), torch.arange(s["longest"], device="cuda")
    live = step < s["new"][:, None]                                           # [n, longest]
    row = (cu[:-1, None] + step).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(n, -1, hkv, group, d).permute(0, 2, 3, 1, 4)
    slots = _slots(s, every[None].expand(n, -1))
    k = kc[slots].permute(0, 2, 3, 1).float()[:, :, None]                     # [n, hkv, 1, d, m]
    v = vc[slots].permute(0, 2, 1, 3).float()[:, :, None]
    at = (pos0[:, None] + step)[..., None]                                    # [n, longest, 1]
    seen = every <= at
    if c["window"]:
        seen = seen & (every > at - c["window"])
    if s["prefix"] is not None:
        seen = seen | (every < s["prefix"].long()[:, None, None])
    seen = seen & (every < (pos0 + s["new"])[:, None, None])
    out, lse = _softmax_pv((q * scale) @ k, seen[:, None, None], v, c["softcap"])
    out = out.permute(0, 3, 1, 2, 4).reshape(n, -1, hq, d)[live]
    return out.to(s["dtype"]), lse.permute(0, 3, 1, 2).reshape(n, -1, hq)[live]


def _plain_append(s):
    c, cu = s["case"], s["cu"].long()
    token = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(cu[1:], token, right=True)
    at = s["pos0"].long()[seq] + token - cu[seq]
    half = c["rope"] // 2
    if s["sections"] is None:
        place = at[:, None].expand(-1, half)
    else:
        axis = torch.repeat_interleave(torch.arange(3, device="cuda"),
                                       torch.tensor(s["sections"], device="cuda"), output_size=half)
        place = s["rope_pos"].long()[axis].T
    angle = place.double() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def rotate(x):
        x = x.float()
        a, b = x[..., :half], x[..., half:c["rope"]]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., c["rope"]:]], -1).to(s["dtype"])

    page = c["page"]
    slot = s["table"].long()[seq, at // page] * page + at % page
    s["k_cache"].view(-1, c["hkv"], c["d"])[slot] = rotate(s["k"])
    s["v_cache"].view(-1, c["hkv"], c["d"])[slot] = s["v"]
    return rotate(s["q"]), s["k_cache"], s["v_cache"]


# ------------------------------------------------------------------- operators in 64 bits
def exact(case, seed):
    """From the definitions, one sequence and head at a time, in 64 bits."""
    s = prepare(case, seed)
    new, past = _lengths(case)
    hq, hkv, d, page, n = case["hq"], case["hkv"], case["d"], case["page"], case["n"]
    dev = "cuda"
    if case["op"] == "append":
        out = s["q"].double()
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        half = case["rope"] // 2
        freq = s["inv_freq"].double()
        first = 0
        for i in range(n):
            rows = torch.arange(first, first + new[i], device=dev)
            pos = torch.arange(past[i], past[i] + new[i], device=dev)
            where = s["table"][i].long()[pos // page], pos % page
            turn = torch.empty(new[i], half, dtype=torch.float64, device=dev)
            for f in range(half):
                p = pos
                if s["sections"] is not None:
                    a = 0 if f < s["sections"][0] else 1 if f < s["sections"][0] + s["sections"][1] else 2
                    p = s["rope_pos"][a, rows].long()
                turn[:, f] = p.double() * freq[f]
            unit = torch.polar(torch.ones_like(turn), turn)[:, None]
            for x, put in ((s["q"], None), (s["k"], kc)):
                x = x[rows].double()
                z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * unit
                x[..., :half], x[..., half:2 * half] = z.real, z.imag
                if put is None:
                    out[rows] = x
                else:
                    put[where] = x
            vc[where] = s["v"][rows].double()
            first += new[i]
        return out, kc, vc
    kc, vc = s["k_cache"].view(-1, hkv, d), s["v_cache"].view(-1, hkv, d)
    shape = s["q"].shape
    q = s["q"].reshape(-1, hq, d)
    out = torch.zeros(q.shape, dtype=torch.float64, device=dev)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=dev)
    first = 0
    for i in range(n):
        end = past[i] + new[i]
        for b in range(0, new[i], 4096 if case["op"] == "prompt" else 1):
            e = min(new[i], b + 4096) if case["op"] == "prompt" else b + 1
            pos = torch.arange(past[i] + b, past[i] + e, device=dev)
            last = end if case["op"] == "prompt" else past[i] + e
            if last <= 0:
                continue
            if case["op"] == "listed":
                x = s["tokens"][i, b].long()
                p = past[i] + b
                near = torch.arange(max(0, p - case["recent"] + 1), p + 1, device=dev)
                tok = torch.cat([x[(x >= 0) & (x <= p - case["recent"])], near])
                ok = torch.ones(1, len(tok), dtype=torch.bool, device=dev)
            else:
                tok = torch.arange(last, device=dev)
                ok = tok <= pos[:, None]
                if case["window"]:
                    ok &= pos[:, None] - tok < case["window"]
                if s.get("prefix") is not None:
                    ok |= tok < s["prefix"][i]
            slot = s["table"][i].long()[tok // page] * page + tok % page
            for h in range(hq):
                if h % (hq // hkv) == 0:
                    k, v = (x[slot, h // (hq // hkv)].double() for x in (kc, vc))
                x = q[first + b:first + e, h].double() @ k.T / math.sqrt(d)
                if case["softcap"]:
                    x = case["softcap"] * torch.tanh(x / case["softcap"])
                x = torch.where(ok, x, -math.inf)
                z = torch.logsumexp(x, -1)
                out[first + b:first + e, h] = torch.exp(x - z[:, None]) @ v
                lse[first + b:first + e, h] = z
        first += new[i]
    return out.view(shape), lse.view(shape[:-1])


# -------------------------------------------------------------------------------- work
def _pairs(case):
    """(query tokens, their visible tokens in all, cached tokens that some query of the sequence sees)."""
    new, past = _lengths(case)
    pairs, read = 0, 0
    prefix = [0] * case["n"]
    if case.get("prefix"):
        rng = random.Random(case["mix"] + 1)
        prefix = [rng.randrange(0, case["prefix"] + 1) for _ in range(case["n"])]
    for m, p, pre in zip(new, past, prefix):
        if case["op"] == "listed":
            for j in range(m):
                at = p + j
                near = max(0, min(case["recent"], at + 1))
                far = min(4 * case["budget"], (at + 1) // 4 * 4) if at >= 0 else 0
                # lists skip the newest tokens: at most a few blocks of a long context
                far = min(far, max(0, at + 1 - near))
                pairs += far + near
                read += far + near
            continue
        w = case["window"] or (1 << 40)
        for j in range(m):
            at = p + j
            pairs += max(max(0, min(w, at + 1)), min(pre, p + m))
        read += max(0, min(p + m, w + m - 1))
    return sum(new), pairs, read


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        rows = case["tokens"]
        turns = rows * (case["hq"] + case["hkv"]) * case["rope"] // 2
        return {"bytes": 2 * rows * (case["hq"] + 2 * case["hkv"]) * case["d"] * size
                + rows * 4 * (case["axes"] if case["axes"] > 1 else 0), "flops": 6 * turns}
    rows, pairs, read = _pairs(case)
    listed_tokens = 16 * case["budget"] * rows if case["op"] == "listed" else 0
    return {"bytes": 2 * read * case["hkv"] * case["d"] * size + 2 * rows * case["hq"] * case["d"] * size
            + rows * case["hq"] * 4 + listed_tokens, "flops": 4 * pairs * case["hq"] * case["d"]}
