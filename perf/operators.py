"""The serving operators of a speculative rollout step, as cases to be timed: keys and values
appended to a paged cache, attention of new tokens over it, and the verification of drafted tokens.

``run`` computes them in plain torch, or with ``own`` through the package's entry points.
"""

import math
import random

import torch

own = False

VPAD, VREAL = 152576, 151936
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------ the cases

def _attention(name, B, n, heads, kv_heads, dim, page, max_len, **kw):
    return {"name": name, "kind": "attention", "B": B, "n": n, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "max_len": max_len, "dtype": "bf16", "order": "token", "window": 0,
            "sinks": 0, "ragged": True} | kw


def _append(name, B, n, kv_heads, dim, page, max_len, **kw):
    return {"name": name, "kind": "append", "B": B, "n": n, "kv_heads": kv_heads, "dim": dim, "page": page,
            "max_len": max_len, "dtype": "bf16", "order": "token", "ragged": True} | kw


def _verify(name, B, n, **kw):
    return {"name": name, "kind": "verify", "B": B, "n": n, "draft_logits": True, "tau": 0.7, "top_k": 50,
            "top_p": 0.95, "mixed": False} | kw


def listed():
    return [
        # one request of about a thousand tokens, one new token: latency is all that counts
        _attention("attend_one", 1, 1, 32, 8, 128, 16, 1003, ragged=False),
        # an ordinary decode batch of unequal requests, one slot of it empty
        _attention("attend_batch", 64, 1, 32, 8, 128, 64, 8192),
        # long contexts, few requests: the split over the length
        _attention("attend_long", 4, 1, 32, 8, 128, 64, 131071),
        # four drafted tokens and the last accepted one, pages ordered by head
        _attention("attend_drafts", 128, 5, 32, 8, 128, 16, 4096, order="head"),
        # a sliding window with sinks, half precision, 64-wide heads, pages of an odd size
        _attention("attend_window", 64, 1, 64, 8, 64, 24, 16384, dtype="f16", window=1024, sinks=4),
        # a decode step's new token
        _append("append_one", 64, 1, 8, 128, 64, 512),
        # prompts written at once
        _append("append_prompts", 16, 2048, 8, 128, 16, 2500),
        # one request, four drafts of a draft model
        _verify("verify_one", 1, 4),
        # drafts without a distribution (looked up in the prompt): point masses
        _verify("verify_lookup", 64, 3, draft_logits=False, tau=1.0, top_k=128, top_p=1.0),
        # a rollout batch with a draft model
        _verify("verify_batch", 128, 4, tau=1.3, top_k=128, top_p=1.0),
        # requests with their own settings (greedy ones among them) and their own numbers of drafts
        _verify("verify_mixed", 96, 7, mixed=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "attention", "append", "verify", "verify"])
    if kind == "attention":
        heads, kv_heads = rng.choice([(32, 8), (64, 8), (16, 16), (28, 4), (8, 1), (40, 8)])
        dim = rng.choice([64, 128])
        B, n = _log_int(rng, 1, 128), rng.choice([1, 1, 1, 2, 3, 5, 8])
        top = min(131072, 400_000_000 // (B * kv_heads * dim), 60_000_000 // (B * heads * n))
        windowed = rng.random() < 0.3
        c = _attention("", B, n, heads, kv_heads, dim, rng.choice([16, 24, 32, 64, 100, 128]),
                       _log_int(rng, n, max(n, top)), dtype=rng.choice(["bf16", "bf16", "f16"]),
                       order=rng.choice(["token", "head"]), window=_log_int(rng, 16, 8192) if windowed else 0,
                       sinks=rng.randrange(9) if windowed else 0, ragged=rng.random() < 0.8)
    elif kind == "append":
        B, n = _log_int(rng, 1, 128), _log_int(rng, 1, 2048)
        n = min(n, 32768 // B)
        c = _append("", B, n, rng.choice([1, 4, 8, 16]), rng.choice([64, 128]), rng.choice([16, 24, 64, 128]),
                    n + rng.randrange(1, 600), dtype=rng.choice(["bf16", "f16"]),
                    order=rng.choice(["token", "head"]), ragged=rng.random() < 0.8)
    else:
        n = rng.randrange(1, 9)
        c = _verify("", _log_int(rng, 1, 1400 // (2 * n + 1)), n, draft_logits=rng.random() < 0.7,
                    tau=rng.choice([0.6, 0.7, 1.0, 1.3]), top_k=rng.choice([20, 50, 100, 128]),
                    top_p=rng.choice([1.0, 1.0, 0.9]), mixed=rng.random() < 0.25)
    del c["name"]
    return c


def _lens(case):
    """Tokens of each sequence, the new ones included: spread over the logarithm where ragged, one of them empty."""
    B, n, top = case["B"], case["n"], case["max_len"]
    if not case["ragged"]:
        return [top] * B
    rng = random.Random(B * 1_000_003 + top)
    lens = [_log_int(rng, max(n, top // 16), top) for _ in range(B)]
    lens[B // 2] = top
    if B >= 8:
        lens[B // 3] = n
        lens[2] = 0
    return lens


def _news(case):
    """New tokens of each sequence: all n, but none in the empty sequence of a larger ragged batch, and one fewer in another."""
    new = [case["n"]] * case["B"]
    if case["ragged"] and case["B"] >= 8:
        new[1], new[2] = max(1, case["n"] - 1), 0
    return new


# ------------------------------------------------------------ inputs

def _cache(case, lens, g, filled):
    """A paged cache [pages, page, kv_heads, dim] (as a view, whatever its order in memory) and a page table."""
    page, H, D, dt = case["page"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    shape = (pages, page, H, D) if case["order"] == "token" else (pages, H, page, D)

    def values():
        if not filled:
            return torch.zeros(shape, dtype=dt, device="cuda")
        out = torch.empty(shape, dtype=dt, device="cuda")
        for a in range(0, pages, 4096):
            part = out[a:a + 4096]
            part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
        return out

    k, v = values(), values()
    if case["order"] == "head":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    # each sequence's pages in the order in which a busy allocator would have given them
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).tolist()
    table, at = torch.zeros((case["B"], max(1, max(need))), dtype=torch.int32), 0
    for b, m in enumerate(need):
        table[b, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
        at += m
    return k, v, table.cuda()


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s = {"case": case}
    if case["kind"] == "verify":
        return _prepare_verify(case, g, s)
    lens, new, dt = _lens(case), _news(case), DTYPES[case["dtype"]]
    s["k_cache"], s["v_cache"], s["table"] = _cache(case, lens, g, case["kind"] == "attention")
    s["lens"], s["new"] = _int32(lens), _int32(new)
    B, n, D = case["B"], case["n"], case["dim"]
    if case["kind"] == "attention":
        s["q"] = (2.0 * randn(B, n, case["heads"], D)).to(dt)
    else:
        # keys and values as they come out of one projection: views of a wider row
        kv = randn(B, n, 2, case["kv_heads"], D).to(dt)
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
    return s


def _settings(case):
    """(temperature, top_p, top_k) of each sequence, for target and draft, where the requests differ."""
    rng = random.Random(case["B"] * 31 + case["n"])
    kinds = [(0.0, 1.0, -1), (0.7, 0.95, 50), (1.0, 1.0, 128), (1.3, 1.0, 20), (0.6, 1.0, 64)]
    return [rng.choice(kinds) for _ in range(case["B"])]


def _num_drafts(case):
    rng = random.Random(case["B"] * 37 + case["n"])
    return [rng.randrange(case["n"] + 1) if case["mixed"] else case["n"] for _ in range(case["B"])]


def _prepare_verify(case, g, s):
    B, n = case["B"], case["n"]

    def words(*shape):
        return torch.randint(-2**31, 2**31, shape, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)

    # a few confident tokens on a noisy background, and a draft model that is near the target
    logits = torch.empty((B * (n + 1), VPAD), dtype=torch.bfloat16, device="cuda")
    draft = torch.empty((B * n, VPAD), dtype=torch.bfloat16, device="cuda")
    token = torch.empty((B, n), dtype=torch.int32, device="cuda")
    for a in range(0, B, 16):
        m = min(B, a + 16) - a
        x = 4.0 * torch.randn((m, n + 1, VPAD), generator=g, device="cuda")
        x += 12.0 * (torch.rand(x.shape, generator=g, device="cuda") < 96.0 / VREAL)
        x[..., VREAL:] = -math.inf
        y = x[:, :n] + 0.4 * torch.randn((m, n, VPAD), generator=g, device="cuda")
        logits[a * (n + 1):(a + m) * (n + 1)] = x.reshape(-1, VPAD).to(torch.bfloat16)
        draft[a * n:(a + m) * n] = y.reshape(-1, VPAD).to(torch.bfloat16)
        top = y.topk(20, dim=-1)      # drafted from among the draft model's first 20 tokens
        noise = torch.rand(top.values.shape, generator=g, device="cuda").clamp_(1e-9).log_().neg_().log_().neg_()
        pick = (top.values / case["tau"] + noise).argmax(-1, keepdim=True)
        token[a:a + m] = top.indices.gather(-1, pick)[..., 0].to(torch.int32)
    if case["mixed"]:
        kinds = _settings(case)
        s["tau"] = torch.tensor([v[0] for v in kinds], device="cuda")
        s["top_p"] = torch.tensor([v[1] for v in kinds], device="cuda")
        s["top_k"] = _int32([v[2] for v in kinds])
        greedy = (s["tau"] == 0).repeat_interleave(n)
        best = draft[:, :VREAL].float().argmax(1).to(torch.int32)
        token = torch.where(greedy, best, token.reshape(-1)).reshape(B, n)
    else:
        s["tau"], s["top_p"], s["top_k"] = case["tau"], case["top_p"], case["top_k"]
    s["logits"], s["draft"], s["token"] = logits, draft if case["draft_logits"] else None, token
    s["num"] = _int32(_num_drafts(case)) if case["mixed"] else None
    s["accept"], s["draw"] = words(B, n), words(B)
    return s


# ------------------------------------------------------------ one pass

def run(s):
    kind = s["case"]["kind"]
    if own:
        import rollout_consistent_vocab_gb300 as rlk
        if kind == "attention":
            out, lse = rlk.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                           new_lens=s["new"], window=s["case"]["window"], sinks=s["case"]["sinks"])
            return {"out": out, "lse": lse}
        if kind == "append":
            rlk.kv_append(s["k_cache"], s["v_cache"], s["table"], s["lens"], s["k"], s["v"], new_lens=s["new"])
            return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        token, accepted, restr, full = rlk.verify_drafts(
            s["logits"], s["token"], s["tau"], s["top_p"], s["top_k"], draft_logits=s["draft"],
            num_drafts=s["num"], accept_uniform=s["accept"], draw_uniform=s["draw"])
        return {"token": token, "accepted": accepted, "restr": restr, "full": full}
    if kind == "attention":
        return _plain_attention(s)
    return _plain_append(s) if kind == "append" else _plain_verify(s)


def _positions(s, n):
    """Position of each new token [B, n], and whether it is there."""
    i = torch.arange(n, device="cuda")
    lens, new = s["lens"].long()[:, None], s["new"].long()[:, None]
    return lens - new + i, i < new


def _plain_attention(s):
    c = s["case"]
    B, n, Hq, Hkv, D = c["B"], c["n"], c["heads"], c["kv_heads"], c["dim"]
    G, L = Hq // Hkv, s["table"].shape[1] * c["page"]
    rows = s["table"].long()
    k = s["k_cache"][rows].reshape(B, L, Hkv, D).permute(0, 2, 3, 1).float()
    v = s["v_cache"][rows].reshape(B, L, Hkv, D).permute(0, 2, 1, 3).float()
    q = s["q"].float().reshape(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    x = torch.matmul(q, k) * (1.0 / math.sqrt(D))
    pos, there = _positions(s, n)
    j = torch.arange(L, device="cuda")
    seen = (j <= pos[..., None]) & there[..., None]
    if c["window"]:
        seen &= (j > pos[..., None] - c["window"]) | (j < c["sinks"])
    x.masked_fill_(~seen[:, None, :, None, :].expand(B, 1, n, G, L).reshape(B, 1, n * G, L), -math.inf)
    m = x.max(-1, keepdim=True).values
    e = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(z == 0, torch.ones_like(z), z)
    lse = torch.log(z) + m
    o = o.reshape(B, Hkv, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D).to(s["q"].dtype)
    return {"out": o, "lse": lse.reshape(B, Hkv, n, G).permute(0, 2, 1, 3).reshape(B, n, Hq)}


def _plain_append(s):
    n, page = s["case"]["n"], s["case"]["page"]
    pos, there = _positions(s, n)
    b, i = torch.nonzero(there, as_tuple=True)
    t = pos[b, i]
    p = s["table"][b, t // page].long()
    s["k_cache"][p, t % page] = s["k"][b, i]
    s["v_cache"][p, t % page] = s["v"][b, i]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _per_row(value, repeat, like):
    """A setting for each of the rows: given once, or by sequence."""
    if isinstance(value, torch.Tensor):
        return value.repeat_interleave(repeat)[:, None]
    return like.new_full((like.shape[0], 1), value)


def _restricted(bits, tau, top_p, top_k):
    """Probabilities under top-k, then top-p; ln of the restricted and the full normaliser; maximum; temperature."""
    x = bits[:, :VREAL].float()
    t = _per_row(tau, x.shape[0] // tau.shape[0] if isinstance(tau, torch.Tensor) else 1, x)
    p = _per_row(top_p, x.shape[0] // top_p.shape[0] if isinstance(top_p, torch.Tensor) else 1, x)
    k = _per_row(top_k, x.shape[0] // top_k.shape[0] if isinstance(top_k, torch.Tensor) else 1, x).long()
    greedy = t == 0
    t = torch.where(greedy, torch.ones_like(t), t)
    m = x.max(1, keepdim=True).values
    e = torch.exp((x - m) / t)
    z = e.sum(1, keepdim=True)
    # every k is at most 128 here (greedy rows aside): the 128 largest hold what top-k and top-p go by
    top = x.topk(128, dim=1).values
    kth = torch.where(k > 0, top.gather(1, k.clamp(1, 128) - 1), torch.full_like(m, -math.inf))
    zk = (e * (x >= kth)).sum(1, keepdim=True)
    mass = torch.exp((top - m) / t)
    above = mass.cumsum(1) - mass
    above = above.gather(1, torch.searchsorted(-top, -top))       # equal values share what is above them
    kept = (above < p * zk) & (top >= kth)
    low = torch.where(kept, top, torch.full_like(top, math.inf)).min(1, keepdim=True).values
    low = torch.where(p < 1, torch.maximum(low, kth), kth)
    e = e * (x >= low)
    zs = e.sum(1, keepdim=True)
    first = torch.zeros_like(e).scatter_(1, x.argmax(1, keepdim=True), 1.0)
    prob = torch.where(greedy, first, e / zs)
    return prob, torch.log(zs), torch.log(z), m, t, greedy


def _plain_verify(s):
    c = s["case"]
    B, n = c["B"], c["n"]
    prob, ln_s, ln_z, m, t, greedy = _restricted(s["logits"], s["tau"], s["top_p"], s["top_k"])
    d = s["token"].long()
    p = prob.reshape(B, n + 1, VREAL)
    if s["draft"] is None:
        q = torch.zeros((B, n, VREAL), device="cuda").scatter_(2, d[..., None], 1.0)
    else:
        q = _restricted(s["draft"], s["tau"], s["top_p"], s["top_k"])[0].reshape(B, n, VREAL)
    u = ((s["accept"].long() & 0xFFFFFFFF) >> 8).float() * 2.0**-24
    num = torch.full((B,), n, device="cuda") if s["num"] is None else s["num"].long()
    i = torch.arange(n, device="cuda")
    ok = u * q.gather(2, d[..., None])[..., 0] < p[:, :n].gather(2, d[..., None])[..., 0]
    accepted = (ok & (i < num[:, None])).long().cumprod(1).sum(1)
    b = torch.arange(B, device="cuda")
    pa = p[b, accepted]
    qa = q[b, accepted.clamp(max=n - 1)] * (accepted < num)[:, None]
    r = (pa - qa).clamp(min=0)
    r = torch.where(r.sum(1, keepdim=True) > 0, r, pa)
    cdf = r.cumsum(1)
    draw_at = (s["draw"].long() & 0xFFFFFFFF).float()[:, None] * 2.0**-32 * cdf[:, -1:]
    drawn = (cdf > draw_at).int().argmax(1)
    i = torch.arange(n + 1, device="cuda")
    token = torch.cat([d, d[:, :1]], 1)
    token = torch.where(i < accepted[:, None], token, drawn[:, None])
    there = i <= accepted[:, None]
    x = s["logits"].reshape(B, n + 1, VPAD).gather(2, token[..., None])[..., 0].float()
    x = (x - m.reshape(B, n + 1)) / t.reshape(B, n + 1)
    there_g = there & ~greedy.reshape(B, n + 1)
    zero = torch.zeros_like(x)
    return {"token": torch.where(there, token, torch.full_like(token, -1)).to(torch.int32),
            "accepted": accepted.to(torch.int32),
            "restr": torch.where(there_g, x - ln_s.reshape(B, n + 1), zero),
            "full": torch.where(there_g, x - ln_z.reshape(B, n + 1), zero)}


# ------------------------------------------------------------ what a pass has to read, write and compute

def work(case):
    B, n = case["B"], case["n"]
    if case["kind"] == "verify":
        num = _num_drafts(case)
        rows = sum(v + 1 for v in num) + (sum(num) if case["draft_logits"] else 0)
        return {"bytes": rows * VREAL * 2 + B * (n + 1) * 20, "flops": rows * VREAL * 4}
    lens, new, D, H = _lens(case), _news(case), case["dim"], case["kv_heads"]
    if case["kind"] == "append":
        return {"bytes": sum(new) * H * D * 2 * 2 * 2 + B * 8, "flops": 0}
    window, sinks = case["window"], case["sinks"]
    tokens = pairs = 0
    for length, m in zip(lens, new):
        seen = set_size = 0
        for i in range(m):
            pos = length - m + i
            low = max(0, pos - window + 1) if window else 0
            set_size += pos + 1 - low + min(sinks if window else 0, low)
        if m:
            low = max(0, length - m - window + 1) if window else 0
            seen = length - low + min(sinks if window else 0, low)
        tokens += seen
        pairs += set_size
    return {"bytes": tokens * H * D * 2 * 2 + sum(new) * case["heads"] * D * 2 + B * n * case["heads"] * (D * 2 + 4),
            "flops": 4 * D * case["heads"] * pairs}


# ------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "attention":
        return _exact_attention(s)
    if case["kind"] == "append":
        return _exact_append(s)
    return _exact_verify(s)


def _exact_attention(s):
    """Sequence by sequence, over the tokens that each query sees."""
    c = s["case"]
    lens, new, page, G = _lens(c), _news(c), c["page"], c["heads"] // c["kv_heads"]
    out = torch.zeros((c["B"], c["n"], c["heads"], c["dim"]), dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], c["n"], c["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        pages = s["table"][b, :-(-lens[b] // page)].long()
        k = s["k_cache"][pages].flatten(0, 1)[:lens[b]].double()
        v = s["v_cache"][pages].flatten(0, 1)[:lens[b]].double()
        for i in range(new[b]):
            end = lens[b] - new[b] + i + 1
            at = list(range(end))
            if c["window"] and end > c["window"]:
                at = list(range(min(c["sinks"], end - c["window"]))) + list(range(end - c["window"], end))
            at = torch.tensor(at, device="cuda") if len(at) < end else slice(0, end)
            for h in range(c["kv_heads"]):
                x = k[at, h] @ s["q"][b, i, h * G:(h + 1) * G].double().T / math.sqrt(c["dim"])
                top = torch.logsumexp(x, 0)
                lse[b, i, h * G:(h + 1) * G] = top
                out[b, i, h * G:(h + 1) * G] = torch.exp(x - top).T @ v[at, h]
    return {"out": out, "lse": lse}


def _exact_append(s):
    c = s["case"]
    lens, new, table = _lens(c), _news(c), s["table"].tolist()
    for cache, fresh in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])):
        for b in range(c["B"]):
            t, i = lens[b] - new[b], 0
            while i < new[b]:                                  # run by run within a page
                m = min(new[b] - i, c["page"] - t % c["page"])
                cache[table[b][t // c["page"]], t % c["page"]:t % c["page"] + m] = fresh[b, i:i + m]
                i, t = i + m, t + m
    return {"k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}


def _exact_row(bits, tau, top_p, top_k):
    """One row's (probabilities, restricted logprobs, full logprobs) in 64 bits, by a sort of the whole row."""
    x = bits[:VREAL].double()
    if tau == 0.0:
        p = torch.zeros_like(x)
        p[int((x == x.max()).nonzero()[0])] = 1.0
        return p, torch.log(p), torch.log(p)
    full = torch.log_softmax(x / tau, 0)
    keep = torch.ones_like(x, dtype=torch.bool)
    if 1 <= top_k < VREAL:
        keep = x >= torch.sort(x, descending=True).values[top_k - 1]
    if top_p < 1.0:
        value, count = torch.unique(x[keep], return_counts=True)
        value, count = value.flip(0), count.flip(0)
        mass = count * torch.exp((value - value[0]) / tau)
        above = torch.cumsum(mass, 0) - mass
        keep &= x >= value[above < top_p * mass.sum()].min()
    restr = torch.where(keep, full - torch.logsumexp(full[keep], 0), -math.inf)
    return torch.exp(restr), restr, full


def _exact_verify(s):
    c = s["case"]
    B, n, num = c["B"], c["n"], _num_drafts(c)
    kinds = _settings(c) if c["mixed"] else [(c["tau"], c["top_p"], c["top_k"])] * B
    # the settings as the 32-bit numbers that a call takes
    kinds = [(float(torch.tensor(t)), float(torch.tensor(p)), k) for t, p, k in kinds]
    token = torch.full((B, n + 1), -1, dtype=torch.int32)
    restr, full = torch.zeros((B, n + 1), dtype=torch.float64), torch.zeros((B, n + 1), dtype=torch.float64)
    accepted = torch.zeros(B, dtype=torch.int32)
    drafted, word, last = s["token"].tolist(), s["accept"].tolist(), s["draw"].tolist()
    for b in range(B):
        for i in range(num[b] + 1):
            p, lr, lf = _exact_row(s["logits"][b * (n + 1) + i], *kinds[b])
            r = p
            if i < num[b]:
                d = drafted[b][i]
                if s["draft"] is None:
                    q = torch.zeros_like(p)
                    q[d] = 1.0
                else:
                    q = _exact_row(s["draft"][b * n + i], *kinds[b])[0]
                if ((word[b][i] & 0xFFFFFFFF) >> 8) / 2.0**24 * float(q[d]) < float(p[d]):
                    token[b, i], restr[b, i], full[b, i] = d, float(lr[d]), float(lf[d])
                    accepted[b] += 1
                    continue
                r = (p - q).clamp(min=0)
                r = r if float(r.sum()) > 0 else p
            cdf = torch.cumsum(r, 0)
            at = int(torch.searchsorted(cdf, (last[b] & 0xFFFFFFFF) / 2.0**32 * cdf[-1], right=True))
            token[b, i], restr[b, i], full[b, i] = at, float(lr[at]), float(lf[at])
            break
    return {"token": token, "accepted": accepted, "restr": restr, "full": full}
