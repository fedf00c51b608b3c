"""Rotary positions, the paged cache's append with the rotation applied on the way, and the
attention of samples that share a long prefix, as cases to be timed.

``run`` computes them in plain torch, or with ``own`` through the package's entry points.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------ the cases

def _rope(name, B, n, heads, dim, **kw):
    return {"name": name, "kind": "rope", "B": B, "n": n, "heads": heads, "dim": dim, "rot": dim, "axes": 1,
            "interleaved": False, "inverse": False, "dtype": "bf16", "theta": 1e6} | kw


def _append(name, B, n, heads, kv_heads, dim, page, max_len, **kw):
    return {"name": name, "kind": "append", "B": B, "n": n, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "max_len": max_len, "rot": dim, "axes": 1, "given": False, "interleaved": False,
            "dtype": "bf16", "order": "token", "theta": 1e6, "ragged": True} | kw


def _prefix(name, groups, members, n, heads, kv_heads, dim, page, shared, tail, **kw):
    return {"name": name, "kind": "prefix", "groups": groups, "members": members, "n": n, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "shared": shared, "tail": tail, "alone": 0,
            "dtype": "bf16", "order": "token", "uneven": False, "ragged": True} | kw


def listed():
    return [
        # queries of a decode step, half of each head rotated, pairs side by side
        _rope("rope_tokens", 64, 1, 32, 128, rot=64, interleaved=True, dtype="f16", theta=1e4),
        # queries of four packed prompts, as the training side recomputes them
        _rope("rope_prompts", 4, 4096, 32, 128),
        # the gradient of queries that turn with time, height and width, at an odd length
        _rope("rope_grad", 2, 4095, 28, 128, axes=3, inverse=True),
        # a decode step's new token: keys turned into the cache, queries turned
        _append("append_one", 64, 1, 32, 8, 128, 64, 512),
        # prompts written at once
        _append("append_prompts", 16, 2048, 32, 8, 128, 16, 2500),
        # prompts with images: positions given, of three axes; half precision, pages ordered by head
        _append("append_axes", 8, 1021, 28, 4, 128, 24, 1500, axes=3, given=True, dtype="f16", order="head"),
        # eight samples of one short prompt: latency is all that counts
        _prefix("prefix_small", 1, 8, 1, 32, 8, 128, 16, 1003, 60, ragged=False),
        # 64 samples of one prompt
        _prefix("prefix_group", 1, 64, 1, 32, 8, 128, 64, 8190, 2048),
        # a rollout batch: 16 prompts, 16 samples of each
        _prefix("prefix_batch", 16, 16, 1, 32, 8, 128, 64, 8192, 2048),
        # two very long contexts with 32 short answers each
        _prefix("prefix_long", 2, 32, 1, 32, 8, 128, 64, 131071, 512),
        # four drafted tokens and the last accepted one of each sample, pages ordered by head
        _prefix("prefix_drafts", 8, 16, 5, 32, 8, 128, 16, 4096, 1024, order="head"),
        # groups of all sizes and requests without one, half precision, 64-wide heads, pages of an odd size
        _prefix("prefix_uneven", 24, 16, 1, 64, 8, 64, 24, 4000, 3000, dtype="f16", uneven=True, alone=9),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "append", "append", "prefix", "prefix", "prefix"])
    dim = rng.choice([64, 128])
    rot = rng.choice([dim, dim, dim // 2, 48])
    axes, theta = rng.choice([1, 1, 2, 3]), rng.choice([1e4, 5e5, 1e6])
    if kind == "rope":
        B, heads = _log_int(rng, 1, 64), rng.choice([1, 8, 28, 32, 64])
        n = _log_int(rng, 1, max(1, 60_000_000 // (B * heads * dim)))
        c = _rope("", B, n, heads, dim, rot=rot, axes=axes, theta=theta, interleaved=rng.random() < 0.4,
                  inverse=rng.random() < 0.5, dtype=rng.choice(["bf16", "f16", "f32"]))
    elif kind == "append":
        heads, kv_heads = rng.choice([(32, 8), (64, 8), (16, 16), (28, 4), (8, 1)])
        B = _log_int(rng, 1, 128)
        n = min(_log_int(rng, 1, 2048), max(1, 180_000_000 // (B * (heads + 2 * kv_heads) * dim)))
        c = _append("", B, n, heads, kv_heads, dim, rng.choice([16, 24, 64, 100]), n + rng.randrange(1, 600), rot=rot,
                    axes=axes, given=axes > 1 or rng.random() < 0.3, interleaved=rng.random() < 0.4, theta=theta,
                    dtype=rng.choice(["bf16", "f16"]), order=rng.choice(["token", "head"]), ragged=rng.random() < 0.8)
    else:
        heads, kv_heads = rng.choice([(32, 8), (64, 8), (16, 16), (28, 4), (8, 1), (40, 8)])
        groups, members, n = _log_int(rng, 1, 32), _log_int(rng, 1, 64), rng.choice([1, 1, 1, 2, 5])
        members = max(1, min(members, 256 // groups, 40_000 // (groups * heads * n)))
        alone = rng.choice([0, 0, 0, 1, 5])
        B = groups * members + alone
        shared = _log_int(rng, 20, min(131072, 160_000_000 // (groups * kv_heads * dim), 220_000_000 // (groups * members * n * heads)))
        tail = _log_int(rng, n, max(n, min(4096, 80_000_000 // (B * kv_heads * dim))))
        c = _prefix("", groups, members, n, heads, kv_heads, dim, rng.choice([16, 24, 32, 64, 100, 128]), shared, tail,
                    alone=alone, dtype=rng.choice(["bf16", "bf16", "f16"]), order=rng.choice(["token", "head"]),
                    uneven=rng.random() < 0.5, ragged=rng.random() < 0.8)
    del c["name"]
    return c


def _sizes(case):
    """(members of each group, shared tokens of each group): the largest of both somewhere among them."""
    rng, G = random.Random(case["groups"] * 1_000_003 + case["shared"]), case["groups"]
    size, shared = [case["members"]] * G, [case["shared"]] * G
    if case["uneven"]:
        size = [rng.randint(1, case["members"]) for _ in range(G)]
        size[rng.randrange(G)] = case["members"]
    if case["ragged"]:
        shared = [_log_int(rng, max(1, case["shared"] // 8), case["shared"]) for _ in range(G)]
        shared[rng.randrange(G)] = case["shared"]
        if G >= 8:
            shared[G // 3] = 0
    return size, shared


def _sequences(case):
    """(start of each group and the end of the last, shared tokens of each sequence, lengths, new tokens)."""
    if case["kind"] == "append":
        B, n = case["B"], case["n"]
        rng = random.Random(B * 1_000_003 + case["max_len"])
        lens, new = [case["max_len"]] * B, [n] * B
        if case["ragged"]:
            lens = [_log_int(rng, max(n, case["max_len"] // 16), case["max_len"]) for _ in range(B)]
            if B >= 8:
                new[1], new[2], lens[2] = max(1, n - 1), 0, 0
        return None, None, lens, new
    n, alone = case["n"], case["alone"]
    size, shared = _sizes(case)
    start, of = [alone // 2], [0] * (alone // 2)
    for m, t in zip(size, shared):
        start.append(start[-1] + m)
        of += [t] * m
    of += [0] * (alone - alone // 2)
    rng, B = random.Random(len(of) * 1_000_033 + case["tail"]), len(of)
    tail, new = [case["tail"]] * B, [n] * B
    if case["ragged"]:
        tail = [_log_int(rng, max(n, case["tail"] // 32), case["tail"]) for _ in range(B)]
        tail[B // 2] = case["tail"]
        if B >= 8:
            new[1], new[2], tail[3] = max(1, n - 1), 0, n
    return start, of, [a + b for a, b in zip(of, tail)], new


# ------------------------------------------------------------ inputs

def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(case, pages, g, filled):
    """A paged cache [pages, page, kv_heads, dim] (as a view, whatever its order in memory)."""
    page, H, D, dt = case["page"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    shape = (pages, page, H, D) if case["order"] == "token" else (pages, H, page, D)
    out = []
    for _ in range(2):
        c = torch.zeros(shape, dtype=dt, device="cuda")
        if filled:
            for a in range(0, pages, 4096):
                part = c[a:a + 4096]
                part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
        out.append(c if case["order"] == "token" else c.transpose(1, 2))
    return out


def _positions(case, base, count, g):
    """Positions [axes, B, n] that begin at `base`: text along one axis; images of 32 patches a row along three."""
    i = torch.arange(count, device="cuda", dtype=torch.int32)
    along = [i] if case["axes"] == 1 else [i // 1024, i // 32 % 32, i % 32][3 - case["axes"]:]
    return torch.stack([base[:, None] + a for a in along]).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s, dt, D, n = {"case": case}, DTYPES[case["dtype"]], case["dim"], case["n"]
    if case["kind"] != "prefix":
        # what the model keeps: its frequencies, and which axis each pair turns with
        P = case["rot"] // 2
        s["inv_freq"] = case["theta"] ** (-torch.arange(P, dtype=torch.float64) / P)
        cut = [0] + [P * (a + 2) // (case["axes"] + 2) for a in range(case["axes"] - 1)]
        s["axis"] = sum((torch.arange(P) >= c).to(torch.uint8) for c in cut[1:]) if case["axes"] > 1 else None
        s["inv_freq_gpu"] = s["inv_freq"].cuda()
        s["axis_gpu"] = torch.zeros(P, dtype=torch.long, device="cuda") if s["axis"] is None else s["axis"].long().cuda()
    if case["kind"] == "rope":
        base = torch.randint(0, 131072, (case["B"],), generator=g, device="cuda", dtype=torch.int32)
        s["positions"] = _positions(case, base, n, g)
        s["x"] = randn(case["B"], n, case["heads"], D).to(dt)
        return s
    start, of, lens, new = _sequences(case)
    B, page, H = len(lens), case["page"], case["kv_heads"]
    s["lens"], s["new"] = _int32(lens), _int32(new)
    need = [-(-t // page) for t in lens]
    table = torch.zeros((B, max(1, max(need))), dtype=torch.int32)
    if case["kind"] == "append":
        pages = sum(need) + 3
        order, at = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu(), 0
        for b, m in enumerate(need):
            table[b, :m] = order[at:at + m]
            at += m
        s["k_cache"], s["v_cache"] = _cache(case, pages, g, False)
        # queries, keys and values as they come out of one projection: views of a wider row
        qkv = randn(B, n, case["heads"] + 2 * H, D).to(dt)
        s["q"], s["k"], s["v"] = qkv.split([case["heads"], H, H], dim=2)
        s["positions"] = _positions(case, s["lens"] - s["new"] + 7, n, g) if case["given"] else None
        s["table"] = table.cuda()
        return s
    # the shared tokens' full pages are held once; a page that they fill in part is each sample's own copy
    size, shared = _sizes(case)
    full = [t // page for t in shared]
    whole = {b: (full[i], start[i]) for i in range(case["groups"]) for b in range(start[i], start[i + 1])}
    pages = sum(m - (whole[b][0] if b in whole and b != whole[b][1] else 0) for b, m in enumerate(need)) + 3
    order, at = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu(), 0
    copies = []
    for b, m in enumerate(need):
        f, first = whole.get(b, (0, b))
        f = 0 if b == first else f
        table[b, :f] = table[first, :f]
        table[b, f:m] = order[at:at + m - f]
        at += m - f
        if b != first and of[b] % page:
            copies.append((int(table[first, f]), int(table[b, f])))
    s["k_cache"], s["v_cache"] = _cache(case, pages, g, True)
    if copies:
        src, dst = (torch.tensor(v, device="cuda") for v in zip(*copies))
        for c in (s["k_cache"], s["v_cache"]):
            c[dst] = c[src]
    s["table"], s["start"], s["shared"] = table.cuda(), _int32(start), _int32(shared)
    s["q"] = (2.0 * randn(B, n, case["heads"], D)).to(dt)
    return s


# ------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "prefix": _plain_prefix}[c["kind"]](s)
    import rollout_consistent_vocab_gb300 as rlk
    if c["kind"] == "rope":
        return rlk.rope(s["x"], s["inv_freq"], s["positions"], pair_axis=s["axis"], interleaved=c["interleaved"],
                        inverse=c["inverse"])
    if c["kind"] == "append":
        q = rlk.kv_append_rope(s["k_cache"], s["v_cache"], s["table"], s["lens"], s["k"], s["v"], s["inv_freq"], q=s["q"],
                               positions=s["positions"], pair_axis=s["axis"], interleaved=c["interleaved"],
                               new_lens=s["new"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    out, lse = rlk.prefix_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["start"], s["shared"],
                                    new_lens=s["new"], max_shared=c["shared"])
    return {"out": out, "lse": lse}


def _turn(s, x, positions):
    """Pair j of each head turned by positions[axis of j] * inv_freq[j] (back, for the gradient); angles in 64 bits."""
    c = s["case"]
    P = c["rot"] // 2
    angle = positions[s["axis_gpu"]].permute(1, 2, 0).double() * s["inv_freq_gpu"]           # [B, n, pairs]
    if c.get("inverse"):
        angle = -angle
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    y = x.float().clone()
    a, b = (y[..., 0:2 * P:2], y[..., 1:2 * P:2]) if c["interleaved"] else (y[..., :P], y[..., P:2 * P])
    u, w = a * cos - b * sin, b * cos + a * sin
    a.copy_(u)
    b.copy_(w)
    return y.to(x.dtype)


def _plain_rope(s):
    return _turn(s, s["x"], s["positions"])


def _new_places(s):
    """Position of each new token [B, n], and whether it is there."""
    i = torch.arange(s["case"]["n"], device="cuda")
    lens, new = s["lens"].long()[:, None], s["new"].long()[:, None]
    return lens - new + i, i < new


def _plain_append(s):
    page = s["case"]["page"]
    pos, there = _new_places(s)
    at = pos[None].to(torch.int32) if s["positions"] is None else s["positions"]
    k, q = _turn(s, s["k"], at), _turn(s, s["q"], at)
    q.masked_fill_(~there[..., None, None], 0.0)              # a place without a new token gets 0
    b, i = torch.nonzero(there, as_tuple=True)
    t = pos[b, i]
    p = s["table"][b, t // page].long()
    s["k_cache"][p, t % page] = k[b, i]
    s["v_cache"][p, t % page] = s["v"][b, i]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _part(q, k, v, seen, scale):
    """Attention of q [X, rows, H, G, D] over k, v [X, L, H, D] where `seen` [X, rows, L]: weighted sum, sum, maximum."""
    X, R, H, G, D = q.shape
    q = q.permute(0, 2, 1, 3, 4).reshape(X, H, R * G, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * scale
    x.masked_fill_(~seen[:, None, :, None, :].expand(X, 1, R, G, -1).reshape(X, 1, R * G, -1), -math.inf)
    m = x.max(-1, keepdim=True).values
    e = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z, o = e.sum(-1, keepdim=True), torch.matmul(e, v.permute(0, 2, 1, 3))
    return [t.reshape(X, H, R, G, -1).permute(0, 2, 1, 3, 4) for t in (o, z, m)]


def _plain_prefix(s):
    """Each group's samples over its shared tokens at once, each sample over the rest, and the two joined."""
    c = s["case"]
    n, Hq, H, D, page = c["n"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    G, M, B, scale = c["groups"], c["members"], s["lens"].shape[0], 1.0 / math.sqrt(D)
    q = s["q"].float().reshape(B, n, H, Hq // H, D)
    start, b = s["start"].long(), torch.arange(B, device="cuda")
    g = torch.searchsorted(start, b, right=True) - 1                                         # -1 or G: in no group
    inside = (g >= 0) & (g < G)
    g = g.clamp(0, G - 1)
    slot = torch.where(inside, b - start[g], torch.zeros_like(b))
    shared = torch.where(inside, s["shared"].long()[g], torch.zeros_like(b))
    # the shared tokens
    L = max(1, c["shared"])
    t = torch.arange(L, device="cuda")
    rows = s["table"][start[:-1]][:, (t // page).clamp(max=s["table"].shape[1] - 1)].long()
    k, v = s["k_cache"][rows, t % page].float(), s["v_cache"][rows, t % page].float()        # [G, L, H, D]
    qg = q.new_zeros((G, M) + q.shape[1:])
    at = torch.nonzero(inside)[:, 0]
    qg[g[at], slot[at]] = q[at]
    seen = (t < s["shared"].long()[:, None])[:, None].expand(G, M * n, L)
    o1, z1, m1 = (x.reshape((G, M, n) + x.shape[2:])[g, slot] for x in _part(qg.flatten(1, 2), k, v, seen, scale))
    m1 = torch.where(inside[:, None, None, None, None], m1, torch.full_like(m1, -math.inf))
    del k, v
    # the rest of each sequence
    t = shared[:, None] + torch.arange(c["tail"], device="cuda")
    rows = s["table"].long().gather(1, (t // page).clamp(max=s["table"].shape[1] - 1))
    k, v = s["k_cache"][rows, t % page].float(), s["v_cache"][rows, t % page].float()
    pos, there = _new_places(s)
    o2, z2, m2 = _part(q, k, v, (t[:, None] <= pos[..., None]) & there[..., None], scale)
    # (a place without a new token sees nothing)
    m1 = torch.where(there[:, :, None, None, None], m1, torch.full_like(m1, -math.inf))
    m = torch.maximum(m1, m2)
    top = torch.where(m == -math.inf, torch.zeros_like(m), m)
    f1, f2 = torch.exp(m1 - top), torch.exp(m2 - top)
    z = z1 * f1 + z2 * f2
    out = (o1 * f1 + o2 * f2) / torch.where(z == 0, torch.ones_like(z), z)
    return {"out": out.reshape(B, n, Hq, D).to(s["q"].dtype), "lse": (torch.log(z) + m).reshape(B, n, Hq)}


# ------------------------------------------------------------ what a pass has to read, write and compute

def work(case):
    D, n = case["dim"], case["n"]
    if case["kind"] == "rope":
        places = case["B"] * n
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": places * (case["heads"] * D * size * 2 + 4 * case["axes"]), "flops": places * case["heads"] * case["rot"] * 3}
    start, of, lens, new = _sequences(case)
    if case["kind"] == "append":
        heads = case["heads"] + 2 * case["kv_heads"]
        return {"bytes": sum(new) * (heads * D * 2 * 2 + (4 * case["axes"] if case["given"] else 0)) + len(lens) * 8,
                "flops": sum(new) * (case["heads"] + case["kv_heads"]) * case["rot"] * 3}
    size, shared = _sizes(case)
    tokens = sum(shared) + sum(t - p for t, p, m in zip(lens, of, new) if m)
    pairs = sum(m * t - m * (m - 1) // 2 for t, m in zip(lens, new))
    return {"bytes": tokens * case["kv_heads"] * D * 4 + sum(new) * case["heads"] * D * 2 + len(lens) * n * case["heads"] * (D * 2 + 4),
            "flops": 4 * D * case["heads"] * pairs}


# ------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "rope":
        return _exact_turned(s, s["x"], s["positions"], -1.0 if case["inverse"] else 1.0)
    return _exact_append(s) if case["kind"] == "append" else _exact_prefix(s)


def _exact_turned(s, x, positions, sign):
    """Pair by pair, as complex numbers times exp(i angle); [B, n] positions of each axis."""
    c, out = s["case"], x.double()
    P = c["rot"] // 2
    for j in range(P):
        first, second = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + P)
        axis = 0 if s["axis"] is None else int(s["axis"][j])
        angle = sign * float(s["inv_freq"][j]) * positions[axis].double()
        z = torch.complex(out[..., first], out[..., second]) * torch.polar(torch.ones_like(angle), angle)[..., None]
        out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_append(s):
    c = s["case"]
    _, _, lens, new = _sequences(c)
    table, page = s["table"].tolist(), c["page"]
    at = s["positions"]
    if at is None:
        at = torch.stack([torch.arange(c["n"], device="cuda") + (t - m) for t, m in zip(lens, new)])[None]
    q, k = _exact_turned(s, s["q"], at, 1.0), _exact_turned(s, s["k"], at, 1.0)
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    for b, m in enumerate(new):
        q[b, m:] = 0.0
        for cache, fresh in zip(caches, (k, s["v"].double())):
            i = 0
            while i < m:                                       # run by run within a page
                t = lens[b] - m + i
                step = min(m - i, page - t % page)
                cache[table[b][t // page], t % page:t % page + step] = fresh[b, i:i + step]
                i += step
    return {"q": q, "k_cache": caches[0], "v_cache": caches[1]}


def _exact_prefix(s):
    """Sequence by sequence through its own pages, over all the tokens that a query sees."""
    c = s["case"]
    _, _, lens, new = _sequences(c)
    page, G = c["page"], c["heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    for b, m in enumerate(new):
        if m == 0:
            continue
        pages = s["table"][b, :-(-lens[b] // page)].long()
        k = s["k_cache"][pages].flatten(0, 1)[:lens[b]].double()
        v = s["v_cache"][pages].flatten(0, 1)[:lens[b]].double()
        for i in range(m):
            end = lens[b] - m + i + 1
            x = torch.einsum("hgd,thd->hgt", s["q"][b, i].double().reshape(-1, G, c["dim"]), k[:end]) / math.sqrt(c["dim"])
            top = torch.logsumexp(x, -1)
            lse[b, i] = top.flatten()
            out[b, i] = torch.einsum("hgt,thd->hgd", torch.exp(x - top[..., None]), v[:end]).flatten(0, 1)
    return {"out": out, "lse": lse}
