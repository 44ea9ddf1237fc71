"""Cases, plain forms and calls of the 8-bit paged cache and of drafted trees over a paged cache.

    append8  PagedCache.append into 8-bit pages (new keys rotated, keys and values quantised as they are written, queries
             rotated), then PagedCache.read of the new tokens: the values that the pages now stand for
    attend8  PagedCache.attend over 8-bit pages: single tokens, drafted tokens, chunks of prompts
    tree     PagedCache.attend of each sequence's tree of drafted tokens, over 16-bit and 8-bit pages
    masks    PagedCache.tree_masks: from each drafted token's parent, which new tokens it sees and its position
    accept   PagedCache.accept: the accepted drafted tokens move up to follow the cached ones, in all layers

A sequence b has kv_len[b] tokens, the last n_b = cu_q[b + 1] - cu_q[b] of them new; new token i lies at
kv_len[b] - n_b + i. Page tables are random permutations of the pool, as after hours of serving; unused entries hold -1.

8-bit pages: a token's D values of a kv head are e4m3 numbers times 2^e, one e for keys and one for values, stored as
e + 127: the smallest e in [-100, 119] for which the largest magnitude is at most 448 * 2^e (119 if there is none); rounded to
the nearest, ties to even, and to at most 448.

Trees: new token i of a sequence sees the cached tokens from its key_lo on and the new tokens c whose bit is set, bit
c % 64 of word c // 64 of its row of masks.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def _case(name, op, **k):
    c = {"name": name, "op": op, "seqs": 1, "new": 1, "kv": 1024, "ragged": False, "idle": 0, "mix": 1, "page": 64,
         "q_heads": 32, "kv_heads": 8, "head_dim": 128}
    if op == "append8":
        c |= {"ragged": True, "sections": "16,24,24", "interleaved": False, "half": True, "base": 5e5}
    elif op in ("attend8", "tree"):
        c |= {"window": 0, "docs": 0, "anchor": False}
        if op == "tree":
            c |= {"bits": 16, "chain": False}
    elif op == "masks":
        c |= {"chain": False}
    elif op == "accept":
        c |= {"kept": 4, "layers": 32}
    c.update(k)
    return c


def listed():
    return [
        # one decoding step of 64 users: rotate q and k, write k and v; latency counts
        _case("append8_step_64", "append8", seqs=64, kv=8192),
        # four ragged prompt chunks of up to 4095 tokens
        _case("append8_chunk_4x4k", "append8", seqs=4, new=4095, kv=16384, page=16),
        # one user, a short context: the smallest call
        _case("attend8_one_1k", "attend8", kv=1000, page=16),
        # 64 users, ragged contexts to 32K, two of the slots idle: bound by reading the cache
        _case("attend8_step_64", "attend8", seqs=64, kv=32768, ragged=True, idle=2),
        # 16 users with 5 drafted tokens each in a row, multi-head layer of dimension 64
        _case("attend8_draft_16x5", "attend8", seqs=16, new=5, kv=8191, ragged=True, q_heads=16, kv_heads=16, head_dim=64,
              page=32),
        # a 2K prompt chunk behind 30K cached tokens: bound by the matrix products
        _case("attend8_chunk_2k_32k", "attend8", new=2048, kv=32768),
        # one user's tree of 7 drafted tokens over a long document, 8-bit pages
        _case("tree8_one_7_64k", "tree", new=7, kv=65536, bits=8, q_heads=28, kv_heads=4),
        # 16 users with trees of up to 64 drafted tokens over ragged contexts to 16K, 16-bit pages
        _case("tree_step_16x64", "tree", seqs=16, new=64, kv=16384, ragged=True, idle=1),
        # the masks and positions of one user's tree: the smallest call
        _case("masks_one_26", "masks", new=26, kv=5000),
        # the masks and positions of 64 users' trees of up to 250 drafted tokens
        _case("masks_step_64x250", "masks", seqs=64, new=250, kv=9000, ragged=True),
        # one user accepts 4 of 26 drafted tokens, all layers
        _case("accept_one", "accept", new=26, kv=400, layers=28),
        # 64 users accept up to 6 of 64 drafted tokens, all layers
        _case("accept_step_64", "accept", seqs=64, new=64, kept=6, kv=256, ragged=True, page=16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _sections(rng, pairs):
    n = rng.choice([1, 2, 3, 3, 4])
    cut = sorted(rng.sample(range(1, pairs), n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cut, cut + [pairs]))


def draw(rng):
    op = rng.choice(["append8", "attend8", "attend8", "attend8", "tree", "tree", "masks", "accept"])
    hq, hkv = rng.choice([(32, 8), (32, 32), (32, 4), (16, 16), (24, 8), (28, 4), (8, 1), (5, 5)])
    k = {"page": rng.choice([16, 32, 64, 128]), "q_heads": hq, "kv_heads": hkv, "head_dim": rng.choice([64, 128, 128]),
         "mix": rng.randrange(1 << 20), "ragged": rng.random() < 0.7}
    seqs = _log(rng, 1, 96)
    k |= {"seqs": seqs, "idle": rng.choice([0, 0, 1]) if seqs > 1 else 0}
    if op == "append8":
        new = min(_log(rng, 1, 3000), max(1, 12000 // seqs))
        k |= {"new": new, "kv": new + _log(rng, 1, max(1, 200000 // seqs)), "sections": _sections(rng, k["head_dim"] // 2),
              "interleaved": rng.random() < 0.5, "half": rng.random() < 0.5, "base": rng.choice([1e4, 5e5, 5e6])}
    elif op in ("attend8", "tree"):
        if op == "tree":
            new = _log(rng, 2, 300)
            k |= {"bits": rng.choice([8, 16]), "chain": rng.random() < 0.15}
        else:
            new = 1 if rng.random() < 0.45 else _log(rng, 2, 2000)
        hist = _log(rng, 1, 120000)
        while seqs > 1 and seqs * new > 8192:
            seqs -= 1
        kv = new + hist
        # scores of the plain form, keys held
        kv = min(kv, max(new + 1, 1_900_000_000 // (seqs * new * hq)), max(new + 1, 1_300_000_000 // (seqs * hkv * k["head_dim"])))
        kind = rng.choice(["all", "all", "window", "docs" if op == "attend8" else "window"])
        k |= {"seqs": seqs, "idle": min(k["idle"], seqs - 1), "new": new, "kv": kv,
              "window": _log(rng, 16, 4096) if kind == "window" else 0, "docs": _log(rng, 50, 4000) if kind == "docs" else 0,
              "anchor": kind == "docs" or rng.random() < 0.3}
    elif op == "masks":
        k |= {"new": _log(rng, 1, 250), "kv": _log(rng, 250, 100000), "chain": rng.random() < 0.2}
    else:
        new = _log(rng, 1, 100)
        k |= {"new": new, "kept": rng.randint(1, min(new, 12)), "kv": new + rng.randint(1, 200),
              "layers": rng.choice([1, 4, 28, 32]), "kv_heads": min(hkv, 8)}
    c = _case("", op, **k)
    del c["name"]
    return c


def _lens(c):
    """(new tokens, tokens held) of each sequence: fixed by the case."""
    rng = random.Random(c["mix"])
    n, kv = [], []
    for b in range(c["seqs"]):
        if b < c["idle"]:
            n.append(0)
            kv.append(0)
        elif c["ragged"]:
            n.append(rng.randint(max(1, c["new"] // 2), c["new"]))
            hist = c["kv"] - c["new"]
            kv.append(n[-1] + rng.randint(hist // 4, hist))
        else:
            n.append(c["new"])
            kv.append(c["kv"])
    return n, kv


def _kept(c):
    """How many of its new tokens each sequence keeps: fixed by the case."""
    rng = random.Random(c["mix"] + 1)
    return [min(x, rng.randint(1, c["kept"]) if c["ragged"] else c["kept"]) for x in _lens(c)[0]]


def _axis_of_pair(c):
    """Which position axis turns each pair: the sections one after the other, or dealt in turn until each is full."""
    left = [int(x) for x in c["sections"].split(",")]
    if not c["interleaved"]:
        return [a for a, x in enumerate(left) for _ in range(x)]
    out = []
    while sum(left):
        for a in range(len(left)):
            if left[a]:
                out.append(a)
                left[a] -= 1
    return out


def _theta(c):
    D = c["head_dim"]
    return [c["base"] ** (-2.0 * p / D) for p in range(D // 2)]


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _positions(c, tokens, seed):
    """[axes, tokens] int32: 512 tokens of text, then four frames of 16 x 16 patches, and so on, from a far start."""
    t = torch.arange(tokens, device=DEV)
    start = seed * 7919 % 100000 + t // 1536 * 528
    w = t % 1536
    text, v = w < 512, (w - 512).clamp(min=0)
    grid = [start + 512 + v // 256, start + 512 + v // 16 % 16, start + 512 + v % 16, start + 512 + v % 7]
    axes = len(c["sections"].split(","))
    return torch.stack([torch.where(text, start + w, x) for x in grid[:axes]]).to(torch.int32).contiguous()


def _codes(g, shape):
    """e4m3 pages of normal values at the spread that their scales give them, and the scales of magnitudes around 1."""
    pages = (_normal(g, *shape) * 120.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    scales = torch.randint(118, 122, shape[:-1], generator=g, device=DEV, dtype=torch.uint8)
    return pages, scales.view(torch.float8_e8m0fnu)


def _parents(c, g, T, i):
    """Each new token's parent among the new ones before it, -1: the last cached token. A tree of logarithmic depth, or a
    chain."""
    if c["chain"]:
        return (i - 1).to(torch.int32)
    r = 0.2 + 0.75 * torch.rand(T, generator=g, device=DEV)
    return torch.minimum((i * r).long() - 1 + (i > 1).long(), i - 1).to(torch.int32)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    n, kv = _lens(c)
    B, T, ps, D, hkv = c["seqs"], sum(n), c["page"], c["head_dim"], c["kv_heads"]
    s["T"], s["max_new"] = T, max(n)
    s["words"] = -(-max(n) // 64)
    s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(n)]), device=DEV, dtype=torch.int32)
    s["kv_len"] = torch.tensor(kv, device=DEV, dtype=torch.int32)
    if own:
        import packed_sequence_rope_gb300 as aa
    if c["op"] == "masks":
        s["parents"] = _parents(c, g, T, _token_rows(s)[1])
        if own:
            s["cache"] = aa.PagedCache(1, 16, 1, 64)
        return s
    need = [-(-x // ps) for x in kv]
    P, W = sum(need) + 3, max(max(need), 1)
    shape = (c.get("layers", 1), P, hkv, ps, D)
    if c["op"] in ("append8", "attend8") or c.get("bits") == 8:
        (s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"]) = _codes(g, shape), _codes(g, shape)
    else:
        s["k_pages"], s["v_pages"] = _normal(g, *shape), _normal(g, *shape)
    pages = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    first = np.concatenate([[0], np.cumsum(need)])[:-1]
    at = np.where(np.arange(W)[None] < np.asarray(need)[:, None], first[:, None] + np.arange(W)[None], -1)
    at = torch.from_numpy(at).to(DEV)
    s["table"] = torch.where(at >= 0, pages[at.clamp(min=0)], torch.full_like(pages[:1], -1)).contiguous()
    if own:
        s["cache"] = aa.PagedCache(P, ps, hkv, D, num_layers=shape[0], k_pages=s["k_pages"], v_pages=s["v_pages"],
                                   k_scales=s.get("k_scales"), v_scales=s.get("v_scales"))
    if c["op"] == "append8":
        qkv = _normal(g, T, c["q_heads"] + 2 * hkv, D)
        # heads differ in size, as a model's do
        qkv *= torch.exp2(torch.randint(-3, 3, (1, qkv.shape[1], 1), generator=g, device=DEV))
        s["q"], s["k"], s["v"] = qkv.split([c["q_heads"], hkv, hkv], dim=1)
        s["pos"] = _positions(c, T, seed)
        s["axis"] = torch.tensor(_axis_of_pair(c), device=DEV)
        s["theta"] = torch.tensor(_theta(c), device=DEV, dtype=torch.float64)
        if own:
            s["rope"] = aa.RopeAxes(D, axis_of_pair=_axis_of_pair(c), base=c["base"],
                                    layout=aa.ROPE_HALF if c["half"] else aa.ROPE_ADJACENT)
    elif c["op"] in ("attend8", "tree"):
        s["q"] = _normal(g, T, c["q_heads"], D)
        seq, i, p = _token_rows(s)
        s["tree"] = None
        if c["op"] == "tree":
            s["parents"] = _parents(c, g, T, i)
            s["tree"], p = _plain_masks(s).values()
        lo = None
        if c["window"]:
            lo = (p - c["window"] + 1).clamp(min=0)
        if c["docs"]:
            lo = torch.where(p > 0, 1 + (p - 1) // c["docs"] * c["docs"], 0)
        s["key_lo"] = None if lo is None else lo.to(torch.int32)
        if own:
            s["work"] = s["cache"].alloc_workspace(B, T, s["max_new"], W, c["q_heads"])
    else:
        kept, order = _kept(c), np.random.RandomState(seed % (1 << 31))
        path = np.full((B, c["kept"]), -1, dtype=np.int32)
        for b in range(B):
            path[b, :kept[b]] = np.sort(order.permutation(n[b])[:kept[b]])
        s["path"] = torch.from_numpy(path).to(DEV)
    return s


# ------------------------------------------------------------------ the operators, plain and the framework's
def _token_rows(s):
    """Each new token's sequence, its index among the new ones and the position that it lies at."""
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=DEV), n, output_size=s["T"])
    i = torch.arange(s["T"], device=DEV) - s["cu"].long()[seq]
    return seq, i, s["kv_len"].long()[seq] - n[seq] + i


def _turn(x, cos, sin, half):
    """Pairs of x [T, H, D] turned by [T, D/2] angles, in 32 bits."""
    x = x.float()
    cos, sin = cos[:, None], sin[:, None]
    if half:
        a, b = x.chunk(2, dim=-1)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)


def _quantise(x):
    """x fp32 [..., D] as e4m3 numbers and their scales' bytes."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = (e - 9 + (m > 0.875).int()).clamp(-100, 119)  # 448 = 0.875 * 2^9
    codes = torch.ldexp(x, -e[..., None].float()).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _values(codes, scales):
    """What 8-bit pages stand for, in 32 bits."""
    return torch.ldexp(codes.float(), scales.view(torch.uint8).float()[..., None] - 127.0)


def _plain_append(s):
    c = s["case"]
    angle = s["pos"].double()[s["axis"]].T * s["theta"]  # 64 bits: far positions
    cos, sin = angle.cos().float(), angle.sin().float()
    seq, _, p = _token_rows(s)
    page, slot = s["table"].long()[seq, p // c["page"]], p % c["page"]
    (k, ks), (v, vs) = _quantise(_turn(s["k"], cos, sin, c["half"])), _quantise(s["v"].float())
    # the pages as bytes: indexing knows no 8-bit floats
    for name, x in (("k_pages", k), ("v_pages", v), ("k_scales", ks), ("v_scales", vs)):
        s[name].view(torch.uint8)[0, page, :, slot] = x.view(torch.uint8)
    read = [_values(s[x + "_pages"].view(torch.uint8)[0, page, :, slot].view(torch.float8_e4m3fn),
                    s[x + "_scales"].view(torch.uint8)[0, page, :, slot]).to(torch.bfloat16) for x in "kv"]
    return {"q": _turn(s["q"], cos, sin, c["half"]).to(torch.bfloat16), "k": read[0], "v": read[1]}


def _own_append(s):
    q = s["cache"].append(s["k"], s["v"], s["table"], s["cu"], s["kv_len"], rope=s["rope"], pos=s["pos"], q=s["q"])
    k, v = s["cache"].read(s["table"], s["cu"], s["kv_len"], s["T"])
    return {"q": q, "k": k, "v": v}


def _plain_attend(s):
    c = s["case"]
    B, D, hq, hkv, Q = c["seqs"], c["head_dim"], c["q_heads"], c["kv_heads"], s["max_new"]
    G = hq // hkv
    at = s["table"].clamp(min=0).long()
    if "k_scales" in s:
        k, v = (_values(s[x + "_pages"].view(torch.uint8)[0][at].view(torch.float8_e4m3fn),
                        s[x + "_scales"].view(torch.uint8)[0][at]) for x in "kv")
    else:
        k, v = (s[x + "_pages"][0][at].float() for x in "kv")
    k, v = (x.permute(0, 2, 1, 3, 4).reshape(B, hkv, -1, D) for x in (k, v))
    seq, i, p = _token_rows(s)
    q = torch.zeros(B, Q, hq, D, device=DEV)
    q[seq, i] = s["q"].float()
    last, lo = torch.full((B, Q), -1, device=DEV), torch.zeros(B, Q, device=DEV, dtype=torch.long)
    last[seq, i] = p if s["tree"] is None else p - i - 1
    if s["key_lo"] is not None:
        lo[seq, i] = s["key_lo"].long()
    j = torch.arange(k.shape[2], device=DEV)
    seen = (j >= lo[..., None]) & (j <= last[..., None])
    if c["anchor"]:
        seen |= (j == 0) & (last[..., None] >= 0)
    if s["tree"] is not None:
        bits = (s["tree"][:, :, None] >> torch.arange(64, device=DEV) & 1).bool().flatten(1)  # [T, 64 words]
        t, bit = bits.nonzero(as_tuple=True)
        seen[seq[t], i[t], (p - i)[t] + bit] = True
    q = q.view(B, Q, hkv, G, D).permute(0, 2, 3, 1, 4)  # [B, hkv, G, Q, D]
    a = (q.reshape(B, hkv, G * Q, D) @ k.transpose(2, 3)).view(B, hkv, G, Q, -1) * (1.0 / math.sqrt(D))
    a.masked_fill_(~seen[:, None, None], -math.inf)
    m = a.amax(-1, keepdim=True).clamp(min=-1e30)
    a = (a - m).exp_()
    total = a.sum(-1, keepdim=True)
    o = (a.view(B, hkv, G * Q, -1) @ v).view(B, hkv, G, Q, D) / total.clamp(min=1e-38)
    lse = (m + total.log()).squeeze(-1)  # [B, hkv, G, Q]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, Q, hq, D)[seq, i]
    lse = lse.permute(1, 2, 0, 3).reshape(hq, B, Q)[:, seq, i]
    return {"o": o.to(torch.bfloat16), "lse": lse}


def _own_attend(s):
    o, lse = s["cache"].attend(s["q"], s["table"], s["cu"], s["kv_len"], s["max_new"], key_lo=s["key_lo"],
                               anchor=s["case"]["anchor"], tree=s["tree"], workspace=s["work"], return_lse=True)
    return {"o": o, "lse": lse}


def _plain_masks(s):
    B, Q = s["kv_len"].numel(), 64 * s["words"]
    seq, i, p = _token_rows(s)
    up = torch.zeros(B, Q, Q, device=DEV)
    up[seq, i, i] = 1.0
    up[seq, i, s["parents"].long().clamp(min=0)] = 1.0 * (s["parents"] >= 0) + 1.0 * (s["parents"] < 0) * (i == 0)
    up[seq, i, i] = 1.0
    for _ in range((Q - 1).bit_length()):  # ancestors twice as far each time
        up = (up @ up).clamp(max=1.0)
    seen = up[seq, i]
    bits = seen.long().view(-1, s["words"], 64) << torch.arange(64, device=DEV)
    depth = seen.sum(-1).long() - 1
    return {"mask": bits.sum(-1), "pos": (p - i + depth).to(torch.int32)}


def _own_masks(s):
    mask, pos = s["cache"].tree_masks(s["parents"], s["cu"], s["kv_len"], s["max_new"])
    return {"mask": mask, "pos": pos}


def _plain_accept(s):
    c = s["case"]
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    b, i = (s["path"] >= 0).nonzero(as_tuple=True)
    base = (s["kv_len"].long() - n)[b]
    source, target = base + s["path"].long()[b, i], base + i
    rows = [(s["table"].long()[b, x // c["page"]], x % c["page"]) for x in (source, target)]
    (sp, ss), (tp, ts) = rows
    s["k_pages"][:, tp, :, ts] = s["k_pages"][:, sp, :, ss]
    s["v_pages"][:, tp, :, ts] = s["v_pages"][:, sp, :, ss]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_accept(s):
    s["cache"].accept(s["table"], s["cu"], s["kv_len"], s["path"])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append8": _own_append, "attend8": _own_attend, "tree": _own_attend, "masks": _own_masks,
                "accept": _own_accept}[op](state)
    return {"append8": _plain_append, "attend8": _plain_attend, "tree": _plain_attend, "masks": _plain_masks,
            "accept": _plain_accept}[op](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, D = case, case["head_dim"]
    n, kv = _lens(c)
    T, hq, hkv = sum(n), c["q_heads"], c["kv_heads"]
    if c["op"] == "masks":
        return {"bytes": T * (4 + 4 + 8 * -(-max(n) // 64)) + 8 * len(n), "flops": 0}
    if c["op"] == "accept":
        return {"bytes": sum(_kept(c)) * c["layers"] * hkv * D * 2 * 2 * 2, "flops": 0}
    if c["op"] == "append8":
        held = T * 2 * hkv * (D + 1)  # written, then read
        return {"bytes": T * (hq + 2 * hkv) * D * 2 + T * hq * D * 2 + 2 * held + T * 2 * hkv * D * 2,
                "flops": 3 * T * (hq + hkv) * D}
    seq = np.repeat(np.arange(len(n)), n)
    i = np.arange(T) - np.concatenate([[0], np.cumsum(n)])[seq]
    base = (np.asarray(kv) - np.asarray(n))[seq]
    p = base + i
    if c["op"] == "tree":
        deep = i if c["chain"] else np.log2(i + 1.0).astype(np.int64)  # about how deep a token lies in its tree
        lo = np.maximum(base + deep - c["window"] + 1, 0) if c["window"] else np.zeros_like(p)
        pairs = int((np.maximum(base - lo, 0) + deep + 1).sum())
        lo = np.minimum(lo, base)
    else:
        lo = np.maximum(p - c["window"] + 1, 0) if c["window"] else np.zeros_like(p)
        if c["docs"]:
            lo = np.where(p > 0, 1 + (p - 1) // c["docs"] * c["docs"], 0)
        pairs = int((p - lo + 1).sum())
    pairs += int(np.sum(lo > 0)) if c["anchor"] else 0
    first = np.full(len(n), 1 << 40)
    np.minimum.at(first, seq, lo)
    keys = sum(int(k - f) + (1 if c["anchor"] and f > 0 else 0) for k, f, x in zip(kv, first, n) if x)
    row = 2 * (D + 1) if c["op"] == "attend8" or c["bits"] == 8 else 4 * D
    more = 8 * -(-max(n) // 64) if c["op"] == "tree" else 0
    return {"bytes": keys * hkv * row + T * hq * (D * 4 + 4) + T * more, "flops": 4 * pairs * D * hq}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_turn(x, s):
    c, D = s["case"], s["case"]["head_dim"]
    x = x.double()
    one, two = (x[..., :D // 2], x[..., D // 2:]) if c["half"] else (x[..., ::2], x[..., 1::2])
    axis = _axis_of_pair(c)
    angle = torch.empty(x.shape[0], D // 2, device=DEV, dtype=torch.float64)
    for p in range(D // 2):
        angle[:, p] = s["pos"][axis[p]].double() * (c["base"] ** (-2.0 * p / D))
    z = torch.complex(one, two) * torch.polar(torch.ones_like(angle), angle)[:, None]
    y = torch.empty_like(x)
    if c["half"]:
        y[..., :D // 2], y[..., D // 2:] = z.real, z.imag
    else:
        y[..., ::2], y[..., 1::2] = z.real, z.imag
    return y


def _exact_held(x):
    """The values that 8-bit pages hold of x [..., D] in 64 bits: multiples of 2^-9 up to 2^-6, then of 1/8 of the power of two
    below, times the row's scale."""
    top = x.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.clamp(torch.ceil(torch.log2(top / 448.0)), -100, 119))
    scale = torch.where((top > 448.0 * scale) & (scale < 2.0 ** 119), 2 * scale, scale)  # should the logarithm have rounded across a border
    scale = torch.where((top <= 224.0 * scale) & (scale > 2.0 ** -100), scale / 2, scale)
    y = (x / scale).clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))) / 8
    return torch.round(y / step) * step * scale  # ties to even


def _exact_seen(s, b, c, n, kv, key_lo, tree):
    """[n, kv] of one sequence, on the host: which keys its new tokens see, token by token."""
    seen = np.zeros((n, kv), dtype=bool)
    base = kv - n
    for i in range(n):
        lo = max(int(key_lo[i]), 0) if key_lo is not None else 0
        if tree is None:
            seen[i, lo:base + i + 1] = True
        else:
            seen[i, lo:base] = True
            for word, bits in enumerate(tree[i]):
                bits = int(bits) & (1 << 64) - 1
                while bits:
                    bit = (bits & -bits).bit_length() - 1
                    seen[i, base + 64 * word + bit] = True
                    bits &= bits - 1
        if c["anchor"]:
            seen[i, 0] |= tree is None or base > 0
    return torch.from_numpy(seen).to(DEV)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    n, kv = _lens(c)
    start = np.concatenate([[0], np.cumsum(n)])
    if c["op"] == "append8":
        return {"q": _exact_turn(s["q"], s), "k": _exact_held(_exact_turn(s["k"], s)), "v": _exact_held(s["v"].double())}
    if c["op"] == "masks":
        parents = s["parents"].tolist()
        masks, pos = np.zeros((s["T"], s["words"]), dtype=np.uint64), np.zeros(s["T"], dtype=np.int32)
        for b in range(c["seqs"]):
            for i in range(n[b]):
                at, depth = i, -1
                while at >= 0:
                    masks[start[b] + i, at // 64] |= np.uint64(1 << at % 64)
                    at, depth = parents[start[b] + at], depth + 1
                pos[start[b] + i] = kv[b] - n[b] + depth
        return {"mask": torch.from_numpy(masks.view(np.int64)), "pos": torch.from_numpy(pos)}
    if c["op"] == "accept":
        out = {x: s[x].clone() for x in ("k_pages", "v_pages")}
        at = lambda b, p: (int(table[b][p // c["page"]]), p % c["page"])  # noqa: E731
        table, path = s["table"].cpu().numpy(), s["path"].cpu().numpy()
        for b in range(c["seqs"]):
            for i, x in enumerate(path[b][path[b] >= 0]):
                (sp, ss), (tp, ts) = at(b, kv[b] - n[b] + int(x)), at(b, kv[b] - n[b] + i)
                for name in out:
                    out[name][:, tp, :, ts] = s[name][:, sp, :, ss]
        return out
    hq, hkv, D = c["q_heads"], c["kv_heads"], c["head_dim"]
    if 4.0 * s["T"] * max(kv) * hq * D > 4e12:
        return None
    o = torch.zeros(s["T"], hq, D, device=DEV, dtype=torch.float64)
    lse = torch.full((hq, s["T"]), -math.inf, device=DEV, dtype=torch.float64)
    key_lo = None if s["key_lo"] is None else s["key_lo"].cpu().numpy()
    tree = None if s["tree"] is None else s["tree"].cpu().numpy()
    for b in range(c["seqs"]):
        if n[b] == 0:
            continue
        rows = slice(int(start[b]), int(start[b + 1]))
        pages = s["table"][b, :-(-kv[b] // c["page"])].long()
        seen = _exact_seen(s, b, c, n[b], kv[b], None if key_lo is None else key_lo[rows], None if tree is None else tree[rows])
        for h in range(hkv):
            held = []
            for x in "kv":
                y = s[x + "_pages"][0].view(torch.uint8 if "k_scales" in s else torch.bfloat16)[pages, h]
                if "k_scales" in s:
                    e = s[x + "_scales"].view(torch.uint8)[0][pages, h].double() - 127
                    y = y.view(torch.float8_e4m3fn).double() * torch.exp2(e)[..., None]
                held.append(y.double().reshape(-1, D)[:kv[b]])
            for e in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                a = s["q"][rows, e].double() @ held[0].T / math.sqrt(D)
                a = a.masked_fill(~seen, -math.inf)
                lse[e, rows] = torch.logsumexp(a, dim=1)
                o[rows, e] = torch.softmax(a, dim=1) @ held[1]
    return {"o": o, "lse": lse}
