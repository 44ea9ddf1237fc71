"""Cases, plain forms and calls of the serving operators and the multi-axis rotation.

    rope    RopeAxes: rotary positions with several axes (time, height, width), forward and with its gradient
    append  PagedCache.append: new keys rotated and written into their pages with the values, queries rotated
    attend  PagedCache.attend: attention of each sequence's new tokens over its paged keys and values
    pages   PagedCache.copy_pages: the page copies of a fork or a compaction, all layers at once

A sequence b has kv_len[b] tokens, the last cu_q[b + 1] - cu_q[b] of them new. New token i of sequence b sits at
p = kv_len[b] - n_b + i and sees keys [key_lo, p], and key 0 (the anchor) where the case has one. Page tables are random
permutations of the pool, as after hours of serving; unused entries hold -1.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def _rope(name, **k):
    c = {"name": name, "op": "rope", "tokens": 1, "q_heads": 32, "kv_heads": 8, "head_dim": 128, "sections": "16,24,24",
         "interleaved": False, "half": True, "train": False, "base": 5e5}
    c.update(k)
    return c


def _append(name, **k):
    c = {"name": name, "op": "append", "seqs": 1, "new": 1, "kv": 1024, "ragged": True, "idle": 0, "mix": 1, "page": 64,
         "q_heads": 32, "kv_heads": 8, "head_dim": 128, "sections": "16,24,24", "interleaved": False, "half": True,
         "base": 5e5}
    c.update(k)
    return c


def _attend(name, **k):
    c = {"name": name, "op": "attend", "seqs": 1, "new": 1, "kv": 1024, "ragged": False, "idle": 0, "mix": 1, "page": 64,
         "q_heads": 32, "kv_heads": 8, "head_dim": 128, "window": 0, "docs": 0, "anchor": False}
    c.update(k)
    return c


def _pages(name, **k):
    c = {"name": name, "op": "pages", "kind": "fork", "pairs": 8, "layers": 32, "page": 64, "kv_heads": 8, "head_dim": 128}
    c.update(k)
    return c


def listed():
    return [
        # one decoding step of 64 users: the rotation alone, latency counts
        _rope("rope_step_64", tokens=64),
        # a 64K training packing of text and video, LLaMA-7B-shaped layer, forward and gradient
        _rope("rope_train_64k", tokens=65536, kv_heads=32, half=False, train=True, base=5e6),
        # one decoding step of 64 users: rotate q and k, write k and v
        _append("append_step_64", seqs=64, kv=8192),
        # four ragged prompt chunks of up to 4095 tokens
        _append("append_chunk_4x4k", seqs=4, new=4095, kv=16384, page=16),
        # one user, a short context: the smallest call
        _attend("attend_one_1k", kv=1000, page=16),
        # one user, a 128K context: the work is split over the keys
        _attend("attend_one_128k", kv=131071, page=64),
        # 64 users, ragged contexts to 32K, two of the slots idle
        _attend("attend_step_64", seqs=64, kv=32768, ragged=True, idle=2),
        # 16 users with 5 drafted tokens each, multi-head layer of dimension 64
        _attend("attend_draft_16x5", seqs=16, new=5, kv=8191, ragged=True, q_heads=16, kv_heads=16, head_dim=64, page=32),
        # ragged prompt chunks of packed documents that see the anchor and their own document
        _attend("attend_docs_8x512", seqs=8, new=512, kv=16384, ragged=True, docs=1500, anchor=True, page=128),
        # a 2K prompt chunk behind 30K cached tokens: bound by the matrix products
        _attend("attend_chunk_2k_32k", new=2048, kv=32768, page=64),
        # a fork of eight sequences: their last pages, all layers
        _pages("pages_fork_8"),
        # a compaction that moves 256 pages, all layers
        _pages("pages_compact_256", kind="compact", pairs=256),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _sections(rng, pairs):
    n = rng.choice([1, 2, 3, 3, 4])
    cut = sorted(rng.sample(range(1, pairs), n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cut, cut + [pairs]))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend", "pages"])
    D = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    hq, hkv = rng.choice([(32, 8), (32, 32), (32, 4), (16, 16), (24, 8), (28, 4), (8, 1), (5, 5)])
    if op == "rope":
        c = _rope("", tokens=_log(rng, 1, 60000), q_heads=hq, kv_heads=hkv, head_dim=D, sections=_sections(rng, D // 2),
                  interleaved=rng.random() < 0.5, half=rng.random() < 0.5, train=rng.random() < 0.5,
                  base=rng.choice([1e4, 5e5, 5e6]))
    elif op == "append":
        seqs, new = _log(rng, 1, 96), _log(rng, 1, 3000)
        new = min(new, max(1, 12000 // seqs))
        c = _append("", seqs=seqs, new=new, kv=new + _log(rng, 1, max(1, 200000 // seqs)), ragged=rng.random() < 0.7,
                    idle=rng.choice([0, 0, 1]) if seqs > 1 else 0, mix=rng.randrange(1 << 20), page=page, q_heads=hq,
                    kv_heads=hkv, head_dim=D, sections=_sections(rng, D // 2), interleaved=rng.random() < 0.5,
                    half=rng.random() < 0.5, base=rng.choice([1e4, 5e5, 5e6]))
    elif op == "attend":
        seqs = _log(rng, 1, 96)
        new = 1 if rng.random() < 0.45 else _log(rng, 2, 2000)
        hist = _log(rng, 1, 120000)
        while seqs > 1 and seqs * new > 8192:
            seqs -= 1
        most = 1_900_000_000  # scores of the plain form
        kv = new + hist
        kv = min(kv, max(new + 1, most // (seqs * new * hq)), max(new + 1, 1_300_000_000 // (seqs * hkv * D)))
        kind = rng.choice(["all", "all", "window", "docs"])
        c = _attend("", seqs=seqs, new=new, kv=kv, ragged=rng.random() < 0.7,
                    idle=rng.choice([0, 0, 1]) if seqs > 1 else 0, mix=rng.randrange(1 << 20), page=page, q_heads=hq,
                    kv_heads=hkv, head_dim=D, window=_log(rng, 16, 4096) if kind == "window" else 0,
                    docs=_log(rng, 50, 4000) if kind == "docs" else 0, anchor=kind == "docs" or rng.random() < 0.3)
    else:
        c = _pages("", kind=rng.choice(["fork", "compact"]), pairs=_log(rng, 1, 250), layers=rng.choice([1, 4, 28, 32]),
                   page=page, kv_heads=min(hkv, 8), head_dim=D)
        if c["page"] > 64:
            c["pairs"] = min(c["pairs"], 120)
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


def _spans(c):
    """(position, first visible key) of every new token in order, as numpy arrays, and each token's sequence."""
    n, kv = _lens(c)
    seq = np.repeat(np.arange(len(n)), n)
    start = np.concatenate([[0], np.cumsum(n)])
    p = np.arange(start[-1]) - start[seq] + np.asarray(kv)[seq] - np.asarray(n)[seq]
    lo = np.zeros_like(p)
    if c["window"]:
        lo = np.maximum(p - c["window"] + 1, 0)
    if c["docs"]:
        lo = np.where(p > 0, 1 + (p - 1) // c["docs"] * c["docs"], 0)
    return p, lo, seq


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


def _theta(c):
    D = c["head_dim"]
    return [c["base"] ** (-2.0 * p / D) for p in range(D // 2)]


def _rope_handle(aa, c):
    return aa.RopeAxes(c["head_dim"], axis_of_pair=_axis_of_pair(c), base=c["base"],
                       layout=aa.ROPE_HALF if c["half"] else aa.ROPE_ADJACENT)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if own:
        import packed_sequence_rope_gb300 as aa
        s["aa"] = aa
    if c["op"] in ("rope", "append"):
        s["axis"] = torch.tensor(_axis_of_pair(c), device=DEV)
        s["theta"] = torch.tensor(_theta(c), device=DEV, dtype=torch.float64)
        if own:
            s["rope"] = _rope_handle(aa, c)
    if c["op"] == "rope":
        # q and k are slices of the layer's joint projection
        T, hq, hk, D = c["tokens"], c["q_heads"], c["kv_heads"], c["head_dim"]
        qkv = _normal(g, T, hq + 2 * hk, D)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["pos"] = _positions(c, T, seed)
        if c["train"]:
            s["gq"], s["gk"] = _normal(g, T, hq, D), _normal(g, T, hk, D)
            s["q"].requires_grad_(True)
            s["k"].requires_grad_(True)
        return s
    if c["op"] == "pages":
        L, n = c["layers"], c["pairs"]
        P = 5 * n // 2 + 2
        s["k_pages"] = _normal(g, L, P, c["kv_heads"], c["page"], c["head_dim"])
        s["v_pages"] = _normal(g, L, P, c["kv_heads"], c["page"], c["head_dim"])
        order = np.random.RandomState(seed % (1 << 31))
        if c["kind"] == "fork":
            both = order.permutation(P)[:2 * n]
            src, dst = both[:n], both[n:]
        else:  # live pages of the upper part move into free ones of the lower part
            src, dst = P // 2 + order.permutation(P - P // 2)[:n], order.permutation(P // 2)[:n]
        s["src"], s["dst"] = src.astype(np.int32), dst.astype(np.int32)
        s["src_t"], s["dst_t"] = (torch.from_numpy(x.astype(np.int64)).to(DEV) for x in (src, dst))
        if own:
            s["cache"] = aa.PagedCache(P, c["page"], c["kv_heads"], c["head_dim"], num_layers=L, k_pages=s["k_pages"],
                                       v_pages=s["v_pages"])
        return s
    n, kv = _lens(c)
    B, T, ps, D = c["seqs"], sum(n), c["page"], c["head_dim"]
    need = [-(-x // ps) for x in kv]
    P, W = sum(need) + 3, max(max(need), 1)
    s["k_pages"] = _normal(g, 1, P, c["kv_heads"], ps, D)
    s["v_pages"] = _normal(g, 1, P, c["kv_heads"], ps, D)
    pages = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    first = np.concatenate([[0], np.cumsum(need)])[:-1]
    at = np.where(np.arange(W)[None] < np.asarray(need)[:, None], first[:, None] + np.arange(W)[None], -1)
    at = torch.from_numpy(at).to(DEV)
    s["table"] = torch.where(at >= 0, pages[at.clamp(min=0)], torch.full_like(pages[:1], -1)).contiguous()
    s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(n)]), device=DEV, dtype=torch.int32)
    s["kv_len"] = torch.tensor(kv, device=DEV, dtype=torch.int32)
    s["max_new"] = max(n)
    s["T"] = T
    if own:
        s["cache"] = aa.PagedCache(P, ps, c["kv_heads"], D, k_pages=s["k_pages"], v_pages=s["v_pages"])
    if c["op"] == "append":
        qkv = _normal(g, T, c["q_heads"] + 2 * c["kv_heads"], D)
        s["q"], s["k"], s["v"] = qkv.split([c["q_heads"], c["kv_heads"], c["kv_heads"]], dim=1)
        s["pos"] = _positions(c, T, seed)
    else:
        s["q"] = _normal(g, T, c["q_heads"], D)
        _, lo, _ = _spans(c)
        s["key_lo"] = torch.from_numpy(lo).to(DEV, torch.int32) if c["window"] or c["docs"] else None
        if own:
            s["work"] = s["cache"].alloc_workspace(B, T, s["max_new"], W, c["q_heads"])
    return s


# ------------------------------------------------------------------ the operators, plain and the framework's
def _turn(x, cos, sin, half):
    """Pairs of x [T, H, D] turned by [T, D/2] angles, in 32 bits, rounded once."""
    x = x.float()
    cos, sin = cos[:, None], sin[:, None]
    if half:
        a, b = x.chunk(2, dim=-1)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1).to(torch.bfloat16)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2).to(torch.bfloat16)


def _cos_sin(s):
    angle = s["pos"].double()[s["axis"]].T * s["theta"]  # 64 bits: far positions
    return angle.cos().float(), angle.sin().float()


def _plain_rope(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    out = {"q": _turn(s["q"].detach(), cos, sin, c["half"]), "k": _turn(s["k"].detach(), cos, sin, c["half"])}
    if c["train"]:
        out["dq"], out["dk"] = _turn(s["gq"], cos, -sin, c["half"]), _turn(s["gk"], cos, -sin, c["half"])
    return out


def _own_rope(s):
    aa, c = s["aa"], s["case"]
    if not c["train"]:
        q, k = s["rope"].apply(s["pos"], s["q"], s["k"])
        return {"q": q, "k": k}
    q, k = aa.rope_axes(s["rope"], s["pos"], s["q"], s["k"])
    dq, dk = torch.autograd.grad((q, k), (s["q"], s["k"]), (s["gq"], s["gk"]))
    return {"q": q.detach(), "k": k.detach(), "dq": dq, "dk": dk}


def _token_rows(s):
    """Each new token's sequence, its index among the new ones and its position."""
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=DEV), n, output_size=s["T"])
    i = torch.arange(s["T"], device=DEV) - s["cu"].long()[seq]
    return seq, i, s["kv_len"].long()[seq] - n[seq] + i


def _plain_append(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    seq, _, p = _token_rows(s)
    page, slot = s["table"].long()[seq, p // c["page"]], p % c["page"]
    s["k_pages"][0, page, :, slot] = _turn(s["k"], cos, sin, c["half"])
    s["v_pages"][0, page, :, slot] = s["v"]
    return {"q": _turn(s["q"], cos, sin, c["half"]), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_append(s):
    q = s["cache"].append(s["k"], s["v"], s["table"], s["cu"], s["kv_len"], rope=s["rope"], pos=s["pos"], q=s["q"])
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attend(s):
    c = s["case"]
    B, D, hq, hkv, Q = c["seqs"], c["head_dim"], c["q_heads"], c["kv_heads"], s["max_new"]
    G = hq // hkv
    at = s["table"].clamp(min=0).long()
    k, v = (x[0][at].float().permute(0, 2, 1, 3, 4).reshape(B, hkv, -1, D) for x in (s["k_pages"], s["v_pages"]))
    seq, i, p = _token_rows(s)
    q = torch.zeros(B, Q, hq, D, device=DEV)
    q[seq, i] = s["q"].float()
    last, lo = torch.full((B, Q), -1, device=DEV), torch.zeros(B, Q, device=DEV, dtype=torch.long)
    last[seq, i] = p
    if s["key_lo"] is not None:
        lo[seq, i] = s["key_lo"].long()
    j = torch.arange(k.shape[2], device=DEV)
    seen = (j >= lo[..., None]) & (j <= last[..., None])
    if c["anchor"]:
        seen |= (j == 0) & (last[..., None] >= 0)
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
                               anchor=s["case"]["anchor"], workspace=s["work"], return_lse=True)
    return {"o": o, "lse": lse}


def _plain_pages(s):
    s["k_pages"][:, s["dst_t"]] = s["k_pages"][:, s["src_t"]]
    s["v_pages"][:, s["dst_t"]] = s["v_pages"][:, s["src_t"]]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_pages(s):
    s["cache"].copy_pages(s["src"], s["dst"])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "attend": _own_attend, "pages": _own_pages}[op](state)
    return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend, "pages": _plain_pages}[op](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, D = case, case["head_dim"]
    if c["op"] == "rope":
        heads = c["q_heads"] + c["kv_heads"]
        axes = len(c["sections"].split(","))
        passes = 2 if c["train"] else 1
        return {"bytes": passes * c["tokens"] * heads * D * 4 + 4 * axes * c["tokens"],
                "flops": passes * 3 * c["tokens"] * heads * D}
    if c["op"] == "pages":
        return {"bytes": 2 * 2 * 2 * c["pairs"] * c["layers"] * c["kv_heads"] * c["page"] * D, "flops": 0}
    n, kv = _lens(c)
    T = sum(n)
    if c["op"] == "append":
        return {"bytes": T * (c["q_heads"] + 2 * c["kv_heads"]) * D * 4, "flops": 3 * T * (c["q_heads"] + c["kv_heads"]) * D}
    p, lo, seq = _spans(c)
    pairs = int((p - lo + 1).sum() + (np.sum(lo > 0) if c["anchor"] else 0))
    first = np.full(len(n), 1 << 40)
    np.minimum.at(first, seq, lo)
    keys = sum(int(k - f) + (1 if c["anchor"] and f > 0 else 0) for k, f, x in zip(kv, first, n) if x)
    return {"bytes": keys * c["kv_heads"] * D * 4 + T * c["q_heads"] * (D * 4 + 4), "flops": 4 * pairs * D * c["q_heads"]}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_turn(x, s, sign=1):
    c = s["case"]
    x = x.detach().double()
    D = x.shape[-1]
    one, two = (x[..., :D // 2], x[..., D // 2:]) if c["half"] else (x[..., ::2], x[..., 1::2])
    axis = _axis_of_pair(c)
    angle = torch.empty(x.shape[0], D // 2, device=DEV, dtype=torch.float64)
    for p in range(D // 2):
        angle[:, p] = s["pos"][axis[p]].double() * (c["base"] ** (-2.0 * p / D)) * sign
    z = torch.complex(one, two) * torch.polar(torch.ones_like(angle), angle)[:, None]
    y = torch.empty_like(x)
    if c["half"]:
        y[..., :D // 2], y[..., D // 2:] = z.real, z.imag
    else:
        y[..., ::2], y[..., 1::2] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        out = {"q": _exact_turn(s["q"], s), "k": _exact_turn(s["k"], s)}
        if c["train"]:
            out["dq"], out["dk"] = _exact_turn(s["gq"], s, -1), _exact_turn(s["gk"], s, -1)
        return out
    if c["op"] == "pages":
        k, v = s["k_pages"].clone(), s["v_pages"].clone()
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            k[:, b], v[:, b] = s["k_pages"][:, a], s["v_pages"][:, a]
        return {"k_pages": k, "v_pages": v}
    n, kv = _lens(c)
    if c["op"] == "append":
        k, v, turned, t = s["k_pages"].double(), s["v_pages"].double(), _exact_turn(s["k"], s), 0
        for b in range(c["seqs"]):
            p = torch.arange(kv[b] - n[b], kv[b], device=DEV)
            page = s["table"][b].long()[p // c["page"]]
            k[0, page, :, p % c["page"]] = turned[t:t + n[b]]
            v[0, page, :, p % c["page"]] = s["v"][t:t + n[b]].double()
            t += n[b]
        return {"q": _exact_turn(s["q"], s), "k_pages": k, "v_pages": v}
    hq, hkv, D = c["q_heads"], c["kv_heads"], c["head_dim"]
    if 4.0 * s["T"] * max(kv) * hq * D > 4e12:
        return None
    o = torch.zeros(s["T"], hq, D, device=DEV, dtype=torch.float64)
    lse = torch.full((hq, s["T"]), -math.inf, device=DEV, dtype=torch.float64)
    pos, lo, _ = (torch.from_numpy(x).to(DEV) for x in _spans(c))
    t = 0
    for b in range(c["seqs"]):
        if n[b] == 0:
            continue
        rows = slice(t, t + n[b])
        t += n[b]
        pages = s["table"][b, :-(-kv[b] // c["page"])].long()
        j = torch.arange(kv[b], device=DEV)
        hidden = ~(((j >= lo[rows, None]) & (j <= pos[rows, None])) | ((j == 0) & bool(c["anchor"])))
        for h in range(hkv):
            k, v = (x[0, pages, h].reshape(-1, D)[:kv[b]].double() for x in (s["k_pages"], s["v_pages"]))
            for e in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                a = s["q"][rows, e].double() @ k.T / math.sqrt(D)
                a = a.masked_fill(hidden, -math.inf)
                lse[e, rows] = torch.logsumexp(a, dim=1)
                o[rows, e] = torch.softmax(a, dim=1) @ v
    return {"o": o, "lse": lse}
