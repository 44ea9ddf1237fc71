"""Plain 64-bit definitions of 8-bit pages and of drafted trees (test infrastructure; CPU only). Bounds are
serving_reference's."""
import math

import torch

import serving_reference as ref

CODES = None  # the values of the 256 e4m3 codes


def code_values():
    """sign, four bits of exponent (bias 7, 0: subnormal), three of significand; float64 [256], NaN for the two NaN codes."""
    global CODES
    if CODES is None:
        x = torch.arange(256)
        e, m = (x >> 3) & 15, (x & 7).double()
        mag = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
        mag[(x & 127) == 127] = math.nan
        CODES = torch.where(x >= 128, -mag, mag)
    return CODES


def values(pages, scales):
    """What 8-bit pages stand for, float64."""
    b = scales.cpu().view(torch.uint8).double()
    p = torch.where(b == 255, math.nan, torch.exp2(b - 127))
    return code_values()[pages.cpu().view(torch.uint8).long()] * p[..., None]


def as_bf16(pages, scales):
    """values() as bf16, which holds them exactly."""
    v = values(pages, scales)
    assert torch.equal(v.to(torch.bfloat16).double().nan_to_num(7.0), v.nan_to_num(7.0))
    return v.to(torch.bfloat16)


def exponent(x):
    """The exponent of each row of x [..., D], float64: the smallest in [-100, 119] with max |x| <= 448 * 2^e."""
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)  # top = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    return torch.where(top == 0, -100, (e - 9 + (m > 0.875).int()).clamp(-100, 119))


def quantise(x):
    """(values held, exponents) of rows x [..., D] float64: the nearest code, ties to the even one."""
    e = exponent(x)
    y = (x * torch.exp2(-e.double())[..., None]).clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * torch.exp2(e.double())[..., None], e


def to_pages(v_bf16):
    """Random bf16 pages as 8-bit ones: (codes, scales) tensors."""
    x = v_bf16.double()
    held, e = quantise(x)
    codes = (held * torch.exp2(-e.double())[..., None]).float().to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def make_batch8(*a, device="cpu", **k):
    """serving_reference.make_batch with 8-bit pages; "kd" and "vd": what they hold, in bf16."""
    d = ref.make_batch(*a, **k)
    g = torch.Generator().manual_seed(17)
    for x in "kv":
        size = torch.randint(-4, 4, d[x + "_pages"].shape[:-1], generator=g)
        codes, scales = to_pages(d[x + "_pages"] * torch.exp2(size)[..., None])
        d[x + "d"], d[x + "_pages"], d[x + "_scales"] = as_bf16(codes, scales), codes, scales
    return {k: v.to(device) if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def masks_of(parents, cu, words):
    """(seen [T][set of new tokens], depth [T]) of trees given by parents."""
    seen, depth = [], []
    for b in range(len(cu) - 1):
        for i in range(cu[b + 1] - cu[b]):
            up = parents[cu[b] + i]
            seen.append(({i} | seen[cu[b] + up]) if up >= 0 else {i})
            depth.append(depth[cu[b] + up] + 1 if up >= 0 else 0)
    return seen, depth


def pack(seen, words):
    """Sets of new tokens as masks int64 [T, words]."""
    out = torch.zeros(len(seen), words, dtype=torch.int64)
    for t, s in enumerate(seen):
        for w in range(words):
            bits = sum(1 << c - 64 * w for c in s if 64 * w <= c < 64 * w + 64)
            out[t, w] = bits - (1 << 64) if bits >> 63 else bits
    return out


def random_tree(gen, new, chain=False):
    """parents int32 [T] of random trees, one per sequence."""
    out = []
    for n in new:
        for i in range(n):
            out.append(i - 1 if chain else int(torch.randint(-1, max(i, 0), (1,), generator=gen)) if i else -1)
    return torch.tensor(out, dtype=torch.int32)


def attend_tree(q, k_pages, v_pages, table, cu_q, kv_len, tree, layer=0, key_lo=None, anchor=False, scale=None):
    """serving_reference.attend with a drafted tree's visible keys: the same result and bounds."""
    q, k_pages, v_pages, table, tree = (x.detach().cpu() for x in (q, k_pages, v_pages, table, tree))
    T, Hq, D = q.shape
    Hkv, G = k_pages.shape[2], Hq // k_pages.shape[2]
    scale = 1.0 / math.sqrt(D) if not scale else scale
    o = torch.full((T, Hq, D), math.nan, dtype=torch.float64)
    ob, lse = torch.zeros_like(o), torch.full((Hq, T), math.nan, dtype=torch.float64)
    lb = torch.zeros_like(lse)
    cu, kv = cu_q.tolist(), kv_len.tolist()
    lo_all = [0] * T if key_lo is None else key_lo.cpu().tolist()
    rows_bits = [[int(w) & (1 << 64) - 1 for w in r] for r in tree.tolist()]
    for b in range(len(kv)):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        m, base = max(kv[b], 0), kv[b] - n
        seen = torch.zeros(n, m, dtype=torch.bool)
        for i in range(n):
            if base + i < 0:
                continue
            seen[i, min(max(lo_all[cu[b] + i], 0), max(base, 0)):max(base, 0)] = True
            if anchor and base > 0:
                seen[i, 0] = True
            for c in range(n):
                if c // 64 < tree.shape[1] and rows_bits[cu[b] + i][c // 64] >> c % 64 & 1 and base + c >= 0:
                    seen[i, base + c] = True
        used = seen.any(0)
        for g in range(Hkv):
            k, v = ref.keys_of(k_pages, table[b], m, layer, g), ref.keys_of(v_pages, table[b], m, layer, g)
            k, v = torch.where(used[:, None], k, 0.0), torch.where(used[:, None], v, 0.0)
            for h in range(g * G, (g + 1) * G):
                qq = q[cu[b]:cu[b + 1], h].double()
                s = (qq @ k.T * scale).masked_fill(~seen, -math.inf)
                some = seen.any(1)
                top = torch.where(some, s.amax(1) if m else torch.zeros(n), 0.0)
                w = torch.exp(s - top[:, None])
                tot = w.sum(1)
                p = w / tot.clamp(min=1e-300)[:, None]
                rows = slice(cu[b], cu[b + 1])
                o[rows, h] = p @ v
                lse[h, rows] = torch.where(some, top + tot.log(), -math.inf)
                d = (qq.abs() @ k.abs().T * seen).amax(1) * scale * D * 2.0 ** -24 if m else torch.zeros(n)
                ob[rows, h] = 2.0 ** -8 * o[rows, h].abs() + (2.0 ** -8 + 2 * d[:, None] + 2.0 ** -14) * (p @ v.abs())
                lb[h, rows] = d + 2.0 ** -14 + 2.0 ** -22 * torch.where(some, lse[h, rows].abs(), 0.0)
    return o, lse, ob, lb


def accept(pages, table, cu, kv, path):
    """pages [L, P, Hkv, ps, ...] after path[b][i] moved to place i behind the cached tokens of each sequence."""
    out, ps = pages.clone(), pages.shape[3]
    for b, p in enumerate(path):
        base = kv[b] - (cu[b + 1] - cu[b])
        for i, x in enumerate(p):
            f, t = base + x, base + i
            out[:, int(table[b, t // ps]), :, t % ps] = pages[:, int(table[b, f // ps]), :, f % ps]
    return out
