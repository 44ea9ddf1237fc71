"""Plain 64-bit definitions of the multi-axis rotation and of attention over a paged cache, with the error bounds
that the GPU tests hold the kernels to (test infrastructure; CPU only)."""
import math

import torch


def turn(x, pos, axis_of_pair, theta, half, inverse=False):
    """x [T, H, D] rotated: pair p by pos[axis_of_pair[p]][t] * theta[p]. float64 [T, H, D]."""
    x = x.detach().double().cpu()
    D = x.shape[-1]
    ang = pos.double().cpu()[torch.tensor(axis_of_pair)].T * torch.tensor(theta, dtype=torch.float64)
    if inverse:
        ang = -ang
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    a, b = (x[..., :D // 2], x[..., D // 2:]) if half else (x[..., 0::2], x[..., 1::2])
    y = torch.empty_like(x)
    ya, yb = a * c - b * s, a * s + b * c
    if half:
        y[..., :D // 2], y[..., D // 2:] = ya, yb
    else:
        y[..., 0::2], y[..., 1::2] = ya, yb
    return y


def turn_bound(ref, x, half):
    """Half a bf16 step of the value (2^-8) and, relative to the pair's length, the angle's error (2^-20 rad for
    |pos| * theta <= 2^30) with six fp32 roundings (2^-24 each): together below 2^-19."""
    x = x.detach().double().cpu()
    D = x.shape[-1]
    if half:
        n = (x[..., :D // 2] ** 2 + x[..., D // 2:] ** 2).sqrt()
        n = torch.cat([n, n], dim=-1)
    else:
        n = (x[..., 0::2] ** 2 + x[..., 1::2] ** 2).sqrt().repeat_interleave(2, dim=-1)
    return ref.abs() * 2.0 ** -8 + n * 2.0 ** -19


def keys_of(pages, table_row, n, layer, head):
    """The first n tokens [n, D] of one head, through the page table. float64."""
    ps = pages.shape[3]
    idx = table_row[: -(-n // ps)].long()
    return pages[layer, idx, head].reshape(-1, pages.shape[-1])[:n].double()


def attend(q, k_pages, v_pages, table, cu_q, kv_len, layer=0, key_lo=None, anchor=False, scale=None):
    """(o, lse, o_bound, lse_bound), float64: o [T, Hq, D], lse [Hq, T]; rows outside [cu_q[0], cu_q[B]) are NaN.

    The bounds: with P_j the softmax weights and A = sum_j P_j |v_j|, a kernel that rounds the weights and the result to
    bf16 is off by at most 2^-8 A + 2^-8 |o| (half a step each). The logits are fp32 sums of D products, off by at most
    d = scale * D * 2^-24 * sum |q||k|, which moves a weight and their sum by a factor within exp(+-d) each; the
    exponential (2^-21), its argument's rounding (|x| 2^-23 for |x| < 128) and the fp32 sums of some hundred terms
    stay below 2^-14 together."""
    q, k_pages, v_pages, table, cu_q, kv_len = (x.detach().cpu() for x in (q, k_pages, v_pages, table, cu_q, kv_len))
    T, Hq, D = q.shape
    Hkv = k_pages.shape[2]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(D) if not scale else scale
    o = torch.full((T, Hq, D), math.nan, dtype=torch.float64)
    ob = torch.zeros_like(o)
    lse = torch.full((Hq, T), math.nan, dtype=torch.float64)
    lb = torch.zeros_like(lse)
    cu, kv = cu_q.tolist(), kv_len.tolist()
    lo_all = [0] * T if key_lo is None else key_lo.cpu().tolist()
    for b in range(len(kv)):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        m = max(kv[b], 0)
        pos = torch.arange(kv[b] - n, kv[b])
        lo = torch.tensor(lo_all[cu[b]:cu[b + 1]])
        j = torch.arange(m)
        seen = (j[None] >= lo[:, None]) & (j[None] <= pos[:, None])
        if anchor and m:
            seen[:, 0] |= pos >= 0
        used = seen.any(0)
        for g in range(Hkv):
            k, v = keys_of(k_pages, table[b], m, layer, g), keys_of(v_pages, table[b], m, layer, g)
            k, v = torch.where(used[:, None], k, 0.0), torch.where(used[:, None], v, 0.0)
            for h in range(g * G, (g + 1) * G):
                qq = q[cu[b]:cu[b + 1], h].double()
                s = (qq @ k.T * scale).masked_fill(~seen, -math.inf)
                any_ = seen.any(1)
                top = torch.where(any_, s.amax(1) if m else torch.zeros(n), 0.0)
                w = torch.exp(s - top[:, None]) if m else torch.zeros(n, 0, dtype=torch.float64)
                tot = w.sum(1)
                p = w / tot.clamp(min=1e-300)[:, None]
                rows = slice(cu[b], cu[b + 1])
                o[rows, h] = p @ v
                lse[h, rows] = torch.where(any_, top + tot.log(), -math.inf)
                d = (qq.abs() @ k.abs().T * seen).amax(1) * scale * D * 2.0 ** -24 if m else torch.zeros(n)
                A = p @ v.abs()
                ob[rows, h] = 2.0 ** -8 * o[rows, h].abs() + (2.0 ** -8 + 2 * d[:, None] + 2.0 ** -14) * A
                lb[h, rows] = d + 2.0 ** -14 + 2.0 ** -22 * torch.where(any_, lse[h, rows].abs(), 0.0)
    return o, lse, ob, lb


def check_attend(o, lse, ref, rows=None, tag=""):
    """Kernel outputs against attend()'s; rows outside the batch are not looked at."""
    ro, rl, ob, lb = ref
    o, lse = o.detach().double().cpu(), lse.detach().double().cpu()
    keep = ~torch.isnan(ro[:, 0, 0])
    err = (o[keep] - ro[keep]).abs() - ob[keep]
    assert not torch.isnan(o[keep]).any(), f"{tag}: NaN in o"
    assert keep.sum() == 0 or err.max() <= 0, f"{tag}: o beyond its bound by {err.max():.3e}"
    g, r = lse[:, keep], rl[:, keep]
    inf = torch.isinf(r)
    assert torch.equal(g[inf], r[inf]), f"{tag}: lse of rows that see nothing"
    err = ((g - r).abs() - lb[:, keep])[~inf]
    assert err.numel() == 0 or err.max() <= 0, f"{tag}: lse beyond its bound by {err.max():.3e}"


def make_batch(seed, kv, new, Hq, Hkv, D, ps, layers=1, spare=3, pad=0, device="cpu", extra_width=1):
    """A random pool, page tables (shuffled pages, -1 behind the last), lengths and rotated queries."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(x, 0) // ps) for x in kv]
    P, W, B = sum(need) + spare, max(max(need), 1) + extra_width, len(kv)
    perm = torch.randperm(P, generator=g).tolist()
    table = torch.full((B, W), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
    cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32)
    T = int(cu[-1]) + pad
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    d = dict(k_pages=r(layers, P, Hkv, ps, D), v_pages=r(layers, P, Hkv, ps, D), table=table, cu=cu,
             kv=torch.tensor(kv, dtype=torch.int32), q=r(T, Hq, D), k=r(T, Hkv, D), v=r(T, Hkv, D))
    return {k: v.to(device) for k, v in d.items()} | {"T": T, "max_q": max(new), "used": set(perm[:at]), "P": P}
