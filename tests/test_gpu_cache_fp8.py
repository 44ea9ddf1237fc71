"""GPU: the paged cache with 8-bit pages (append, read, attend, copies, the bookkeeping) against plain 64-bit definitions,
element by element."""
import math

import pytest
import torch

import drafts_reference as dr
import serving_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def aa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import packed_sequence_rope_gb300 as pkg
    return pkg


def _cache(aa, d, ps, Hkv, D, **kw):
    return aa.PagedCache(d["P"], ps, Hkv, D, num_layers=d["k_pages"].shape[0],
                         **{x: d[x] for x in ("k_pages", "v_pages", "k_scales", "v_scales")}, **kw)


def _attend(aa, d, ps, Hkv, D, tag="", layer=0, **kw):
    with _cache(aa, d, ps, Hkv, D) as c:
        o, lse = c.attend(d["q"], d["table"], d["cu"], d["kv"], d["max_q"], layer=layer, return_lse=True, **kw)
        torch.cuda.synchronize()
        c.check_device_error()
    want = ref.attend(d["q"], d["kd"], d["vd"], d["table"], d["cu"], d["kv"], layer, kw.get("key_lo"),
                      kw.get("anchor", False), kw.get("softmax_scale"))
    ref.check_attend(o, lse, want, tag=tag)
    return o, lse


# ------------------------------------------------------------------ what pages hold
@pytest.mark.parametrize("D", [64, 128])
def test_read_gives_every_code_at_every_scale(aa, D):
    """254 codes and the scales at which bf16 holds all of them; 255 makes a row NaN."""
    codes = torch.tensor([x for x in range(256) if x & 127 != 127], dtype=torch.uint8)
    rows = -(-len(codes) // D)
    bytes_ = list(range(10, 247)) + [255]
    n = rows * len(bytes_)
    P = -(-n // 16)
    pages = torch.zeros(1, P, 1, 16, D, dtype=torch.uint8)
    scales = torch.full((1, P, 1, 16), 127, dtype=torch.uint8)
    flat = torch.zeros(rows * D, dtype=torch.uint8)
    flat[:len(codes)] = codes
    pages.view(-1, D)[:n] = flat.view(rows, D).repeat(len(bytes_), 1)
    scales.view(-1)[:n] = torch.tensor(bytes_, dtype=torch.uint8).repeat_interleave(rows)
    k, s = pages.view(torch.float8_e4m3fn).cuda(), scales.view(torch.float8_e8m0fnu).cuda()
    table = torch.arange(P, dtype=torch.int32)[None].cuda()
    cu, kv = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([0, n], [n]))
    with aa.PagedCache(P, 16, 1, D, k_pages=k, v_pages=k.flip(1).contiguous(), k_scales=s, v_scales=s.view(torch.uint8).flip(1)
                       .contiguous().view(torch.float8_e8m0fnu)) as c:
        got_k, got_v = c.read(table, cu, kv, n)
        back = c.read(table.flip(1).contiguous(), cu, kv, n)[1]
    want = dr.values(pages, scales).view(-1, D)[:n]
    for got in (got_k, back):
        got = got.cpu().double().view(n, D)
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(9.0), want.nan_to_num(9.0))


@pytest.mark.parametrize("byte", [3, 4, 9, 246, 255])
def test_read_at_the_ends_of_the_range(aa, byte):
    codes = torch.tensor([x for x in range(256) if x & 127 != 127] + [0, 0], dtype=torch.uint8).view(4, 64)
    pages = torch.zeros(1, 1, 1, 16, 64, dtype=torch.uint8)
    pages[0, 0, 0, :4] = codes
    scales = torch.full((1, 1, 1, 16), byte, dtype=torch.uint8)
    k, s = pages.view(torch.float8_e4m3fn).cuda(), scales.view(torch.float8_e8m0fnu).cuda()
    table, cu, kv = (torch.tensor(t, dtype=torch.int32).cuda() for t in ([[0]], [0, 4], [4]))
    with aa.PagedCache(1, 16, 1, 64, k_pages=k, v_pages=k.clone(), k_scales=s, v_scales=s.clone()) as c:
        got = c.read(table, cu, kv, 4)
    want = dr.values(pages, scales)[0, 0, 0, :4]
    assert torch.equal(want.to(torch.bfloat16).double().nan_to_num(9.0), want.nan_to_num(9.0))  # bf16 holds them
    for g in got:
        g = g.cpu().double().view(4, 64)
        assert torch.equal(g.isnan(), want.isnan()) and torch.equal(g.nan_to_num(9.0), want.nan_to_num(9.0))


@pytest.mark.parametrize("ps", [16, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("half", [False, True, None])
@pytest.mark.parametrize("new", [[1, 1, 1, 0, 1], [1, 0, 130, 57, 3]])
def test_append_quantises_what_it_writes(aa, ps, D, half, new):
    """The held values are the nearest codes of the rotated ones; nothing else of the pool changes. Rotated values are
    off by 2^-19 of their pair's length before they are rounded (serving_reference.turn_bound), so a value is held
    within half a step of its own, 2^-4 of its size or 2^-10 of the scale, and that error, at a scale that the row's
    maximum gives within the same error."""
    torch.manual_seed(ps + D)
    kv = [n + x for n, x in zip(new, (0, 5, 40, 16, 200))]
    Hq, Hkv = 6, 2
    d = dr.make_batch8(ps + D, kv, new, Hq, Hkv, D, ps, layers=2, pad=2, device="cuda")
    k, v = (d[x] * torch.exp2(torch.randint(-9, 9, d[x].shape[:2], device="cuda"))[..., None] for x in "kv")
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    T, n = d["T"], sum(new)
    before = {x: d[x].view(torch.uint8).clone() for x in ("k_pages", "v_pages", "k_scales", "v_scales")}
    rope = pos = None
    if half is not None:
        rope = aa.RopeAxes(D, sections=(D // 2,), base=1e4, layout=aa.ROPE_HALF if half else aa.ROPE_ADJACENT)
        pos = torch.randint(0, 100000, (1, T), dtype=torch.int32, device="cuda")
    with _cache(aa, d, ps, Hkv, D) as c:
        q = c.append(k, v, d["table"], d["cu"], d["kv"], layer=1, rope=rope, pos=pos, q=d["q"] if rope else None)
        rk, rv = c.read(d["table"], d["cu"], d["kv"], T, layer=1)
        torch.cuda.synchronize()
        c.check_device_error()
    touched = torch.zeros(before["k_scales"].shape, dtype=torch.bool, device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
    p = torch.cat([torch.arange(a - b, a) for a, b in zip(kv, new)])
    page = d["table"].cpu()[seq, p // ps].long()
    touched[1, page, :, p % ps] = True
    for x in before:
        m = touched if "scales" in x else touched[..., None].expand_as(before[x])
        assert torch.equal(d[x].view(torch.uint8)[~m], before[x][~m]), x
    if rope:
        want = ref.turn(k, pos, rope.axis_of_pair, [1e4 ** (-2.0 * i / D) for i in range(D // 2)], half)
        off = ref.turn_bound(want, k, half) - want.abs() * 2.0 ** -8
        wq = ref.turn(d["q"], pos, rope.axis_of_pair, [1e4 ** (-2.0 * i / D) for i in range(D // 2)], half)
        assert ((q.cpu().double() - wq).abs() <= ref.turn_bound(wq, d["q"], half))[:n].all()
    else:
        want, off = k.cpu().double(), torch.zeros(k.shape, dtype=torch.float64)
    scale_k = torch.exp2(d["k_scales"].view(torch.uint8).cpu()[1, page, :, p % ps].double() - 127)
    got = dr.values(d["k_pages"], d["k_scales"])[1, page, :, p % ps]
    assert torch.equal(rk[:n].cpu().double(), got)
    want, off = want[:n], off[:n]
    assert ((got - want).abs() <= torch.maximum(want.abs() * 2.0 ** -4, scale_k[..., None] * 2.0 ** -10) + off * 1.0625).all()
    top, slack = want.abs().amax(-1), off.amax(-1)
    assert (top <= 448 * scale_k + slack).all() and (top >= 224 * scale_k - slack).all()
    held, e = dr.quantise(v.cpu().double()[:n])
    assert torch.equal(rv[:n].cpu().double(), held)
    assert torch.equal(d["v_scales"].view(torch.uint8).cpu()[1, page, :, p % ps].int() - 127, e.int())
    if not rope:
        assert torch.equal(rk[:n].cpu().double(), dr.quantise(k.cpu().double()[:n])[0])


def test_append_of_rows_at_the_borders(aa):
    """Maxima at and around 448 times a power of two, zeros, the type's largest and smallest values, ties; NaN and infinities
    make their row NaN and no other."""
    rows = [[0.0], [448.0], [450.0], [224.0], [226.0], [2.0 ** 127 * 1.75], [3.3895e38], [2.0 ** -126], [2.0 ** -133],
            [448 * 2.0 ** -100], [450 * 2.0 ** -100], [447.0 * 2.0 ** -100], [1.0, 1.0625, 1.1875, -1.0625, 2.0 ** -9],
            [448.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11, -2.0 ** -10], [math.inf], [-math.inf, 1.0], [math.nan, 3.0]]
    x = torch.zeros(len(rows), 1, 64)
    for i, r in enumerate(rows):
        x[i, 0, 5:5 + len(r)] = torch.tensor(r, dtype=torch.float64).float()
        if i % 2 == 0:
            x[i, 0, 63] = x[i, 0, 5]
    x = x.to(torch.bfloat16).cuda()
    n = len(rows)
    table, cu, kv = torch.tensor([[1, 0]], dtype=torch.int32).cuda(), *(torch.tensor(t, dtype=torch.int32).cuda() for t in ([0, n], [n]))
    with aa.PagedCache(2, 16 if n <= 32 else 32, 1, 64, dtype=torch.float8_e4m3fn, device="cuda") as c:
        c.append(x, x, table, cu, kv)
        k, v = c.read(table, cu, kv, n)
        c.check_device_error()
    fine = torch.isfinite(x.float()).all(-1).all(-1).cpu()
    assert fine.sum() == n - 3
    held, _ = dr.quantise(x.cpu().double())
    for got in (k, v):
        assert torch.equal(got.cpu().double()[fine], held[fine]) and got.cpu()[~fine].isnan().all()


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_append_of_rotated_keys_that_fp32_does_not_hold(aa, half, D):
    """Pairs of bf16's largest values are longer than fp32's largest: what passes 448 * 2^119 becomes that, and no row is NaN.
    Bound: the angle's 2^-19 of the pair's length, then half a code's step."""
    n = 40
    top = 3.3895e38
    k = torch.zeros(n, 1, D, dtype=torch.float64)
    k[:, 0, :] = top * torch.where(torch.arange(n * D).view(n, D) % 7 < 3, 1.0, -1.0)
    k[::3, 0, 2:] = 1.0e30
    k = k.to(torch.bfloat16).cuda()
    rope = aa.RopeAxes(D, sections=(D // 2,), base=1e4, layout=aa.ROPE_HALF if half else aa.ROPE_ADJACENT)
    pos = (torch.arange(n, dtype=torch.int32) * 3).cuda()
    table, cu, kv = torch.tensor([[2, 0, 1]], dtype=torch.int32).cuda(), *(torch.tensor(t, dtype=torch.int32).cuda() for t in ([0, n], [n]))
    with aa.PagedCache(3, 16, 1, D, dtype=torch.float8_e4m3fn, device="cuda") as c:
        c.append(k, k, table, cu, kv, rope=rope, pos=pos)
        got, _ = c.read(table, cu, kv, n)
        c.check_device_error()
    want = ref.turn(k, pos[None], rope.axis_of_pair, [1e4 ** (-2.0 * i / D) for i in range(D // 2)], half)
    off = ref.turn_bound(want, k, half) - want.abs() * 2.0 ** -8
    assert (want.abs() > 3.5e38).any()
    held = want.clamp(-448 * 2.0 ** 119, 448 * 2.0 ** 119)
    err = (got.cpu().double() - held).abs()
    assert (err <= torch.maximum(held.abs() * 2.0 ** -4, torch.tensor(2.0 ** 109, dtype=torch.float64)) + off * 1.0625).all()


def test_append_of_slices_many_sequences_and_steps(aa):
    """Token by token, from slices of a joint projection, what one call writes."""
    B, ps, Hkv, D = 150, 32, 3, 128
    kv = [1 + 7 * b % 60 for b in range(B)]
    d = dr.make_batch8(1, kv, [1] * B, 6, Hkv, D, ps, device="cuda")
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(B, 6 + 2 * Hkv, D, generator=g).to(torch.bfloat16).cuda()
    q, k, v = qkv.split([6, Hkv, Hkv], dim=1)
    rope = aa.RopeAxes(D, sections=(64,), base=5e5)
    pos = torch.arange(B, dtype=torch.int32, device="cuda")[None] * 17
    with _cache(aa, d, ps, Hkv, D) as c:
        out = c.append(k, v, d["table"], d["cu"], d["kv"], rope=rope, pos=pos, q=q)
        rk, rv = c.read(d["table"], d["cu"], d["kv"], B)
        one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        for b in (0, 1, 77, 149):
            s = slice(b, b + 1)
            assert torch.equal(c.append(k[s], v[s], d["table"][s], one, d["kv"][s], rope=rope, pos=pos[:, s], q=q[s]), out[s])
            again = c.read(d["table"][s], one, d["kv"][s], 1)
            assert torch.equal(again[0], rk[s]) and torch.equal(again[1], rv[s])
        c.check_device_error()
    assert torch.equal(rv.cpu().double(), dr.quantise(v.cpu().double())[0])


@pytest.mark.parametrize("fp8", [False, True])
def test_read_leaves_other_rows_and_reports_bad_pages(aa, fp8):
    kv, new, ps, Hkv, D = [40, 0, 21], [7, 0, 21], 16, 2, 64
    d = (dr.make_batch8 if fp8 else ref.make_batch)(3, kv, new, 2, Hkv, D, ps, layers=2, pad=3, device="cuda")
    kw = {x: d[x] for x in ("k_scales", "v_scales")} if fp8 else {}
    want = [d["kd"], d["vd"]] if fp8 else [d["k_pages"], d["v_pages"]]
    with aa.PagedCache(d["P"], ps, Hkv, D, num_layers=2, k_pages=d["k_pages"], v_pages=d["v_pages"], **kw) as c:
        out = [torch.full((d["T"], Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        got = c.read(d["table"], d["cu"], d["kv"], d["T"], layer=1, out_k=out[0], out_v=out[1])
        assert got[0] is out[0] or got[0].data_ptr() == out[0].data_ptr()
        c.check_device_error()
        for o, w in zip(out, want):
            assert (o[28:] == 7.0).all()
            for b, t in ((0, 0), (2, 7)):
                for g in range(Hkv):
                    rows = ref.keys_of(w.cpu(), d["table"][b].cpu(), kv[b], 1, g)[kv[b] - new[b]:]
                    assert torch.equal(o[t:t + new[b], g].cpu().double(), rows)
        bad = d["table"].clone()
        bad[2, 1] = d["P"]  # positions 16 to 20 of the last sequence
        k, v = c.read(bad, d["cu"], d["kv"], d["T"], layer=1)
        assert (k[23:28] == 0).all() and (v[23:28] == 0).all() and torch.equal(k[:23], out[0][:23])
        with pytest.raises(aa.AAError):
            c.check_device_error()
        c.read(d["table"][:, :2].contiguous(), d["cu"], d["kv"], d["T"])  # position 33 lies behind two pages of 16
        with pytest.raises(aa.AAError):
            c.check_device_error()
        k, v = c.read(d["table"], d["cu"], d["kv"], 0)
        assert k.shape == (0, Hkv, D)


# ------------------------------------------------------------------ attention
LENGTHS = [0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 513]


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 2), (7, 1), (16, 1), (20, 4)])
def test_single_tokens(aa, ps, D, Hq, Hkv):
    d = dr.make_batch8(ps + D + Hq, LENGTHS, [1] * len(LENGTHS), Hq, Hkv, D, ps, device="cuda")
    _attend(aa, d, ps, Hkv, D)


@pytest.mark.parametrize("Hq,Hkv", [(32, 1), (64, 1), (33, 1), (17, 1), (100, 2)])
def test_single_tokens_many_heads_per_group(aa, Hq, Hkv):
    d = dr.make_batch8(Hq, [1, 64, 300, 1030], [1] * 4, Hq, Hkv, 128, 64, device="cuda")
    _attend(aa, d, 64, Hkv, 128)


@pytest.mark.parametrize("kv,B", [(9000, 1), (4097, 3), (70000, 1)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 64)])
def test_single_tokens_over_long_contexts(aa, kv, B, Hq, Hkv, D):
    lens = [max(kv // (b + 1), 1) for b in range(B)]
    d = dr.make_batch8(kv, lens, [1] * B, Hq, Hkv, D, 32, device="cuda")
    _attend(aa, d, 32, Hkv, D)


@pytest.mark.parametrize("anchor", [False, True])
def test_single_tokens_masks(aa, anchor):
    kv = [1, 5, 64, 65, 130, 300, 300, 300, 300, 1000, 0, 2000]
    lo = [0, -4, 63, 64, 128, 299, 300, 10 ** 9, -2 ** 31, 937, 0, 1]
    for Hq, Hkv, ps, D in ((8, 2, 16, 128), (4, 4, 64, 64)):
        d = dr.make_batch8(11, kv, [1] * len(kv), Hq, Hkv, D, ps, device="cuda")
        o, lse = _attend(aa, d, ps, Hkv, D, key_lo=torch.tensor(lo, dtype=torch.int32, device="cuda"), anchor=anchor)
        empty = [10] + ([] if anchor else [6, 7])
        assert (o[empty] == 0).all() and (lse[:, empty] == -math.inf).all()


CHUNKS = [([1, 2, 5, 17], [1, 2, 100, 64]), ([0, 3, 0, 0, 40, 0], [50, 3, 0, 7, 333, 1]), ([130, 1, 257], [130, 700, 1000]),
          ([33, 16, 64], [33, 1500, 65]), ([500], [1300])]


@pytest.mark.parametrize("chunk", range(len(CHUNKS)))
@pytest.mark.parametrize("ps", [16, 32, 128])
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 64), (8, 2, 128), (6, 2, 128), (7, 1, 64), (16, 1, 128)])
def test_chunks(aa, chunk, ps, Hq, Hkv, D):
    new, kv = CHUNKS[chunk]
    d = dr.make_batch8(chunk, kv, new, Hq, Hkv, D, ps, device="cuda")
    _attend(aa, d, ps, Hkv, D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [2, 40])
@pytest.mark.parametrize("most", [500, 1500])
def test_up_to_64_rows(aa, D, B, most):
    for new in (8, 13, 16):
        kv = [max(new, most - 37 * b % most) for b in range(B)]
        d = dr.make_batch8(new + B, kv, [new - b % 3 for b in range(B)], 8, 2, D, 32, device="cuda")
        _attend(aa, d, 32, 2, D)


@pytest.mark.parametrize("anchor", [False, True])
@pytest.mark.parametrize("new", [3, 70, 300])
def test_chunk_masks(aa, anchor, new):
    """Packed documents, a sliding window, and rows that see nothing in between."""
    kv = [new, new + 41, new + 700]
    p = torch.cat([torch.arange(k - new, k) for k in kv])
    docs = torch.where(p > 0, 1 + torch.div(p - 1, 90, rounding_mode="floor") * 90, torch.zeros_like(p))
    window = (p - 33).clamp(min=-5)
    g = torch.Generator().manual_seed(4)
    mixed = torch.where(torch.rand(3 * new, generator=g) < 0.2, p + 1 + torch.randint(0, 3, (3 * new,), generator=g),
                        (p * torch.rand(3 * new, generator=g)).long())
    for name, lo in (("docs", docs), ("window", window), ("mixed", mixed)):
        for Hq, Hkv, D, ps in ((4, 1, 128, 32), (2, 2, 64, 128)):
            d = dr.make_batch8(new, kv, [new] * 3, Hq, Hkv, D, ps, device="cuda")
            _attend(aa, d, ps, Hkv, D, tag=name, key_lo=lo.to(torch.int32).cuda(), anchor=anchor)


@pytest.mark.parametrize("new,kv,Hq,Hkv,D", [(17, 52000, 8, 1, 128), (5, 70000, 16, 1, 64), (33, 2200, 8, 2, 128),
                                              (130, 9000, 16, 2, 128), (300, 5000, 4, 4, 64)])
def test_few_units_with_many_parts(aa, new, kv, Hq, Hkv, D):
    d = dr.make_batch8(new, [kv, kv // 3], [new, new // 2], Hq, Hkv, D, 64, device="cuda")
    _attend(aa, d, 64, Hkv, D)
    lo = torch.full((new + new // 2,), kv // 5, dtype=torch.int32, device="cuda")
    lo[::7] = kv
    _attend(aa, d, 64, Hkv, D, key_lo=lo, anchor=True)


@pytest.mark.parametrize("new", [1, 4, 40, 200])
@pytest.mark.parametrize("ps", [16, 64])
def test_what_no_row_sees_does_not_reach_the_result(aa, new, ps):
    """NaN scales and codes in unused pages, behind the last token, in front of every window, and between seen keys."""
    kv, Hq, Hkv, D = [new + 70, new + 333, new], 4, 2, 128
    d = dr.make_batch8(new, kv, [new] * 3, Hq, Hkv, D, ps, device="cuda")
    first = [40, 300, 0]
    lo = torch.cat([torch.full((new,), x) for x in first])
    if new > 1:
        lo[new // 2] = 10 ** 6  # sees nothing: its own key lies between seen ones, or behind the last
    seen = torch.zeros(d["P"], ps, dtype=torch.bool, device="cuda")
    for b in range(3):
        p = torch.arange(kv[b] - new, kv[b])
        j = torch.arange(kv[b])
        j = j[((j >= lo[b * new:(b + 1) * new, None]) & (j <= p[:, None])).any(0)]
        seen[d["table"][b].cpu()[j // ps].long(), j % ps] = True
    for x in "kv":
        d[x + "_scales"].view(torch.uint8).masked_fill_(~seen[None, :, None], 255)
        d[x + "_pages"].view(torch.uint8).masked_fill_(~seen[None, :, None, :, None], 127)
    o, _ = _attend(aa, d, ps, Hkv, D, key_lo=lo.to(torch.int32).cuda())
    assert torch.isfinite(o.float()).all()


@pytest.mark.parametrize("new", [1, 150])
def test_a_token_that_is_nan_makes_the_rows_that_see_it_nan(aa, new):
    kv = 300 + new
    for x in "kv":
        d = dr.make_batch8(new, [kv, 50], [new, 1], 4, 2, 64, 64, device="cuda")
        at = 10
        d[x + "_scales"].view(torch.uint8)[0, d["table"][0, 0], :, at] = 255
        with _cache(aa, d, 64, 2, 64) as c:
            o = c.attend(d["q"], d["table"], d["cu"], d["kv"], new)
            late = c.attend(d["q"], d["table"], d["cu"], d["kv"], new,
                            key_lo=torch.full((new + 1,), at + 1, dtype=torch.int32, device="cuda"))
        assert o[:new].isnan().all() and not o[new:].isnan().any() and not late.isnan().any()


def test_large_logits_scales_and_values_far_apart(aa):
    for new in (1, 150):
        for scale in (0.5, 4.0):
            d = dr.make_batch8(6, [new + 400], [new], 4, 2, 64, 64, device="cuda")
            _attend(aa, d, 64, 2, 64, softmax_scale=scale)
        # tokens whose scales differ by a factor of 2^80
        d = dr.make_batch8(7, [new + 400], [new], 4, 2, 128, 16, device="cuda")
        e = d["v_scales"].view(torch.uint8)
        e.copy_(torch.randint(80, 160, e.shape, dtype=torch.uint8))
        d["vd"] = dr.as_bf16(d["v_pages"], d["v_scales"]).cuda()
        _attend(aa, d, 16, 2, 128)


def test_scales_far_from_one(aa):
    """Values at the ends of bf16's range: 2^-100 and 2^100 times ordinary ones, at every length of product."""
    for new in (1, 150):
        for shift in (-93, 7, 8, 9, 100):
            d = dr.make_batch8(8, [new + 90], [new], 4, 2, 128, 16, device="cuda")
            e = d["v_scales"].view(torch.uint8)
            e.copy_((e.int() - e.int().min() + max(27, 127 + shift - 4)).clamp(27, 247).to(torch.uint8))
            d["vd"] = dr.as_bf16(d["v_pages"], d["v_scales"]).cuda()
            e = d["k_scales"].view(torch.uint8)
            if shift > 0:  # queries that bring the logits back to ordinary sizes
                e.copy_((e.int() + shift).clamp(27, 247).to(torch.uint8))
                d["q"] = (d["q"].float() * 2.0 ** -shift).to(torch.bfloat16)
                d["kd"] = dr.as_bf16(d["k_pages"], d["k_scales"]).cuda()
            _attend(aa, d, 16, 2, 128, tag=f"{new} {shift}")


def _set_scales(d, x, top):
    """Keys or values (x) moved by a power of two: the largest scale becomes 2^(top - 127)."""
    e = d[x + "_scales"].view(torch.uint8)
    by = top - int(e.max())
    e.copy_((e.int() + by).clamp(27, 246).to(torch.uint8))
    d[x + "d"] = dr.as_bf16(d[x + "_pages"], d[x + "_scales"]).cuda()
    return by


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [1, 5, 150])
@pytest.mark.parametrize("top", [27, 60, 220, 232, 246])
def test_queries_and_keys_far_from_one_that_meet_in_the_middle(aa, new, D, top):
    """Keys at both ends of the range, queries that bring the logits back to ordinary sizes."""
    d = dr.make_batch8(12, [new + 90, new + 300], [new, new], 4, 2, D, 16, device="cuda")
    by = _set_scales(d, "k", top)
    d["q"] = (d["q"].double() * 2.0 ** -by).to(torch.bfloat16)
    lo = torch.arange(2 * new, dtype=torch.int32, device="cuda") % 40
    _attend(aa, d, 16, 2, D, tag=str(top))
    _attend(aa, d, 16, 2, D, tag=str(top), key_lo=lo, anchor=True)


@pytest.mark.parametrize("x", ["k", "v"])
@pytest.mark.parametrize("new", [1, 5, 40, 150])
@pytest.mark.parametrize("D", [64, 128])
def test_the_smallest_scales(aa, x, new, D):
    """Scales from 2^-124 on, where bf16 still holds every code: keys under queries that meet them, and values."""
    d = dr.make_batch8(16, [new + 90, new + 300], [new, new], 4, 2, D, 16, device="cuda")
    e = d[x + "_scales"].view(torch.uint8)
    by = 3 - int(e.min())
    e.copy_((e.int() + by).to(torch.uint8))
    d[x + "d"] = dr.as_bf16(d[x + "_pages"], d[x + "_scales"]).cuda()
    if x == "k":
        d["q"] = (d["q"].double() * 2.0 ** -by).to(torch.bfloat16)
    with _cache(aa, d, 16, 2, D) as c:
        o, lse = c.attend(d["q"], d["table"], d["cu"], d["kv"], new, return_lse=True)
        c.check_device_error()
    ro, rl, ob, lb = ref.attend(d["q"], d["kd"], d["vd"], d["table"], d["cu"], d["kv"])
    # results below 2^-126 lie 2^-133 apart: rounding one is off by up to half of that, whatever its size
    ref.check_attend(o, lse, (ro, rl, ob + 2.0 ** -134, lb))


@pytest.mark.parametrize("new", [1, 5, 150])
@pytest.mark.parametrize("scale", [1e-30, 1e-38, 1e-44])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -120, 1.0])
def test_tiny_softmax_scales(aa, new, scale, size):
    """All visible keys weigh the same; those that a mask hides weigh nothing, whatever the queries are."""
    d = dr.make_batch8(14, [new + 130, new + 40], [new, new], 4, 2, 64, 16, device="cuda")
    d["q"].mul_(size)
    lo = (torch.arange(2 * new, dtype=torch.int32, device="cuda") * 5 % 37)
    _attend(aa, d, 16, 2, 64, softmax_scale=scale)
    _attend(aa, d, 16, 2, 64, softmax_scale=scale, key_lo=lo, anchor=True)


@pytest.mark.parametrize("new", [1, 5, 40, 150])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_keys_under_ordinary_queries(aa, new, sign):
    """Logits of 2^100 and more that fp32 holds, of one sign: the largest takes all of the weight."""
    D = 128
    d = dr.make_batch8(13, [new + 150], [new], 4, 2, D, 64, device="cuda")
    _set_scales(d, "k", 232)  # 2^105
    d["q"].fill_(1.0)
    codes = d["k_pages"].view(torch.uint8)
    codes.copy_(codes & 127 if sign > 0 else codes | 128)
    d["kd"] = dr.as_bf16(d["k_pages"], d["k_scales"]).cuda()
    o, lse = _attend(aa, d, 64, 2, D)
    assert torch.isfinite(o.float()).all() and (lse * sign > 2.0 ** 100).all()
    # a row's heads of a kv head see the same keys with the same queries; its result is one key's value
    p = torch.arange(150, new + 150)
    for g in range(2):
        k, v = (ref.keys_of(d[x].cpu(), d["table"][0].cpu(), new + 150, 0, g) for x in ("kd", "vd"))
        s = k.sum(-1)
        for i in range(new):
            best = s[:p[i] + 1].argmax()
            second = s[:p[i] + 1].clone()
            second[best] = -math.inf
            if s[best] - second.max() > 2.0 ** -16 * s.abs().max():
                assert ((o[i, 2 * g].cpu().double() - v[best]).abs() <= 2.0 ** -8 * v[best].abs()).all()


def _logits(kind, n):
    """A logit per key that 8 bits hold, and the keys that may have weight; between the others and these lie more than 2^9."""
    j = torch.arange(n)
    near = ((j * 37 % 25).double() - 12) / 4
    if kind == "behind":  # far below the ones that come later
        s, of = torch.where(j < n - n // 3, -2.0 ** 30, near), j >= n - n // 3
    elif kind == "ahead":
        s, of = torch.where(j < n // 3, near, -2.0 ** (10 + j % 90)), j < n // 3
    elif kind == "low":  # all of them low, one the least
        s = -2.0 ** 24 * torch.exp2((j * 7 % 60 + 1).double())
        s[n // 2] = -2.0 ** 24
        of = j == n // 2
    elif kind == "growing":
        s, of = torch.exp2(10 + (j // 4).double() * 100 // n), j == n - 1
        s[-1] = 2.0 ** 112
    else:  # one far above, early
        s, of = near.clone(), j == 5
        s[5] = 2.0 ** float(kind)
    return s, of


def check_far_logits(aa, kind, new, D, fp8, n=700):
    """Queries and keys whose products are exact (one code times a power of two per key), over values whose scales lie far
    apart: what has weight is known, and the result is off by the roundings of the weights and its own alone."""
    Hq, Hkv, ps = 4, 2, 64
    d = dr.make_batch8(15, [n], [new], Hq, Hkv, D, ps, device="cuda")
    s, of = _logits(kind, n)
    e = d["v_scales"].view(torch.uint8)
    e.copy_(torch.randint(100, 150, e.shape, generator=torch.Generator().manual_seed(3), dtype=torch.uint8))
    d["vd"] = dr.as_bf16(d["v_pages"], d["v_scales"]).cuda()
    held, exp = dr.quantise(s[:, None])
    assert torch.equal(held[:, 0], s)
    codes = (held[:, 0] * torch.exp2(-exp.double())).float().to(torch.float8_e4m3fn).cuda()
    j = torch.arange(n, device="cuda")
    page = d["table"][0, j // ps].long()
    d["k_pages"].view(torch.uint8)[0, page, :, j % ps] = codes.view(torch.uint8)[:, None, None]
    d["k_scales"].view(torch.uint8)[0, page, :, j % ps] = (exp + 127).to(torch.uint8).cuda()[:, None]
    d["kd"] = dr.as_bf16(d["k_pages"], d["k_scales"]).cuda()
    d["q"].fill_(1.0)
    pool = {x: d[x] for x in ("k_pages", "v_pages", "k_scales", "v_scales")} if fp8 else dict(k_pages=d["kd"], v_pages=d["vd"])
    hi = torch.arange(n - new, n) if kind not in ("growing", "behind") else torch.full((new,), n - 1)
    tree = torch.full((new, -(-new // 64)), -1, dtype=torch.int64, device="cuda") if kind in ("growing", "behind") else None
    with aa.PagedCache(d["P"], ps, Hkv, D, **pool) as c:
        o, lse = c.attend(d["q"], d["table"], d["cu"], d["kv"], new, softmax_scale=1.0 / D, return_lse=True, tree=tree)
        c.check_device_error()
    o, lse = o.double().cpu(), lse.double().cpu()
    for g in range(Hkv):
        v = ref.keys_of(d["vd"].cpu(), d["table"][0].cpu(), n, 0, g)
        for i in range(new):
            seen = of & (j.cpu() <= hi[i])
            top = s[seen].max()
            w = torch.where(seen, (s - top).exp(), 0.0)
            p = w / w.sum()
            want, bound = p @ v, (2.0 ** -8 + 2.0 ** -14) * (p @ v.abs())
            for h in range(g * Hq // Hkv, (g + 1) * Hq // Hkv):
                assert ((o[i, h] - want).abs() <= bound + 2.0 ** -8 * want.abs()).all(), (kind, i, h)
                r = float(top + w.sum().log())
                assert abs(float(lse[h, i]) - r) <= 2.0 ** -14 + 2.0 ** -21 * abs(r)


FAR = ["behind", "ahead", "low", "growing", "11", "20", "40", "100"]


@pytest.mark.parametrize("kind", FAR)
@pytest.mark.parametrize("new", [1, 5, 16])
@pytest.mark.parametrize("D", [64, 128])
def test_logits_of_any_size(aa, kind, new, D):
    check_far_logits(aa, kind, new, D, True)


@pytest.mark.parametrize("kind", FAR)
@pytest.mark.parametrize("new", [40, 150])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [700, 3000])
def test_logits_of_any_size_in_chunks(aa, kind, new, D, n):
    check_far_logits(aa, kind, new, D, True, n)


@pytest.mark.parametrize("new", [1, 7, 90])
def test_growing_logits_over_large_values(aa, new):
    """Later keys outweigh earlier ones by up to 2^60, step by step, over values of 2^100: what rows keep on the way stays in range."""
    d = dr.make_batch8(9, [new + 1500], [new], 4, 2, 128, 64, device="cuda")
    e = d["v_scales"].view(torch.uint8)
    e.copy_((e.int() - e.int().min() + 217).clamp(27, 246).to(torch.uint8))
    d["vd"] = dr.as_bf16(d["v_pages"], d["v_scales"]).cuda()
    d["q"].fill_(0.25)
    j = torch.arange(new + 1500, device="cuda")
    # one code for all channels; logits 0.25 * 128 * value / sqrt(128) from 0 to 42 in steps
    code = torch.round(j * 14.0 / len(j)).to(torch.float8_e4m3fn)
    page = d["table"][0, (j // 64)].long()
    d["k_pages"].view(torch.uint8)[0, page, :, j % 64] = code.view(torch.uint8)[:, None, None]
    d["k_scales"].view(torch.uint8)[0, page, :, j % 64] = 127
    d["kd"] = dr.as_bf16(d["k_pages"], d["k_scales"]).cuda()
    o, _ = _attend(aa, d, 64, 2, 128)
    assert torch.isfinite(o.float()).all()


@pytest.mark.parametrize("new", [1, 5, 90])
def test_layers_strides_streams_and_graphs(aa, new):
    kv, ps, Hq, Hkv, D = [new + 300, new + 7], 32, 8, 2, 128
    d = dr.make_batch8(new, kv, [new, new], Hq, Hkv, D, ps, layers=3, pad=2, device="cuda")
    wide = torch.zeros(d["T"], Hq + 5, D, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:2 + Hq] = d["q"]
    o, lse = _attend(aa, d, ps, Hkv, D, layer=2)
    with _cache(aa, d, ps, Hkv, D) as c:
        args = (wide[:, 2:2 + Hq], d["table"], d["cu"], d["kv"], new)
        work = c.alloc_workspace(2, d["T"], new, d["table"].shape[1], Hq)
        out = torch.full_like(d["q"], 3.0)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        c.attend(*args, layer=2, out=out, workspace=work, stream=s)
        s.synchronize()
        assert torch.equal(out[:2 * new], o[:2 * new]) and (out[2 * new:] == 3.0).all()
        graph = torch.cuda.CUDAGraph()
        k, v = d["k"], d["v"]
        c.append(k, v, d["table"], d["cu"], d["kv"], layer=2)
        with torch.cuda.graph(graph):
            c.append(k, v, d["table"], d["cu"], d["kv"], layer=2)
            c.attend(*args, layer=2, out=out, workspace=work)
        d["kv"].sub_(1)  # both sequences one token shorter
        graph.replay()
        torch.cuda.synchronize()
        c.check_device_error()
        d["kd"], d["vd"] = dr.as_bf16(d["k_pages"], d["k_scales"]), dr.as_bf16(d["v_pages"], d["v_scales"])
        want = ref.attend(d["q"], d["kd"], d["vd"], d["table"], d["cu"], d["kv"], 2)
        ref.check_attend(out, c.attend(*args, layer=2, return_lse=True)[1], want)


@pytest.mark.parametrize("max_q", [0, 1, 4, 60, 1000])
def test_max_q_is_a_hint(aa, max_q):
    d = dr.make_batch8(8, [60, 500, 129], [1, 150, 40], 8, 2, 128, 64, device="cuda") | {"max_q": max_q}
    _attend(aa, d, 64, 2, 128)


@pytest.mark.parametrize("width", [1030, 4700])
@pytest.mark.parametrize("lo", [0, 170])
def test_wide_tables(aa, width, lo):
    """Rows for which 16-bit copies are made, of four sequences at a time because of their tables' width; and, where one
    sequence's would be too large, are not."""
    new, kv, ps, Hq, Hkv, D = [70, 0, 90, 66, 80], [300, 50, 90, 200, 700], 64, 32, 8, 128
    d = dr.make_batch8(width, kv, new, Hq, Hkv, D, ps, device="cuda")
    d["table"] = torch.cat([d["table"], torch.full((5, width - d["table"].shape[1]), -1, dtype=torch.int32, device="cuda")], 1)
    key_lo = torch.full((sum(new),), lo, dtype=torch.int32, device="cuda")
    key_lo[::9] += 40
    _attend(aa, d, ps, Hkv, D)
    _attend(aa, d, ps, Hkv, D, key_lo=key_lo, anchor=True)


@pytest.mark.parametrize("new,max_q", [(1, 1), (6, 6), (40, 1), (100, 100)])
@pytest.mark.parametrize("ps", [16, 64])
@pytest.mark.parametrize("D", [64, 128])
def test_buffers_of_unread_pages_are_used_again(aa, new, max_q, ps, D):
    """Pages that are not read, for a bad number, in front of a window or behind the last key, leave zeros for scales; the same
    buffers then take tiles whose scales are far from those. A bad page's keys and values are zeros."""
    Hq, Hkv, kv = 4, 2, [new + 3000, new + 1777]
    d = dr.make_batch8(new + ps, kv, [new, new], Hq, Hkv, D, ps, device="cuda")
    spare = next(p for p in range(d["P"]) if p not in d["used"])  # what the bad numbers stand for
    for x in "kv":
        d[x + "_pages"].view(torch.uint8)[:, spare].zero_()
        d[x + "d"] = dr.as_bf16(d[x + "_pages"], d[x + "_scales"]).cuda()
    holes = torch.zeros(d["table"].shape, dtype=torch.bool)
    holes[:, 1::5] = True  # behind the last page too, where nothing is looked up
    holes[:, (max(kv) - new) // ps:] = False
    holes &= (d["table"] >= 0).cpu()
    bad = torch.where(holes.cuda(), d["P"] + 5, d["table"])
    zeros = torch.where(holes.cuda(), spare, d["table"])
    p = torch.cat([torch.arange(k - new, k) for k in kv])
    with _cache(aa, d, ps, Hkv, D) as c:
        for lo, anchor in ((None, False), ((p - 1500).clamp(min=0), True)):
            lo = None if lo is None else lo.to(torch.int32).cuda()
            first = c.attend(d["q"], bad, d["cu"], d["kv"], max_q, key_lo=lo, anchor=anchor, return_lse=True)
            with pytest.raises(aa.AAError):
                c.check_device_error()
            want = ref.attend(d["q"], d["kd"], d["vd"], zeros, d["cu"], d["kv"], 0, lo, anchor)
            ref.check_attend(*first, want)
            for _ in range(3):
                again = c.attend(d["q"], bad, d["cu"], d["kv"], max_q, key_lo=lo, anchor=anchor, return_lse=True)
                assert all(torch.equal(a, b) for a, b in zip(again, first))


@pytest.mark.parametrize("chunk,width", [(300, 1030), (60, 1030), (300, 40)])
@pytest.mark.parametrize("D", [64, 128])
def test_a_chunk_among_single_tokens(aa, chunk, width, D):
    """One prompt chunk beside single tokens, sequences without any and rows that see nothing: where tables are wide, in several slices."""
    new = [1, 1, 0, chunk, 1, 1, 1, 7, 1, 1, 0, 1]
    kv = [1, 700, 50, chunk + 1000, 64, 65, 1, 300, 0, 2000, 0, 129]
    ps, Hq, Hkv = 64, 16 if D == 128 else 32, 8
    d = dr.make_batch8(chunk + width, kv, new, Hq, Hkv, D, ps, device="cuda")
    d["table"] = torch.cat([d["table"], torch.full((len(kv), width - d["table"].shape[1]), -1, dtype=torch.int32, device="cuda")], 1)
    _attend(aa, d, ps, Hkv, D)
    lo = torch.tensor([max(0, k - n - 100) for k, n in zip(kv, new) for _ in range(n)], dtype=torch.int32, device="cuda")
    lo[5::11] = 2 ** 30
    for anchor in (False, True):
        _attend(aa, d, ps, Hkv, D, key_lo=lo, anchor=anchor)


# ------------------------------------------------------------------ pages and bookkeeping
@pytest.mark.parametrize("n,ps,Hkv,D,L", [(1, 16, 1, 64, 1), (70, 16, 3, 64, 2), (9, 128, 8, 128, 3)])
def test_copy_pages(aa, n, ps, Hkv, D, L):
    d = dr.make_batch8(n, [ps * 2 * n], [1], Hkv, Hkv, D, ps, layers=L, device="cuda")
    order = torch.randperm(d["P"], generator=torch.Generator().manual_seed(n))[:2 * n].numpy().astype("int32")
    before = {x: d[x].view(torch.uint8).clone() for x in ("k_pages", "v_pages", "k_scales", "v_scales")}
    with _cache(aa, d, ps, Hkv, D) as c:
        c.copy_pages(order[:n], order[n:])
        torch.cuda.synchronize()
    for x, y in before.items():
        y[:, order[n:].tolist()] = y[:, order[:n].tolist()]
        assert torch.equal(d[x].view(torch.uint8), y), x


def test_a_run_with_forks_and_compaction(aa):
    """Prompts in chunks, a fork that grows into a shared page, steps of single tokens, a compaction: the cache holds
    each token's quantised key and value, and the attention over it is that of the definition."""
    ps, Hq, Hkv, D, L = 16, 8, 2, 64, 2
    rope = aa.RopeAxes(D, sections=(D // 2,), base=1e4, layout=aa.ROPE_HALF)
    theta = [1e4 ** (-2.0 * i / D) for i in range(D // 2)]
    g = torch.Generator().manual_seed(9)
    held = {}  # sequence -> (keys, values) per layer as bf16, all tokens
    with aa.PagedCache(64, ps, Hkv, D, num_layers=L, max_seqs=4, dtype=torch.float8_e4m3fn) as c:
        assert c.k_pages.dtype == torch.float8_e4m3fn and c.k_scales.shape == (L, 64, Hkv, ps)
        lens = {}

        def step(seqs, new):
            for s in seqs:
                lens[s] = lens.get(s, 0) + new
            c.resize(seqs, [lens[s] for s in seqs])
            table, kv = c.tables(seqs, device="cuda")
            T = new * len(seqs)
            cu = torch.arange(0, T + 1, new, dtype=torch.int32, device="cuda")
            pos = torch.cat([torch.arange(lens[s] - new, lens[s]) for s in seqs]).to(torch.int32).cuda()
            for layer in range(L):
                q, k, v = (torch.randn(T, h, D, generator=g).to(torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv))
                qr = c.append(k, v, table, cu, kv, layer=layer, rope=rope, pos=pos, q=q)
                o, lse = c.attend(qr, table, cu, kv, new, layer=layer, return_lse=True)
                rk, rv = c.read(table, cu, kv, T, layer=layer)
                want = ref.turn(k, pos[None], [0] * (D // 2), theta, True)
                scale = dr.exponent(want).double().exp2()[..., None]
                assert ((rk.cpu().double() - want).abs() <= torch.maximum(want.abs() * 2.0 ** -4, scale * 2.0 ** -9) * 1.001).all()
                assert torch.equal(rv.cpu().double(), dr.quantise(v.cpu().double())[0])
                for i, s in enumerate(seqs):
                    h = held.setdefault((s, layer), [torch.empty(0, Hkv, D, dtype=torch.bfloat16)] * 2)
                    held[s, layer] = [torch.cat([h[0], rk[i * new:(i + 1) * new].cpu()]), torch.cat([h[1], rv[i * new:(i + 1) * new].cpu()])]
                check(seqs, new, layer, qr, o, lse)
            c.check_device_error()

        def check(seqs, new, layer, q, o, lse):
            need = [-(-lens[s] // ps) for s in seqs]
            pages = [torch.zeros(1, sum(need), Hkv, ps, D, dtype=torch.bfloat16) for _ in range(2)]
            table, at = torch.full((len(seqs), max(need)), -1, dtype=torch.int32), 0
            for i, s in enumerate(seqs):
                table[i, :need[i]] = torch.arange(at, at + need[i])
                for x in range(2):
                    for t in range(lens[s]):
                        pages[x][0, at + t // ps, :, t % ps] = held[s, layer][x][t]
                at += need[i]
            cu = torch.arange(0, new * len(seqs) + 1, new)
            want = ref.attend(q, pages[0], pages[1], table, cu, torch.tensor([lens[s] for s in seqs]))
            ref.check_attend(o, lse, want)

        step([0, 1], 37)
        step([0, 1], 1)
        c.fork(0, 2)
        lens[2] = lens[0]
        for layer in range(L):
            held[2, layer] = list(held[0, layer])
        step([0, 2], 1)
        step([0, 1, 2], 3)
        c.free([1])
        del lens[1]
        assert c.compact() > 0
        step([0, 2], 1)
        step([2], 90)


def test_long_pool_offsets_pass_32_bits(aa):
    """Pages whose byte offsets pass 2^32, at the end of a large pool."""
    ps, Hkv, D = 128, 8, 128
    P = (1 << 32) // (ps * Hkv * D) + 300
    k, v = (torch.zeros(1, P, Hkv, ps, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((1, P, Hkv, ps), 127, dtype=torch.uint8, device="cuda") for _ in range(2))
    d = dr.make_batch8(5, [200, 300], [1, 1], 8, Hkv, D, ps, spare=0, device="cuda")
    n, at = d["P"], P - d["P"]
    for big, small in ((k, "k_pages"), (v, "v_pages"), (ks, "k_scales"), (vs, "v_scales")):
        big[:, at:] = d[small].view(torch.uint8)
    want = ref.attend(d["q"], d["kd"], d["vd"], d["table"], d["cu"], d["kv"])
    table = torch.where(d["table"] >= 0, d["table"] + at, d["table"])
    with aa.PagedCache(P, ps, Hkv, D, k_pages=k.view(torch.float8_e4m3fn), v_pages=v.view(torch.float8_e4m3fn),
                       k_scales=ks.view(torch.float8_e8m0fnu), v_scales=vs.view(torch.float8_e8m0fnu)) as c:
        o, lse = c.attend(d["q"], table, d["cu"], d["kv"], 1, return_lse=True)
        c.append(d["k"], d["v"], table, d["cu"], d["kv"])
        rk, rv = c.read(table, d["cu"], d["kv"], 2)
        c.check_device_error()
    ref.check_attend(o, lse, want)
    for got, x in ((rk, "k"), (rv, "v")):
        assert torch.equal(got.cpu().double(), dr.quantise(d[x].cpu().double())[0])
    assert n < 300 and k[:, :at].max() == 0 and v[:, :at].max() == 0


# ------------------------------------------------------------------ refusals
@pytest.mark.parametrize("new", [1, 130])
def test_bad_pages_are_reported_and_never_used(aa, new):
    d = dr.make_batch8(1, [new + 60, 40], [new, 1], 4, 2, 64, 16, device="cuda")
    for bad in (-1, d["P"], 2 ** 31 - 1, -2 ** 31):
        t = d["table"].clone()
        t[0, 1] = bad
        with _cache(aa, d, 16, 2, 64) as c:
            o = c.attend(d["q"], t, d["cu"], d["kv"], new)
            assert torch.isfinite(o.float()).all()
            with pytest.raises(aa.AAError):
                c.check_device_error()
            before = [d[x].view(torch.uint8).clone() for x in ("k_pages", "v_pages", "k_scales", "v_scales")]
            t[0].fill_(bad)
            c.append(d["k"][:new], d["v"][:new], t[:1], d["cu"][:2], d["kv"][:1])
            with pytest.raises(aa.AAError):
                c.check_device_error()
            for x, y in zip(("k_pages", "v_pages", "k_scales", "v_scales"), before):
                assert torch.equal(d[x].view(torch.uint8), y)


def test_refusals(aa):
    d = dr.make_batch8(1, [30], [2], 4, 2, 64, 16, device="cuda")
    pool = {x: d[x] for x in ("k_pages", "v_pages", "k_scales", "v_scales")}
    make = lambda **k: aa.PagedCache(d["P"], 16, 2, 64, **(pool | k))  # noqa: E731
    for wrong in (dict(k_scales=None), dict(k_scales=None, v_scales=None), dict(k_pages=d["kd"], v_pages=d["vd"]),
                  dict(k_scales=d["k_scales"].view(torch.uint8)), dict(v_scales=d["v_scales"][:, :-1]),
                  dict(v_pages=d["vd"]), dict(dtype=torch.float16), dict(dtype=torch.bfloat16),
                  dict(k_scales=d["k_scales"].cpu()), dict(k_pages=None, v_pages=None)):
        with pytest.raises((ValueError, aa.AAError)):
            make(**wrong)
    with pytest.raises(aa.AAError):
        make(v_pages=d["k_pages"])
    with pytest.raises(aa.AAError):
        make(v_scales=d["k_scales"])
    with make() as c:
        for out_k in (torch.empty(2, 2, 64, device="cuda"), torch.empty(2, 2, 64, dtype=torch.bfloat16),
                      torch.empty(3, 2, 64, dtype=torch.bfloat16, device="cuda")):
            with pytest.raises(ValueError):
                c.read(d["table"], d["cu"], d["kv"], 2, out_k=out_k)
        with pytest.raises(ValueError):
            c.read(d["table"], d["cu"], d["kv"], -1)
        with pytest.raises(aa.AAError):
            c.read(d["table"], d["cu"], d["kv"], 2, layer=1)
        both = torch.empty(2, 2, 64, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(aa.AAError):
            c.read(d["table"], d["cu"], d["kv"], 2, out_k=both, out_v=both)
        scales = d["k_scales"].view(torch.uint8).view(-1)
        with pytest.raises(aa.AAError, match="scales"):  # a result that lies among the scales
            c.attend(d["q"], d["table"], d["cu"], d["kv"], 2, lse=scales[:32].view(torch.float32).view(4, 2))
