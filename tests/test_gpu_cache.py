"""GPU: the paged cache (append, attend, copy_pages and the whole run of them) against plain 64-bit definitions, element
by element: every page size, head layout and length at which a tile, a page or a mask can go wrong."""
import ctypes
import math

import pytest
import torch

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
    return aa.PagedCache(d["P"], ps, Hkv, D, num_layers=d["k_pages"].shape[0], k_pages=d["k_pages"], v_pages=d["v_pages"], **kw)


def _attend(aa, d, ps, Hkv, D, tag="", layer=0, **kw):
    with _cache(aa, d, ps, Hkv, D) as c:
        o, lse = c.attend(d["q"], d["table"], d["cu"], d["kv"], d["max_q"], layer=layer, return_lse=True, **kw)
        torch.cuda.synchronize()
        c.check_device_error()
    want = ref.attend(d["q"], d["k_pages"], d["v_pages"], d["table"], d["cu"], d["kv"], layer, kw.get("key_lo"),
                      kw.get("anchor", False), kw.get("softmax_scale"))
    ref.check_attend(o, lse, want, tag=tag)
    return o, lse


# ------------------------------------------------------------------ attend: single tokens
LENGTHS = [0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 513]


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 2), (7, 1), (16, 1), (20, 4)])
def test_single_tokens(aa, ps, D, Hq, Hkv):
    d = ref.make_batch(ps + D + Hq, LENGTHS, [1] * len(LENGTHS), Hq, Hkv, D, ps, device="cuda")
    _attend(aa, d, ps, Hkv, D)


@pytest.mark.parametrize("Hq,Hkv", [(32, 1), (64, 1), (33, 1), (17, 1), (100, 2)])
def test_single_tokens_many_heads_per_group(aa, Hq, Hkv):
    d = ref.make_batch(Hq, [1, 64, 300, 1030], [1] * 4, Hq, Hkv, 128, 64, device="cuda")
    _attend(aa, d, 64, Hkv, 128)


@pytest.mark.parametrize("kv,B", [(9000, 1), (4097, 3), (70000, 1)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 64)])
def test_single_tokens_over_long_contexts(aa, kv, B, Hq, Hkv, D):
    lens = [max(kv // (b + 1), 1) for b in range(B)]
    d = ref.make_batch(kv, lens, [1] * B, Hq, Hkv, D, 32, device="cuda")
    _attend(aa, d, 32, Hkv, D)


@pytest.mark.parametrize("anchor", [False, True])
def test_single_tokens_masks(aa, anchor):
    """Windows that start inside a tile, at its border and past the end (an empty row), with and without the anchor."""
    kv = [1, 5, 64, 65, 130, 300, 300, 300, 300, 1000, 0, 2000]
    lo = [0, -4, 63, 64, 128, 299, 300, 10 ** 9, -2 ** 31, 937, 0, 1]
    for Hq, Hkv, ps, D in ((8, 2, 16, 128), (4, 4, 64, 64)):
        d = ref.make_batch(11, kv, [1] * len(kv), Hq, Hkv, D, ps, device="cuda")
        o, lse = _attend(aa, d, ps, Hkv, D, key_lo=torch.tensor(lo, dtype=torch.int32, device="cuda"), anchor=anchor)
        empty = [10] + ([] if anchor else [6, 7])
        assert (o[empty] == 0).all() and (lse[:, empty] == -math.inf).all()


# ------------------------------------------------------------------ attend: chunks
CHUNKS = [  # new tokens, tokens held
    ([1, 2, 5, 17], [1, 2, 100, 64]),
    ([0, 3, 0, 0, 40, 0], [50, 3, 0, 7, 333, 1]),
    ([130, 1, 257], [130, 700, 1000]),
    ([33, 16, 64], [33, 1500, 65]),
    ([500], [1300]),
]


@pytest.mark.parametrize("chunk", range(len(CHUNKS)))
@pytest.mark.parametrize("ps", [16, 128])
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 64), (8, 2, 128), (6, 2, 128), (7, 1, 64), (16, 1, 128)])
def test_chunks(aa, chunk, ps, Hq, Hkv, D):
    new, kv = CHUNKS[chunk]
    d = ref.make_batch(chunk, kv, new, Hq, Hkv, D, ps, device="cuda")
    _attend(aa, d, ps, Hkv, D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [2, 40])
@pytest.mark.parametrize("most", [500, 1500])
def test_up_to_64_rows(aa, D, B, most):
    """Rows where the choice of kernel depends on the head size, the batch and the contexts."""
    for new in (8, 9, 13, 16):
        kv = [max(new, most - 37 * b % most) for b in range(B)]
        d = ref.make_batch(new + B, kv, [new - b % 3 for b in range(B)], 8, 2, D, 32, device="cuda")
        _attend(aa, d, 32, 2, D)


@pytest.mark.parametrize("Hq,Hkv", [(64, 1), (45, 1), (33, 1), (10, 2)])
@pytest.mark.parametrize("ps", [32, 64])
def test_chunks_many_heads_per_group(aa, Hq, Hkv, ps):
    d = ref.make_batch(5, [50, 400], [9, 131], Hq, Hkv, 128, ps, device="cuda")
    _attend(aa, d, ps, Hkv, 128)


@pytest.mark.parametrize("anchor", [False, True])
@pytest.mark.parametrize("new", [3, 70, 300])
def test_chunk_masks(aa, anchor, new):
    """Packed documents, a sliding window, and rows that see nothing in between."""
    kv = [new, new + 41, new + 700]
    T = 3 * new
    p = torch.cat([torch.arange(k - new, k) for k in kv])
    docs = torch.where(p > 0, 1 + torch.div(p - 1, 90, rounding_mode="floor") * 90, torch.zeros_like(p))
    window = (p - 33).clamp(min=-5)
    g = torch.Generator().manual_seed(4)
    mixed = torch.where(torch.rand(T, generator=g) < 0.2, p + 1 + torch.randint(0, 3, (T,), generator=g),
                        (p * torch.rand(T, generator=g)).long())
    for name, lo in (("docs", docs), ("window", window), ("mixed", mixed)):
        for Hq, Hkv, D, ps in ((4, 1, 128, 32), (2, 2, 64, 128)):
            d = ref.make_batch(new, kv, [new] * 3, Hq, Hkv, D, ps, device="cuda")
            _attend(aa, d, ps, Hkv, D, tag=name, key_lo=lo.to(torch.int32).cuda(), anchor=anchor)


def test_fewer_tokens_held_than_new(aa):
    """kv_len below the number of new tokens: the first rows have no position and see nothing."""
    d = ref.make_batch(3, [4, 0, 300], [10, 6, 301], 4, 2, 64, 16, device="cuda")
    for anchor in (False, True):
        o, lse = _attend(aa, d, 16, 2, 64, anchor=anchor)
        assert (o[:6] == 0).all() and (lse[:, 10:17] == -math.inf).all()


@pytest.mark.parametrize("max_q", [0, 1, 4, 1000])
def test_max_q_is_a_hint(aa, max_q):
    d = ref.make_batch(8, [60, 500, 129], [1, 150, 40], 8, 2, 128, 64, device="cuda") | {"max_q": max_q}
    _attend(aa, d, 64, 2, 128)


def test_long_chunk_over_long_context(aa):
    d = ref.make_batch(21, [6000], [700], 4, 1, 128, 64, device="cuda")
    _attend(aa, d, 64, 1, 128)


# ------------------------------------------------------------------ attend: values, layouts, streams
@pytest.mark.parametrize("new,kv,Hq,Hkv,D", [(17, 52000, 8, 1, 128), (5, 70000, 16, 1, 64), (40, 20000, 8, 1, 64),
                                              (33, 2200, 8, 2, 128), (130, 9000, 16, 2, 128), (300, 5000, 4, 4, 64)])
def test_few_units_with_many_parts(aa, new, kv, Hq, Hkv, D):
    """Long contexts of one or two sequences: a unit's keys are split among many CTAs."""
    for lens, n in (([kv], [new]), ([kv, kv // 3], [new, new // 2])):
        d = ref.make_batch(new, lens, n, Hq, Hkv, D, 64, device="cuda")
        _attend(aa, d, 64, Hkv, D)
        lo = torch.full((sum(n),), kv // 5, dtype=torch.int32, device="cuda")
        lo[::7] = kv  # rows that see nothing but the anchor
        for anchor in (False, True):
            _attend(aa, d, 64, Hkv, D, key_lo=lo, anchor=anchor)


@pytest.mark.parametrize("new", [1, 4, 200])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_what_no_row_sees_does_not_reach_the_result(aa, new, bad):
    """NaN and infinities in unused pages, behind the last token of a page, and in front of every row's window."""
    kv, ps, Hq, Hkv, D = [new + 70, new + 333, new], 32, 4, 2, 128
    d = ref.make_batch(new, kv, [new] * 3, Hq, Hkv, D, ps, device="cuda")
    first = [40, 300, 0]
    lo = torch.cat([torch.full((new,), x) for x in first]).to(torch.int32).cuda()
    for pages in (d["k_pages"], d["v_pages"]):
        seen = torch.zeros(d["P"], ps, dtype=torch.bool, device="cuda")
        for b in range(3):
            j = torch.arange(first[b], kv[b])
            seen[d["table"][b].cpu()[j // ps].long(), j % ps] = True
        pages.masked_fill_(~seen[None, :, None, :, None], bad)
    o, _ = _attend(aa, d, ps, Hkv, D, key_lo=lo)
    assert torch.isfinite(o.float()).all()


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("wide", [1, 90])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_chunks_that_see_only_the_anchor(aa, ps, wide, bad):
    """Every row's first key lies behind its position, in the page of the last one: of that page, and of the anchor's, no
    row sees anything but key 0."""
    for kv, new, Hq, D in ((6, 6, 16, 128), (100, 40, 4, 128), (100, 90, 2, 64), (127, 40, 4, 64), (300, 40, 4, 128)):
        d = ref.make_batch(kv, [kv], [new], Hq, 1, D, ps, device="cuda", extra_width=wide)
        for pages in (d["k_pages"], d["v_pages"]):
            first = pages[0, d["table"][0, 0], 0, 0].clone()
            pages.fill_(bad)
            pages[0, d["table"][0, 0], 0, 0] = first
        for lo in {kv, -(-(kv + 1) // ps) * ps - 1, kv + 1000}:
            key_lo = torch.full((new,), lo, dtype=torch.int32, device="cuda")
            o, _ = _attend(aa, d, ps, 1, D, key_lo=key_lo, anchor=True)
            # one key of weight 1
            assert torch.equal(o, d["v_pages"][0, d["table"][0, 0], 0, 0].expand_as(o))


def test_large_logits_and_scales(aa):
    for new in (1, 150):
        for scale in (0.5, 4.0):
            d = ref.make_batch(6, [new + 400], [new], 4, 2, 64, 64, device="cuda")
            _attend(aa, d, 64, 2, 64, softmax_scale=scale)


@pytest.mark.parametrize("new,Hq,Hkv,D,ps", [(5, 8, 2, 128, 16), (16, 4, 4, 64, 64), (15, 4, 1, 64, 32), (40, 4, 1, 128, 64),
                                             (90, 14, 2, 128, 16), (300, 2, 2, 64, 128)])
@pytest.mark.parametrize("anchor", [False, True])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_rows_that_see_nothing_hide_their_own_keys(aa, new, Hq, Hkv, D, ps, anchor, bad):
    """Rows whose first key lies behind their position leave keys between seen ones that no row sees: behind the last row
    that sees any, in front of the first, and in between. NaN and infinities there stay out of the result."""
    g = torch.Generator().manual_seed(new)
    for held in (0, 77, 1500):
        kv = held + new
        p = torch.arange(held, kv)
        tail, middle, front = torch.zeros(new, dtype=torch.long), p - 3, p.clone()
        tail[new * 2 // 3:] = 1 << 30
        middle[new // 4:new // 2] = kv + 5
        front[:new // 3] = held + new // 3 + 1
        some = torch.where(torch.rand(new, generator=g) < 0.4, p + 1 + torch.randint(0, 4, (new,), generator=g), p - 1)
        for name, lo in (("tail", tail), ("middle", middle), ("front", front), ("some", some)):
            d = ref.make_batch(new, [kv, 40], [new, 1], Hq, Hkv, D, ps, device="cuda")
            j = torch.arange(kv)
            seen = ((j >= lo[:, None]) & (j <= p[:, None])).any(0)
            seen[0] |= anchor
            hidden = j[~seen]
            for pages in (d["k_pages"], d["v_pages"]):
                pages[0, d["table"][0].cpu()[hidden // ps].long().cuda(), :, (hidden % ps).cuda()] = bad
            key_lo = torch.cat([lo, torch.zeros(1, dtype=torch.long)]).to(torch.int32).cuda()
            o, _ = _attend(aa, d, ps, Hkv, D, tag=f"{name} {held}", key_lo=key_lo, anchor=anchor)
            assert torch.isfinite(o.float()).all()


@pytest.mark.parametrize("logit", [2e4, 5e4, -2e4, -5e4])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,kv", [(1, 500), (1, 20000), (120, 500), (120, 3500)])
def test_logits_of_tens_of_thousands(aa, logit, D, new, kv):
    """Maxima far from 0 on both sides: a row's base has to be within a few units of its maximum, whatever its size.
    Both kernels, with whole and with cut units; the rows' logits differ by some tens."""
    d = ref.make_batch(kv, [kv], [new], 4, 2, D, 64, device="cuda")
    a = math.sqrt(abs(logit) / math.sqrt(D))
    g = torch.Generator().manual_seed(7)
    rows = a * (1.0 + 0.2 * torch.rand(d["q"].shape[:2] + (1,), generator=g)).cuda()
    d["q"].copy_(rows + 0.1 * d["q"])
    d["k_pages"].copy_(math.copysign(a, logit) + 0.3 * d["k_pages"])
    o, lse = _attend(aa, d, 64, 2, D)
    assert torch.isfinite(lse).all() and (o.float().abs().amax(-1) > 0).all()


def test_values_far_apart(aa):
    """One key far above the others, first, in the middle or last; and logits of -inf from infinite keys."""
    for new in (1, 130):
        for at in (0, 150, 299):
            d = ref.make_batch(at, [300], [new], 2, 1, 64, 16, device="cuda")
            page = int(d["table"][0, at // 16])
            d["k_pages"][0, page, 0, at % 16] = d["q"][-1, 0] * 4
            _attend(aa, d, 16, 1, 64)
    for new in (1, 130):
        d = ref.make_batch(2, [300], [new], 2, 2, 64, 16, device="cuda")
        d["q"].abs_()
        page = int(d["table"][0, 3])
        d["k_pages"][0, page, 0, 5, 7] = -math.inf
        with _cache(aa, d, 16, 2, 64) as c:
            o, lse = c.attend(d["q"], d["table"], d["cu"], d["kv"], new, return_lse=True)
            d["k_pages"][0, page, 0, 5, 7] = -3e38
            o2, lse2 = c.attend(d["q"], d["table"], d["cu"], d["kv"], new, return_lse=True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("new,kv", [(1, 500), (1, 20000), (4, 300), (100, 300), (100, 3000)])
def test_nan_in_a_visible_key_shows(aa, new, kv):
    """A NaN in a key makes every row that sees it NaN (never 0), and no row of another sequence."""
    d = ref.make_batch(3, [kv, kv], [new, new], 4, 2, 64, 64, device="cuda")
    at = kv - new // 2 - 1  # seen by the later half of the new tokens
    d["k_pages"][0, int(d["table"][1, at // 64]), 1, at % 64, 3] = math.nan
    with _cache(aa, d, 64, 2, 64) as c:
        o, lse = c.attend(d["q"], d["table"], d["cu"], d["kv"], new, return_lse=True)
        c.check_device_error()
    sees = torch.zeros(2 * new, 4, dtype=torch.bool)
    sees[new + at - (kv - new):, 2:] = True
    assert torch.isnan(lse.T.cpu()).equal(sees)
    assert torch.isnan(o.cpu()).all(-1).equal(sees) and torch.isnan(o.cpu()).any(-1).equal(sees)


@pytest.mark.parametrize("page_tokens", [16, 128])
def test_mixed_batch_of_many_sequences(aa, page_tokens):
    """Hundreds of sequences, most idle or with one token, some with chunks: the kernel for chunks, whole units and cut ones."""
    g = torch.Generator().manual_seed(8)
    pick = torch.randint(0, 10, (300,), generator=g).tolist()
    new = [0 if x < 4 else 1 if x < 9 else 50 + i % 97 for i, x in enumerate(pick)]
    kv = [n + int(x) for n, x in zip(new, torch.randint(0, 90, (300,), generator=g))]
    d = ref.make_batch(8, kv, new, 4, 1, 64, page_tokens, device="cuda")
    _attend(aa, d, page_tokens, 1, 64)
    kv[7] += 2500  # one long context: wide tables, units are cut
    d = ref.make_batch(8, kv, new, 4, 1, 64, page_tokens, device="cuda")
    _attend(aa, d, page_tokens, 1, 64)


@pytest.mark.parametrize("group", [1, 4, 16])
def test_chunks_with_wide_tables(aa, group):
    """Short and long contexts in one batch under tables of 4096 keys: pieces of units on many SMs."""
    d = ref.make_batch(group, [3900, 64, 5, 1000], [80, 64, 5, 300], 2 * group, 2, 128, 32, device="cuda", extra_width=6)
    _attend(aa, d, 32, 2, 128)


def test_strides_layers_and_rows_behind_the_batch(aa):
    for new in (1, 90):
        T, pad, Hq, Hkv, D, ps = 2 * new, 5, 4, 2, 128, 64
        d = ref.make_batch(new, [new + 50, new + 9], [new, new], Hq, Hkv, D, ps, layers=3, pad=pad, device="cuda")
        joint = torch.randn(T + pad, Hq + 2 * Hkv, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
        joint[:, :Hq] = d["q"]
        out = torch.full((T + pad, Hq, D), 7.0, device="cuda", dtype=torch.bfloat16)
        lse = torch.full((Hq, T + pad), 7.0, device="cuda")
        with _cache(aa, d, ps, Hkv, D) as c:
            o, _ = c.attend(joint[:, :Hq], d["table"], d["cu"], d["kv"], new, layer=2, out=out, lse=lse, return_lse=True)
            assert o is out and (out[T:] == 7).all() and (lse[:, T:] == 7).all()
            want = ref.attend(d["q"], d["k_pages"], d["v_pages"], d["table"], d["cu"], d["kv"], 2)
            ref.check_attend(out, lse, want)
            # without the log-sum-exp, the same bits
            assert torch.equal(c.attend(joint[:, :Hq], d["table"], d["cu"], d["kv"], new, layer=2)[:T], out[:T])
            c.check_device_error()


def test_calls_of_whole_units_need_no_workspace(aa):
    """Tables of at most 768 keys: a unit's keys are never split, so there is nothing to keep; above, there is."""
    for ps in (16, 64, 128):
        W = 768 // ps
        d = ref.make_batch(ps, [700, 300, 90], [90, 40, 90], 8, 2, 128, ps, device="cuda", extra_width=0)
        table = torch.nn.functional.pad(d["table"], (0, W - d["table"].shape[1]), value=-1)
        with _cache(aa, d, ps, 2, 128) as c:
            assert c.workspace_bytes(3, d["T"], 90, W, 8) == 256
            assert c.workspace_bytes(3, d["T"], 90, W + 1, 8) > 1 << 20
            work = torch.zeros(256, dtype=torch.uint8, device="cuda")
            got = c.attend(d["q"], table, d["cu"], d["kv"], 90, workspace=work, return_lse=True)
            c.check_device_error()
            assert (work == 0).all()
            wide = torch.nn.functional.pad(table, (0, 1), value=-1)
            with pytest.raises(aa.AAError, match="workspace"):
                c.attend(d["q"], wide, d["cu"], d["kv"], 90, workspace=work)
        want = ref.attend(d["q"], d["k_pages"], d["v_pages"], d["table"], d["cu"], d["kv"])
        ref.check_attend(*got, want)


def test_batches_of_nothing(aa):
    d = ref.make_batch(1, [5, 0], [0, 0], 2, 1, 64, 16, pad=3, device="cuda")
    out = torch.full_like(d["q"], 7.0)
    with _cache(aa, d, 16, 1, 64) as c:
        c.attend(d["q"], d["table"], d["cu"], d["kv"], 0, out=out)
        assert (out == 7).all()
        assert c.attend(d["q"][:0], d["table"], d["cu"], d["kv"], 0).shape == (0, 2, 64)
        c.append(d["k"][:0], d["v"][:0], d["table"], d["cu"], d["kv"])
        before = d["k_pages"].clone()
        c.append(d["k"], d["v"], d["table"], d["cu"], d["kv"])
        c.check_device_error()
        assert torch.equal(before, d["k_pages"])


def test_append_of_no_tokens_with_queries(aa):
    d = ref.make_batch(1, [5, 0], [0, 0], 2, 1, 64, 16, pad=3, device="cuda")
    rope, pos = aa.RopeAxes(64, (32,)), torch.zeros(1, 0, dtype=torch.int32, device="cuda")
    with _cache(aa, d, 16, 1, 64) as c:
        q = c.append(d["k"][:0], d["v"][:0], d["table"], d["cu"], d["kv"], rope=rope, pos=pos, q=d["q"][:0])
        assert q.shape == (0, 2, 64)
        c.check_device_error()


def test_runs_agree_bit_for_bit_and_across_streams(aa):
    for new, kv in ((1, [3000, 17]), (5, [900, 40]), (160, [2000, 160])):
        d = ref.make_batch(4, kv, [new, new], 8, 2, 128, 64, device="cuda")
        with _cache(aa, d, 64, 2, 128) as c:
            want = c.attend(d["q"], d["table"], d["cu"], d["kv"], new)
            streams = [torch.cuda.Stream() for _ in range(2)]
            for s in streams:
                s.wait_stream(torch.cuda.current_stream())
            got = [c.attend(d["q"], d["table"], d["cu"], d["kv"], new, stream=s) for s in streams for _ in range(3)]
            torch.cuda.synchronize()
            assert all(torch.equal(x, want) for x in got)


@pytest.mark.parametrize("Hq,Hkv,D", [(6, 2, 128), (14, 2, 128), (5, 1, 64), (7, 1, 64)])
def test_rows_that_hold_no_token_change_nothing(aa, Hq, Hkv, D):
    """Groups that do not divide 128 leave rows of a tile without a token, over whatever shared memory holds: the same
    call after calls with other queries, which leave small and large values there, gives the same bits."""
    ps = 64
    for kv in (700, 2600):  # whole units; cut ones
        d = ref.make_batch(Hq, [kv] * 12, [80] * 12, Hq, Hkv, D, ps, device="cuda", extra_width=0)
        n = 160 * 256
        q = torch.randn(n, Hkv, D, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
        table = d["table"][:1].expand(160, -1).contiguous()
        cu = torch.arange(0, n + 1, 256, dtype=torch.int32, device="cuda")
        length = torch.full((160,), 256, dtype=torch.int32, device="cuda")
        with _cache(aa, d, ps, Hkv, D) as c:
            got = []
            for times in (0.0, 1.0, 30.0, 1000.0):
                c.attend(q * times, table, cu, length, 256)
                got.append(c.attend(d["q"], d["table"], d["cu"], d["kv"], 80, return_lse=True))
            torch.cuda.synchronize()
            c.check_device_error()
        assert all(torch.equal(x[0], got[0][0]) and torch.equal(x[1], got[0][1]) for x in got)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (6, 2, 128), (4, 4, 64)])
def test_a_sequence_does_not_depend_on_the_next_ones_queries(aa, Hq, Hkv, D):
    """The rows behind a sequence's last token hold the next sequence's queries: the first one's bits are the same
    whatever those are, and without them."""
    ps, new = 64, 300 // (Hq // Hkv) - 7
    d = ref.make_batch(Hq, [700, 700], [new, new], Hq, Hkv, D, ps, device="cuda", extra_width=0)
    with _cache(aa, d, ps, Hkv, D) as c:
        want = c.attend(d["q"][:new], d["table"][:1], d["cu"][:2], d["kv"][:1], new, return_lse=True)
        for times in (1.0, 30.0, 1000.0):
            q = d["q"].clone()
            q[new:] *= times
            o, lse = c.attend(q, d["table"], d["cu"], d["kv"], new, return_lse=True)
            assert torch.equal(o[:new], want[0]) and torch.equal(lse[:, :new], want[1])
        c.check_device_error()


def test_graph_replay_follows_lengths_and_tables(aa):
    for new in (1, 100):
        Hq, Hkv, D, ps = 8, 2, 128, 32
        d = ref.make_batch(9, [new + 900, new + 31], [new, new], Hq, Hkv, D, ps, device="cuda")
        rope = aa.RopeAxes(D, (64,), base=1e4, layout=aa.ROPE_HALF)
        pos = torch.zeros(1, d["T"], dtype=torch.int32, device="cuda")
        with _cache(aa, d, ps, Hkv, D) as c:
            ws = c.alloc_workspace(2, d["T"], new, d["table"].shape[1], Hq)

            def step():
                q = c.append(d["k"], d["v"], d["table"], d["cu"], d["kv"], rope=rope, pos=pos, q=d["q"])
                return q, c.attend(q, d["table"], d["cu"], d["kv"], new, workspace=ws)
            step()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                q, o = step()
            for kv in ([new + 3, new + 30], [new + 500, new + 1]):
                d["kv"].copy_(torch.tensor(kv, dtype=torch.int32))
                pos.copy_(torch.cat([torch.arange(k - new, k) for k in kv])[None])
                d["table"].copy_(d["table"].flip(0))  # there and back
                graph.replay()
                torch.cuda.synchronize()
                c.check_device_error()
                want = ref.attend(q, d["k_pages"], d["v_pages"], d["table"].clamp(min=0), d["cu"], d["kv"])
                ref.check_attend(o, want[1], want)
                eq, eo = step()
                assert torch.equal(eq, q) and torch.equal(eo, o)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("D,half", [(64, False), (64, True), (128, False), (128, True)])
def test_append_writes_the_new_rows_and_nothing_else(aa, ps, D, half):
    new, kv = [1, 0, 40, 3, 129], [1, 77, 40, 130, 400]
    Hq, Hkv = 6, 3
    d = ref.make_batch(ps, kv, new, Hq, Hkv, D, ps, layers=2, pad=2, device="cuda")
    T = d["T"] - 2
    sections = (D // 8, D // 8, D // 4)
    rope = aa.RopeAxes(D, sections, base=5e5, layout=aa.ROPE_HALF if half else aa.ROPE_ADJACENT)
    theta = [5e5 ** (-2.0 * p / D) for p in range(D // 2)]
    pos = torch.randint(0, 100000, (3, T + 2), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    k0, v0 = d["k_pages"].clone(), d["v_pages"].clone()
    with _cache(aa, d, ps, Hkv, D) as c:
        out = torch.full_like(d["q"], 7.0)
        got = c.append(d["k"], d["v"], d["table"], d["cu"], d["kv"], layer=1, rope=rope, pos=pos, q=d["q"], out_q=out)
        torch.cuda.synchronize()
        c.check_device_error()
    assert got is out and (out[T:] == 7).all()
    want = ref.turn(d["q"], pos, rope.axis_of_pair, theta, half)
    assert ((out[:T].double().cpu() - want[:T]).abs() <= ref.turn_bound(want, d["q"], half)[:T]).all()
    want, bound = ref.turn(d["k"], pos, rope.axis_of_pair, theta, half), None
    bound = ref.turn_bound(want, d["k"], half)
    k1, v1, t = d["k_pages"].cpu(), d["v_pages"].cpu(), 0
    for b, n in enumerate(new):
        for i in range(n):
            p = kv[b] - n + i
            page, slot = int(d["table"][b, p // ps]), p % ps
            assert ((k1[1, page, :, slot].double() - want[t]).abs() <= bound[t]).all()
            assert torch.equal(v1[1, page, :, slot], d["v"][t].cpu())
            k0[1, page, :, slot], v0[1, page, :, slot] = d["k_pages"][1, page, :, slot], d["v_pages"][1, page, :, slot]
            t += 1
    assert torch.equal(d["k_pages"], k0) and torch.equal(d["v_pages"], v0)


def test_append_without_rotation_and_from_slices(aa):
    new, kv, ps, Hkv, D = [30, 2], [50, 64], 32, 2, 128
    d = ref.make_batch(2, kv, new, 4, Hkv, D, ps, device="cuda")
    joint = torch.cat([d["q"], d["k"], d["v"]], dim=1)
    k, v = joint[:, 4:6], joint[:, 6:]
    with _cache(aa, d, ps, Hkv, D) as c:
        assert c.append(k, v, d["table"], d["cu"], d["kv"]) is None
        for b, t in ((0, 0), (1, 30)):
            got = ref.keys_of(d["k_pages"].cpu(), d["table"][b].cpu(), kv[b], 0, 1)[kv[b] - new[b]:]
            assert torch.equal(got, d["k"][t:t + new[b], 1].double().cpu())
        rope = aa.RopeAxes(D, (64,), base=1e4)
        pos = torch.arange(32, dtype=torch.int32, device="cuda")[None]
        yq = c.append(k, v, d["table"], d["cu"], d["kv"], rope=rope, pos=pos, q=joint[:, :4])
        assert torch.equal(yq, rope.apply(pos, d["q"]))
        assert torch.equal(ref.keys_of(d["k_pages"].cpu(), d["table"][0].cpu(), 50, 0, 0)[20:],
                           rope.apply(pos, d["k"])[:30, 0].double().cpu())
        c.check_device_error()


def test_append_many_sequences(aa):
    """More sequences than a warp looks at in one step, most without new tokens."""
    g = torch.Generator().manual_seed(3)
    new = [int(x) if x < 3 else 0 for x in torch.randint(0, 9, (2500,), generator=g)]
    kv = [n + int(x) for n, x in zip(new, torch.randint(0, 20, (2500,), generator=g))]
    d = ref.make_batch(3, kv, new, 1, 1, 64, 16, device="cuda")
    with _cache(aa, d, 16, 1, 64) as c:
        c.append(d["k"], d["v"], d["table"], d["cu"], d["kv"])
        c.check_device_error()
    table, pages, t = d["table"].cpu(), d["v_pages"].cpu(), 0
    for b, n in enumerate(new):
        for i in range(n):
            p = kv[b] - n + i
            assert torch.equal(pages[0, table[b, p // 16], 0, p % 16], d["v"][t, 0].cpu())
            t += 1
    _attend(aa, d, 16, 1, 64)


# ------------------------------------------------------------------ page copies
@pytest.mark.parametrize("n", [1, 3, 64, 65, 1100])
@pytest.mark.parametrize("ps,Hkv,D,L", [(16, 1, 64, 1), (32, 3, 128, 2)])
def test_copy_pages(aa, n, ps, Hkv, D, L):
    P = 2 * n + 5
    g = torch.Generator().manual_seed(n)
    d = {"k_pages": torch.randn(L, P, Hkv, ps, D, generator=g).to(torch.bfloat16).cuda(), "P": P}
    d["v_pages"] = -d["k_pages"]
    order = torch.randperm(P, generator=g).tolist()
    src, dst = order[:n], order[n:2 * n]
    want = d["k_pages"].clone()
    want[:, dst] = d["k_pages"][:, src]
    with _cache(aa, d, ps, Hkv, D) as c:
        c.copy_pages(src + [order[-1]], dst + [order[-1]])  # the last one onto itself: nothing
        torch.cuda.synchronize()
    assert torch.equal(d["k_pages"], want) and torch.equal(d["v_pages"], -want)


def test_copy_pages_refusals(aa):
    d = ref.make_batch(1, [100], [1], 1, 1, 64, 16, device="cuda")
    before = d["k_pages"].clone()
    with _cache(aa, d, 16, 1, 64) as c:
        P = d["P"]
        for src, dst, msg in (([0], [P], "page numbers"), ([-1], [0], "page numbers"), ([0, 1], [2, 2], "two pairs"),
                              ([0, 1], [1, 2], "both"), ([0, 1], [1, 1], "both")):
            with pytest.raises(aa.AAError) as e:
                c.copy_pages(src, dst)
            assert e.value.status == 1 and msg in str(e.value)
        with pytest.raises(ValueError):
            c.copy_pages([0, 1], [2])
        c.copy_pages([0, 0], [1, 2])  # one source for two targets is a fork of three
        torch.cuda.synchronize()
        assert torch.equal(d["k_pages"][:, 2], before[:, 0]) and torch.equal(d["k_pages"][:, 1], before[:, 0])


# ------------------------------------------------------------------ bad pages and refusals
@pytest.mark.parametrize("new", [1, 4, 200])
def test_bad_pages_are_reported_and_never_used(aa, new):
    kv, ps, Hkv, D = [new + 100, new + 300], 16, 2, 64
    for bad in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
        d = ref.make_batch(1, kv, [new, new], 4, Hkv, D, ps, device="cuda")
        d["table"][1, 2] = bad
        with _cache(aa, d, ps, Hkv, D) as c:
            o, lse = c.attend(d["q"], d["table"], d["cu"], d["kv"], new, return_lse=True)
            with pytest.raises(aa.AAError) as e:
                c.check_device_error()
            assert e.value.status == 1 and "page number" in str(e.value)
            c.check_device_error()  # cleared
            # the other sequence is whole
            want = ref.attend(d["q"][:new], d["k_pages"], d["v_pages"], d["table"][:1], d["cu"][:2], d["kv"][:1])
            ref.check_attend(o[:new], lse[:, :new], want)
            # append: the token on the bad page is skipped
            last = (kv[1] - 1) // ps
            d["table"][1, last] = bad
            k0 = d["k_pages"].clone()
            c.append(d["k"][-1:], d["v"][-1:], d["table"], torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda"), d["kv"])
            with pytest.raises(aa.AAError):
                c.check_device_error()
            assert torch.equal(k0, d["k_pages"])


def test_positions_outside_the_table(aa):
    for new in (1, 150):
        d = ref.make_batch(1, [new + 60], [new], 2, 1, 64, 16, extra_width=0, device="cuda")
        d["kv"] += 16 * 5
        with _cache(aa, d, 16, 1, 64) as c:
            c.attend(d["q"], d["table"], d["cu"], d["kv"], new)
            with pytest.raises(aa.AAError) as e:
                c.check_device_error()
            assert "position" in str(e.value)
            k0 = d["k_pages"].clone()
            c.append(d["k"][-1:], d["v"][-1:], d["table"], torch.tensor([0, 1], dtype=torch.int32, device="cuda"), d["kv"])
            with pytest.raises(aa.AAError):
                c.check_device_error()
            d["kv"].fill_(0)  # a new token at position -1
            c.append(d["k"][-1:], d["v"][-1:], d["table"], torch.tensor([0, 1], dtype=torch.int32, device="cuda"), d["kv"])
            with pytest.raises(aa.AAError):
                c.check_device_error()
            assert torch.equal(k0, d["k_pages"])


def test_refusals(aa):
    d = ref.make_batch(1, [20, 30], [2, 1], 4, 2, 64, 16, device="cuda")
    with _cache(aa, d, 16, 2, 64) as c:
        good = dict(q=d["q"], page_table=d["table"], cu_q=d["cu"], kv_len=d["kv"], max_q=2)
        out = torch.full_like(d["q"], 7.0)
        for change in (dict(q=d["q"].float()), dict(q=d["q"][..., :32]), dict(q=d["q"].cpu()), dict(page_table=d["table"].long()),
                       dict(page_table=d["table"][:, ::2]), dict(cu_q=d["cu"][1:]), dict(kv_len=d["kv"][:1]),
                       dict(kv_len=d["kv"].cpu()), dict(key_lo=torch.zeros(2, dtype=torch.int32, device="cuda")),
                       dict(out=out[1:]), dict(lse=torch.zeros(3, 4, device="cuda")),
                       dict(workspace=torch.zeros(4, device="cuda"))):
            with pytest.raises(ValueError):
                c.attend(**(good | change))
        for change, msg in ((dict(layer=1), "layer"), (dict(layer=-1), "layer"), (dict(max_q=-1), "max_q"),
                            (dict(q=d["q"][:, :3].contiguous()), "multiple"), (dict(softmax_scale=float("nan")), "scale"),
                            (dict(out=d["q"]), "overlaps"), (dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")), "workspace"),
                            (dict(q=torch.zeros(3, 130, 64, dtype=torch.bfloat16, device="cuda")), "at most 64")):
            with pytest.raises(aa.AAError) as e:
                c.attend(**((good if "q" in change else good | dict(out=out)) | change))
            assert msg in str(e.value), change
        rope, pos = aa.RopeAxes(64, (32,)), torch.zeros(1, 3, dtype=torch.int32, device="cuda")
        good = dict(k=d["k"], v=d["v"], page_table=d["table"], cu_q=d["cu"], kv_len=d["kv"])
        for change in (dict(k=d["k"].half()), dict(v=d["v"][1:]), dict(v=d["v"][:, :1]), dict(rope=rope), dict(pos=pos),
                       dict(q=d["q"]), dict(rope=rope, pos=pos[:, 1:]), dict(rope=rope, pos=pos, out_q=out),
                       dict(rope=rope, pos=pos, q=d["q"][1:])):
            with pytest.raises(ValueError):
                c.append(**(good | change))
        with pytest.raises(aa.AAError):
            c.append(**good, rope=aa.RopeAxes(128, (64,)), pos=pos)
        with pytest.raises(aa.AAError):
            c.append(**good, layer=3)
        c.check_device_error()
        # the library's own checks, past the binding's
        L, b = aa.lib(), aa.binding.AACacheBatch(d["table"].data_ptr(), d["cu"].data_ptr(), d["kv"].data_ptr(), 2, 3, 3, 0)
        for field, value in (("num_seqs", 0), ("table_width", 0), ("total_tokens", -1), ("page_table", None), ("cu_q", None),
                             ("kv_len", None), ("table_width", 1 << 27)):
            x = aa.binding.AACacheBatch.from_buffer_copy(b)
            setattr(x, field, value)
            assert L.aa_cache_append(c._h, ctypes.addressof(x), d["k"].data_ptr(), 128, d["v"].data_ptr(), 128, None, None,
                                     None, 0, None, 0, None) == 1
        torch.cuda.synchronize()
        assert (out == 7).all()


def test_results_written_into_given_tensors_are_seen_by_autograd(aa):
    d = ref.make_batch(1, [20, 30], [2, 1], 4, 2, 64, 16, device="cuda")
    rope, pos = aa.RopeAxes(64, (32,)), torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    with _cache(aa, d, 16, 2, 64) as c:
        append = lambda **kw: c.append(d["k"], d["v"], d["table"], d["cu"], d["kv"], rope=rope, pos=pos, q=d["q"], **kw)
        attend = lambda **kw: c.attend(d["q"], d["table"], d["cu"], d["kv"], 2, **kw)
        lse = torch.zeros(4, 3, device="cuda")
        for call, out in ((lambda x: append(out_q=x), torch.zeros_like(d["q"])), (lambda x: attend(out=x), torch.zeros_like(d["q"])),
                          (lambda x: attend(lse=x), lse)):
            leaf = out.requires_grad_(True)
            a = leaf * 1
            y = a * a  # saves a
            for x in (leaf, a):
                with pytest.raises(ValueError, match="grad"):
                    call(x)
            with torch.no_grad():
                call(a)
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                y.sum().backward()
        c.check_device_error()


def test_results_in_the_pool_are_refused(aa):
    d = ref.make_batch(2, [20, 30], [2, 1], 4, 2, 64, 16, device="cuda")
    rope, pos = aa.RopeAxes(64, (32,)), torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    with _cache(aa, d, 16, 2, 64) as c:
        good = dict(q=d["q"], page_table=d["table"], cu_q=d["cu"], kv_len=d["kv"], max_q=2)
        for pool in (c.k_pages, c.v_pages):
            before = pool.clone()
            inside = pool.reshape(-1)[-3 * 4 * 64:].view(3, 4, 64)
            lse = pool.reshape(-1)[:24].view(torch.float32).view(4, 3)
            for change in (dict(out=inside), dict(lse=lse)):
                with pytest.raises(aa.AAError, match="pages"):
                    c.attend(**(good | change))
            with pytest.raises(aa.AAError, match="pages"):
                c.append(d["k"], d["v"], d["table"], d["cu"], d["kv"], rope=rope, pos=pos, q=d["q"], out_q=inside)
            torch.cuda.synchronize()
            assert torch.equal(pool, before)
        c.check_device_error()


def test_results_that_overlap_are_refused(aa):
    """o, lse and the part of the workspace that is used: apart from one another, from q and key_lo, and from the pool.
    Nothing is launched."""
    T, Hq, D = 100, 4, 64
    d = ref.make_batch(2, [1300], [T], Hq, 2, D, 16, device="cuda")
    with _cache(aa, d, 16, 2, D) as c:
        W = d["table"].shape[1]
        need = c.workspace_bytes(1, T, T, W, Hq)
        arena = torch.full((need + (1 << 20),), 7, dtype=torch.uint8, device="cuda")
        o_bytes, lse_bytes = T * Hq * D * 2, T * Hq * 4
        o_at = lambda at: arena[at:at + o_bytes].view(torch.bfloat16).view(T, Hq, D)
        lse_at = lambda at: arena[at:at + lse_bytes].view(torch.float32).view(Hq, T)
        lo_at = lambda at: arena[at:at + 4 * T].view(torch.int32)
        before, pools = arena.clone(), [p.clone() for p in (c.k_pages, c.v_pages)]
        good = dict(q=d["q"], page_table=d["table"], cu_q=d["cu"], kv_len=d["kv"], max_q=T)
        tail = need // 256 * 256 + 256
        q = o_at(tail)
        for change in (dict(out=o_at(0), lse=lse_at(256)), dict(out=o_at(0), lse=lse_at(o_bytes - 16)),
                       dict(out=o_at(0), workspace=arena), dict(out=o_at(need - 256), workspace=arena),
                       dict(lse=lse_at(need - 256), workspace=arena), dict(lse=lse_at(tail), q=q),
                       dict(q=o_at(need - 256), workspace=arena), dict(key_lo=lo_at(need - 256), workspace=arena),
                       dict(key_lo=lo_at(tail), lse=lse_at(tail)), dict(key_lo=lo_at(tail), out=o_at(tail)),
                       dict(cu_q=lo_at(tail)[:2], lse=lse_at(tail)), dict(kv_len=lo_at(tail)[:1], out=o_at(tail)),
                       dict(page_table=lo_at(need - 256)[:W][None], workspace=arena)):
            with pytest.raises(aa.AAError, match="overlap"):
                c.attend(**(good | change))
        L, b = aa.lib(), aa.binding.AACacheBatch(d["table"].data_ptr(), d["cu"].data_ptr(), d["kv"].data_ptr(), 1, W, T, 0)
        out = torch.zeros_like(d["q"])
        for at in (c.k_pages.data_ptr(), c.v_pages.data_ptr() - need + 256):  # its first, its last bytes in the pool
            st = L.aa_cache_attend(c._h, ctypes.addressof(b), d["q"].data_ptr(), Hq * D, Hq, T, None, 0, 0.0, out.data_ptr(),
                                   None, at, need, None)
            assert st == 1 and "overlap" in L.aa_last_error().decode()
        torch.cuda.synchronize()
        assert torch.equal(arena, before) and torch.equal(c.k_pages, pools[0]) and torch.equal(c.v_pages, pools[1])
        # behind the bytes that the call needs an arena may hold the results
        o, lse = c.attend(**good, out=o_at(tail), lse=lse_at(tail + o_bytes), workspace=arena, return_lse=True)
        c.check_device_error()
        ref.check_attend(o, lse, ref.attend(d["q"], *pools, d["table"], d["cu"], d["kv"]))


# ------------------------------------------------------------------ the run of them together
def test_serving_run_against_the_packed_forward(aa):
    """A packed sequence of documents is prefilled in chunks and then continued token by token through the cache, with
    pages forked, compacted and freed on the way; every output is the packed forward's (Plan.fwd on the same tokens), which
    shares no code with it, within both bounds."""
    import oracle as orc
    from gpu_common import f64, inputs, problem
    docs = [70, 150, 201]
    T, Hq, Hkv, D, ps = 1 + sum(docs), 8, 2, 128, 16
    cu = [1]
    for n in docs:
        cu.append(cu[-1] + n)
    q, k, v, _ = inputs(T, Hq, Hkv, D, seed=91)
    with aa.Plan(cu, T, Hq, Hkv, D, 5e5, rope_layout=aa.ROPE_HALF) as plan:
        packed, lse_packed = plan.fwd(q, k, v)
        doc, position = plan.metadata()
        torch.cuda.synchronize()
        plan.check_device_error()
    O, LSE = orc.forward(problem(cu, T, Hq, Hkv, D, 5e5, layout=orc.ROPE_HALF), q.cpu(), k.cpu(), v.cpu())
    pos = torch.from_numpy(position).cuda()[None]
    lo = torch.tensor([0] + [cu[x - 1] for x in doc[1:]], dtype=torch.int32, device="cuda")
    rope = aa.RopeAxes(D, (64,), base=5e5, layout=aa.ROPE_HALF)
    o, lse = torch.zeros_like(q), torch.zeros_like(lse_packed)
    cuts = [0, 100, 101, 230, 400] + list(range(401, T + 1))
    with aa.PagedCache(64, ps, Hkv, D, num_layers=2, max_seqs=4) as c:
        c.k_pages.fill_(math.nan), c.v_pages.fill_(math.nan)
        c.resize([3], [90])  # pages of another sequence in front
        seq = 0
        for a, b in zip(cuts, cuts[1:]):
            c.resize([seq], [b])
            table, kv = c.tables([seq], width=40, device="cuda")
            at = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
            rq = c.append(k[a:b], v[a:b], table, at, kv, layer=1, rope=rope, pos=pos[:, a:b].contiguous(), q=q[a:b])
            o[a:b], lse[:, a:b] = c.attend(rq, table, at, kv, b - a, layer=1, key_lo=lo[a:b].contiguous(), anchor=True,
                                           return_lse=True)
            if b == 230:  # go on in a fork; the first sequence is given up
                c.fork(0, 1)
                seq = 1
            elif b == 400:
                c.free([0, 3])
            elif b == 405:
                assert c.compact() > 0
            elif b == 410:  # two rejected tokens, written again
                c.fork(1, 2)
                c.resize([2], [408])
                c.resize([2], [410])
                t2, kv2 = c.tables([2], width=40, device="cuda")
                c.append(k[408:410] * 2, v[408:410] * 2, t2, torch.tensor([0, 2], dtype=torch.int32, device="cuda"), kv2, layer=1)
                c.free([2])
        torch.cuda.synchronize()
        c.check_device_error()
        assert c.stats()["free_pages"] == 64 - -(-T // ps)
    # the acceptance bounds of the packed forward (tests/gpu_common.py)
    err = abs(f64(o) - O)
    assert err.max() <= 2e-2 and err.mean() <= 2e-3
    assert abs(f64(lse) - LSE).max() <= 1e-2
    assert (o.double() - packed.double()).abs().max() <= 4e-2


def test_growing_a_fork_copies_its_page_on_the_device(aa):
    ps, Hkv, D = 16, 1, 64
    with aa.PagedCache(8, ps, Hkv, D, num_layers=3, max_seqs=3) as c:
        c.k_pages.normal_(), c.v_pages.normal_()
        c.resize([0], [20])
        c.fork(0, 1)
        c.resize([1], [21])
        a, b = c.tables([0])[0][0], c.tables([1])[0][0]
        torch.cuda.synchronize()
        assert a[0] == b[0] and a[1] != b[1]
        assert torch.equal(c.k_pages[:, a[1]], c.k_pages[:, b[1]]) and torch.equal(c.v_pages[:, a[1]], c.v_pages[:, b[1]])
        # while a stream is captured, a call that has to copy is refused and changes nothing
        c.fork(0, 2)
        x = torch.zeros(1, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            x += 1
            with pytest.raises(aa.AAError) as e:
                c.resize([2], [22])
            c.resize([1], [33])  # takes a page, copies nothing
        assert "captured" in str(e.value)
        assert (c.tables([2])[0] == c.tables([0])[0]).all() and c.tables([1])[1][0] == 33


def test_long_pool_offsets_pass_32_bits(aa):
    """A pool of more than 2^32 bytes and 2^31 elements: pages at its far end."""
    ps, Hkv, D, L = 128, 8, 128, 2
    P = 9000  # L * P * Hkv * ps * D = 2.36e9 elements
    k = torch.zeros(L, P, Hkv, ps, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    d = ref.make_batch(6, [300, 140], [1, 140], 16, Hkv, D, ps, device="cuda")
    far = torch.tensor([P - 1, P - 2, P - 3, P - 4, P - 5], device="cuda")
    table = torch.tensor([[P - 1, P - 2, P - 3], [P - 4, P - 5, -1]], dtype=torch.int32, device="cuda")
    used = [int(d["table"][b, w]) for b, n in ((0, 3), (1, 2)) for w in range(n)]
    k[1, far], v[1, far] = d["k_pages"][0, used], d["v_pages"][0, used]
    with aa.PagedCache(P, ps, Hkv, D, num_layers=L, k_pages=k, v_pages=v) as c:
        o, lse = c.attend(d["q"], table, d["cu"], d["kv"], 140, layer=1, return_lse=True)
        o1, lse1 = c.attend(d["q"][:1], table, torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda"), d["kv"], 1, layer=1,
                            return_lse=True)
        want = ref.attend(d["q"], d["k_pages"], d["v_pages"], d["table"], d["cu"], d["kv"])
        ref.check_attend(o, lse, want)
        ref.check_attend(o1, lse1, [x[:1] if x.dim() == 3 else x[:, :1] for x in want])
        c.append(d["k"][:1], d["v"][:1], table, torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda"), d["kv"], layer=1)
        c.copy_pages([P - 3], [5])
        torch.cuda.synchronize()
        c.check_device_error()
        assert torch.equal(v[1, P - 3, :, 299 % ps], d["v"][0]) and torch.equal(v[1, 5], v[1, P - 3])
        assert torch.equal(k[1, P - 3, :, 299 % ps], d["k"][0])
