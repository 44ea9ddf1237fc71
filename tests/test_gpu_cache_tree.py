"""GPU: drafted trees over the paged cache (masks and positions, attention, moving the accepted tokens) against plain
definitions, for 16-bit and 8-bit pages."""
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


def _batch(fp8, *a, **k):
    d = (dr.make_batch8 if fp8 else ref.make_batch)(*a, **k)
    if not fp8:
        d["kd"], d["vd"] = d["k_pages"], d["v_pages"]
    return d


def _cache(aa, d, ps, Hkv, D, **kw):
    pool = {x: d[x] for x in ("k_pages", "v_pages", "k_scales", "v_scales") if x in d}
    return aa.PagedCache(d["P"], ps, Hkv, D, num_layers=d["k_pages"].shape[0], **pool, **kw)


def _attend(aa, d, ps, Hkv, D, tree, tag="", layer=0, **kw):
    with _cache(aa, d, ps, Hkv, D) as c:
        o, lse = c.attend(d["q"], d["table"], d["cu"], d["kv"], d["max_q"], layer=layer, tree=tree, return_lse=True, **kw)
        torch.cuda.synchronize()
        c.check_device_error()
    want = dr.attend_tree(d["q"], d["kd"], d["vd"], d["table"], d["cu"], d["kv"], tree, layer, kw.get("key_lo"),
                          kw.get("anchor", False), kw.get("softmax_scale"))
    ref.check_attend(o, lse, want, tag=tag)
    return o, lse


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ masks
@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("new", [[1], [26], [64], [65, 0, 1, 128], [3] * 90, [0, 0, 7, 300, 0, 2, 0], [1100]])
def test_tree_masks(aa, new, chain):
    g = torch.Generator().manual_seed(len(new))
    parents = dr.random_tree(g, new, chain)
    cu = [0] + torch.tensor(new).cumsum(0).tolist()
    kv = [n + 11 * b for b, n in enumerate(new)]
    words = -(-max(new) // 64)
    seen, depth = dr.masks_of(parents.tolist(), cu, words)
    with aa.PagedCache(1, 16, 1, 64) as c:
        mask, pos = c.tree_masks(parents.cuda(), _i32(cu), _i32(kv), max(new))
        c.check_device_error()
        # into given tensors, with rows behind the batch that stay
        more = torch.cat([parents, torch.tensor([5, 5], dtype=torch.int32)]).cuda()
        om, op = torch.full((len(seen) + 2, words), 77, device="cuda"), torch.full((len(seen) + 2,), 77, dtype=torch.int32, device="cuda")
        c.tree_masks(more, _i32(cu), _i32(kv), max(new), out_mask=om, out_pos=op)
        c.check_device_error()
    assert torch.equal(mask.cpu(), dr.pack(seen, words))
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
    assert torch.equal(pos.cpu().long(), torch.tensor(kv)[seq] - torch.tensor(new)[seq] + torch.tensor(depth))
    assert torch.equal(om[:-2], mask) and torch.equal(op[:-2], pos) and (om[-2:] == 77).all() and (op[-2:] == 77).all()


def test_tree_masks_narrower_than_the_tree(aa):
    parents = dr.random_tree(torch.Generator().manual_seed(3), [200])
    seen, _ = dr.masks_of(parents.tolist(), [0, 200], 4)
    with aa.PagedCache(1, 16, 1, 64) as c:
        mask, _ = c.tree_masks(parents.cuda(), _i32([0, 200]), _i32([200]), 100)
        assert torch.equal(mask.cpu(), dr.pack(seen, 2))
        wide, _ = c.tree_masks(parents.cuda(), _i32([0, 200]), _i32([200]), 1000)
        assert torch.equal(wide.cpu(), dr.pack(seen, 16))
        none = c.tree_masks(parents[:0].cuda(), _i32([0, 0]), _i32([9]), 0)
        assert none[0].shape == (0, 1) and none[1].shape == (0,)
        c.check_device_error()


def test_bad_parents_count_as_roots_and_are_reported(aa):
    for at, bad in ((0, 0), (3, 3), (3, 7), (2, -2), (4, 2 ** 31 - 1), (4, -2 ** 31)):
        p = [-1, 0, 1, 1, 3]
        p[at] = bad
        seen, depth = dr.masks_of([x if -1 <= x < i else -1 for i, x in enumerate(p)], [0, 5], 1)
        with aa.PagedCache(1, 16, 1, 64) as c:
            mask, pos = c.tree_masks(_i32(p), _i32([0, 5]), _i32([25]), 5)
            with pytest.raises(aa.AAError, match="parent"):
                c.check_device_error()
            c.check_device_error()
        assert torch.equal(mask.cpu(), dr.pack(seen, 1)) and pos.tolist() == [20 + x for x in depth]


# ------------------------------------------------------------------ attention
SHAPES = [(8, 2, 128), (2, 2, 64), (7, 1, 64), (16, 1, 128), (20, 4, 128)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ps", [16, 64, 128])
@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("new", [[1, 2, 3, 0, 4], [7, 16, 0, 9], [26, 64, 33], [65, 130, 1], [300]])
def test_trees(aa, fp8, ps, Hq, Hkv, D, new):
    g = torch.Generator().manual_seed(len(new) + ps)
    kv = [n + (0, 1, 70, 500, 63)[b % 5] for b, n in enumerate(new)]
    d = _batch(fp8, ps + D, kv, new, Hq, Hkv, D, ps, device="cuda")
    seen, _ = dr.masks_of(dr.random_tree(g, new).tolist(), d["cu"].tolist(), 0)
    _attend(aa, d, ps, Hkv, D, dr.pack(seen, -(-max(new) // 64)).cuda())


@pytest.mark.parametrize("fp8", [False, True])
def test_a_chain_is_what_attend_does_without_a_tree(aa, fp8):
    """The two calls add the same terms, in an order of their own: each within its bound of the same definition."""
    for new in (1, 6, 130):
        kv = [new + 300, new + 65]
        d = _batch(fp8, new, kv, [new, new], 8, 2, 128, 32, device="cuda")
        seen, _ = dr.masks_of(dr.random_tree(None, [new, new], chain=True).tolist(), d["cu"].tolist(), 0)
        tree = dr.pack(seen, -(-new // 64)).cuda()
        _attend(aa, d, 32, 2, 128, tree)
        want = ref.attend(d["q"], d["kd"], d["vd"], d["table"], d["cu"], d["kv"])
        assert torch.equal(want[0], dr.attend_tree(d["q"], d["kd"], d["vd"], d["table"], d["cu"], d["kv"], tree)[0])
        with _cache(aa, d, 32, 2, 128) as c:
            ref.check_attend(*c.attend(d["q"], d["table"], d["cu"], d["kv"], new, return_lse=True), want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("max_q", [0, 1, 5, 40, 1000])
@pytest.mark.parametrize("Hq,D", [(8, 128), (2, 64)])
def test_max_q_is_a_hint(aa, fp8, max_q, Hq, D):
    new = [1, 150, 40]
    d = _batch(fp8, 8, [60, 500, 129], new, Hq, 2, D, 64, device="cuda") | {"max_q": max_q}
    seen, _ = dr.masks_of(dr.random_tree(torch.Generator().manual_seed(max_q), new).tolist(), d["cu"].tolist(), 0)
    lo = torch.arange(sum(new), dtype=torch.int32, device="cuda") * 7 % 90
    _attend(aa, d, 64, 2, D, dr.pack(seen, 3).cuda())
    _attend(aa, d, 64, 2, D, dr.pack(seen, 3).cuda(), key_lo=lo, anchor=True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("anchor", [False, True])
@pytest.mark.parametrize("new", [3, 40, 150])
def test_any_mask_with_windows_anchors_and_empty_rows(aa, fp8, anchor, new):
    """Rows that see later tokens, none, or bits that stand for none; first keys in front of, at and behind the cached
    ones; no cached tokens; fewer tokens held than new ones."""
    g = torch.Generator().manual_seed(new)
    kv = [new, new + 41, new + 700, max(new - 2, 1), 0]
    news = [new, new, new, new, 2]
    T, words = sum(news), -(-new // 64) + 1
    bits = torch.randint(-2 ** 63, 2 ** 63 - 1, (T, words), generator=g) & torch.randint(-2 ** 63, 2 ** 63 - 1, (T, words), generator=g)
    bits[torch.rand(T, generator=g) < 0.3] = 0
    base = torch.cat([torch.full((n,), k - n) for k, n in zip(kv, news)])
    lo = torch.where(torch.rand(T, generator=g) < 0.4, base + torch.randint(-2, 3, (T,), generator=g),
                     (base * torch.rand(T, generator=g)).long())
    for Hq, Hkv, D, ps in ((4, 1, 128, 32), (2, 2, 64, 128), (16, 1, 128, 16)):
        d = _batch(fp8, new, kv, news, Hq, Hkv, D, ps, device="cuda")
        for key_lo in (None, lo.to(torch.int32).cuda()):
            o, lse = _attend(aa, d, ps, Hkv, D, bits.cuda(), key_lo=key_lo, anchor=anchor)
            assert (lse[:, -2:] == -math.inf).all() and (o[-2:] == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,kv,Hq,Hkv,D", [(7, 52000, 8, 1, 128), (30, 20000, 8, 2, 128), (64, 9000, 16, 2, 64),
                                              (100, 3000, 4, 4, 128)])
def test_trees_over_long_contexts(aa, fp8, new, kv, Hq, Hkv, D):
    """Units whose keys are split among CTAs, with the new tokens in the last part, or across two."""
    g = torch.Generator().manual_seed(new)
    for lens, n in (([kv], [new]), ([kv, kv // 3], [new, new // 2])):
        d = _batch(fp8, new, lens, n, Hq, Hkv, D, 64, device="cuda")
        seen, _ = dr.masks_of(dr.random_tree(g, n).tolist(), d["cu"].tolist(), 0)
        lo = torch.full((sum(n),), kv // 5, dtype=torch.int32, device="cuda")
        lo[::7] = kv
        tree = dr.pack(seen, -(-new // 64)).cuda()
        _attend(aa, d, 64, Hkv, D, tree)
        _attend(aa, d, 64, Hkv, D, tree, key_lo=lo, anchor=True)


@pytest.mark.parametrize("width", [1030, 4700])
def test_trees_over_wide_tables(aa, width):
    """Ragged trees over 8-bit pages for which 16-bit copies are made of some sequences at a time, or of none."""
    g = torch.Generator().manual_seed(width)
    new, kv, ps, Hq, Hkv, D = [70, 0, 1, 90, 66, 33, 80], [300, 50, 900, 90, 200, 33, 700], 64, 32, 8, 128
    d = _batch(True, width, kv, new, Hq, Hkv, D, ps, device="cuda")
    d["table"] = torch.cat([d["table"], torch.full((len(kv), width - d["table"].shape[1]), -1, dtype=torch.int32, device="cuda")], 1)
    seen, _ = dr.masks_of(dr.random_tree(g, new).tolist(), d["cu"].tolist(), 0)
    lo = torch.randint(0, 300, (sum(new),), generator=g, dtype=torch.int32).cuda()
    _attend(aa, d, ps, Hkv, D, dr.pack(seen, 2).cuda())
    _attend(aa, d, ps, Hkv, D, dr.pack(seen, 2).cuda(), key_lo=lo, anchor=True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [5, 24, 130])
@pytest.mark.parametrize("ps", [16, 128])
def test_tokens_that_no_row_sees_do_not_reach_the_result(aa, fp8, new, ps):
    """NaN in new tokens that no mask names, behind the last token, and in cached ones in front of every first key."""
    g = torch.Generator().manual_seed(new)
    kv, Hq, Hkv, D = [new + 70, new], 4, 2, 128
    d = _batch(fp8, new, kv, [new, new], Hq, Hkv, D, ps, device="cuda")
    hidden = set(torch.randperm(new, generator=g)[:new // 3].tolist()) | {new - 1}
    seen = [{c for c in range(new) if c not in hidden and int(torch.randint(0, 3, (1,), generator=g))} for _ in range(2 * new)]
    lo = torch.full((2 * new,), 30, dtype=torch.int32, device="cuda")
    some = torch.zeros(d["P"], ps, dtype=torch.bool)
    for b in range(2):
        base = kv[b] - new
        for j in list(range(30, base)) + [base + c for s in seen[b * new:(b + 1) * new] for c in s]:
            some[int(d["table"][b, j // ps]), j % ps] = True
    some = some.cuda()
    for x in "kv":
        if fp8:
            d[x + "_scales"].view(torch.uint8).masked_fill_(~some[None, :, None], 255)
            d[x + "_pages"].view(torch.uint8).masked_fill_(~some[None, :, None, :, None], 127)
        else:
            d[x + "_pages"].masked_fill_(~some[None, :, None, :, None], math.nan)
    o, _ = _attend(aa, d, ps, Hkv, D, dr.pack(seen, -(-new // 64)).cuda(), key_lo=lo)
    assert torch.isfinite(o.float()).all()


def test_masks_that_are_slices_other_streams_and_graphs(aa):
    new, ps, Hq, Hkv, D = 30, 32, 8, 2, 128
    kv = [new + 300, new + 7]
    d = _batch(False, 1, kv, [new, new], Hq, Hkv, D, ps, layers=2, pad=2, device="cuda")
    g = torch.Generator().manual_seed(1)
    parents = torch.cat([dr.random_tree(g, [new, new]), torch.full((2,), -1, dtype=torch.int32)]).cuda()
    seen, _ = dr.masks_of(parents.tolist()[:2 * new], d["cu"].tolist(), 0)
    tree = torch.cat([dr.pack(seen, 1), torch.zeros(2, 1, dtype=torch.int64)]).cuda()
    o, _ = _attend(aa, d, ps, Hkv, D, tree, layer=1)
    wide = torch.full((d["T"], 3), -1, device="cuda")
    wide[:, 1:2] = tree
    with _cache(aa, d, ps, Hkv, D) as c:
        args = (d["q"], d["table"], d["cu"], d["kv"], new)
        out = torch.full_like(d["q"], 3.0)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        c.attend(*args, layer=1, out=out, tree=wide[:, 1:2], stream=s)
        s.synchronize()
        assert torch.equal(out[:2 * new], o[:2 * new]) and (out[2 * new:] == 3.0).all()
        work, path = c.alloc_workspace(2, d["T"], new, d["table"].shape[1], Hq), _i32([[0, 2], [1, -1]])
        mask, pos = c.tree_masks(parents, d["cu"], d["kv"], new)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.tree_masks(parents, d["cu"], d["kv"], new, out_mask=mask, out_pos=pos)
            c.attend(*args, layer=1, out=out, tree=mask, workspace=work)
            c.accept(d["table"], d["cu"], d["kv"], path)
        other = dr.random_tree(g, [new, new])  # another tree, lengths and path in the same graph
        parents[:2 * new] = other.cuda()
        d["kv"].sub_(3)
        path.copy_(_i32([[4, 9], [-1, 5]]))
        before = d["k_pages"].cpu().clone()
        want_o, _, ob, _ = dr.attend_tree(d["q"], d["k_pages"], d["v_pages"], d["table"], d["cu"], d["kv"],
                                          dr.pack(dr.masks_of(other.tolist(), d["cu"].tolist(), 0)[0], 1), 1)
        graph.replay()
        torch.cuda.synchronize()
        c.check_device_error()
        assert ((out[:2 * new].cpu().double() - want_o[:2 * new]).abs() <= ob[:2 * new]).all()
        want = dr.accept(before, d["table"].cpu(), d["cu"].tolist(), d["kv"].tolist(), [[4, 9], []])
        assert torch.equal(d["k_pages"].cpu(), want)


def test_attend_refusals(aa):
    d = _batch(False, 1, [30], [2], 4, 2, 64, 16, device="cuda")
    with _cache(aa, d, 16, 2, 64) as c:
        args = (d["q"], d["table"], d["cu"], d["kv"], 2)
        for tree in (torch.zeros(2, 1, dtype=torch.int32, device="cuda"), torch.zeros(3, 1, dtype=torch.int64, device="cuda"),
                     torch.zeros(2, 0, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda"),
                     torch.zeros(2, 1, dtype=torch.int64), [[1], [3]]):
            with pytest.raises(ValueError):
                c.attend(*args, tree=tree)
        with pytest.raises(aa.AAError):
            c.attend(*args, tree=torch.zeros(2, (1 << 14) + 1, dtype=torch.int64, device="cuda"))
        masks = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
        with pytest.raises(aa.AAError, match="tree"):  # a result in the masks
            c.attend(*args, tree=masks[:2], lse=masks[1:3].view(-1).view(torch.float32).view(4, 2))
        for bad in (dict(parents=_i32([[0]])), dict(parents=_i32([0]).long()), dict(cu=_i32([0])), dict(kv=_i32([1, 2])),
                    dict(max_q=-1), dict(out_mask=torch.zeros(1, 2, dtype=torch.int64, device="cuda"))):
            a = dict(parents=_i32([-1]), cu=_i32([0, 1]), kv=_i32([1]), max_q=1) | bad
            with pytest.raises(ValueError):
                c.tree_masks(a["parents"], a["cu"], a["kv"], a["max_q"], out_mask=a.get("out_mask"))
        for path in (_i32([0]), _i32([[0], [1]]), _i32([[0]]).long(), _i32([[0]]).cpu(), _i32([[0, 1, 2, 3]])[:, ::2]):
            with pytest.raises(ValueError):
                c.accept(d["table"], d["cu"], d["kv"], path)
        c.accept(d["table"], d["cu"], d["kv"], _i32([[]]).view(1, 0))
        c.check_device_error()


def test_sizes_out_of_range_are_refused_before_results_are_allocated(aa):
    d = _batch(False, 1, [30], [2], 4, 2, 64, 16, device="cuda")
    torch.cuda.synchronize()
    with _cache(aa, d, 16, 2, 64) as c:
        before = torch.cuda.max_memory_allocated()
        for max_q in ((1 << 20) + 1, 2 ** 31 - 1):
            with pytest.raises(ValueError):
                c.tree_masks(_i32([-1] * 5000), _i32([0, 5000]), _i32([5000]), max_q)
        for T in (1 << 30, 2 ** 31 - 1):
            with pytest.raises(ValueError):
                c.read(d["table"], d["cu"], d["kv"], T)
        assert torch.cuda.max_memory_allocated() - before < 1 << 20


# ------------------------------------------------------------------ accepting
PATHS = [[[0], [3], []], [[0, 1, 2], [0, 2, 3], [9]], [[5, 6, 7, 39], [1, 2, 3, 4], list(range(20))], [[], [], []],
         [list(range(1, 40)), list(range(25)), [0, 24]]]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ps", [16, 128])
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("Hkv,D,L", [(1, 64, 1), (3, 128, 2), (40, 128, 1)])
def test_accept(aa, fp8, ps, path, Hkv, D, L):
    """Rows that are read after they would have been overwritten, that cross pages and batches of rows, that stay."""
    new, kv = [40, 25, 25], [40, 25 + 13, 25 + 150]
    d = _batch(fp8, ps, kv, new, Hkv, Hkv, D, ps, layers=L, device="cuda")
    names = [x for x in ("k_pages", "v_pages", "k_scales", "v_scales") if x in d]
    raw = lambda x: d[x].view(torch.uint8).cpu().clone() if fp8 else d[x].cpu().clone()  # noqa: E731
    before = {x: raw(x) for x in names}
    width = max(len(p) for p in path) + 2
    table = torch.full((3, width), -1, dtype=torch.int32)
    for b, p in enumerate(path):
        table[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        table[b, len(p) + 1:] = 1  # what lies behind the first negative entry is not looked at
    with _cache(aa, d, ps, Hkv, D) as c:
        c.accept(d["table"], d["cu"], d["kv"], table.cuda())
        torch.cuda.synchronize()
        c.check_device_error()
    for x in names:
        assert torch.equal(raw(x), dr.accept(before[x], d["table"].cpu(), d["cu"].tolist(), kv, path)), x


@pytest.mark.parametrize("bad", [[2, 1], [1, 1], [0, 40], [40], [0, 2 ** 31 - 1], [3, 2, 5]])
def test_accept_moves_nothing_along_a_bad_path(aa, bad):
    d = _batch(False, 1, [60, 30], [40, 20], 2, 2, 64, 16, layers=2, device="cuda")
    before = d["k_pages"].cpu().clone()
    path = torch.full((2, 4), -1, dtype=torch.int32)
    path[0, :len(bad)] = torch.tensor(bad, dtype=torch.int32)
    path[1, :2] = torch.tensor([3, 7], dtype=torch.int32)
    with _cache(aa, d, 16, 2, 64) as c:
        c.accept(d["table"], d["cu"], d["kv"], path.cuda())
        with pytest.raises(aa.AAError, match="path"):
            c.check_device_error()
        assert torch.equal(d["k_pages"].cpu(), dr.accept(before, d["table"].cpu(), d["cu"].tolist(), [60, 30], [[], [3, 7]]))
        # positions and pages that are none
        for kv, table, match in ((_i32([39, 30]), d["table"], "position"), (_i32([160, 30]), d["table"], "position"),
                                 (d["kv"], torch.where(d["table"] >= 0, d["table"] + 1000, d["table"]), "page")):
            now = d["k_pages"].clone()
            c.accept(table, d["cu"], kv, _i32([[0, 7], [-1, -1]]))
            with pytest.raises(aa.AAError, match=match):
                c.check_device_error()
            assert torch.equal(d["k_pages"], now)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [3, 60])
def test_a_captured_step_on_several_streams(aa, fp8, new):
    """The calls behind a copy, a clear and another stream's work, in one graph: what they read is there."""
    ps, Hq, Hkv, D = 32, 8, 2, 128
    kv = [new + 300, new + 7]
    d = _batch(fp8, 4, kv, [new, new], Hq, Hkv, D, ps, layers=2, device="cuda")
    g = torch.Generator().manual_seed(2)
    parents = dr.random_tree(g, [new, new]).cuda()
    path = _i32([[1, 2], [2, -1]])
    with _cache(aa, d, ps, Hkv, D) as c:
        work = [c.alloc_workspace(2, d["T"], new, d["table"].shape[1], Hq) for _ in range(2)]
        q, out, here = torch.empty_like(d["q"]), torch.empty_like(d["q"]), torch.zeros_like(parents)
        plain = torch.empty_like(d["q"])
        k, v = torch.empty_like(d["k"]), torch.empty_like(d["v"])
        mask, pos = c.tree_masks(parents, d["cu"], d["kv"], new)
        rk, rv = c.read(d["table"], d["cu"], d["kv"], d["T"])

        def step(side):
            main = torch.cuda.current_stream()
            q.copy_(d["q"])
            k.copy_(d["k"])
            v.copy_(d["v"])
            side.wait_stream(main)
            with torch.cuda.stream(side):  # the first call behind another stream's copies
                c.append(k, v, d["table"], d["cu"], d["kv"])
                c.attend(q, d["table"], d["cu"], d["kv"], new, out=plain, workspace=work[0])
            here.zero_()
            here.copy_(parents)
            mask.zero_()
            c.tree_masks(here, d["cu"], d["kv"], new, out_mask=mask, out_pos=pos)
            main.wait_stream(side)
            c.attend(q, d["table"], d["cu"], d["kv"], new, out=out, tree=mask, workspace=work[1])
            out.mul_(1.0)
            c.accept(d["table"], d["cu"], d["kv"], path)
            rk.zero_()
            rv.zero_()
            c.read(d["table"], d["cu"], d["kv"], d["T"], out_k=rk, out_v=rv)

        side = torch.cuda.Stream()
        step(side)
        torch.cuda.synchronize()
        want = [x.clone() for x in (out, plain, mask, pos, rk, rv)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(side)
        for _ in range(3):
            for x in (q, out, plain, mask, pos, rk, rv, here, k, v):
                x.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip((out, plain, mask, pos, rk, rv), want))
        c.check_device_error()
        seen, _ = dr.masks_of(parents.tolist(), d["cu"].tolist(), 0)
        assert torch.equal(mask.cpu(), dr.pack(seen, 1))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("fp8", [False, True])
def test_drafting_run(aa, fp8):
    """A user's tokens are drafted as trees, verified and kept along a path, step after step: every kept token's attention,
    and what the cache holds in the end, are those of the same tokens appended one by one."""
    ps, Hq, Hkv, D, L, N = 16, 8, 2, 128, 2, 60
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(L, N, h, D, generator=g).to(torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv))
    rope = aa.RopeAxes(D, sections=(D // 2,), base=1e4)
    kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
    plain, spec = (aa.PagedCache(32, ps, Hkv, D, num_layers=L, max_seqs=2, dtype=kind, device="cuda") for _ in range(2))
    start = 21
    ref_o = torch.empty(L, N, Hq, D, dtype=torch.bfloat16, device="cuda")
    for t in [range(start)] + [[x] for x in range(start, N)]:  # the prompt, then token by token
        t, n = list(t), len(t)
        plain.resize([1], [t[-1] + 1])
        table, kv = plain.tables([1], device="cuda")
        for layer in range(L):
            qr = plain.append(k[layer, t], v[layer, t], table, _i32([0, n]), kv, layer=layer, rope=rope, pos=_i32(t), q=q[layer, t])
            ref_o[layer, t] = plain.attend(qr, table, _i32([0, n]), kv, n, layer=layer)
    spec.resize([0], [start])
    table, kv = spec.tables([0], device="cuda")
    for layer in range(L):
        spec.append(k[layer, :start], v[layer, :start], table, _i32([0, start]), kv, layer=layer, rope=rope, pos=_i32(list(range(start))))
    at = start
    while at < N:
        n = int(torch.randint(1, 20, (1,), generator=g))
        parents = dr.random_tree(g, [n]).tolist()
        depth = dr.masks_of(parents, [0, n], 1)[1]
        # the path to the deepest drafted token is right, as far as there are tokens; the others are wrong
        leaf, path = depth.index(max(depth)), []
        while leaf >= 0:
            path.insert(0, leaf)
            leaf = parents[leaf]
        path = path[:N - at]
        spec.resize([0], [at + n])
        table, kv = spec.tables([0], device="cuda")
        cu = _i32([0, n])
        mask, pos = spec.tree_masks(_i32(parents), cu, kv, n)
        assert pos.tolist() == [at + x for x in depth]
        for layer in range(L):
            qn, kn, vn = (torch.randn(n, h, D, generator=g).to(torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv))
            right = list(range(at, at + len(path)))
            qn[path], kn[path], vn[path] = q[layer, right], k[layer, right], v[layer, right]
            qr = spec.append(kn, vn, table, cu, kv, layer=layer, rope=rope, pos=pos, q=qn)
            o = spec.attend(qr, table, cu, kv, n, layer=layer, tree=mask)
            # two kernels' results of the same sums, each within its bound: 2^-8 of the weighted values and of the result
            want = ref_o[layer, right].float()
            assert (o[path].float() - want).abs().max() <= 2 * (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -14) * float(v.abs().max())
        keep = torch.full((1, n + 1), -1, dtype=torch.int32)
        keep[0, :len(path)] = torch.tensor(path, dtype=torch.int32)
        spec.accept(table, cu, kv, keep.cuda())
        at += len(path)
        spec.resize([0], [at])
    for c in (plain, spec):
        c.check_device_error()
    everything = [c.read(*c.tables([s], device="cuda")[:1], _i32([0, N]), _i32([N]), N, layer=layer)
                  for c, s in ((plain, 1), (spec, 0)) for layer in range(L)]
    for layer in range(L):
        for a, b in zip(everything[layer], everything[L + layer]):
            assert torch.equal(a, b)
    plain.close()
    spec.close()
