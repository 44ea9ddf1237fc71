"""The paged cache's bookkeeping and every refusal, through the C ABI without a GPU: which page belongs to which sequence
after growing, shrinking, forking, compacting and freeing, against a plain model of it; arguments that must be
refused before anything is launched."""
import ctypes
import os

import numpy as np
import pytest


@pytest.fixture(scope="module")
def aa():
    import __graft_entry__
    __graft_entry__.build()
    import packed_sequence_rope_gb300 as pkg
    return pkg


def _cache(aa, pages=16, ps=16, seqs=4):
    return aa.PagedCache(pages, ps, 2, 64, num_layers=2, max_seqs=seqs, host_only=True)


def _pages(c, seq):
    table, lens = c.tables([seq], width=64)
    n = -(-int(lens[0]) // c.ps)
    assert (table[0, n:] == -1).all() and (table[0, :n] >= 0).all()
    return table[0, :n].tolist()


def test_growing_and_shrinking_hand_out_the_lowest_pages(aa):
    with _cache(aa) as c:
        c.resize([0, 1], [17, 16])
        assert _pages(c, 0) == [0, 1] and _pages(c, 1) == [2]
        c.resize([0], [33])
        assert _pages(c, 0) == [0, 1, 3]
        c.resize([0], [16])            # exactly one page left
        assert _pages(c, 0) == [0] and c.stats()["free_pages"] == 14
        c.resize([2], [16 * 3])
        assert _pages(c, 2) == [1, 3, 4]
        c.free([0, 1, 2])
        assert c.stats() == {"free_pages": 16, "shared_pages": 0, "longest": 0}
        assert _pages(c, 2) == []


def test_shrinking_serves_growing_in_the_same_call(aa):
    with _cache(aa, pages=4) as c:
        c.resize([0], [64])
        c.resize([0, 1], [16, 48])
        assert _pages(c, 0) == [0] and _pages(c, 1) == [1, 2, 3]


def test_too_few_pages_changes_nothing(aa):
    with _cache(aa, pages=4) as c:
        c.resize([0], [40])
        before = _pages(c, 0), c.stats()
        with pytest.raises(aa.AAError) as e:
            c.resize([0, 1], [41, 17])
        assert e.value.status == 4
        assert (_pages(c, 0), c.stats()) == before and _pages(c, 1) == []


def test_fork_shares_and_growing_copies_the_partly_filled_page(aa):
    with _cache(aa) as c:
        c.resize([0], [40])
        c.fork(0, 1)
        assert _pages(c, 1) == _pages(c, 0) == [0, 1, 2] and c.stats()["shared_pages"] == 3
        c.resize([1], [41])            # grows into the shared third page: a page of its own
        assert _pages(c, 1) == [0, 1, 3] and _pages(c, 0) == [0, 1, 2]
        c.resize([0], [41])            # now the only holder of page 2
        assert _pages(c, 0) == [0, 1, 2]
        c.free([0])
        assert _pages(c, 1) == [0, 1, 3] and c.stats() == {"free_pages": 13, "shared_pages": 0, "longest": 3}


def test_two_forks_that_grow_in_one_call(aa):
    with _cache(aa) as c:
        c.resize([0], [20])
        c.fork(0, 1)
        c.fork(0, 2)
        c.resize([0, 1, 2], [21, 21, 33])
        tails = [_pages(c, s)[1] for s in range(3)]
        assert len(set(tails)) == 3 and c.stats()["shared_pages"] == 1


def test_fork_at_a_page_border_copies_nothing(aa):
    with _cache(aa) as c:
        c.resize([0], [32])
        c.fork(0, 1)
        c.resize([1], [33])
        assert _pages(c, 0) == [0, 1] and _pages(c, 1) == [0, 1, 2]


def test_shrinking_into_a_shared_full_page_then_growing_copies_it(aa):
    with _cache(aa) as c:
        c.resize([0], [32])
        c.fork(0, 1)
        c.resize([1], [20])            # inside page 1, which sequence 0 holds in full
        assert _pages(c, 1) == [0, 1]
        c.resize([1], [21])
        assert _pages(c, 1) == [0, 2] and _pages(c, 0) == [0, 1]


def test_compact_moves_used_pages_to_the_front(aa):
    with _cache(aa) as c:
        c.resize([0, 1, 2], [32, 32, 64])
        c.fork(2, 3)
        c.free([0])
        assert c.compact() == 2
        assert sorted(_pages(c, 1) + _pages(c, 2)) == list(range(6)) and _pages(c, 3) == _pages(c, 2)
        assert c.compact() == 0
        c.resize([0], [16])
        assert _pages(c, 0) == [6]


def test_random_walk_against_a_plain_model(aa):
    rng = np.random.default_rng(5)
    P, ps, S = 24, 16, 6
    with _cache(aa, pages=P, ps=ps, seqs=S) as c:
        for _ in range(600):
            op = rng.integers(0, 4)
            before = [_pages(c, s) for s in range(S)]
            lens = c.tables(range(S), width=64)[1].tolist()
            try:
                if op <= 1:
                    ids = rng.choice(S, rng.integers(1, 4), replace=False)
                    want = [int(max(0, lens[s] + rng.integers(-30, 60))) for s in ids]
                    c.resize(ids, want)
                    for s, n in zip(ids, want):
                        lens[s] = n
                elif op == 2:
                    a, b = (int(x) for x in rng.integers(0, S, 2))
                    c.fork(a, b)
                    lens[b] = lens[a]
                else:
                    c.compact()
            except aa.AAError:
                assert [_pages(c, s) for s in range(S)] == before
            now, got = [_pages(c, s) for s in range(S)], c.tables(range(S), width=64)[1].tolist()
            assert got == lens
            held = {}
            for s in range(S):
                assert len(set(now[s])) == len(now[s]) == -(-lens[s] // ps)
                for w, p in enumerate(now[s]):
                    held.setdefault(p, set()).add(w)
            assert all(len(w) == 1 for w in held.values())  # a shared page serves the same positions everywhere
            st = c.stats()
            assert st["free_pages"] == P - len(held)
            assert st["shared_pages"] == sum(sum(p in now[s] for s in range(S)) > 1 for p in held)
            if op == 3:
                assert all(p < len(held) for p in held)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(page_size=48), 2, "page_size"), (dict(page_size=256), 2, "page_size"), (dict(head_dim=96), 2, "head_dim"),
    (dict(num_layers=0), 1, "num_layers"), (dict(num_pages=0), 1, "num_pages"), (dict(num_kv_heads=0), 1, "num_kv_heads"),
    (dict(num_pages=1 << 24, num_kv_heads=8), 1, "2^31"), (dict(max_seqs=-1), 1, "max_seqs"),
])
def test_create_refusals(aa, kw, status, msg):
    args = dict(num_pages=4, page_size=16, num_kv_heads=1, head_dim=64) | kw
    with pytest.raises(aa.AAError) as e:
        aa.PagedCache(**args, host_only=True)
    assert e.value.status == status and msg in str(e.value)


def test_pool_pointers_are_refused_before_any_device_call(aa):
    cfg = aa.binding.AACacheConfig(1, 4, 16, 1, 64, 0, 0)
    h = ctypes.c_void_p()
    for k, v, msg in ((None, 4096, "16-byte"), (4096, 1 << 20 | 8, "16-byte"), (4096, 4096 + 64, "overlap")):
        assert aa.lib().aa_cache_create(ctypes.byref(cfg), k, v, ctypes.byref(h)) == 1 and not h.value
        assert msg in aa.lib().aa_last_error().decode()


@pytest.mark.parametrize("call,msg", [
    (lambda c: c.resize([4], [1]), "max_seqs"), (lambda c: c.resize([-1], [1]), "max_seqs"),
    (lambda c: c.resize([1, 1], [1, 2]), "twice"), (lambda c: c.resize([0], [-1]), "lengths"),
    (lambda c: c.fork(0, 1), "empty"), (lambda c: c.fork(0, 4), "max_seqs"), (lambda c: c.fork(0, 0), "empty"),
    (lambda c: c.tables([0], width=1), "table_width"), (lambda c: c.tables([9]), "max_seqs"),
    (lambda c: c.copy_pages([0], [1]), "host_only"),
])
def test_bookkeeping_refusals(aa, call, msg):
    with _cache(aa) as c:
        c.resize([0, 1], [20, 20])
        before = [_pages(c, s) for s in range(4)]
        with pytest.raises(aa.AAError) as e:
            call(c)
        assert e.value.status == 1 and msg in str(e.value)
        assert [_pages(c, s) for s in range(4)] == before


def test_a_cache_is_not_copied(aa):
    """Two objects with one handle would free it twice."""
    import copy
    import pickle
    with _cache(aa) as c:
        c.resize([0], [20])
        for call in (copy.copy, copy.deepcopy, pickle.dumps):
            with pytest.raises(TypeError, match="PagedCache"):
                call(c)
        assert _pages(c, 0) == [0, 1]


def test_cache_without_sequences_refuses_bookkeeping(aa):
    with _cache(aa, seqs=0) as c:
        for call in (lambda: c.resize([0], [1]), lambda: c.fork(0, 0), c.compact):
            with pytest.raises(aa.AAError):
                call()
        c.resize([], [])


def test_python_checks(aa):
    with _cache(aa) as c:
        with pytest.raises(ValueError):
            c.resize([0, 1], [3])
        with pytest.raises(ValueError):
            c.resize([0.5], [3])
        with pytest.raises(ValueError):
            c.resize([2 ** 40], [3])


@pytest.mark.parametrize("kw,msg", [
    (dict(head_dim=96, axis_of_pair=[0] * 48), "head_dim"), (dict(sections=(16, 24, 23)), "add up"),
    (dict(sections=(16, 16, 16, 8, 8)), "num_axes"), (dict(axis_of_pair=[0] * 63), "entries"),
    (dict(axis_of_pair=[0] * 63 + [-1]), "axis_of_pair"), (dict(sections=(64,), base=1.0), "base"),
    (dict(sections=(64,), theta=[1.0] * 63 + [float("nan")]), "theta"), (dict(sections=(64,), theta=[-1.0] * 64), "theta"),
    (dict(sections=(64,), layout=2), "layout"), (dict(), "either"), (dict(sections=(64,), axis_of_pair=[0] * 64), "either"),
])
def test_rope_axes_refusals(aa, kw, msg):
    with pytest.raises((aa.AAError, ValueError)) as e:
        aa.RopeAxes(**(dict(head_dim=128) | kw))
    assert msg in str(e.value)


def test_rope_axes_sections_and_fixed_point_angles(aa):
    r = aa.RopeAxes(64, sections=(4, 12, 16), interleaved=True, base=1e4)
    assert r.axis_of_pair[:12] == [0, 1, 2] * 4 and sorted(r.axis_of_pair) == [0] * 4 + [1] * 12 + [2] * 16
    assert aa.RopeAxes(64, sections=(4, 12, 16)).axis_of_pair == [0] * 4 + [1] * 12 + [2] * 16
    # the 64-bit fraction of a turn times the position, modulo one turn, is the angle
    for p in (0, 5, 31):
        theta = 1e4 ** (-2.0 * p / 64)
        for pos in (0, 1, 12345, 10 ** 9, -7, -2 ** 31):
            turns = (pos * r._c.turn[p]) % 2 ** 64 / 2 ** 64
            want = pos * theta / (2 * np.pi)
            d = turns - want
            assert abs(d - round(d)) * 2 * np.pi < 2.0 ** -20, (p, pos)


def test_copies_of_a_rotation_are_their_own(aa):
    """A copied, pickled or unpickled RopeAxes has a table of its own, which outlives the original's."""
    import copy
    import gc
    import pickle
    make = lambda: aa.RopeAxes(128, sections=(16, 24, 24), base=5e6, layout=aa.ROPE_HALF)
    original = make()
    want = bytes(original._c)
    copies = [copy.copy(original), copy.deepcopy(original), pickle.loads(pickle.dumps(original)), copy.deepcopy({"r": original})["r"]]
    del original
    gc.collect()
    others = [aa.RopeAxes(64, sections=(32,), base=1e4) for _ in range(64)]  # what reuses freed memory
    for r in copies:
        assert r._at == ctypes.addressof(r._c) and bytes(r._c) == want
        assert (r.head_dim, r.num_axes, r.layout, r.axis_of_pair) == (128, 3, aa.ROPE_HALF, make().axis_of_pair)
    assert len({r._at for r in copies[1:] + others}) == 3 + 64


def test_rope_axes_apply_refusals(aa):
    r, A = aa.RopeAxes(64, sections=(16, 16)), 1 << 20  # addresses that are never read: refused first
    ok = dict(T=4, q=A, qs=128, qo=A * 2, hq=2, k=A * 3, ks=128, ko=A * 4, hk=2, pos=A * 5)
    bad = [(dict(T=-1), "total_tokens"), (dict(hq=0), "q_heads"), (dict(hk=0), "NULL"), (dict(k=None), "NULL"),
           (dict(q=None), "q must"), (dict(q=A + 8), "16-byte"), (dict(qo=None), "q_out"), (dict(qs=120), "stride"),
           (dict(qs=132), "stride"), (dict(ko=A * 2 + 512), "overlap"), (dict(qo=A + 256), "overlaps"),
           (dict(qo=A, qs=256), "overlaps"), (dict(qo=A * 3), "overlap"), (dict(pos=None), "pos"), (dict(pos=A + 2), "pos")]
    for change, msg in bad:
        a = ok | change
        st = aa.lib().aa_rope_axes_apply(r._at, a["pos"], a["T"], a["q"], a["qs"], a["qo"], a["hq"], a["k"], a["ks"], a["ko"],
                                         a["hk"], 0, None)
        assert st == 1 and msg in aa.lib().aa_last_error().decode(), (change, aa.lib().aa_last_error())
    assert aa.lib().aa_rope_axes_apply(None, A, 4, A, 128, 2 * A, 2, None, 0, None, 0, 0, None) == 1
    blank = aa.binding.AARopeAxes()
    assert aa.lib().aa_rope_axes_apply(ctypes.addressof(blank), A, 4, A, 128, 2 * A, 2, None, 0, None, 0, 0, None) == 1
    assert "init" in aa.lib().aa_last_error().decode()
    # an empty call is accepted without pointers
    assert aa.lib().aa_rope_axes_apply(r._at, None, 0, None, 0, None, 2, None, 0, None, 0, 0, None) == 0


def test_empty_rotation_with_keys_is_accepted(aa):
    """No tokens: tensors without elements have no address, and none is read."""
    r = aa.RopeAxes(64, sections=(16, 16))
    for k_heads in (0, 2):
        assert aa.lib().aa_rope_axes_apply(r._at, None, 0, None, 128, None, 2, None, 128, None, k_heads, 0, None) == 0
    for q_heads, k_heads in ((0, 2), (2, -1), (65537, 0)):  # sizes are still looked at
        assert aa.lib().aa_rope_axes_apply(r._at, None, 0, None, 128, None, q_heads, None, 128, None, k_heads, 0, None) == 1


def test_device_calls_refuse_a_host_only_cache(aa):
    with _cache(aa) as c:
        L = aa.lib()
        for st in (L.aa_cache_append(c._h, None, None, 0, None, 0, None, None, None, 0, None, 0, None),
                   L.aa_cache_attend(c._h, None, None, 0, 1, 1, None, 0, 0.0, None, None, None, 0, None),
                   L.aa_cache_check_error(c._h, None), L.aa_cache_copy_pages(c._h, None, None, 0, None)):
            assert st == 1 and "host_only" in L.aa_last_error().decode()
        assert L.aa_cache_attend_workspace_bytes(None, 1, 1, 1, 1, 1) == 0
        assert L.aa_cache_attend_workspace_bytes(c._h, 0, 1, 1, 1, 2) == 0


def test_native_calls_are_rebuilt_for_another_torch(aa, tmp_path, monkeypatch):
    """_calls.so fits the torch that it was compiled for: with another one the build is stale."""
    from packed_sequence_rope_gb300 import _build
    assert not _build._stale()
    real = _build._torch()
    with open(os.path.join(real, "version.py")) as f:
        text = f.read()
    (tmp_path / "version.py").write_text(text + "\n# another build\n")
    with monkeypatch.context() as m:
        m.setattr(_build, "_torch", lambda: str(tmp_path))
        assert _build._stale()
    assert not _build._stale()
