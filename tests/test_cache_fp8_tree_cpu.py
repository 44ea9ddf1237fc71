"""8-bit pages and drafted trees through the C ABI without a GPU: what must be refused before anything is launched, and the
definitions that the GPU tests use."""
import ctypes

import pytest
import torch

import drafts_reference as dr


@pytest.fixture(scope="module")
def aa():
    import __graft_entry__
    __graft_entry__.build()
    import packed_sequence_rope_gb300 as pkg
    return pkg


def test_code_values_are_the_types():
    x = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    assert torch.equal(dr.code_values().nan_to_num(1000.0), x.nan_to_num(1000.0))


def test_quantise_is_the_nearest_code_at_the_smallest_scale():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(500, 64, generator=g, dtype=torch.float64) * torch.exp2(torch.randint(-130, 117, (500, 1), generator=g))
    held, e = dr.quantise(x)
    p = torch.exp2(e.double())[:, None]
    codes = dr.code_values()[torch.tensor([c for c in range(256) if c & 127 != 127])]
    best = ((x.clamp(-448 * p, 448 * p) / p)[..., None] - codes).abs().amin(-1)
    assert torch.allclose((x.clamp(-448 * p, 448 * p) - held).abs() / p, best, rtol=0, atol=1e-12)
    top = x.abs().amax(-1, keepdim=True)
    assert (top <= 448 * p).all() and ((top > 224 * p) | (e[:, None] == -100)).all()


def test_create_refusals(aa):
    cfg = aa.binding.AACacheConfig(1, 4, 16, 2, 64, 0, 0)
    out = ctypes.c_void_p()
    size = 4 * 2 * 16
    k, v, ks, vs = 1 << 20, 1 << 21, 1 << 22, 1 << 23
    for a in ((0, ks, v, vs), (k, 0, v, vs), (k, ks, 0, vs), (k, ks, v, 0), (k + 8, ks, v, vs), (k, ks + 8, v, vs),
              (k, ks, k + 64 * size - 16, vs), (k, k + 64, v, vs), (k, ks, v, v + 16), (k, ks, v, ks + size - 16)):
        assert aa.lib().aa_cache_create_fp8(ctypes.addressof(cfg), *a, ctypes.byref(out)) == 1, a
        assert not out.value
    assert aa.lib().aa_cache_create_fp8(None, k, ks, v, vs, ctypes.byref(out)) == 1
    assert aa.lib().aa_cache_create_fp8(ctypes.addressof(cfg), k, ks, v, vs, None) == 1
    cfg.head_dim = 96
    assert aa.lib().aa_cache_create_fp8(ctypes.addressof(cfg), k, ks, v, vs, ctypes.byref(out)) == 2


def test_device_calls_refuse_a_host_only_cache(aa):
    with aa.PagedCache(16, 16, 2, 64, max_seqs=2, host_only=True, dtype=torch.float8_e4m3fn) as c:
        c.resize([0], [33])
        assert c.tables([0])[0].shape == (1, 3) and c.k_scales is None
        batch = aa.binding.AACacheBatch(16, 16, 16, 1, 1, 1, 0)
        at = ctypes.addressof(batch)
        L = aa.lib()
        for call in (lambda h: L.aa_cache_read(h, at, 16, 32, None),
                     lambda h: L.aa_cache_accept(h, at, 16, 1, None),
                     lambda h: L.aa_cache_tree_masks(h, 16, 16, 16, 1, 1, 1, 16, 16, None),
                     lambda h: L.aa_cache_attend_tree(h, at, 16, 128, 2, 1, None, 0, 16, 1, 0.0, 16, None, 256, 256, None)):
            assert call(c._h) == 1 and b"host_only" in L.aa_last_error()
            assert call(None) == 1
        for words in (0, -1, (1 << 14) + 1):
            assert L.aa_cache_attend_tree(c._h, at, 16, 128, 2, 1, None, 0, 16, words, 0.0, 16, None, 256, 256, None) == 1
        with pytest.raises(ValueError):
            c.tree_masks(torch.zeros(1, dtype=torch.int32), None, None, 1)
        with pytest.raises(ValueError):
            c.accept(None, None, None, None)
        with pytest.raises(ValueError):
            c.read(None, None, None, 1)


def test_types_that_are_none_are_refused(aa):
    for dtype in (torch.float16, torch.float8_e5m2, torch.uint8):
        with pytest.raises(ValueError):
            aa.PagedCache(16, 16, 2, 64, host_only=True, dtype=dtype)


def test_masks_and_paths_of_the_definitions():
    seen, depth = dr.masks_of([-1, 0, 0, 2, -1], [0, 5], 1)
    assert seen == [{0}, {0, 1}, {0, 2}, {0, 2, 3}, {4}] and depth == [0, 1, 1, 2, 0]
    assert dr.pack([{0, 63, 64}], 2).tolist() == [[1 - (1 << 63), 1]]
    pages = torch.arange(6.0).view(1, 3, 1, 2, 1)
    table = torch.tensor([[2, 0, 1]])
    got = dr.accept(pages, table, [0, 5], [6], [[1, 3]])  # base 1: positions 2 and 4 to 1 and 2
    rows = [pages[0, table[0, p // 2], 0, p % 2, 0].item() for p in range(6)]
    after = [got[0, table[0, p // 2], 0, p % 2, 0].item() for p in range(6)]
    assert after == [rows[0], rows[2], rows[4], rows[3], rows[4], rows[5]]
