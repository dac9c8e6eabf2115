"""The indexer's operators without a GPU: exported symbols, host-side refusals of the C
entry points and of the binding, and the frequencies of scaled rotary positions."""

import ctypes
import math
import os
import re

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_sm_gb300 import build
    build.build()
    import sparse_attention_indexer_sm_gb300 as pkg
    return pkg.load_library()


def test_every_declared_function_is_exported_and_bound(lib):
    text = open(os.path.join(ROOT, "include", "indexer_ops.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^\s*(?:int|size_t)\s+(indexer_\w+)\s*\(", text, flags=re.M)
    assert {"indexer_rotary", "indexer_quantise", "indexer_cache_write", "indexer_cache_read",
            "indexer_scores", "indexer_guard_hits"} <= set(names)
    for name in names:
        assert hasattr(lib, name) and getattr(lib, name).argtypes is not None


ONE = 256  # a pointer that is never followed: every call below is refused on the host


def rotary(lib, **kw):
    a = dict(x=ONE, xts=512, xhs=128, pos=ONE, freqs=ONE, dtype=0, tokens=4, heads=4, dim=128, rot=64,
             start=64, layout=0, scale=1.0, transpose=0, out=1 << 20, ots=512, ohs=128)
    a.update(kw)
    return lib.indexer_rotary(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(dtype=-1), dict(layout=2), dict(layout=-1), dict(tokens=-1), dict(heads=-1),
    dict(dim=1, rot=2, start=0), dict(rot=0), dict(rot=3), dict(rot=66), dict(start=-1), dict(start=65),
    dict(dim=65538), dict(start=2**31 - 2), dict(xts=-1), dict(xhs=-1), dict(ots=-1), dict(ohs=-1),
    dict(x=None), dict(pos=None), dict(freqs=None), dict(out=None), dict(x=257), dict(out=257),
    dict(dtype=2, x=258), dict(ohs=127), dict(ots=511), dict(ots=128, ohs=128), dict(ots=128, ohs=511),
    dict(tokens=2**31)])
def test_rotary_refusals(lib, bad):
    assert rotary(lib, **bad) == 1


def test_rotary_of_nothing(lib):
    assert rotary(lib, tokens=0, x=None, out=None) == 0
    assert rotary(lib, heads=0, x=None, out=None) == 0


def quantise(lib, **kw):
    a = dict(x=ONE, xts=512, xhs=128, dtype=0, tokens=4, heads=4, dim=128, fmt=0, weights=None, codes=ONE,
             scales=ONE)
    a.update(kw)
    return lib.indexer_quantise(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(fmt=2), dict(fmt=-1), dict(tokens=-1), dict(heads=-1), dict(dim=0), dict(dim=65537),
    dict(xts=-1), dict(xhs=-1), dict(x=None), dict(codes=None), dict(scales=None), dict(x=257),
    dict(scales=258), dict(weights=258), dict(weights=ONE, dim=129), dict(tokens=2**31)])
def test_quantise_refusals(lib, bad):
    assert quantise(lib, **bad) == 1


def cache(**kw):
    import sparse_attention_indexer_sm_gb300.indexer as ix
    a = dict(codes=ONE, scales=ONE, num_pages=8, code_page_stride=64 * 128, code_token_stride=128,
             scale_page_stride=64, scale_token_stride=1, page_size=64, dim=128)
    a.update(kw)
    return ix.IndexerCache(*a.values())


BAD_CACHES = [dict(num_pages=-1), dict(page_size=0), dict(dim=0), dict(dim=65537), dict(codes=None),
              dict(scales=None), dict(scales=258), dict(code_token_stride=127), dict(code_page_stride=127),
              dict(scale_token_stride=0), dict(scale_page_stride=0), dict(num_pages=2**26, page_size=32)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_cache_refusals(lib, bad):
    c = cache(**bad)
    p = ctypes.addressof(c)
    assert lib.indexer_cache_write(ONE, 128, 0, 4, ONE, 0, p, None) == 1
    assert lib.indexer_cache_read(p, ONE, 4, 0, ONE, None) == 1
    assert lib.indexer_scores(ONE, ONE, p, ONE, 1, ONE, 1, 1, 64, 64, ONE, None) == 1


def test_write_and_read_refusals(lib):
    c = cache()
    p = ctypes.addressof(c)
    write, read = lib.indexer_cache_write, lib.indexer_cache_read
    assert write(ONE, 128, 0, 4, ONE, 0, None, None) == 1
    assert write(ONE, 128, 3, 4, ONE, 0, p, None) == 1
    assert write(ONE, 128, 0, 4, ONE, 2, p, None) == 1
    assert write(ONE, 128, 0, -1, ONE, 0, p, None) == 1
    assert write(ONE, -1, 0, 4, ONE, 0, p, None) == 1
    assert write(None, 128, 0, 4, ONE, 0, p, None) == 1
    assert write(ONE, 128, 0, 4, None, 0, p, None) == 1
    assert write(ONE, 128, 0, 4, 258, 0, p, None) == 1
    assert write(257, 128, 0, 4, ONE, 0, p, None) == 1
    assert write(None, 128, 0, 0, None, 0, p, None) == 0
    assert read(None, ONE, 4, 0, ONE, None) == 1
    assert read(p, ONE, 4, 3, ONE, None) == 1
    assert read(p, ONE, -1, 0, ONE, None) == 1
    assert read(p, None, 4, 0, ONE, None) == 1
    assert read(p, ONE, 4, 0, None, None) == 1
    assert read(p, ONE, 4, 2, 258, None) == 1
    assert read(p, 258, 4, 0, ONE, None) == 1
    assert read(p, None, 0, 0, None, None) == 0


def scores(lib, c, **kw):
    a = dict(q=ONE, w=ONE, cache=ctypes.addressof(c), pt=ONE, pts=4, lens=ONE, batch=2, queries=2, heads=64,
             row_len=256, out=ONE)
    a.update(kw)
    return lib.indexer_scores(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(w=None), dict(pt=None), dict(lens=None), dict(out=None), dict(q=264), dict(w=258),
    dict(pt=258), dict(lens=258), dict(out=258), dict(batch=-1), dict(queries=-1), dict(heads=0),
    dict(heads=129), dict(row_len=0), dict(row_len=2**31), dict(pts=3), dict(cache=None),
    dict(batch=65536, queries=65536)])
def test_scores_refusals(lib, bad):
    assert scores(lib, cache(), **bad) == 1


def test_scores_refuse_other_rows_and_alignments(lib):
    assert scores(lib, cache(dim=256, code_token_stride=256, code_page_stride=64 * 256)) == 1
    assert scores(lib, cache(codes=ONE + 8)) == 1
    assert scores(lib, cache(code_token_stride=132, code_page_stride=64 * 132)) == 1
    assert scores(lib, cache(code_page_stride=64 * 128 + 8)) == 1
    assert scores(lib, cache(), batch=0, q=None) == 0
    assert scores(lib, cache(), queries=0, q=None) == 0
    assert lib.indexer_guard_hits(None) == 1


def test_binding_refuses_cpu_tensors_and_other_types():
    import sparse_attention_indexer_sm_gb300 as fw
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    pos, freqs = torch.zeros(4, dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        fw.indexer_rotary(x, pos, freqs)
    with pytest.raises(TypeError, match="x must be"):
        fw.indexer_rotary(x.double(), pos, freqs)
    with pytest.raises(ValueError, match="layout"):
        fw.indexer_rotary(x, pos, freqs, layout="neox")
    with pytest.raises(ValueError, match="CUDA"):
        fw.indexer_quantise(x)
    with pytest.raises(ValueError, match="scale_format"):
        fw.indexer_quantise(x, scale_format="e8m0")
    codes = torch.zeros(2, 64, 128, dtype=torch.float8_e4m3fn)
    scales = torch.zeros(2, 64, 1)
    with pytest.raises(ValueError, match="CUDA"):
        fw.indexer_cache_write(x[:, 0], pos, codes, scales)
    with pytest.raises(ValueError, match="CUDA"):
        fw.indexer_cache_read(codes, scales, pos)
    with pytest.raises(ValueError, match="dtype"):
        fw.indexer_cache_read(codes, scales, pos, dtype=torch.float64)
    with pytest.raises(TypeError, match="codes must be"):
        fw.indexer_cache_read(codes.view(torch.uint8), scales, pos)
    with pytest.raises(ValueError, match="CUDA"):
        fw.indexer_scores(torch.zeros(1, 1, 64, 128, dtype=torch.float8_e4m3fn), torch.zeros(1, 1, 64), codes,
                          scales, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32), 128)


def test_frequencies():
    import sparse_attention_indexer_sm_gb300 as fw
    f, scale = fw.indexer_rotary_freqs(64, device="cpu")
    assert scale == 1.0 and f.dtype == torch.float64 and f.shape == (32,)
    assert f[0] == 1.0 and math.isclose(f[31].item(), 10000.0 ** (-62 / 64), rel_tol=1e-14)
    lin, _ = fw.indexer_rotary_freqs(64, scaling="linear", factor=8.0, device="cpu")
    assert torch.allclose(lin * 8.0, f, rtol=1e-14, atol=0)
    ntk, _ = fw.indexer_rotary_freqs(64, scaling="ntk", factor=8.0, device="cpu")
    assert ntk[0] == 1.0 and math.isclose(ntk[31].item() * 8.0, f[31].item(), rel_tol=1e-12)
    yarn, scale = fw.indexer_rotary_freqs(64, scaling="yarn", factor=40.0, original_len=4096, device="cpu")
    turns = 4096.0 * f / (2.0 * math.pi)
    fast, slow = turns >= 32.0, turns <= 1.0
    assert fast.any() and slow.any() and (~fast & ~slow).any()
    assert torch.equal(yarn[fast], f[fast]) and torch.allclose(yarn[slow] * 40.0, f[slow], rtol=1e-14, atol=0)
    between = ~fast & ~slow
    assert ((yarn < f) & (yarn > f / 40.0))[between].all()
    assert math.isclose(scale, 0.1 * math.log(40.0) + 1.0)
    for bad in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=64, scaling="dynamic"), dict(rot_dim=64, factor=0.5),
                dict(rot_dim=64, base=1.0), dict(rot_dim=64, scaling="yarn", beta_fast=1.0, beta_slow=1.0)):
        with pytest.raises(ValueError):
            fw.indexer_rotary_freqs(**bad, device="cpu")
