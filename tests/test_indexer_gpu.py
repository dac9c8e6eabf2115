"""The indexer's operators against plain implementations in 64 bits (needs a GB300).

Tolerances. A product of two values rounded to p bits is off by at most half a step,
``torch.finfo(t).eps / 2`` relative; each test states how many such steps its operator
takes. Codes, scales and read-back rows have one right value and are compared exactly.
"""

from __future__ import annotations

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24  # half a step of fp32
TYPES = [torch.bfloat16, torch.float16, torch.float32]
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def fw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_indexer_sm_gb300 as p
    p.load_library()
    return p


@pytest.fixture(autouse=True)
def no_guard_hits(fw):
    fw.indexer_reset_guard_hits()
    yield
    assert fw.indexer_guard_hits() == 0, "a slot or a page outside the cache, or a wait that ran out"


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------- rotary positions

def rotary_ref(x, positions, freqs, layout, start, scale, transpose):
    """(result, tolerance) in 64 bits on the CPU."""
    x, freqs = x.double().cpu(), freqs.cpu()
    r2 = freqs.shape[0]
    i = torch.arange(r2)
    ia, ib = (start + i, start + r2 + i) if layout == "half" else (start + 2 * i, start + 2 * i + 1)
    angle = positions.cpu().double()[:, None] * freqs
    if x.dim() == 3:
        angle = angle[:, None]
    c, s = scale * angle.cos(), scale * angle.sin() * (-1 if transpose else 1)
    a, b = x[..., ia], x[..., ib]
    y, tol = x.clone(), torch.zeros_like(x)
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    # the angle: half a step of its 24 bits as a share of half a turn (pi), and the 64-bit
    # products' own (the frequency's two, the reference's); sine and cosine: 2 steps; the
    # factor, the product, the sum: a half step each
    off = scale * (a.abs() + b.abs()) * (math.pi * U32 + angle.abs() * 2.0 ** -51 + (2 * 2 + 3) * U32)
    tol[..., ia] = tol[..., ib] = off
    return y, tol


def check(out, ref, tol):
    assert out.shape == ref.shape
    half = torch.finfo(out.dtype).eps / 2
    smallest = torch.finfo(out.dtype).smallest_normal * torch.finfo(out.dtype).eps
    got = out.detach().double().cpu()
    bound = tol + (ref.abs() + tol) * half + smallest
    worst = ((got - ref).abs() / bound).nan_to_num(0.0, math.inf, math.inf).max().item() if ref.numel() else 0.0
    assert worst <= 1.0, f"off by {worst:.3g} of the tolerance"


ROTARY = [  # tokens, heads (0: no such axis), dim, rot, start
    (1, 1, 2, 2, 0), (1, 64, 128, 64, 64), (3, 5, 128, 128, 0), (17, 7, 80, 80, 0), (5, 2, 192, 64, 128),
    (33, 0, 64, 64, 0), (4, 3, 130, 6, 7), (2, 9, 63, 62, 1), (300, 1, 576, 64, 512), (7, 33, 96, 16, 40),
    (2, 1, 4100, 4096, 4)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("shape", ROTARY)
def test_rotary_and_its_gradient(fw, shape, layout, dtype):
    tokens, heads, dim, rot, start = shape
    g = gen(dim + tokens)
    x = torch.randn((tokens, heads, dim) if heads else (tokens, dim), generator=g).to(dtype).cuda()
    positions = torch.randint(-100, 300000, (tokens,), generator=g, dtype=torch.int32).cuda()
    freqs, scale = fw.indexer_rotary_freqs(rot, scaling="yarn", factor=4.0)
    x.requires_grad_(True)
    y = fw.indexer_rotary(x, positions, freqs, layout=layout, start=start, scale=scale)
    check(y, *rotary_ref(x.detach(), positions, freqs, layout, start, scale, False))
    dy = torch.randn(y.shape, generator=g).to(dtype).cuda()
    y.backward(dy)
    check(x.grad, *rotary_ref(dy, positions, freqs, layout, start, scale, True))
    rest = [i for i in range(dim) if not start <= i < start + rot]
    assert torch.equal(y.detach()[..., rest], x.detach()[..., rest])


def test_rotary_gradient_against_differences(fw):
    """The rotation is linear: <R(x + d) - R(x), v> equals <d, R^T v>. In fp32 with small whole
    numbers for x, d and v, each side is a sum of 2 * 6 * 32 rounded terms of a few units."""
    g = gen(3)
    x, d, v = (torch.randint(-4, 5, (6, 2, 32), generator=g).float().cuda() for _ in range(3))
    positions = torch.arange(6, dtype=torch.int32).cuda() * 1000
    freqs, scale = fw.indexer_rotary_freqs(16, scaling="yarn", factor=8.0)
    leaf = x.clone().requires_grad_(True)
    for layout in ("half", "interleaved"):
        how = dict(layout=layout, start=8, scale=scale)
        (grad,) = torch.autograd.grad(fw.indexer_rotary(leaf, positions, freqs, **how), leaf, v)
        moved = (fw.indexer_rotary(x + d, positions, freqs, **how).double()
                 - fw.indexer_rotary(x, positions, freqs, **how).double())
        left, right = (moved * v.double()).sum().item(), (grad.double() * d.double()).sum().item()
        terms = 6 * 2 * 32 * (16 * scale * 2) * 4  # values up to 8 sqrt 2 times 4, both sides
        assert abs(left - right) <= terms * 16 * U32


def test_rotary_twice_differentiable_and_broadcast_inputs(fw):
    positions = torch.tensor([0, 5, 70000], dtype=torch.int32).cuda()
    freqs, _ = fw.indexer_rotary_freqs(8)
    key = torch.randn((3, 1, 8), generator=gen(1)).cuda().requires_grad_(True)
    y = fw.indexer_rotary(key.expand(3, 4, 8), positions, freqs)       # one head shared by four
    dy = torch.randn((3, 4, 8), generator=gen(2)).cuda().requires_grad_(True)
    (grad,) = torch.autograd.grad(y, key, dy, create_graph=True)
    ref, tol = rotary_ref(dy.detach(), positions, freqs, "half", 0, 1.0, True)
    check(grad, ref.sum(1, keepdim=True), tol.sum(1, keepdim=True) + 4 * U32 * ref.abs().sum(1, keepdim=True))
    (second,) = torch.autograd.grad(grad.sum(), dy)
    ones = torch.ones(3, 4, 8)
    check(second, *rotary_ref(ones, positions, freqs, "half", 0, 1.0, False))
    (flat,) = torch.autograd.grad(fw.indexer_rotary(key, positions, freqs).sum(), key)  # an expanded gradient
    check(flat, *rotary_ref(torch.ones(3, 1, 8), positions, freqs, "half", 0, 1.0, True))


def test_rotary_far_positions(fw):
    """Positions to the ends of int32, with frequencies above one turn a position too."""
    positions = torch.tensor([0, 1, -1, 2**20, 2**31 - 1, -2**31], dtype=torch.int32).cuda()
    freqs = torch.tensor([1.0, 0.1, 1e-6, 3.0, 7.5, 0.0], dtype=torch.float64).cuda()
    x = torch.randn((6, 3, 12), generator=gen(5)).cuda()
    for layout in ("half", "interleaved"):
        y = fw.indexer_rotary(x, positions, freqs, layout=layout)
        check(y, *rotary_ref(x, positions, freqs, layout, 0, 1.0, False))
    back = fw.indexer_rotary(y, positions, freqs, layout="interleaved", transpose=True)
    assert torch.allclose(back, x, rtol=0, atol=2 * 20 * U32 * 12)


def test_rotary_strides_in_place_and_streams(fw):
    g = gen(9)
    big = torch.randn((6, 4, 300), generator=g).to(torch.bfloat16).cuda()
    positions = torch.randint(0, 9999, (6,), generator=g, dtype=torch.int32).cuda()
    freqs, _ = fw.indexer_rotary_freqs(32)
    for x in (big[:, :, 40:168], big[:, :, 41:169], big.transpose(0, 1)[:, :, :128][:4],
              big[:, 1, :64], big[::2][:, ::3, 8:136], big[:1, :1, 3:67]):
        pos = positions[:x.shape[0]].contiguous()
        ref = rotary_ref(x, pos, freqs, "half", 16, 1.0, False)
        check(fw.indexer_rotary(x, pos, freqs, start=16), *ref)
        holder = torch.zeros((*x.shape[:-1], x.shape[-1] + 9), dtype=x.dtype, device="cuda")
        out = holder[..., 5:5 + x.shape[-1]]
        assert fw.indexer_rotary(x, pos, freqs, start=16, out=out) is out
        check(out, *ref)
        assert not holder[..., :5].any() and not holder[..., 5 + x.shape[-1]:].any()
    y = big.clone()
    z = y[:, :, 40:168]
    fw.indexer_rotary(z, positions, freqs, start=16, out=z)
    check(z, *rotary_ref(big[:, :, 40:168], positions, freqs, "half", 16, 1.0, False))
    assert torch.equal(y[:, :, :56], big[:, :, :56]) and torch.equal(y[:, :, 88:], big[:, :, 88:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = fw.indexer_rotary(big, positions, freqs, stream=side)
    side.synchronize()
    check(out, *rotary_ref(big, positions, freqs, "half", 0, 1.0, False))
    for shape in ((0, 4, 128), (6, 0, 128)):
        empty = torch.empty(shape, device="cuda")
        assert fw.indexer_rotary(empty, positions[:shape[0]].contiguous(), freqs).shape == shape


def test_rotary_keeps_what_is_not_finite_where_it_is(fw):
    x = torch.zeros((2, 2, 16)).cuda()
    x[0, 0, 0], x[0, 1, 15], x[1, 0, 9] = math.inf, math.nan, -math.inf
    positions = torch.tensor([3, 4], dtype=torch.int32).cuda()
    freqs, _ = fw.indexer_rotary_freqs(8)
    y = fw.indexer_rotary(x, positions, freqs)
    assert torch.isinf(y[0, 0, [0, 4]]).all() and torch.isnan(y[0, 1, 15]) and y[1, 0, 9] == -math.inf
    hit = torch.zeros((2, 2, 16), dtype=torch.bool)
    hit[0, 0, [0, 4]] = hit[0, 1, 15] = hit[1, 0, 9] = True
    assert not y.cpu()[~hit].any()


def test_rotary_refusals(fw):
    x = torch.zeros((4, 2, 128)).cuda()
    pos, freqs = torch.zeros(4, dtype=torch.int32).cuda(), torch.ones(32, dtype=torch.float64).cuda()
    bad = [dict(x=x.half().double()), dict(x=x[0, 0]), dict(x=x.transpose(1, 2)), dict(positions=pos[:3]),
           dict(positions=pos.long()), dict(positions=pos.cpu()), dict(freqs=freqs.float()), dict(freqs=freqs[:0]),
           dict(start=65), dict(start=-1), dict(layout="other"), dict(out=x[:, :1]), dict(out=x.half()),
           dict(out=x.as_strided((4, 2, 128), (0, 128, 1))), dict(freqs=torch.ones(65, dtype=torch.float64).cuda())]
    for kw in bad:
        args = dict(dict(x=x, positions=pos, freqs=freqs), **kw)
        with pytest.raises((ValueError, TypeError, fw.TopkError)):
            fw.indexer_rotary(args.pop("x"), args.pop("positions"), args.pop("freqs"), **args)
    buf = torch.zeros(4 * 256 + 64).cuda()
    a, b = buf[:1024].view(4, 2, 128), buf[64:1088].view(4, 2, 128)
    with pytest.raises(ValueError, match="overlap"):
        fw.indexer_rotary(a, pos, freqs, out=b)
    with pytest.raises(ValueError, match="differentiable"):
        fw.indexer_rotary(x.clone().requires_grad_(True), pos, freqs, out=torch.empty_like(x))


# ---------------------------------------------------------------- 8-bit rows

GRID = None


def grid():
    """The 127 finite magnitudes of e4m3, by their codes."""
    global GRID
    if GRID is None:
        GRID = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
                         for e in range(16) for m in range(8)][:127])
    return GRID


def quantise_ref(x, fmt):
    """(codes as bytes, scales) by comparisons with the middles between codes, in 64 bits."""
    x = x.double().cpu().numpy()
    dim = x.shape[-1]
    g = grid()
    mid = (g[1:] + g[:-1]) / 2
    codes = np.zeros(x.shape, dtype=np.uint8)
    scales = np.zeros(x.shape[:-1] + (-(-dim // 128),), dtype=np.float32)
    for k in range(scales.shape[-1]):
        v = x[..., 128 * k:128 * (k + 1)]
        fine = np.isfinite(v).all(-1)
        top = np.maximum(np.where(fine[..., None], np.abs(v), 0).max(-1), 2.0 ** -64)
        if fmt == "fp32":
            s = (top / 448.0).astype(np.float32)
        else:
            m, e = np.frexp(top)
            s = np.ldexp(1.0, np.where(m <= 0.875, e - 9, e - 8)).astype(np.float32)
        edge = mid * s.astype(np.float64)[..., None]           # exact: 5 bits by 24
        a = np.abs(np.where(fine[..., None], v, 0))
        c = (a[..., None] > edge[..., None, :]).sum(-1)
        tie = (a[..., None] == edge[..., None, :]).any(-1) & (c % 2 == 1)
        c = np.where(tie, c + 1, c).astype(np.uint8) | (np.signbit(v).astype(np.uint8) << 7)
        codes[..., 128 * k:128 * (k + 1)] = np.where(fine[..., None], c, 0x7F)
        scales[..., k] = np.where(fine, s, np.nan)
    return codes, scales


def same_quantised(codes, scales, ref):
    c, s = codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy()
    # a code's sign of zero is not part of its value
    c, r = np.where(c == 0x80, 0, c), np.where(ref[0] == 0x80, 0, ref[0])
    return np.array_equal(c, r) and np.array_equal(s, ref[1], equal_nan=True)


@pytest.mark.parametrize("fmt", ["fp32", "pow2"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 1, 128), (3, 64, 128), (37, 128), (5, 3, 576), (2, 7, 200), (9, 63), (4, 1),
                                   (33, 129), (2, 2, 1032)])
def test_quantise(fw, shape, dtype, fmt):
    g = gen(sum(shape))
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-12, 12, shape[:-1] + (1,), generator=g).float())
    x[..., ::37] *= 30.0
    x[0] = 0.0
    x = x.to(dtype).cuda()
    assert same_quantised(*fw.indexer_quantise(x, scale_format=fmt), quantise_ref(x, fmt))


def test_quantise_at_the_borders_between_codes(fw):
    """fp32 values on, and one step beside, the middles between codes, for scales whose
    quotients are not exact; and subnormal codes."""
    g = grid()
    mid = (g[1:] + g[:-1]) / 2
    rows = []
    for top in (1.0, 3.0, 447.0, 448.0, 1e-3, 7.1e4, 1e30, 2.0 ** -60):
        s = float(np.float32(np.float64(np.float32(top)) / 448.0))
        at = (mid * s).astype(np.float32)
        v = np.concatenate([at, np.nextafter(at, np.float32(np.inf)), np.nextafter(at, np.float32(0))])
        v = np.minimum(v, np.float32(top))
        for i in range(0, len(v), 127):
            part = np.zeros(128, dtype=np.float32)
            part[:len(v[i:i + 127])] = v[i:i + 127]
            part[1::2] *= -1
            part[127] = top
            rows.append(part)
    x = torch.from_numpy(np.stack(rows)).cuda()
    for fmt in ("fp32", "pow2"):
        assert same_quantised(*fw.indexer_quantise(x, scale_format=fmt), quantise_ref(x, fmt))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantise_16_bit_values_on_every_border(fw, dtype):
    """For every mantissa of the largest value, all values of the type whose quotients come near a border
    between codes: those on it depend on the rounding of the scale alone."""
    bits = 8 if dtype is torch.bfloat16 else 11
    g = grid()
    mid = (g[1:] + g[:-1]) / 2
    rows = []
    for a in range(2 ** (bits - 1), 2 ** bits):
        top = float(a)
        at = torch.from_numpy(mid * top / 448.0).to(dtype).double()
        step = torch.exp2(torch.floor(torch.log2(at.clamp(min=2.0 ** -24))) - (bits - 1))
        v = torch.cat([at, at + step, at - step]).clamp(0.0, top)
        v[1::2] *= -1
        for i in range(0, len(v), 127):
            part = torch.zeros(128, dtype=torch.float64)
            part[:len(v[i:i + 127])] = v[i:i + 127]
            part[127] = top
            rows.append(part)
    x = torch.stack(rows).to(dtype).cuda()
    for fmt in ("fp32", "pow2"):
        assert same_quantised(*fw.indexer_quantise(x, scale_format=fmt), quantise_ref(x, fmt))


@pytest.mark.parametrize("dtype", TYPES)
def test_quantise_extremes_and_what_is_not_finite(fw, dtype):
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    x = torch.zeros(8, 256, dtype=dtype)
    x[0], x[1, :128], x[1, 128:], x[2, 5], x[2, 200] = big, -big, tiny, tiny * torch.finfo(dtype).eps, big
    x[3, 7], x[4, 130], x[5, 255] = math.inf, -math.inf, math.nan
    x[6] = torch.randn(256, generator=gen(4)).to(dtype) * tiny
    x = x.cuda()
    for fmt in ("fp32", "pow2"):
        codes, scales = fw.indexer_quantise(x, scale_format=fmt)
        assert same_quantised(codes, scales, quantise_ref(x, fmt))
        assert torch.isnan(codes[3, :128].float()).all() and not torch.isnan(codes[3, 128:].float()).any()


def test_quantise_folds_weights_and_takes_strides(fw):
    g = gen(8)
    big = torch.randn((5, 6, 400), generator=g).to(torch.bfloat16).cuda()
    w = torch.randn((5, 6), generator=g).cuda()
    for x in (big[:, :, 16:144], big[:, :, 17:145], big[:, :, :100], big[:, :, 1:2]):
        ref = quantise_ref(x, "fp32")
        codes, folded = fw.indexer_quantise(x, weights=w)
        assert same_quantised(codes, (folded * 0 + torch.from_numpy(ref[1][..., 0]).cuda())[..., None], ref)
        assert np.array_equal(folded.cpu().numpy(), w.cpu().numpy() * ref[1][..., 0])
    for x in (big.transpose(0, 1)[:, :, :256], big[::2, ::2], big[:1].expand(5, 6, 400), big[:, 2]):
        assert same_quantised(*fw.indexer_quantise(x), quantise_ref(x, "fp32"))
    codes, scales = torch.empty((5, 6, 400), dtype=E4M3, device="cuda"), torch.empty((5, 6, 4), device="cuda")
    got = fw.indexer_quantise(big, codes=codes, scales=scales)
    assert got[0] is codes and got[1] is scales and same_quantised(codes, scales, quantise_ref(big, "fp32"))
    for n in (0, 1):
        c, s = fw.indexer_quantise(big[:n])
        assert c.shape == (n, 6, 400) and s.shape == (n, 6, 4)
    for kw in (dict(weights=w), dict(codes=codes[:4]), dict(scales=scales[..., :3]), dict(codes=codes.view(torch.uint8))):
        with pytest.raises((ValueError, TypeError)):
            fw.indexer_quantise(big, **kw)


# ---------------------------------------------------------------- the cache

def make_cache(pages, size, dim, layout="apart"):
    """A cache full of a pattern, with guard bytes between what belongs to it."""
    nb = -(-dim // 128)
    if layout == "apart":
        codes = torch.full((pages, size, dim), 3, dtype=torch.uint8, device="cuda").view(E4M3)
        return codes, torch.full((pages, size, nb), 7.0, device="cuda"), None
    if layout == "page":      # a page: its codes, then its scales, in one buffer
        width = size * dim + -(size * dim) % 4
        buf = torch.full((pages, width + size * nb * 4 + 16), 3, dtype=torch.uint8, device="cuda")
        codes = buf.view(E4M3).as_strided((pages, size, dim), (buf.shape[1], dim, 1))
        scales = buf.view(-1)[: buf.numel() // 4 * 4].view(torch.float32).as_strided(
            (pages, size, nb), (buf.shape[1] // 4, nb, 1), width // 4)
        assert buf.shape[1] % 4 == 0
        return codes, scales, buf
    stride = dim + 16 - dim % 16 + nb * 4 + (-nb * 4) % 16       # a row: its codes, then its scales
    buf = torch.full((size, pages, stride), 3, dtype=torch.uint8, device="cuda")  # pages inside rows
    codes = buf.view(E4M3).as_strided((pages, size, dim), (stride, stride * pages, 1))
    scales = buf.view(-1).view(torch.float32).as_strided(
        (pages, size, nb), (stride // 4, stride * pages // 4, 1), (dim + 16 - dim % 16) // 4)
    return codes, scales, buf


@pytest.mark.parametrize("layout", ["apart", "page", "row"])
@pytest.mark.parametrize("page_size", [1, 4, 48, 64])
@pytest.mark.parametrize("dim", [128, 576, 200, 63])
@pytest.mark.parametrize("dtype", TYPES)
def test_cache_write_and_read(fw, dtype, dim, page_size, layout):
    if layout == "page" and page_size * dim % 4:
        pytest.skip("scales would not be aligned")
    pages, tokens = 400 // page_size + 2, 133
    g = gen(dim + page_size)
    codes, scales, buf = make_cache(pages, page_size, dim, layout)
    before = buf.clone() if buf is not None else None
    x = torch.randn((tokens, dim), generator=g).to(dtype).cuda()
    slots = torch.randperm(pages * page_size, generator=g)[:tokens].int()
    slots[5], slots[tokens - 1] = -1, -1
    slots = slots.cuda()
    fw.indexer_cache_write(x, slots, codes, scales)
    ref = quantise_ref(x, "fp32")
    want_c = np.full((pages * page_size, dim), 3, dtype=np.uint8)
    want_s = np.full((pages * page_size, -(-dim // 128)), 7.0, dtype=np.float32)
    if buf is not None:
        want_s[:] = np.frombuffer(bytes([3] * 4), dtype=np.float32)[0]
    at = slots.cpu().numpy()
    want_c[at[at >= 0]], want_s[at[at >= 0]] = ref[0][at >= 0], ref[1][at >= 0]
    assert same_quantised(codes.reshape(-1, dim), scales.reshape(-1, want_s.shape[1]), (want_c, want_s))
    if buf is not None:  # nothing else of the buffer has changed
        mark = buf.clone()
        codes.view(torch.uint8).fill_(3)
        scales.view(torch.int32).fill_(0x03030303)
        assert torch.equal(buf, before)
        buf.copy_(mark)
    pick = torch.randint(-1, pages * page_size, (3, 50), generator=g, dtype=torch.int32)
    pick[0, 0], pick[2, 49], pick[1, 0] = -1, pages * page_size - 1, 0
    got = fw.indexer_cache_read(codes, scales, pick.cuda(), dtype=dtype)
    at = pick.numpy()
    c = torch.from_numpy(want_c).view(E4M3).float()[at.clip(0)]
    s = torch.from_numpy(np.repeat(want_s, 128, axis=1)[:, :dim])[at.clip(0)]
    want = torch.where(torch.from_numpy(at >= 0)[..., None], (c * s).to(dtype), torch.zeros((), dtype=dtype))
    assert got.shape == (3, 50, dim) and torch.equal(got.cpu(), want)


def test_cache_rows_that_are_not_finite_and_ranges(fw):
    codes, scales, _ = make_cache(4, 8, 256)
    x = torch.ones(3, 256)
    x[0, 3], x[1, 200] = math.nan, math.inf
    x[2] = 1e6
    slots = torch.tensor([0, 9, 31], dtype=torch.int32).cuda()
    fw.indexer_cache_write(x.cuda(), slots, codes, scales, scale_format="pow2")
    y = fw.indexer_cache_read(codes, scales, slots, dtype=torch.float16).cpu()
    assert torch.isnan(y[0, :128]).all() and (y[0, 128:] == 1).all()
    assert (y[1, :128] == 1).all() and torch.isnan(y[1, 128:]).all()
    assert torch.isinf(y[2]).all()  # past fp16's range


def test_slots_outside_the_cache_are_not_followed(fw):
    codes, scales, _ = make_cache(4, 8, 128)
    x = torch.randn((5, 128), generator=gen(1)).cuda()
    slots = torch.tensor([-2, 32, 2**31 - 1, -2**31, 7], dtype=torch.int32).cuda()
    fw.indexer_cache_write(x, slots, codes, scales)
    assert fw.indexer_guard_hits() == 4
    ref = quantise_ref(x, "fp32")
    assert same_quantised(codes.view(-1, 128)[7:8], scales.view(-1, 1)[7:8], (ref[0][4:], ref[1][4:]))
    rest = [i for i in range(32) if i != 7]
    assert (codes.view(torch.uint8).view(-1, 128)[rest] == 3).all() and (scales.view(-1)[rest] == 7).all()
    fw.indexer_reset_guard_hits()
    y = fw.indexer_cache_read(codes, scales, slots)
    assert fw.indexer_guard_hits() == 4 and not y[:4].any() and y[4].any()
    fw.indexer_reset_guard_hits()
    none = codes[:0], scales[:0]  # a cache of no pages
    assert not fw.indexer_cache_read(*none, torch.full((3,), -1, dtype=torch.int32).cuda()).any()
    fw.indexer_cache_write(x[:1], torch.full((1,), -1, dtype=torch.int32).cuda(), *none)


def test_cache_refusals(fw):
    codes, scales, _ = make_cache(4, 8, 128)
    x, slots = torch.zeros((5, 128)).cuda(), torch.zeros(5, dtype=torch.int32).cuda()
    for kw in (dict(x=x[:, :64]), dict(x=x[:, None]), dict(slots=slots[:4]), dict(slots=slots.long()),
               dict(codes=codes.view(torch.uint8)), dict(codes=codes[0]), dict(scales=scales[..., 0]),
               dict(scales=scales.half()), dict(scales=scales[:3]), dict(codes=codes[:1].expand(4, 8, 128)),
               dict(codes=codes.as_strided((4, 8, 128), (128, 128, 1))),
               dict(scales=scales[:, :1].expand(4, 8, 1)), dict(x=x.cpu()), dict(slots=slots.cpu())):
        a = dict(dict(x=x, slots=slots, codes=codes, scales=scales), **kw)
        with pytest.raises((ValueError, TypeError)):
            fw.indexer_cache_write(a["x"], a["slots"], a["codes"], a["scales"])
    with pytest.raises(ValueError):
        fw.indexer_cache_read(codes, scales, torch.zeros((4, 2), dtype=torch.int32).cuda().t())
    with pytest.raises(TypeError):
        fw.indexer_cache_read(codes, scales, slots, out=torch.empty((5, 128)).cuda())


def test_offsets_past_32_bits(fw):
    """A cache of 4.6 GB: rows at its far end are written, read and scored where they belong."""
    size, dim, pages = 64, 128, 36_000_000 // 64
    codes = torch.zeros((pages, size, dim), dtype=torch.uint8, device="cuda").view(E4M3)
    scales = torch.zeros((pages, size, 1), device="cuda")
    x = torch.randn((200, dim), generator=gen(6)).cuda()
    slots = (pages * size - 1 - 7 * torch.arange(200)).int().cuda()
    fw.indexer_cache_write(x, slots, codes, scales)
    ref = quantise_ref(x, "fp32")
    at = slots.long()
    assert same_quantised(codes.view(torch.uint8).view(-1, dim)[at].view(E4M3), scales.view(-1, 1)[at], ref)
    y = fw.indexer_cache_read(codes, scales, slots, dtype=torch.float32)
    want = torch.from_numpy(ref[0]).view(E4M3).float() * torch.from_numpy(ref[1])
    assert torch.equal(y.cpu(), want)
    q, w = fw.indexer_quantise(torch.randn((1, 8, 128), generator=gen(7)).cuda(), weights=torch.ones(1, 8).cuda())
    table = torch.arange(pages - 23, pages, dtype=torch.int32).cuda()[None]
    lens = torch.full((1, 1), 23 * size, dtype=torch.int32).cuda()
    got = fw.indexer_scores(q[None], w[None], codes, scales, table, lens, 23 * size)
    check_scores(got, q[None], w[None], codes[-23:], scales[-23:], table - (pages - 23), lens, 23 * size)


# ---------------------------------------------------------------- scores

def scores_ref(q, weights, codes, scales, table, lens, row_len):
    """(scores, tolerance) in 64 bits."""
    size = codes.shape[1]
    b, n, h, d = q.shape
    j = torch.arange(row_len)
    table, lens = table.cpu().long(), lens.cpu().long()
    slot = table[:, j // size] * size + j % size
    keys = codes.reshape(-1, d).cpu().float().double()[slot]                 # [b, row_len, d]
    s = scales.reshape(-1).cpu().double()[slot][:, None]
    q, w = q.cpu().float().double(), weights.cpu().double()
    dots = torch.einsum("bnhd,bjd->bnhj", q, keys)
    size_of = torch.einsum("bnhd,bjd->bnhj", q.abs(), keys.abs())
    relu = dots.clamp(min=0)
    y = (w[..., None] * relu).sum(2) * s
    # each of 128 additions keeps 24 bits or more, rounded or cut off (a step at most); so do
    # the heads' products and sums, and the scale
    tol = (w.abs()[..., None] * (128 * 2 * U32 * size_of + (h + 3) * 2 * U32 * relu)).sum(2) * s.abs()
    seen = j < lens.clamp(0, row_len)[..., None]
    y = torch.where(seen, y, torch.full_like(y, -math.inf)).view(b * n, row_len)
    return y, torch.where(seen, tol, torch.zeros_like(tol)).view(b * n, row_len)


def check_scores(got, *args):
    ref, tol = scores_ref(*args)
    got = got.double().cpu()
    assert got.shape == ref.shape
    fine = torch.isfinite(ref)
    assert torch.equal(got[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)])
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    off = (got - ref).abs()[fine]
    bound = tol[fine] + 1e-37
    assert bool((off <= bound).all()), f"off by {(off / bound).max().item():.3g} of the tolerance"


def scores_inputs(seed, b, n, h, row_len, page_size, lens=None, layout="apart"):
    g = gen(seed)
    pages = -(-row_len // page_size)
    total = b * pages + 3
    codes, scales, _ = make_cache(total, page_size, 128, layout)
    codes.copy_((torch.randn((total, page_size, 128), generator=g) * 90).clamp(-448, 448).to(E4M3))
    scales.copy_(torch.rand((total, page_size, 1), generator=g) * 0.02 + 0.001)
    table = torch.randperm(total, generator=g)[:b * pages].view(b, pages).int().cuda()
    q = (torch.randn((b, n, h, 128), generator=g) * 90).clamp(-448, 448).to(E4M3).cuda()
    w = torch.randn((b, n, h), generator=g).cuda()
    if lens is None:
        lens = torch.randint(0, row_len + 1, (b, n), generator=g).int()
    else:
        lens = torch.tensor(lens, dtype=torch.int32).view(b, n)
    return q, w, codes, scales, table, lens.cuda(), row_len


@pytest.mark.parametrize("case", [
    # batch, queries, heads, row_len, page_size
    (1, 1, 64, 1, 64), (1, 1, 64, 2048, 64), (3, 1, 64, 1000, 64), (2, 2, 64, 777, 64), (2, 4, 64, 300, 64),
    (1, 7, 64, 513, 64), (1, 33, 64, 640, 64), (2, 1, 128, 257, 64), (1, 5, 128, 400, 64), (3, 1, 1, 500, 64),
    (2, 3, 24, 333, 64), (1, 9, 8, 700, 64), (2, 1, 17, 129, 64), (1, 20, 33, 300, 64), (2, 1, 64, 300, 1),
    (2, 2, 32, 500, 48), (1, 1, 64, 1000, 128), (1, 3, 64, 900, 256), (2, 1, 64, 200, 16), (1, 2, 64, 130, 100),
    (2, 1, 64, 90, 7), (5, 2, 96, 260, 2), (1, 130, 16, 200, 64), (40, 1, 64, 200, 64)])
def test_scores(fw, case):
    args = scores_inputs(sum(case), *case)
    check_scores(fw.indexer_scores(*args), *args)


@pytest.mark.parametrize("case", [(400, 1, 64, 300, 64), (90, 5, 64, 1000, 64), (70, 3, 128, 700, 64), (30, 50, 32, 600, 64),
                                  (200, 2, 24, 900, 16), (3, 1, 64, 40000, 64)])
def test_scores_of_many_rows(fw, case):
    """More work than the chip holds at once, rows of every length among it (empty ones too), checked against
    the same rows scored a few at a time, and some of them against the reference."""
    q, w, codes, scales, table, lens, n = scores_inputs(sum(case), *case)
    got = fw.indexer_scores(q, w, codes, scales, table, lens, n)
    queries = case[1]
    for b in range(0, case[0], max(1, case[0] // 9)):
        part = q[b:b + 1], w[b:b + 1], codes, scales, table[b:b + 1], lens[b:b + 1], n
        few = fw.indexer_scores(*part)
        assert torch.equal(got[b * queries:(b + 1) * queries], few)
        if b % 2 == 0:
            check_scores(few, *part)
    for _ in range(3):
        assert torch.equal(fw.indexer_scores(q, w, codes, scales, table, lens, n), got)


def test_scores_of_every_length(fw):
    """No keys, one key, both sides of every border of pages and tiles, past the row, negative."""
    lens = [0, 1, 2, 63, 64, 65, 127, 128, 129, 191, 192, 255, 256, 257, 383, 384, 385, 399, 400, 401, 2**31 - 1,
            -1, -2**31, 300]
    args = scores_inputs(5, len(lens), 1, 64, 400, 64, lens)
    check_scores(fw.indexer_scores(*args), *args)
    args = scores_inputs(6, 4, 6, 64, 400, 64, lens)
    check_scores(fw.indexer_scores(*args), *args)


@pytest.mark.parametrize("layout", ["page", "row"])
@pytest.mark.parametrize("page_size", [64, 20, 1])
def test_scores_over_other_layouts(fw, layout, page_size):
    args = scores_inputs(7, 3, 2, 64, 500, page_size, layout=layout)
    if args[2].stride(0) % 16:  # pages of one row, 148 bytes apart
        with pytest.raises(ValueError, match="16 bytes"):
            fw.indexer_scores(*args)
        return
    check_scores(fw.indexer_scores(*args), *args)


def test_scores_table_stride_outputs_and_streams(fw):
    q, w, codes, scales, table, lens, n = scores_inputs(8, 3, 2, 64, 500, 64)
    ref = fw.indexer_scores(q, w, codes, scales, table, lens, n)
    wide = torch.full((3, table.shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    holder = torch.full((6 * n + 8,), 5.0, device="cuda")
    out = holder[3:3 + 6 * n].view(6, n)  # not on 16 bytes
    assert torch.equal(fw.indexer_scores(q, w, codes, scales, wide, lens, n, out=out), ref)
    assert (holder[:3] == 5).all() and (holder[3 + 6 * n:] == 5).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fw.indexer_scores(q, w, codes, scales, table, lens, n, stream=side)
    side.synchronize()
    assert torch.equal(got, ref)
    assert fw.indexer_scores(q[:0], w[:0], codes, scales, table[:0], lens[:0], n).shape == (0, n)
    for _ in range(3):  # the same bits every time
        assert torch.equal(fw.indexer_scores(q, w, codes, scales, table, lens, n), ref)


def test_scores_with_what_is_not_finite(fw):
    """A row with a NaN scale makes its own scores NaN and no others; so does a NaN weight.
    Past the length nothing of a key is seen, whatever the cache holds there."""
    q, w, codes, scales, table, lens, n = scores_inputs(9, 2, 1, 64, 300, 64, [300, 200])
    codes, scales = codes.clone(), scales.clone()
    t = table.cpu()
    bad = [(0, 5), (0, 299), (1, 199)]
    for b, j in bad + [(1, 200), (1, 299)]:
        codes[t[b, j // 64], j % 64] = float("nan")
        scales[t[b, j // 64], j % 64] = math.nan
    y = fw.indexer_scores(q, w, codes, scales, table, lens, n).cpu()
    nan = torch.zeros(2, n, dtype=torch.bool)
    for b, j in bad:
        nan[b, j] = True
    assert torch.equal(torch.isnan(y), nan) and (y[1, 200:] == -math.inf).all()
    w = w.clone()
    w[1, 0, 3] = math.nan
    y = fw.indexer_scores(q, w, codes, scales, table, lens, n).cpu()
    assert torch.isnan(y[1, :200]).all() and torch.equal(torch.isnan(y[0]), nan[0])


def test_scores_of_pages_outside_the_cache(fw):
    q, w, codes, scales, table, lens, n = scores_inputs(10, 2, 3, 64, 300, 64, [300] * 6)
    good = fw.indexer_scores(q, w, codes, scales, table, lens, n).cpu()
    table = table.clone()
    table[0, 1], table[1, 4], table[1, 0] = -1, codes.shape[0], 2**31 - 1
    y = fw.indexer_scores(q, w, codes, scales, table, lens, n).cpu()
    assert fw.indexer_guard_hits() > 0
    fw.indexer_reset_guard_hits()
    want = good.clone()
    want[0:3, 64:128] = want[3:6, 256:300] = want[3:6, 0:64] = -math.inf
    assert torch.equal(y, want)
    short = [100] * 3 + [200] * 3  # the last bad page of the second sequence lies past its length
    lens = torch.tensor(short, dtype=torch.int32).view(2, 3).cuda()
    table[0, 1], table[1, 0] = 0, 0
    fw.indexer_scores(q, w, codes, scales, table, lens, n)
    assert fw.indexer_guard_hits() == 0


def test_scores_refusals(fw):
    q, w, codes, scales, table, lens, n = scores_inputs(11, 2, 3, 64, 300, 64)
    ok = dict(q=q, weights=w, codes=codes, scales=scales, page_table=table, seq_lens=lens, row_len=n)
    for kw in (dict(q=q[..., :64]), dict(q=q.view(torch.uint8)), dict(q=q[0]), dict(q=q.transpose(0, 1)),
               dict(weights=w[:, :, :3]), dict(weights=w.half()), dict(row_len=0), dict(row_len=10**6),
               dict(page_table=table.long()), dict(page_table=table[:1]), dict(page_table=table[:1].expand(2, -1)),
               dict(seq_lens=lens[:, :2]), dict(seq_lens=lens.long()), dict(codes=codes[..., :64]),
               dict(out=torch.empty((6, n - 1)).cuda()), dict(out=torch.empty((6, n)).half().cuda()),
               dict(q=torch.empty((2, 3, 129, 128), dtype=E4M3, device="cuda"),
                    weights=torch.empty((2, 3, 129)).cuda())):
        a = dict(ok, **kw)
        with pytest.raises((ValueError, TypeError)):
            fw.indexer_scores(*(a.pop(k) for k in ("q", "weights", "codes", "scales", "page_table", "seq_lens",
                                                   "row_len")), **a)


# ---------------------------------------------------------------- together

def test_captured_step_replays_with_new_inputs(fw):
    """Rotation, write, quantise, scores, selection and read-back in one CUDA graph."""
    g = gen(12)
    b, h, n, size = 3, 64, 700, 64
    pages = -(-n // size)
    freqs, scale = fw.indexer_rotary_freqs(64)
    codes, scales, _ = make_cache(b * pages, size, 128)
    codes.copy_((torch.randn(codes.shape, generator=g) * 90).clamp(-448, 448).to(E4M3))
    scales.fill_(0.01)
    table = torch.randperm(b * pages, generator=g).view(b, pages).int().cuda()
    q, k = torch.empty(b, h, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(b, 128, dtype=torch.bfloat16, device="cuda")
    w, pos = torch.empty(b, h, device="cuda"), torch.empty(b, dtype=torch.int32, device="cuda")
    lens, slots = torch.empty(b, dtype=torch.int32, device="cuda"), torch.empty(b, dtype=torch.int32, device="cuda")

    def feed(seed):
        gg = gen(seed)
        q.copy_(torch.randn(q.shape, generator=gg))
        k.copy_(torch.randn(k.shape, generator=gg))
        w.copy_(torch.randn(w.shape, generator=gg))
        at = torch.randint(300, n, (b,), generator=gg)
        pos.copy_(at.int())
        lens.copy_((at + 1).int())
        slots.copy_((table.cpu().long()[torch.arange(b), at // size] * size + at % size).int())

    def step():
        qr = fw.indexer_rotary(q, pos, freqs, start=64, scale=scale)
        kr = fw.indexer_rotary(k, pos, freqs, start=64, scale=scale)
        fw.indexer_cache_write(kr, slots, codes, scales)
        q8, w8 = fw.indexer_quantise(qr, weights=w)
        s = fw.indexer_scores(q8[:, None], w8[:, None], codes, scales, table, lens[:, None], n)
        picked = fw.topk_transform_paged(s, lens, table, size, 64)
        return q8, w8, s, picked, fw.indexer_cache_read(codes, scales, picked)

    feed(1)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (2, 3):
        feed(seed)
        graph.replay()
        torch.cuda.synchronize()
        q8, w8, s, picked, rows = held
        check_scores(s, q8[:, None], w8[:, None], codes, scales, table, lens[:, None], n)
        for i in range(b):
            best = s[i].topk(64).indices.cpu()
            want = table[i].cpu().long()[best // size] * size + best % size
            assert set(picked[i].cpu().tolist()) == set(want.tolist())
        assert torch.equal(rows, fw.indexer_cache_read(codes, scales, picked))


def test_captured_backward(fw):
    """Forward and backward of the rotation in a graph of their own leaves."""
    x = torch.zeros((5, 3, 64), device="cuda", requires_grad=True)
    dy = torch.zeros((5, 3, 64), device="cuda")
    positions = torch.arange(5, dtype=torch.int32).cuda() * 100
    freqs, _ = fw.indexer_rotary_freqs(32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(fw.indexer_rotary(x, positions, freqs), x, dy)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = fw.indexer_rotary(x, positions, freqs)
        (grad,) = torch.autograd.grad(y, x, dy)
    for seed in (1, 2):
        with torch.no_grad():
            x.copy_(torch.randn(x.shape, generator=gen(seed)))
        dy.copy_(torch.randn(x.shape, generator=gen(seed + 9)))
        graph.replay()
        torch.cuda.synchronize()
        check(y, *rotary_ref(x.detach(), positions, freqs, "half", 0, 1.0, False))
        check(grad, *rotary_ref(dy, positions, freqs, "half", 0, 1.0, True))


def test_example_decodes(fw):
    """examples/indexer_decode.py: its last step's scores, selection and rows."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "indexer_decode.py")
    spec = importlib.util.spec_from_file_location("indexer_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.main(["--batch", "3", "--context", "300", "--k", "50", "--steps", "4"])
    ix = got["indexer"]
    assert ix.lens.tolist() == [300] * 3
    q = fw.indexer_rotary(ix.q, ix.lens - 1, ix.freqs, start=64, scale=ix.scale)
    q8, w = fw.indexer_quantise(q, weights=ix.weights)
    check_scores(got["scores"], q8[:, None], w[:, None], ix.codes, ix.scales, ix.page_table, ix.lens[:, None], 300)
    slot = ix.page_table.long()[:, torch.arange(300).cuda() // 64] * 64 + torch.arange(300).cuda() % 64
    want = slot.gather(1, got["scores"].topk(50, 1).indices)
    assert torch.equal(got["picked"].long().sort(1).values, want.sort(1).values)
    assert torch.equal(got["rows"], fw.indexer_cache_read(ix.codes, ix.scales, got["picked"]))


def test_calls_of_more_parts_than_one_launch_numbers(fw):
    """More than 2**30 rows: they are cut into launches, which have to fit together."""
    heads, tokens = 16384, 66000
    row = torch.randn((1, heads, 1), generator=gen(3)).to(torch.bfloat16).cuda()
    codes, scales = fw.indexer_quantise(row.expand(tokens, heads, 1))
    one = fw.indexer_quantise(row)
    assert same_quantised(*one, quantise_ref(row, "fp32"))
    for t in range(0, tokens, 4000):  # a piece at a time: comparisons make copies
        part = slice(t, t + 4000)
        assert bool((codes[part].view(torch.uint8) == one[0].view(torch.uint8)).all())
        assert bool((scales[part] == one[1]).all())
    del codes, scales
    cache = torch.randint(0, 120, (64, 16, 16), generator=gen(4), dtype=torch.uint8).cuda().view(E4M3)
    factors = torch.rand((64, 16, 1), generator=gen(5)).cuda()
    slots = torch.arange(1024, dtype=torch.int32).cuda()
    want = fw.indexer_cache_read(cache, factors, slots, dtype=torch.bfloat16)
    got = fw.indexer_cache_read(cache, factors, slots.repeat((1 << 20) + 3), dtype=torch.bfloat16)
    got = got.view(-1, 1024, 16)
    for r in range(0, got.shape[0], 1 << 17):
        assert bool((got[r:r + (1 << 17)] == want).all())


@pytest.mark.parametrize("seed", range(12))
def test_scores_of_drawn_shapes(fw, seed):
    """Shapes from the whole range, ragged, with pages of every kind."""
    import random
    rng = random.Random(seed)
    b, n, h = rng.randint(1, 40), rng.choice([1, 1, 2, 3, 5, 8, 40]), rng.choice([1, 8, 15, 16, 31, 48, 64, 65, 128])
    row_len, size = rng.randint(1, 5000), rng.choice([1, 2, 3, 12, 16, 48, 64, 128, 192, 256])
    args = scores_inputs(seed + 100, b, n, h, row_len, size, layout=rng.choice(["apart", "row"]))
    got = fw.indexer_scores(*args)
    q, w, codes, scales, table, lens, _ = args
    for i in {0, b // 2, b - 1}:
        check_scores(got[i * n:(i + 1) * n], q[i:i + 1], w[i:i + 1], codes, scales, table[i:i + 1], lens[i:i + 1], row_len)


def test_calls_on_two_streams_at_once(fw):
    """Scores and writes of two independent streams, overlapping in time, give what each gives alone."""
    jobs = []
    for seed, case in ((21, (150, 1, 64, 900, 64)), (22, (3, 40, 64, 2000, 64))):
        args = scores_inputs(seed, *case)
        x = torch.randn((5000, 128), generator=gen(seed)).to(torch.bfloat16).cuda()
        jobs.append((args, x, fw.indexer_scores(*args), fw.indexer_quantise(x), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for k, (args, x, _, _, stream) in enumerate(jobs):
            with torch.cuda.stream(stream):
                got[k].append((fw.indexer_scores(*args), fw.indexer_quantise(x)))
    torch.cuda.synchronize()
    for k, (_, _, scores, (codes, scales), _) in enumerate(jobs):
        for s, (c, f) in got[k]:
            assert torch.equal(s, scores) and torch.equal(f, scales)
            assert torch.equal(c.view(torch.uint8), codes.view(torch.uint8))


@pytest.mark.parametrize("case", [(64, 1, 64, 12000, 64), (1, 1, 64, 700000, 64), (40, 3, 64, 16000, 64), (9, 60, 32, 9000, 64),
                                  (300, 1, 24, 3000, 16), (2, 40, 128, 40000, 64), (700, 1, 8, 1100, 1)])
def test_scores_in_spans(fw, case):
    """Calls large enough that CTAs share the tiles out by the rows' lengths: mostly short rows, some empty, a few full;
    all rows empty; only the last one not."""
    b, n, _, row_len, _ = case
    g = gen(sum(case))
    short = (torch.rand((b, n), generator=g) ** 4 * row_len).int()
    full = torch.rand((b, 1), generator=g) < 0.1
    last = torch.zeros((b, n), dtype=torch.int32)
    last[-1, -1] = row_len - 3
    steps = (row_len - n + 1 + torch.arange(n, dtype=torch.int32)).clamp(min=0).expand(b, n).contiguous()
    for lens in (torch.where(full, row_len, short).int(), torch.zeros((b, n), dtype=torch.int32), last, steps):
        q, w, codes, scales, table, lens, _ = scores_inputs(sum(case), *case, lens=lens.tolist())
        got = fw.indexer_scores(q, w, codes, scales, table, lens, row_len)
        seen = torch.arange(row_len).cuda() < lens.view(-1, 1)
        assert torch.equal(got == -math.inf, ~seen)
        for i in range(0, b, max(1, b // 5)):  # a few at a time they are items in turn
            few = fw.indexer_scores(q[i:i + 1], w[i:i + 1], codes, scales, table[i:i + 1], lens[i:i + 1], row_len)
            assert torch.equal(got[i * n:(i + 1) * n], few)
        small = slice(0, min(n, 4))
        check_scores(got[small], q[:1, small], w[:1, small], codes, scales, table[:1], lens[:1, small], row_len)
