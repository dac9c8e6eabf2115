"""Edges of the layer norm, the appends to a block-scaled cache and the attention over it (needs a
GB300): means of widths whose reciprocal fp32 does not have, codes at borders between two of them,
NaN codes wherever the work is cut, caches without pages, captured gradients."""

from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
from test_indexer_attention_gpu import (  # noqa: E402
    MANY, append_ref, attention_ref, ints, make_cache, make_case, same, slots_of)

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
E4M3 = torch.float8_e4m3fn
TYPES = [torch.bfloat16, torch.float16, torch.float32]


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
    assert fw.indexer_guard_hits() == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------- layer norm

# widths of every split of the rows over lanes, most of them without an exact reciprocal: by pieces of 16 bytes, value by
# value, and long rows of both kinds
DIMS = [24, 112, 200, 1000, 1536, 3584, 7168, 8200, 20000, 3, 31, 127, 1001, 5001]
ROWS = [200.0, 1000.0, -7.0, 0.0703125, 3.0, 1.0 / 3.0, -60000.0]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", DIMS)
def test_norm_of_constant_rows(fw, dim, dtype):
    """A constant row is its shift, and gives the weight no gradient, to the last bit. (The mean that the row's sum gives is
    off by a few steps of fp32; the differences from it are exact, all alike and a whole number of steps, so what it lacks is
    known to within 2^-22 of those few steps, and the corrected mean is the row's value.)"""
    x = torch.tensor(ROWS).to(dtype)[:, None].expand(-1, dim).contiguous().cuda().requires_grad_(True)
    g = gen(dim)
    w = torch.randn(dim, generator=g).cuda().requires_grad_(True)
    b = torch.randn(dim, generator=g).to(dtype).float().cuda()
    dy = torch.randn((len(ROWS), dim), generator=g).to(dtype).cuda()
    y = fw.indexer_layer_norm(x, w, b, eps=1e-6)
    assert torch.equal(y, b.to(dtype).expand_as(y))
    assert not fw.indexer_layer_norm(x.detach(), w.detach(), eps=1e-6).any()
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    assert not dw.any()
    # dx = (gw - mean(gw)) / sqrt(eps): products, their sum of up to 40 + dim / 256 additions in a row, the mean, the root
    gw = dy.double().cpu() * w.detach().double().cpu()
    rstd = 1e-6 ** -0.5
    want = (gw - gw.mean(-1, keepdim=True)) * rstd
    tol = rstd * U * (6 * gw.abs() + (50 + dim / 256) * gw.abs().mean(-1, keepdim=True))
    half, tiny = torch.finfo(dtype).eps / 2, torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    fits = want.abs() < 0.9 * torch.finfo(dtype).max
    assert ((dx.double().cpu() - want).abs() <= tol + (want.abs() + tol) * half + tiny)[fits].all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", DIMS)
def test_norm_of_nearly_constant_rows(fw, dim, dtype):
    """All values but a few are one large number. The mean is rounded once to fp32, whatever the width: it is off by half a step,
    and by DEPTH additions of differences that are small."""
    depth = 50 + dim / 256
    x = torch.tensor(ROWS).to(dtype)[:, None].repeat(1, dim)
    g = gen(dim + 1)
    at = torch.randint(0, dim, (len(ROWS), max(1, dim // 50)), generator=g)
    x.scatter_(1, at, (x.gather(1, at).float() * (1 + 4 * torch.finfo(dtype).eps)).to(dtype))
    w = torch.randn(dim, generator=g)
    eps = 1e-6
    y = fw.indexer_layer_norm(x.cuda(), w.cuda(), eps=eps).double().cpu()
    x, w = x.double(), w.double()
    mean = x.mean(-1, keepdim=True)
    d = x - mean
    var = d.square().mean(-1, keepdim=True)
    rstd = (var + eps).rsqrt()
    first = (depth + 2) * U * x.abs().mean(-1, keepdim=True)  # how far the first mean may be off
    spread = d.abs().mean(-1, keepdim=True) + first
    e_mean = U * mean.abs() + (depth + 4) * U * spread
    # squares around the first mean, less the square of what it lacked
    e_var = (depth + 8) * U * (var + first.square()) + 4 * U * first * spread * (depth + 4)
    r_rstd = 0.5 * e_var / (var + eps) + 4 * U
    n = d * rstd
    tol = (rstd * (e_mean + U * d.abs()) + n.abs() * (r_rstd + r_rstd.square() + 3 * U)) * w.abs()
    want = n * w
    half, tiny = torch.finfo(dtype).eps / 2, torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    worst = ((y - want).abs() / (tol + (want.abs() + tol) * half + tiny)).max().item()
    assert worst <= 1.0, f"off by {worst:.3g} of the tolerance"


# ---------------------------------------------------------------- appends

def borders():
    """Halfway between neighbouring e4m3 values, normal ones."""
    grid = torch.arange(8, 127, dtype=torch.uint8).view(E4M3).float().double()
    return (grid[1:] + grid[:-1]) / 2


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [4, 64])
def test_append_under_scales_that_are_no_powers_of_two(fw, block, dtype):
    """Blocks whose scale from before is any number: quotients within a step of fp32 of a border between two codes, above it,
    below it and on it, become the code that is nearest to the real quotient."""
    pages, heads, dim, rows = 300, 2, 128, 3
    g = gen(block)
    codes, scales = make_cache(g, pages, block, heads, dim, block)
    mids = borders()
    shape = (pages, heads)
    at = torch.rand(shape, generator=g).add(1.0).to(dtype).double() * 2.0 ** -3  # a value of the row's type, and its border
    m = mids[torch.randint(24, 109, shape, generator=g)]  # below 224: half of what the scale holds, so none grows
    s = (at / m).float()
    # that value times powers of two, and for fp32 its neighbours too; all of them within what the scale holds
    x = at[:, None, :, None] * torch.exp2(torch.randint(-5, 1, (pages, rows, heads, dim), generator=g).double())
    x = x * (torch.randint(0, 2, x.shape, generator=g).double() * 2 - 1)
    x = x.float()
    if dtype == torch.float32:
        x = torch.nextafter(x, torch.full_like(x, 1e9) * torch.randint(-1, 2, x.shape, generator=g).float() + x)
    x = x.to(dtype).flatten(0, 1).cuda()
    starts = (torch.arange(pages + 1) * rows).int().cuda()
    lens = torch.full((pages,), rows + 1, dtype=torch.int32).cuda()  # one position is there already
    table = torch.randperm(pages, generator=g).int().view(pages, 1)
    scales[table[:, 0].long(), 0] = s.cuda()
    args = (x, starts, lens, table.cuda(), codes, scales)
    ref = append_ref(*args)
    assert torch.equal(ref[1][:, 0][table[:, 0].long()], s.double())  # the scales stay
    fw.indexer_cache_append(*args)
    same(codes, scales, ref)


@pytest.mark.parametrize("dtype", TYPES)
def test_append_where_any_scale_grows(fw, dtype):
    """Codes from before that come near a border between two codes as their scale, any number, gives way to a power of two."""
    pages, heads, dim, block = 300, 2, 128, 8
    g = gen(5)
    codes, scales = make_cache(g, pages, block, heads, dim, block)
    grid = torch.arange(8, 127, dtype=torch.uint8).view(E4M3).float().double()
    mids = borders()
    c = grid[torch.randint(0, len(grid), (pages, heads), generator=g)]
    s = (mids[torch.randint(0, len(mids), (pages, heads), generator=g)] / c).float()
    s = s * torch.exp2(-6 - torch.frexp(s)[1].float())  # 2^-7 to 2^-6: the power of two takes its place
    scales[:, 0] = s.cuda()
    codes[:, :3] = (c[:, None, :, None] * (torch.randint(0, 2, (pages, 3, heads, dim), generator=g).double() * 2 - 1)).float().to(E4M3).cuda()
    x = torch.full((pages, heads, dim), 5.0).to(dtype).cuda()
    starts = torch.arange(pages + 1).int().cuda()
    lens = torch.full((pages,), 4, dtype=torch.int32).cuda()
    table = torch.arange(pages, dtype=torch.int32).view(pages, 1).cuda()
    args = (x, starts, lens, table, codes, scales)
    ref = append_ref(*args)
    assert (ref[1] == 2.0 ** -6).all()
    fw.indexer_cache_append(*args)
    same(codes, scales, ref)


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("size", [16, 5])
@pytest.mark.parametrize("group,dim", [(3, 64), (20, 128), (40, 128), (100, 128), (200, 112), (4, 256)])
def test_attention_over_a_cache_without_pages(fw, group, dim, size):
    """Every slot and page id is outside it: nothing is seen, and each that is asked for is counted."""
    codes, scales = torch.empty((0, size, 2, dim), dtype=torch.uint8, device="cuda").view(E4M3), torch.empty((0, 1, 2), device="cuda")
    cache = (codes, scales, codes.clone(), scales.clone())
    q = torch.randn((3, 2, 2 * group, dim), generator=gen(1)).bfloat16().cuda()
    slots = torch.full((6, 300), -1, dtype=torch.int32)
    slots[0, 7], slots[1, ::2], slots[3, 299], slots[5, 0] = 0, 3, 2**31 - 1, -2
    out, lse = fw.indexer_attention(q, *cache, slots=slots.cuda(), return_lse=True)
    assert not out.any() and (lse == -math.inf).all()
    assert fw.indexer_guard_hits() >= 153
    fw.indexer_reset_guard_hits()
    assert not fw.indexer_attention(q, *cache, slots=torch.full_like(slots, -1).cuda()).any()
    assert fw.indexer_guard_hits() == 0  # none is asked for
    table = torch.tensor([[0, 1, 2, 3], [-1, 7, 0, 0], [0, 0, 0, 0]], dtype=torch.int32).cuda()
    lens = torch.tensor([[3 * size, 4 * size], [1, 2], [0, 0]], dtype=torch.int32).cuda()
    out, lse = fw.indexer_attention(q, *cache, page_table=table, seq_lens=lens, return_lse=True)
    assert not out.any() and (lse == -math.inf).all()
    assert fw.indexer_guard_hits() >= 5
    fw.indexer_reset_guard_hits()


NAN_CODES = [  # batch, queries, kv heads, group, dim, pages of a sequence, page size, block
    (2, 3, 2, 2, 128, 60, 16, 16), (3, 1, 1, 8, 64, 40, 16, 4), (1, 2, 2, 9, 128, 50, 16, 16), (2, 1, 1, 30, 128, 30, 7, 7),
    (1, 5, 1, 13, 64, 40, 16, 16), (2, 1, 2, 14, 256, 30, 16, 16), (1, 4, 1, 5, 192, 20, 5, 1), (2, 1, 2, 40, 128, 50, 16, 16),
    (1, 9, 1, 7, 112, 60, 16, 2), (2, 1, 1, 100, 128, 40, 16, 16), (1, 50, 2, 4, 128, 30, 16, 16), (1, 130, 1, 2, 80, 40, 16, 16)]


@pytest.mark.parametrize("softmax_scale", [0.1, 4.0])
@pytest.mark.parametrize("dtype", TYPES[:2])
@pytest.mark.parametrize("case", NAN_CODES)
def test_attention_a_nan_code_of_a_value_stays_in_its_column(fw, case, dtype, softmax_scale):
    """The formula's own result: that column of the queries that see the key is NaN, however little the key weighs, wherever the
    work is cut and whatever other queries of the tile see; other columns, queries and the logarithm are as without it."""
    batch, queries, kv, group, dim, width, size, block = case
    g, q, k, v, table = make_case(sum(case) + 1, *case, dtype)
    length = width * size
    lens = (ints(g, length // 2, length + 1, (batch, 1)) - queries + 1 + torch.arange(queries)).int()
    lens[0] += length - lens[0, -1]
    clean = v[0].clone()
    spoiled = v[0].view(torch.uint8)
    for b in range(batch):  # a few keys anywhere, the first, and those around each query's last
        at = torch.cat([torch.tensor([0]), torch.randint(0, length, (4,), generator=g), (lens[b, ::3].long() - 1), lens[b, -1:].long()])
        for j in at.clamp(0, length - 1).tolist():
            slot = int(slots_of(table[b], size, length)[j])
            h, col = int(ints(g, 0, kv, ())), int(ints(g, 0, dim, ()))
            spoiled[slot // size, slot % size, h, col] = 0x7f + 128 * (j % 2)
            clean.view(torch.uint8)[slot // size, slot % size, h, col] = 0
    nan = v[0].cpu().float().isnan().flatten(0, 1)

    def compare(out, got, sees):
        ref, tol, lse, lse_tol = attention_ref(q.flatten(0, 1), k, (clean, v[1]), sees, softmax_scale)
        want = torch.stack([nan[sees(r)].any(0).repeat_interleave(group, 0) for r in range(batch * queries)])
        out, got = out.double().cpu().flatten(0, 1), got.double().cpu().flatten(0, 1)
        assert want.any() and torch.equal(out.isnan(), want)
        eps = torch.finfo(dtype).eps
        bound = tol + (ref.abs() + tol) * eps / 2 + torch.finfo(dtype).smallest_normal * eps
        assert (((out - ref).abs() <= bound) | want).all()
        assert ((got - lse).abs() <= lse_tol).all()

    args = dict(softmax_scale=softmax_scale, return_lse=True)
    whole = lambda r: slots_of(table[r // queries], size, int(lens[r // queries, r % queries]))  # noqa: E731
    compare(*fw.indexer_attention(q, *k, *v, page_table=table.cuda(), seq_lens=lens.cuda(), **args), whole)
    slots = torch.full((batch * queries, length), -1, dtype=torch.int32)
    for r in range(batch * queries):  # the same rows as picks in another order, some places empty
        mine = whole(r)
        slots[r, torch.randperm(length, generator=g)[:len(mine)]] = mine.int()
    compare(*fw.indexer_attention(q, *k, *v, slots=slots.cuda(), **args), lambda r: slots[r][slots[r] >= 0].long())


@pytest.mark.parametrize("dtype", TYPES[:2])
@pytest.mark.parametrize("case", MANY + [(300, 1, 2, 8, 128, 4, 16, 16), (200, 1, 1, 30, 128, 5, 16, 16), (200, 2, 1, 16, 64, 5, 7, 7)])
def test_attention_nan_codes_in_many_tiles_of_a_cta(fw, case, dtype):
    """To the last bit what the same call gives with 0 in their place, but for NaN in these columns of the queries that see them:
    nothing goes from one tile of a CTA to the next ones. In every run."""
    batch, queries, kv, group, dim, width, size, block = case
    g, q, k, v, table = make_case(sum(case) + 2, *case, dtype)
    length = width * size
    lens = (ints(g, 0, length + 1, (batch, 1)) - queries + 1 + torch.arange(queries)).int()
    args = dict(page_table=table.cuda(), seq_lens=lens.cuda(), return_lse=True)
    codes = v[0].view(torch.uint8)
    place = torch.rand((batch, length), generator=g) < 1.5 / length  # one or two of a sequence's keys, many sequences none
    place[::3] = False
    want = torch.zeros((batch, queries, kv, dim), dtype=torch.bool)
    put = []
    for b, j in place.nonzero().tolist():
        slot, h, col = int(slots_of(table[b], size, length)[j]), int(ints(g, 0, kv, ())), int(ints(g, 0, dim, ()))
        put.append((slot // size, slot % size, h, col))
        want[b, :, h, col] |= lens[b] > j
    at = tuple(torch.tensor(i).cuda() for i in zip(*put))
    codes[at] = 0
    out, lse = fw.indexer_attention(q, *k, *v, **args)
    codes[at] = 0xff
    assert want.any()
    want = out.masked_fill(want.repeat_interleave(group, 2).cuda(), math.nan)
    for _ in range(20):
        got, other = fw.indexer_attention(q, *k, *v, **args)
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))
        assert torch.equal(other, lse)


# ---------------------------------------------------------------- captured gradients

@pytest.mark.parametrize("made", ["in the capture", "before it"])
@pytest.mark.parametrize("name", ["norm", "rotary"])
def test_captured_backward_to_a_graph_of_the_default_stream(fw, name, made):
    """Inputs made from a leaf that such a graph holds: the backward is refused, before torch meets the default stream; the
    forward alone can be captured, and all of it once that graph is gone."""
    leaf = torch.randn((30, 64), generator=gen(3)).cuda().requires_grad_(True)
    w, dy = torch.randn(64, generator=gen(4)).cuda(), torch.randn((30, 64), generator=gen(5)).cuda()
    freqs, _ = fw.indexer_rotary_freqs(64)
    positions = torch.arange(30, dtype=torch.int32).cuda()
    call = {"norm": lambda x: fw.indexer_layer_norm(x, w), "rotary": lambda x: fw.indexer_rotary(x, positions, freqs)}[name]
    held = leaf * 3.0
    want = call(leaf.detach() * 3.0)
    for wanted in ("leaf", "all"):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            x = held if made == "before it" else leaf * 3.0
            y = call(x)
            with pytest.raises(RuntimeError, match="gradient graph"):
                if wanted == "leaf":
                    torch.autograd.grad(y, leaf, dy)
                else:
                    y.backward(dy)
            y = y.detach()
        graph.replay()
        assert torch.equal(y, want) and leaf.grad is None
        del x
    want = torch.autograd.grad(call(held), leaf, dy)[0]  # nothing is captured: as ever
    del held
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(call(leaf * 3.0), leaf, dy)[0]
    graph.replay()
    assert torch.equal(got, want)


def test_captured_backward_past_a_graph_of_the_default_stream(fw):
    """Only the nodes that the backward goes on to matter: a weight's gradient alone, though the rows come from a held graph."""
    leaf = torch.randn((30, 64), generator=gen(6)).cuda().requires_grad_(True)
    w = torch.randn(64, generator=gen(7)).cuda().requires_grad_(True)
    dy = torch.randn((30, 64), generator=gen(8)).cuda()
    held = leaf * 3.0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(fw.indexer_layer_norm(held, w), w, dy)[0]
    graph.replay()
    assert torch.equal(got, torch.autograd.grad(fw.indexer_layer_norm(held, w), w, dy)[0])
