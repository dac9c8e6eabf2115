"""The indexer's operators at the edges of their contracts (needs a GB300): counts read while
other streams work, and what autograd and the allocator are owed."""

from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
LONG = 200_000_000  # cycles of torch.cuda._sleep: a tenth of a second


@pytest.fixture(scope="module")
def fw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_attention_indexer_sm_gb300 as p
    p.load_library()
    return p


@pytest.fixture(autouse=True)
def no_guard_hits(fw):
    torch.cuda.synchronize()
    fw.indexer_reset_guard_hits()
    fw.topk_reset_guard_hits()
    yield
    torch.cuda.synchronize()
    assert fw.indexer_guard_hits() == 0 and fw.topk_guard_hits() == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def make_cache(pages, size, dim=128):
    return (torch.zeros((pages, size, dim), device="cuda").to(E4M3),
            torch.zeros((pages, size, -(-dim // 128)), device="cuda"))


# ---------------------------------------------------------------- counts

def test_count_waits_for_other_streams(fw):
    """A bad slot met on a stream that is behind is in the count, and a reset comes after it."""
    codes, scales = make_cache(4, 8)
    x, slots = torch.ones((3, 128), device="cuda"), torch.tensor([-5, 1, 32], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG)
        fw.indexer_cache_write(x, slots, codes, scales)
    assert fw.indexer_guard_hits() == 2
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG)
        fw.indexer_cache_write(x, slots, codes, scales)
    fw.indexer_reset_guard_hits()
    torch.cuda.synchronize()
    assert fw.indexer_guard_hits() == 0


def test_topk_count_waits_for_other_streams(fw):
    """The same of the top-k's count: a row that needs more pages than its table's stride (through the C
    ABI, as the binding refuses such a table)."""
    lib = fw.load_library()
    n, size, pages, k = 8192, 64, 100, 64
    scores = torch.randn((2, n), generator=gen(1)).cuda()
    lens = torch.tensor([n, 6400], dtype=torch.int32, device="cuda")
    table = torch.arange(2 * pages, dtype=torch.int32, device="cuda").view(2, pages)
    out = torch.empty((2, k), dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()

    def call():
        torch.cuda._sleep(LONG)
        st = lib.topk_transform_paged(scores.data_ptr(), n, lens.data_ptr(), table.data_ptr(), pages, size, 2, k,
                                      out.data_ptr(), None, 0, side.cuda_stream)
        assert st == 0

    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call()
    assert fw.topk_guard_hits() == 1
    with torch.cuda.stream(side):
        call()
    fw.topk_reset_guard_hits()
    torch.cuda.synchronize()
    assert fw.topk_guard_hits() == 0


# ---------------------------------------------------------------- outputs on other streams

def pending_block(nbytes):
    """Frees a block of the current stream's pool that queued work has still to write; its address."""
    block = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(LONG)
    block.fill_(0x5A)
    return block.data_ptr()


def on_side_calls(fw):
    """(name, bytes of each output, call) of everything that makes its own outputs, on inputs that are ready."""
    g = gen(2)
    n, k, size = 1000, 50, 20
    x = torch.randn((200, 8, 128), generator=g).to(torch.bfloat16).cuda()
    positions = torch.arange(200, dtype=torch.int32).cuda()
    freqs, _ = fw.indexer_rotary_freqs(64)
    codes, scales = make_cache(200, size)
    flat = torch.randperm(200 * size, generator=g).int().cuda()
    fw.indexer_cache_write(torch.randn((200 * size, 128), generator=g).cuda(), flat, codes, scales)
    q, w = fw.indexer_quantise(x[:4], weights=torch.ones((4, 8), device="cuda"))
    table = torch.randperm(200, generator=g).int().cuda().view(4, 50)
    lens = torch.tensor([1000, 1, 500, 999], dtype=torch.int32).cuda()
    return [
        ("rotary", [x.numel() * 2], lambda **kw: (fw.indexer_rotary(x, positions, freqs, **kw),)),
        ("quantise", [x.numel(), 200 * 8 * 4], lambda **kw: fw.indexer_quantise(x, **kw)),
        ("read", [flat.numel() * 128 * 2], lambda **kw: (fw.indexer_cache_read(codes, scales, flat, **kw),)),
        ("scores", [4 * n * 4], lambda **kw: (
            fw.indexer_scores(q[:, None], w[:, None], codes, scales, table, lens[:, None], n, **kw),)),
    ]


@pytest.mark.parametrize("which", range(4))
def test_output_made_on_another_stream(fw, which):
    """A call on a stream that is not behind the current one: its output is no block that work queued on the
    current stream has still to write."""
    name, sizes, call = on_side_calls(fw)[which]
    want = call()
    side = torch.cuda.Stream()
    call(stream=side)  # loads what is loaded once
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    pending = {pending_block(nbytes) for nbytes in sizes}
    got = call(stream=side)
    assert not pending & {t.data_ptr() for t in got}, name
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), name


def test_output_read_on_the_current_stream_and_dropped(fw):
    """An output that work queued on the current stream still reads is not handed out again to the stream it
    was made on."""
    x = torch.ones((4096, 128), device="cuda")
    positions = torch.zeros(4096, dtype=torch.int32, device="cuda")
    freqs, _ = fw.indexer_rotary_freqs(64)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = fw.indexer_rotary(x, positions, freqs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(LONG)
    seen = y.clone()
    at = y.data_ptr()
    del y
    with torch.cuda.stream(side):
        other = torch.full((4096, 128), 9.0, device="cuda")
        assert other.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(seen, x)


@pytest.mark.parametrize("which", ["raw", "paged", "ragged", "window", "grouped", "sorted", "split"])
def test_topk_output_made_on_another_stream(fw, which):
    """The same of the top-k's calls, their workspaces among them."""
    b, n, k = 8, 4000, 64
    scores = torch.randn((b, n), generator=gen(6)).cuda()
    lens = torch.full((b,), n, dtype=torch.int32, device="cuda")
    starts = (torch.arange(b, dtype=torch.int32) * n).cuda()
    table = torch.arange(b * 125, dtype=torch.int32, device="cuda").view(b, 125)
    problem = {"form": "raw", "k": k, "scores": scores, "seq_lens": lens, "sorted": which == "sorted"}
    calls = {
        "raw": lambda **kw: fw.topk_transform_raw(scores, lens, k, **kw),
        "paged": lambda **kw: fw.topk_transform_paged(scores, lens, table, 32, k, **kw),
        "ragged": lambda **kw: fw.topk_transform_ragged(scores.view(-1), starts, lens, k, **kw),
        "window": lambda **kw: fw.topk_transform_window(scores, torch.zeros_like(lens), lens, k, **kw),
        "grouped": lambda **kw: fw.topk_transform_grouped([problem], **kw)[0],
        "sorted": lambda **kw: fw.topk_transform_grouped([problem], **kw)[0],
        "split": lambda **kw: fw.topk_transform_raw(scores, lens, k, **kw),
    }
    before = fw.topk_set_chip_split(2 if which == "split" else 1)
    try:
        call, spare = calls[which], fw.topk_workspace_bytes(b, n, k) if which == "split" else 0
        want = call().sort(1).values
        side = torch.cuda.Stream()
        call(stream=side)
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        pending = {pending_block(nbytes) for nbytes in (b * k * 4, max(spare, 1 << 16))}
        got = call(stream=side)
        assert got.data_ptr() not in pending
        torch.cuda.synchronize()
        assert torch.equal(got.sort(1).values, want)
        with torch.cuda.stream(side):  # an output dropped while the current stream still reads it
            torch.cuda._sleep(1)
        side.synchronize()
        torch.cuda._sleep(LONG)
        seen, at = got.clone(), got.data_ptr()
        del got
        with torch.cuda.stream(side):
            assert torch.zeros((b, k), dtype=torch.int32, device="cuda").data_ptr() != at
        torch.cuda.synchronize()
        assert torch.equal(seen.sort(1).values, want)
    finally:
        fw.topk_set_chip_split(before)


# ---------------------------------------------------------------- autograd

def test_forward_mode_is_refused(fw):
    """No forward derivative is dropped silently."""
    import torch.autograd.forward_ad as fwd
    x, v = torch.randn((4, 2, 16), generator=gen(3)).cuda(), torch.ones((4, 2, 16), device="cuda")
    positions = torch.arange(4, dtype=torch.int32).cuda()
    freqs, _ = fw.indexer_rotary_freqs(8)
    codes, scales = make_cache(2, 4, 16)
    slots = torch.arange(4, dtype=torch.int32).cuda()
    side = torch.cuda.Stream()
    with fwd.dual_level():
        dual = fwd.make_dual(x, v)
        with pytest.raises(ValueError, match="forward-mode"):
            fw.indexer_rotary(dual, positions, freqs)
        with pytest.raises(ValueError, match="forward-mode"):
            fw.indexer_rotary(dual, positions, freqs, stream=side)
        with pytest.raises(ValueError, match="forward-mode"):
            fw.indexer_rotary(x, positions, freqs, out=dual)
        with pytest.raises(ValueError, match="forward-mode"):
            fw.indexer_quantise(dual)
        with pytest.raises(ValueError, match="forward-mode"):
            fw.indexer_cache_write(dual[:, 0], slots, codes, scales)
        plain = fw.indexer_rotary(fwd.unpack_dual(dual).primal, positions, freqs)  # without its tangent
        with torch.no_grad():  # backward is off, forward is not
            with pytest.raises(ValueError, match="forward-mode"):
                fw.indexer_rotary(dual, positions, freqs)
        with torch.inference_mode():  # both are off
            assert torch.equal(fw.indexer_rotary(dual, positions, freqs), plain)
    assert torch.equal(fw.indexer_rotary(x, positions, freqs), plain)


def test_writing_over_a_saved_tensor_is_noticed(fw):
    """An output that another operation saved for its backward: autograd says that it was changed."""
    positions = torch.arange(4, dtype=torch.int32).cuda()
    freqs, _ = fw.indexer_rotary_freqs(8)
    rows = torch.randn((4, 16), generator=gen(4)).cuda()
    codes, scales = make_cache(2, 2, 16)
    slots = torch.arange(4, dtype=torch.int32).cuda()
    q = torch.zeros((1, 1, 2, 128), device="cuda").to(E4M3)
    wide = make_cache(2, 2)
    table, lens = torch.arange(2, dtype=torch.int32).cuda()[None], torch.full((1, 1), 4, dtype=torch.int32).cuda()
    held = torch.zeros((4, 1), device="cuda")
    spare = torch.empty((4, 16), device="cuda").to(E4M3)
    calls = [
        ((4, 16), lambda t: fw.indexer_rotary(rows, positions, freqs, out=t)),
        ((4, 16), lambda t: fw.indexer_rotary(t, positions, freqs, out=t)),
        ((4, 16), lambda t: fw.indexer_rotary(rows, positions, freqs, out=t, stream=torch.cuda.current_stream())),
        ((4, 1), lambda t: fw.indexer_quantise(rows, codes=spare, scales=t)),
        ((2, 2, 1), lambda t: fw.indexer_cache_write(rows, slots, codes, t)),
        ((4, 16), lambda t: fw.indexer_cache_read(codes, scales, slots, dtype=torch.float32, out=t)),
        ((1, 4), lambda t: fw.indexer_scores(q, torch.ones((1, 1, 2), device="cuda"), *wide, table, lens, 4, out=t)),
    ]
    for shape, write in calls:
        saved = torch.ones(shape, device="cuda")
        leaf = torch.ones(shape, device="cuda", requires_grad=True)
        y = (leaf * saved).sum()
        write(saved)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    for t, write in ((spare, lambda: fw.indexer_quantise(rows, codes=spare, scales=held)),
                     (codes, lambda: fw.indexer_cache_write(rows, slots, codes, scales))):
        before = t._version
        write()
        assert t._version == before + 1
    with torch.inference_mode():
        out = torch.empty((4, 16), device="cuda")
    assert fw.indexer_rotary(rows, positions, freqs, out=out) is out  # an inference tensor has no version


def test_gradients_that_do_not_exist_are_refused(fw):
    """The 8-bit operators have no gradient: an input that asks for one is not detached silently."""
    rows = torch.randn((4, 2, 128), generator=gen(5)).cuda()
    w = torch.ones((4, 2), device="cuda")
    codes, scales = make_cache(2, 4)
    slots = torch.arange(4, dtype=torch.int32).cuda()
    q8, w8 = fw.indexer_quantise(rows, weights=w)
    table, lens = torch.arange(2, dtype=torch.int32).cuda()[None], torch.full((1, 4), 8, dtype=torch.int32).cuda()

    def scores(weights=w8, s=scales, out=None):
        return fw.indexer_scores(q8[None], weights[None], codes, s, table, lens, 8, out=out)

    def leaf(t):
        return t.clone().requires_grad_(True)

    calls = [lambda: fw.indexer_quantise(leaf(rows)), lambda: fw.indexer_quantise(rows, weights=leaf(w)),
             lambda: fw.indexer_quantise(rows, weights=w, scales=leaf(w)),
             lambda: fw.indexer_cache_write(leaf(rows)[:, 0], slots, codes, scales),
             lambda: fw.indexer_cache_write(rows[:, 0], slots, codes, leaf(scales)),
             lambda: fw.indexer_cache_read(codes, leaf(scales), slots),
             lambda: fw.indexer_cache_read(codes, scales, slots, dtype=torch.float32,
                                           out=leaf(torch.zeros((4, 128), device="cuda"))),
             lambda: scores(weights=leaf(w8)), lambda: scores(s=leaf(scales)),
             lambda: scores(out=leaf(torch.zeros((4, 8), device="cuda")))]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call()
    with torch.no_grad():
        for call in calls:
            call()
    assert torch.equal(scores(weights=leaf(w8).detach()), scores())


# ---------------------------------------------------------------- scores

@pytest.mark.parametrize("page_size,strided", [(64, False), (64, True), (3, False), (1, False)])
def test_every_nan_scale_makes_its_scores_nan(fw, page_size, strided):
    """Every bit pattern of a NaN, those that a kernel might use as a mark among them."""
    n = 24
    pages = -(-n // page_size)
    patterns = [0x7fc00000, 0x7fc00001, 0x7f800001, 0x7fffffff, -1, -0x400000, -0x3fffff, 0x7fc00002]
    codes = torch.full((pages, page_size, 128), 1.0, device="cuda").to(E4M3)
    bits = torch.full((pages, page_size, 2 if strided else 1), 0x3f800000, dtype=torch.int32, device="cuda")
    for i, v in enumerate(patterns):
        j = 3 * i
        bits[j // page_size, j % page_size] = v
    scales = bits.view(torch.float32)[..., :1]
    q, w = torch.ones((1, 1, 4, 128), device="cuda").to(E4M3), torch.ones((1, 1, 4), device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    got = fw.indexer_scores(q, w, codes, scales, table, torch.full((1, 1), n, dtype=torch.int32, device="cuda"), n)
    want = torch.full((1, n), 512.0)
    want[0, ::3] = math.nan
    assert torch.equal(got.cpu().nan_to_num(-1.0), want.nan_to_num(-1.0))


def scores_inputs(seed, b, n, h, row_len, page_size, lens=None):
    g = gen(seed)
    pages = -(-row_len // page_size)
    codes = (torch.randn((b * pages, page_size, 128), generator=g) * 90).clamp(-448, 448).to(E4M3).cuda()
    scales = (torch.rand((b * pages, page_size, 1), generator=g) * 0.02 + 0.001).cuda()
    table = torch.randperm(b * pages, generator=g).view(b, pages).int().cuda()
    q = (torch.randn((b, n, h, 128), generator=g) * 90).clamp(-448, 448).to(E4M3).cuda()
    w = torch.randn((b, n, h), generator=g).cuda()
    if lens is None:
        lens = torch.randint(0, row_len + 1, (b, n), generator=g).int()
    return q, w, codes, scales, table, lens.cuda(), row_len


@pytest.mark.parametrize("case", [(3, 1, 64, 1000, 64), (2, 2, 128, 600, 64), (5, 4, 64, 700, 48), (2, 33, 16, 500, 1),
                                  (200, 1, 64, 6000, 64), (40, 5, 32, 24000, 64)])
def test_a_call_that_gives_up_has_no_wrong_scores(fw, case):
    """What was computed around a wait that ran out is NaN, and so is everything where the kernel cannot start;
    both are counted. Later calls are as before."""
    lib = fw.load_library()
    args = scores_inputs(sum(case), *case)
    want = fw.indexer_scores(*args)
    seen = torch.arange(case[3], device="cuda") < args[5].view(-1, 1)
    for mode in (1, 2):
        out = torch.zeros_like(want)
        assert lib.indexer_set_scores_failure(mode) == 0
        try:
            fw.indexer_scores(*args, out=out)
            torch.cuda.synchronize()
        finally:
            assert lib.indexer_set_scores_failure(0) == mode
        assert fw.indexer_guard_hits() > 0
        fw.indexer_reset_guard_hits()
        assert bool(torch.isnan(out[seen]).all())
        if mode == 1:
            assert bool((out[~seen] == -math.inf).all())
        else:
            assert bool(torch.isnan(out).all())
        assert torch.equal(fw.indexer_scores(*args), want)


KEY_TILE, ITEM_COST, MOST_SLICES = 128, 4, 8192  # csrc/indexer_scores.cu: kTile, kItemCost, kMaxSpanSlices


def in_spans(b, n, h, row_len):
    """Whether CTAs of a call share its tiles out by the rows' lengths, or take items in turn."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    columns = next(c for c in (16, 32, 64, 128) if h <= c)
    slices, tiles = b * -(-n // min(256 // columns, n)), -(-row_len // KEY_TILE)
    return (slices <= MOST_SLICES and slices * (tiles + ITEM_COST) < 2**31 and slices * tiles >= sms * (32 + slices // 64))


@pytest.mark.parametrize("n,h,row_len,page_size", [
    (1, 64, 12000, 64), (1, 64, 12001, 1), (1, 64, 11999, 3), (16, 16, 12000, 64), (16, 16, 9000, 1), (4, 64, 9001, 1),
    (4, 64, 9000, 3), (3, 128, 6000, 20), (3, 128, 6001, 1), (8, 32, 9000, 48), (9, 24, 9000, 1), (5, 64, 7000, 128)])
def test_spans_against_items_in_turn(fw, n, h, row_len, page_size):
    """As many sequences as it takes for spans, of every mix of lengths: the same bits as each sequence by itself,
    in items in turn, and some rows against 64 bits."""
    from test_indexer_gpu import check_scores
    b = next(b for b in range(1, MOST_SLICES) if in_spans(b, n, h, row_len)) * 9 // 8 + 1
    assert in_spans(b, n, h, row_len) and not in_spans(1, n, h, row_len)
    g = gen(n + h + page_size)
    q, w, codes, scales, table, _, _ = scores_inputs(n * h + page_size, b, n, h, row_len, page_size)
    short = (torch.rand((b, n), generator=g) ** 4 * row_len).int()
    mixed = torch.where(torch.rand((b, 1), generator=g) < 0.2, row_len, short).int()
    mixed[::7] = 0
    last = torch.zeros((b, n), dtype=torch.int32)
    last[-1, -1] = row_len - 3
    steps = (row_len - n + 1 + torch.arange(n, dtype=torch.int32)).expand(b, n).contiguous()
    for lens in (mixed, torch.zeros((b, n), dtype=torch.int32), last, steps):
        lens = lens.cuda()
        got = fw.indexer_scores(q, w, codes, scales, table, lens, row_len)
        seen = torch.arange(row_len, device="cuda") < lens.view(-1, 1)
        assert torch.equal(got == -math.inf, ~seen)
        for i in range(b):
            few = fw.indexer_scores(q[i:i + 1], w[i:i + 1], codes, scales, table[i:i + 1], lens[i:i + 1], row_len)
            assert torch.equal(got[i * n:(i + 1) * n], few), i
        for i in {0, b // 2, b - 1}:
            k = i % n  # one query of the sequence
            check_scores(got[i * n + k:i * n + k + 1], q[i:i + 1, k:k + 1], w[i:i + 1, k:k + 1], codes, scales,
                         table[i:i + 1], lens[i:i + 1, k:k + 1], row_len)
