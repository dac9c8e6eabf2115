"""The indexer's operators at the edges of their contracts (needs a GB300): counts read while
other streams work, and what autograd and the allocator are owed."""

from __future__ import annotations

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
