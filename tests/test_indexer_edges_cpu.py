"""The indexer's operators at the edges of their contracts, without a GPU."""

import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")


# ---------------------------------------------------------------- frequencies

def by_pairs(rot, base, factor, trained, fast, slow):
    """The blend by the pair's index, one pair at a time."""
    def index(turns):  # where a pair turns so often within the trained positions
        return rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))

    low, high = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rot - 1)
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if i <= low:
            share = 0.0
        elif i >= high:
            share = 1.0
        else:
            share = (i - low) / (high - low)
        out.append(f * (1 - share) + f / factor * share)
    return out


@pytest.mark.parametrize("how", [(64, 10000.0, 40.0, 4096, 32.0, 1.0), (128, 10000.0, 4.0, 32768, 32.0, 1.0),
                                 (64, 500000.0, 8.0, 8192, 4.0, 1.0), (64, 10000.0, 16.0, 100, 32.0, 1.0),
                                 (2, 10000.0, 4.0, 4096, 32.0, 1.0), (64, 10000.0, 4.0, 4096, 1.0001, 1.0),
                                 (32, 1000.0, 4.0, 10**9, 32.0, 1.0)])
def test_yarn_frequencies_blended_by_the_pairs_index(how):
    import sparse_attention_indexer_sm_gb300 as fw
    rot, base, factor, trained, fast, slow = how
    f, scale = fw.indexer_rotary_freqs(rot, base, scaling="yarn", factor=factor, original_len=trained, beta_fast=fast,
                                       beta_slow=slow, ramp="pairs", device="cpu")
    # each frequency: a power, a quotient, two products and a sum in 64 bits, of numbers that are all positive
    torch.testing.assert_close(f, torch.tensor(by_pairs(*how), dtype=torch.float64), rtol=64 * 2.0 ** -53, atol=0)
    assert math.isclose(scale, 0.1 * math.log(factor) + 1.0)


def test_yarn_ramps():
    import sparse_attention_indexer_sm_gb300 as fw
    plain, _ = fw.indexer_rotary_freqs(64, device="cpu")
    kw = dict(scaling="yarn", factor=40.0, original_len=4096, device="cpu")
    turns, _ = fw.indexer_rotary_freqs(64, **kw)
    pairs, _ = fw.indexer_rotary_freqs(64, ramp="pairs", **kw)
    assert torch.equal(turns, fw.indexer_rotary_freqs(64, ramp="turns", **kw)[0])
    # pair 16 of 64 columns: 6 of the 13 steps from pair 10 to pair 23; 6.52 turns of 32 down to 1
    assert math.isclose((pairs / plain)[16].item(), 1 - 6 / 13 * (1 - 1 / 40), rel_tol=1e-12)
    share = (4096 * 0.01 / (2 * math.pi) - 1) / 31
    assert math.isclose((turns / plain)[16].item(), share + (1 - share) / 40, rel_tol=1e-12)
    with pytest.raises(ValueError, match="ramp"):
        fw.indexer_rotary_freqs(64, ramp="other", **kw)


# ---------------------------------------------------------------- build

@pytest.mark.parametrize("compiler", ["false", "no-such-compiler"])
def test_library_stands_without_the_binding(compiler, tmp_path, monkeypatch):
    """A binding that does not compile ends the build with an error, but after the library is linked."""
    from sparse_attention_indexer_sm_gb300 import build
    stub = tmp_path / "bin" / "nvcc"  # writes the file that follows -o
    stub.parent.mkdir()
    stub.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\necho "$@" > "$2"\n')
    stub.chmod(0o755)
    out = tmp_path / "_build"
    monkeypatch.setattr(build, "BUILD_DIR", str(out))
    monkeypatch.setattr(build, "LIB_PATH", str(out / "libtopk_transform.so"))
    monkeypatch.setattr(build, "nvcc", lambda: str(stub))
    monkeypatch.setenv("CXX", compiler)
    with pytest.raises(RuntimeError, match="compiler failed"):
        build.build()
    assert (out / "libtopk_transform.so").exists() and not os.path.exists(build.binding_path())
    with monkeypatch.context() as m:  # no PyTorch: the library alone
        m.setattr(build, "_pytorch", lambda: False)
        m.delattr(build, "binding_path")
        assert build.build(force=True) == build.build() == build.LIB_PATH
    monkeypatch.setenv("CXX", str(stub))
    assert build.build() == build.LIB_PATH and os.path.exists(build.binding_path())


def test_binding_belongs_to_its_interpreter_and_pytorch():
    from sparse_attention_indexer_sm_gb300 import build
    name = os.path.basename(build.binding_path())
    assert sys.implementation.cache_tag in name and torch.__version__ in name


def test_failure_mode_of_scores():
    from sparse_attention_indexer_sm_gb300 import build
    build.build()
    import sparse_attention_indexer_sm_gb300 as fw
    lib = fw.load_library()
    assert [lib.indexer_set_scores_failure(m) for m in (1, 2, 3, 0)] == [0, 1, 2, 0]
