"""More calls of the paged cache that are refused on the host (no GPU needed: addresses are made up, and
validation must end before any use)."""

import pytest
import torch

from exact_io_aware_77_b200 import _lib, paged
from tests.test_paged_refusals import A, _append, _cache, _name, _paged, _shared, lib  # noqa: F401


@pytest.mark.parametrize("call", [_paged, _shared], ids=["paged", "shared"])
@pytest.mark.parametrize("scale,k_scale", [(1e-30, 1e-20), (1e30, 1e20), (1e38, 3.0)])
def test_score_factors_out_of_range_are_refused(lib, call, scale, k_scale):  # noqa: F811
    """scale * k_scale gone to 0 or past fp32's range: every score would be NaN."""
    assert _name(call(cache=_cache(fp8=1, k_scale=k_scale), scale=scale)) == "FA_ERR_SCALE"


@pytest.mark.parametrize("call", [_paged, _shared], ids=["paged", "shared"])
def test_scales_past_the_exponentials_base_are_refused(lib, call):  # noqa: F811
    assert _name(call(scale=3e38)) == "FA_ERR_SCALE"     # scale * log2(e) is past fp32's range


@pytest.mark.parametrize("kw", [dict(k_scale=1e-39), dict(v_scale=1e-39)])
def test_scales_without_an_inverse_are_refused(lib, kw):  # noqa: F811
    """1 / scale past fp32's range: zeros would become NaN codes."""
    assert _name(_append(cache=_cache(fp8=1, **kw))) == "FA_ERR_SCALE"


def test_ragged_forwards_refuse_like_the_plain_ones(lib):  # noqa: F811
    """counts may be left out, and must be aligned; the masks, shapes and scratch are checked as ever."""
    c, ws = A + 65536, 1 << 40

    def paged(counts, window=0, ws_bytes=ws):
        return _name(_lib.fa_fwd_paged_ragged(A, _cache(), A, counts, A, A, 2, 8, 4, 1, 128, None, 0.1, 1, window, c, ws_bytes, None))

    def shared(counts, prefix=1000, ws_bytes=ws):
        return _name(_lib.fa_fwd_shared_ragged(A, _cache(), A, prefix, A, counts, A, A, 2, 8, 4, 1, 128, None, 0.1, 1, c, ws_bytes,
                                               None))
    for call in (paged, shared):
        assert call(A + 2) == "FA_ERR_ALIGN"
        assert call(A, ws_bytes=100) == "FA_ERR_WORKSPACE"
    assert paged(A, window=-1) == "FA_ERR_MASK" and shared(A, prefix=-1) == "FA_ERR_SHAPE"


def test_scales_of_bf16_pages_are_refused():
    """They would be ignored, and a cache read as if it were unscaled."""
    k, t = torch.empty(5, 4, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 3, dtype=torch.int32)
    for scales in ((0.5, 1.0), (1.0, 2.0), (float("nan"), 1.0)):
        with pytest.raises(ValueError):
            paged._cache(k, k, t, 2, 64, -1, *scales)
        paged._cache(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn), t, 2, 64, -1, *scales)


def test_sizes_past_32_bits_are_refused():
    """The library takes ints: 2^32 + 1 must not reach it as 1."""
    for at in range(5):
        sizes = [2, 8, 4, 1, 128]
        sizes[at] += 1 << 32
        for call in (paged.paged_workspace_size, lambda *s: paged.shared_workspace_size(*s, 100)):
            with pytest.raises(ValueError):
                call(*sizes)
    pages = torch.zeros(1, dtype=torch.int32).expand(1 << 18)
    assert paged._prefix_length(100, pages, 32768) == 100
    for n in (1 << 32, (1 << 32) + 100, -1, (1 << 33) + 1):
        with pytest.raises(ValueError):
            paged._prefix_length(n, pages, 32768)
    with pytest.raises(ValueError):
        paged.shared_workspace_size(2, 8, 4, 1, 128, 1 << 32)


def test_the_last_tokens_that_a_block_could_index_are_refused(lib):  # noqa: F811
    """A block of the append has room for up to 64 tokens: indices past the last one must not wrap round."""
    for n in ((1 << 31) - 1, (1 << 31) - 64):
        assert _name(_append(B=1, H=0, q=0, q_out=0, H_kv=1, N=n, d=64)) == "FA_ERR_SHAPE"
