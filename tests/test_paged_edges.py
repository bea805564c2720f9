"""The paged cache operators on the GPU at the edges of what their calls may meet (see
test_paged_edges_emulated.py for the same on the CPU)."""

import pytest
import torch

from tests import paged_ref as ref
from tests.test_paged_edges_emulated import assert_sink, sink
from tests.test_paged_parity import _cuda, _i32, fa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("where", [0, 1])
@pytest.mark.parametrize("gap", [14, 16, 18, 20, 22])
def test_small_weights_over_e4m3_pages(fa, gap, where, d):  # noqa: F811
    """Keys far below the largest score carry the result where the largest key's V is 0."""
    n = 1999
    q, k, v, table, (ks, vs), want = sink(ref.rng(0), gap, n, where, d=d)
    q, k, v, table, length = _cuda(q, k, v, table, _i32([n + 1]))
    o, lse = fa.decode_paged(q, k, v, table[None], length, scale=0.125, k_scale=ks, v_scale=vs)
    assert_sink(o.cpu(), lse.cpu(), gap, n, want, 2.0 ** -39)
    if gap <= 20:
        for H in (1, 70):   # both forms of the prefix kernel
            o, lse = fa.decode_shared(q.expand(3, H, -1, -1).contiguous(), k, v, table, n + 1, table[None, :1].expand(3, -1).contiguous(),
                                      torch.zeros(3, dtype=torch.int32, device="cuda"), scale=0.125, k_scale=ks, v_scale=vs)
            assert (lse == lse[0, 0]).all() and (o == o[0, 0]).all()
            assert_sink(o[:1, :1].cpu(), lse[:1, :1].cpu(), gap, n, want, 2.0 ** -35)
    assert fa.check_status() == 0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_huge_scores_over_e4m3_pages(fa, d):  # noqa: F811
    """Scores of 2^32: the largest weight stays within f16."""
    gen = ref.rng(8)
    k, v, table, _ = ref.make_cache(gen, [300], 1, 16, d, True, spare=0)
    q = (torch.randn(1, 3, 1, d, generator=gen).clamp(-1, 1) * 60000).bfloat16()
    keys, values = (torch.from_numpy(ref.sequence(x, table[0].tolist(), 300)[0]) for x in (k, v))
    s = (q.double()[0, :, 0] @ keys.T) * 6000.0 * d ** -0.5
    assert s.amax(1).min() > 2.0 ** 32
    rows = values[s.argmax(1)] * 0.01
    q, k, v, table, n = _cuda(q, k, v, table, _i32([300]))
    for o, lse in (fa.decode_paged(q, k, v, table, n, k_scale=6000.0, v_scale=0.01),
                   fa.decode_shared(q, k, v, table[0].contiguous(), 300, table, n * 0, k_scale=6000.0, v_scale=0.01)):
        assert lse.isfinite().all()
        assert (o.cpu().double()[0, :, 0] - rows).abs().max() <= 2.0 ** -7 * 4.48
    assert fa.check_status() == 0
