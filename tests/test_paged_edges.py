"""The paged cache operators on the GPU at the edges of what their calls may meet (see
test_paged_edges_emulated.py for the same on the CPU)."""

import pytest
import torch

from tests import paged_ref as ref
from tests.test_paged_edges_emulated import assert_sink, ragged_attention, sink
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


RAGGED = [
    # lengths after the append, counts, N, H, H_kv, d, page, window, fp8, prefix
    ([50, 4, 0, 130, 2999], [2, 4, 0, 1, 3], 4, 8, 2, 128, 16, 0, False, 0),
    ([50, 4, 0, 130, 2999], [2, 4, 0, 1, 3], 4, 8, 2, 128, 48, 0, True, 0),
    ([50, 7, 3, 130, 2999], [5, 0, 2, 1, 4], 5, 20, 1, 64, 16, 70, False, 0),
    ([50, 7, 3, 130, 2999], [5, 0, 2, 1, 4], 5, 14, 2, 64, 32, 70, True, 0),
    ([600, 33], [600, 1], 600, 4, 4, 64, 16, 0, False, 0),               # prompts, one of a single token
    ([40, 21], [11, 3], 13, 6, 2, 256, 64, 0, False, 0),
    ([40, 4, 0, 130], [2, 4, 0, 1], 4, 8, 2, 128, 64, 0, False, 700),
    ([40, 4, 0, 130], [2, 4, 0, 1], 4, 8, 2, 128, 64, 0, True, 700),
    ([3] * 60, [0, 1, 2] * 20, 2, 28, 4, 64, 16, 0, False, 1300),
    ([3, 40], [0, 3], 3, 68, 1, 256, 16, 0, True, 500),
]


@pytest.mark.parametrize("case", RAGGED, ids=range(len(RAGGED)))
def test_append_then_attention_of_a_ragged_batch(fa, case):  # noqa: F811
    """Padded rows through append_kv(counts) and the attention after it with the same lengths and counts,
    eager and captured; padding rows give 0 and -inf, whatever they hold."""
    lengths, counts, N, H, H_kv, d, page, window, fp8, prefix = case
    gen = ref.rng(90 + N + d)
    B, need = len(lengths), -(-prefix // page)
    k_pages, v_pages, table, spare = ref.make_cache(gen, lengths, H_kv, page, d, fp8, spare=need + 1)
    q, k, v = (torch.randn(B, h, N, d, generator=gen).bfloat16() for h in (H, H_kv, H_kv))
    angle = torch.rand(3200, d // 2, generator=gen) * 6.3
    for b, c in enumerate(counts):
        for x in (q, k, v):
            x[b, :, c:] = float("nan")
    scales = dict(k_scale=0.0125, v_scale=0.01) if fp8 else {}
    kp, vp, tab, pages, n, c = _cuda(k_pages, v_pages, table.clamp(min=0), spare[:need].contiguous(), _i32(lengths), _i32(counts))
    q, k, v, cos, sin = _cuda(q, k, v, angle.cos(), angle.sin())

    def step():
        qr = fa.append_kv(k, v, kp, vp, tab, n, counts=c, q=q, q_out=q.clone(), cos=cos, sin=sin, **scales)
        if prefix:
            return qr, *fa.decode_shared(qr, kp, vp, pages, prefix, tab, n, causal=True, counts=c, **scales)
        return qr, *fa.decode_paged(qr, kp, vp, tab, n, causal=True, window=window, counts=c, **scales)

    qr, o, lse = step()
    assert fa.check_status() == 0
    want = ragged_attention(qr.cpu(), kp.cpu(), vp.cpu(), table, lengths, counts, d ** -0.5, True, window, *scales.values(),
                            prefix=(spare[:need].tolist(), prefix) if prefix else None)
    ref.assert_attention(o, lse, want, case)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    graph.replay()
    assert torch.equal(out[1], o) and torch.equal(out[2], lse)
    # without counts every row is a new one, as before
    full = torch.full_like(c, N)
    args = (q.nan_to_num(), kp, vp)
    for more in ({}, dict(counts=full)):
        got = fa.decode_shared(*args, pages, prefix, tab, n, causal=True, **more, **scales)
        first = got if not more else first
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    assert fa.check_status() == 0


def test_counts_are_checked(fa):  # noqa: F811
    k = torch.zeros(2, 1, 16, 64, device="cuda", dtype=torch.bfloat16)
    q = torch.zeros(2, 1, 1, 64, device="cuda", dtype=torch.bfloat16)
    table, n = _cuda(_i32([[0], [1]]), _i32([3, 4]))
    for bad in (n.long(), n[:1], n.cpu(), torch.zeros(4, device="cuda", dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            fa.decode_paged(q, k, k, table, n, counts=bad)
        with pytest.raises(ValueError):
            fa.decode_shared(q, k, k, table[0], 10, table, n, counts=bad)


@pytest.mark.parametrize("N", [4, 700])   # one head a thread, and four
def test_a_row_with_a_bad_position_is_not_stored_at_all(fa, N):  # noqa: F811
    gen = ref.rng(70 + N)
    H, H_kv, d, page = 32, 8, 128, 16
    table = torch.arange(2 * (-(-N // page)), dtype=torch.int32).reshape(2, -1)
    kp, vp = (torch.full((table.numel(), H_kv, page, d), 3.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q, k, v = (torch.randn(2, h, N, d, generator=gen).bfloat16().cuda() for h in (H, H_kv, H_kv))
    positions = torch.randint(0, 99, (3, 2, N), generator=gen, dtype=torch.int32)
    bad = [(0, 0, 1), (1, 1, 3), (2, 0, N - 1)]
    for (a, b, i), x in zip(bad, (99, -1, 1 << 30)):
        positions[a, b, i] = x
    angle = torch.rand(99, d // 4, generator=gen).cuda()
    n, q_out = _i32([N, N]).cuda(), torch.full_like(q, 7.0)
    fa.append_kv(k, v, kp, vp, table.cuda(), n, q=q, q_out=q_out, cos=angle.cos(), sin=angle.sin(),
                 positions=positions.cuda(), sections=(8, 12, 12))
    assert fa.STATUS_NAMES[fa.check_status()] == "FA_ERR_INDEX"
    missing = torch.zeros(2, N, dtype=torch.bool)
    for _, b, i in bad:
        missing[b, i] = True
    for x, old in ((q_out, 7.0), (kp, 3.0), (vp, 3.0)):
        rows = x.cpu().transpose(1, 2) if x is q_out else \
            x.cpu().transpose(1, 2).reshape(2, -1, H_kv, d)[:, :N]
        assert torch.equal((rows == old).all(-1).all(-1), missing)
        assert not (rows == old).all(-1)[~missing].any()


def test_counts_out_of_range_are_reported(fa):  # noqa: F811
    gen = ref.rng(80)
    lengths, N = [20, 33], 4
    k_pages, v_pages, table, _ = ref.make_cache(gen, lengths, 1, 16, 64, False)
    q, k, v = (torch.randn(2, h, N, 64, generator=gen).bfloat16() for h in (2, 1, 1))
    for bad in (-1, 5, -(1 << 31), (1 << 31) - 1):
        taken = [2, min(max(bad, 0), N)]
        kp, vp = k_pages.cuda(), v_pages.cuda()
        c, n = _i32([2, bad]).cuda(), _i32(lengths).cuda()
        q_out = torch.full_like(q, 7.0).cuda()
        fa.append_kv(*_cuda(k, v), kp, vp, table.cuda(), n, counts=c, q=q.cuda(), q_out=q_out)
        assert fa.STATUS_NAMES[fa.check_status()] == "FA_ERR_INDEX"
        ref.assert_append(q_out, kp, vp, ref.append(q, k, v, k_pages, v_pages, table, lengths, taken, None, None, None, (), False,
                                                    1.0, 1.0), torch.full_like(q, 7.0))
        o, lse = fa.decode_paged(q.cuda(), kp, vp, table.cuda(), n, causal=True, counts=c)
        assert fa.STATUS_NAMES[fa.check_status()] == "FA_ERR_INDEX"
        ref.assert_attention(o, lse, ragged_attention(q, kp.cpu(), vp.cpu(), table, lengths, taken, 0.125, True))
    assert fa.check_status() == 0
