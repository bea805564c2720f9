"""The paged cache kernels' own CUDA source on the CPU (see test_paged_emulated.py), at the edges of
what their calls may meet."""

import subprocess

import numpy as np
import pytest
import torch

from tests import paged_ref as ref
from tests.test_paged_emulated import _bf16, _run, _strides


@pytest.fixture(scope="module")
def exes(tmp_path_factory):
    """late: as in test_paged_emulated.py; unordered: under ThreadSanitizer, with warps whose votes,
    shuffles, matrix loads and MMAs order no memory."""
    from tests.host_emu.build_emu import build_many
    try:
        return build_many(str(tmp_path_factory.mktemp("paged_edges")), {
            "late": ("prefix_kernel.cuh", "emu_paged_main.cpp", "emu_paged", ()),
            "unordered": ("prefix_kernel.cuh", "emu_paged_main.cpp", "emu_paged_tsan", ("EMU_UNORDERED",))})
    except FileNotFoundError:
        pytest.skip("g++ not available")


def _paged(exe, pre, q, k, v, table, lengths, H_kv, causal=True, window=0, fp8=False, ctas=3, prefix=None, hidden=False,
           files=(), scales=(0.0125, 0.01), second=False):
    """Runs the paged kernels, or (prefix = (page numbers, length, splits, keys form)) the shared form's;
    returns O, L and the status.  hidden: every grid's inputs appear with its wait; second: the paged
    grid's second CTA runs first."""
    B, H, N_q, d = q.shape
    ks, vs = scales if fp8 else (1.0, 1.0)
    args = ["shared" if prefix else "paged", B, H, H_kv, N_q, d, k.shape[2], k.shape[0], table.shape[1], causal, window,
            d ** -0.5, fp8, ks, vs, ctas, *_strides(k), *_strides(v)]
    inputs = dict(q=q, k=k, v=v, table=table, lengths=np.array(lengths, dtype=np.int32), **dict(files))
    if prefix:
        args += list(prefix[1:])
        inputs["pages"] = prefix[0]
    status = _run(exe, (["hidden"] if hidden else ["second"] if second else []) + args, inputs, pre)
    lse = torch.from_numpy(np.fromfile(pre + ".lse", dtype=np.float32)).reshape(B, H, N_q)
    return _bf16(pre + ".o", q.shape), lse, status


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_nothing_is_read_before_the_wait(exes, tmp_path, shared, fp8):
    """Every grid may be scheduled while the one before it runs, and sees what other grids have written
    (lengths, tables, queries, pages, partial results) only once it has waited for it."""
    gen = ref.rng(51)
    lengths, page, d = [150, 3, 70], 16, 64
    k, v, table, spare = ref.make_cache(gen, lengths, 2, page, d, fp8, spare=9)
    q = torch.randn(3, 4, 2, d, generator=gen).bfloat16()
    pages, prefix = spare.contiguous(), 140
    o, lse, status = _paged(exes["late"], str(tmp_path / "x"), q, k, v, table, lengths, 2, fp8=fp8,
                            prefix=(pages, prefix, 2, 1) if shared else None, hidden=True)
    assert status == 0
    ks, vs = (0.0125, 0.01) if fp8 else (1.0, 1.0)
    ref.assert_attention(o, lse, ref.attention(q, k, v, table, lengths, d ** -0.5, True, 0, ks, vs,
                                               prefix=(pages.tolist(), prefix) if shared else None))


@pytest.mark.parametrize("fp8", [False, True])
def test_lanes_meet_before_they_read_cleared_rows(exes, tmp_path, fp8):
    """V rows behind the mask are cleared by some lanes and read by others: no data race (a race
    makes the binary's exit status 66)."""
    if subprocess.run([exes["unordered"]], capture_output=True).returncode != 2:   # its answer to no arguments
        pytest.skip("ThreadSanitizer does not run here")
    gen = ref.rng(12)
    lengths, N_q, window = [21, 0, 50, 5], 3, 30
    k, v, table, q, want, hit = ref.poisoned(gen, lengths, N_q, window, 16, fp8)
    o, lse, status = _paged(exes["unordered"], str(tmp_path / "x"), q, k, v, table, lengths, 2, window=window, fp8=fp8)
    assert status == 0
    ref.assert_poisoned(o, lse, want, hit)


def sink(gen, gap, n, where, page=16, d=64):
    """n equal keys and one, with V = 0, whose score lies `gap` above theirs, in E4M3 pages of one head;
    the key stands first (where = 0) or last.  Returns (q, k, v, numbers, scales, O of the exact result)."""
    pages = -(-(n + 1) // page)
    k = torch.zeros(pages, 1, page, d).to(torch.float8_e4m3fn)
    v = torch.full((pages, 1, page, d), 1.5).to(torch.float8_e4m3fn)
    at = 0 if where == 0 else n
    k[at // page, 0, at % page, 0] = 8.0
    v[at // page, 0, at % page] = 0.0
    q = torch.zeros(1, 1, 1, d)
    q[..., 0] = gap           # the score: gap * 8 * k_scale / sqrt(64), with k_scale = 1
    w = n * np.exp(-float(gap))
    return q.bfloat16(), k, v, torch.arange(pages, dtype=torch.int32), (1.0, 1.0), 1.5 * w / (1 + w)


def assert_sink(o, lse, gap, n, want, lost):
    """The equal keys' weights are off by half an f16 step, 2^-11 of themselves or `lost` / 2 of the largest
    weight; scores and exponentials by 2^-16, for the weights and their sum; the result by half a bf16
    step."""
    bound = max(2.0 ** -11, lost / 2 * np.exp(float(gap))) + 2 * 2.0 ** -16 + 2.0 ** -8
    assert (o.double() / want - 1).abs().max() <= bound, (gap, float(o.flatten()[0]), want)
    assert abs(float(lse) - (gap + np.log1p(n * np.exp(-float(gap))))) <= 2.0 ** -16 + 2.0 ** -20 * gap


@pytest.mark.parametrize("where", [0, 1])
@pytest.mark.parametrize("gap", [14, 18, 22])
def test_small_weights_over_e4m3_pages(exes, tmp_path, gap, where):
    """Keys far below the largest score carry the result where the largest key's V is 0."""
    n = 799
    q, k, v, table, scales, want = sink(ref.rng(0), gap, n, where)
    o, lse, status = _paged(exes["late"], str(tmp_path / "x"), q, k, v, table[None], [n + 1], 1, fp8=True, scales=scales)
    assert status == 0
    assert_sink(o, lse, gap, n, want, 2.0 ** -39)


@pytest.mark.parametrize("where", [0, 1])
@pytest.mark.parametrize("gap", [14, 18])
def test_small_weights_over_an_e4m3_prefix(exes, tmp_path, gap, where):
    n = 450
    q, k, v, table, scales, want = sink(ref.rng(0), gap, n, where, page=64)
    o, lse, status = _paged(exes["late"], str(tmp_path / "x"), q, k, v, table[None, :1], [0], 1, fp8=True, scales=scales,
                            prefix=(table, n + 1, 1, 1))
    assert status == 0
    assert_sink(o, lse, gap, n, want, 2.0 ** -35)


@pytest.mark.parametrize("shared", [False, True])
def test_huge_scores_over_e4m3_pages(exes, tmp_path, shared):
    """Scores of 2^32: the largest weight stays within f16, whatever the rounding of its exponent."""
    gen = ref.rng(8)
    k, v, table, _ = ref.make_cache(gen, [100], 1, 16, 64, True, spare=0)
    q = (torch.randn(1, 3, 1, 64, generator=gen).clamp(-1, 1) * 60000).bfloat16()
    pages = table[0].contiguous()
    o, lse, status = _paged(exes["late"], str(tmp_path / "x"), q, k, v, table, [0 if shared else 100], 1, fp8=True,
                            scales=(6000.0, 0.01), prefix=(pages, 100, 1, 1) if shared else None)
    assert status == 0 and lse.isfinite().all()
    keys, values = (torch.from_numpy(ref.sequence(x, pages, 100)[0]) for x in (k, v))
    s = (q.double()[0, :, 0] @ keys.T) * 6000.0 / 8
    assert s.amax(1).min() > 2.0 ** 32
    rows = values[s.argmax(1)] * 0.01
    assert (o[0, :, 0].double() - rows).abs().max() <= 2.0 ** -7 * 4.48


def ragged_attention(q, k, v, table, lengths, counts, *args, **kw):
    """ref.attention() where sequence b has counts[b] new rows; padding gives O = 0 and L = -inf."""
    got = None
    for b, c in enumerate(counts):
        one = ref.attention(q[b:b + 1, :, :c], k, v, table[b:b + 1], lengths[b:b + 1], *args, **kw)
        got = got or [np.full((*q.shape[:x.ndim],), -np.inf if i == 1 else 0.0) for i, x in enumerate(one)]
        for x, y in zip(got, one):
            x[b, :, :c] = y[0]
    return got


RAGGED = [
    # lengths, counts, N_q, H, H_kv, page, causal, window, fp8, (prefix, splits, keys form)
    ([50, 7, 0, 130, 33], [2, 4, 0, 1, 0], 4, 4, 2, 16, True, 0, False, None),
    ([50, 7, 3, 130, 33], [2, 3, 3, 1, 0], 4, 4, 2, 48, True, 0, True, None),
    ([50, 7, 0, 130, 33], [2, 4, 0, 1, 3], 4, 12, 2, 16, True, 20, False, None),       # two row blocks
    ([50, 7, 0, 130, 33], [5, 4, 0, 1, 3], 5, 2, 1, 16, False, 9, True, None),
    ([50, 7, 0, 130], [2, 4, 0, 1], 4, 2, 1, 16, False, 0, False, None),
    ([5, 7, 0, 60], [2, 4, 0, 1], 4, 4, 2, 16, True, 0, False, (100, 1, 1)),
    ([5, 7, 0, 60], [3, 1, 0, 4], 4, 2, 1, 64, True, 0, True, (300, 2, 1)),
    ([3] * 9, [0, 1, 2] * 3, 2, 20, 1, 16, True, 0, False, (140, 2, 0)),               # 360 rows
]


@pytest.mark.parametrize("case", RAGGED, ids=range(len(RAGGED)))
def test_ragged_rows(exes, tmp_path, case):
    """A sequence's first counts[b] rows stand where an append with the same counts put them; what the
    padding rows hold does not matter."""
    lengths, counts, N_q, H, H_kv, page, causal, window, fp8, prefix = case
    gen = ref.rng(61 + N_q + page)
    need = -(-prefix[0] // page) if prefix else 0
    k, v, table, spare = ref.make_cache(gen, lengths, H_kv, page, 64, fp8, spare=need + 1)
    q = torch.randn(len(lengths), H, N_q, 64, generator=gen).bfloat16()
    scales = (0.0125, 0.01) if fp8 else (1.0, 1.0)
    pages = spare[:need].contiguous()
    want = ragged_attention(q, k, v, table, lengths, counts, 0.125, causal, window, *scales,
                            prefix=(pages.tolist(), prefix[0]) if prefix else None)
    for b, c in enumerate(counts):
        q[b, :, c:] = float("nan")
    o, lse, status = _paged(exes["late"], str(tmp_path / "x"), q, k, v, table, lengths, H_kv, causal, window, fp8, ctas=4,
                            prefix=(pages, *prefix) if prefix else None, files=dict(counts=np.array(counts, dtype=np.int32)))
    assert status == 0
    ref.assert_attention(o, lse, want, case)


@pytest.mark.parametrize("heads", [1, 4])
@pytest.mark.parametrize("axes", [1, 3])
def test_a_row_with_a_bad_position_is_not_stored_at_all(exes, tmp_path, axes, heads):
    """Not its V, not the part of it that does not turn, not the pairs of its other axes; the other rows are."""
    gen = ref.rng(70)
    lengths, N, H, H_kv, d, page, rot, n_angles = [20, 9], 4, 2, 1, 64, 16, 32, 30
    k_pages, v_pages, table, _ = ref.make_cache(gen, lengths, H_kv, page, d, False)
    q, k, v = (torch.randn(2, h, N, d, generator=gen).bfloat16() for h in (H, H_kv, H_kv))
    angle = torch.rand(n_angles, rot // 2, generator=gen)
    sections = [16] if axes == 1 else [4, 4, 8]
    positions = torch.randint(0, n_angles, (axes, 2, N), generator=gen, dtype=torch.int32)
    positions[axes - 1, 0, 1], positions[0, 1, 3] = n_angles, -1
    pre = str(tmp_path / "x")
    files = dict(q=q, k=k, v=v, kp=k_pages, vp=v_pages, table=table, lengths=np.array(lengths, dtype=np.int32),
                 cos=angle.cos(), sin=angle.sin(), positions=positions)
    status = _run(exes["late"], ["append", 2, H, H_kv, N, d, page, k_pages.shape[0], table.shape[1], rot, n_angles, axes,
                                 *(sections + [0] * 3)[:4], 0, 0, 1.0, 1.0, heads, 0, 1, *_strides(k_pages),
                                 *_strides(v_pages)], files, pre)
    assert status == 4
    good = positions.clone()
    good[axes - 1, 0, 1], good[0, 1, 3] = 0, 0
    out, q_bound, pools, bounds = ref.append(q, k, v, k_pages, v_pages, table, lengths, None, angle.cos(), angle.sin(), good,
                                             tuple(sections), False, 1.0, 1.0)
    for b, i in ((0, 1), (1, 3)):   # as they were: q_out's filling, the pages' contents
        out[b, :, i], slot = np.nan, lengths[b] - N + i
        for pool, bound, x in zip(pools, bounds, (k_pages, v_pages)):
            at = int(table[b, slot // page]), slice(None), slot % page
            pool[at], bound[at] = ref._np(x)[at], 0.0
    before = torch.full(q.shape, 0x4242, dtype=torch.int16).view(torch.bfloat16)
    got = [torch.from_numpy(np.fromfile(f"{pre}.{x}", dtype=np.uint8)).view(torch.bfloat16).reshape(k_pages.shape)
           for x in ("kp", "vp")]
    ref.assert_append(_bf16(pre + ".q_out", q.shape), *got, (out, q_bound, pools, bounds), before)


@pytest.mark.parametrize("ctas", [1, 3])
def test_too_long_lengths_are_reported_whoever_runs(exes, tmp_path, ctas):
    """The report does not depend on CTA 0 of the paged grid, whose work another CTA may take over."""
    gen = ref.rng(6)
    k, v, table, _ = ref.make_cache(gen, [64, 600], 1, 16, 64, False, width=38)
    table = table.clamp(min=0)
    q = torch.randn(2, 1, 1, 64, generator=gen).bfloat16()
    for lengths, expected in (([64, 600], 0), ([64, 609], 4)):
        o, lse, status = _paged(exes["late"], str(tmp_path / "x"), q, k, v, table, lengths, 1, ctas=ctas, second=True)
        assert status == expected
        ref.assert_attention(o, lse, ref.attention(q, k, v, table, [64, min(lengths[1], 608)], 0.125, True))


@pytest.mark.parametrize("bad", [-1, 5, -(1 << 31), (1 << 31) - 1])
def test_counts_out_of_range(exes, tmp_path, bad):
    """A count outside 0 .. N is read as the nearer of the two, and reported, by the append and the attention."""
    gen = ref.rng(80)
    lengths, N, counts = [20, 33], 4, [2, bad]
    taken = [2, min(max(bad, 0), N)]
    k_pages, v_pages, table, _ = ref.make_cache(gen, lengths, 1, 16, 64, False)
    q, k, v = (torch.randn(2, h, N, 64, generator=gen).bfloat16() for h in (2, 1, 1))
    counts = np.array(counts, dtype=np.int32)
    pre = str(tmp_path / "x")
    files = dict(q=q, k=k, v=v, kp=k_pages, vp=v_pages, table=table, lengths=np.array(lengths, dtype=np.int32),
                 cos=torch.ones(1), sin=torch.ones(1), counts=counts)
    status = _run(exes["late"], ["append", 2, 2, 1, N, 64, 16, k_pages.shape[0], table.shape[1], 0, 1, 0, 0, 0, 0, 0, 0, 0,
                                 1.0, 1.0, 1, 1, 0, *_strides(k_pages), *_strides(v_pages)], files, pre)
    assert status == 4
    want = ref.append(q, k, v, k_pages, v_pages, table, lengths, taken, None, None, None, (), False, 1.0, 1.0)
    got = [torch.from_numpy(np.fromfile(f"{pre}.{x}", dtype=np.uint8)).view(torch.bfloat16).reshape(k_pages.shape)
           for x in ("kp", "vp")]
    ref.assert_append(_bf16(pre + ".q_out", q.shape), *got, want, torch.full(q.shape, 0x4242, dtype=torch.int16).view(torch.bfloat16))
    o, lse, status = _paged(exes["late"], pre, q, k_pages, v_pages, table, lengths, 1, files=dict(counts=counts))
    assert status == 4
    ref.assert_attention(o, lse, ragged_attention(q, k_pages, v_pages, table, lengths, taken, 0.125, True))


@pytest.mark.parametrize("length", [-1, -(1 << 31)])
def test_a_negative_length_is_an_idle_slot(exes, tmp_path, length):
    """Nothing of its rows is stored, whatever the count, and it is no error."""
    gen = ref.rng(81)
    k_pages, v_pages, table, _ = ref.make_cache(gen, [20, 20], 1, 16, 64, False)
    q, k, v = (torch.randn(2, 1, 4, 64, generator=gen).bfloat16() for _ in range(3))
    pre = str(tmp_path / "x")
    files = dict(q=q, k=k, v=v, kp=k_pages, vp=v_pages, table=table, lengths=np.array([20, length], dtype=np.int32),
                 cos=torch.ones(1), sin=torch.ones(1))
    status = _run(exes["late"], ["append", 2, 1, 1, 4, 64, 16, k_pages.shape[0], table.shape[1], 0, 1, 0, 0, 0, 0, 0, 0, 0,
                                 1.0, 1.0, 1, 0, 0, *_strides(k_pages), *_strides(v_pages)], files, pre)
    assert status == 0
    want = ref.append(q, k, v, k_pages, v_pages, table, [20, 0], None, None, None, None, (), False, 1.0, 1.0)
    got = [torch.from_numpy(np.fromfile(f"{pre}.{x}", dtype=np.uint8)).view(torch.bfloat16).reshape(k_pages.shape)
           for x in ("kp", "vp")]
    ref.assert_append(_bf16(pre + ".q_out", q.shape), *got, want, torch.full(q.shape, 0x4242, dtype=torch.int16).view(torch.bfloat16))
