"""The paged cache kernels' own CUDA source on the CPU (see test_paged_emulated.py), at the edges of
what their calls may meet."""

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
           files=(), scales=(0.0125, 0.01)):
    """Runs the paged kernels, or (prefix = (page numbers, length, splits, keys form)) the shared form's;
    returns O, L and the status."""
    B, H, N_q, d = q.shape
    ks, vs = scales if fp8 else (1.0, 1.0)
    args = ["shared" if prefix else "paged", B, H, H_kv, N_q, d, k.shape[2], k.shape[0], table.shape[1], causal, window,
            d ** -0.5, fp8, ks, vs, ctas, *_strides(k), *_strides(v)]
    inputs = dict(q=q, k=k, v=v, table=table, lengths=np.array(lengths, dtype=np.int32), **dict(files))
    if prefix:
        args += list(prefix[1:])
        inputs["pages"] = prefix[0]
    status = _run(exe, (["hidden"] if hidden else []) + args, inputs, pre)
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
    gen = ref.rng(12)
    lengths, N_q, window = [21, 0, 50, 5], 3, 30
    k, v, table, q, want, hit = ref.poisoned(gen, lengths, N_q, window, 16, fp8)
    o, lse, status = _paged(exes["unordered"], str(tmp_path / "x"), q, k, v, table, lengths, 2, window=window, fp8=fp8)
    assert status == 0
    ref.assert_poisoned(o, lse, want, hit)
