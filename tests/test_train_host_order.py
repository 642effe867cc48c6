"""Sizes that no grid can cover are refused before any CUDA call (no kernel launched)."""
import ctypes

import pytest
import torch

from gemm_epilogue_transformer_02_b200 import binding as C
from gemm_epilogue_transformer_02_b200.build import build

SHAPE = 2
P, Q, R, S = (ctypes.c_void_p(v) for v in (0x10000, 0x20000, 0x30000, 0x40000))
MOST = (1 << 31) - 8  # the largest feature size

# fake pointers: only where no kernel can launch
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: CPU-only check")


@pytest.fixture(scope="module")
def lib():
    build()
    return C.load_library()


def test_embed_grid(lib):
    assert lib.coda_embed(P, Q, 1.0, R, S, S, S, (1 << 31) - 1, MOST, 10, None) == SHAPE


@pytest.mark.parametrize("M,D,V,accumulate", [(1 << 14, MOST, 10, 0), (1 << 14, MOST, 10, 1),
                                              (1, 16384, (1 << 31) - 2, 0), (1, 16384, (1 << 31) - 2, 1)])
def test_embed_bwd_grid(lib, M, D, V, accumulate):
    assert lib.coda_embed_bwd(P, Q, 1.0, R, accumulate, S, (1 << 63) - 1, M, D, V, None) == SHAPE
    assert lib.coda_embed_bwd_workspace_size(M, D, V) == 0


def test_newton_schulz_longest_side(lib):
    """A sum over 2^29 takes longer than the waits for it last (0.25 us for 64 of them)."""
    f, size, c = lib.coda_newton_schulz, lib.coda_newton_schulz_workspace_size, (3.4445, -4.775, 2.0315)
    long = 1 << 28
    assert size(1, 8, long) > 0 and size(1, long, 8) > 0
    for m, n in ((8, long + 8), (long + 8, 8), (8, 1 << 29), (1 << 29, 16)):
        assert size(1, m, n) == 0
        assert f(P, Q, 1, m, n, 5, *c, 1e-7, R, (1 << 63) - 1, None) == SHAPE
