"""Host-side checks of the calls around the GEMM chain (no kernel launched):
argument errors with their status codes, workspace sizes, the binding's checks."""
import ctypes

import pytest
import torch

from gemm_epilogue_transformer_02_b200 import binding as C
from gemm_epilogue_transformer_02_b200.build import build

OK, NULL, SHAPE, ALIGN, WS = 0, 1, 2, 3, 4
P, Q, R, S = (ctypes.c_void_p(v) for v in (0x10000, 0x20000, 0x30000, 0x40000))
MIS = ctypes.c_void_p(0x30008)  # 8-byte aligned only
BIG = 1 << 40

# fake pointers: only where no kernel can launch
no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: CPU-only check")


@pytest.fixture(scope="module")
def lib():
    build()
    return C.load_library()


@no_gpu_only
def test_embed_refusals(lib):
    f = lib.coda_embed
    assert f(P, Q, 1.0, R, S, S, S, 0, 64, 10, None) == OK
    assert f(None, Q, 1.0, R, S, S, S, 4, 64, 10, None) == NULL
    assert f(P, None, 1.0, R, S, S, S, 4, 64, 10, None) == NULL
    assert f(P, Q, 1.0, R, None, None, None, 4, 64, 10, None) == NULL   # no output
    assert f(P, Q, 1.0, None, None, S, None, 4, 64, 10, None) == NULL   # hg needs gamma
    for M, D, V in ((-1, 64, 10), (4, 60, 10), (4, 0, 10), (4, 64, 0), (4, 64, 1 << 31), (1 << 31, 64, 10)):
        assert f(P, Q, 1.0, R, S, S, S, M, D, V, None) == SHAPE
    for i in (0, 1, 3, 4, 5, 6):
        a = [P, Q, 1.0, R, S, S, S]
        a[i] = MIS
        assert f(*a, 4, 64, 10, None) == ALIGN


@no_gpu_only
def test_embed_bwd_refusals(lib):
    f, size = lib.coda_embed_bwd, lib.coda_embed_bwd_workspace_size
    n = size(4, 64, 10)
    assert n >= 2 * 4 * 8 + 2 * 64 * 4
    assert size(4, 64, 1 << 20) >= (1 << 20) // 8
    assert size(0, 64, 10) == 0 and size(4, 60, 10) == 0 and size(-1, 64, 10) == 0 and size(4, 64, 0) == 0
    assert f(P, Q, 1.0, R, 0, S, n - 1, 4, 64, 10, None) == WS
    assert f(P, Q, 1.0, R, 0, None, n, 4, 64, 10, None) == WS
    assert f(P, Q, 1.0, R, 1, None, 0, 0, 64, 10, None) == OK    # an empty batch adds nothing
    assert f(None, Q, 1.0, R, 0, S, n, 4, 64, 10, None) == NULL
    assert f(P, None, 1.0, R, 0, S, n, 4, 64, 10, None) == NULL
    assert f(P, Q, 1.0, None, 0, S, n, 4, 64, 10, None) == NULL
    last = (1 << 31) - 1024  # the sort's row numbers stay in 32 bits
    assert size(last, 8, 10) > 16 * last and size(last + 1, 8, 10) == 0
    for M, D, V in ((-1, 64, 10), (4, 60, 10), (4, 64, 0), (4, 64, (1 << 31) - 1), (last + 1, 8, 10)):
        assert f(P, Q, 1.0, R, 0, S, BIG, M, D, V, None) == SHAPE
    for i in (0, 1, 3, 5):
        a = [P, Q, 1.0, R, 0, S]
        a[i] = MIS
        assert f(*a, BIG, 4, 64, 10, None) == ALIGN


@no_gpu_only
def test_norm_refusals(lib):
    f = lib.coda_add_rmsnorm_mx
    assert f(P, Q, R, 1e-6, S, P, Q, R, 0, 128, None) == OK
    for M, N, eps in ((-1, 128, 0), (4, 64, 0), (4, 16512, 0), (4, 128, -1), (1 << 31, 128, 0)):
        assert f(P, Q, R, eps, S, P, Q, R, M, N, None) == SHAPE
    for i in (0, 2, 5, 6):
        a = [P, Q, R, 1e-6, S, P, Q, R]
        a[i] = None
        assert f(*a, 4, 128, None) == NULL
    for i in (0, 1, 2, 4, 5, 6, 7):
        a = [P, Q, R, 1e-6, S, P, Q, R]
        a[i] = MIS
        assert f(*a, 4, 128, None) == ALIGN
    f = lib.coda_add_rmsnorm_fp8
    assert f(P, Q, R, 1e-6, S, S, P, Q, R, 0, 16, None) == OK
    for M, N, eps in ((-1, 16, 0), (4, 24, 0), (4, 16400, 0), (4, 16, -1)):
        assert f(P, Q, R, eps, S, S, P, Q, R, M, N, None) == SHAPE
    for i in (0, 2, 4, 6, 7):
        a = [P, Q, R, 1e-6, S, S, P, Q, R]
        a[i] = None
        assert f(*a, 4, 16, None) == NULL
    for i in (0, 1, 2, 4, 5, 6, 7, 8):
        a = [P, Q, R, 1e-6, S, S, P, Q, R]
        a[i] = MIS
        assert f(*a, 4, 16, None) == ALIGN
    assert f(P, Q, R, float("nan"), S, S, P, Q, R, 4, 16, None) == SHAPE


@no_gpu_only
def test_norm_bwd_refusals(lib):
    f, size = lib.coda_add_rmsnorm_bwd, lib.coda_add_rmsnorm_bwd_workspace_size
    n = size(5, 64)
    assert 64 * 4 <= n <= 5 * 64 * 4 and size(0, 64) == 0 and size(5, 60) == 0
    assert size(1 << 20, 64) < 1 << 24  # the blocks, not the rows
    a0 = [P, Q, R, S, P, Q, R, S]
    assert f(*a0, n - 1, 5, 64, None) == WS
    for M, N in ((-1, 64), (5, 60), (5, 16392)):
        assert f(*a0, BIG, M, N, None) == SHAPE
    for i in (0, 1, 2, 3, 5, 6):
        a = list(a0)
        a[i] = None
        assert f(*a, n, 5, 64, None) == NULL
    for i in range(8):
        a = list(a0)
        a[i] = MIS
        assert f(*a, n, 5, 64, None) == ALIGN


@no_gpu_only
def test_newton_schulz_refusals(lib):
    f, size = lib.coda_newton_schulz, lib.coda_newton_schulz_workspace_size
    n = size(2, 64, 128)
    assert n >= 2 * (4 * 64 * 128 + 2 * 64 * 64) * 2
    assert size(0, 64, 64) == 0 and size(1, 60, 64) == 0 and size(1, 64, 0) == 0
    assert size(65536, 64, 64) == 0 and size(1, 1 << 20, 1 << 20) == 0
    c = (3.4445, -4.775, 2.0315)
    assert f(P, Q, 0, 64, 128, 5, *c, 1e-7, None, 0, None) == OK
    assert f(P, Q, 2, 64, 128, 5, *c, 1e-7, R, n - 1, None) == WS
    assert f(P, Q, 2, 64, 128, 5, *c, 1e-7, None, n, None) == WS
    assert f(None, Q, 2, 64, 128, 5, *c, 1e-7, R, n, None) == NULL
    assert f(P, None, 2, 64, 128, 5, *c, 1e-7, R, n, None) == NULL
    assert f(MIS, Q, 2, 64, 128, 5, *c, 1e-7, R, n, None) == ALIGN
    assert f(P, MIS, 2, 64, 128, 5, *c, 1e-7, R, n, None) == ALIGN
    assert f(P, Q, 2, 64, 128, 5, *c, 1e-7, MIS, n, None) == ALIGN
    for b, m, k, steps, eps in ((-1, 64, 128, 5, 0), (65536, 64, 128, 5, 0), (1, 60, 128, 5, 0), (1, 64, 0, 5, 0),
                                (1, 64, 128, 0, 0), (1, 64, 128, 101, 0), (1, 64, 128, 5, -1.0),
                                (1, 1 << 20, 1 << 20, 5, 0)):
        assert f(P, Q, b, m, k, steps, *c, eps, R, BIG, None) == SHAPE


def test_binding_constants(lib):
    assert C.PARTIAL_TILE == C.partial_tile_width()
    assert lib.coda_version() >= 4


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: C.embed(t, x), lambda: C.embed_bwd(t, x, 10), lambda: C.add_rmsnorm_mx(x, None, x[0], 1e-6),
                 lambda: C.add_rmsnorm_fp8(x, None, x[0], 1e-6, torch.ones(1)),
                 lambda: C.add_rmsnorm_bwd(x, x, torch.ones(4), x[0]),
                 lambda: C.newton_schulz(torch.zeros(8, 8))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


@pytest.mark.gpu
def test_binding_refusals_on_a_gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    r, g = torch.ones(4, device="cuda"), x[0]
    f = torch.zeros(64, 72, device="cuda")
    bad = [
        (TypeError, lambda: C.embed(t.int(), x)),
        (ValueError, lambda: C.embed(t.view(2, 2), x)),
        (ValueError, lambda: C.embed(t, x[:, ::2])),
        (ValueError, lambda: C.embed(t, x, gamma=g[:64])),
        (ValueError, lambda: C.embed(t, x, hg_out=x)),
        (ValueError, lambda: C.embed(t, x, h_out=x[:2])),
        (C.CodaError, lambda: C.embed(t, x, h=False, partial=False)),
        (ValueError, lambda: C.embed_bwd(t[:3], x, 10)),
        (ValueError, lambda: C.embed_bwd(t, x, 10, accumulate=True)),
        (ValueError, lambda: C.embed_bwd(t, x, 10, dE_out=torch.zeros(9, 128, device="cuda"))),
        (C.CodaError, lambda: C.embed_bwd(t, x, 10, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))),
        (C.CodaError, lambda: C.embed_bwd(t, x, 0)),
        (ValueError, lambda: C.add_rmsnorm_mx(x, x[:2], g, 1e-6)),
        (ValueError, lambda: C.add_rmsnorm_mx(x[:, :64].contiguous(), None, g[:64], 1e-6)),
        (C.CodaError, lambda: C.add_rmsnorm_mx(x, None, g, -1.0)),
        (ValueError, lambda: C.add_rmsnorm_fp8(x, None, g, 1e-6, r)),
        (TypeError, lambda: C.add_rmsnorm_bwd(x, x, r.double(), g)),
        (ValueError, lambda: C.add_rmsnorm_bwd(x, x, r, g, x[:3])),
        (TypeError, lambda: C.newton_schulz(f.bfloat16())),
        (ValueError, lambda: C.newton_schulz(f[0])),
        (ValueError, lambda: C.newton_schulz(f.t())),
        (C.CodaError, lambda: C.newton_schulz(f[:, :12].contiguous())),
        (C.CodaError, lambda: C.newton_schulz(f, steps=0)),
        (C.CodaError, lambda: C.newton_schulz(f, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))),
    ]
    for k, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"call {k} was not refused")
    torch.cuda.synchronize()
