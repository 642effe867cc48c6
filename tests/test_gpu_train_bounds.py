"""The error bounds that the calls around the GEMM chain state, and their edges,
on the GPU against 64 bits."""
import math

import pytest
import torch

from gemm_epilogue_transformer_02_b200 import binding as C

pytestmark = pytest.mark.gpu

BF, F32, F64, U8 = torch.bfloat16, torch.float32, torch.float64, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    C.load_library()
    yield
    C.poll_status()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


# ----------------------------------------------------------- Newton-Schulz


def ns_exact(G, steps=5, eps=1e-7):
    a, b, c = C.NEWTON_SCHULZ_COEFFS
    X = G.to(F64)
    X = X / (X.norm() + eps)
    X = X.t() if X.shape[0] > X.shape[1] else X
    for _ in range(steps):
        A = X @ X.t()
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.t() if G.shape[0] > G.shape[1] else X


def ns_error(out, ref):
    """|X - ref| / |ref| of X before its rounding to bf16: the output's error less
    the rounding's own (they are independent, so the squares add; the latter is
    taken from ref's rounding and known to 1 / sqrt(elements) of itself)."""
    n2 = float(ref.square().sum())
    all2 = float((out.to(F64) - ref).square().sum()) / n2
    own2 = float((ref.to(BF).to(F64) - ref).square().sum()) / n2
    return math.sqrt(max(0.0, all2 - own2)), own2 * 3.0 / math.sqrt(ref.numel())


def low_rank(g, m, n, rank, noise):
    return randn(g, m, rank) @ randn(g, rank, n) / math.sqrt(rank) + noise * randn(g, m, n)


def stated(m, n):
    """The header's bound for a G whose norm lies in a few directions."""
    return 1.5e-3 + 0.65 / min(m, n)


@pytest.mark.parametrize("m,n", [(512, 1016), (512, 1024), (1024, 2040), (1024, 2048), (520, 4104), (256, 512),
                                 (64, 72), (136, 264), (64, 1024)])
@pytest.mark.parametrize("rank,noise", [(1, 1e-2), (1, 3e-3), (1, 3e-4), (4, 1e-3), (16, 1e-3)])
def test_newton_schulz_few_directions(m, n, rank, noise):
    """One or a few directions hold the norm, as in the gradient of a layer whose
    inputs are not centred: whatever the shape and the orientation."""
    G = low_rank(gen(m + n + rank), m, n, rank, noise)
    ref = ns_exact(G)
    e, slack = ns_error(C.newton_schulz(G), ref)
    assert e <= math.sqrt(stated(m, n) ** 2 + slack), e
    e, slack = ns_error(C.newton_schulz(G.t().contiguous()).t(), ref)
    assert e <= math.sqrt(stated(m, n) ** 2 + slack), e


@pytest.mark.parametrize("m,n", [(512, 512), (512, 1024), (1024, 4096), (4096, 1024)])
@pytest.mark.parametrize("means", [1.0, 3.0])
def test_newton_schulz_of_a_gradient_with_feature_means(m, n, means):
    """X^T dY whose features have means as large as their deviation, and three
    times that."""
    g = gen(m + 2 * n)
    T = 2 * min(m, n)
    G = (randn(g, m, T) + means * randn(g, m, 1)) @ (randn(g, T, n) + means * randn(g, 1, n))
    e, slack = ns_error(C.newton_schulz(G), ns_exact(G))
    assert e <= math.sqrt(stated(m, n) ** 2 + slack), e
