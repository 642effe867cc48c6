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


# The kernel's roundings restated: fp16 values scaled by powers of two, the
# symmetric results' lower halves mirrored, what fp16 drops of a diagonal kept
# beside it, X in two parts of which the last update takes the first.


def f16(x, scale):
    return (x * scale).to(torch.float16).to(F64) / scale


class Sym:
    def __init__(self, v, scale, diag):
        v = torch.tril(v) + torch.tril(v, -1).t()
        self.m = f16(v, scale)
        self.f = torch.diagonal(self.m)
        self.d = (torch.diagonal(v) - self.f) * (1.0 if diag else 0.0)


def truncated_product(x, y):
    """Sums of 16 products at a time, each addition cut to fp32's 24 bits."""
    acc = torch.zeros(x.shape[0], y.shape[1], dtype=F64, device="cuda")
    for k in range(0, x.shape[1], 16):
        mant, ex = torch.frexp(acc + x[:, k:k + 16] @ y[k:k + 16])
        acc = torch.ldexp(torch.trunc(mant * 2.0 ** 24) / 2.0 ** 24, ex)
    return acc


def ns_restated(G, product=torch.matmul, diag=True, low=True):
    a, b, c = C.NEWTON_SCHULZ_COEFFS
    X = G.to(F64)
    X = X / (X.norm() + 1e-7)
    X = X.t() if X.shape[0] > X.shape[1] else X
    for step in range(5):
        hi = f16(X, 4096.0)
        lo = f16(X - hi, 4096.0) * (1.0 if low and step < 4 else 0.0)
        A = Sym(product(hi, hi.t()), 1024.0, diag)
        corr = c * (2 * A.d * A.f + A.d * A.d) + b * A.d + a
        P = Sym(c * product(A.m, A.m) + b * A.m + torch.diag(corr), 256.0, diag)
        X = product(P.m, hi) + P.d[:, None] * hi + (P.d + P.f)[:, None] * lo
    return X.t() if G.shape[0] > G.shape[1] else X


def ns_case(kind, m, n):
    g = gen(m + 3 * n)
    if kind == "gaussian":
        return randn(g, m, n)
    if kind == "one direction":
        return low_rank(g, m, n, 1, 1e-3)
    if kind == "means":
        T = 2 * min(m, n)
        return (randn(g, m, T) + 3 * randn(g, m, 1)) @ (randn(g, T, n) + 3 * randn(g, 1, n))
    q, r = torch.linalg.qr(randn(g, max(m, n), min(m, n)))  # every A and P a multiple of the identity
    return (q if m > n else q.t()).contiguous()


@pytest.mark.parametrize("kind,m,n", [(k, m, n) for k in ("gaussian", "one direction", "means")
                                      for m, n in ((512, 512), (384, 1160), (1160, 384), (1024, 1032))]
                         + [("orthogonal", 512, 512), ("orthogonal", 384, 1160)])
def test_newton_schulz_rounds_as_stated(kind, m, n):
    """The result is that of the stated roundings with exact sums, up to what the
    tensor core's fp32 sums move: an entry whose sum is cut differently may round
    to the fp16 value beside it.  How far that reaches is worked out with sums cut
    after every 16 products (3e-4 to 1.1e-3 for these inputs); the bar is a third
    above it.  Without the diagonals' corrections the result would be 1.0e-3 to
    2.3e-3 away, without X's low part up to 0.12: both beyond the bar."""
    G = ns_case(kind, m, n)
    ref = ns_restated(G)

    def away(X):
        return float((X - ref).norm() / ref.norm())

    bar = 4 / 3 * away(ns_restated(G, truncated_product)) + 5e-5
    assert bar < away(ns_restated(G, diag=False))
    if kind != "gaussian":
        assert bar < away(ns_restated(G, low=False))
    e, slack = ns_error(C.newton_schulz(G), ref)
    assert e <= math.sqrt(bar ** 2 + slack), (e, bar)


@pytest.mark.parametrize("batch,m,n", [(9, 264, 256), (3, 520, 512), (40, 72, 136), (2, 1032, 520)])
def test_newton_schulz_matrix_of_a_batch_is_what_it_is_alone(batch, m, n):
    """To the last bit where the sums' k-blocks stay whole (K below 1024).  A K of
    1032 has 17 k-blocks, which the batch's 128 x 128 tiles take in two parts and
    the 128 x 64 ones of a matrix alone in one: another order of sums, so there
    each is within the stated bound of the exact X and within half a bf16 step of
    its own, and the two differ by no more than twice both."""
    G = randn(gen(batch + m), batch, m, n)
    out = C.newton_schulz(G)
    for i in range(batch):
        alone = C.newton_schulz(G[i])
        if max(m, n) < 1024:
            assert torch.equal(alone, out[i])
        else:
            far = (alone.to(F64) - out[i].to(F64)).norm() / out[i].to(F64).norm()
            assert float(far) <= 2 * (stated(m, n) + 2.0 ** -8)


# --------------------------------------------------------------- 8-bit norm


@pytest.mark.parametrize("M,N", [(5, 264), (40, 2048), (3, 8200)])
@pytest.mark.parametrize("k", [-60, -45, 40, 60])
def test_norm_backward_of_rows_far_from_one(M, N, k):
    """dx of 2^k h with 2^-k r is 2^-k dx, and dgamma is the same, to the last bit:
    every product only changes its exponent."""
    g = gen(M + N)
    h = randn(g, M, N).to(BF)
    r = torch.rsqrt(h.float().square().mean(1))
    dy, gamma = randn(g, M, N).to(BF), randn(g, N).to(BF)
    dx, dgamma = C.add_rmsnorm_bwd(dy, h, r, gamma)
    dx2, dgamma2 = C.add_rmsnorm_bwd(dy, h * 2.0 ** k, r * 2.0 ** -k, gamma)
    assert torch.equal(dx2.float(), dx.float() * 2.0 ** -k) and torch.equal(dgamma2, dgamma)


def test_norm_of_a_stream_far_from_one():
    """The same forward and back: with eps 0 only the exponents of h and r change."""
    M, N = 9, 640
    g = gen(12)
    x, gamma = randn(g, M, N).to(BF), randn(g, N).to(BF)
    dy, d_h = randn(g, M, N).to(BF), randn(g, M, N).to(BF)
    h, q, sf, r = C.add_rmsnorm_mx(x, x, gamma, 0.0)
    dx, dgamma = C.add_rmsnorm_bwd(dy, h, r, gamma, d_h)
    for k in (-58, 58):
        s = 2.0 ** k
        h2, q2, sf2, r2 = C.add_rmsnorm_mx(x * s, x * s, gamma, 0.0)
        assert torch.equal(h2.float(), h.float() * s) and torch.equal(q2, q) and torch.equal(sf2, sf)
        assert torch.equal(r2, r / s)
        dx2, dgamma2 = C.add_rmsnorm_bwd(dy, h2, r2, gamma, (d_h / s).to(BF))
        assert torch.equal(dx2.float(), dx.float() / s) and torch.equal(dgamma2, dgamma)


def test_amax_of_an_empty_batch_is_zero():
    """A new amax is never left as it was allocated (a given one stays as it is)."""
    old = [torch.full((1,), 3.0, device="cuda") for _ in range(64)]
    del old  # the allocator's next small blocks hold 3
    for N in (16, 512, 2048):
        e, gamma = torch.empty(0, N, dtype=BF, device="cuda"), torch.ones(N, dtype=BF, device="cuda")
        amax = C.add_rmsnorm_fp8(e, None, gamma, 1e-6, torch.ones(1, device="cuda"))[2]
        assert float(amax) == 0.0


# ------------------------------------------------------- embedding gradient


# Rows past the first 48 MiB + 4096 M bytes of dE are zeroed by blocks of 8, 8, 2
# and 1 rows of a 32-row word of the bitmap.
@pytest.mark.parametrize("D,V", [(2048, 8003), (1032, 16001), (4104, 4001), (16392, 1003)])
@pytest.mark.parametrize("kind", ["none", "borders", "every third"])
def test_embed_bwd_zeroes_every_row_that_does_not_occur(D, V, kind):
    g = gen(D + V)
    first = ((48 << 20) + 4096 * 64) // (32 * 4 * D) * 32
    assert first < V - 64
    if kind == "none":
        tokens = torch.full((5,), -1, device="cuda")
    elif kind == "borders":
        at = [0, 31, 32, V - 1, V - 2]
        for k in range(first - 64, first + 64, 8):
            at += [k - 1, k, k + 1]
        tokens = torch.tensor(sorted(set(at)), device="cuda")
    else:
        tokens = torch.arange(first - 40, V, 3, device="cuda")
    tokens = tokens[torch.randperm(len(tokens), generator=g, device="cuda")]
    dh = randn(g, len(tokens), D).to(BF)
    raw = torch.full((V + 2, D), float("nan"), device="cuda")
    dE = C.embed_bwd(tokens, dh, V, dE_out=raw[1:-1])
    ref = torch.zeros(V, D, device="cuda")
    if kind != "none":
        ref[tokens] = dh.float()  # each occurs once
    assert torch.equal(dE, ref)
    assert bool(raw[0].isnan().all()) and bool(raw[-1].isnan().all())
