"""The calls around the GEMM chain on the GPU: embedding, 8-bit norms and
Newton-Schulz against plain formulas in 64 bits.

Roundings: u(t) is half a step of type t relative to the value (bf16 2^-8,
fp32 2^-24, fp16 2^-11)."""
import math

import numpy as np
import pytest
import torch

from gemm_epilogue_transformer_02_b200 import binding as C
from oracle import coda_oracle_fp8 as F8
from oracle import coda_oracle_mx as MX

pytestmark = pytest.mark.gpu

BF, F32, F64, U8 = torch.bfloat16, torch.float32, torch.float64, torch.uint8
U_BF, U_32, U_16 = 2.0 ** -8, 2.0 ** -24, 2.0 ** -11
GUARD, PATTERN = 8192, 0xA5


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


class Guarded:
    """A tensor with a known pattern before and after it."""

    def __init__(self, shape, dtype):
        n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((2 * GUARD + n,), PATTERN, dtype=U8, device="cuda")
        self.n = n
        self.t = self.raw[GUARD:GUARD + n].view(dtype).view(shape)

    def intact(self):
        return bool((self.raw[:GUARD] == PATTERN).all()) and bool((self.raw[GUARD + self.n:] == PATTERN).all())


def near(got, ref, rel, floor=0.0):
    """|got - ref| <= rel * |ref| + floor, element by element."""
    got, ref = got.to(F64), ref.to(F64)
    assert got.shape == ref.shape
    bad = ((got - ref).abs() > rel * ref.abs() + floor) | ~torch.isfinite(got)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off, worst {(got - ref).abs().max().item():.3e}"


# ---------------------------------------------------------------- embedding


@pytest.mark.parametrize("M,D,V", [(1, 8, 1), (5, 264, 17), (4, 128, 300), (257, 520, 1000), (33, 2048, 128256),
                                   (1030, 1000, 50)])
def test_embed(M, D, V):
    g = gen(M + D)
    tokens = torch.randint(-2, V + 2, (M,), generator=g, device="cuda")
    E = randn(g, V, D).to(BF)
    gamma = randn(g, D).to(BF)
    scale = math.sqrt(D)
    T = C.partial_cols(D)
    h, hg, partial = Guarded((M, D), BF), Guarded((M, D), BF), Guarded((T, M), F32)
    C.embed(tokens, E, scale, gamma, h_out=h.t, hg_out=hg.t, partial_out=partial.t)
    assert h.intact() and hg.intact() and partial.intact()
    ok = (tokens >= 0) & (tokens < V)
    ref = torch.where(ok[:, None], E.to(F64)[tokens.clamp(0, V - 1)] * float(np.float32(scale)), 0.0)
    near(h.t, ref, U_BF + 2 * U_32)
    near(hg.t, ref * gamma.to(F64), U_BF + 4 * U_32)
    sq = torch.nn.functional.pad(ref.square(), (0, T * 128 - D)).view(M, T, 128).sum(2).t()
    near(partial.t, sq, 128 * U_32)  # 128 non-negative terms
    h2, hg2, p2 = C.embed(tokens, E, scale, partial=False)
    assert torch.equal(h2, h.t) and hg2 is None and p2 is None
    h3, hg3, p3 = C.embed(tokens, E, scale, gamma, h=False)
    assert h3 is None and torch.equal(hg3, hg.t) and torch.equal(p3, partial.t)


def embed_bwd_ref(tokens, dh, V, scale):
    """(sum, sum of magnitudes) in 64 bits."""
    ok = (tokens >= 0) & (tokens < V)
    x = dh.to(F64)[ok] * float(np.float32(scale))
    z = torch.zeros(V, dh.shape[1], dtype=F64, device="cuda")
    return z.index_add(0, tokens[ok], x), z.index_add(0, tokens[ok], x.abs())


def tokens_of(kind, M, V, g):
    if kind == "uniform":
        return torch.randint(0, V, (M,), generator=g, device="cuda")
    if kind == "one":
        return torch.full((M,), V - 1, dtype=torch.int64, device="cuda")
    if kind == "padding":
        return torch.where(torch.rand(M, generator=g, device="cuda") < 0.5, V + 5, -1)
    if kind == "runs":  # a token's run is 1, 31, 32, 33, 65 or 200 rows, shuffled
        lens, t = [1, 31, 32, 33, 65, 200], []
        while len(t) < M:
            t += [(len(t) * 7) % V] * lens[len(t) % 6]
        return torch.tensor(t[:M], device="cuda")[torch.randperm(M, generator=g, device="cuda")]
    half = torch.rand(M, generator=g, device="cuda") < 0.5  # "half": every second row is one token
    return torch.where(half, 0, torch.randint(-1, V + 1, (M,), generator=g, device="cuda"))


@pytest.mark.parametrize("kind", ["uniform", "one", "padding", "runs", "half"])
@pytest.mark.parametrize("M,D,V", [(1, 8, 1), (31, 16, 3), (33, 264, 40), (1000, 2056, 97), (4097, 64, 5000),
                                   (300, 8, 300000), (700, 512, 30011)])
def test_embed_bwd(kind, M, D, V):
    g = gen(M * 3 + D)
    tokens = tokens_of(kind, M, V, g)
    dh = randn(g, M, D).to(BF)
    dE = Guarded((V, D), F32)
    ws = Guarded((C.load_library().coda_embed_bwd_workspace_size(M, D, V),), U8)
    C.embed_bwd(tokens, dh, V, 3.0, dE_out=dE.t, ws=ws.t)
    assert dE.intact() and ws.intact()
    ref, mag = embed_bwd_ref(tokens, dh, V, 3.0)
    # at most M fp32 additions of rounded partial sums, and the scale
    err = (dE.t.to(F64) - ref).abs()
    assert bool((err <= (M + 2) * U_32 * mag).all()), err.max().item()
    again = C.embed_bwd(tokens, dh, V, 3.0)
    assert torch.equal(again, dE.t)
    base = randn(g, V, D)
    acc = base.clone()
    C.embed_bwd(tokens, dh, V, 3.0, dE_out=acc, accumulate=True)
    assert torch.equal(acc, base + dE.t)  # one fp32 addition; base + 0 elsewhere


def test_embed_bwd_many_tokens():
    """Over 65536 rows: blocks of more than 32 pairs; a token in half of them."""
    M, D, V = 131072 + 77, 40, 1000
    g = gen(9)
    tokens = tokens_of("half", M, V, g)
    dh = randn(g, M, D).to(BF)
    dE = C.embed_bwd(tokens, dh, V)
    ref, mag = embed_bwd_ref(tokens, dh, V, 1.0)
    # each sum: 64 or fewer rows, then up to 2 * 2048 / 8 parts, then 8 groups
    assert bool(((dE.to(F64) - ref).abs() <= 700 * U_32 * mag).all())


def test_embed_bwd_order_does_not_depend_on_the_rows_before():
    """A token's sum is that of its rows in increasing order within a block."""
    g = gen(4)
    dh = (randn(g, 30, 16) * torch.logspace(-6, 6, 30, device="cuda")[:, None]).to(BF)
    tokens = torch.tensor([2, 1] * 15, device="cuda")
    dE = C.embed_bwd(tokens, dh, 3)
    for v, first in ((2, 0), (1, 1)):
        s = torch.zeros(16, device="cuda")
        for i in range(first, 30, 2):
            s = s + dh[i].float()
        assert torch.equal(dE[v], s)
    assert not bool(dE[0].any())


def test_embed_bwd_empty_batch():
    dE = torch.ones(5, 16, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    C.embed_bwd(none, torch.empty(0, 16, dtype=BF, device="cuda"), 5, dE_out=dE, accumulate=True)
    assert bool((dE == 1).all())
    C.embed_bwd(none, torch.empty(0, 16, dtype=BF, device="cuda"), 5, dE_out=dE)
    assert not bool(dE.any())


def test_empty_batches():
    """No rows (their tensors have no address): nothing is launched or refused."""
    e = torch.empty(0, 256, dtype=BF, device="cuda")
    g = torch.ones(256, dtype=BF, device="cuda")
    h, hg, partial = C.embed(torch.empty(0, dtype=torch.int64, device="cuda"), g.view(1, 256), 1.0, g)
    assert h.shape == hg.shape == (0, 256) and partial.shape == (2, 0)
    h, q, sf, r = C.add_rmsnorm_mx(e, e, g, 1e-6)
    assert h.shape == q.shape == (0, 256) and sf.numel() == r.numel() == 0
    amax = torch.full((1,), 3.0, device="cuda")
    _, q8, _, _ = C.add_rmsnorm_fp8(e, None, g, 1e-6, torch.ones(1, device="cuda"), amax_out=amax)
    assert q8.shape == (0, 256) and float(amax) == 3.0
    dx, dgamma = C.add_rmsnorm_bwd(e, e, torch.empty(0, device="cuda"), g, e)
    assert dx.shape == (0, 256) and not bool(dgamma.any())
    assert C.newton_schulz(torch.empty(0, 64, 128, device="cuda")).shape == (0, 64, 128)


# --------------------------------------------------------------- 8-bit norm


def norm_ref(x, res, gamma, eps):
    h = x.to(F64) + (0 if res is None else res.to(F64))
    r = 1 / torch.sqrt((h * h).mean(1) + float(np.float32(eps)))
    return h, r, gamma.to(F64) * h * r[:, None]


def norm_inputs(M, N, with_res, seed):
    g = gen(seed)
    x = randn(g, M, N).to(BF)
    x[M // 2] = 0  # a row of zeros
    res = (2 * randn(g, M, N)).to(BF) if with_res else None
    if with_res:
        res[M // 2] = 0
    gamma = randn(g, N).to(BF)
    gamma[:32] = 0  # a block of zeros
    return x, res, gamma


# y's relative error: r's sum of N non-negative terms (half of it in r), rsqrt
# and the products; far below half a step of e4m3 (2^-4)
def y_err(N):
    return (N / 2 + 8) * U_32


@pytest.mark.parametrize("with_res", [True, False])
@pytest.mark.parametrize("M,N", [(1, 128), (3, 384), (130, 512), (257, 2048), (20, 8192), (129, 640), (2, 16384),
                                 (131, 128), (70, 4224), (5, 8320)])
def test_add_rmsnorm_mx(M, N, with_res):
    x, res, gamma = norm_inputs(M, N, with_res, M + N)
    eps = 1e-6
    h, q, r = Guarded((M, N), BF), Guarded((M, N), U8), Guarded((M,), F32)
    sf = Guarded((C.mx_sf_bytes(M, N, C.MX_A),), U8)
    C.add_rmsnorm_mx(x, res, gamma, eps, h_out=h.t, yq_out=q.t, ysf_out=sf.t, r_out=r.t)
    assert h.intact() and q.intact() and sf.intact() and r.intact()
    h64, r64, y = norm_ref(x, res, gamma, eps)
    near(h.t, h64, U_BF + U_32)
    near(r.t, r64, y_err(N))
    sfh = sf.t.cpu().numpy()
    exps = MX.sf_untile(sfh, M, N)
    tiled, used = MX.sf_tile(exps, M)
    assert np.array_equal(tiled[used], sfh[used]) and used.all()  # padding rows hold 127
    got = torch.from_numpy(MX.mx_dequantize(q.t.cpu().numpy(), exps)).cuda()
    s = torch.from_numpy(np.ldexp(1.0, exps)).cuda().repeat_interleave(32, 1)
    # e4m3: half a step of the value (2^-4), or of the smallest step 2^-9
    assert bool(((got - y).abs() <= (2.0 ** -4 + y_err(N)) * y.abs() + 2.0 ** -10 * s).all())
    amax = y.view(M, N // 32, 32).abs().amax(2).cpu().numpy()
    sc = np.ldexp(1.0, exps)
    e = y_err(N)
    assert np.all(amax <= 448 * sc * (1 + e))          # no element saturates
    assert np.all((amax >= 224 * sc * (1 - e)) | (amax == 0))  # and no smaller scale would do
    assert np.all(exps[amax == 0] == 0)
    h0, q0, sf0, r0 = C.add_rmsnorm_mx(x, res, gamma, eps, h=False)
    assert h0 is None and torch.equal(q0, q.t) and torch.equal(sf0, sf.t) and torch.equal(r0, r.t)


@pytest.mark.parametrize("with_res", [True, False])
@pytest.mark.parametrize("M,N", [(1, 16), (1, 4096), (3, 528), (300, 512), (64, 2064), (9, 16384),
                                 (2, 512), (301, 48), (6, 8208)])
def test_add_rmsnorm_fp8(M, N, with_res):
    x, res, gamma = norm_inputs(M, N, with_res, M * 7 + N)
    eps = 1e-5
    s_y = torch.tensor([2.0 / 448], device="cuda")  # some of y saturates
    h, q, r, amax = Guarded((M, N), BF), Guarded((M, N), U8), Guarded((M,), F32), Guarded((1,), F32)
    C.add_rmsnorm_fp8(x, res, gamma, eps, s_y, h_out=h.t, y8_out=q.t, amax_out=amax.t, r_out=r.t)
    assert h.intact() and q.intact() and r.intact() and amax.intact()
    h64, r64, y = norm_ref(x, res, gamma, eps)
    near(h.t, h64, U_BF + U_32)
    near(r.t, r64, y_err(N))
    near(amax.t, y.abs().max().reshape(1), y_err(N))
    got = torch.from_numpy(F8.e4m3_decode(q.t.cpu().numpy())).cuda()
    want = (y / s_y.to(F64)).clamp(-448, 448)
    assert bool(((got - want).abs() <= (2.0 ** -4 + y_err(N)) * want.abs() + 2.0 ** -10).all())


def test_norm8_agrees_with_the_separate_calls():
    """The same codes as add -> norm -> quantise where those round nothing away:
    gamma 1 and rows whose h and r are powers of two."""
    M, N = 128, 256
    g = gen(3)
    x = torch.where(torch.rand(M, N, generator=g, device="cuda") < 0.5, 1.0, -1.0).to(BF)
    x *= 2.0 ** torch.randint(-3, 4, (M, 1), generator=g, device="cuda").to(BF)
    gamma = torch.ones(N, dtype=BF, device="cuda")
    _, q, sf, r = C.add_rmsnorm_mx(x, None, gamma, 0.0)
    y = C.unfused_rmsnorm(x, gamma, 0.0)
    q2, sf2 = C.mx_quantize(y, C.MX_A)
    assert torch.equal(q, q2) and torch.equal(sf, sf2)
    s_y = torch.tensor([1.0 / 64], device="cuda")
    _, q8, amax, _ = C.add_rmsnorm_fp8(x, None, gamma, 0.0, s_y)
    q82, amax2, _ = C.unfused_rmsnorm_fp8(x, gamma, 0.0, s_y)
    assert torch.equal(q8, q82) and torch.equal(amax, amax2)


def test_norm8_keeps_a_bad_row_to_itself():
    M, N = 4, 256
    g = gen(8)
    x = randn(g, M, N).to(BF)
    gamma = randn(g, N).to(BF)
    clean = C.add_rmsnorm_mx(x, None, gamma, 1e-6)
    x[1, 7], x[2, 9] = float("nan"), float("inf")
    h, q, sf, r = C.add_rmsnorm_mx(x, None, gamma, 1e-6)
    for i in (0, 3):
        assert torch.equal(q[i], clean[1][i]) and torch.equal(h[i], clean[0][i]) and r[i] == clean[3][i]
    assert torch.isnan(r[1]) and r[2] == 0
    assert int(q[2, 9]) & 0x7f == 0x7f  # inf * 0


@pytest.mark.parametrize("with_dh", [True, False])
@pytest.mark.parametrize("M,N", [(1, 8), (5, 264), (257, 512), (130, 2048), (1500, 1032), (40, 8192), (7, 16384),
                                 (5000, 40), (2401, 512), (1900, 2568), (700, 4104), (301, 8200)])
def test_add_rmsnorm_bwd(M, N, with_dh):
    g = gen(M + 5 * N)
    h = (2 * randn(g, M, N)).to(BF)
    r = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    dy, gamma = randn(g, M, N).to(BF), randn(g, N).to(BF)
    d_h = randn(g, M, N).to(BF) if with_dh else None
    dx, dgamma = Guarded((M, N), BF), Guarded((N,), F32)
    ws = Guarded((C.load_library().coda_add_rmsnorm_bwd_workspace_size(M, N),), U8)
    C.add_rmsnorm_bwd(dy, h, r, gamma, d_h, dx_out=dx.t, dgamma_out=dgamma.t, ws=ws.t)
    assert dx.intact() and dgamma.intact() and ws.intact()
    dy64, h64, r64, g64 = dy.to(F64), h.to(F64), r.to(F64)[:, None], gamma.to(F64)
    gg = dy64 * g64
    terms = gg * h64
    coef = -(r64 ** 3) * terms.mean(1, keepdim=True)
    ref = r64 * gg + coef * h64 + (0 if d_h is None else d_h.to(F64))
    # fp32: the mean's N additions relative to its terms' magnitudes, a few operations on each addend
    mag = (r64 * gg).abs() + (coef * h64).abs() + (0 if d_h is None else d_h.to(F64).abs())
    floor = 8 * U_32 * mag + N * U_32 * (r64 ** 3 * terms.abs().mean(1, keepdim=True) * h64.abs())
    assert bool(((dx.t.to(F64) - ref).abs() <= U_BF * ref.abs() + floor).all())
    t = dy64 * h64 * r64
    assert bool(((dgamma.t.to(F64) - t.sum(0)).abs() <= (M + 4) * U_32 * t.abs().sum(0)).all())
    again = C.add_rmsnorm_bwd(dy, h, r, gamma, d_h)
    assert torch.equal(again[0], dx.t) and torch.equal(again[1], dgamma.t)


def test_add_rmsnorm_bwd_against_differences():
    """<dy, y(h + t v) - y(h - t v)> / 2t in 64 bits for directions of h and gamma."""
    M, N, eps = 6, 128, 1e-6
    g = gen(21)
    x, gamma, dy = randn(g, M, N).to(BF), randn(g, N).to(BF), randn(g, M, N).to(BF)
    h, _, _, r = C.add_rmsnorm_mx(x, None, gamma, eps)
    dx, dgamma = C.add_rmsnorm_bwd(dy, h, r, gamma)

    def f(h, gam):
        return (dy.to(F64) * gam * h / torch.sqrt((h * h).mean(1, keepdim=True) + eps)).sum()

    h64, g64, t = h.to(F64), gamma.to(F64), 1e-5
    for k in range(3):
        v, w = randn(g, M, N).to(F64), randn(g, N).to(F64)
        d = (f(h64 + t * v, g64) - f(h64 - t * v, g64)) / (2 * t)
        # each dx is off by up to half a bf16 step
        assert abs(float((dx.to(F64) * v).sum() - d)) <= float(1.1 * U_BF * (dx.to(F64) * v).abs().sum())
        d = (f(h64, g64 + t * w) - f(h64, g64 - t * w)) / (2 * t)
        assert abs(float((dgamma.to(F64) * w).sum() - d)) <= 1e-5 * float((dgamma.to(F64) * w).abs().sum())


# ----------------------------------------------------------- Newton-Schulz


def ns_ref(G, steps=5, coeffs=C.NEWTON_SCHULZ_COEFFS, eps=1e-7):
    a, b, c = coeffs
    X = G.to(F64)
    X = X / (X.square().sum((-2, -1), keepdim=True).sqrt() + float(np.float32(eps)))
    for _ in range(steps):
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    return X


# Relative to |X|_F: the output's rounding (2^-8 at most), and three fp16
# operands per step (X, A, B), each off by at most 2^-11 in independent
# directions, grown by at most a factor of 2 on the way out (the slope of the
# polynomial on the singular values it maps among themselves is below 1.7).
def ns_tol(steps):
    return U_BF + 2 * math.sqrt(3 * steps) * U_16


def ns_check(out, G, steps=5, more=0.0, **kw):
    ref = ns_ref(G, steps, **kw)
    err = (out.to(F64) - ref).flatten(-2).norm(dim=-1) / ref.flatten(-2).norm(dim=-1).clamp(min=1e-300)
    assert bool((err <= ns_tol(steps) + more).all()), err
    return err


@pytest.mark.parametrize("m,n", [(8, 8), (8, 1000), (72, 8), (128, 128), (136, 264), (264, 136), (512, 512),
                                 (1000, 264), (136, 1032), (1024, 1024), (1096, 1032), (1032, 2056), (2056, 1032),
                                 (1544, 4104), (4104, 1544), (2056, 2568)])
@pytest.mark.parametrize("batch", [None, 3])
def test_newton_schulz(m, n, batch):
    g = gen(m + n)
    shape = (m, n) if batch is None else (batch, m, n)
    G = 1e-3 * randn(g, *shape)
    out = Guarded(shape, BF)
    ws = Guarded((C.load_library().coda_newton_schulz_workspace_size(batch or 1, m, n),), U8)
    C.newton_schulz(G, out=out.t, ws=ws.t)
    assert out.intact() and ws.intact()
    ns_check(out.t, G)
    assert torch.equal(C.newton_schulz(G), out.t)


@pytest.mark.parametrize("batch,m,n", [(2, 8, 8), (40, 72, 136), (5, 520, 512), (16, 512, 512), (90, 264, 256),
                                       (600, 64, 64), (12, 1032, 1024), (5, 1032, 2072), (3, 1544, 1640)])
def test_newton_schulz_batches(batch, m, n):
    """Matrices go from phase to phase by themselves where there are few tiles,
    and together where there are many; each is what it is alone, in every run."""
    G = randn(gen(batch), batch, m, n)
    G[batch // 2, m // 2, n // 3] = float("nan")
    out = C.newton_schulz(G)
    assert not out[batch // 2].isfinite().any()
    keep = torch.arange(batch, device="cuda") != batch // 2
    ns_check(out[keep], G[keep])
    for _ in range(3):
        assert torch.equal(C.newton_schulz(G)[keep], out[keep])


@pytest.mark.parametrize("steps", [1, 2, 3, 7])
def test_newton_schulz_steps(steps):
    G = randn(gen(steps), 200, 328)
    ns_check(C.newton_schulz(G, steps=steps), G, steps)
    ns_check(C.newton_schulz(G.t().contiguous(), steps=steps), G.t(), steps)


@pytest.mark.parametrize("m,n", [(512, 768), (1024, 1280)])
def test_newton_schulz_nearly_low_rank(m, n):
    """A few directions hold nearly all of the norm; the rest grow by up to
    3.4^5 and with them whatever rounding left there."""
    g = gen(17)
    G = randn(g, m, 16) @ randn(g, 16, n) + 0.01 * randn(g, m, n)
    ns_check(C.newton_schulz(G), G)
    ns_check(C.newton_schulz(G.t().contiguous()), G.t())


@pytest.mark.parametrize("m,n", [(512, 2048), (1024, 2560)])
def test_newton_schulz_nearly_low_rank_in_groups(m, n):
    """Steps 1-3 and 4-5 are taken on the Gram matrix A.  Its fp16 rounding is a
    symmetric matrix of spectral norm e <= 2 |A|_F 2^-12 / sqrt(m) (entries off by
    2^-12 of theirs in random directions), which the small directions take
    through the later steps of a group, growing by a^2 = 11.9 a step, and which
    moves P by |b| e / a = 1.4 e of itself.  16 directions hold the norm: |A|_F is
    1/4 at first and at most 4 * 1.44 in the second group, so for m >= 512 that
    is 1.4 * 5.4e-6 * 11.9^2 + 1.4 * 1.25e-4 * 11.9 = 3.2e-3; P A and A' are
    rounded in the same way: sqrt(3) of that, and sqrt(2) for the mirrored half."""
    g = gen(18)
    G = randn(g, m, 16) @ randn(g, 16, n) + 0.01 * randn(g, m, n)
    more = math.sqrt(6) * 3.2e-3
    ns_check(C.newton_schulz(G), G, more=more)
    ns_check(C.newton_schulz(G.t().contiguous()), G.t(), more=more)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 9])
def test_newton_schulz_groups_of_every_length(steps):
    """Wide enough for groups: 1, 2, 3, 3 + 1, 3 + 2 + 1, 3 + 2 + 2 + 2 steps; odd
    sizes, and a batch."""
    G = randn(gen(40 + steps), 2, 520, 1048)
    ns_check(C.newton_schulz(G, steps=steps), G, steps)
    T = G.mT.contiguous()
    ns_check(C.newton_schulz(T, steps=steps), T, steps)


def test_newton_schulz_scale():
    """The norm is taken in 64 bits: only eps sees the scale of G."""
    G = randn(gen(2), 136, 136)
    ref = C.newton_schulz(G, eps=0.0)
    for k in (-100, -40, 40, 100):
        assert torch.equal(C.newton_schulz(G * 2.0 ** k, eps=0.0), ref)
    assert not bool(C.newton_schulz(torch.zeros(64, 72, device="cuda")).any())


def test_newton_schulz_other_coefficients():
    G = randn(gen(5), 256, 136)
    kw = {"coeffs": (1.875, -1.25, 0.375)}  # converges to one from below
    ns_check(C.newton_schulz(G, steps=6, **kw), G, 6, **kw)


def test_newton_schulz_keeps_a_bad_matrix_to_itself():
    G = randn(gen(6), 3, 136, 200)
    clean = C.newton_schulz(G)
    G[1, 5, 7] = float("nan")
    out = C.newton_schulz(G)
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2], clean[2])
    assert not bool(torch.isfinite(out[1]).all())


# ------------------------------------------------------ streams and graphs


def step_inputs(seed):
    g = gen(seed)
    M, D, V = 300, 256, 500
    return {"tokens": torch.randint(-1, V, (M,), generator=g, device="cuda"), "E": randn(g, V, D).to(BF),
            "gamma": randn(g, D).to(BF), "dh": randn(g, M, D).to(BF), "res": randn(g, M, D).to(BF),
            "s_y": torch.tensor([0.01], device="cuda"), "G": randn(g, D, 512)}


def all_calls(s):
    h, hg, partial = C.embed(s["tokens"], s["E"], 2.0, s["gamma"])
    h2, q, sf, r = C.add_rmsnorm_mx(h, s["res"], s["gamma"], 1e-6)
    _, q8, amax, _ = C.add_rmsnorm_fp8(h, s["res"], s["gamma"], 1e-6, s["s_y"], h=False)
    dx, dgamma = C.add_rmsnorm_bwd(s["dh"], h2, r, s["gamma"], s["res"])
    dE = C.embed_bwd(s["tokens"], dx, 500, 2.0)
    out = C.newton_schulz(s["G"])
    return [h, hg, partial, h2, q, sf, r, q8, amax, dx, dgamma, dE, out]


def test_calls_capture_into_a_graph_and_replay_on_new_inputs():
    a, b = step_inputs(1), step_inputs(2)
    want_a, want_b = all_calls(a), all_calls(b)
    s = {k: v.clone() for k, v in a.items()}
    all_calls(s)  # kernels' attributes are set outside of the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_calls(s)
    for inputs, want in ((a, want_a), (b, want_b), (a, want_a)):
        for k, v in inputs.items():
            s[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_two_streams_at_once():
    """Each call has its own workspace, so calls on two streams do not meet."""
    a, b = step_inputs(3), step_inputs(4)
    want_a, want_b = all_calls(a), all_calls(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            got_a = all_calls(a)
        with torch.cuda.stream(s2):
            got_b = all_calls(b)
        torch.cuda.synchronize()
        for x, y in zip(got_a + got_b, want_a + want_b):
            assert torch.equal(x, y)


# ---------------------------------------------------------- together, as used


def test_a_training_step_from_tokens_to_updates():
    """Tokens -> embedding -> row-scaled GEMM from hg and partial -> loss; its
    gradients back to the table; the weight's update orthogonalised."""
    M, D, V = 512, 256, 1024
    g = gen(31)
    eps = 1e-6
    tokens = torch.randint(0, V, (M,), generator=g, device="cuda")
    labels = torch.randint(0, V, (M,), generator=g, device="cuda")
    E = randn(g, V, D).to(BF)
    gamma = (1 + 0.1 * randn(g, D)).to(BF)
    W = (randn(g, D, D) / 16).to(BF)
    head = (randn(g, D, V) / 16).to(BF)
    h, hg, partial = C.embed(tokens, E, 1.0, gamma)
    out, r = C.gemm_rowscale_partial(hg, W, partial, D, eps)
    loss, lse, _ = C.lmhead_ce(out, head, labels)
    dOut, dHead = C.lmhead_ce_bwd(out, head, labels, lse)
    d_hg, dW, pdr = C.gemm_rowscale_bwd(dOut.to(BF), hg, W, r)
    dh, dgamma = C.rms_reduce_bwd(pdr, r, d_hg, h, gamma)
    dE = C.embed_bwd(tokens, dh, V)
    ups = [C.newton_schulz(dW), C.newton_schulz(dHead)]
    C.poll_status()
    E64, g64, W64, H64 = (t.to(F64).requires_grad_() for t in (E, gamma, W, head))
    x = E64[tokens]
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + eps) * g64
    L = torch.nn.functional.cross_entropy(y @ W64 @ H64, labels, reduction="none")
    L.mean().backward()
    # the chain rounds its intermediates to bf16 (2^-8 each): out, the loss gradient, dOut, y, hg, dh
    near(loss, L.detach(), 0.0, floor=2e-2)
    for got, ref in ((dE, E64.grad), (dW, W64.grad), (dHead, H64.grad), (dgamma, g64.grad)):
        assert float((got.to(F64) - ref).norm() / ref.norm()) <= 6 * U_BF
    for u, d in zip(ups, (dW, dHead)):
        ns_check(u, d)


def test_8bit_norm_feeds_the_8bit_gemms():
    M, N, N2 = 300, 256, 384
    g = gen(41)
    x, res = randn(g, M, N).to(BF), randn(g, M, N).to(BF)
    gamma = (1 + 0.1 * randn(g, N)).to(BF)
    W = (randn(g, N, N2) / 16).to(BF)
    _, _, y = norm_ref(x, res, gamma, 1e-6)
    ref = y @ W.to(F64)
    # both operands in e4m3: each product off by 2 * 2^-4 at most in random directions;
    # relative to the rms that is below 2 * 2^-4 / sqrt(3) on average
    bar = 2 * 2.0 ** -4 / math.sqrt(3)
    Wq, Wsf = C.mx_quantize(W.t().contiguous(), C.MX_B)
    _, q, sf, _ = C.add_rmsnorm_mx(x, res, gamma, 1e-6)
    out, _ = C.gemm_rowscale_partial_mx(q, sf, Wq, Wsf)
    assert float((out.to(F64) - ref).norm() / ref.norm()) <= bar
    W8, _, sw = C.fp8_quantize(W, transpose=True)
    s_y = torch.ones(1, device="cuda")
    _, _, amax, _ = C.add_rmsnorm_fp8(x, res, gamma, 1e-6, s_y)
    s_y = C.fp8_scale_from_amax(amax)
    _, y8, _, _ = C.add_rmsnorm_fp8(x, res, gamma, 1e-6, s_y)
    assert float((C.gemm_fp8(y8, s_y, W8, sw).to(F64) - ref).norm() / ref.norm()) <= bar
    C.poll_status()
