"""Timed cases of the training-step operators around the GEMM chain: the token
embedding with its gradient, the residual add + RMSNorm that hands 8-bit
operands to the FP8 and MXFP8 GEMMs with its backward, and the Newton-Schulz
orthogonalisation of a weight's update.

With ``own`` false ``run`` computes an operator from elementary torch
operations in fp32; with ``own`` true it calls the library."""
import math

import torch

own = False

EPS = 1e-6
NS = (3.4445, -4.775, 2.0315)  # the Muon optimiser's quintic
NS_EPS = 1e-7
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one token through a 1B model's table: what a call costs by itself
        {"name": "embed_1_token", "op": "embed", "M": 1, "D": 2048, "V": 128256},
        # a 1B training batch (4 x 2048 tokens), with gamma * h and the norm's partial sums
        {"name": "embed_1b", "op": "embed", "M": 8192, "D": 2048, "V": 128256},
        # a small model's table gradient, a ragged batch
        {"name": "embed_bwd_small", "op": "embed_bwd", "M": 253, "D": 512, "V": 4096},
        # the 1B table's dense fp32 gradient: 1 GB written, word frequencies as in text
        {"name": "embed_bwd_1b", "op": "embed_bwd", "M": 8192, "D": 2048, "V": 128256},
        # one token, delayed per-tensor scale
        {"name": "norm_fp8_1_token", "op": "norm", "form": "fp8", "M": 1, "N": 4096, "res": True},
        # the 1B batch's first norm for the MXFP8 GEMMs
        {"name": "norm_mx_1b", "op": "norm", "form": "mx", "M": 8192, "N": 2048, "res": True},
        # a small ragged batch's norm backward
        {"name": "norm_bwd_small", "op": "norm_bwd", "M": 257, "N": 512, "res": True},
        # the 1B batch's norm backward with the residual stream's gradient
        {"name": "norm_bwd_1b", "op": "norm_bwd", "M": 8192, "N": 2048, "res": True},
        # the tiny block's first weight
        {"name": "ns_512", "op": "ns", "batch": 1, "m": 512, "n": 512},
        # the first-GEMM weights of four layers of the 1B model at once
        {"name": "ns_1b_square_x4", "op": "ns", "batch": 4, "m": 2048, "n": 2048},
        # its down projection
        {"name": "ns_1b_down", "op": "ns", "batch": 1, "m": 8192, "n": 2048},
        # its fused gate/up projection
        {"name": "ns_1b_gate_up", "op": "ns", "batch": 1, "m": 2048, "n": 16384},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["embed", "embed_bwd", "norm", "norm", "norm_bwd", "ns", "ns"])
    if op in ("embed", "embed_bwd"):
        return {"op": op, "M": _log(rng, 1, 8192), "D": _log(rng, 64, 2048, 8), "V": _log(rng, 100, 128256)}
    if op == "norm":
        form = rng.choice(["mx", "fp8"])
        N = _log(rng, 128, 8192, 128) if form == "mx" else _log(rng, 16, 8192, 16)
        return {"op": op, "form": form, "M": _log(rng, 1, min(8192, 8192 * 4096 // N)), "N": N,
                "res": rng.random() < 0.8}
    if op == "norm_bwd":
        N = _log(rng, 16, 8192, 8)
        return {"op": op, "M": _log(rng, 1, min(8192, 8192 * 4096 // N)), "N": N, "res": rng.random() < 0.8}
    m, n = _log(rng, 64, 2048, 8), _log(rng, 64, 4096, 8)
    if rng.random() < 0.3:
        n = m
    if rng.random() < 0.3:
        m, n = n, m
    most = max(1, int(2048 * 2048 * 16384 / (min(m, n) ** 2 * max(m, n))))
    return {"op": op, "batch": _log(rng, 1, min(8, most)), "m": m, "n": n}


def work(c):
    op = c["op"]
    if op == "embed":
        rows = c["M"] * c["D"]
        return {"bytes": 6 * rows + 8 * c["M"] + 4 * c["M"] * -(-c["D"] // 128), "flops": 4 * rows}
    if op == "embed_bwd":
        return {"bytes": 2 * c["M"] * c["D"] + 8 * c["M"] + 4 * c["V"] * c["D"], "flops": 2 * c["M"] * c["D"]}
    if op == "norm":
        e = c["M"] * c["N"]
        b = e * (7 if c["res"] else 3)  # x, res and h in bf16, codes in 8 bits; without res h is x
        return {"bytes": b + (e // 32 if c["form"] == "mx" else 0) + 4 * c["M"] + 2 * c["N"], "flops": 8 * e}
    if op == "norm_bwd":
        e = c["M"] * c["N"]
        return {"bytes": e * (8 if c["res"] else 6) + 4 * c["M"] + 6 * c["N"], "flops": 12 * e}
    m, n = min(c["m"], c["n"]), max(c["m"], c["n"])
    # a step: half of the symmetric X X^T, half of the symmetric square, the update
    return {"bytes": c["batch"] * 6 * m * n, "flops": 5 * c["batch"] * (3 * m * m * n + m ** 3)}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _tokens(g, M, V):
    """Token numbers with Zipf's frequencies; one in fifty is padding (-1)."""
    u = torch.rand(M, generator=g, device="cuda", dtype=F64)
    rank = torch.exp(u * math.log(V)).long().clamp_(1, V) - 1
    tok = (rank * 40503 + 17) % V  # frequent words lie anywhere in the table
    return torch.where(torch.rand(M, generator=g, device="cuda") < 0.02, torch.full_like(tok, -1), tok)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op == "embed":
        s["tokens"] = _tokens(g, case["M"], case["V"])
        s["E"] = _randn(g, case["V"], case["D"]).mul_(0.02).to(BF16)
        s["gamma"] = _randn(g, case["D"]).mul_(0.1).add_(1.0).to(BF16)
        s["scale"] = math.sqrt(case["D"])
    elif op == "embed_bwd":
        s["tokens"] = _tokens(g, case["M"], case["V"])
        s["dh"] = _randn(g, case["M"], case["D"]).mul_(0.01).to(BF16)
        s["scale"] = math.sqrt(case["D"])
    elif op == "norm":
        M, N = case["M"], case["N"]
        s["x"] = _randn(g, M, N).to(BF16)
        s["skip"] = _randn(g, M, N).mul_(2.0).to(BF16) if case["res"] else None
        s["gamma"] = _randn(g, N).mul_(0.1).add_(1.0).to(BF16)
        s["s_y"] = torch.full((1,), 5.0 / 448.0, device="cuda")  # an earlier step's max |y| was 5: a few larger saturate
    elif op == "norm_bwd":
        M, N = case["M"], case["N"]
        h = _randn(g, M, N).mul_(2.0)
        s["h"] = h.to(BF16)
        s["r"] = torch.rsqrt(h.square().mean(1) + EPS)
        s["dy"] = _randn(g, M, N).mul_(0.01).to(BF16)
        s["dskip"] = _randn(g, M, N).mul_(0.01).to(BF16) if case["res"] else None
        s["gamma"] = _randn(g, N).mul_(0.1).add_(1.0).to(BF16)
    else:
        # a weight's gradient: products of activations and output gradients whose features differ in size
        B, m, n = case["batch"], case["m"], case["n"]
        T = 2 * min(m, n)
        fm = torch.logspace(0, -1, m, device="cuda")[torch.randperm(m, generator=g, device="cuda")]
        fn = torch.logspace(0, -1, n, device="cuda")[torch.randperm(n, generator=g, device="cuda")]
        s["G"] = torch.stack([(_randn(g, m, T) * fm[:, None]) @ (_randn(g, T, n) * fn) * 1e-4 for _ in range(B)])
    return s


# --------------------------------------------------------------- operators


def run(s):
    op = s["op"]
    if own:
        return _own(s)
    if op == "embed":
        tok, M, D = s["tokens"], s["M"], s["D"]
        ok = (tok >= 0) & (tok < s["V"])
        h = s["E"][torch.where(ok, tok, 0)].float() * s["scale"] * ok[:, None]
        T = -(-D // 128)
        sq = torch.nn.functional.pad(h.square(), (0, T * 128 - D))
        partial = sq.view(M, T, 128).sum(2).t().contiguous()
        return {"h": h.to(BF16), "hg": (s["gamma"].float() * h).to(BF16), "partial": partial}
    if op == "embed_bwd":
        tok = s["tokens"]
        ok = (tok >= 0) & (tok < s["V"])
        dE = torch.zeros(s["V"], s["D"], device="cuda")
        return dE.index_add_(0, torch.where(ok, tok, 0), s["dh"].float() * (s["scale"] * ok[:, None]))
    if op == "norm":
        h = s["x"].float() if s["skip"] is None else s["x"].float() + s["skip"].float()
        r = torch.rsqrt(h.square().mean(1) + EPS)
        y = s["gamma"].float() * h * r[:, None]
        out = {"r": r}
        if s["skip"] is not None:
            out["h"] = h.to(BF16)
        if s["form"] == "fp8":
            out["amax"] = y.abs().amax().reshape(1)
            out["y8"] = (y / s["s_y"]).clamp(-448, 448).to(torch.float8_e4m3fn)
            return out
        M, N = s["M"], s["N"]
        yb = y.view(M, N // 32, 32)
        amax = yb.abs().amax(2)
        # the smallest power of two 2^e with amax <= 448 * 2^e; 448 = 0.875 * 2^9
        frac, exp = torch.frexp(amax)
        e = torch.where(frac <= 0.875, exp - 9, exp - 8)
        e = torch.where(amax == 0, 0, e).clamp(-127, 127)
        out["yq"] = torch.ldexp(yb, -e[:, :, None]).view(M, N).to(torch.float8_e4m3fn)
        # scale bytes in 512-byte atoms (k-block of four scales, 128 rows), padding rows 2^0
        nrb = -(-M // 128)
        b = torch.full((nrb * 128, N // 32), 127, dtype=torch.uint8, device="cuda")
        b[:M] = (e + 127).to(torch.uint8)
        b = b.view(nrb, 4, 32, N // 128, 4).permute(3, 0, 2, 1, 4).contiguous()
        out["ysf"] = b.reshape(-1).view(torch.float8_e8m0fnu)
        return out
    if op == "norm_bwd":
        h, r, gamma = s["h"].float(), s["r"], s["gamma"].float()
        dy = s["dy"].float()
        g = dy * gamma
        coef = -(r ** 3) * (g * h).sum(1) / s["N"]
        dx = g * r[:, None] + coef[:, None] * h
        if s["dskip"] is not None:
            dx = dx + s["dskip"].float()
        return {"dx": dx.to(BF16), "dgamma": (dy * h * r[:, None]).sum(0)}
    X = s["G"]
    tall = s["m"] > s["n"]
    X = X.mT if tall else X
    X = X / (X.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    a, b, c = NS
    for _ in range(5):
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    return (X.mT if tall else X).to(BF16).contiguous()


def _own(s):
    from gemm_epilogue_transformer_02_b200 import binding as coda

    op = s["op"]
    if op == "embed":
        h, hg, partial = coda.embed(s["tokens"], s["E"], s["scale"], s["gamma"])
        return {"h": h, "hg": hg, "partial": partial}
    if op == "embed_bwd":
        return coda.embed_bwd(s["tokens"], s["dh"], s["V"], s["scale"])
    if op == "norm":
        keep = s["skip"] is not None  # without a residual h is x itself
        if s["form"] == "fp8":
            h, y8, amax, r = coda.add_rmsnorm_fp8(s["x"], s["skip"], s["gamma"], EPS, s["s_y"], h=keep)
            out = {"r": r, "amax": amax, "y8": y8.view(torch.float8_e4m3fn)}
        else:
            h, yq, ysf, r = coda.add_rmsnorm_mx(s["x"], s["skip"], s["gamma"], EPS, h=keep)
            out = {"r": r, "yq": yq.view(torch.float8_e4m3fn), "ysf": ysf.view(torch.float8_e8m0fnu)}
        return {**out, "h": h} if keep else out
    if op == "norm_bwd":
        dx, dgamma = coda.add_rmsnorm_bwd(s["dy"], s["h"], s["r"], s["gamma"], s["dskip"])
        return {"dx": dx, "dgamma": dgamma}
    return coda.newton_schulz(s["G"], steps=5, coeffs=NS, eps=NS_EPS)


# ------------------------------------------------------------------- exact


def exact(case, seed):
    """What run returns, in 64 bits; codes as the values before their rounding."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        h = torch.zeros(case["M"], case["D"], dtype=F64, device="cuda")
        rows = ((s["tokens"] >= 0) & (s["tokens"] < case["V"])).nonzero()[:, 0]
        h[rows] = s["E"].index_select(0, s["tokens"][rows]).to(F64) * s["scale"]
        partial = torch.stack([t.pow(2).sum(1) for t in h.split(128, 1)])
        return {"h": h, "hg": h * s["gamma"].to(F64), "partial": partial}
    if op == "embed_bwd":
        order = torch.argsort(s["tokens"], stable=True)
        tok = s["tokens"][order]
        order, tok = order[tok >= 0], tok[tok >= 0]
        dE = torch.zeros(case["V"], case["D"], dtype=F64, device="cuda")
        return dE.index_put_((tok,), s["dh"][order].to(F64), accumulate=True).mul_(s["scale"])
    if op == "norm":
        h = s["x"].to(F64)
        if s["skip"] is not None:
            h = h + s["skip"].to(F64)
        r = 1.0 / torch.sqrt((h * h).sum(1) / case["N"] + EPS)
        y = torch.einsum("ij,i,j->ij", h, r, s["gamma"].to(F64))
        out = {"r": r, "h": h if s["skip"] is not None else None}
        if case["form"] == "fp8":
            return {**out, "amax": torch.max(torch.abs(y)).reshape(1), "y8": (y / s["s_y"].to(F64)).clamp(-448, 448)}
        yb = y.reshape(case["M"], -1, 32)
        amax = yb.abs().max(2).values
        e = torch.ceil(torch.log2(amax / 448.0))  # no block of these inputs is all zero
        return {**out, "yq": (yb / torch.exp2(e)[:, :, None]).reshape(case["M"], -1), "ysf": None}
    if op == "norm_bwd":
        h, r, gamma, dy = s["h"].to(F64), s["r"].to(F64), s["gamma"].to(F64), s["dy"].to(F64)
        xhat = h * r[:, None]
        g = dy * gamma
        dx = r[:, None] * (g - xhat * (g * xhat).mean(1, keepdim=True))
        if s["dskip"] is not None:
            dx = dx + s["dskip"].to(F64)
        return {"dx": dx, "dgamma": torch.einsum("ij,ij->j", dy, xhat)}
    # U f(sigma) V^T through the eigenvectors of the smaller Gram matrix
    a, b, c = NS
    out = []
    for G in s["G"].to(F64):
        X = G / (torch.linalg.norm(G) + NS_EPS)
        tall = case["m"] > case["n"]
        lam, U = torch.linalg.eigh(X.T @ X if tall else X @ X.T)
        sig2, f = lam.clamp(min=0), torch.ones_like(lam)
        for _ in range(5):  # f = product of the factors a + b s^2 + c s^4, s the running singular value
            q = a + b * sig2 + c * sig2 * sig2
            f, sig2 = f * q, sig2 * q * q
        P = (U * f) @ U.T
        out.append(X @ P if tall else P @ X)
    return torch.stack(out)
