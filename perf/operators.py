"""Cases of the expert products and of the Newton-Schulz orthogonalisation, to be timed and checked.

Grouped products: the rows of x (rows, k) are sorted by expert, expert e owns the rows
offsets[e] .. offsets[e+1]-1, and w (experts, n, k) holds one weight matrix for each expert.
  forward    y[r]  = w[e] x[r]                              y  (rows, n)
  backward   dx[r] = w[e]^T dy[r],  dw[e] = sum_r dy[r] x[r]^T    dx (rows, k), dw (experts, n, k)

Newton-Schulz: each matrix g (m, n) of a batch becomes x = g / (|g|_F + eps) and then, steps times,
x <- a x + (b A + c A^2) x with A = x x^T, which takes its singular values towards 1 (the update of
an optimiser that orthogonalises its momentum).  For m > n the same polynomial acts from the right.

`own` chooses between the plain form (elementary torch operations in 32 bits) and the library.
"""
import math

import torch

own = False

STEPS = 5
COEFFS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # Serving one token: eight of 64 experts see one row each.  Latency and the weights' bytes.
        {"name": "forward one token", "op": "forward", "dtype": "bf16", "rows": 8, "experts": 64, "k": 2048, "n": 1024, "skew": 0.0},
        # Serving a batch of 64 tokens, four experts each, among 128: a few rows for each expert.
        {"name": "forward decode batch", "op": "forward", "dtype": "bf16", "rows": 256, "experts": 128, "k": 2048, "n": 2048, "skew": 0.5},
        # A prompt through 32 experts, unevenly routed.
        {"name": "forward prompt", "op": "forward", "dtype": "f16", "rows": 8192, "experts": 32, "k": 4096, "n": 2048, "skew": 0.6},
        # Odd everything: rows, widths that no 16-byte row stride fits, experts without rows.
        {"name": "forward odd", "op": "forward", "dtype": "bf16", "rows": 1777, "experts": 7, "k": 1001, "n": 517, "skew": 3.0},
        # A training step's backward pass over an ordinary layer.
        {"name": "backward ordinary", "op": "backward", "dtype": "bf16", "rows": 16384, "experts": 16, "k": 2048, "n": 4096, "skew": 0.6},
        # The largest: a training batch of 65536 routed rows over 64 experts.
        {"name": "backward large", "op": "backward", "dtype": "bf16", "rows": 65536, "experts": 64, "k": 4096, "n": 2048, "skew": 0.6},
        # One small projection, where the chain of short products is all latency.
        {"name": "orthogonalise small", "op": "orthogonalise", "dtype": "f32", "batch": 1, "m": 128, "n": 128},
        # The update of all experts of a layer at once.
        {"name": "orthogonalise experts", "op": "orthogonalise", "dtype": "bf16", "batch": 24, "m": 1024, "n": 512},
        # A square projection of a middling model.
        {"name": "orthogonalise square", "op": "orthogonalise", "dtype": "bf16", "batch": 1, "m": 2048, "n": 2048},
        # Odd sizes in full precision.
        {"name": "orthogonalise odd", "op": "orthogonalise", "dtype": "f32", "batch": 1, "m": 1023, "n": 2777},
        # A tall matrix in full precision.
        {"name": "orthogonalise tall", "op": "orthogonalise", "dtype": "f32", "batch": 1, "m": 8192, "n": 2048},
        # The up projection of a large model.
        {"name": "orthogonalise large", "op": "orthogonalise", "dtype": "bf16", "batch": 1, "m": 4096, "n": 8192},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of its range; half of them multiples of 64, a quarter odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    kind = rng.random()
    if kind < 0.5:
        v = max(64, v // 64 * 64)
    elif kind < 0.75:
        v |= 1
    v = max(lo, min(hi, v))
    return v if v != 3072 else v - 64


def draw(rng):
    op = rng.choice(["forward", "backward", "orthogonalise"])
    if op == "orthogonalise":
        while True:
            c = {"op": op, "dtype": rng.choice(["bf16", "f32", "f16"]), "batch": int(round(math.exp(rng.uniform(0, math.log(32))))),
                 "m": _size(rng, 64, 8192), "n": _size(rng, 64, 8192)}
            small, big = min(c["m"], c["n"]), max(c["m"], c["n"])
            if c["batch"] * small * small * (3 * big + small) * (3 if c["dtype"] == "f32" else 1) <= 4096 * 4096 * (3 * 8192 + 4096):
                return c
    while True:
        c = {"op": op, "dtype": rng.choice(["bf16", "f16"]), "rows": _size(rng, 1, 65536), "experts": int(round(math.exp(rng.uniform(math.log(2), math.log(128))))),
             "k": _size(rng, 64, 4096), "n": _size(rng, 64, 4096), "skew": round(rng.uniform(0.0, 1.0), 2)}
        if c["rows"] * c["k"] * c["n"] <= 65536 * 4096 * 2048 and c["experts"] * c["k"] * c["n"] <= 64 * 4096 * 2048:
            return c


def _counts(case):
    """Rows of each expert, largest first: shares (i + 1)^-skew, summing to rows."""
    shares = [(i + 1) ** -case["skew"] for i in range(case["experts"])]
    total, run, cum = sum(shares), 0.0, [0]
    for s in shares:
        run += s
        cum.append(int(case["rows"] * run / total + 0.5))
    cum[-1] = case["rows"]
    return [b - a for a, b in zip(cum, cum[1:])]


def work(case):
    if case["op"] == "orthogonalise":
        m, n = sorted((case["m"], case["n"]))
        size = 4 if case["dtype"] == "f32" else 2
        # x x^T and A^2 are symmetric: half of each product is enough
        flops = case["batch"] * STEPS * (m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n)
        return {"bytes": 2 * size * case["batch"] * m * n, "flops": flops}
    rows, k, n = case["rows"], case["k"], case["n"]
    active = sum(1 for c in _counts(case) if c)
    x, y, w, offsets = 2 * rows * k, 2 * rows * n, 2 * active * n * k, 4 * (case["experts"] + 1)
    if case["op"] == "forward":
        return {"bytes": x + w + y + offsets, "flops": 2 * rows * k * n}
    dw = 2 * case["experts"] * n * k
    return {"bytes": (y + w + x) + (x + dw) + offsets, "flops": 4 * rows * k * n}


# ------------------------------------------------------------------ inputs
def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    if case["op"] == "orthogonalise":
        # A momentum: noise whose columns differ in scale, and a part of low rank as strong as it.
        b, m, n, rank = case["batch"], case["m"], case["n"], 8
        f = {"generator": gen, "device": "cuda"}
        noise = torch.randn(b, m, n, **f) * torch.exp(0.5 * torch.randn(b, 1, n, **f))
        low = torch.randn(b, m, rank, **f) @ torch.randn(b, rank, n, **f)
        g = noise + low * (noise.norm(dim=(1, 2), keepdim=True) / low.norm(dim=(1, 2), keepdim=True))
        return {"g": (0.01 * g).to(dtype)}
    rows, k, n, experts = case["rows"], case["k"], case["n"], case["experts"]
    counts = _counts(case)
    order = torch.randperm(experts, generator=torch.Generator().manual_seed(seed)).tolist()
    offsets, most = [0], 1
    for e in order:
        offsets.append(offsets[-1] + counts[e])
        most = max(most, counts[e])
    s = {"offsets": torch.tensor(offsets, dtype=torch.int32, device="cuda"), "most": most, "x": randn(rows, k)}
    w = torch.empty(experts, n, k, dtype=dtype, device="cuda")
    for e in range(experts):  # one at a time: the 32-bit noise of all experts would be twice the weights
        w[e] = randn(n, k, scale=k ** -0.5)
    s["w"] = w
    if case["op"] == "backward":
        s["dy"] = randn(rows, n, scale=0.1)
    return s


def prepare(case, seed):
    return {"op": case["op"], **_inputs(case, seed)}


# ------------------------------------------------------------------ plain forms
def _padded(s, t):
    """Rows sorted by expert as (experts, most, width) in 32 bits, zeros past each expert's rows; and where each row went."""
    offsets = s["offsets"].long()
    row = torch.arange(t.shape[0], device=t.device)
    e = torch.searchsorted(offsets[1:].contiguous(), row, right=True)
    at = e * s["most"] + row - offsets[e]
    p = torch.zeros((offsets.numel() - 1) * s["most"], t.shape[1], dtype=torch.float32, device=t.device)
    p[at] = t.float()
    return p.view(-1, s["most"], t.shape[1]), at, e


def _plain_forward(s):
    x, w = s["x"], s["w"]
    if x.shape[0] <= w.shape[0]:  # a few rows: each with its own weights
        _, _, e = _padded(s, x[:, :1])
        return torch.matmul(w[e].float(), x.float()[:, :, None])[:, :, 0].to(x.dtype)
    xp, at, _ = _padded(s, x)
    return torch.matmul(xp, w.float().transpose(1, 2)).flatten(0, 1)[at].to(x.dtype)


def _plain_backward(s):
    x, w, dy = s["x"], s["w"], s["dy"]
    yp, at, _ = _padded(s, dy)
    dx = torch.matmul(yp, w.float()).flatten(0, 1)[at].to(x.dtype)
    xp, _, _ = _padded(s, x)
    return {"dx": dx, "dw": torch.matmul(yp.transpose(1, 2), xp).to(x.dtype)}


def _plain_orthogonalise(g):
    a, b, c = COEFFS
    x = g.float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        gram = torch.matmul(x, x.transpose(1, 2))
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    return (x.transpose(1, 2) if tall else x).to(g.dtype).contiguous()


def run(state):
    op = state["op"]
    if own:
        from fp64_gemm_emulation_gb300 import ozaki as oz

        if op == "forward":
            return oz.ozaki_grouped_gemm(state["x"], state["w"], state["offsets"])
        if op == "backward":
            return {"dx": oz.ozaki_grouped_gemm_dgrad(state["dy"], state["w"], state["offsets"]),
                    "dw": oz.ozaki_grouped_gemm_wgrad(state["dy"], state["x"], state["offsets"])}
        return oz.ozaki_newton_schulz(state["g"], steps=STEPS, coeffs=COEFFS, eps=EPS)
    if op == "forward":
        return _plain_forward(state)
    if op == "backward":
        return _plain_backward(state)
    return _plain_orthogonalise(state["g"])


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "orthogonalise":
        # All steps on the smaller Gram matrix: with x = P g and A = x x^T, a step is q = a + bA + cA^2,
        # P <- q P and A <- q A q (q and A commute).
        a, b, c = COEFFS
        g = s["g"].double()
        tall = g.shape[1] > g.shape[2]
        if tall:
            g = g.transpose(1, 2)
        norm = torch.linalg.matrix_norm(g) + EPS
        gram = torch.einsum("bij,bkj->bik", g, g) / norm[:, None, None] ** 2
        eye = torch.eye(g.shape[1], dtype=torch.float64, device=g.device).expand_as(gram)
        p = eye
        for i in range(STEPS):
            q = a * eye + b * gram + c * torch.bmm(gram, gram)
            p = q if i == 0 else torch.bmm(q, p)
            if i + 1 < STEPS:
                gram = torch.bmm(q, torch.bmm(gram, q))
        x = torch.bmm(p, g) / norm[:, None, None]
        return x.transpose(1, 2).contiguous() if tall else x
    offsets = s["offsets"].tolist()
    x, w = s["x"], s["w"]
    y = torch.zeros(x.shape[0], w.shape[1] if case["op"] == "forward" else w.shape[2], dtype=torch.float64, device=x.device)
    if case["op"] == "forward":
        for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
            y[lo:hi] = torch.einsum("rk,nk->rn", x[lo:hi].double(), w[e].double())
        return y
    dw = torch.zeros(w.shape, dtype=torch.float64, device=x.device)
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        dy = s["dy"][lo:hi].double()
        y[lo:hi] = torch.einsum("rn,nk->rk", dy, w[e].double())
        dw[e] = torch.einsum("rn,rk->nk", dy, x[lo:hi].double())
    return {"dx": y, "dw": dw}
