"""Cases of the 8-bit products and of what stands around them in a training step, to be timed and checked.

8-bit values (e4m3, e5m2) come with a 32-bit scale for each block of 128: value = q * scale.  A block is
128 neighbours of a row ("row"), 128 rows of one column ("column") or 128 x 128 of a matrix ("matrix"), the
last ones shorter; scale = max|v| / (the type's largest value), 1 for a block of zeros.
With rows sorted by expert (offsets), the blocks of a column start anew with each expert: expert e's first
block is number offsets[e] // 128 + e, and the values lie in rows 128 b .. of their block b, zeros behind
an expert's last row.

Products: rows r of expert e (one expert: a dense layer), w (experts, n, k) in matrix blocks.
  forward    y[r]  = w[e] x[r]           x in row blocks
  gradients  dx[r] = w[e]^T dy[r]        dy in row blocks
             dw[e] = sum_r dy[r] x[r]^T  both in column blocks
Quantisation: a matrix, or the rows of an activation or gradient both ways in one pass.
Root-mean-square norm: h = x + residual, y = h / sqrt(mean(h^2) + eps) * w; its results are y in 8 bits
(row blocks), h and the rows' 1 / sqrt(...).  Backward: from dy and the gradient dh that reaches h by the
residual path, dx = dh + rstd (g - h rstd^2 mean(g h)) with g = dy w, and dw = sum_r dy h rstd.
Clipping: the 2-norm over all gradients, and each times min(1, limit / (norm + 1e-6)).

`own` chooses between the plain form (elementary torch operations in 32 bits) and the library.
"""
import math

import torch

own = False

EPS = 1e-6
BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EIGHT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # Serving one token: eight of 64 experts see one row each.  Latency and the weights' bytes.
        {"name": "product one token", "op": "product", "rows": 8, "experts": 64, "k": 2048, "n": 1024, "skew": 0.0},
        # Serving a batch of 64 tokens through one wide projection.
        {"name": "product decode batch", "op": "product", "rows": 64, "experts": 1, "k": 4096, "n": 8192, "skew": 0.0},
        # A prompt through a dense layer.
        {"name": "product prompt", "op": "product", "rows": 8192, "experts": 1, "k": 4096, "n": 8192, "skew": 0.0},
        # Both gradients, odd everything: rows, widths, unevenly routed experts.
        {"name": "gradients odd", "op": "gradients", "rows": 1777, "experts": 7, "k": 1001, "n": 517, "skew": 1.0, "format": "e5m2"},
        # Both gradients of a training step's expert layer, the largest.
        {"name": "gradients large", "op": "gradients", "rows": 32768, "experts": 16, "k": 2048, "n": 4096, "skew": 0.6, "format": "e4m3"},
        # The weights of eight experts, after an update of their 32-bit masters.
        {"name": "quantise weights", "op": "quantise", "dtype": "f32", "block": "matrix", "rows": 2048, "experts": 8, "k": 4096, "skew": 0.0, "format": "e4m3"},
        # A gradient on its way into both products of the backward pass, rows sorted by expert.
        {"name": "quantise gradient", "op": "quantise", "dtype": "bf16", "block": "both", "rows": 16384, "experts": 16, "k": 4096, "skew": 0.6, "format": "e5m2"},
        # One token between two layers: latency.
        {"name": "norm one token", "op": "norm", "dtype": "bf16", "rows": 1, "k": 4096},
        # A prompt between two layers.
        {"name": "norm prompt", "op": "norm", "dtype": "bf16", "rows": 16384, "k": 4096},
        # The norm's gradients in a training step, a width that no 16-byte row stride fits.
        {"name": "norm backward odd", "op": "norm_backward", "dtype": "bf16", "rows": 7777, "k": 2049},
        # The gradients of a small model's 50 tensors.
        {"name": "clip small", "op": "clip", "dtype": "f32", "tensors": 50, "total": 400000, "limit": 1.0},
        # The gradients of a large layer stack.
        {"name": "clip large", "op": "clip", "dtype": "bf16", "tensors": 160, "total": 600000000, "limit": 1.0},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of its range; half of them multiples of 64, a quarter odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    kind = rng.random()
    if kind < 0.5:
        v = v // 64 * 64 or v
    elif kind < 0.75:
        v |= 1
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["product", "gradients", "quantise", "norm", "norm_backward", "clip"])
    skew, fmt = round(rng.uniform(0.0, 1.0), 2), rng.choice(["e4m3", "e5m2"])
    dtype = rng.choice(["bf16", "f32", "f16"])
    while True:
        experts = 1 if rng.random() < 0.4 else int(round(math.exp(rng.uniform(math.log(2), math.log(64)))))
        rows, k, n = _size(rng, 1, 32768), _size(rng, 64, 8192), _size(rng, 64, 8192)
        if op in ("product", "gradients"):
            c = {"op": op, "rows": rows, "experts": experts, "k": k, "n": n, "skew": skew}
            if op == "gradients":
                c["format"] = fmt
            if rows * k * n <= 32768 * 2048 * 4096 and experts * k * n <= 16 * 2048 * 4096:
                return c
        elif op == "quantise":
            block = rng.choice(["row", "column", "both", "matrix"])
            c = {"op": op, "dtype": dtype, "block": block, "rows": rows, "experts": experts, "k": k, "skew": skew, "format": fmt}
            if (experts if block == "matrix" else 1) * rows * k <= 8 * 2048 * 4096:
                return c
        elif op == "clip":
            total = _size(rng, 1000, 600000000)
            return {"op": op, "dtype": dtype, "tensors": min(total, _size(rng, 1, 600)), "total": total // (2 if dtype == "f32" and total > 1000 else 1),
                    "limit": rng.choice([1.0, 1e6])}
        elif rows * k <= 16384 * 4096:
            return {"op": op, "dtype": dtype, "rows": rows, "k": k}


def _counts(rows, experts, skew):
    """Rows of each expert, largest first: shares (i + 1)^-skew, summing to rows."""
    shares = [(i + 1) ** -skew for i in range(experts)]
    total, run, cum = sum(shares), 0.0, [0]
    for s in shares:
        run += s
        cum.append(int(rows * run / total + 0.5))
    cum[-1] = rows
    return [b - a for a, b in zip(cum, cum[1:])]


def _blocks(x):
    return -(-x // BLOCK)


def _lengths(case):
    """Elements of each tensor of a clip case: a few large matrices and many small vectors."""
    count, total = case["tensors"], case["total"]
    shares = [1.0 if i % 3 == 0 else 0.01 if i % 3 == 1 else 0.3 for i in range(count)]
    whole = sum(shares)
    lengths = [max(1, int(total * s / whole)) for s in shares]
    lengths[0] = max(1, lengths[0] + total - sum(lengths))
    return lengths


def work(case):
    op = case["op"]
    if op in ("product", "gradients"):
        rows, k, n, experts = case["rows"], case["k"], case["n"], case["experts"]
        active = sum(1 for c in _counts(rows, experts, case["skew"]) if c)
        w = active * (n * k + 4 * _blocks(n) * _blocks(k))
        offsets = 4 * (experts + 1) if experts > 1 else 0
        if op == "product":
            return {"bytes": rows * k + 4 * rows * _blocks(k) + w + 2 * rows * n + offsets, "flops": 2 * rows * k * n}
        columns = rows * (n + k) + 4 * (n + k) * _blocks(rows)
        return {"bytes": rows * n + 4 * rows * _blocks(n) + w + columns + 2 * rows * k + 2 * experts * n * k + offsets, "flops": 4 * rows * k * n}
    if op == "clip":
        total = sum(_lengths(case))
        return {"bytes": total * 2 * DTYPES[case["dtype"]].itemsize, "flops": 3 * total}
    rows, k, size = case["rows"], case["k"], DTYPES[case["dtype"]].itemsize
    if op == "quantise":
        if case["block"] == "matrix":
            return {"bytes": case["experts"] * (rows * k * (size + 1) + 4 * _blocks(rows) * _blocks(k)), "flops": 2 * case["experts"] * rows * k}
        row, column = case["block"] in ("row", "both"), case["block"] in ("column", "both")
        return {"bytes": rows * k * (size + row + column) + 4 * (row * rows * _blocks(k) + column * _blocks(rows) * k), "flops": 2 * rows * k * (row + column)}
    if op == "norm":
        return {"bytes": rows * k * (3 * size + 1) + size * k + 4 * rows * (_blocks(k) + 1), "flops": 7 * rows * k}
    return {"bytes": rows * k * 4 * size + 2 * size * k + 4 * rows, "flops": 10 * rows * k}


# ------------------------------------------------------------------ plain forms of the quantisation
def _scales(amax, eight):
    s = amax / LARGEST[eight]
    return torch.where(amax == 0, torch.ones_like(s), s.clamp(min=2.0 ** -126))


def _pad_to(t, rows, cols):
    return torch.nn.functional.pad(t, (0, cols - t.shape[-1], 0, rows - t.shape[-2]))


def _plain_quantise(t, block, eight):
    """t (..., rows, k) in 32 bits: its 8-bit values and their scales."""
    rows, k = t.shape[-2:]
    br, bk = {"row": (1, BLOCK), "column": (BLOCK, 1), "matrix": (BLOCK, BLOCK)}[block]
    nr, nk = -(-rows // br), -(-k // bk)
    p = _pad_to(t, nr * br, nk * bk).unflatten(-1, (nk, bk)).unflatten(-3, (nr, br))  # (..., nr, br, nk, bk)
    s = _scales(p.abs().amax(dim=(-3, -1)), eight)
    q = (p / s[..., :, None, :, None]).to(eight)
    return q.flatten(-4, -3).flatten(-2, -1)[..., :rows, :k], s


def _padded_row(offsets, rows):
    """Where row r lies once each expert's rows start a block of their own."""
    row = torch.arange(rows, device=offsets.device)
    e = torch.searchsorted(offsets[1:].contiguous(), row, right=True)
    return BLOCK * (offsets[e] // BLOCK + e) + row - offsets[e]


def _by_expert(t, offsets):
    """t's rows laid out so that column blocks start anew with each expert."""
    if offsets is None:
        return t
    rows = t.shape[0]
    p = torch.zeros(BLOCK * (rows // BLOCK + offsets.numel() - 1), t.shape[1], dtype=t.dtype, device=t.device)
    p[_padded_row(offsets.long(), rows)] = t
    return p


def _values(q, s, block):
    """The 32-bit values of 8-bit ones and their scales."""
    rows, k = q.shape[-2:]
    if block in ("row", "matrix"):
        s = s.repeat_interleave(BLOCK, -1)[..., :k]
    if block in ("column", "matrix"):
        s = s.repeat_interleave(BLOCK, -2)[..., :rows, :]
    return q.to(s.dtype) * s


# ------------------------------------------------------------------ inputs
def _padded_stride(q):
    """The same values with rows that start at multiples of 16 bytes."""
    k = q.shape[-1]
    out = torch.zeros(*q.shape[:-1], -(-k // 16) * 16, dtype=torch.uint8, device=q.device).view(q.dtype)[..., :k]
    out.copy_(q)
    return out


def _row_scales(s):
    """Scales of row blocks as the library keeps them: the rows of a block next to each other."""
    return s.t().contiguous().t()


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def randn(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    def outliers(rows, k, scale=1.0, dtype=torch.float32):  # columns of different size, as activations have
        return (torch.randn(rows, k, generator=gen, device="cuda") * (scale * torch.exp(0.7 * torch.randn(k, generator=gen, device="cuda")))).to(dtype)

    if op == "clip":
        dtype, spans, at = DTYPES[case["dtype"]], [], 0
        for length in _lengths(case):  # every tensor at a multiple of 512 bytes, as an allocator places them
            spans.append((at, length))
            at += -(-length // 256) * 256
        flat = torch.zeros(at, dtype=dtype, device="cuda")
        for start, length in spans:
            flat[start:start + length] = torch.randn(length, generator=gen, device="cuda") * 0.01
        return {"flat": flat, "out": torch.zeros_like(flat), "spans": spans, "limit": case["limit"]}
    rows, k = case["rows"], case["k"]
    if op in ("norm", "norm_backward"):
        dtype = DTYPES[case["dtype"]]
        s = {"w": (1.0 + randn(k, scale=0.1)).to(dtype)}
        if op == "norm":
            return {**s, "x": outliers(rows, k, dtype=dtype), "residual": outliers(rows, k, 2.0, dtype)}
        h = outliers(rows, k, 2.0, dtype)
        rstd = (h.float().square().mean(1) + EPS).rsqrt()
        return {**s, "h": h, "rstd": rstd, "dy": randn(rows, k, scale=0.1, dtype=dtype), "dh": randn(rows, k, scale=0.1, dtype=dtype)}
    experts, s = case["experts"], {"offsets": None, "most": rows}
    if experts > 1 and case.get("block") != "matrix":
        counts = _counts(rows, experts, case["skew"])
        order = torch.randperm(experts, generator=torch.Generator().manual_seed(seed)).tolist()
        offsets = [0]
        for e in order:
            offsets.append(offsets[-1] + counts[e])
        s["offsets"], s["most"] = torch.tensor(offsets, dtype=torch.int32, device="cuda"), max(counts)
    if op == "quantise":
        s.update(block=case["block"], eight=EIGHT[case["format"]])
        dtype = DTYPES[case["dtype"]]
        if case["block"] == "matrix":
            s["x"] = torch.stack([randn(rows, k, scale=k ** -0.5, dtype=dtype) for _ in range(experts)])
        else:
            s["x"] = outliers(rows, k, 1e-3, dtype)
        return s
    n = case["n"]
    w = [_plain_quantise(randn(n, k, scale=k ** -0.5), "matrix", torch.float8_e4m3fn) for _ in range(experts)]
    s["wq"], s["ws"] = _padded_stride(torch.stack([q for q, _ in w])), torch.stack([t for _, t in w])
    x = outliers(rows, k)
    if op == "product":
        q, t = _plain_quantise(x, "row", torch.float8_e4m3fn)
        return {**s, "xq": _padded_stride(q), "xs": _row_scales(t)}
    dy = outliers(rows, n, 0.1)
    q, t = _plain_quantise(dy, "row", EIGHT[case["format"]])
    s.update(dyq=_padded_stride(q), dys=_row_scales(t))
    for name, v, eight in (("x", x, torch.float8_e4m3fn), ("dy", dy, EIGHT[case["format"]])):
        q, t = _plain_quantise(_by_expert(v, s["offsets"]), "column", eight)
        s[name + "qc"], s[name + "sc"] = _padded_stride(q), t
    return s


def prepare(case, seed):
    s = {"op": case["op"], **_inputs(case, seed)}
    if case["op"] == "clip":
        s["grads"] = [s["flat"][at:at + length] for at, length in s["spans"]]
        s["outs"] = [s["out"][at:at + length] for at, length in s["spans"]]
    return s


# ------------------------------------------------------------------ plain forms
def _padded(s, t):
    """Rows sorted by expert as (experts, most, width), zeros past each expert's rows; where each row went, and its expert."""
    if s["offsets"] is None:
        row = torch.arange(t.shape[0], device=t.device)
        return t[None], row, torch.zeros_like(row)
    offsets = s["offsets"].long()
    row = torch.arange(t.shape[0], device=t.device)
    e = torch.searchsorted(offsets[1:].contiguous(), row, right=True)
    at = e * s["most"] + row - offsets[e]
    p = torch.zeros((offsets.numel() - 1) * s["most"], t.shape[1], dtype=t.dtype, device=t.device)
    p[at] = t
    return p.view(-1, s["most"], t.shape[1]), at, e


def _plain_product(s):
    x = _values(s["xq"], s["xs"], "row")
    rows, experts = x.shape[0], s["wq"].shape[0]
    if 1 < experts and rows <= experts:  # a few rows: each with its own weights
        _, _, e = _padded(s, x[:, :1])
        w = _values(s["wq"][e], s["ws"][e], "matrix")
        return torch.matmul(w, x[:, :, None])[:, :, 0].to(torch.bfloat16)
    xp, at, _ = _padded(s, x)
    w = _values(s["wq"], s["ws"], "matrix")
    return torch.matmul(xp, w.transpose(1, 2)).flatten(0, 1)[at].to(torch.bfloat16)


def _plain_gradients(s):
    rows = s["dyq"].shape[0]
    w = _values(s["wq"], s["ws"], "matrix")
    dyp, at, _ = _padded(s, _values(s["dyq"], s["dys"], "row"))
    dx = torch.matmul(dyp, w).flatten(0, 1)[at].to(torch.bfloat16)
    x, dy = _values(s["xqc"], s["xsc"], "column"), _values(s["dyqc"], s["dysc"], "column")
    if s["offsets"] is not None:
        row = _padded_row(s["offsets"].long(), rows)
        x, dy = x[row], dy[row]
    dw = torch.matmul(_padded(s, dy)[0].transpose(1, 2), _padded(s, x)[0]).to(torch.bfloat16)
    return {"dx": dx, "dw": dw}


def _quantised(s, t):
    out = {}
    if s["block"] == "matrix":
        out["q"], out["s"] = _plain_quantise(t, "matrix", s["eight"])
    if s["block"] in ("row", "both"):
        out["q"], out["s"] = _plain_quantise(t, "row", s["eight"])
    if s["block"] in ("column", "both"):
        out["qc"], out["sc"] = _plain_quantise(_by_expert(t, s["offsets"]), "column", s["eight"])
    return out


def _normed(s, bits):
    h = s["x"].to(bits) + s["residual"].to(bits)
    rstd = (h.square().mean(1) + EPS).rsqrt()
    q, t = _plain_quantise(h * rstd[:, None] * s["w"].to(bits), "row", torch.float8_e4m3fn)
    return {"q": q, "s": t, "h": h, "rstd": rstd}


def _norm_gradients(s, bits):
    dy, h, w, rstd = s["dy"].to(bits), s["h"].to(bits), s["w"].to(bits), s["rstd"].to(bits)[:, None]
    g = dy * w
    dx = s["dh"].to(bits) + rstd * (g - h * rstd.square() * (g * h).mean(1, keepdim=True))
    return {"dx": dx, "dw": (dy * h * rstd).sum(0)}


def run(state):
    s, op = state, state["op"]
    if own:
        return _run_own(s)
    if op == "product":
        return _plain_product(s)
    if op == "gradients":
        return _plain_gradients(s)
    if op == "quantise":
        return _quantised(s, s["x"].float())
    if op == "norm":
        r = _normed(s, torch.float32)
        return {**r, "h": r["h"].to(s["x"].dtype)}
    if op == "norm_backward":
        r = _norm_gradients(s, torch.float32)
        return {"dx": r["dx"].to(s["h"].dtype), "dw": r["dw"].to(s["w"].dtype)}
    g = s["flat"].float()  # the tensors lie in one buffer, zeros between them
    norm = g.square().sum().sqrt()
    s["out"].copy_(g * (s["limit"] / (norm + 1e-6)).clamp(max=1.0))  # (g is flat itself where that is in 32 bits)
    return {"norm": norm, "grads": s["out"]}


def _run_own(s):
    from fp64_gemm_emulation_gb300 import ozaki as oz

    op = s["op"]
    if op == "product":
        return oz.ozaki_grouped_gemm_f8(s["xq"], s["xs"], s["wq"], s["ws"], s["offsets"])
    if op == "gradients":
        return {"dx": oz.ozaki_grouped_gemm_f8_dgrad(s["dyq"], s["dys"], s["wq"], s["ws"], s["offsets"]),
                "dw": oz.ozaki_grouped_gemm_f8_wgrad(s["dyqc"], s["dysc"], s["xqc"], s["xsc"], s["offsets"])}
    if op == "quantise":
        r = oz.ozaki_quantize_f8(s["x"], s["block"], s["offsets"], s["eight"])
        names = {"both": ("q", "s", "qc", "sc"), "column": ("qc", "sc")}.get(s["block"], ("q", "s"))
        return dict(zip(names, r))
    if op == "norm":
        q, t, h, rstd = oz.ozaki_rms_norm_f8(s["x"], s["w"], s["residual"], EPS)
        return {"q": q, "s": t, "h": h, "rstd": rstd}
    if op == "norm_backward":
        dx, dw = oz.ozaki_rms_norm_backward(s["dy"], s["h"], s["w"], s["rstd"], s["dh"])
        return {"dx": dx, "dw": dw}
    norm = oz.ozaki_clip_grad_norm(s["grads"], s["limit"], out=s["outs"])
    return {"norm": norm, "grads": s["out"]}


# ------------------------------------------------------------------ 64 bits
def _exact_values(q, s, block):
    """q times its block's scale, in 64 bits, block by block."""
    v = q.double()
    step_r, step_k = (1 if block == "row" else BLOCK), (1 if block == "column" else BLOCK)
    r = torch.arange(v.shape[-2], device=v.device) // step_r
    c = torch.arange(v.shape[-1], device=v.device) // step_k
    return v * s.double()[..., r, :][..., c]


def exact(case, seed):
    s, op = _inputs(case, seed), case["op"]
    if op == "product":
        x, offsets = _exact_values(s["xq"], s["xs"], "row"), s["offsets"].tolist() if s["offsets"] is not None else [0, case["rows"]]
        y = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device=x.device)
        for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
            if lo < hi:
                y[lo:hi] = torch.einsum("rk,nk->rn", x[lo:hi], _exact_values(s["wq"][e], s["ws"][e], "matrix"))
        return y
    if op == "gradients":
        rows, experts = case["rows"], case["experts"]
        offsets = s["offsets"].tolist() if s["offsets"] is not None else [0, rows]
        dy = _exact_values(s["dyq"], s["dys"], "row")
        xc, dyc = _exact_values(s["xqc"], s["xsc"], "column"), _exact_values(s["dyqc"], s["dysc"], "column")
        dx = torch.zeros(rows, case["k"], dtype=torch.float64, device=dy.device)
        dw = torch.zeros(experts, case["n"], case["k"], dtype=torch.float64, device=dy.device)
        for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
            if lo < hi:
                dx[lo:hi] = torch.einsum("rn,nk->rk", dy[lo:hi], _exact_values(s["wq"][e], s["ws"][e], "matrix"))
                at = BLOCK * (lo // BLOCK + e)
                dw[e] = torch.einsum("rn,rk->nk", dyc[at:at + hi - lo], xc[at:at + hi - lo])
        return {"dx": dx, "dw": dw}
    if op == "clip":
        total, coef = torch.zeros((), dtype=torch.float64, device=s["flat"].device), None
        for at, length in s["spans"]:
            total = total + s["flat"][at:at + length].double().square().sum()
        coef = torch.clamp(s["limit"] / (total.sqrt() + 1e-6), max=1.0)
        return {"norm": total.sqrt(), "grads": s["flat"].double() * coef}
    if op == "quantise":
        return _exact_quantised(s)
    if op == "norm":
        h = s["x"].double().add(s["residual"].double())
        rstd = 1.0 / torch.sqrt(torch.einsum("rk,rk->r", h, h) / h.shape[1] + EPS)
        q, t = _exact_blocks((h * rstd[:, None]) * s["w"].double(), "row", torch.float8_e4m3fn)
        return {"q": q, "s": t, "h": h, "rstd": rstd}
    # By the chain rule through z = h rstd: dz = dy w, dh = rstd (dz - z mean(dz z)).
    rstd = s["rstd"].double()[:, None]
    z, dz = s["h"].double() * rstd, s["dy"].double() * s["w"].double()
    along = torch.einsum("rk,rk->r", dz, z) / z.shape[1]
    return {"dx": s["dh"].double() + (dz - z * along[:, None]) * rstd, "dw": torch.einsum("rk,rk->k", s["dy"].double(), z)}


def _exact_blocks(t, block, eight):
    """8-bit values and scales by the definition, in 64 bits: a block after another along its direction."""
    if block == "column":
        q, s = _exact_blocks(t.transpose(-2, -1), "row", eight)
        return q.transpose(-2, -1), s.transpose(-2, -1)
    tall = BLOCK if block == "matrix" else 1
    rows, k = t.shape[-2:]
    q, scales = torch.zeros_like(t), []
    for c in range(0, k, BLOCK):
        part = t[..., c:c + BLOCK]
        amax = part.abs().amax(-1)
        if tall > 1:
            amax = torch.stack([amax[..., r:r + tall].amax(-1) for r in range(0, rows, tall)], -1)
        s = torch.where(amax > 0, amax / LARGEST[eight], torch.ones_like(amax))
        scales.append(s)
        each = s.repeat_interleave(tall, -1)[..., :rows] if tall > 1 else s
        q[..., c:c + BLOCK] = (part / each[..., None]).float().to(eight).double()
    return q, torch.stack(scales, -1)


def _exact_quantised(s):
    x, out = s["x"].double(), {}
    if s["block"] == "matrix":
        out["q"], out["s"] = _exact_blocks(x, "matrix", s["eight"])
    if s["block"] in ("row", "both"):
        out["q"], out["s"] = _exact_blocks(x, "row", s["eight"])
    if s["block"] in ("column", "both"):
        if s["offsets"] is None:
            p = x
        else:
            offsets = s["offsets"].tolist()
            p = torch.zeros(BLOCK * (x.shape[0] // BLOCK + len(offsets) - 1), x.shape[1], dtype=x.dtype, device=x.device)
            for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
                at = BLOCK * (lo // BLOCK + e)
                p[at:at + hi - lo] = x[lo:hi]
        out["qc"], out["sc"] = _exact_blocks(p, "column", s["eight"])
    return out
