"""8-bit products, quantisation, RMS norm and clipping as programs call them: streams, graphs, workspaces, refusals, a training step (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from fp64_gemm_emulation_gb300 import ozaki as oz
    from fp64_gemm_emulation_gb300 import run_experts

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(autouse=True)
def clean_status():
    oz.ozaki_get_device_status()
    yield
    assert oz.ozaki_get_device_status() == oz.OZ_OK


def randn(*shape, dtype=torch.float32, seed=0, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def layer(rows=700, n=320, k=264, counts=(300, 0, 250, 150), seed=0):
    at = [0]
    for c in counts:
        at.append(at[-1] + c)
    o = torch.tensor(at, dtype=torch.int32, device="cuda")
    return (randn(rows, k, dtype=torch.bfloat16, seed=seed), randn(rows, k, dtype=torch.bfloat16, seed=seed + 1), randn(len(counts), n, k, dtype=torch.bfloat16, seed=seed + 2),
            (1 + randn(k, seed=seed + 3, scale=0.1)).to(torch.bfloat16), randn(rows, n, dtype=torch.bfloat16, seed=seed + 4, scale=0.1), o)


def chain(x, res, w, gain, dy, o, stream=None):
    """A norm, the layer's three products with what quantises their operands, the norm's gradients, and clipping."""
    q, s, h, rstd = oz.ozaki_rms_norm_f8(x, gain, res, stream=stream)
    wq, ws = oz.ozaki_quantize_f8(w, "matrix", stream=stream)
    y = oz.ozaki_grouped_gemm_f8(q, s, wq, ws, o, stream=stream)
    dq, ds, dqc, dsc = oz.ozaki_quantize_f8(dy, "both", o, E5M2, stream=stream)
    dn = oz.ozaki_grouped_gemm_f8_dgrad(dq, ds, wq, ws, o, stream=stream)
    xc, xs = oz.ozaki_quantize_f8(h, "column", o, stream=stream)
    dw = oz.ozaki_grouped_gemm_f8_wgrad(dqc, dsc, xc, xs, o, stream=stream)
    dx, dgain = oz.ozaki_rms_norm_backward(dn, h, gain, rstd, stream=stream)
    out = [torch.empty_like(dw), torch.empty_like(dgain)]
    norm = oz.ozaki_clip_grad_norm([dw, dgain], 1.0, out=out, stream=stream)
    return [q.float(), s, h, rstd, y, dn, dw, dx, dgain, norm, *out]


def same(a, b):
    assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_chain_repeats_bit_for_bit():
    ops = layer()
    want = chain(*ops)
    for _ in range(20):
        same(chain(*ops), want)


def test_chain_on_other_streams_at_once():
    sets = [layer(seed=10 * i) for i in range(4)]
    want = [chain(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = [chain(*s, stream=st) for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        same(g, w)
    with torch.cuda.stream(streams[0]):
        inner = chain(*sets[1])
    torch.cuda.synchronize()
    same(inner, want[1])


def test_chain_captured_and_replayed_with_new_values():
    ops, other = layer(), layer(seed=100)
    want = chain(*other)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        chain(*ops)
        first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(first, stream=stream):
            a = chain(*ops)
        with torch.cuda.graph(second, stream=stream):
            b = chain(*ops)
    torch.cuda.synchronize()
    for t, u in zip(ops, other):
        t.copy_(u)
    for _ in range(3):
        first.replay()
        second.replay()
    torch.cuda.synchronize()
    same(a, want)
    same(b, want)


def test_group_sizes_are_read_on_the_device_at_replay():
    x, _, w, _, dy, o = layer()
    q, s = oz.ozaki_quantize_f8(x, "row")
    wq, ws = oz.ozaki_quantize_f8(w, "matrix")

    def both():
        return [oz.ozaki_grouped_gemm_f8(q, s, wq, ws, o),
                oz.ozaki_grouped_gemm_f8_wgrad(*oz.ozaki_quantize_f8(dy, "column", o), *oz.ozaki_quantize_f8(x, "column", o), o)]

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        both()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = both()
    torch.cuda.synchronize()
    for counts in ([0, 0, 0, 0, 700], [0, 1, 2, 699, 700], [5, 5, 400, 401, 690]):
        o.copy_(torch.tensor(counts, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        same(got, both())


def test_workspaces_of_the_caller():
    x, _, w, gain, dy, _ = layer(k=264, n=264)
    _, _, h, rstd = oz.ozaki_rms_norm_f8(x, gain)
    ws = torch.empty(oz.ozaki_rms_norm_backward_workspace_bytes(264, 700), dtype=torch.uint8, device="cuda")
    same(oz.ozaki_rms_norm_backward_ws(dy, h, gain, rstd, ws), oz.ozaki_rms_norm_backward(dy, h, gain, rstd))
    cw = torch.empty(oz.ozaki_clip_grad_norm_workspace_bytes(), dtype=torch.uint8, device="cuda")
    a, b = [x.clone(), w.clone()], [x.clone(), w.clone()]
    assert torch.equal(oz.ozaki_clip_grad_norm_ws(a, 1.0, cw), oz.ozaki_clip_grad_norm(b, 1.0))
    same(a, b)
    for bad in (ws.cpu(), torch.empty(2 * ws.numel(), dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            oz.ozaki_rms_norm_backward_ws(dy, h, gain, rstd, bad)
        with pytest.raises(ValueError, match="workspace"):
            oz.ozaki_clip_grad_norm_ws(a, 1.0, bad)
    with pytest.raises(oz.OzakiError):
        oz.ozaki_rms_norm_backward_ws(dy, h, gain, rstd, ws[:256])


def test_given_outputs_are_used_and_checked():
    x, _, w, _, dy, o = layer()
    q, s = oz.ozaki_quantize_f8(x, "row")
    wq, ws = oz.ozaki_quantize_f8(w, "matrix")
    y = torch.empty(700, 320, dtype=torch.float16, device="cuda")
    assert oz.ozaki_grouped_gemm_f8(q, s, wq, ws, o, Y=y) is y
    assert torch.equal(y, oz.ozaki_grouped_gemm_f8(q, s, wq, ws, o, dtype=torch.float16))
    for bad in (y[:, :300], y[:10], y.t(), y.cpu()):
        with pytest.raises(ValueError):
            oz.ozaki_grouped_gemm_f8(q, s, wq, ws, o, Y=bad)
    with pytest.raises(ValueError):
        oz.ozaki_grouped_gemm_f8(q, s, wq, ws, o, Y=y, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        oz.ozaki_grouped_gemm_f8(q, s, wq, ws, o, dtype=torch.float32)


def test_refusals():
    x, res, w, gain, dy, o = layer()
    q, s = oz.ozaki_quantize_f8(x, "row")
    wq, ws = oz.ozaki_quantize_f8(w, "matrix")
    dqc, dsc = oz.ozaki_quantize_f8(dy, "column", o)
    xqc, xsc = oz.ozaki_quantize_f8(x, "column", o)
    _, _, h, rstd = oz.ozaki_rms_norm_f8(x, gain)
    value = [
        lambda: oz.ozaki_grouped_gemm_f8(q, s.contiguous(), wq, ws, o),                 # scales by row
        lambda: oz.ozaki_grouped_gemm_f8(q, s[:, :2], wq, ws, o),
        lambda: oz.ozaki_grouped_gemm_f8(q, s.double(), wq, ws, o),
        lambda: oz.ozaki_grouped_gemm_f8(q, s, wq, ws[:, :1], o),
        lambda: oz.ozaki_grouped_gemm_f8(q, s, wq, ws.transpose(1, 2), o),
        lambda: oz.ozaki_grouped_gemm_f8(q, s, wq[..., :200], ws, o),
        lambda: oz.ozaki_grouped_gemm_f8(q, s, wq, ws),                                 # four groups without offsets
        lambda: oz.ozaki_grouped_gemm_f8(q, s, wq, ws, o[:4]),
        lambda: oz.ozaki_grouped_gemm_f8(q, s, wq, ws, o.long()),
        lambda: oz.ozaki_grouped_gemm_f8(q, s, wq, ws, o.cpu()),
        lambda: oz.ozaki_grouped_gemm_f8(q.float().to(E4M3)[:, :264].contiguous()[:, 8:], s, wq, ws, o),  # rows at odd addresses
        lambda: oz.ozaki_grouped_gemm_f8(q.contiguous(), s, wq, ws, o) if 264 % 16 else 1 / 0,
        lambda: oz.ozaki_grouped_gemm_f8(q, s, wq.cpu(), ws, o),
        lambda: oz.ozaki_grouped_gemm_f8_wgrad(dqc, dsc, xqc[:-128], xsc[:-1], o),
        lambda: oz.ozaki_grouped_gemm_f8_wgrad(dqc, dsc[:-1], xqc, xsc, o),
        lambda: oz.ozaki_grouped_gemm_f8_wgrad(dqc, dsc, xqc, xsc, o, rows=100),
        lambda: oz.ozaki_grouped_gemm_f8_wgrad(dqc, dsc, xqc, xsc, rows=100),
        lambda: oz.ozaki_grouped_gemm_f8_wgrad(dqc, dsc, xqc, xsc, o, dW=torch.empty(4, 320, 260, dtype=torch.bfloat16, device="cuda")),
        lambda: oz.ozaki_quantize_f8(x, "matrix", o),
        lambda: oz.ozaki_quantize_f8(x[0], "row"),
        lambda: oz.ozaki_quantize_f8(x.t(), "row"),
        lambda: oz.ozaki_quantize_f8(x, "column", o.cpu()),
        lambda: oz.ozaki_rms_norm_f8(x, gain[:-1]),
        lambda: oz.ozaki_rms_norm_f8(x, gain.float()),
        lambda: oz.ozaki_rms_norm_f8(x, gain, res[:-1]),
        lambda: oz.ozaki_rms_norm_f8(x, gain, res.float()),
        lambda: oz.ozaki_rms_norm_f8(torch.empty(1, 40000, device="cuda"), torch.empty(40000, device="cuda")),
        lambda: oz.ozaki_rms_norm_backward(x, h, gain, rstd.double()),
        lambda: oz.ozaki_rms_norm_backward(x, h[:, :-1], gain, rstd),
        lambda: oz.ozaki_rms_norm_backward(x, h, gain, rstd[:-1]),
        lambda: oz.ozaki_clip_grad_norm([x, w.cpu()], 1.0),
        lambda: oz.ozaki_clip_grad_norm([x.t()], 1.0),
        lambda: oz.ozaki_clip_grad_norm([x], 1.0, out=[]),
        lambda: oz.ozaki_clip_grad_norm([x], 1.0, out=[x[:-1]]),
        lambda: oz.ozaki_clip_grad_norm([x], 1.0, out=[x.float()]),
    ]
    for i, call in enumerate(value):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was not refused")
    for call in (lambda: oz.ozaki_quantize_f8(x.double()), lambda: oz.ozaki_quantize_f8(x, dtype=torch.float16), lambda: oz.ozaki_grouped_gemm_f8(x, s, wq, ws, o),
                 lambda: oz.ozaki_rms_norm_f8(x.double(), gain.double()), lambda: oz.ozaki_clip_grad_norm([x.double()], 1.0)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(oz.OzakiError):
        oz.ozaki_rms_norm_f8(x, gain, eps=-1.0)
    with pytest.raises(oz.OzakiError):
        oz.ozaki_clip_grad_norm([x], -1.0)


def test_offsets_past_32_bits():
    # 2^17 + 200 rows, 2^15 features: elements past 2^32 of the operands, past 2^31 of the outputs
    rows, k, n = (1 << 17) + 200, 1 << 15, 64
    x = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(0))
    q, s = oz.ozaki_quantize_f8(x, "row")
    tail = slice(rows - 300, rows)
    for got, want in zip((q[tail], s[tail]), oz.ozaki_quantize_f8(x[tail], "row")):
        assert torch.equal(got.float(), want.float())
    wq, ws = oz.ozaki_quantize_f8(randn(n, k, seed=1, scale=k ** -0.5), "matrix")
    y = oz.ozaki_grouped_gemm_f8(q, s, wq, ws)
    want = oz.ozaki_grouped_gemm_f8(*oz.ozaki_quantize_f8(x[tail], "row"), wq, ws)
    assert torch.equal(y[tail], want)
    o = torch.tensor([0, rows - 300, rows], dtype=torch.int32, device="cuda")
    dyq, dys = oz.ozaki_quantize_f8(randn(rows, n, dtype=torch.bfloat16, seed=2), "column", o)
    del q, s
    xq, xs = oz.ozaki_quantize_f8(x, "column", o)
    dw = oz.ozaki_grouped_gemm_f8_wgrad(dyq, dys, xq, xs, o)
    first = torch.zeros(2, dtype=torch.int32, device="cuda")
    first[1] = 300
    alone = oz.ozaki_grouped_gemm_f8_wgrad(*oz.ozaki_quantize_f8(randn(rows, n, dtype=torch.bfloat16, seed=2)[tail].contiguous(), "column", first),
                                           *oz.ozaki_quantize_f8(x[tail], "column", first), first)
    assert torch.equal(dw[1], alone[0])
    del xq, xs, dyq, dys
    gain = randn(k, dtype=torch.bfloat16, seed=3)
    got = oz.ozaki_rms_norm_f8(x, gain, x)
    for a, b in zip(got, oz.ozaki_rms_norm_f8(x[tail], gain, x[tail])):
        assert torch.equal(a[tail].float(), b.float())


# ------------------------------------------------------------------ a wait that runs out
def test_an_expired_wait_is_reported_and_the_next_call_is_right():
    x, _, w, _, dy, o = layer()
    q, s = oz.ozaki_quantize_f8(x, "row")
    wq, ws = oz.ozaki_quantize_f8(w, "matrix")
    dq, ds, dqc, dsc = oz.ozaki_quantize_f8(dy, "both", o)
    xqc, xsc = oz.ozaki_quantize_f8(x, "column", o)
    calls = [lambda: oz.ozaki_grouped_gemm_f8(q, s, wq, ws, o), lambda: oz.ozaki_grouped_gemm_f8_dgrad(dq, ds, wq, ws, o),
             lambda: oz.ozaki_grouped_gemm_f8_wgrad(dqc, dsc, xqc, xsc, o)]
    for call in calls:
        want = call()
        oz.ozaki_set_epilogue_wait_ns(0)
        try:
            call()
            assert oz.ozaki_get_device_status() == oz.OZ_ETIMEOUT
        finally:
            oz.ozaki_set_epilogue_wait_ns(-1)
        assert torch.equal(call(), want)


# ------------------------------------------------------------------ a training step
def test_eight_bit_layer_gradients():
    rows, experts, k, n = 500, 3, 200, 160
    gen = torch.Generator(device="cuda").manual_seed(0)
    _, o = run_experts.route(torch.randint(experts, (rows,), generator=gen, device="cuda"), experts)
    x, w = randn(rows, k, dtype=torch.bfloat16, seed=1), randn(experts, n, k, dtype=torch.bfloat16, seed=2, scale=k ** -0.5)
    gain, target = (1 + randn(k, seed=3, scale=0.1)).to(torch.bfloat16), randn(rows, n, dtype=torch.bfloat16, seed=4)
    lay = run_experts.EightBitExpertLayer(w.clone(), gain.clone())
    loss, dx, dw, dgain = lay.gradients(x, o, target)

    X, G = x.double(), gain.double()
    rstd = (X.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    normed = X * rstd * G
    at = o.tolist()

    def by_expert(a, b, f):
        return torch.cat([f(a[lo:hi], b[e]) for e, (lo, hi) in enumerate(zip(at, at[1:]))])

    y = by_expert(normed, w.double(), lambda t, m: t @ m.T)
    dy = (y - target.double()) / rows
    dn = by_expert(dy, w.double(), lambda t, m: t @ m)
    want_w = torch.stack([dy[lo:hi].T @ normed[lo:hi] for lo, hi in zip(at, at[1:])])
    dz = dn * G
    z = X * rstd
    want_x = rstd * (dz - z * (dz * z).mean(1, keepdim=True))
    want_gain = (dn * z).sum(0)
    # Quantising moves a value by at most 2^-4 (e4m3) or 2^-3 (e5m2) of it, or by 2^-10 / 448 of its block's largest,
    # which 2^-4 of 2^-13 of the matrix's largest covers; with 2^-8 for what was rounded to bfloat16 before (the norm's result
    # for the column blocks, dy, dn), and 2^-6 of it all for FP32's roundings and products of small terms.
    q4, q5, more = 1 + 2.0 ** -4, 1 + 2.0 ** -3, 1 + 2.0 ** -6

    def size(t):
        return t.abs() + 2.0 ** -13 * t.abs().max()

    sx, sw = size(normed) * (1 + 2.0 ** -8), size(w.double())
    ey = by_expert(sx, sw, lambda t, m: t @ m.T) * (q4 * q4 - 1) * more
    sdy = (dy.abs() + ey / rows) * (1 + 2.0 ** -8)
    sdy = sdy + 2.0 ** -13 * sdy.max()
    edn = (by_expert(sdy, sw, lambda t, m: t @ m) * q5 * q4 * (1 + 2.0 ** -8) - by_expert(dy.abs(), w.double().abs(), lambda t, m: t @ m)) * more
    ew = (torch.stack([sdy[lo:hi].T @ sx[lo:hi] for lo, hi in zip(at, at[1:])]) * q5 * q4
          - torch.stack([dy[lo:hi].abs().T @ normed[lo:hi].abs() for lo, hi in zip(at, at[1:])])) * more
    ez = edn * G.abs()
    ex = rstd * (ez + z.abs() * (ez * z.abs()).mean(1, keepdim=True)) * more
    eg = (edn * z.abs()).sum(0) * more
    for got, want, off in ((dx, want_x, ex), (dw, want_w, ew), (dgain, want_gain, eg)):
        assert ((got.double() - want).abs() <= off + 2.0 ** -8 * (want.abs() + off)).all()
    d, e = (y - target.double()).abs(), ey + 2.0 ** -8 * (y.abs() + ey)
    want = 0.5 * d.square().sum() / rows
    assert abs(loss.item() - want.item()) <= (0.5 * (2 * d * e + e.square()).sum() / rows).item() * more


def test_eight_bit_training_runs():
    losses = run_experts.train(300, 4, 128, 96, 3, eight_bit=True)
    assert len(losses) == 3 and all(l == l and l < float("inf") for l in losses)


def test_sixteen_bit_training_is_as_it_was():
    assert run_experts.train(300, 4, 128, 96, 2) == run_experts.train(300, 4, 128, 96, 2, eight_bit=False, clip=0.5)
