"""Calls from several host threads at once (GPU)."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from fp64_gemm_emulation_gb300 import ozaki as oz


@pytest.mark.parametrize("k", [8192, 8191, 16384])
def test_norm_gradients_with_and_without_dh_at_once(k):
    # The two forms need different amounts of shared memory, whose limit all threads share.  The library is called without the
    # binding's work around it, so that the threads are inside it at the same time.
    gen = torch.Generator(device="cuda").manual_seed(k)
    rows, calls = 2, 20000
    dy, h, dh = (torch.randn(rows, k, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3))
    w, rstd = torch.randn(k, generator=gen, device="cuda").to(torch.bfloat16), torch.rand(rows, generator=gen, device="cuda")
    nbytes = oz.ozaki_rms_norm_backward_workspace_bytes(k, rows)
    lanes = []
    for i in range(4):
        more = dh if i % 2 else None
        stream, ws = torch.cuda.Stream(), torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        dx, dw = torch.empty_like(dy), torch.empty_like(w)
        args = (k, rows, oz.OZ_BF16, dy.data_ptr(), k, h.data_ptr(), k, w.data_ptr(), rstd.data_ptr(), more.data_ptr() if i % 2 else None, k,
                dx.data_ptr(), k, dw.data_ptr(), ws.data_ptr(), nbytes, stream.cuda_stream)
        lanes.append((args, dx, dw, oz.ozaki_rms_norm_backward(dy, h, w, rstd, more), ws, stream))
    torch.cuda.synchronize()
    start, refused = threading.Barrier(len(lanes)), [0] * len(lanes)

    def work(i):
        args, call = lanes[i][0], oz._lib.ozaki_rms_norm_backward_ws
        start.wait()
        for _ in range(calls):
            refused[i] += call(*args) != oz.OZ_OK

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(lanes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0] * len(lanes)
    for _, dx, dw, want, _, _ in lanes:
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
