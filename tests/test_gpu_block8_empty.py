"""8-bit quantisation of matrices without elements (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from fp64_gemm_emulation_gb300 import ozaki as oz


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("block", ["column", "both"])
def test_no_rows_with_offsets(block, dtype):
    # every block that the groups are laid out in is there, with zeros and scales of 1
    o = torch.zeros(4, dtype=torch.int32, device="cuda")
    got = oz.ozaki_quantize_f8(torch.empty(0, 136, dtype=dtype, device="cuda"), block, o)
    q, s = got[-2:]
    assert q.shape == (3 * 128, 136) and (q.float() == 0).all() and s.shape == (3, 136) and (s == 1).all()
    if block == "both":
        assert got[0].shape == (0, 136) and got[1].shape == (0, 2)
    assert oz.ozaki_get_device_status() == oz.OZ_OK


@pytest.mark.parametrize("shape", [(0, 3, 40, 136), (2, 3, 0, 136), (2, 3, 40, 0), (0, 40, 136), (0, 136), (3, 2, 1, 1)])
def test_batches_without_elements(shape):
    q, s = oz.ozaki_quantize_f8(torch.ones(shape, dtype=torch.bfloat16, device="cuda"), "matrix")
    assert q.shape == shape and s.shape == (*shape[:-2], -(-shape[-2] // 128), -(-shape[-1] // 128))
    assert torch.equal(q.float(), torch.full(shape, 448.0, device="cuda"))


def test_batches_that_lie_unevenly_are_refused():
    x = torch.ones(3, 4, 40, 136, dtype=torch.bfloat16, device="cuda")[:, :2]
    with pytest.raises((ValueError, RuntimeError)):
        oz.ozaki_quantize_f8(x, "matrix")
