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
