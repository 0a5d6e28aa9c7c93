"""A product prepared with a weight that has been freed since is refused, not run."""
import pytest
import torch

from dense_fp8_gemm_b200 import spense

pytestmark = pytest.mark.gpu


def test_prepared_product_of_a_freed_weight_is_refused():
    q, s = spense.mx4_quantize(torch.randn(256, 512, device="cuda"), scale_rows=True)
    pw = spense.mx4_pack(q, s)
    xq, xs = spense.mx4_quantize(torch.randn(5, 512, device="cuda"))
    y = torch.zeros(5, 256, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    ws = spense.new_workspace(spense.mx4_workspace_size(pw, 5))
    calls = [spense.PreparedMx4Gemm(pw, xq, xs, y, ws), spense.PreparedMx4Gemm(pw, xq, xs, y, ws, offsets=off)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    before = y.clone()
    pw.free()
    pw.free()                                                 # a second time is nothing
    for call in calls:
        with pytest.raises(spense.SpenseError) as e:
            call()
        assert e.value.code == 1
    for again in (lambda: spense.mx4_gemm(pw, xq, xs, Y=y, workspace=ws), lambda: spense.mx4_workspace_size(pw, 5)):
        with pytest.raises(spense.SpenseError):
            again()
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), before.view(torch.int16)) and spense.workspace_status(ws) == 0
