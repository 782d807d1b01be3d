"""Layer norm backward for the weight's and bias's gradient alone: without a dx there
is nothing that the flag to add to dx could add to."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(3, 100), (70, 512), (70, 4096), (40, 9000), (5, 13001)])
def test_add_dx_without_dx(rows, cols):
    import torch
    import gradient_sync_zr_amd as z
    for dt in (torch.bfloat16, torch.float32):
        x, dy = (torch.randn(rows, cols, device="cuda").to(dt) for _ in range(2))
        w, mean, rstd = torch.randn(cols, device="cuda"), torch.randn(rows, device="cuda"), torch.rand(rows, device="cuda")
        ws = torch.empty(max(4, z.zr_layernorm_workspace_bytes(rows, cols)), dtype=torch.uint8, device="cuda")
        sides = []
        for add in (False, True):
            dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
            z.zr_layernorm_bwd(dy, x, rows, cols, mean, rstd, w, dweight=dw, dbias=db, add_dx=add, workspace=ws)
            sides.append((dw, db))
        assert all(torch.equal(a, b) for a, b in zip(*sides))
