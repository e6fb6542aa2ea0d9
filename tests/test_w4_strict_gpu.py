"""Products with 4-bit weights at the edges of what include/cf_w4.h allows."""
import pytest
import torch

from attention_block_gb300 import binding
from test_w4_gpu import DT, Mat

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows", [1, 5, 16])
def test_a_product_reads_what_the_launches_in_front_wrote(dtype, rows):
    """y += x W1 in place, then z = y W2, over and over without a pause: rows of y whose bytes are no multiple of 32, so
    that blocks share sectors.  The same calls with a pause behind each give the same bits."""
    first, second = Mat(512, 520, 64, True, dtype, rows, 3), Mat(512, 264, 128, False, dtype, rows, 4)

    def run(pause):
        y = first.residual.clone()
        out = []
        for _ in range(60):
            z = torch.empty(rows, 264, dtype=DT[dtype], device="cuda")
            first.mv(rows, first.x, first.packed, y, residual=y)
            if pause:
                torch.cuda.synchronize()
            second.mv(rows, y[:, :512], second.packed, z)
            if pause:
                torch.cuda.synchronize()
            out.append(z)
        return torch.stack(out + [y[:, :264].clone()])

    want = run(True)
    for _ in range(3):
        assert torch.equal(run(False), want)
    assert first.mv.status() == binding.CF_OK and second.mv.status() == binding.CF_OK
