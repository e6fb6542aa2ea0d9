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


@pytest.mark.parametrize("bits", [0x7f800001, 0x7f80ffff, 0xff800001, 0xff801234, 0x7fc00000])
@pytest.mark.parametrize("rows", [2, 20])
def test_every_nan_of_32_bits_makes_its_row_nan(bits, rows):
    m = Mat(384, 140, 128, True, "f32", rows)
    m.codes[77], m.zeros[0] = 0xff, 3  # all of the same sign, and none zero
    m.scales.abs_()
    m.packed = m.mv.pack(m.codes, m.scales, m.zeros)
    clean = torch.empty(rows, 140, device="cuda")
    m.mv(rows, m.x, m.packed, clean)
    m.x.view(torch.int32)[1, 77] = bits - (1 << 32 if bits >> 31 else 0)
    out = torch.empty_like(clean)
    m.mv(rows, m.x, m.packed, out)
    assert out[1].isnan().all()
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2:], clean[2:])
