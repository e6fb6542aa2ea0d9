"""The operators of the paged cache of 8-bit codes at the edges of what include/cf_paged8.h allows."""
import pytest
import torch

from attention_block_gb300 import binding
from paged8_util import DT, Problem8

pytestmark = pytest.mark.gpu
OK, RANGE = binding.CF_OK, binding.CF_ERR_DEVICE_POS_RANGE
CODES = ["e4m3", "int8"]
NAN = float("nan")


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("q_len", [[1, 1, 1], [40, 3, 90]], ids=str)
def test_reading_back_sees_the_append_in_front(code, q_len):
    """Other keys and values appended to the same slots and read back, over and over without a pause."""
    pr = Problem8(q_len, [n + 30 for n in q_len], 4, 2, code=code)
    kv = binding.Paged8Kv(**pr.config())
    n = sum(pr.kv_len)
    start = torch.tensor([sum(pr.kv_len[:b]) for b in range(4)], dtype=torch.int32, device="cuda")
    gain = [2.0 ** (i % 7 - 3) for i in range(40)]
    ks, vs = [pr.k * x for x in gain], [pr.v / x for x in gain]
    q_out = torch.empty_like(pr.q)

    def run(pause):
        out = []
        for k, v in zip(ks, vs):
            o = torch.full((2, n, pr.nkv, pr.d), NAN, dtype=DT[pr.dtype], device="cuda")
            kv.append(3, pr.tokens, pr.q, k, v, pr.q_start, pr.lens, pr.table, pr.k_pages, pr.v_pages, pr.scales, q_out)
            if pause:
                torch.cuda.synchronize()
            kv.read(3, n, start, None, pr.table, pr.k_pages, pr.v_pages, pr.scales, o[0], o[1])
            if pause:
                torch.cuda.synchronize()
            out.append(o)
        return torch.stack(out)

    want = run(True)
    assert not want.isnan().any()
    for _ in range(3):
        assert torch.equal(run(False), want)
    assert kv.status() == OK
