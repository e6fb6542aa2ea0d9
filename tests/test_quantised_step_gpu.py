"""A decode step in 8 and 4 bits as it is used: projections with 4-bit weights
around a paged cache of 8-bit codes, for a batch whose lengths grow, captured
once and replayed; each stage against float64 on what the stage in front gave
it, and the whole against the block in float64."""
import math

import pytest
import torch

from attention_block_gb300 import binding
from paged8_util import E, Problem8, half_step, ref_attention8

pytestmark = pytest.mark.gpu
OK = binding.CF_OK


def quantise4(w, group):
    """Codes, scales and zeros of w [K, N], a scale and a zero point per group and column."""
    k, n = w.shape
    g = w.view(k // group, group, n)
    lo, hi = g.amin(1), g.amax(1)
    scale = ((hi - lo) / 15).to(torch.bfloat16)
    zero = (-lo / scale.float()).round().clamp(0, 15)
    c = ((g / scale.float()[:, None]).round() + zero[:, None]).clamp(0, 15).to(torch.uint8).view(k, n)
    return c[:, 0::2] | c[:, 1::2] << 4, scale, zero.to(torch.uint8), \
        ((c.view(k // group, group, n).double() - zero.double()[:, None]) * scale.double()[:, None]).view(k, n)


class Linear:
    def __init__(self, k, n, rows, g, group=64):
        w = torch.randn(k, n, generator=g, device="cuda") / math.sqrt(k)
        codes, scales, zeros, self.w = quantise4(w, group)
        self.mv = binding.W4Matvec(in_features=k, out_features=n, group=group, zeros=True, max_rows=rows, dtype="bf16")
        self.packed = self.mv.pack(codes, scales, zeros)
        self.k, self.rows = k, rows

    def __call__(self, x, out, residual=None):
        return self.mv(x.shape[0], x, self.packed, out, residual=residual)

    def check(self, x, out, residual=None):
        y = x.double() @ self.w
        tol = (self.k + 8) * E * (x.double().abs() @ self.w.abs())
        if residual is not None:
            y, tol = y + residual.double(), tol + 16 * E * residual.double().abs()
        assert ((out.double() - y).abs() <= tol + half_step("bf16") * y.abs()).all()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("q_len,heads", [([1] * 5, (8, 2)), ([4, 4, 4], (4, 4)), ([9, 1, 20], (8, 2))], ids=["step", "drafts", "chunks"])
def test_a_step_of_the_block(code, q_len, heads):
    nq, nkv = heads
    d, T = 64, sum(q_len)
    hidden = nq * d
    g = torch.Generator(device="cuda").manual_seed(5)
    pr = Problem8(q_len, [n + 30 + 17 * b for b, n in enumerate(q_len)], nq, nkv, d=d, code=code, max_pages=12, spare=30)
    spare = sorted(set(range(pr.num_pages)) - set(pr.table.flatten().tolist()))
    for b in range(pr.batch):  # pages for what is to come
        for i in range(pr.max_pages):
            if pr.table[b, i] < 0 and i * pr.page < pr.kv_len[b] + 4 * q_len[b]:
                pr.table[b, i] = spare.pop()
    qkv_lin, o_lin = Linear(hidden, (nq + 2 * nkv) * d, T, g), Linear(hidden, hidden, T, g)
    kv = binding.Paged8Kv(**pr.config())
    x = torch.empty(T, hidden, dtype=torch.bfloat16, device="cuda")
    qkv = torch.empty(T, (nq + 2 * nkv) * d, dtype=torch.bfloat16, device="cuda")
    q, k, v = (t.view(T, -1, d) for t in (qkv[:, :nq * d], qkv[:, nq * d:(nq + nkv) * d], qkv[:, (nq + nkv) * d:]))
    qr, attn, out = (torch.empty(T, nq, d, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    out = out.view(T, hidden)
    starts = None if max(q_len) == 1 else pr.q_start

    def step():
        norm = (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)
        qkv_lin(norm, qkv)
        kv.append(pr.batch, T, q, k, v, starts, pr.lens, pr.table, pr.k_pages, pr.v_pages, pr.scales, qr)
        kv.attention(pr.batch, T, pr.max_q, qr, starts, pr.lens, pr.table, pr.k_pages, pr.v_pages, pr.scales, attn)
        o_lin(attn.view(T, hidden), out, residual=x)
        return norm

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    x.normal_(generator=g)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
        with torch.cuda.graph(graph, stream=side):
            norm = step()
    for turn in range(3):
        x.normal_(generator=g)
        pr.lens += torch.tensor(q_len, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert kv.status() == OK and qkv_lin.mv.status() == OK
        pr.kv_len = pr.lens.tolist()
        qkv_lin.check(norm, qkv)
        pr.q = qr
        want, tol, _, _ = ref_attention8(pr)
        assert ((attn.double() - want).abs() <= tol).all()
        o_lin.check(attn.view(T, hidden), out, residual=x)
        # the whole in float64, over what the cache holds: bf16 between the stages, four roundings
        xd = x.double()
        y = (xd * torch.rsqrt(xd.square().mean(-1, keepdim=True) + 1e-6)) @ qkv_lin.w
        rate = 1e4 ** (-torch.arange(0, d, 2, device="cuda").double() / d)
        pos = torch.cat([torch.arange(pr.kv_len[b] - n, pr.kv_len[b], device="cuda") for b, n in enumerate(q_len)])
        z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos.double()[:, None] * rate)[:, None]
        yq = y[:, :nq * d].view(T, nq, d)
        yq = torch.complex(yq[..., :d // 2], yq[..., d // 2:]) * z
        pr.q = torch.cat([yq.real, yq.imag], -1)
        block = xd + ref_attention8(pr)[0].view(T, hidden) @ o_lin.w
        assert (out.double() - block).norm() <= 8 * half_step("bf16") * block.norm()
