"""Products with 4-bit weights on the GPU against float64.

Tolerance: x, codes and zeros enter exactly; a sum of k products in fp32 is off
by k e sum|x w| at most, e = 2^-23 (tensor-core sums may truncate), the scales'
products and the sum of the groups by as much per group, and out is rounded by
half a step of its type: u |out| + (k + 8) e sum_k |x_k| |W_kn| + (8 e + u) |residual|
(the residual is added in fp32)."""
import math

import pytest
import torch

from attention_block_gb300 import binding

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E = 2.0 ** -23
INVALID, ALIAS = binding.CF_ERR_INVALID_ARG, binding.CF_ERR_ALIAS


class Mat:
    def __init__(self, k, n, group=128, zeros=False, dtype="bf16", rows=1, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = DT[dtype]
        self.k, self.n, self.group, self.dtype, self.rows = k, n, group, dtype, rows
        self.codes = torch.randint(0, 256, (k, n // 2), generator=g, device="cuda", dtype=torch.uint8)
        self.scales = (0.01 * torch.randn(k // group, n, generator=g, device="cuda")).to(dt)
        self.zeros = torch.randint(0, 16, (k // group, n), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
        self.x = torch.randn(rows, k, generator=g, device="cuda").to(dt)
        self.residual = torch.randn(rows, n, generator=g, device="cuda").to(dt)
        self.mv = binding.W4Matvec(in_features=k, out_features=n, group=group, zeros=zeros, max_rows=rows, dtype=dtype)
        self.packed = self.mv.pack(self.codes, self.scales, self.zeros)

    def weights(self):
        c = torch.stack([self.codes & 15, self.codes >> 4], -1).view(self.k, self.n).double()
        z = self.zeros.double() if self.zeros is not None else torch.full_like(self.scales, 8).double()
        return (c - z.repeat_interleave(self.group, 0)) * self.scales.double().repeat_interleave(self.group, 0)

    def want(self, x=None, residual=None):
        x = self.x if x is None else x
        W, xd = self.weights(), x.double()
        y = xd @ W
        u = torch.finfo(DT[self.dtype]).eps / 2
        tol = (self.k + 8) * E * (xd.abs() @ W.abs())
        if residual is not None:
            y = y + residual.double()
            tol = tol + (8 * E + u) * residual.double().abs()
        tol = tol + u * y.abs()
        if self.dtype == "f16":
            tol = tol + 2.0 ** -25
        return y, tol

    def check(self, residual=False, x=None):
        out = torch.full((self.rows, self.n), float("nan"), dtype=DT[self.dtype], device="cuda")
        r = self.residual if residual else None
        self.mv(self.rows, self.x if x is None else x, self.packed, out, residual=r)
        y, tol = self.want(x, r)
        same = (out.double() == y) | (out.isnan() & y.isnan())
        bad = ~same & ~((out.double() - y).abs() <= tol)
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: " \
            f"{out[bad][0]} for {y[bad][0]} (tol {tol[bad][0]})"
        return out


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 16, 17, 33, 64])
def test_rows_groups_and_types(dtype, group, zeros, rows):
    Mat(5 * group, 210, group, zeros, dtype, rows).check(residual=rows % 2 == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("k,n,group", [(32, 2, 32), (32, 64, 32), (64, 66, 64), (96, 130, 32), (128, 62, 128), (160, 18, 32),
                                       (4096, 4096, 128), (11008, 514, 64), (14336, 1000, 128), (256, 30000, 128),
                                       (1 << 20, 8, 128)])
@pytest.mark.parametrize("rows", [1, 16])
def test_sizes(dtype, k, n, group, rows):
    Mat(k, n, group, True, dtype, rows, seed=k + n).check(residual=True)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_strided_rows_and_fewer_rows_than_the_handle_has(dtype):
    m = Mat(256, 130, 64, True, dtype, 12)
    wide = torch.full((12, 512), float("nan"), dtype=DT[dtype], device="cuda")
    wide[:, 128:384] = m.x
    a = m.check()
    b = m.check(x=wide[:, 128:384])
    assert torch.equal(a, b)
    for rows in (0, 1, 3, 9):
        out = torch.full((12, 130), 5.0, dtype=DT[dtype], device="cuda")
        m.mv(rows, m.x, m.packed, out)
        assert torch.equal(out[:rows], a[:rows]) and (out[rows:] == 5).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows", [3, 20])
def test_what_is_not_finite_stays_in_its_row(dtype, rows):
    m = Mat(384, 140, 128, True, dtype, rows)
    clean = m.check()
    m.x[1, 5], m.x[2, 200], m.x[0, 383] = math.inf, math.nan, 6e4 if dtype == "f16" else 2.0 ** 100
    out = m.check()
    assert not out[1].isfinite().any() and out[2].isnan().all()
    assert torch.equal(out[3:], clean[3:])


def test_residual_in_place_and_streams():
    m = Mat(512, 200, 128, False, "bf16", 4)
    want = m.check(residual=True)
    out = m.residual.clone()
    m.mv(4, m.x, m.packed, out, residual=out)
    assert torch.equal(out, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out2 = torch.empty_like(out)
    m.mv(4, m.x, m.packed, out2, residual=m.residual, stream=s)
    s.synchronize()
    assert torch.equal(out2, want)


@pytest.mark.parametrize("rows", [1, 16])
def test_packing_and_products_in_a_row_and_in_a_graph(rows):
    """Weights are packed anew right in front of the product that reads them."""
    a, b = Mat(1024, 700, 64, True, "f16", rows, 1), Mat(1024, 700, 64, True, "f16", rows, 2)
    want = [a.check(), b.check()]
    packed = torch.empty_like(a.packed)
    outs = [torch.empty_like(want[0]) for _ in range(2)]

    def step():
        for m, o in zip((a, b), outs):
            a.mv.pack(m.codes, m.scales, m.zeros, packed=packed)
            a.mv(rows, m.x, packed, o)

    for _ in range(5):
        step()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_refusals():
    m = Mat(256, 128, 64, True, "bf16", 4)
    out = torch.empty(4, 128, dtype=torch.bfloat16, device="cuda")
    lib, h = binding.lib(), m.mv.handle
    x, p, o = m.x.data_ptr(), m.packed.data_ptr(), out.data_ptr()
    for args, code in [((-1, x, 256, p, None, o), INVALID), ((5, x, 256, p, None, o), INVALID),
                       ((1, None, 256, p, None, o), INVALID), ((1, x + 2, 256, p, None, o), INVALID),
                       ((1, x, 248, p, None, o), INVALID), ((1, x, 257, p, None, o), INVALID),
                       ((1, x, 256, None, None, o), INVALID), ((1, x, 256, p + 8, None, o), INVALID),
                       ((1, x, 256, p, None, None), INVALID), ((1, x, 256, p, o + 1, o), INVALID),
                       ((4, x, 1 << 41, p, None, o), INVALID),
                       ((4, x, 256, p, None, x + 1024), ALIAS), ((4, x, 256, p, None, p + 128), ALIAS),
                       ((4, x, 256, p, o + 256, o), ALIAS)]:
        assert lib.cf_w4_matvec(h, *args, None) == code, args
    c, s, z = m.codes.data_ptr(), m.scales.data_ptr(), m.zeros.data_ptr()
    for args, code in [((None, s, z, p), INVALID), ((c, None, z, p), INVALID), ((c, s, None, p), INVALID),
                       ((c, s, z, None), INVALID), ((c, s, z, p + 4), INVALID), ((c, s + 1, z, p), INVALID),
                       ((p, s, z, p), ALIAS), ((c, p + 16, z, p), ALIAS), ((c, s, p, p), ALIAS)]:
        assert lib.cf_w4_pack(h, *args, None) == code, args
    for bad in (lambda: m.mv(4, m.x.float(), m.packed, out), lambda: m.mv(4, m.x[:3], m.packed, out),
                lambda: m.mv(4, m.x, m.packed[:100], out), lambda: m.mv(4, m.x, m.packed, out[:, :64]),
                lambda: m.mv(4, m.x.cpu(), m.packed, out), lambda: m.mv.pack(m.codes, m.scales),
                lambda: m.mv.pack(m.codes.T, m.scales, m.zeros), lambda: m.mv.pack(m.codes, m.scales.float(), m.zeros)):
        with pytest.raises(binding.CfError):
            bad()
