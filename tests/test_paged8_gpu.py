"""The operators of the paged cache of 8-bit codes on the GPU against float64 (paged8_util)."""
import math

import pytest
import torch

from attention_block_gb300 import binding
from paged8_util import CODE, DT, E, Problem8, check_codes, half_step, quantise, ref_attention8, ref_rope
from paged_util import axes_of

pytestmark = pytest.mark.gpu
OK, RANGE = binding.CF_OK, binding.CF_ERR_DEVICE_POS_RANGE
TYPES = ["bf16", "f16"]
CODES = ["e4m3", "int8"]
NAN = float("nan")


def close(got, want, tol, what):
    got, want = got.double(), want.double()
    same = (got == want) | (got.isnan() & want.isnan())
    err = torch.where(same, torch.zeros_like(want), (got - want).abs())
    bad = ~(err <= tol.nan_to_num(0))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at " \
        f"{bad.nonzero()[0].tolist()}: {got[bad][0]} for {want[bad][0]} (tol {tol[bad][0]})"


class Run8:
    def __init__(self, pr, poison=True, **cfg):
        self.pr = pr
        if poison:
            self.poison()
        self.kv = binding.Paged8Kv(**pr.config(**cfg))
        self.out = torch.full((pr.tokens, pr.nq, pr.d), NAN, dtype=DT[pr.dtype], device="cuda")
        self.lse = torch.full((pr.tokens, pr.nq), NAN, device="cuda")

    def poison(self):
        """Scales of slots that no row sees are NaN."""
        pr = self.pr
        seen = torch.zeros(pr.num_pages, pr.page, dtype=torch.bool, device="cuda")
        for b in range(pr.batch):
            j = torch.arange(max(pr.kv_len[b], 0), device="cuda")
            seen[pr.table[b][j // pr.page].long(), j % pr.page] = True
        pr.scales[~seen[:, None, :, None].expand_as(pr.scales)] = NAN

    def attend(self, window=0, sinks=0, q_start="own", max_q=None, stream=None, lse=True, q=None):
        pr = self.pr
        self.kv.attention(pr.batch, pr.tokens, max_q or pr.max_q, pr.q if q is None else q,
                          pr.q_start if isinstance(q_start, str) else q_start, pr.lens, pr.table, pr.k_pages,
                          pr.v_pages, pr.scales, self.out, lse=self.lse if lse else None, window=window,
                          n_sinks=sinks, stream=stream)
        return self

    def check(self, window=0, sinks=0, what="", **kw):
        assert self.kv.status() == OK
        out, tol, lse, ltol = ref_attention8(self.pr, window, sinks, **kw)
        close(self.out, out, tol, what + " out")
        close(self.lse, lse, ltol, what + " lse")
        return self


def both(pr, window=0, sinks=0, **cfg):
    Run8(pr, **cfg).attend(window, sinks).check(window, sinks)


# ------------------------------------------------------------------ attention --
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads", [(4, 4), (8, 2), (7, 1), (16, 1), (6, 2), (32, 1)], ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_single_tokens(code, dtype, heads, d):
    kv = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 777]
    both(Problem8([1] * len(kv), kv, *heads, d=d, dtype=dtype, code=code))


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("page", [1, 2, 8, 16, 64, 256])
@pytest.mark.parametrize("layout,inter", [(0, False), (1, False), (0, True), (1, True)])
def test_pages(code, page, layout, inter):
    for q_len in ([1, 2, 1], [40, 90, 3]):
        both(Problem8(q_len, [300, 257, 31], 8, 2, page=page, code=code, layout=layout, interleaved=inter))


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_len,kv_len", [
    ([3, 0, 2, 4], [40, 9, 2, 130]), ([1, 5, 16, 0, 7], [1, 5, 300, 20, 1000]),
    ([64, 1, 129, 2], [64, 400, 500, 7]), ([300, 17], [2000, 17]), ([257], [1281])], ids=str)
def test_ragged_tokens(code, dtype, d, q_len, kv_len):
    both(Problem8(q_len, kv_len, 8, 2, d=d, dtype=dtype, code=code, extra_tokens=2))
    both(Problem8(q_len, kv_len, 4, 4, d=d, dtype=dtype, code=code))


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (17, 0), (64, 4), (100, 130), (128, 1), (513, 16),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("q_len,kv_len", [([1, 1, 1, 1], [1, 65, 300, 513]), ([5, 70, 300], [700, 70, 900])], ids=str)
def test_window_and_sinks(code, window, sinks, q_len, kv_len):
    both(Problem8(q_len, kv_len, 8, 2, code=code, dtype="f16"), window, sinks)
    both(Problem8(q_len, kv_len, 3, 3, d=64, code=code), window, sinks)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("q_len", [[1, 1, 0], [9, 3, 2], [200, 40, 30]], ids=str)
def test_rows_that_see_nothing(code, q_len):
    # sequences of no positions, and more tokens than positions: p < 0
    pr = Problem8(q_len, [0, max(q_len[1] - 1, 0), 0], 4, 2, code=code)
    r = Run8(pr).attend()
    out, tol, lse, ltol = ref_attention8(pr)
    close(r.out, out, tol, "out")
    close(r.lse, lse, ltol, "lse")


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", TYPES)
def test_large_and_small_queries_share_a_tile(code, dtype):
    """bf16 queries far beyond fp16's range beside ordinary and tiny ones."""
    pr = Problem8([4, 70], [90, 200], 4, 1, dtype=dtype, code=code)
    big = 2.0 ** 20 if dtype == "bf16" else 2.0 ** 8
    for t in (1, 10, 40):
        pr.q[t] *= big
        pr.q[t + 1] /= big
    pr.scales[..., 0] /= big  # scores of the large rows stay finite and ordinary
    both(pr)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_len,kv_len", [([4, 1], [90, 33]), ([300, 700, 40], [500, 700, 2000])], ids=str)
def test_queries_that_are_not_finite_stay_in_their_rows(dtype, q_len, kv_len):
    pr = Problem8(q_len, kv_len, 8, 2, dtype=dtype)
    if dtype == "bf16":  # a power of two of its own for this row, beside the others
        pr.q[2] *= 2.0 ** 20
        pr.scales[..., 0] /= 2.0 ** 20
    out, tol, lse, ltol = ref_attention8(pr)
    q = pr.q.clone()
    q[0, 3, 5] = NAN
    q[1, 6, 0] = float("inf")
    q[pr.tokens - 1, 0, pr.d - 1] = -float("inf")
    r = Run8(pr).attend(q=q)
    assert r.kv.status() == OK
    assert r.out[0, 3].isnan().all() and r.lse[0, 3].isnan()
    for t, h in ((0, 3), (1, 6), (pr.tokens - 1, 0)):
        out[t, h], tol[t, h] = r.out[t, h].to(out), 0
        lse[t, h], ltol[t, h] = r.lse[t, h].to(lse), 0
    close(r.out, out, tol, "out")
    close(r.lse, lse, ltol, "lse")


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("q_len", [[1, 1, 1], [3, 2, 1], [100, 40, 17]], ids=str)
def test_scales_of_many_sizes_and_zero(code, q_len):
    pr = Problem8(q_len, [300, 140, 17], 4, 2, code=code, dtype="f16")
    g = torch.Generator(device="cuda").manual_seed(3)
    pr.scales[..., 1] *= torch.exp2(torch.randint(-20, 6, pr.scales.shape[:-1], generator=g, device="cuda").float())
    zero = torch.rand(pr.scales.shape, generator=g, device="cuda") < 0.2
    pr.scales[zero] = 0
    for i, pool in enumerate((pr.k_pages, pr.v_pages)):  # as append leaves them
        z = zero[..., i].transpose(1, 2) if pr.layout == 0 else zero[..., i]
        pool.view(torch.uint8)[z] = 0
    both(pr)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("q_len,kv_len,window", [([1, 1], [50, 300], 0), ([4, 3], [50, 300], 0),
                                                 ([60, 130], [300, 131], 0), ([60, 130], [300, 131], 20)], ids=str)
def test_nan_heads_reach_the_rows_that_see_them(code, q_len, kv_len, window):
    """A NaN scale of a key makes o and lse of the rows that see it NaN, one of a value o alone."""
    pr = Problem8(q_len, kv_len, 4, 2, code=code, dtype="f16")
    at = [(0, kv_len[0] - 1, 0, 0), (1, kv_len[1] - 2, 1, 1), (0, 3, 1, 0), (1, 7, 0, 1)]  # sequence, position, head, side
    for b, j, h, side in at:
        pr.scales[pr.table[b, j // pr.page].long(), h, j % pr.page, side] = NAN
    out, tol, lse, ltol = ref_attention8(pr, window)
    r = Run8(pr).attend(window)
    G = pr.nq // pr.nkv
    for b in range(2):
        for i in range(q_len[b]):
            p, t = kv_len[b] - q_len[b] + i, pr.starts[b] + i
            for h in range(pr.nq):
                hit = [any(x[0] == b and x[2] == h // G and x[3] == side and x[1] <= p and
                           (not window or p - x[1] < window) for x in at) for side in (0, 1)]
                assert bool(r.out[t, h].isnan().all()) == (hit[0] or hit[1]), (b, i, h)
                assert bool(r.out[t, h].isnan().any()) == (hit[0] or hit[1]), (b, i, h)
                assert bool(r.lse[t, h].isnan()) == hit[0], (b, i, h)


@pytest.mark.parametrize("code", CODES)
def test_scale_strided_queries_and_no_lse(code):
    for q_len, kv_len in (([1, 1], [40, 70]), ([30, 50], [40, 70])):
        pr = Problem8(q_len, kv_len, 4, 2, code=code)
        wide = torch.full((pr.tokens, 7, pr.d), NAN, dtype=pr.q.dtype, device="cuda")
        wide[:, 2:6] = pr.q
        r = Run8(pr, scale=0.2).attend(q=wide[:, 2:6]).check(scale=0.2)
        got = r.out.clone()
        r.out.fill_(NAN)
        r.attend(q=wide[:, 2:6], lse=False)
        assert torch.equal(r.out, got)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_len,heads", [([1] * 300, (8, 2)), ([1] * 37 + [2] * 50, (4, 4)), ([1, 40] * 40, (8, 1))],
                         ids=["300", "mixed", "prompts"])
def test_many_sequences(code, dtype, q_len, heads):
    kv = [n + (i * 37) % 401 for i, n in enumerate(q_len)]
    both(Problem8(q_len, kv, *heads, dtype=dtype, code=code))


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("q_len,kv_len,heads", [([1], [40000], (8, 2)), ([4], [33333], (4, 1)), ([513], [9000], (8, 2)),
                                                ([1, 1, 1], [20000, 5, 300], (4, 4))], ids=str)
def test_long_contexts(code, q_len, kv_len, heads):
    both(Problem8(q_len, kv_len, *heads, code=code, page=64))


# --------------------------------------------------------------------- append --
def append(pr, q_out=None, rope_pos=None, q=None, k=None, v=None, status=OK, **cfg):
    kv = binding.Paged8Kv(**pr.config(**cfg))
    q_out = torch.full_like(pr.q, NAN) if q_out is None else q_out
    kv.append(pr.batch, pr.tokens, pr.q if q is None else q, pr.k if k is None else k, pr.v if v is None else v,
              pr.q_start, pr.lens, pr.table, pr.k_pages, pr.v_pages, pr.scales, q_out, rope_pos=rope_pos)
    assert kv.status() == status
    return q_out


def check_append(pr, rope_pos=None, theta=1e4, rope_dim=0, sections=None, inter=False, **cfg):
    r = rope_dim or pr.d
    if rope_pos is None:
        pos = [pr.kv_len[b] - pr.q_len[b] + i for b in range(pr.batch) for i in range(pr.q_len[b])]
        P = [pos + [0] * (pr.tokens - len(pos))] * 3
    else:
        P = rope_pos.cpu().tolist()
    before = [pr.k_pages.clone(), pr.v_pages.clone(), pr.scales.clone()]
    q_out = append(pr, rope_pos=rope_pos, rope_theta=theta, rope_dim=rope_dim, rope_sections=sections,
                   rope_interleaved=inter, **cfg)
    n = pr.starts[-1]
    ax = axes_of(r, sections, inter)
    u = half_step(pr.dtype)
    want, s = ref_rope(pr.q.double().cpu(), P, theta, r, ax)
    close(q_out[:n].cpu(), want[:n], u * want[:n].abs() + 2.0 ** -20 * s[:n] + (2.0 ** -25 if pr.dtype == "f16" else 0), "q")
    assert q_out[n:].isnan().all()
    k, ksum = (x.cuda() for x in ref_rope(pr.k.double().cpu(), P, theta, r, ax))
    written = torch.zeros(pr.num_pages, pr.page, dtype=torch.bool, device="cuda")
    for b in range(pr.batch):
        lo = pr.kv_len[b] - pr.q_len[b]
        rows = slice(pr.starts[b], pr.starts[b + 1])
        K, V, ks, vs = pr.held(b, lo, pr.kv_len[b])
        check_codes(K, ks, k[rows], 2.0 ** -20 * ksum[rows], pr.code, f"keys of {b}")
        v = pr.v[rows].double()
        check_codes(V, vs, v, torch.zeros_like(v), pr.code, f"values of {b}")
        j = torch.arange(lo, pr.kv_len[b], device="cuda")
        written[pr.table[b][j // pr.page].long(), j % pr.page] = True
    # other slots stay as they were
    for old, new in zip(before[:2], (pr.k_pages, pr.v_pages)):
        w = written if pr.layout == 0 else written[:, None].expand(-1, pr.nkv, -1)
        assert torch.equal(old.view(torch.uint8)[~w], new.view(torch.uint8)[~w])
    w = written[:, None].expand(-1, pr.nkv, -1)
    assert torch.equal(before[2][~w], pr.scales[~w])


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout,inter", [(0, False), (1, True)])
def test_append(code, dtype, d, layout, inter):
    check_append(Problem8([3, 0, 1, 17], [40, 9, 1, 17], 6, 2, d=d, dtype=dtype, code=code, layout=layout,
                          interleaved=inter, extra_tokens=2))


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("q_len", [[1], [1400, 3]], ids=str)
def test_append_many_and_single(code, q_len):
    check_append(Problem8(q_len, [n + 5 for n in q_len], 8, 2, code=code, page=32), theta=5e5)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("d,sections,inter,rope_dim", [(128, (16, 24, 24), False, 0), (64, (12, 10, 10), True, 0),
                                                       (128, None, False, 32), (64, None, False, 16)])
def test_append_axes_and_partial_rotation(code, d, sections, inter, rope_dim):
    pr = Problem8([3, 8], [40, 8], 4, 2, d=d, code=code)
    rp = torch.randint(0, 30000, (3, pr.tokens), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).cuda()
    check_append(pr, rope_pos=rp if sections else None, sections=sections, inter=inter, rope_dim=rope_dim)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", TYPES)
def test_append_of_zeros_tiny_values_and_what_is_not_finite(code, dtype):
    pr = Problem8([6], [22], 2, 2, code=code, dtype=dtype)
    pr.k[0], pr.v[0] = 0, 0
    tiny = 2.0 ** -110 if dtype == "bf16" else 2.0 ** -24
    pr.k[1], pr.v[1] = tiny, -tiny
    pr.k[2, 0, 5], pr.v[2, 1, 7] = math.inf, -math.inf
    pr.k[3, 1, 100], pr.v[3, 0, 0] = NAN, NAN
    q = append(pr)
    K, V, ks, vs = pr.held(0, 16, 22)
    assert (K[0] == 0).all() and (V[0] == 0).all() and (ks[0] == 0).all() and (vs[0] == 0).all()
    if dtype == "bf16":
        assert (K[1] == 0).all() and (V[1] == 0).all() and (ks[1] == 0).all() and (vs[1] == 0).all()
    else:
        assert (V[1] == -CODE[code][1]).all() and (vs[1] > 0).all()
    assert ks[2, 0].isnan() and not ks[2, 1].isnan() and vs[2, 1].isnan() and not vs[2, 0].isnan()
    assert ks[3, 1].isnan() and vs[3, 0].isnan() and not q.isnan().any()
    for x, s in ((K, ks), (V, vs)):
        assert (x[s.isnan()] == 0).all()
        assert x.abs().max() == CODE[code][1]


def test_append_in_place_without_queries_and_before_the_start():
    pr = Problem8([2, 3], [20, 3], 4, 2)
    merged = torch.cat([pr.q.flatten(1), pr.k.flatten(1), pr.v.flatten(1)], 1)
    q, k, v = (merged[:, a:b].view(5, -1, 128) for a, b in ((0, 512), (512, 768), (768, 1024)))
    want = append(pr)
    kept = [pr.k_pages.clone(), pr.v_pages.clone(), pr.scales.clone()]
    pr.k_pages.view(torch.uint8).zero_(), pr.scales.zero_()
    append(pr, q=q, k=k, v=v, q_out=q)
    assert torch.equal(q, want)
    kv = binding.Paged8Kv(**pr.config())
    kv.append(pr.batch, pr.tokens, None, pr.k, pr.v, pr.q_start, pr.lens, pr.table, pr.k_pages, pr.v_pages,
              pr.scales, None)
    for b in range(2):
        j = torch.arange(pr.kv_len[b] - pr.q_len[b], pr.kv_len[b], device="cuda")
        ids = pr.table[b][j // pr.page].long()
        for i, pool in enumerate((pr.k_pages, pr.v_pages)):
            assert torch.equal(pool.view(torch.uint8)[ids, j % pr.page], kept[i].view(torch.uint8)[ids, j % pr.page])
        assert torch.equal(pr.scales[ids, :, j % pr.page], kept[2][ids, :, j % pr.page])
    pr = Problem8([4], [2], 4, 2)  # two tokens before the start
    q = append(pr, status=RANGE)
    assert q[:2].isnan().all()  # rows of tokens that are not appended stay as they were
    assert not q[2:].isnan().any()


# ----------------------------------------------------------------------- read --
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,layout,inter,page", [(64, 0, False, 16), (128, 1, True, 8), (128, 0, True, 1), (64, 1, False, 64)])
def test_read_back(code, dtype, d, layout, inter, page):
    pr = Problem8([1] * 4, [40, 9, 131, 300], 4, 2, d=d, page=page, dtype=dtype, code=code, layout=layout, interleaved=inter)
    pr.scales[pr.table[1, 3 // page].long(), :, 3 % page] = NAN
    first, count = [5, 0, 130, 17], [35, 9, 0, 200]
    start = [7 + sum(count[:b]) for b in range(5)]  # rows before the first sequence's, and behind the last's
    n = start[-1] + 3
    kv = binding.Paged8Kv(**pr.config())
    wide = torch.full((n, 5 * pr.nkv * d), 99.0, dtype=DT[dtype], device="cuda")
    k, v = wide[:, d * pr.nkv:2 * d * pr.nkv], wide[:, 3 * d * pr.nkv:4 * d * pr.nkv]
    rs = torch.tensor(start, dtype=torch.int32, device="cuda")
    kv.read(4, n, rs, torch.tensor(first, dtype=torch.int32, device="cuda"), pr.table, pr.k_pages, pr.v_pages, pr.scales, k, v)
    assert kv.status() == OK
    want = torch.full((n, 5 * pr.nkv * d), 99.0, dtype=torch.float64, device="cuda")
    for b in range(4):
        K, V, ks, vs = pr.held(b, first[b], first[b] + count[b])
        want[start[b]:start[b + 1], d * pr.nkv:2 * d * pr.nkv] = (K * ks[..., None]).flatten(1)
        want[start[b]:start[b + 1], 3 * d * pr.nkv:4 * d * pr.nkv] = (V * vs[..., None]).flatten(1)
    tol = half_step(dtype) * want.abs() * (1 + 2.0 ** -10) + (2.0 ** -25 if dtype == "f16" else 0)
    close(wide, want, tol, "rows")
    for one in (0, 1):  # keys or values alone, from position 0
        got = torch.zeros(9, pr.nkv, d, dtype=DT[dtype], device="cuda")
        rs2 = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
        kv.read(1, 9, rs2, None, pr.table[1:2].contiguous(), pr.k_pages, pr.v_pages, pr.scales, *((got, None) if one == 0 else (None, got)))
        x = pr.held(1, 0, 9)
        want = x[one] * x[2 + one][..., None]
        close(got, want, half_step(dtype) * want.abs() * (1 + 2.0 ** -10) + 2.0 ** -25, "alone")


def test_read_reports_what_lies_outside():
    pr = Problem8([1] * 3, [20, 30, 40], 4, 2, code="int8")
    kv = binding.Paged8Kv(**pr.config())

    def rows(start, first, table=None):
        k = torch.full((30, pr.nkv, pr.d), 7.0, dtype=torch.bfloat16, device="cuda")
        v = k.clone()
        kv.read(3, 30, torch.tensor(start, dtype=torch.int32, device="cuda"),
                torch.tensor(first, dtype=torch.int32, device="cuda"), pr.table if table is None else table,
                pr.k_pages, pr.v_pages, pr.scales, k, v)
        return k, v

    k, v = rows([0, 5, 8, 10], [-2, 0, 0])
    assert kv.status() == RANGE and (k[:2] == 7).all() and not (k[2:10] == 7).all() and (k[10:] == 7).all()
    k, v = rows([0, 5, 8, 10], [0, pr.max_pages * pr.page - 1, 2 ** 31 - 1])
    # (the second sequence's last entry is unset: a page outside the pool reads as zeros)
    assert kv.status() == RANGE and (k[5] == 0).all() and (k[6:8] == 7).all() and (k[8:] == 7).all()
    k, v = rows([0, 5, 3, 10], [0, 0, 0])
    assert kv.status() == RANGE
    k, v = rows([0, 5, 8, 31], [0, 0, 0])
    assert kv.status() == RANGE and (k[8:] == 7).all()
    bad = pr.table.clone()
    bad[0, 0] = pr.num_pages
    k, v = rows([0, 5, 8, 10], [0, 0, 0], bad)
    assert kv.status() == RANGE and (k[:5] == 0).all() and (v[:5] == 0).all()
    assert kv.status() == OK


# ------------------------------------------------- what the device reports --
def with_starts(starts, kv_len, tokens, heads, **kw):
    """A problem whose q_start is given as it is: malformed entries have no tokens."""
    q_len = [b - a if 0 <= a <= b <= tokens else 0 for a, b in zip(starts, starts[1:])]
    pr = Problem8(q_len, kv_len, *heads, extra_tokens=tokens - sum(q_len), **kw)
    pr.starts = list(starts)
    pr.q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    return pr


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("starts,kv_len,tokens,heads", [
    ([0, 64, 2000, 128, 192, 256, 320, 384, 448], [1000, 5, 5, 3000, 100, 64, 80, 90], 512, (8, 2)),
    ([300, 400, 200, 300, 100, 200, 0, 100], [400, 1, 300, 1, 250, 1, 700], 400, (4, 2)),
    ([8, 12, 0, 4], [20, 9, 30], 12, (1, 1)),
    ([t if t not in (100, 170) else (-3, 10 ** 9)[t > 100] for t in range(251)],
     [1 + 3 * (b % 50) for b in range(250)], 250, (8, 2)),
    ([3 * t if t != 31 else 2 ** 31 - 1 for t in range(61)], [9 + b for b in range(60)], 180, (16, 1)),
    ([5, 4, 3, 2, 1, 0], [5, 4, 3, 2, 1], 5, (8, 2)),
    ([-2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1], [50, 40, 30], 70, (8, 2)),
], ids=["far", "falling", "swapped", "singles", "drafts", "none", "limits"])
def test_sequences_beside_malformed_starts(code, starts, kv_len, tokens, heads):
    pr = with_starts(starts, kv_len, tokens, heads, code=code, d=64)
    r = Run8(pr)
    want = ref_attention8(pr)
    for _ in range(2):
        r.out.fill_(NAN), r.lse.fill_(NAN)
        r.attend()
        assert r.kv.status() == RANGE
        close(r.out, want[0], want[1], "out")
        close(r.lse, want[2], want[3], "lse")


@pytest.mark.parametrize("n", [3, 70])
def test_tokens_claimed_twice_leave_the_rest_alone(n):
    batch = 41
    pr = Problem8([n] + [0] * (batch - 1), [n + 40 + 3 * b for b in range(batch)], 8, 2, d=64, extra_tokens=2)
    r = Run8(pr)
    good = pr.q_start.clone()
    big = torch.full((3 * pr.tokens, pr.nq, pr.d), 7.0, dtype=r.out.dtype, device="cuda")
    big_lse = torch.full((3 * pr.tokens, pr.nq), 7.0, device="cuda")
    r.out, r.lse = big[pr.tokens:2 * pr.tokens], big_lse[pr.tokens:2 * pr.tokens]
    for _ in range(3):
        pr.q_start.copy_(torch.tensor([n * (b % 2) for b in range(batch + 1)], dtype=torch.int32))
        r.attend()
        assert r.kv.status() == RANGE
        pr.q_start.copy_(good)
        r.out.fill_(NAN), r.lse.fill_(NAN)
        r.attend()
        r.check()
    for x in (big, big_lse):
        assert (x[:pr.tokens] == 7).all() and (x[2 * pr.tokens:] == 7).all()


@pytest.mark.parametrize("q_len", [[1, 2, 1, 1], [60, 70, 1, 40]], ids=str)
def test_bad_lengths_and_pages_are_reported_and_stay_in_bounds(q_len):
    pr = Problem8(q_len, [80, 90, 40, 93], 4, 2, max_pages=9)
    r = Run8(pr)
    good = ref_attention8(pr)
    lens, table = pr.lens.clone(), pr.table.clone()
    pr.lens[0] = -1
    pr.lens[1] = pr.max_pages * pr.page + 1
    pr.table[2, 1] = pr.num_pages  # positions 16..31 of sequence 2 have no page
    r.attend()
    assert r.kv.status() == RANGE and r.kv.status() == OK
    n = pr.starts[2]
    assert (r.out[:n] == 0).all() and torch.isinf(r.lse[:n]).all()
    close(r.out[n + 1:], good[0][n + 1:], good[1][n + 1:], "the good sequence")
    # zeros stand for the lost positions: as if their scales were zero
    pr.table.copy_(table), pr.lens.copy_(lens)
    ids = pr.table[2, 1].long()
    pr.scales[ids] = 0
    for pool in (pr.k_pages, pr.v_pages):
        pool.view(torch.uint8)[ids] = 0
    want = ref_attention8(pr)
    close(r.out[n], want[0][n], want[1][n], "the sequence with a lost page")
    close(r.lse[n], want[2][n], want[3][n], "the sequence with a lost page")


@pytest.mark.parametrize("q_len,max_q", [([2, 3, 1], 2), ([70, 3, 40], 69)], ids=str)
def test_more_tokens_than_max_q_are_reported(q_len, max_q):
    pr = Problem8(q_len, [90, 30, 40], 4, 2)
    r = Run8(pr)
    good = ref_attention8(pr)
    r.attend(max_q=max_q)
    assert r.kv.status() == RANGE
    for b in range(3):
        rows = slice(pr.starts[b], pr.starts[b + 1])
        if q_len[b] > max_q:
            assert (r.out[rows] == 0).all() and torch.isinf(r.lse[rows]).all()
        else:
            close(r.out[rows], good[0][rows], good[1][rows], "a good sequence")


# -------------------------------------------------------------- refusals --
def test_refusals():
    pr = Problem8([1, 2], [20, 30], 4, 2)
    r = Run8(pr)
    kv, INV, ALIAS = r.kv, binding.CF_ERR_INVALID_ARG, binding.CF_ERR_ALIAS
    L, s = binding.lib(), torch.cuda.current_stream().cuda_stream
    qp, kp, vp, sp, op = (x.data_ptr() for x in (pr.q, pr.k_pages, pr.v_pages, pr.scales, r.out))
    base = dict(h=kv.handle, batch=2, n=3, max_q=2, q=qp, qs=512, st=pr.q_start.data_ptr(), kl=pr.lens.data_ptr(),
                tab=pr.table.data_ptr(), k=kp, v=vp, sc=sp, w=0, sk=0, out=op, lse=None, stream=s)

    def att(**kw):
        return L.cf_paged8_attention(*dict(base, **kw).values())

    for kw in (dict(batch=3), dict(n=4), dict(max_q=0), dict(max_q=4), dict(q=None), dict(q=qp + 2), dict(qs=511),
               dict(qs=2 ** 62), dict(st=None), dict(kl=None), dict(tab=None), dict(k=None), dict(v=vp + 8), dict(sc=None),
               dict(sc=sp + 4), dict(w=-1), dict(sk=-1), dict(out=None), dict(lse=r.lse.data_ptr() + 2)):
        assert att(**kw) == INV, kw
    for kw in (dict(out=qp), dict(out=kp), dict(out=vp), dict(out=sp), dict(lse=sp + 8), dict(lse=op),
               dict(lse=pr.table.data_ptr())):
        assert att(**kw) == ALIAS, kw
    assert att(batch=0) == OK and att(n=0) == OK
    ap = dict(h=kv.handle, b=2, n=3, q=qp, k=pr.k.data_ptr(), v=pr.v.data_ptr(), qs=512, ks=256, st=base["st"],
              kl=base["kl"], rp=None, tab=base["tab"], kp=kp, vp=vp, sc=sp, qo=op, qos=512, stream=s)

    def app(**kw):
        return L.cf_paged8_append(*dict(ap, **kw).values())

    for kw in (dict(b=3), dict(n=4), dict(st=None), dict(q=None), dict(qo=None), dict(k=None), dict(ks=255),
               dict(qos=8), dict(kp=None), dict(vp=vp + 4), dict(sc=None), dict(sc=sp + 4), dict(rp=base["st"] + 2)):
        assert app(**kw) == INV, kw
    for kw in (dict(qo=qp, qos=520), dict(qo=ap["k"]), dict(qo=kp), dict(qo=sp), dict(k=kp), dict(v=vp), dict(vp=kp),
               dict(tab=kp), dict(sc=kp), dict(sc=vp + 64), dict(k=sp)):
        assert app(**kw) == ALIAS, kw
    assert app(n=0) == OK
    out = torch.empty(2, 8, pr.nkv, pr.d, dtype=torch.bfloat16, device="cuda")
    rs = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    rd = dict(h=kv.handle, b=2, n=8, rs=rs.data_ptr(), first=None, tab=base["tab"], kp=kp, vp=vp, sc=sp,
              ko=out[0].data_ptr(), vo=out[1].data_ptr(), os=256, stream=s)

    def read(**kw):
        return L.cf_paged8_read(*dict(rd, **kw).values())

    for kw in (dict(b=3), dict(b=-1), dict(n=-1), dict(n=2 ** 30 + 1), dict(rs=None), dict(rs=rs.data_ptr() + 1),
               dict(first=rs.data_ptr() + 2), dict(tab=None), dict(kp=None), dict(vp=vp + 8), dict(sc=None),
               dict(sc=sp + 4), dict(ko=None, vo=None), dict(ko=rd["ko"] + 8), dict(os=255), dict(os=260)):
        assert read(**kw) == INV, kw
    for kw in (dict(ko=kp), dict(vo=vp), dict(ko=sp), dict(vo=rd["ko"]), dict(vo=rd["ko"] + 16), dict(ko=base["tab"] & ~15)):
        assert read(**kw) == ALIAS, kw
    assert read(n=0) == OK and read() == OK
    assert kv.status() == OK
    args = (2, 3, 2, pr.q, pr.q_start, pr.lens, pr.table, pr.k_pages, pr.v_pages, pr.scales, r.out)
    for at, bad in ((3, pr.q.float()), (3, pr.q.cpu()), (3, pr.q[:2]), (4, pr.q_start.long()), (6, pr.table[:, :1].contiguous()),
                    (7, pr.k_pages[1:]), (7, pr.k_pages.view(torch.int8)), (8, pr.v_pages.bfloat16()),
                    (9, pr.scales[1:]), (9, pr.scales.double()), (9, pr.scales.transpose(0, 1)), (10, r.out[:2])):
        with pytest.raises(binding.CfError):
            kv.attention(*args[:at], bad, *args[at + 1:])
    with pytest.raises(binding.CfError):
        kv.prefix_attention(*args)
    torch.cuda.synchronize()
    assert r.out.isnan().all()


# ------------------------------------------- streams, graphs, whole runs --
def test_offsets_past_32_bits():
    """Pools of more than 2^32 codes, scales of more than 2^31 bytes; the sequence's pages lie at their end."""
    nkv, d, page = 8, 64, 64
    num = 2 ** 32 // (nkv * d * page) + 1 << 1
    if torch.cuda.mem_get_info()[0] < 4 * num * page * nkv * d:
        pytest.skip("needs 35 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(60)
    kp, vp = (torch.zeros(num, page, nkv, d, dtype=torch.int8, device="cuda") for _ in range(2))
    scales = torch.zeros(num, nkv, page, 2, device="cuda")
    kv = binding.Paged8Kv(n_q_heads=8, n_kv_heads=nkv, head_dim=d, page_size=page, num_pages=num, max_pages=4,
                          max_batch=2, max_tokens=300, dtype="f16", code="int8")
    table = torch.tensor([[num - 1, num - 5, num - 9, num - 2], [0, 1, 2, num - 3]], dtype=torch.int32, device="cuda")
    for n in ((200, 100), (1, 1)):
        lens = torch.tensor([250, 256], dtype=torch.int32, device="cuda")
        T = sum(n)
        st = torch.tensor([0, n[0], T], dtype=torch.int32, device="cuda")
        q, k, v = (torch.randn(T, 8, d, generator=g, device="cuda").half() for _ in range(3))
        qr, o = torch.empty_like(q), torch.empty_like(q)
        kv.append(2, T, q, k, v, st, lens, table, kp, vp, scales, qr)
        kv.attention(2, T, max(n), qr, st, lens, table, kp, vp, scales, o)
        rows = torch.tensor([0, 250, 506], dtype=torch.int32, device="cuda")
        K, V = (torch.empty(506, nkv, d, dtype=torch.float16, device="cuda") for _ in range(2))
        kv.read(2, 506, rows, None, table, kp, vp, scales, K, V)
        assert kv.status() == OK
        for b in range(2):
            Kb, Vb = (x[int(rows[b]):int(rows[b + 1])].double() for x in (K, V))
            new = v[int(st[b]):int(st[b + 1])].double()
            assert ((Vb[int(lens[b]) - n[b]:] - new).abs() <= new.abs().amax(-1, keepdim=True) * (0.5 / 127 + 2.0 ** -10)).all()
            s = torch.einsum("nhd,shd->hns", qr[int(st[b]):int(st[b + 1])].double(), Kb) / math.sqrt(d)
            p = torch.arange(int(lens[b]) - n[b], int(lens[b]), device="cuda")[:, None]
            s.masked_fill_(torch.arange(int(lens[b]), device="cuda")[None] > p, -math.inf)
            want = torch.einsum("hns,shd->nhd", s.softmax(-1), Vb)
            # keys and values are read back in fp16, half a step off each
            err = (o[int(st[b]):int(st[b + 1])].double() - want).norm() / want.norm()
            assert err <= 8 * 2.0 ** -11, err


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("q_len", [[1], [3], [40]], ids=str)
def test_flat_tails_far_below_the_largest_weight_count(code, q_len):
    """One key of weight 1 and a value of 0, 20000 of 2^-26 and values of 1: the product has the tail as the sum has it.
    Scores of 0 and 18 are off by (64 + 4) 2^-23 18 at most, and by 3 2^-23 (26 + 30 + 4) with the scales' logarithms,
    weights relatively by twice that.  A weight of 2^-26 is held to 2^-33 (40 tokens) or 2^-41 of the largest."""
    n, d = q_len[0], 64
    pr = Problem8(q_len, [20000], 8, 2, d=d, page=64, code=code, dtype="f16")
    top = CODE[code][1]
    pr.k_pages.view(torch.uint8).zero_()
    ones = torch.full((1,), top, device="cuda").to(CODE[code][0]).view(torch.uint8)
    pr.v_pages.view(torch.uint8).fill_(int(ones))
    pr.scales[..., 0] = 0
    pr.scales[..., 1] = 1 / top
    pr.q.zero_()
    pr.q[..., 0] = 16.0
    ids = pr.table[0, 0].long()
    pr.k_pages.view(torch.uint8)[ids, 7, :, 0] = ones
    pr.scales[ids, :, 7, 0] = 26 * math.log(2) * 8 / 16 / top
    pr.v_pages.view(torch.uint8)[ids, 7] = 0
    pr.scales[ids, :, 7, 1] = 0
    r = Run8(pr, poison=False).attend()
    assert r.kv.status() == OK
    s = float(pr.scales[ids, 0, 7, 0]) * top * 16 / 8
    w = math.exp(-s)
    seen = torch.arange(20000 - n, 20000, dtype=torch.float64, device="cuda")
    want = (seen * w / (1 + seen * w))[:, None, None].expand(r.out.shape)
    ds, db = 68 * 2.0 ** -23 * s, 3 * 2.0 ** -23 * 60
    held = 2.0 ** -11 + (2.0 ** -34 if n * 4 > 16 else 2.0 ** -42) / w
    tol = want * (2.0 ** -11 + held + 2 * ds + 2 * db + 20008 * 2.0 ** -23) + 2.0 ** -25
    close(r.out, want, tol, "out")


@pytest.mark.parametrize("code", CODES)
def test_calls_of_every_kind_repeat_their_bits_and_graphs_replay_with_other_lengths(code):
    prs = [Problem8(q, kv, 8, 2, code=code, max_pages=40, spare=3) for q, kv in
           (([1] * 5, [600, 3, 17, 250, 1]), ([4, 2, 0, 3], [500, 90, 5, 77]), ([200, 3, 90], [600, 30, 90]))]
    runs = [Run8(p) for p in prs]
    first = []
    for r in runs:
        r.attend().check()
        first.append((r.out.clone(), r.lse.clone()))
    for _ in range(4):
        for r, f in zip(runs, first):
            r.out.fill_(NAN)
            r.attend()
            assert torch.equal(r.out, f[0]) and torch.equal(r.lse, f[1])
    graphs, streams = [], []
    for r in runs:
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            r.attend()
        graphs.append(g), streams.append(s)
    for cut in (0, 1, 0):  # the graphs at once, each on its own handle and stream
        for p, r in zip(prs, runs):
            p.lens.copy_(torch.tensor([max(n - cut * 7, q) for n, q in zip(p.kv_len, p.q_len)], dtype=torch.int32))
            r.out.fill_(NAN)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for p, r, f in zip(prs, runs, first):
            if cut == 0:
                assert torch.equal(r.out, f[0])
            else:
                out, tol, lse, ltol = ref_attention8(p, kv_len=[int(x) for x in p.lens])
                close(r.out, out, tol, "out")


def test_current_stream_and_a_stream_that_is_given():
    pr = Problem8([1, 1], [300, 17], 4, 2)
    r = Run8(pr)
    want = ref_attention8(pr)
    s = torch.cuda.Stream()
    for how in ("current", "given", "raw"):
        r.out.fill_(NAN)
        s.wait_stream(torch.cuda.current_stream())
        if how == "current":
            with torch.cuda.stream(s):
                r.attend()
        else:
            r.attend(stream=s if how == "given" else s.cuda_stream)
        s.synchronize()
        close(r.out, want[0], want[1], how)


@pytest.mark.parametrize("code,dtype", [("e4m3", "bf16"), ("int8", "f16")])
def test_prompt_in_chunks_then_steps(code, dtype):
    """A prompt appended and attended in chunks of 1, 7, 64 and 200 tokens, then steps: the cache holds the same codes
    as after one append of everything, and each row is what the reference makes of that cache."""
    n = 330
    one = Problem8([n], [n], 8, 2, code=code, dtype=dtype, max_pages=32, spare=12)
    q_rot = append(one)
    whole = [one.k_pages.clone(), one.v_pages.clone(), one.scales.clone()]
    kv = binding.Paged8Kv(**one.config())
    one.k_pages.view(torch.uint8).zero_(), one.v_pages.view(torch.uint8).zero_(), one.scales.zero_()
    out = torch.full_like(one.q, NAN)
    at = 0
    for c in (200, 64, 7, 1, 50, 1, 1, 1, 5):
        rows = slice(at, at + c)
        at += c
        lens = torch.tensor([at], dtype=torch.int32, device="cuda")
        st = torch.tensor([0, c], dtype=torch.int32, device="cuda")
        qr = torch.empty_like(one.q[rows])
        kv.append(1, c, one.q[rows], one.k[rows], one.v[rows], st, lens, one.table, one.k_pages, one.v_pages, one.scales, qr)
        assert torch.equal(qr, q_rot[rows])
        kv.attention(1, c, c, qr, st, lens, one.table, one.k_pages, one.v_pages, one.scales, out[rows])
    assert at == n and kv.status() == OK
    held = one.held(0, 0, n)
    for i, pool in enumerate((one.k_pages, one.v_pages)):
        ids = one.table[0, :-(-n // one.page)].long()
        assert torch.equal(pool.view(torch.uint8)[ids][:n // one.page], whole[i].view(torch.uint8)[ids][:n // one.page])
    assert all(torch.isfinite(x).all() for x in held)
    one.q = q_rot
    want, tol, _, _ = ref_attention8(one)
    close(out, want, tol, "out")
