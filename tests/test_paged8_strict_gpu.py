"""The operators of the paged cache of 8-bit codes at the edges of what include/cf_paged8.h allows."""
import pytest
import torch

from attention_block_gb300 import binding
from paged8_util import DT, Problem8, half_step, ref_attention8
from test_paged8_gpu import Run8, both, close

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


@pytest.mark.parametrize("q_len", [[1, 1, 1], [40, 3, 90]], ids=str)
def test_page_tables_and_lengths_written_right_in_front(q_len):
    """The page table and the lengths change on the device between calls, without a pause."""
    pr = Problem8(q_len, [300, 400, 500], 8, 2)
    other = Problem8(q_len, [290, 410, 470], 8, 2, seed=1, max_pages=pr.max_pages)
    n = pr.num_pages
    pr.k_pages, pr.v_pages = (torch.cat([a.view(torch.uint8), b.view(torch.uint8)]).view(a.dtype) for a, b in
                              ((pr.k_pages, other.k_pages), (pr.v_pages, other.v_pages)))
    pr.scales, pr.num_pages = torch.cat([pr.scales, other.scales]), n + other.num_pages
    inputs = [(pr.table.clone(), pr.lens.clone()), (torch.where(other.table >= 0, other.table + n, -7), other.lens)]
    r = Run8(pr, poison=False)

    def run(pause):
        out = []
        for i in range(40):
            pr.table.copy_(inputs[i % 2][0])
            pr.lens.copy_(inputs[i % 2][1])
            if pause:
                torch.cuda.synchronize()
            r.attend()
            if pause:
                torch.cuda.synchronize()
            out.append(r.out.clone())
        return torch.stack(out)

    want = run(True)
    assert not torch.equal(want[0], want[1])
    for _ in range(3):
        assert torch.equal(run(False), want)
    assert r.kv.status() == OK


# ------------------------------------------------------------- value scales --
def set_values(pr, scale, zero=None):
    """Value scales [num_pages, nkv, page]; heads in `zero` are held as zeros."""
    pr.scales[..., 1] = scale
    if zero is not None:
        pr.scales[..., 1][zero] = 0
        z = zero.transpose(1, 2) if pr.layout == 0 else zero
        pr.v_pages.view(torch.uint8)[z] = 0


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("log2", [-60, -45, -30, -19, 0, 40, 60])
@pytest.mark.parametrize("q_len", [[1, 1], [3, 4], [60, 130]], ids=str)
def test_zero_heads_beside_value_scales_of_any_size(code, d, log2, q_len):
    """A head of zeros weighs in the sum as exp(s), and takes nothing from the others' weights."""
    pr = Problem8(q_len, [300, 190], 4, 2, d=d, code=code)
    g = torch.Generator(device="cuda").manual_seed(7)
    shape = pr.scales.shape[:-1]
    set_values(pr, 2.0 ** log2 * (1 + torch.rand(shape, generator=g, device="cuda")) / 2 ** (log2 > 0),
               torch.rand(shape, generator=g, device="cuda") < 0.2)
    both(pr)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("log2", [-60, -45, -9])
@pytest.mark.parametrize("ahead", [3, 12, 18])
@pytest.mark.parametrize("q_len", [[1], [4], [70]], ids=str)
def test_a_first_position_of_zeros_that_takes_most_of_the_weight(code, log2, ahead, q_len):
    """Position 0 holds a value of zeros and scores some `ahead` octaves above the others."""
    pr = Problem8(q_len, [700], 4, 2, code=code)
    pr.q[..., 0] = 8.0
    at = int(pr.table[0, 0])
    top = 127.0 if code == "int8" else 448.0
    pr.k_pages.view(torch.uint8)[at, 0] = 0
    pr.k_pages[at, 0, :, 0] = int(top) if code == "int8" else torch.tensor(top).to(pr.k_pages.dtype)
    pr.scales[at, :, 0, 0] = ahead * 0.6931 * pr.d ** 0.5 / (8 * top)
    zero = torch.zeros(pr.scales.shape[:-1], dtype=torch.bool, device="cuda")
    zero[at, :, 0] = True
    set_values(pr, 2.0 ** log2, zero)
    both(pr)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("q_len", [[1], [4], [70]], ids=str)
@pytest.mark.parametrize("low,high", [(-60, 60), (-60, -9), (-33, 9), (-19, 60), (-20, 60)], ids=str)
def test_one_large_value_scale_beside_many_small_ones(code, q_len, low, high):
    """Most of exp(s) lies at positions whose values are 2^-(high - low) of the largest: they count in the sum."""
    pr = Problem8(q_len, [20000], 4, 2, code=code, page=64, q_scale=0.5)
    scale = torch.full(pr.scales.shape[:-1], 2.0 ** low, device="cuda")
    scale[int(pr.table[0, 100]), :, 5] = 2.0 ** high
    set_values(pr, scale)
    pr.scales[int(pr.table[0, 100]), :, 5, 0] = 0.5
    both(pr)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("q_len,window", [([1, 1], 0), ([4, 3], 0), ([70, 200], 0), ([70, 200], 150)], ids=str)
@pytest.mark.parametrize("order", ["up", "down", "mixed", "small"])
def test_value_scales_that_grow_fall_and_mix_along_a_sequence(code, q_len, window, order):
    """Scales from 2^-50 to 2^50, zeros among them, and NaN heads behind them; all of them small in the last case."""
    pr = Problem8(q_len, [1500, 900], 4, 2, code=code)
    g = torch.Generator(device="cuda").manual_seed(11)
    zero = torch.rand(pr.scales.shape[:-1], generator=g, device="cuda") < 0.05
    log2 = torch.randint(-50, 51, pr.scales.shape[:-1], generator=g, device="cuda").float()
    if order == "small":
        log2 = -40 - log2.abs() / 5
    for b in range(2):
        if order in ("up", "down"):
            j = torch.arange(pr.kv_len[b], device="cuda")
            x = -50 + 100 * j / (pr.kv_len[b] - 1)
            log2[pr.table[b][j // pr.page].long(), :, j % pr.page] = (x if order == "up" else -x)[:, None]
    set_values(pr, log2.exp2(), zero)
    both(pr, window)
    for b, h in ((0, 1), (1, 0)):
        pr.scales[pr.table[b, 40].long(), h, 5, 1] = NAN  # position 645
    r = Run8(pr).attend(window)
    out, tol, lse, ltol = ref_attention8(pr, window)
    for b in range(2):
        p = torch.arange(pr.kv_len[b] - q_len[b], pr.kv_len[b], device="cuda")
        hit = (p >= 645) & (p - 645 < (window or 10 ** 6))
        rows = slice(pr.starts[b], pr.starts[b + 1])
        sick = torch.zeros(q_len[b], 4, dtype=torch.bool, device="cuda")
        sick[:, 2 - 2 * b:4 - 2 * b] = hit[:, None]
        assert (r.out[rows].isnan().all(-1) == sick).all() and (r.out[rows].isnan().any(-1) == sick).all()
        assert ((r.out[rows].double() - out[rows]).abs() <= tol[rows])[~sick].all()
    assert ((r.lse.double() - lse).abs() <= ltol).all()


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("q_len", [[1, 2], [60, 130]], ids=str)
def test_scales_outside_what_is_read(code, q_len):
    """A value scale below 2^-60 counts as 0; one above 2^60 or below 0, of a key or a value, as NaN."""
    pr = Problem8(q_len, [200, 190], 4, 2, code=code)
    ids, slot = pr.table[:, 2].long(), 3  # position 35 of both sequences
    pr.scales[ids[0], 0, slot, 1] = 2.0 ** -61
    pr.scales[ids[0], 1, slot, 1] = 2.0 ** -108
    want = Problem8(q_len, [200, 190], 4, 2, code=code)
    want.scales[ids[0], :, slot, 1] = 0
    want.v_pages.view(torch.uint8)[ids[0], slot] = 0
    r = Run8(pr).attend()
    out, tol, lse, ltol = ref_attention8(want)
    rows = slice(0, q_len[0])
    assert ((r.out[rows].double() - out[rows]).abs() <= tol[rows]).all()
    assert ((r.lse[rows].double() - lse[rows]).abs() <= ltol[rows]).all()
    G, rows = pr.nq // pr.nkv, slice(q_len[0], sum(q_len))
    for side, bad in ((0, 2.0 ** 61), (0, -1.0), (0, float("inf")), (1, 2.0 ** 61), (1, -2.0 ** -70), (1, float("inf"))):
        kept = pr.scales.clone()
        pr.scales[ids[1], 1, slot, side] = bad
        r.attend()
        pr.scales.copy_(kept)
        assert r.kv.status() == OK
        assert r.out[rows, G:].isnan().all() and not r.out[rows, :G].isnan().any(), (side, bad)
        assert r.lse[rows, G:].isnan().all() == (side == 0) and not r.lse[rows, :G].isnan().any(), (side, bad)
        assert not r.out[:q_len[0]].isnan().any()


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("q_len", [[1], [4], [70]], ids=str)
@pytest.mark.parametrize("log2", [-99, -70, -53, -49, 65], ids=str)
def test_heads_of_any_size_are_appended_and_attended(code, q_len, log2):
    """bf16 values of one size, from where append holds them to the largest that attention reads: o is what is read back,
    or 0 where the scales lie below 2^-60."""
    n = 100
    pr = Problem8(q_len, [n], 4, 2, code=code)
    ap = Problem8([n], [n], 4, 2, code=code)
    ap.v = (ap.v.double().clamp(-1.9, 1.9) * 2.0 ** log2).bfloat16()
    pr.table, pr.k_pages, pr.v_pages, pr.scales = ap.table, ap.k_pages, ap.v_pages, ap.scales
    pr.num_pages = ap.num_pages
    kv = binding.Paged8Kv(**ap.config())
    kv.append(1, n, ap.q, ap.k, ap.v, ap.q_start, ap.lens, ap.table, ap.k_pages, ap.v_pages, ap.scales, ap.q)
    K, V, ks, vs = pr.held(0, 0, n)
    back = torch.full((n, 2, pr.d), NAN, dtype=torch.bfloat16, device="cuda")
    kv.read(1, n, ap.q_start, None, ap.table, ap.k_pages, ap.v_pages, ap.scales, None, back)
    want = V * vs[..., None]
    assert kv.status() == OK and want.abs().amax() > 2.0 ** log2
    assert ((back.double() - want).abs() <= 2.0 ** -8 * want.abs()).all()
    low = vs < 2.0 ** -60
    assert low.all() or not low.any()
    if low.any():
        r = Run8(pr, poison=False).attend()
        assert (r.out.double().abs() <= 2.0 ** -70).all()
        _, _, lse, ltol = ref_attention8(pr)
        assert ((r.lse.double() - lse).abs() <= ltol).all()
    else:
        both(pr)


# ----------------------------------------------------------------- queries --
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_len", [[1], [4], [70]], ids=str)
@pytest.mark.parametrize("log2", [-30, -11, -10, 0, 20])
def test_elements_of_bf16_queries_far_below_the_largest(code, d, q_len, log2):
    """A row's largest element meets keys of zero; the scores come from elements 2^-15 of it.  They count whole but in the
    many-row kernel where the largest lies between 2^-10 and 2^15: there they are multiples of 2^-24."""
    pr = Problem8(q_len, [300], 4, 2, d=d, code=code)
    pr.q = (pr.q.double() * 2.0 ** (log2 - 16)).bfloat16()
    pr.q[..., 0] = 1.5 * 2.0 ** log2
    pr.k_pages.view(torch.uint8)[..., 0] = 0
    pr.scales[..., 0] *= 2.0 ** (15 - log2)
    r = Run8(pr).attend()
    if q_len[0] * 2 > 16 and -10 <= log2 < 15:
        pr.q = pr.q.half().double()
    r.check()


# ------------------------------------------------------------------- append --
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
def test_appends_of_any_size_leave_the_same_codes_and_scales(code, dtype, d):
    """A sequence appended at once, by a call of one token to a block or of four, and in chunks down to single tokens: codes
    and scales of every position, the last page's among them, and the rotated queries are the same bits."""
    n = 1301
    pr = Problem8([n], [n], 8, 2, d=d, code=code, dtype=dtype, max_pages=90, spare=20)
    kv = binding.Paged8Kv(**pr.config())

    def appended(chunks):
        pr.k_pages.view(torch.uint8).fill_(9), pr.v_pages.view(torch.uint8).fill_(9), pr.scales.fill_(NAN)
        q_out = torch.full_like(pr.q, NAN)
        at = 0
        for c in chunks:
            rows = slice(at, at + c)
            at += c
            lens = torch.tensor([at], dtype=torch.int32, device="cuda")
            st = torch.tensor([0, c], dtype=torch.int32, device="cuda")
            kv.append(1, c, pr.q[rows], pr.k[rows], pr.v[rows], st, lens, pr.table, pr.k_pages, pr.v_pages, pr.scales, q_out[rows])
        assert at == n and kv.status() == OK
        return [q_out] + list(pr.held(0, 0, n)) + [pr.k_pages.clone(), pr.v_pages.clone(), pr.scales.clone()]

    want = appended([n])
    assert all(torch.isfinite(x).all() for x in want[:5])
    for chunks in ([1221, 64, 1, 7, 1, 1, 5, 1], [400, 1, 900], [1] * 21 + [1280]):
        for a, b in zip(appended(chunks), want):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ------------------------------------------------------------- reading back --
@pytest.mark.parametrize("start,rows", [
    ([0, 100, 8, 10], 10), ([0, 5, 3, 10], 10), ([9, 30, -1, 4, 9, 6, 9, 30], 30), ([40, 0, 20, 40], 40),
    ([0] + [2 ** 31 - 1] * 3 + [4, 9, 17], 20), ([t if t % 7 else 1000 for t in range(301)], 300),
    ([3, 3, 3, 7, 7, 20], 23)], ids=["far", "falling", "mixed", "swapped", "limit", "many", "in order"])
def test_rows_beside_malformed_starts_are_read(start, rows):
    """A sequence whose starts decrease or leave the rows has none, the others have theirs."""
    batch = len(start) - 1
    pr = Problem8([1] * batch, [30 + 3 * (b % 9) for b in range(batch)], 4, 2, d=64, max_pages=4)
    kv = binding.Paged8Kv(**pr.config())
    k, v = (torch.full((rows, 2, 64), 99.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kv.read(batch, rows, torch.tensor(start, dtype=torch.int32, device="cuda"), None, pr.table, pr.k_pages, pr.v_pages,
            pr.scales, k, v)
    ordered = all(0 <= a <= b <= rows for a, b in zip(start, start[1:]))
    assert kv.status() == (OK if ordered else RANGE)
    want = [torch.full((rows, 2, 64), 99.0, dtype=torch.float64, device="cuda") for _ in range(2)]
    twice = torch.zeros(rows, dtype=torch.int32, device="cuda")
    for b, (a, e) in enumerate(zip(start, start[1:])):
        if 0 <= a <= e <= rows and e - a <= pr.kv_len[b]:
            K, V, ks, vs = pr.held(b, 0, e - a)
            want[0][a:e], want[1][a:e] = K * ks[..., None], V * vs[..., None]
            twice[a:e] += 1
    assert (twice == 1).any()
    for got, w in zip((k, v), want):
        one = twice < 2  # what a row holds that two claim is unspecified
        close(got[one], w[one], half_step("bf16") * (1 + 2.0 ** -10) * w[one].abs(), "rows")


# ------------------------------------------------------ calls without tokens --
@pytest.mark.parametrize("batch", [1, 32, 33, 300])
@pytest.mark.parametrize("max_q", [1, 40])
def test_tokens_of_no_sequence_are_left_alone(batch, max_q):
    """A padded call: n_tokens rows, none of which belongs to a sequence."""
    pr = Problem8([0] * batch, [30 + b % 7 for b in range(batch)], 8, 2, d=64, extra_tokens=50)
    r = Run8(pr)
    before = [pr.k_pages.clone(), pr.v_pages.clone(), pr.scales.clone()]
    q_out = torch.full_like(pr.q, 7.0)
    r.out.fill_(7), r.lse.fill_(7)
    for _ in range(2):
        r.attend(max_q=max_q)
        r.kv.append(batch, pr.tokens, pr.q, pr.k, pr.v, pr.q_start, pr.lens, pr.table, pr.k_pages, pr.v_pages, pr.scales, q_out)
        assert r.kv.status() == OK
    for x in (r.out, r.lse, q_out):
        assert (x == 7).all()
    for x, y in zip(before, (pr.k_pages, pr.v_pages, pr.scales)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("code,dtype", [("e4m3", "bf16"), ("int8", "f16")])
@pytest.mark.parametrize("heads", [(300, 1), (257, 1), (514, 2), (1000, 1)], ids=str)
def test_more_grouped_heads_than_a_tile_has_rows(code, dtype, heads):
    both(Problem8([1, 3, 2], [40, 70, 2], *heads, d=64, dtype=dtype, code=code))
