"""The paged cache's operators at the edges of what include/cf_paged.h allows:
malformed starts, values that are no numbers, overlaps, shapes."""
import math
from decimal import Decimal, getcontext

import pytest
import torch

from attention_block_gb300 import binding
from paged_util import Problem, half_step, ref_attention
from test_paged_gpu import OK, RANGE, TYPES, Run, check_append, close, dev, run_append

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------- malformed starts --
def with_starts(starts, kv_len, tokens, heads, **kw):
    """A problem whose starts are given: a sequence has none of the tokens
    where its start decreases or leaves them."""
    q_len = [b - a if 0 <= a <= b <= tokens else 0 for a, b in zip(starts, starts[1:])]
    pr = Problem(q_len, kv_len, *heads, extra_tokens=tokens - sum(q_len), **kw)
    pr.starts = list(starts)
    return pr


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("prefix", [0, 60])
@pytest.mark.parametrize("starts,kv_len,tokens,heads", [
    # a start far too large in front of a long sequence, which all the work lies in
    ([0, 64, 2000, 128, 192, 256, 320, 384, 448], [1000, 5, 5, 3000, 100, 64, 80, 90], 512, (8, 2)),
    ([0, 64, 2000, 128, 192, 256, 320, 384, 448], [3000, 5, 5, 70, 100, 64, 80, 90], 512, (8, 2)),
    # the sequences in falling order, the bad ones between them
    ([300, 400, 200, 300, 100, 200, 0, 100], [400, 1, 300, 1, 250, 1, 700], 400, (4, 2)),
    ([8, 12, 0, 4], [20, 9, 30], 12, (1, 1)),
    # single tokens of many sequences, two entries lost
    ([t if t not in (100, 170) else (-3, 10 ** 9)[t > 100] for t in range(251)],
     [1 + 3 * (b % 50) for b in range(250)], 250, (8, 2)),
    ([3 * t if t != 31 else 2 ** 31 - 1 for t in range(61)], [9 + b for b in range(60)], 180, (16, 1)),
    ([5, 4, 3, 2, 1, 0], [5, 4, 3, 2, 1], 5, (8, 2)),
    ([-2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1], [50, 40, 30], 70, (8, 2)),
], ids=["far", "near", "falling", "swapped", "singles", "drafts", "none", "limits"])
def test_sequences_beside_malformed_starts(dtype, prefix, starts, kv_len, tokens, heads):
    """Malformed entries are reported, their sequences have no tokens, and
    every other sequence gets its rows; twice, so that nothing stays behind."""
    pr = with_starts(starts, kv_len, tokens, heads, dtype=dtype, prefix=prefix, seed=81, d=64)
    r = Run(pr)
    want = ref_attention(pr)
    for _ in range(2):
        r.out.fill_(float("nan")), r.lse.fill_(float("nan"))
        r.attend()
        assert r.kv.status() == RANGE
        close(r.out, want[0], want[1], "out")
        close(r.lse, want[2], want[3], "lse")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("prefix", [0, 90])
@pytest.mark.parametrize("n", [3, 70])
def test_tokens_claimed_twice_leave_the_rest_alone(dtype, prefix, n):
    """Many sequences that claim the same tokens: the call ends, reports them,
    writes nothing beside its outputs, and the next call finds all as it was."""
    batch = 41
    pr = Problem([n] + [0] * (batch - 1), [n + 40 + 3 * b for b in range(batch)], 8, 2, d=64,
                 dtype=dtype, prefix=prefix, extra_tokens=2, seed=88)
    r = Run(pr)
    good = r.q_start.clone()
    big = torch.full((3 * pr.tokens, pr.nq, pr.d), 7.0, dtype=r.out.dtype, device="cuda")
    big_lse = torch.full((3 * pr.tokens, pr.nq), 7.0, device="cuda")
    r.out, r.lse = big[pr.tokens:2 * pr.tokens], big_lse[pr.tokens:2 * pr.tokens]
    for _ in range(3):
        r.q_start.copy_(torch.tensor([n * (b % 2) for b in range(batch + 1)], dtype=torch.int32))
        r.attend()
        assert r.kv.status() == RANGE
        r.q_start.copy_(good)
        r.out.fill_(float("nan")), r.lse.fill_(float("nan"))
        r.attend()
        r.check()
    for x in (big, big_lse):
        assert (x[:pr.tokens] == 7).all() and (x[2 * pr.tokens:] == 7).all()


def test_a_token_whose_page_is_lost_keeps_its_query_row():
    pr = Problem([3, 2], [20, 30], 4, 2, seed=89)
    r = Run(pr)
    q, k, v = dev(pr.q), dev(pr.k), dev(pr.v)
    r.table[0, 1] = pr.num_pages  # positions 16..31 of the first sequence: all three tokens
    before = r.k_pages.clone().nan_to_num(7.0), r.v_pages.clone().nan_to_num(7.0)
    r.kv.append(2, 5, q, k, v, r.q_start, r.kv_len, r.table, r.k_pages, r.v_pages, r.out)
    assert r.kv.status() == RANGE
    assert r.out[:3].isnan().all() and r.out[3:].isfinite().all()
    for got, old in zip((r.k_pages, r.v_pages), before):
        assert int((got.nan_to_num(7.0) != old).flatten(2).any(-1).sum()) == 2  # two slots, of the second


def test_angles_are_as_exact_as_stated():
    """cos and sin of every angle, read off rotated unit vectors in fp32, against
    angles in 60 digits.  The header's 2^-25 and 2^-23 of a turn, and 2^-24 for
    sincospif (2 ulp of 1 and the fp32 results' rounding: (2 + 1) 2^-24 / 2 pi)."""
    d, n = 128, 64
    g = torch.Generator().manual_seed(90)
    near = torch.cat([torch.arange(16), torch.randint(0, 2 ** 28, (n - 16,), generator=g)])
    far = torch.randint(-2 ** 31, 2 ** 31, (n,), generator=g)
    far[:3] = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1])
    kv = binding.PagedKv(n_q_heads=1, n_kv_heads=1, head_dim=d, page_size=16, num_pages=4,
                         max_pages=4, max_batch=1, max_tokens=n, dtype="f32", rope_theta=5e5)
    x = torch.zeros(n, 1, d, device="cuda")
    x[..., :d // 2] = 1.0  # a = 1, b = 0: the pair becomes (cos, sin)
    pools = torch.zeros(2, 4, 16, 1, d, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    st, table = torch.tensor([0, n], **i32), torch.arange(4, **i32).view(1, 4)
    getcontext().prec = 60
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    rate = [Decimal(500000) ** (Decimal(-2 * i) / d) / (2 * pi) for i in range(d // 2)]
    for pos, bound in ((near, 2.0 ** -25), (far, 2.0 ** -23)):
        out = torch.empty_like(x)
        kv.append(1, n, x, x, x, st, st[1:], table, pools[0], pools[1], out,
                  rope_pos=pos.to(**i32).view(1, n))
        assert kv.status() == OK
        c, s = out[:, 0, :d // 2].double().cpu(), out[:, 0, d // 2:].double().cpu()
        turns = torch.atan2(s, c) / (2 * math.pi)
        want = torch.tensor([[float(int(p) * r - (int(p) * r).to_integral_value()) for r in rate]
                             for p in pos], dtype=torch.float64)
        off = (turns - want + 0.5) % 1 - 0.5
        assert off.abs().max() <= bound + 2.0 ** -24, off.abs().max()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("starts,kv_len,tokens", [
    ([0, 4, -5, 4, 6], [9, 3, 20, 30], 6),      # one from -5 to 4: claims nothing
    ([0, 3, 1], [9, 30], 3),                     # decreases, and owns no token
    ([0, 3, 99, 3, 5], [9, 3, 8, 30], 5),
    ([20, 40, 0, 20], [30, 7, 45], 40),
], ids=str)
def test_append_reports_malformed_starts(dtype, starts, kv_len, tokens):
    pr = with_starts(starts, kv_len, tokens, (4, 2), dtype=dtype, seed=82)
    for _ in range(5):
        r, q = run_append(pr)
        check_append(pr, r, q, status=RANGE)
        owned = torch.zeros(tokens, dtype=torch.bool)
        for b, n in enumerate(pr.q_len):
            owned[starts[b]:starts[b] + n] = True
        assert q[~owned].isnan().all()


# ----------------------------------------------------- infinities and NaN --
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,q_len,kv_len,prefix", [
    ((4, 4), [1, 1, 1], [40, 300, 517], 0),
    ((8, 2), [1], [2000], 0),             # one sequence over many warps and blocks
    ((16, 1), [1, 1], [33, 120], 0),
    ((4, 2), [3, 2], [200, 90], 0),       # short drafts: early tiles that all rows see
    ((4, 2), [1, 1], [20, 9], 150),       # a prefix, few rows in all
    ((8, 2), [1] * 20, [5] * 20, 150),    # a prefix, many
    ((4, 2), [150], [400], 0), ((4, 2), [100, 40], [130, 60], 200)], ids=str)
def test_infinities_that_every_row_sees(dtype, d, heads, q_len, kv_len, prefix):
    """Values of +-infinity, with probabilities above 2^-24 of the largest, stay
    infinities of their sign (NaN where both meet); other columns stay exact."""
    pr = Problem(q_len, kv_len, *heads, d=d, dtype=dtype, prefix=prefix, seed=80, q_scale=0.5)
    vp = pr.split(pr.pools)[1]
    at = [(pr.table[b], j) for b in range(pr.batch) for j in (0, kv_len[b] // 2)]
    at += [(pr.prefix_table, j) for j in (3, prefix - 2) if prefix]
    for n, (row, j) in enumerate(at):
        v = pr.slot(vp, row, j)
        v[:, n % 2::7] = (math.inf, -math.inf)[n % 2]
        v[:, 5::14] = -(math.inf, -math.inf)[n % 2]
        v[:, 12] = math.nan
    want = ref_attention(pr)
    r = Run(pr)
    r.attend()
    assert r.kv.status() == OK
    got, finite = r.out.double().cpu(), want[0].isfinite()
    assert want[0].isinf().any() and want[0].isnan().any()
    assert torch.equal(got.isnan(), want[0].isnan())
    assert (got[want[0].isinf()] == want[0][want[0].isinf()]).all()
    close(torch.where(finite, got, 0.0), torch.where(finite, want[0], 0.0),
          torch.where(finite, want[1], 0.0), "finite values")
    close(r.lse, want[2], want[3], "lse")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_len,kv_len,prefix,window", [
    ([1, 1, 1], [1, 200, 900], 0, 0), ([3, 2], [3, 90], 0, 0), ([3, 2], [3, 90], 0, 1),
    ([150, 1], [300, 1], 0, 0), ([150, 1], [300, 1], 0, 1), ([1, 2], [1, 40], 70, 0),
    ([60, 1], [90, 1], 70, 0)], ids=str)
def test_rows_of_nan_say_so_in_lse(dtype, q_len, kv_len, prefix, window):
    """-infinity stands for rows without a key; a NaN in a query, or in every
    key that a row sees, is NaN in o and in lse."""
    pr = Problem(q_len, kv_len, 4, 2, dtype=dtype, prefix=prefix, seed=83)
    kp = pr.split(pr.pools)[0]
    pr.q[0, 1, 5] = math.nan            # one head of the first token
    pr.q[-1, :, 0] = math.nan           # every head of the last one
    for j in range(kv_len[0] - q_len[0], kv_len[0]):  # with a window of 1: all that a row sees
        pr.slot(kp, pr.table[0], j)[0] = math.nan
    want = ref_attention(pr, window)
    r = Run(pr)
    r.attend(window)
    assert r.kv.status() == OK
    assert want[2].isnan().any() and want[2].isfinite().any()
    assert torch.equal(r.out.isnan().cpu(), want[0].isnan())
    close(r.lse, want[2], want[3], "lse")
    finite = want[0].isfinite()
    close(torch.where(finite, r.out.double().cpu(), 0.0), torch.where(finite, want[0], 0.0),
          torch.where(finite, want[1], 0.0), "finite values")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_len,prefix", [([1], 0), ([2], 0), ([40], 0), ([1], 20000), ([40], 20000)],
                         ids=str)
def test_flat_tails_far_below_the_largest_weight_count(dtype, q_len, prefix):
    """One key of weight 1 and a value of 0, 20000 of 2^-26 and values of 1: the
    product has the tail as the sum has it.  Scores of 0 and 2 ln 2^13 = 18.02
    are off by (64 + 2) 2^-23 18.02 at most, their weights relatively by twice
    that; the weights' rounding and the result's are half a step each, and a
    fp16 result below 2^-14 is off by 2^-25."""
    n, d, own = q_len[0], 64, 20000 - prefix
    own = own or 64
    pr = Problem(q_len, [own], 8, 2, d=d, page=64, dtype=dtype, prefix=prefix, seed=91)
    kp, vp = pr.split(pr.pools)
    kp.zero_(), vp.fill_(1.0)
    pr.q.zero_()
    pr.q[..., 0] = 16.0
    top = torch.tensor(26 * math.log(2) * 8 / 16).to(pr.q.dtype)  # times 16 / sqrt(64)
    row = pr.prefix_table if prefix else pr.table[0]
    pr.slot(kp, row, 7)[:, 0] = top
    pr.slot(vp, row, 7)[...] = 0.0
    r = Run(pr, poison=False)
    r.attend()
    assert r.kv.status() == OK
    w = math.exp(-2 * float(top))
    seen = torch.arange(own - n, own, dtype=torch.float64) + prefix  # keys but for the one
    want = (seen * w / (1 + seen * w))[:, None, None].expand(r.out.shape)
    u, ds = half_step(dtype), 66 * 2.0 ** -23 * 2 * float(top)
    tol = want * (2 * u + 2 * ds + (20064 + 8) * 2.0 ** -23) + 2.0 ** -25
    close(r.out, want, tol, "out")


# ---------------------------------------------------------------- overlaps --
def test_in_place_append_refuses_keys_that_share_the_queries_elements():
    """q_out == q lets k and v lie between the rows of q, not on them."""
    pr = Problem([2, 3], [9, 30], 4, 2, seed=84)
    r = Run(pr)
    L, s = binding.lib(), torch.cuda.current_stream().cuda_stream
    row = (4 + 2 * 2) * 128
    x = torch.zeros(8 * row, dtype=torch.bfloat16, device="cuda")
    at = x.data_ptr()

    def append(n, k, v, ks=row, qs=row, q=at + 2 * row):
        return L.cf_paged_append(r.kv.handle, 2 if n > 1 else 1, n, q, k, v, qs, ks,
                                 r.q_start.data_ptr() if n > 1 else None, r.kv_len.data_ptr(), None,
                                 r.table.data_ptr(), r.k_pages.data_ptr(), r.v_pages.data_ptr(), q,
                                 qs, s)

    q, w = at + 2 * row, 2 * 512  # w: bytes of a row's queries
    other = torch.zeros(8 * row, dtype=torch.bfloat16, device="cuda")
    free = other.data_ptr()
    for n in (5, 1):
        assert append(n, q + w, q + w + 512) == OK               # the merged projection
        assert append(n, q + w + 512, q + w) == OK
        assert append(n, free, free + 512) == OK
        for bad in (q, q + 16, q + w - 16, q + 512, q - 512 + 16):
            assert append(n, bad, q + w) == binding.CF_ERR_ALIAS, bad - q
            assert append(n, q + w, bad) == binding.CF_ERR_ALIAS, bad - q
    assert append(5, q - 512, q + w) == OK                       # the row before, behind its queries
    assert append(5, q + 2 * row, q + w) == binding.CF_ERR_ALIAS     # the next row's queries
    assert append(5, q + 8 * row, q + w) == binding.CF_ERR_ALIAS     # the last row's
    assert append(1, q + 2 * row, q + w) == OK                   # there is no next row
    assert append(5, free, free + 512, ks=256) == OK
    assert append(5, q + w, free, ks=256) == binding.CF_ERR_ALIAS    # rows of another stride among q's
    assert r.kv.status() == OK


@pytest.mark.parametrize("layout", [0, 1])
def test_pools_that_share_pages_are_refused(layout):
    """With a page stride of two pages keys and values may alternate; they may
    not share a page."""
    pr = Problem([2, 3], [9, 30], 4, 2, seed=85, interleaved=True, layout=layout)
    r = Run(pr)
    L, s = binding.lib(), torch.cuda.current_stream().cuda_stream
    x = [t.cuda() for t in (pr.q, pr.k, pr.v)]
    page = 2 * pr.page * pr.nkv * pr.d  # bytes

    def append(k, v):
        return L.cf_paged_append(r.kv.handle, 2, 5, x[0].data_ptr(), x[1].data_ptr(),
                                 x[2].data_ptr(), 512, 256, r.q_start.data_ptr(),
                                 r.kv_len.data_ptr(), None, r.table.data_ptr(), k, v,
                                 r.out.data_ptr(), 512, s)

    k = r.k_pages.data_ptr()
    assert append(k, k + page) == OK and append(k + page, k) == OK
    for off in (0, 16, page // 2, page - 16, page + 16, 2 * page, 3 * page + 16):
        assert append(k, k + off) == binding.CF_ERR_ALIAS, off
        assert append(k + off, k) == binding.CF_ERR_ALIAS, off
    assert r.kv.status() == OK


# ------------------------------------------------------- handles and shapes --
def test_a_new_handle_serves_every_stream():
    """Its workspace is ready when create returns, also for streams that do not
    wait for the default one, and however much that still has to do."""
    a = torch.randn(8192, 8192, device="cuda")
    side = torch.cuda.Stream()
    pr = Problem([1], [900], 4, 2, seed=86)
    r = Run(pr)
    want = ref_attention(pr)
    torch.cuda.synchronize()
    done = torch.cuda.Event()
    with torch.cuda.stream(torch.cuda.default_stream()):
        for _ in range(20):
            a @ a
        done.record()
    r.kv = binding.PagedKv(**pr.config())
    assert done.query()
    r.attend(stream=side)
    side.synchronize()
    r.check()


def test_strides_whose_span_overflows_are_refused():
    """Rows so far apart that the tensor's bytes pass 63 bits: nothing runs."""
    n = 1 << 20
    kv = binding.PagedKv(n_q_heads=1, n_kv_heads=1, head_dim=64, page_size=16, num_pages=1,
                         max_pages=1, max_batch=1, max_tokens=n, dtype="bf16")
    x = torch.zeros(64 * 64, dtype=torch.bfloat16, device="cuda")
    i32 = torch.zeros(64, dtype=torch.int32, device="cuda")
    L, s = binding.lib(), torch.cuda.current_stream().cuda_stream
    a = [x[i:].data_ptr() for i in range(0, 1024, 64)]
    far = 1 << 40
    assert L.cf_paged_attention(kv.handle, 1, n, 1, a[0], far, i32.data_ptr(), i32.data_ptr(),
                                i32.data_ptr(), a[1], a[2], 0, 0, a[3], None, s) == \
        binding.CF_ERR_INVALID_ARG
    for strides in ((far, 64, 64), (64, far, 64), (64, 64, far)):
        q, kv_, out = strides
        assert L.cf_paged_append(kv.handle, 1, n, a[0], a[1], a[2], q, kv_, i32.data_ptr(),
                                 i32.data_ptr(), None, i32.data_ptr(), a[3], a[4], a[5], out, s) == \
            binding.CF_ERR_INVALID_ARG
    assert kv.status() == OK and (x == 0).all()


def test_tables_of_another_width_are_refused():
    """[batch, max_pages] and [axes, n_tokens] arrays are read by those widths:
    a tensor of two axes has to have them."""
    pr = Problem([2, 3], [9, 30], 4, 2, max_pages=4, seed=87)
    r = Run(pr, rope_sections=(16, 24, 24))
    rest = (r.k_pages, r.v_pages)
    wide = torch.zeros(2, pr.max_pages + 1, dtype=torch.int32, device="cuda")
    q, k, v = dev(pr.q), dev(pr.k), dev(pr.v)
    i32 = dict(dtype=torch.int32, device="cuda")
    for table in (wide, wide.T.contiguous()):
        with pytest.raises(binding.CfError) as e:
            r.kv.attention(2, 5, 3, q, r.q_start, r.kv_len, table, *rest, r.out)
        assert e.value.code == binding.CF_ERR_INVALID_ARG
        with pytest.raises(binding.CfError):
            r.kv.prefix_attention(2, 5, 3, q, r.q_start, r.kv_len, table, r.ptable, 0, *rest, r.out)
        with pytest.raises(binding.CfError):
            r.kv.append(2, 5, q, k, v, r.q_start, r.kv_len, table, *rest, r.out)
    for shape in ((3, 6), (5, 3), (4, 6)):
        with pytest.raises(binding.CfError):
            r.kv.append(2, 5, q, k, v, r.q_start, r.kv_len, r.table, *rest, r.out,
                        rope_pos=torch.zeros(*shape, **i32))
    assert r.out.isnan().all()
    # rows beyond the call's, and arrays of one axis, are fine
    more = torch.cat([r.table, r.table])
    for table in (r.table, more, r.table.flatten()):
        for pos in (torch.zeros(3, 5, **i32), torch.zeros(15, **i32), None):
            r.kv.append(2, 5, q, k, v, r.q_start, r.kv_len, table, *rest, r.out, rope_pos=pos)
        r.kv.attention(2, 5, 3, q, r.q_start, r.kv_len, table, *rest, r.out)
    assert r.kv.status() == OK
