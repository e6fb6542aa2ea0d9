"""Work cases of a decode step in 8 and 4 bits: appending to a paged KV cache whose keys and values are held as 8-bit
codes with a scale per position and head, attention over that cache, reading it back, and products of a few rows with
weights of 4 bits and group scales.

A case fixes every size; its values come from the seed.  Sequence b has q_len[b] new tokens behind ctx[b] older ones;
both are derived from the case alone, so that every seed gives the same shapes."""
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FORMATS = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}  # type of a code, largest magnitude
TINY = 2.0 ** -100  # heads whose largest magnitude is below are held as zeros


def _kv(op, name, dtype, fmt, heads, page, batch, ctx, q, theta=1e4, window=0, sinks=0):
    nq, nkv, d = heads
    return {"name": name, "op": op, "dtype": dtype, "fmt": fmt, "nq": nq, "nkv": nkv, "d": d, "page": page,
            "batch": batch, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "q_lo": q[0], "q_hi": q[1], "theta": theta,
            "window": window, "sinks": sinks}


def _mv(name, dtype, k, n, group, rows, zeros=False, residual=False):
    return {"name": name, "op": "matvec", "dtype": dtype, "k": k, "n": n, "group": group, "rows": rows,
            "zeros": zeros, "residual": residual}


MHA128 = (32, 32, 128)   # 32 heads of 128, hidden 4096
MHA64 = (32, 32, 64)     # 32 heads of 64, hidden 2048
GQA128 = (32, 8, 128)    # 32 query heads on 8 KV heads of 128


def listed():
    return [
        # one new token of one sequence: the per-step latency of a chat with one user
        _kv("append", "append8_1_token", "bf16", "e4m3", GQA128, 16, 1, (4096, 4096), (1, 1), 5e5),
        # prompts of a batch entering the cache together, odd lengths, behind older turns
        _kv("append", "append8_prompts", "bf16", "e4m3", GQA128, 16, 8, (0, 4097), (333, 2048), 5e5),
        # sequences that move on to a cache in 16 bits: the step's tokens appended, everything read back
        _kv("read", "read8_sequences", "f16", "int8", MHA64, 64, 16, (1024, 2048), (1, 5)),
        # one sequence handed to a dense cache after a prompt's last chunk
        _kv("read", "read8_one_sequence", "bf16", "e4m3", GQA128, 16, 1, (3585, 3585), (511, 511), 5e5),
        # one user, 1024 tokens of context: latency
        _kv("attention", "attn8_decode_b1", "f16", "int8", MHA128, 16, 1, (1024, 1024), (1, 1)),
        # a full decode batch with grouped heads
        _kv("attention", "attn8_decode_gqa_b16", "bf16", "e4m3", GQA128, 16, 16, (4096, 4096), (1, 1)),
        # ragged long contexts: what a cache of 8 bits is for
        _kv("attention", "attn8_decode_long", "bf16", "int8", GQA128, 32, 32, (2048, 32768), (1, 1)),
        # four draft tokens of each sequence of a batch
        _kv("attention", "attn8_drafts", "f16", "e4m3", GQA128, 16, 32, (1001, 4096), (4, 4)),
        # a chunk of a long prompt behind what is in the cache already
        _kv("attention", "attn8_chunk", "bf16", "e4m3", GQA128, 16, 1, (15872, 15872), (512, 512)),
        # chunks of several prompts in one call, odd lengths
        _kv("attention", "attn8_chunks", "f16", "int8", MHA128, 64, 4, (0, 2049), (257, 1024)),
        # one token through a merged projection of queries, keys and values
        _mv("w4_qkv_1_row", "f16", 4096, 12288, 128, 1),
        # a decode batch through a down projection, with zero points and the residual
        _mv("w4_down_16_rows", "bf16", 11008, 4096, 64, 16, zeros=True, residual=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(("append", "read", "attention", "attention", "attention", "matvec", "matvec"))
    if op == "matvec":
        group = rng.choice((32, 64, 128))
        k = group * log(max(1, 256 // group), 14336 // group)
        n = 2 * log(64, 14336)
        c = _mv("", rng.choice(("f16", "bf16", "bf16", "f32")), k, n, group, rng.choice((1, 1, 2, 3, 4, 8, 13, 16, 32, 64)),
                rng.random() < 0.5, rng.random() < 0.5)
    else:
        dtype, fmt = rng.choice(("bf16", "f16")), rng.choice(("int8", "e4m3"))
        d = rng.choice((64, 128))
        nkv = rng.choice((1, 2, 4, 8))
        nq = nkv * rng.choice((1, 2, 3, 4, 7, 8))
        page = rng.choice((16, 32, 64, 128))
        theta = rng.choice((1e4, 5e5, 1e6))
        window, sinks = 0, 0
        batch = log(1, 64)
        if op == "attention":
            q_hi = 1 if rng.random() < 0.5 else log(2, max(2, 2048 // batch))
            ctx_hi = log(16, max(16, min(32768, 400000 // batch)))
            if q_hi > 64:
                ctx_hi = min(ctx_hi, 4096)
            if rng.random() < 0.3:
                window, sinks = log(16, 4096), rng.choice((0, 4, 16))
        else:
            if op == "append":  # codes are compared as values of a float type
                fmt = "e4m3"
            ctx_hi = log(1, max(1, min(16384, 65536 // batch)))
            q_hi = log(1, max(1, 8192 // batch))
        c = _kv(op, "", dtype, fmt, (nq, nkv, d), page, batch, (rng.randint(0, ctx_hi), ctx_hi),
                (rng.randint(1, q_hi), q_hi), theta, window, sinks)
    del c["name"]
    return c


def _lens(c):
    """q_len and ctx of every sequence."""
    r = random.Random(c["batch"] * 7919 + c["ctx_hi"] * 31 + c["q_hi"])
    return ([r.randint(c["q_lo"], c["q_hi"]) for _ in range(c["batch"])],
            [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["batch"])])


def _quantise(x, fmt):
    """Codes of x [.., d] and a scale per head: the largest magnitude gets the format's largest code."""
    dt, top = FORMATS[fmt]
    amax = x.abs().amax(-1, keepdim=True)
    zero = amax < TINY
    y = x * torch.where(zero, 0.0, top / torch.where(zero, 1.0, amax))
    codes = y.round().to(dt) if fmt == "int8" else y.to(dt)
    return codes, torch.where(zero, 0.0, amax / top).squeeze(-1)


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    dt = DTYPES[c["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    if c["op"] == "matvec":
        return _prepare_matvec(c, dt, g, dev)
    q_len, ctx = _lens(c)
    kv = [a + b for a, b in zip(q_len, ctx)]
    T, B, page, nq, nkv, d = sum(q_len), c["batch"], c["page"], c["nq"], c["nkv"], c["d"]
    per_seq = -(-max(kv) // page)
    used = [-(-x // page) for x in kv]
    n_pages = sum(used) + 3
    order = torch.randperm(n_pages, generator=g, device=dev).int()  # pages are handed out in no order
    first = torch.tensor([sum(used[:b]) for b in range(B)], device=dev)
    cols = torch.arange(per_seq, device=dev)
    table = torch.where(cols[None] < torch.tensor(used, device=dev)[:, None],
                        order[(first[:, None] + cols[None]).clamp(max=n_pages - 1)], order[-1:])
    s = {"case": c, "batch": B, "tokens": T, "max_q": max(q_len),
         "q_start": torch.tensor([sum(q_len[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev),
         "kv_len": torch.tensor(kv, dtype=torch.int32, device=dev), "page_table": table.int().contiguous(),
         "scales": torch.empty(n_pages, nkv, page, 2, device=dev)}
    # what the cache holds: channels of keys differ in size, as behind a projection; values by position
    for i, pool in enumerate(("k_pages", "v_pages")):
        s[pool] = torch.empty(n_pages, page, nkv, d, dtype=FORMATS[c["fmt"]][0], device=dev)
        wide = 0.3 + 1.4 * torch.rand(nkv, d, generator=g, device=dev)
        step = max(1, (1 << 26) // (page * nkv * d))
        for lo in range(0, n_pages, step):
            x = torch.randn(min(step, n_pages - lo), page, nkv, d, generator=g, device=dev)
            x *= wide if i == 0 else 0.3 + 1.4 * torch.rand(x.shape[:3], generator=g, device=dev)[..., None]
            codes, scale = _quantise(x, c["fmt"])
            s[pool][lo:lo + step] = codes
            s["scales"][lo:lo + step, ..., i] = scale.transpose(1, 2)
    if c["op"] == "attention":
        # scores with a standard deviation of about two: attention that picks some keys out
        s["q"] = (2 * torch.randn(T, nq, d, generator=g, device=dev)).to(dt)
        s["out"] = torch.empty(T, nq, d, dtype=dt, device=dev)
    else:
        # the merged projection's output; a projected channel has its own scale
        x = torch.randn(T, (nq + 2 * nkv) * d, generator=g, device=dev)
        x *= 0.5 + torch.rand((nq + 2 * nkv) * d, generator=g, device=dev)
        s["qkv"] = x.to(dt)
        s["q"] = s["qkv"][:, :nq * d].view(T, nq, d)
        s["k"] = s["qkv"][:, nq * d:(nq + nkv) * d].view(T, nkv, d)
        s["v"] = s["qkv"][:, (nq + nkv) * d:].view(T, nkv, d)
        s["q_out"] = torch.empty(T, nq, d, dtype=dt, device=dev)
    if c["op"] == "read":
        rows = sum(kv)
        s["rows"] = rows
        s["row_start"] = torch.tensor([sum(kv[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
        s["k_out"] = torch.empty(rows, nkv, d, dtype=dt, device=dev)
        s["v_out"] = torch.empty(rows, nkv, d, dtype=dt, device=dev)
    if own:
        from attention_block_gb300 import binding
        s["kv"] = binding.Paged8Kv(n_q_heads=nq, n_kv_heads=nkv, head_dim=d, page_size=page, num_pages=n_pages,
                                   max_batch=B, max_tokens=T, max_pages=per_seq, rope_theta=c["theta"],
                                   dtype=c["dtype"], code=c["fmt"])
    return s


def _prepare_matvec(c, dt, g, dev):
    k, n, groups = c["k"], c["n"], c["k"] // c["group"]
    s = {"case": c, "rows": c["rows"],
         # two columns' codes in a byte, the even one's in the low half
         "codes": torch.randint(0, 256, (k, n // 2), generator=g, device=dev, dtype=torch.uint8),
         "scales": (0.02 / 4 * (0.5 + torch.rand(groups, n, generator=g, device=dev))).to(dt),
         "zeros": torch.randint(4, 12, (groups, n), generator=g, device=dev, dtype=torch.uint8) if c["zeros"] else None,
         "x": torch.randn(c["rows"], k, generator=g, device=dev).to(dt),
         "residual": torch.randn(c["rows"], n, generator=g, device=dev).to(dt) if c["residual"] else None,
         "out": torch.empty(c["rows"], n, dtype=dt, device=dev)}
    if own:
        from attention_block_gb300 import binding
        s["w4"] = binding.W4Matvec(in_features=k, out_features=n, group=c["group"], zeros=c["zeros"],
                                   max_rows=c["rows"], dtype=c["dtype"])
        s["packed"] = s["w4"].pack(s["codes"], s["scales"], s["zeros"])
    return s


# ------------------------------------------------------------ plain forms --
def _token_grid(s):
    """Row of each (sequence, i) in the token arrays, which of them exist, and their positions: [B, N]."""
    i = torch.arange(s["max_q"], device=s["kv_len"].device)
    a, b = s["q_start"][:-1, None].long(), s["q_start"][1:, None].long()
    tok = a + i
    return tok.clamp(max=s["tokens"] - 1), tok < b, s["kv_len"][:, None].long() - (b - a) + i


def _plain_rope(x, pos, c):
    """x [T, heads, d] at positions pos [T], rotate-half, in 32 bits."""
    half = c["d"] // 2
    i = torch.arange(half, device=x.device, dtype=torch.float64)
    freq = torch.pow(torch.tensor(c["theta"], dtype=torch.float64, device=x.device), -2.0 * i / c["d"])
    ang = pos.double()[:, None] * freq  # far positions lose their angle in 32 bits
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(s):
    c = s["case"]
    tok, there, pos = _token_grid(s)
    seq = torch.arange(s["batch"], device=tok.device)[:, None].expand_as(tok)[there]
    p = pos[there]  # tokens lie in the order of their sequences
    page, slot = s["page_table"][seq, p // c["page"]].long(), p % c["page"]
    k, ks = _quantise(_plain_rope(s["k"], p, c), c["fmt"])
    v, vs = _quantise(s["v"].float(), c["fmt"])
    s["k_pages"].view(torch.uint8)[page, slot] = k.view(torch.uint8)
    s["v_pages"].view(torch.uint8)[page, slot] = v.view(torch.uint8)
    s["scales"][page, :, slot] = torch.stack([ks, vs], -1)
    return _plain_rope(s["q"], p, c).to(s["q"].dtype)


def _values(s, pages, pool):
    """Values in 32 bits of the pages [..]: [.., page, nkv, d]."""
    i = ("k_pages", "v_pages").index(pool)
    return s[pool].view(torch.uint8)[pages].view(s[pool].dtype).float() * \
        s["scales"][pages][..., i].transpose(-1, -2)[..., None]


def _plain_read(s):
    q = _plain_append(s)
    row = torch.arange(s["rows"], device=q.device)
    seq = torch.searchsorted(s["row_start"][1:].long(), row, right=True)
    j, page = row - s["row_start"][seq].long(), s["case"]["page"]
    pages = s["page_table"][seq, j // page].long()
    out = {"q": q}
    out["k"], out["v"] = (
        (s[pool].view(torch.uint8)[pages, j % page].view(s[pool].dtype).float() *
         s["scales"][pages, :, j % page, i][..., None]).to(q.dtype) for i, pool in enumerate(("k_pages", "v_pages")))
    return out


def _plain_attention(s):
    c = s["case"]
    tok, there, pos = _token_grid(s)
    B, N = tok.shape
    G = c["nq"] // c["nkv"]
    K = _values(s, s["page_table"].long(), "k_pages").flatten(1, 2).transpose(1, 2)
    j = torch.arange(K.shape[2], device=K.device)
    p = pos[:, :, None]
    see = (j <= p) & (j < s["kv_len"][:, None, None])
    if c["window"]:
        see &= (p - j < c["window"]) | (j < c["sinks"])
    rows = s["q"][tok].float().view(B, N, c["nkv"], G, c["d"]).transpose(1, 2).reshape(B, c["nkv"], -1, c["d"])
    sc = rows @ K.transpose(2, 3)
    del K
    sc *= c["d"] ** -0.5
    sc.view(B, c["nkv"], N, G, -1).masked_fill_(~see[:, None, :, None], float("-inf"))
    sc.sub_(sc.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    total = sc.sum(-1, keepdim=True)
    V = _values(s, s["page_table"].long(), "v_pages").flatten(1, 2).transpose(1, 2)
    o = (sc @ V) / total
    o = o.view(B, c["nkv"], N, G, c["d"]).transpose(1, 2).reshape(B, N, c["nq"], c["d"])
    out = torch.zeros(s["tokens"], c["nq"], c["d"], dtype=s["q"].dtype, device=o.device)
    out[tok[there]] = o[there].to(out.dtype)
    return {"out": out}


def _plain_matvec(s):
    c = s["case"]
    k, n, group = c["k"], c["n"], c["group"]
    w = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).view(k // group, group, n).float()
    w -= s["zeros"][:, None].float() if c["zeros"] else 8.0
    w *= s["scales"][:, None].float()
    y = s["x"].float() @ w.view(k, n)
    if c["residual"]:
        y += s["residual"].float()
    return {"out": y.to(s["x"].dtype)}


def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if not own:
        if op == "append":
            return {"q": _plain_append(s), "k_pages": s["k_pages"], "v_pages": s["v_pages"], "scales": s["scales"]}
        return {"read": _plain_read, "attention": _plain_attention, "matvec": _plain_matvec}[op](s)
    if op == "matvec":
        s["w4"](s["rows"], s["x"], s["packed"], s["out"], residual=s["residual"])
        return {"out": s["out"]}
    kv = s["kv"]
    starts = s["q_start"] if s["max_q"] > 1 else None  # one token per sequence needs no starts
    if op == "attention":
        kv.attention(s["batch"], s["tokens"], s["max_q"], s["q"], starts, s["kv_len"], s["page_table"], s["k_pages"],
                     s["v_pages"], s["scales"], s["out"], window=c["window"], n_sinks=c["sinks"])
        return {"out": s["out"]}
    kv.append(s["batch"], s["tokens"], s["q"], s["k"], s["v"], starts, s["kv_len"], s["page_table"], s["k_pages"],
              s["v_pages"], s["scales"], s["q_out"])
    if op == "append":
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"], "scales": s["scales"]}
    kv.read(s["batch"], s["rows"], s["row_start"], None, s["page_table"], s["k_pages"], s["v_pages"], s["scales"],
            s["k_out"], s["v_out"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


# ----------------------------------------------------------------- the work --
def _visible(p, window, sinks):
    """Number of keys that position p sees."""
    if not window or p < window:
        return p + 1
    return window + min(sinks, p + 1 - window)


def work(case):
    c = case
    es = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "matvec":
        groups = c["k"] // c["group"]
        return {"bytes": c["k"] * c["n"] // 2 + groups * c["n"] * (es + (1 if c["zeros"] else 0)) +
                c["rows"] * (c["k"] + c["n"] * (2 if c["residual"] else 1)) * es, "flops": 2 * c["rows"] * c["k"] * c["n"]}
    q_len, ctx = _lens(c)
    T = sum(q_len)
    held = c["nkv"] * (2 * c["d"] + 8)  # bytes of a position in the cache: codes and two scales
    if c["op"] != "attention":
        new = T * (c["nq"] + 2 * c["nkv"]) * c["d"] * es + T * c["nq"] * c["d"] * es + T * held + 4 * (2 * c["batch"] + 1)
        # sequences whole: the new tokens' codes are still to be written, and read
        back = (T + sum(ctx)) * (held + 2 * c["nkv"] * c["d"] * es) if c["op"] == "read" else 0
        return {"bytes": new + back, "flops": 5 * T * (c["nq"] + c["nkv"]) * c["d"]}
    pairs = keys = 0
    for n, a in zip(q_len, ctx):
        pairs += sum(_visible(p, c["window"], c["sinks"]) for p in range(a, a + n))
        lo = max(0, a - c["window"] + 1) if c["window"] else 0  # the first token's window starts here
        keys += a + n - lo + min(c["sinks"] if c["window"] else 0, lo)
    return {"bytes": keys * held + 4 * (-(-keys // c["page"])) + 2 * T * c["nq"] * c["d"] * es,
            "flops": 4 * pairs * c["nq"] * c["d"]}


# ------------------------------------------------------------ in 64 bits --
def _code64(x, fmt):
    """Codes, as values, and scales of heads x [.., d] in 64 bits."""
    top = FORMATS[fmt][1]
    peak = x.abs().max(-1, keepdim=True).values
    y = torch.where(peak < TINY, torch.zeros_like(x), x / peak.clamp(min=TINY) * top)
    if fmt == "int8":
        y = torch.round(y)
    else:  # three bits behind the leading one, steps of 2^-9 below 2^-6
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        y = torch.round(y / step) * step
    return y, torch.where(peak < TINY, torch.zeros_like(peak), peak / top)[..., 0]


def exact(case, seed):
    s = prepare(case, seed)
    c, f64 = case, torch.float64
    if c["op"] == "matvec":
        k, n = c["k"], c["n"]
        out = torch.zeros(c["rows"], n, dtype=f64, device=s["x"].device)
        if c["residual"]:
            out += s["residual"].to(f64)
        for i in range(k // c["group"]):
            part = slice(i * c["group"], (i + 1) * c["group"])
            w = torch.empty(c["group"], n, dtype=f64, device=out.device)
            w[:, 0::2] = (s["codes"][part] % 16).to(f64)
            w[:, 1::2] = (s["codes"][part] // 16).to(f64)
            w -= s["zeros"][i].to(f64) if c["zeros"] else 8
            out += (s["x"][:, part].to(f64) @ w) * s["scales"][i].to(f64)
        return {"out": out}
    nq, nkv, d, page = c["nq"], c["nkv"], c["d"], c["page"]
    q_len, ctx = _lens(c)
    dev = s["q"].device

    def held(b, lo, hi, i):
        """Values of positions lo .. hi - 1 of sequence b."""
        j = torch.arange(lo, hi, device=dev)
        ids = s["page_table"][b][j // page].long()
        return s[("k_pages", "v_pages")[i]].float()[ids, j % page].to(f64) * s["scales"][ids, :, j % page, i].to(f64)[..., None]

    if c["op"] != "attention":
        rate = torch.tensor([float(c["theta"]) ** (-2.0 * i / d) for i in range(d // 2)], dtype=f64, device=dev)
        pools, scales = [s["k_pages"].to(f64), s["v_pages"].to(f64)], s["scales"].to(f64)
        qs, ks, vs, at = [], [], [], 0
        for b in range(c["batch"]):
            n = q_len[b]
            p = torch.arange(ctx[b], ctx[b] + n, device=dev)
            ang = p.to(f64)[:, None] * rate
            z = torch.polar(torch.ones_like(ang), ang)[:, None]

            def turn(x):
                y = torch.complex(x[..., :d // 2].to(f64), x[..., d // 2:].to(f64)) * z
                return torch.cat([y.real, y.imag], -1)

            ids = s["page_table"][b][p // page].long()
            new = [_code64(turn(s["k"][at:at + n]), c["fmt"]), _code64(s["v"][at:at + n].to(f64), c["fmt"])]
            for i in range(2):
                pools[i][ids, p % page] = new[i][0]
                scales[ids, :, p % page, i] = new[i][1]
            qs.append(turn(s["q"][at:at + n]))
            for i, kept in enumerate((ks, vs)):
                kept += [held(b, 0, ctx[b], i), new[i][0] * new[i][1][..., None]]
            at += n
        if c["op"] == "append":
            return {"q": torch.cat(qs), "k_pages": pools[0], "v_pages": pools[1], "scales": scales}
        return {"q": torch.cat(qs), "k": torch.cat(ks), "v": torch.cat(vs)}
    if work(case)["flops"] > 4e12:
        return None
    out = torch.zeros(sum(q_len), nq, d, dtype=f64, device=dev)
    at = 0
    for b in range(c["batch"]):
        n, a = q_len[b], ctx[b]
        K, V = held(b, 0, a + n, 0), held(b, 0, a + n, 1)
        own_j = torch.arange(a + n, device=dev)
        for lo in range(0, n, 512):
            hi = min(n, lo + 512)
            p = torch.arange(a + lo, a + hi, device=dev)[:, None]
            hide = own_j > p
            if c["window"]:
                hide |= (own_j <= p - c["window"]) & (own_j >= c["sinks"])
            for h in range(nkv):
                heads = slice(h * (nq // nkv), (h + 1) * (nq // nkv))
                x = torch.einsum("nhd,sd->hns", s["q"][at + lo:at + hi, heads].to(f64), K[:, h]) / d ** 0.5
                w = torch.softmax(x.masked_fill(hide, float("-inf")), -1)
                out[at + lo:at + hi, heads] = torch.einsum("hns,sd->nhd", w, V[:, h])
        at += n
    return {"out": out}
