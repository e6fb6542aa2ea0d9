"""Work cases of the paged KV cache's operators: appending with rotary positions (one or three axes), attention with a
sliding window and sinks, attention of a batch that shares a prefix.

A case fixes every size; its values come from the seed.  Sequence b has q_len[b] new tokens behind ctx[b] older ones;
both are derived from the case alone, so that every seed gives the same shapes."""
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _case(op, name, dtype, heads, page, batch, ctx, q, theta=1e4, axes="", window=0, sinks=0, prefix=0):
    nq, nkv, d = heads
    return {"name": name, "op": op, "dtype": dtype, "nq": nq, "nkv": nkv, "d": d, "page": page, "batch": batch,
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "q_lo": q[0], "q_hi": q[1], "theta": theta, "axes": axes,
            "window": window, "sinks": sinks, "prefix": prefix}


MHA128 = (32, 32, 128)   # 32 heads of 128, hidden 4096
MHA64 = (32, 32, 64)     # 32 heads of 64, hidden 2048
GQA128 = (32, 8, 128)    # 32 query heads on 8 KV heads of 128


def listed():
    return [
        # one new token of one sequence: the per-step latency of a chat with one user
        _case("append", "append_1_token", "bf16", GQA128, 16, 1, (4096, 4096), (1, 1), 5e5),
        # the decode step of a full batch, ragged lengths
        _case("append", "append_decode_b64", "f16", MHA64, 64, 64, (1024, 2048), (1, 1)),
        # prompts of a batch entering the cache together, odd lengths, behind older turns
        _case("append", "append_prompts", "bf16", GQA128, 16, 8, (0, 4097), (333, 2048), 5e5),
        # a picture of several thousand patches: positions by time, height and width
        _case("append", "append_axes_picture", "bf16", GQA128, 32, 2, (17, 1031), (4097, 4097), 1e6, "16,24,24"),
        # video frames of a batch, head size 64, the axes interleaved over the frequencies
        _case("append", "append_axes_video", "f16", MHA64, 64, 6, (0, 257), (1200, 3601), 1e4, "12,10,10,i"),
        # one user, 1024 tokens of context: latency
        _case("attention", "attn_decode_b1", "f16", MHA128, 16, 1, (1024, 1024), (1, 1)),
        # a full decode batch with grouped heads
        _case("attention", "attn_decode_gqa_b16", "bf16", GQA128, 16, 16, (4096, 4096), (1, 1)),
        # ragged long contexts behind a window with four sinks
        _case("attention", "attn_decode_window", "bf16", GQA128, 32, 48, (5000, 32768), (1, 1), window=4096, sinks=4),
        # prompts of several users in one call, odd lengths, one of them behind older turns
        _case("attention", "attn_prompts", "bf16", GQA128, 16, 4, (0, 2049), (517, 2048)),
        # one long prompt under a window with sinks
        _case("attention", "attn_prompt_window", "f16", MHA64, 64, 1, (0, 0), (8191, 8191), window=1024, sinks=4),
        # a decode batch that shares a system prompt
        _case("prefix", "prefix_decode_b64", "bf16", GQA128, 16, 64, (32, 515), (1, 1), prefix=8192),
        # sampling many answers to one long document, four draft tokens a step
        _case("prefix", "prefix_draft_b128", "bf16", GQA128, 64, 128, (8, 1030), (4, 4), prefix=16385),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(("append", "attention", "attention", "prefix"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f16", "f32"))
    d = rng.choice((64, 128))
    nkv = rng.choice((1, 2, 4, 8))
    nq = nkv * rng.choice((1, 2, 3, 4, 7, 8))
    page = rng.choice((16, 32, 64, 128))
    theta = rng.choice((1e4, 5e5, 1e6))
    axes, window, sinks, prefix = "", 0, 0, 0
    if op == "append":
        batch = log(1, 64)
        ctx_hi = log(1, 16384)
        q_hi = log(1, max(1, 16384 // batch))
        if rng.random() < 0.5:
            h = rng.randint(1, d // 2 // 3)
            axes = "%d,%d,%d" % (d // 2 - 2 * h, h, h) + rng.choice(("", ",i"))
    else:
        batch = log(1, 96)
        q_hi = 1 if rng.random() < 0.5 else log(2, max(2, 4096 // batch))
        ctx_hi = log(16, max(16, min(32768, 400000 // batch)))
        if q_hi > 64:
            ctx_hi = min(ctx_hi, 2048)
        if dtype == "f32":  # a type for checking models, not for serving them
            batch, q_hi, ctx_hi = min(batch, 8), min(q_hi, 128), min(ctx_hi, 2048)
        if op == "prefix":
            prefix = log(100, 16384 if dtype != "f32" else 1024)
            ctx_hi = min(ctx_hi, 1024)
            q_hi = min(q_hi, 16)
        elif rng.random() < 0.5:
            window, sinks = log(16, 4096), rng.choice((0, 4, 16))
    ctx_lo = rng.randint(0, ctx_hi)
    q_lo = rng.randint(1, q_hi)
    c = _case(op, "", dtype, (nq, nkv, d), page, batch, (ctx_lo, ctx_hi), (q_lo, q_hi), theta, axes, window, sinks, prefix)
    del c["name"]
    return c


def _lens(c):
    """q_len and ctx of every sequence."""
    r = random.Random(c["batch"] * 7919 + c["ctx_hi"] * 31 + c["q_hi"])
    return ([r.randint(c["q_lo"], c["q_hi"]) for _ in range(c["batch"])],
            [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["batch"])])


def _axes(c):
    """Pairs for each axis, and whether the axes are interleaved."""
    parts = c["axes"].split(",") if c["axes"] else []
    return [int(x) for x in parts[:3]], parts[3:] == ["i"]


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    dt = DTYPES[c["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    q_len, ctx = _lens(c)
    kv = [a + b for a, b in zip(q_len, ctx)]
    T, B, page, nq, nkv, d = sum(q_len), c["batch"], c["page"], c["nq"], c["nkv"], c["d"]
    per_seq = -(-max(kv) // page)
    used = [-(-x // page) for x in kv]
    n_prefix = -(-c["prefix"] // page)
    n_pages = sum(used) + n_prefix + 3
    order = torch.randperm(n_pages, generator=g, device=dev).int()  # pages are handed out in no order
    first = torch.tensor([sum(used[:b]) for b in range(B)], device=dev)
    cols = torch.arange(per_seq, device=dev)
    table = torch.where(cols[None] < torch.tensor(used, device=dev)[:, None],
                        order[(first[:, None] + cols[None]).clamp(max=n_pages - 1)], order[-1:])
    s = {"case": c, "batch": B, "tokens": T, "max_q": max(q_len),
         "q_start": torch.tensor([sum(q_len[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev),
         "kv_len": torch.tensor(kv, dtype=torch.int32, device=dev), "page_table": table.int().contiguous(),
         "prefix_table": order[sum(used):sum(used) + n_prefix].clone(),
         "k_pages": torch.randn(n_pages, page, nkv, d, generator=g, device=dev).to(dt),
         "v_pages": torch.randn(n_pages, page, nkv, d, generator=g, device=dev).to(dt)}
    if c["op"] == "append":
        # the merged projection's output; a projected channel has its own scale
        x = torch.randn(T, (nq + 2 * nkv) * d, generator=g, device=dev)
        x *= 0.5 + torch.rand((nq + 2 * nkv) * d, generator=g, device=dev)
        s["qkv"] = x.to(dt)
        s["q"] = s["qkv"][:, :nq * d].view(T, nq, d)
        s["k"] = s["qkv"][:, nq * d:(nq + nkv) * d].view(T, nkv, d)
        s["v"] = s["qkv"][:, (nq + nkv) * d:].view(T, nkv, d)
        s["q_out"] = torch.empty(T, nq, d, dtype=dt, device=dev)
        s["rope_pos"] = None
        if c["axes"]:
            # text, then frames of 40 x 30 patches behind it: time, row and column of each
            i = torch.cat([torch.arange(a, a + n, device=dev) for a, n in zip(ctx, q_len)])
            at = torch.randint(0, 900, (1,), generator=g, device=dev)
            s["rope_pos"] = torch.stack([at + i // 1200, at + i // 40 % 30, at + i % 40]).int().contiguous()
    else:
        # scores with a standard deviation of about two: attention that picks some keys out
        s["q"] = (2 * torch.randn(T, nq, d, generator=g, device=dev)).to(dt)
        s["out"] = torch.empty(T, nq, d, dtype=dt, device=dev)
    if own:
        from attention_block_gb300 import binding
        sections, inter = _axes(c)
        s["kv"] = binding.PagedKv(n_q_heads=nq, n_kv_heads=nkv, head_dim=d, page_size=page, num_pages=n_pages,
                                  max_batch=B, max_tokens=T, max_pages=per_seq, rope_theta=c["theta"],
                                  rope_sections=sections or None, rope_interleaved=inter, dtype=c["dtype"])
    return s


# ------------------------------------------------------------ plain forms --
def _token_grid(s):
    """Row of each (sequence, i) in the token arrays, which of them exist, and their positions: [B, N]."""
    i = torch.arange(s["max_q"], device=s["kv_len"].device)
    a, b = s["q_start"][:-1, None].long(), s["q_start"][1:, None].long()
    tok = a + i
    return tok.clamp(max=s["tokens"] - 1), tok < b, s["kv_len"][:, None].long() - (b - a) + i


def _plain_rope(x, pos, c):
    """x [T, heads, d] with positions pos [axes, T], rotate-half."""
    half = c["d"] // 2
    i = torch.arange(half, device=x.device)
    sections, inter = _axes(c)
    if not sections:
        axis = torch.zeros_like(i)
    elif inter:
        axis = torch.where((i % 3 == 1) & (i < 3 * sections[1]), 1, torch.where((i % 3 == 2) & (i < 3 * sections[2]), 2, 0))
    else:
        axis = (i >= sections[0]).long() + (i >= sections[0] + sections[1]).long()
    freq = torch.pow(torch.tensor(c["theta"], dtype=torch.float64, device=x.device), -2.0 * i.double() / c["d"])
    ang = pos.double()[axis].T * freq  # [T, half]: far positions lose their angle in 32 bits
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(x.dtype)


def _plain_append(s):
    c = s["case"]
    tok, there, pos = _token_grid(s)
    seq = torch.arange(s["batch"], device=tok.device)[:, None].expand_as(tok)[there]
    p = pos[there]  # tokens lie in the order of their sequences
    rp = s["rope_pos"] if s["rope_pos"] is not None else p[None]
    page = s["page_table"][seq, p // c["page"]].long()
    s["k_pages"][page, p % c["page"]] = _plain_rope(s["k"], rp, c)
    s["v_pages"][page, p % c["page"]] = s["v"]
    return {"q": _plain_rope(s["q"], rp, c), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _rows(s, x):
    """[B, N, nq, d] -> [B, nkv, N*G, d]"""
    c = s["case"]
    B, N = x.shape[:2]
    return x.view(B, N, c["nkv"], c["nq"] // c["nkv"], c["d"]).transpose(1, 2).reshape(B, c["nkv"], -1, c["d"])


def _plain_scores(s):
    """Scores of every sequence over its own pages, masked, [B, nkv, N*G, S], and the values [B, nkv, S, d]."""
    c = s["case"]
    tok, there, pos = _token_grid(s)
    G = c["nq"] // c["nkv"]
    K = s["k_pages"][s["page_table"].long()].flatten(1, 2).float().transpose(1, 2)
    V = s["v_pages"][s["page_table"].long()].flatten(1, 2).float().transpose(1, 2)
    j = torch.arange(K.shape[2], device=K.device)
    p = pos[:, :, None]
    see = (j <= p) & (j < s["kv_len"][:, None, None])
    if c["window"]:
        see &= (p - j < c["window"]) | (j < c["sinks"])
    sc = _rows(s, s["q"][tok].float()) @ K.transpose(2, 3)
    sc *= c["d"] ** -0.5
    sc.view(*sc.shape[:2], -1, G, sc.shape[3]).masked_fill_(~see[:, None, :, None], float("-inf"))
    return sc, V, tok, there


def _take_rows(s, o, tok, there):
    c = s["case"]
    B, N = tok.shape
    o = o.view(B, c["nkv"], N, -1, c["d"]).transpose(1, 2).reshape(B, N, c["nq"], c["d"])
    out = torch.zeros(s["tokens"], c["nq"], c["d"], dtype=s["q"].dtype, device=o.device)
    out[tok[there]] = o[there].to(out.dtype)
    return out


def _plain_attention(s):
    sc, V, tok, there = _plain_scores(s)
    sc.sub_(sc.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    total = sc.sum(-1, keepdim=True)
    return {"out": _take_rows(s, (sc @ V) / total, tok, there)}


def _plain_prefix(s):
    c = s["case"]
    nkv, P = c["nkv"], c["prefix"]
    sc, V, tok, there = _plain_scores(s)
    Kp = s["k_pages"][s["prefix_table"].long()].flatten(0, 1)[:P].float().transpose(0, 1)
    Vp = s["v_pages"][s["prefix_table"].long()].flatten(0, 1)[:P].float().transpose(0, 1)
    B, N = tok.shape
    rows = _rows(s, s["q"][tok].float()).transpose(0, 1).reshape(nkv, -1, c["d"])
    sp = rows @ Kp.transpose(1, 2)
    sp *= c["d"] ** -0.5
    top = torch.maximum(sp.amax(-1).view(nkv, B, -1).transpose(0, 1), sc.amax(-1))[..., None]
    sc.sub_(top).exp_()
    sp.sub_(top.transpose(0, 1).reshape(nkv, -1, 1)).exp_()
    total = sc.sum(-1, keepdim=True) + sp.sum(-1).view(nkv, B, -1, 1).transpose(0, 1)
    o = sc @ V + (sp @ Vp).view(nkv, B, -1, c["d"]).transpose(0, 1)
    return {"out": _take_rows(s, o / total, tok, there)}


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"append": _plain_append, "attention": _plain_attention, "prefix": _plain_prefix}[op](s)
    kv, c = s["kv"], s["case"]
    starts = s["q_start"] if s["max_q"] > 1 else None  # one token per sequence needs no starts
    if op == "append":
        kv.append(s["batch"], s["tokens"], s["q"], s["k"], s["v"], starts, s["kv_len"], s["page_table"], s["k_pages"],
                  s["v_pages"], s["q_out"], rope_pos=s["rope_pos"])
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "attention":
        kv.attention(s["batch"], s["tokens"], s["max_q"], s["q"], starts, s["kv_len"], s["page_table"], s["k_pages"],
                     s["v_pages"], s["out"], window=c["window"], n_sinks=c["sinks"])
    else:
        kv.prefix_attention(s["batch"], s["tokens"], s["max_q"], s["q"], starts, s["kv_len"], s["page_table"],
                            s["prefix_table"], c["prefix"], s["k_pages"], s["v_pages"], s["out"])
    return {"out": s["out"]}


# ----------------------------------------------------------------- the work --
def _visible(p, window, sinks):
    """Number of keys that position p sees."""
    if not window or p < window:
        return p + 1
    return window + min(sinks, p + 1 - window)


def work(case):
    c = case
    es = 4 if c["dtype"] == "f32" else 2
    q_len, ctx = _lens(c)
    T = sum(q_len)
    if c["op"] == "append":
        n = (c["nq"] + 2 * c["nkv"]) * c["d"]
        pos = 4 * T * (3 if c["axes"] else 0)
        return {"bytes": 2 * T * n * es + 4 * (2 * c["batch"] + 1) + pos, "flops": 3 * T * (c["nq"] + c["nkv"]) * c["d"]}
    pairs, keys = c["prefix"] * T, c["prefix"]
    for n, a in zip(q_len, ctx):
        pairs += sum(_visible(p, c["window"], c["sinks"]) for p in range(a, a + n))
        lo = max(0, a - c["window"] + 1) if c["window"] else 0  # the first token's window starts here
        keys += a + n - lo + min(c["sinks"] if c["window"] else 0, lo)
    kv_bytes = 2 * keys * c["nkv"] * c["d"] * es + 4 * (-(-keys // c["page"]))
    return {"bytes": kv_bytes + 2 * T * c["nq"] * c["d"] * es, "flops": 4 * pairs * c["nq"] * c["d"]}


# ------------------------------------------------------------ in 64 bits --
def exact(case, seed):
    s = prepare(case, seed)
    c, f64 = case, torch.float64
    nq, nkv, d, page = c["nq"], c["nkv"], c["d"], c["page"]
    q_len, ctx = _lens(c)
    dev = s["q"].device
    if c["op"] == "append":
        sections, inter = _axes(c)
        rate = [float(c["theta"]) ** (-2.0 * i / d) for i in range(d // 2)]
        which = [0] * (d // 2)
        for i in range(d // 2):
            if sections and inter:
                which[i] = i % 3 if i < 3 * sections[i % 3] else 0
            elif sections:
                which[i] = 0 if i < sections[0] else 1 if i < sections[0] + sections[1] else 2
        k_pool, v_pool = s["k_pages"].to(f64), s["v_pages"].to(f64)
        qs, at = [], 0
        for b in range(c["batch"]):
            n = q_len[b]
            p = torch.arange(ctx[b], ctx[b] + n, device=dev)
            axes = s["rope_pos"][:, at:at + n].to(f64) if s["rope_pos"] is not None else p.to(f64).expand(3, n)
            ang = torch.stack([axes[which[i]] * rate[i] for i in range(d // 2)], 1)
            z = torch.polar(torch.ones_like(ang), ang)[:, None]

            def turn(x):
                y = torch.complex(x[..., :d // 2].to(f64), x[..., d // 2:].to(f64)) * z
                return torch.cat([y.real, y.imag], -1)

            ids = s["page_table"][b][p // page].long()
            k_pool[ids, p % page] = turn(s["k"][at:at + n])
            v_pool[ids, p % page] = s["v"][at:at + n].to(f64)
            qs.append(turn(s["q"][at:at + n]))
            at += n
        return {"q": torch.cat(qs), "k_pages": k_pool, "v_pages": v_pool}
    pairs = work(case)["flops"]
    if pairs > 4e12:
        return None
    out = torch.zeros(sum(q_len), nq, d, dtype=f64, device=dev)
    pre = s["prefix_table"].long()
    Kp = s["k_pages"][pre].reshape(-1, nkv, d)[:c["prefix"]].to(f64)
    Vp = s["v_pages"][pre].reshape(-1, nkv, d)[:c["prefix"]].to(f64)
    at = 0
    for b in range(c["batch"]):
        n, a = q_len[b], ctx[b]
        ids = s["page_table"][b].long()
        K = torch.cat([Kp, s["k_pages"][ids].reshape(-1, nkv, d)[:a + n].to(f64)])
        V = torch.cat([Vp, s["v_pages"][ids].reshape(-1, nkv, d)[:a + n].to(f64)])
        own_j = torch.arange(a + n, device=dev)
        for lo in range(0, n, 512):
            hi = min(n, lo + 512)
            p = torch.arange(a + lo, a + hi, device=dev)[:, None]
            hide = own_j > p
            if c["window"]:
                hide |= (own_j <= p - c["window"]) & (own_j >= c["sinks"])
            hide = torch.cat([torch.zeros(hi - lo, c["prefix"], dtype=torch.bool, device=dev), hide], 1)
            for h in range(nkv):
                heads = slice(h * (nq // nkv), (h + 1) * (nq // nkv))
                x = torch.einsum("nhd,sd->hns", s["q"][at + lo:at + hi, heads].to(f64), K[:, h]) / d ** 0.5
                w = torch.softmax(x.masked_fill(hide, float("-inf")), -1)
                out[at + lo:at + hi, heads] = torch.einsum("hns,sd->nhd", w, V[:, h])
        at += n
    return {"out": out}
