"""The 8-bit paged KV cache's operators, as cases to measure: appending keys and values with
the rotary rotation applied on the way, attention over the cache, and attention over
picked regions of the cache.

Notation: N query rows, ``rows`` consecutive ones for each of B sequences (row j of
sequence b at position start_b + j), G KV groups, Hq query heads, head dim 128, regions of
8 tokens.  A pool has pages of ``page_tokens`` tokens, [P][G][page_tokens][128], and a
block table [B][T] of page numbers in a random order.  In 8 bits the pool holds e4m3 codes and a
scale for each region and group, [P][G][page_tokens / 8]; a scale is the smallest power of
two that brings the region within 448.
"""
import math

import torch

own = False

D = 128          # head dim
RT = 8           # tokens of a region
DEV = "cuda" if torch.cuda.is_available() else "cpu"


def listed():
    return [
        # one decode row of a 4,608-token context into the framework's own bf16 caches
        {"name": "append_bf16_decode_1x4608", "op": "append", "bits": 16, "B": 1, "rows": 1, "lo": 4608, "hi": 4608,
         "G": 4, "hq": 8, "page_tokens": 4616, "rot": 128},
        # a prompt chunk of 2,048 tokens, q rotated beside k, into 64-token bf16 pages
        {"name": "append_bf16_chunk_2048", "op": "append", "bits": 16, "B": 1, "rows": 2048, "lo": 4096, "hi": 4096,
         "G": 4, "hq": 8, "page_tokens": 64, "rot": 64},
        # a decode batch: 16 rows at ragged positions, most of them inside a half-filled region
        {"name": "append_e4m3_decode_16", "op": "append", "bits": 8, "B": 16, "rows": 1, "lo": 1000, "hi": 4607,
         "G": 4, "hq": 8, "page_tokens": 64, "rot": 128},
        # prompt chunks of four sequences, each starting and ending inside a region
        {"name": "append_e4m3_chunk_4x1021", "op": "append", "bits": 8, "B": 4, "rows": 1021, "lo": 1000, "hi": 4000,
         "G": 4, "hq": 8, "page_tokens": 64, "rot": 64},
        # one decode row over all of a 4,608-token context: latency
        {"name": "paged_decode_1x4608", "op": "paged", "B": 1, "rows": 1, "lo": 4608, "hi": 4608, "G": 4, "hq": 8,
         "page_tokens": 64, "window": 0},
        # a ragged decode batch at 16K to 32K tokens
        {"name": "paged_decode_16x16k-32k", "op": "paged", "B": 16, "rows": 1, "lo": 16384, "hi": 32768, "G": 4,
         "hq": 8, "page_tokens": 64, "window": 0},
        # one decode row at 1M tokens
        {"name": "paged_decode_1x1m", "op": "paged", "B": 1, "rows": 1, "lo": 1048576, "hi": 1048576, "G": 4, "hq": 8,
         "page_tokens": 64, "window": 0},
        # a prompt chunk whose rows still see every token (within the selection's 512 regions)
        {"name": "paged_chunk_2048_on_2k", "op": "paged", "B": 1, "rows": 2048, "lo": 2048, "hi": 2048, "G": 4, "hq": 8,
         "page_tokens": 64, "window": 0},
        # a prompt chunk of a sliding-window layer, window 512
        {"name": "paged_chunk_2048_window_512", "op": "paged", "B": 1, "rows": 2048, "lo": 6144, "hi": 6144, "G": 4,
         "hq": 8, "page_tokens": 64, "window": 512},
        # one decode row at 1M tokens over its 512 picked regions and its own: latency
        {"name": "sparse_decode_1x1m", "op": "sparse", "B": 1, "rows": 1, "lo": 1048576, "hi": 1048576, "G": 4, "hq": 8,
         "page_tokens": 64, "top_k": 512},
        # the ragged decode batch over picked regions
        {"name": "sparse_decode_16x16k-32k", "op": "sparse", "B": 16, "rows": 1, "lo": 16384, "hi": 32768, "G": 4,
         "hq": 8, "page_tokens": 64, "top_k": 512},
        # a prompt chunk of 2,048 rows at 64K tokens over picked regions
        {"name": "sparse_chunk_2048_on_64k", "op": "sparse", "B": 1, "rows": 2048, "lo": 65536, "hi": 65536, "G": 4,
         "hq": 8, "page_tokens": 64, "top_k": 512},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "paged", "paged", "sparse", "sparse"])
    G, hq = rng.choice([1, 2, 4, 4, 8]), rng.choice([4, 8, 8, 16])
    c = {"op": op, "G": G, "hq": hq, "page_tokens": rng.choice([8, 16, 24, 32, 64, 128, 200, 256])}
    if op == "append":
        c["bits"] = rng.choice([8, 8, 16])
        c["rot"] = rng.choice([0, 16, 32, 64, 96, 128])
        c["B"] = _log_int(rng, 1, 64)
        most = min(2048, 65536 // (G * hq)) // c["B"]
        c["rows"] = rng.choice([1, _log_int(rng, 1, max(1, most))])
        c["lo"], c["hi"] = sorted(_log_int(rng, 1, min(6000, 60000 // c["B"])) - 1 for _ in range(2))
        return c
    if rng.random() < 0.65:      # decode rows, up to four of a sequence
        c["B"] = _log_int(rng, 1, 32)
        c["rows"] = rng.choice([1, 1, 1, 2, 4])
        longest, top = min(131072, (4 << 20) // (c["B"] * G)), 1024
    else:                        # chunks
        c["B"] = rng.choice([1, 1, 2, 3])
        c["rows"] = _log_int(rng, 16, min(1500, 65536 // (G * hq)) // c["B"])
        longest, top = (1500 if op == "paged" else 16384), 512
    c["lo"], c["hi"] = sorted(_log_int(rng, 1, longest) - 1 for _ in range(2))
    if op == "paged":
        c["window"] = rng.choice([0, 0, 0, 1, 100, 512, _log_int(rng, 2, 2000)])
    else:
        c["top_k"] = rng.choice([512, 512, 64, _log_int(rng, 1, top)])
    return c


# ---------------------------------------------------------------- what a program has in hand

def _starts(case, gen):
    """First position of each sequence's rows, uniform on [lo, hi]."""
    u = torch.rand(case["B"], generator=gen, device=DEV, dtype=torch.float64)
    return (case["lo"] + (u * (case["hi"] - case["lo"] + 1)).floor().long()).clamp(max=case["hi"])


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _pool_of_codes(gen, pages, G, pt):
    """A pool as an e4m3 cache holds it: codes of normal values within 448 and the power-of-two
    scale of each region and group (values of about unit size, within two binades)."""
    codes = torch.empty((pages, G, pt, D), device=DEV, dtype=torch.uint8)
    flat = codes.view(-1)
    step = 1 << 27
    for at in range(0, flat.numel(), step):
        x = torch.randn(min(step, flat.numel() - at), generator=gen, device=DEV).mul_(100.0).clamp_(-448.0, 448.0)
        flat[at:at + step] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    e = torch.randint(-8, -5, (pages, G, pt // RT), generator=gen, device=DEV)
    return codes, torch.exp2(e.float())


def _picks(gen, starts, case, G):
    """sel_ids [N][G][top_k] and sel_count [N][G]: min(top_k, regions before the row's own)
    distinct regions of each row, in a random order, -1 behind them."""
    B, rows, top_k = case["B"], case["rows"], case["top_k"]
    ids = torch.full((B * rows, G, top_k), -1, device=DEV, dtype=torch.int32)
    regions = ((starts[:, None] + torch.arange(rows, device=DEV)) // RT).reshape(-1)
    count = regions.clamp(max=top_k)
    most = max(1, int(regions.max()))
    step = max(1, (1 << 28) // (G * most))
    for n in range(0, B * rows, step):
        r = regions[n:n + step]
        s = torch.rand((r.numel(), G, most), generator=gen, device=DEV)
        s.masked_fill_(torch.arange(most, device=DEV) >= r[:, None, None], -1.0)
        got = s.topk(min(top_k, most), dim=-1)
        ids[n:n + step, :, :got.indices.shape[-1]] = torch.where(got.values >= 0, got.indices, -1).int()
    return ids, count[:, None].expand(-1, G).contiguous().int()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    B, rows, G, pt = case["B"], case["rows"], case["G"], case["page_tokens"]
    Hq, N = G * case["hq"], case["B"] * case["rows"]
    starts = _starts(case, gen)
    table_len = -(-(case["hi"] + rows) // pt)
    pages = B * table_len
    s = {"case": dict(case), "starts": starts,
         "table": torch.randperm(pages, generator=gen, device=DEV).int().view(B, table_len).contiguous(),
         "row_seq": torch.arange(B, device=DEV).repeat_interleave(rows).int(),
         "row_pos": (starts[:, None] + torch.arange(rows, device=DEV)).reshape(-1).int()}
    if case["op"] == "append":
        # q, k and v as they come out of one projection: [N][(Hq + 2 G) * 128]
        qkv = _normal(gen, N, Hq + 2 * G, D) * torch.exp(_normal(gen, N, Hq + 2 * G, 1) * 0.5)
        s["qkv"] = qkv.bfloat16()
        pos = torch.arange(table_len * pt, device=DEV, dtype=torch.float64)
        if case["rot"]:
            inv = 10000.0 ** (-torch.arange(case["rot"] // 2, device=DEV, dtype=torch.float64) * 2 / case["rot"])
            s["cos"], s["sin"] = ((pos[:, None] * inv).cos().float().bfloat16(), (pos[:, None] * inv).sin().float().bfloat16())
        else:
            s["cos"] = s["sin"] = None
        s["q_out"] = torch.zeros((N, Hq, D), device=DEV, dtype=torch.bfloat16)
        if case["bits"] == 8:
            s["k"], s["k_scale"] = _pool_of_codes(gen, pages, G, pt)
            s["v"], s["v_scale"] = _pool_of_codes(gen, pages, G, pt)
        else:
            s["k"], s["v"] = (_normal(gen, pages, G, pt, D).bfloat16() for _ in range(2))
            s["k_scale"] = s["v_scale"] = None
        return s
    s["q"] = (_normal(gen, N, Hq, D) * 1.5).bfloat16()
    s["k"], s["k_scale"] = _pool_of_codes(gen, pages, G, pt)
    s["v"], s["v_scale"] = _pool_of_codes(gen, pages, G, pt)
    s["out"] = torch.zeros((N, Hq, D), device=DEV, dtype=torch.bfloat16)
    if case["op"] == "sparse":
        s["sel_ids"], s["sel_count"] = _picks(gen, starts, case, G)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _own_append, "paged": _own_paged, "sparse": _own_sparse}[op](s)
    return {"append": _plain_append, "paged": _plain_paged, "sparse": _plain_sparse}[op](s)


def _handles(s):
    """The framework's geometry, cache handle and workspace, made once for a state, as a program keeps them."""
    if "cache" not in s:
        import block_sparse_attention_step5_gb300 as s5

        c = s["case"]
        s["s5"] = s5
        s["geom"] = s5.Geometry.step5(num_q_heads=c["G"] * c["hq"], num_kv_groups=c["G"], idx_heads=c["G"] * 4,
                                      top_k=c.get("top_k", 512))
        s["cache"] = s5.PagedCache(s["k"], s["v"], s["table"], s["k_scale"], s["v_scale"])
        s["ws"] = s5.PagedWorkspace.create(s["geom"]) if c["op"] != "append" else None
    return s["s5"], s["geom"], s["cache"], s["ws"]


def _own_append(s):
    s5, geom, cache, _ = _handles(s)
    Hq, G = geom.num_q_heads, geom.num_kv_groups
    q, k, v = s["qkv"].split((Hq, G, G), dim=1)
    call = s5.step5_kv_append_e4m3 if s["case"]["bits"] == 8 else s5.step5_kv_append
    call(geom, k, v, cache, s["row_seq"], s["row_pos"], s["cos"], s["sin"], q=q, q_out=s["q_out"])
    return _append_outputs(s)


def _own_paged(s):
    s5, geom, cache, ws = _handles(s)
    s5.step5_paged_attn_e4m3(geom, s["q"], cache, s["row_seq"], s["row_pos"], s["out"], ws, window=s["case"]["window"])
    return s["out"]


def _own_sparse(s):
    s5, geom, cache, ws = _handles(s)
    s5.step5_sparse_attn_e4m3(geom, s["q"], cache, s["row_seq"], s["row_pos"], s["sel_ids"], s["sel_count"], s["out"], ws)
    return s["out"]


def _append_outputs(s):
    out = {"q": s["q_out"]}
    if s["case"]["bits"] == 8:  # the codes as e4m3 numbers, each region's scale beside them
        out.update(k=s["k"].view(torch.float8_e4m3fn), v=s["v"].view(torch.float8_e4m3fn), k_scale=s["k_scale"],
                   v_scale=s["v_scale"])
    else:
        out.update(k=s["k"], v=s["v"])
    return out


# ---------------------------------------------------------------- plain forms (32 bits)

def _to_bf16(x):
    """bf16 of 64-bit values, rounded once: first to 32 bits, to odd, then to bf16."""
    f = x.float()
    u = f.view(torch.int32)
    u = torch.where(f.double().abs() > x.abs(), u - 1, u)
    u = torch.where(f.double() != x, u | 1, u)
    return u.view(torch.float32).bfloat16()


def _plain_rotate(x, cos, sin, pos):
    """x [N][H][128], the first rot dims rotated: pairs (i, i + rot / 2)."""
    if cos is None:
        return x
    half = cos.shape[1]
    c, n = (t[pos.long()].double()[:, None, :] for t in (cos, sin))
    a, b = x[..., :half].double(), x[..., half:2 * half].double()
    return torch.cat((_to_bf16(a * c - b * n), _to_bf16(b * c + a * n), x[..., 2 * half:]), dim=-1)


def _plain_scale(amax):
    """The smallest power of two s with amax <= 448 s (0 for amax 0)."""
    m, e = torch.frexp(amax / 1.75)
    return torch.where(amax > 0, torch.exp2((e - 8 - (m == 0.5).int()).float()), 0.0)


def _plain_append(s):
    c = s["case"]
    B, rows, G, pt = c["B"], c["rows"], c["G"], c["page_tokens"]
    Hq = G * c["hq"]
    q, k, v = s["qkv"].split((Hq, G, G), dim=1)
    s["q_out"].copy_(_plain_rotate(q, s["cos"], s["sin"], s["row_pos"]))
    k = _plain_rotate(k, s["cos"], s["sin"], s["row_pos"])
    seq, pos = s["row_seq"].long(), s["row_pos"].long()
    page, slot = s["table"].long()[seq, pos // pt], pos % pt
    if c["bits"] == 16:
        s["k"][page, :, slot] = k
        s["v"][page, :, slot] = v
        return _append_outputs(s)
    first = s["starts"]                                          # the first region's tokens before the rows stay
    p0, r0 = s["table"].long()[torch.arange(B, device=DEV), first // pt], first % pt // RT
    kept = torch.arange(RT, device=DEV) < (first % RT)[:, None]  # [B][8]
    for x, codes, scales in ((k, s["k"], s["k_scale"]), (v, s["v"], s["v_scale"])):
        regions = codes.view(codes.shape[0], G, pt // RT, RT, D)
        before = scales[p0, :, r0].clone()                       # [B][G]
        # the largest value of each region, from the rows that fall into it
        span = (first % RT + rows + RT - 1) // RT
        most = (rows + 2 * RT - 2) // RT
        amax = torch.zeros((B, most, G), device=DEV)
        local = pos // RT - (first // RT)[seq]
        amax.view(B * most, G).scatter_reduce_(0, (seq * most + local)[:, None].expand(-1, G),
                                               x.float().abs().amax(-1), "amax")
        new = _plain_scale(amax).clamp(min=2.0 ** -126)
        new[:, 0] = torch.where(kept.any(1)[:, None], torch.maximum(new[:, 0], before), new[:, 0])
        reg = (first // RT)[:, None] + torch.arange(most, device=DEV)
        b_at, m_at = (torch.arange(most, device=DEV) < span[:, None]).nonzero(as_tuple=True)
        reg = reg[b_at, m_at]
        scales[s["table"].long()[b_at, reg * RT // pt], :, reg * RT % pt // RT] = new[b_at, m_at]
        old = regions[p0, :, r0]                                 # [B][G][8][128], requantised where the scale grew
        val = old.view(torch.float8_e4m3fn).float() * (before / new[:, 0])[:, :, None, None]
        regions[p0, :, r0] = torch.where(kept[:, None, :, None], val.to(torch.float8_e4m3fn).view(torch.uint8), old)
        val = x.float() / new[seq, local][:, :, None]
        codes[page, :, slot] = val.to(torch.float8_e4m3fn).view(torch.uint8)
    return _append_outputs(s)


def _plain_values(s, codes, scales, seq, tok):
    """fp32 values of tokens tok [..., L] of sequences seq [..., 1]: [..., G, L, 128]."""
    pt = s["case"]["page_tokens"]
    page = s["table"].long()[seq, tok // pt]
    x = codes[page, :, tok % pt].view(torch.float8_e4m3fn).float() * scales[page, :, tok % pt // RT][..., None]
    return x.transpose(-3, -2)


def _plain_softmax_av(q, k, v, seen):
    """q [..., G, R, 128] against k, v [..., G, L, 128], seen [..., G, R, L]: [..., G, R, 128]."""
    x = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D))
    x.masked_fill_(~seen, -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    return (x @ v) / x.sum(-1, keepdim=True)


def _plain_paged(s):
    c = s["case"]
    B, rows, G, hq, W = c["B"], c["rows"], c["G"], c["hq"], c["window"]
    first = s["starts"]
    lo = (first - W + 1).clamp(min=0) if W else torch.zeros_like(first)
    L = c["hi"] + rows if not W else min(c["hi"] + rows, rows + W - 1)
    tok = lo[:, None] + torch.arange(L, device=DEV)               # [B][L]
    at = tok.clamp(max=s["table"].shape[1] * c["page_tokens"] - 1)
    seq = torch.arange(B, device=DEV)[:, None]
    k, v = (_plain_values(s, s[x], s[x + "_scale"], seq, at) for x in "kv")
    pos = first[:, None] + torch.arange(rows, device=DEV)         # [B][rows]
    seen = tok[:, None, :] <= pos[:, :, None]
    if W:
        seen &= tok[:, None, :] > pos[:, :, None] - W
    seen = seen[:, None, :, None, :].expand(-1, -1, -1, hq, -1).reshape(B, 1, rows * hq, L)
    q = s["q"].float().view(B, rows, G, hq, D).transpose(1, 2).reshape(B, G, rows * hq, D)
    o = _plain_softmax_av(q, k, v, seen).view(B, G, rows, hq, D).transpose(1, 2)
    s["out"].copy_(o.reshape(B * rows, G * hq, D))
    return s["out"]


def _plain_sparse(s):
    c = s["case"]
    G, hq, N = c["G"], c["hq"], c["B"] * c["rows"]
    step = max(1, (1 << 30) // (G * (c["top_k"] + 1) * RT * D))   # rows whose gathered keys fit in 4 GB
    for n in range(0, N, step):
        pos = s["row_pos"][n:n + step].long()
        m = pos.numel()
        ids = torch.cat((s["sel_ids"][n:n + step].long(), (pos // RT)[:, None, None].expand(m, G, 1)), dim=2)
        tok = (ids[..., None] * RT + torch.arange(RT, device=DEV)).view(m, G, -1)
        seen = (tok >= 0) & (tok <= pos[:, None, None])
        at = tok.clamp(min=0, max=s["table"].shape[1] * c["page_tokens"] - 1)
        page, slot = s["table"].long()[s["row_seq"][n:n + step].long()[:, None, None], at // c["page_tokens"]], at % c["page_tokens"]
        g = torch.arange(G, device=DEV)[None, :, None]
        k, v = (s[x][page, g, slot].view(torch.float8_e4m3fn).float() * s[x + "_scale"][page, g, slot // RT][..., None]
                for x in "kv")
        q = s["q"][n:n + step].float().view(m, G, hq, D)
        s["out"][n:n + step] = _plain_softmax_av(q, k, v, seen[:, :, None, :]).reshape(m, G * hq, D).bfloat16()
    return s["out"]


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _near(x, bits, low):
    """x (64 bits) to the nearest number of ``bits`` significant bits, ties to even, with
    no step finer than 2^low."""
    m, e = torch.frexp(x)
    ulp = torch.exp2((e - bits).clamp(min=low).double())
    return torch.round(x / ulp) * ulp


def _exact_append(s):
    c = s["case"]
    B, rows, G, pt = c["B"], c["rows"], c["G"], c["page_tokens"]
    Hq = G * c["hq"]
    x = s["qkv"].double()
    if c["rot"]:
        h, p = c["rot"] // 2, s["row_pos"].long()
        z = torch.complex(x[..., :h], x[..., h:2 * h])
        w = torch.complex(s["cos"].double()[p], s["sin"].double()[p])
        z = z * w[:, None]
        turned = torch.cat((_near(z.real, 8, -133), _near(z.imag, 8, -133), x[..., 2 * h:]), -1)
        x = torch.cat((turned[:, :Hq + G], x[:, Hq + G:]), 1)
    out = {"q": x[:, :Hq]}
    for name, new in (("k", x[:, Hq:Hq + G]), ("v", x[:, Hq + G:])):
        if c["bits"] == 16:
            pool = s[name].double()
            for b in range(B):
                t = torch.arange(rows, device=DEV) + s["starts"][b]
                pool[s["table"][b].long()[t // pt], :, t % pt] = new[b * rows:(b + 1) * rows]
            out[name] = pool
            continue
        pool, scale = s[name].view(torch.float8_e4m3fn).double(), s[name + "_scale"].double()
        for b in range(B):
            start = int(s["starts"][b])
            table = s["table"][b].long()
            # whole regions: tokens kept, then the rows' tokens, the last region's rest absent
            r0, r1 = start // RT, (start + rows - 1) // RT
            reg = torch.arange(r0, r1 + 1, device=DEV)
            page, at = table[reg * RT // pt], reg * RT % pt // RT
            tok = reg[:, None] * RT + torch.arange(RT, device=DEV)
            fresh = (tok >= start) & (tok < start + rows)
            val = torch.zeros((len(reg), RT, G, D), device=DEV, dtype=torch.float64)
            val[fresh] = new[b * rows:(b + 1) * rows]
            top = val.abs().amax((1, 3))                                  # [regions][G]
            e = torch.ceil(torch.log2(top / 448.0)).clamp(min=-126)
            e = e + (top > 448.0 * torch.exp2(e)).double() - (top <= 448.0 * torch.exp2(e - 1)).double()
            e = e.clamp(min=-126)
            if start % RT:
                e[0] = torch.maximum(e[0], torch.log2(scale[page[0], :, at[0]]).round())
            s8 = torch.exp2(e)
            shape = pool.view(pool.shape[0], G, pt // RT, RT, D)
            held = shape[page, :, at].transpose(1, 2)                     # [regions][8][G][128]
            held = held * torch.where((tok < start)[:, :, None], (scale[page, :, at] / s8)[:, None], 1.0)[..., None]
            val = torch.where(fresh[:, :, None, None], val / s8[:, None, :, None], held)
            shape[page, :, at] = _near(val, 4, -9).transpose(1, 2)
            scale[page, :, at] = s8
        out[name], out[name + "_scale"] = pool, scale
    return out


def _exact_attend(q, k, v):
    """One (row, group): q [hq][128], k, v [L][128]."""
    x = torch.softmax(q @ k.T / math.sqrt(D), dim=-1)
    return x @ v


def _exact_values(s, name, b, g, tok):
    pt = s["case"]["page_tokens"]
    page = s["table"][b].long()[tok // pt]
    return s[name][page, g, tok % pt].view(torch.float8_e4m3fn).double() * s[name + "_scale"][page, g, tok % pt // RT].double()[:, None]


def _exact_paged(s):
    c = s["case"]
    rows, G, hq, W = c["rows"], c["G"], c["hq"], c["window"]
    out = torch.zeros((c["B"] * rows, G, hq, D), device=DEV, dtype=torch.float64)
    for b, start in enumerate(s["starts"].tolist()):
        lo = max(0, start - W + 1) if W else 0
        tok = torch.arange(lo, start + rows, device=DEV)
        for g in range(G):
            k, v = (_exact_values(s, x, b, g, tok) for x in "kv")
            q = s["q"].view(-1, G, hq, D)[b * rows:(b + 1) * rows, g].double()
            for j in range(0, rows, 256):
                pos = torch.arange(start + j, start + min(rows, j + 256), device=DEV)[:, None, None]
                x = torch.einsum("rhd,ld->rhl", q[j:j + 256], k) / math.sqrt(D)
                hide = (tok > pos) | (tok <= pos - W if W else False)
                x = torch.softmax(x.masked_fill(hide, -math.inf), -1)
                out[b * rows + j:b * rows + j + pos.shape[0], g] = torch.einsum("rhl,ld->rhd", x, v)
    return out.view(-1, G * hq, D)


def _exact_sparse(s):
    c = s["case"]
    G, hq, N = c["G"], c["hq"], c["B"] * c["rows"]
    out = torch.zeros((N, G, hq, D), device=DEV, dtype=torch.float64)
    pos, seq, count = s["row_pos"].tolist(), s["row_seq"].tolist(), s["sel_count"].tolist()
    q = s["q"].view(N, G, hq, D).double()
    eight = torch.arange(RT, device=DEV)
    for n in range(N):
        mine = torch.arange(pos[n] // RT * RT, pos[n] + 1, device=DEV)
        for g in range(G):
            tok = torch.cat(((s["sel_ids"][n, g, :count[n][g]].long()[:, None] * RT + eight).reshape(-1), mine))
            out[n, g] = _exact_attend(q[n, g], *(_exact_values(s, x, seq[n], g, tok) for x in "kv"))
    return out.view(N, G * hq, D)


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "paged": _exact_paged, "sparse": _exact_sparse}[case["op"]](s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    B, rows, G, hq = case["B"], case["rows"], case["G"], case["hq"]
    N, Hq = B * rows, G * case["hq"]
    mid = (case["lo"] + case["hi"]) / 2
    if case["op"] == "append":
        # qkv read, q, k and v written, a scale for each region touched; table rows and positions
        kv = 2 * N * G * D * (2 if case["bits"] == 16 else 1)
        scales = 0 if case["bits"] == 16 else 2 * 4 * G * B * (rows / RT + 1)
        tables = 2 * 2 * N * case["rot"] // 2
        return {"bytes": N * (Hq + 2 * G) * D * 2 + N * Hq * D * 2 + kv + scales + tables, "flops": N * (Hq + G) * case["rot"] * 3}
    qo = 2 * N * Hq * D * 2
    per_token = G * (2 * D + 2 * 4 / RT)
    if case["op"] == "paged":
        W = case["window"]
        ends = [mid + j + 1 for j in range(rows)]
        keys = sum(min(e, W) if W else e for e in ends)
        span = mid + rows if not W else min(mid + rows, rows + W - 1)
        return {"bytes": qo + B * span * per_token, "flops": 4 * D * Hq * B * keys}
    picked = min(case["top_k"], mid / RT) * RT + RT / 2
    touched = min(rows * picked, mid + rows)
    return {"bytes": qo + B * touched * per_token + N * G * 4 * min(case["top_k"], mid / RT), "flops": 4 * D * Hq * N * picked}
