"""The bf16 paged KV cache's operators, as cases to measure: attention of decode rows, drafts and
prompt chunks over the pages, attention over picked regions of them, and the step's plan (pages
handed out and taken back, block tables, the rows' sequences and positions) made on the GPU.

Notation: N query rows, ``rows`` consecutive ones for each of B sequences (row j of sequence b at
position start_b + j; ragged cases give each sequence its own number of them), G KV groups, Hq query
heads, head dim 128, regions of 8 tokens.  A pool has pages of ``page_tokens`` tokens,
[P][G][page_tokens][128], and a block table [B][T] of page numbers in a random order.
"""
import math

import numpy as np
import torch

own = False

D = 128          # head dim
RT = 8           # tokens of a region
DEV = "cuda" if torch.cuda.is_available() else "cpu"


def listed():
    return [
        # one decode row over all of a 4,608-token context: latency
        {"name": "paged_decode_1x4608", "op": "paged", "B": 1, "rows": 1, "lo": 4608, "hi": 4608, "G": 4, "hq": 8,
         "page_tokens": 64, "window": 0, "gate": False, "apart": False},
        # a ragged decode batch at 16K to 32K tokens
        {"name": "paged_decode_16x16k-32k", "op": "paged", "B": 16, "rows": 1, "lo": 16384, "hi": 32768, "G": 4,
         "hq": 8, "page_tokens": 64, "window": 0, "gate": False, "apart": False},
        # eight sequences with four drafted tokens each, on pages that end inside a tile, with the output gate
        {"name": "paged_drafts_8x4_on_8k", "op": "paged", "B": 8, "rows": 4, "lo": 6000, "hi": 8191, "G": 4, "hq": 8,
         "page_tokens": 24, "window": 0, "gate": True, "apart": False},
        # a prompt chunk whose rows still see every token (within the selection's 512 regions)
        {"name": "paged_chunk_2048_on_2k", "op": "paged", "B": 1, "rows": 2048, "lo": 2048, "hi": 2048, "G": 4, "hq": 8,
         "page_tokens": 64, "window": 0, "gate": False, "apart": False},
        # a prompt chunk of a sliding-window layer, window 512, gated, q a slice of the projection's output
        {"name": "paged_chunk_2048_window_512", "op": "paged", "B": 1, "rows": 2048, "lo": 6144, "hi": 6144, "G": 4,
         "hq": 8, "page_tokens": 64, "window": 512, "gate": True, "apart": True},
        # three prompts of odd lengths from their first token on, 16 heads a group
        {"name": "paged_prompts_3x701", "op": "paged", "B": 3, "rows": 701, "lo": 0, "hi": 0, "G": 2, "hq": 16,
         "page_tokens": 16, "window": 0, "gate": False, "apart": False},
        # a prompt chunk of a dense layer deep in a long context
        {"name": "paged_chunk_2048_on_64k", "op": "paged", "B": 1, "rows": 2048, "lo": 65536, "hi": 65536, "G": 4,
         "hq": 8, "page_tokens": 64, "window": 0, "gate": False, "apart": False},
        # one decode row at 1M tokens over its 512 picked regions and its own: latency
        {"name": "sparse_decode_1x1m", "op": "sparse", "B": 1, "rows": 1, "lo": 1048576, "hi": 1048576, "G": 4, "hq": 8,
         "page_tokens": 64, "top_k": 512, "gate": True, "apart": False},
        # the ragged decode batch over picked regions
        {"name": "sparse_decode_16x16k-32k", "op": "sparse", "B": 16, "rows": 1, "lo": 16384, "hi": 32768, "G": 4,
         "hq": 8, "page_tokens": 64, "top_k": 512, "gate": False, "apart": False},
        # a prompt chunk of 2,048 rows at 64K tokens over picked regions
        {"name": "sparse_chunk_2048_on_64k", "op": "sparse", "B": 1, "rows": 2048, "lo": 65536, "hi": 65536, "G": 4,
         "hq": 8, "page_tokens": 64, "top_k": 512, "gate": False, "apart": False},
        # the plan of a decode step of 64 sequences (a token each, some at a page's end), and the roll-back of it
        {"name": "plan_decode_64", "op": "plan", "B": 64, "N": 64, "most": 1, "lo": 16384, "hi": 32768,
         "page_tokens": 64, "spare": 1.0},
        # a mixed step of 1,024 slots, prompts and decode rows and idle ones, more tokens than the free pages hold
        {"name": "plan_mixed_1024", "op": "plan", "B": 1024, "N": 65536, "most": 127, "lo": 0, "hi": 4095,
         "page_tokens": 16, "spare": 0.9},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["paged", "paged", "paged", "sparse", "sparse", "plan"])
    if op == "plan":
        B = _log_int(rng, 1, 1024)
        most = rng.choice([1, 4, _log_int(rng, 1, 127)])
        c = {"op": op, "B": B, "N": B * rng.choice([most, (most + 1) // 2 + 1]), "most": most,
             "page_tokens": rng.choice([8, 16, 24, 64, 128, 256]), "spare": rng.choice([0.0, 0.5, 0.9, 1.0, 1.0])}
        c["lo"], c["hi"] = sorted(_log_int(rng, 1, 4096) - 1 for _ in range(2))
        return c
    G, hq = rng.choice([1, 2, 4, 4, 8]), rng.choice([4, 8, 8, 16])
    c = {"op": op, "G": G, "hq": hq, "page_tokens": rng.choice([8, 16, 24, 32, 64, 128, 200, 256]),
         "gate": rng.random() < 0.4, "apart": rng.random() < 0.4}
    if rng.random() < 0.6:       # decode rows, up to four of a sequence
        c["B"] = _log_int(rng, 1, 32)
        c["rows"] = rng.choice([1, 1, 1, 2, 4])
        longest, top = min(131072, (4 << 20) // (c["B"] * G)), 1024
    else:                        # chunks
        c["B"] = rng.choice([1, 1, 2, 3])
        c["rows"] = _log_int(rng, 16, min(1500, 65536 // (G * hq)) // c["B"])
        longest, top = (8000 if op == "paged" else 16384), 512
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
    """bf16 normal values, drawn a part at a time."""
    x = torch.empty(shape, device=DEV, dtype=torch.bfloat16)
    flat, step = x.view(-1), 1 << 27
    for at in range(0, flat.numel(), step):
        part = flat[at:at + step]
        part.copy_(torch.randn(part.numel(), generator=gen, device=DEV))
    return x


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


def _prepare_plan(case, gen):
    """Slots of a serving program: some idle, some about to start, the others of lo .. hi tokens with their
    pages held; the tokens each gets next; the free pages, in a random order."""
    B, pt, N = case["B"], case["page_tokens"], case["N"]
    lengths = _starts(case, gen).int()
    kind = torch.rand(B, generator=gen, device=DEV)
    lengths[kind < 0.1] = 0
    new = (1 + torch.rand(B, generator=gen, device=DEV) * case["most"]).floor().clamp(max=case["most"]).int()
    new[(kind > 0.05) & (kind < 0.15)] = 0
    table_len = -(-(case["hi"] + case["most"]) // pt) + 1
    held = ((lengths + pt - 1) // pt).int()
    need = ((lengths + new + pt - 1) // pt - held).clamp(min=0)
    used, pages = int(held.sum()), B * table_len                   # (pages that are neither held nor free are others')
    free = max(1, int(int(need.sum()) * case["spare"])) + (1 if case["spare"] >= 1.0 else 0)
    order = torch.randperm(pages, generator=gen, device=DEV).int()
    table = torch.full((B, table_len), -1, device=DEV, dtype=torch.int32)
    mine = torch.arange(table_len, device=DEV) < held[:, None]
    table[mine] = order[:used]
    stack = torch.full((pages,), -1, device=DEV, dtype=torch.int32)
    stack[:free] = order[used:used + free]
    return {"case": dict(case), "lengths": lengths, "new": new, "none": torch.zeros_like(new), "pages": pages,
            "table": table, "held": held, "free_pages": stack, "free_count": torch.tensor([free], device=DEV).int(),
            "N": N}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] == "plan":
        return _prepare_plan(case, gen)
    B, rows, G, pt = case["B"], case["rows"], case["G"], case["page_tokens"]
    Hq, N = G * case["hq"], case["B"] * case["rows"]
    starts = _starts(case, gen)
    table_len = -(-(case["hi"] + rows) // pt)
    pages = B * table_len
    s = {"case": dict(case), "starts": starts,
         "table": torch.randperm(pages, generator=gen, device=DEV).int().view(B, table_len).contiguous(),
         "row_seq": torch.arange(B, device=DEV).repeat_interleave(rows).int(),
         "row_pos": (starts[:, None] + torch.arange(rows, device=DEV)).reshape(-1).int()}
    if case["apart"]:            # q where one projection left it, beside k and v
        s["q"] = (_normal(gen, N, Hq + 2 * G, D) * 1.5)[:, :Hq]
    else:
        s["q"] = _normal(gen, N, Hq, D) * 1.5
    s["k"], s["v"] = (_normal(gen, pages, G, pt, D) for _ in range(2))
    s["gate"] = _normal(gen, N, Hq) if case["gate"] else None
    s["out"] = torch.zeros((N, Hq, D), device=DEV, dtype=torch.bfloat16)
    if case["op"] == "sparse":
        s["sel_ids"], s["sel_count"] = _picks(gen, starts, case, G)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"paged": _own_paged, "sparse": _own_sparse, "plan": _own_plan}[op](s)
    return {"paged": _plain_paged, "sparse": _plain_sparse, "plan": _plain_plan}[op](s)


def _handles(s):
    """The framework's geometry, cache handle and workspace, made once for a state, as a program keeps them."""
    if "cache" not in s:
        import block_sparse_attention_step5_gb300 as s5

        c = s["case"]
        s["s5"] = s5
        s["geom"] = s5.Geometry.step5(num_q_heads=c["G"] * c["hq"], num_kv_groups=c["G"], idx_heads=c["G"] * 4,
                                      top_k=c.get("top_k", 512))
        s["cache"] = s5.PagedCache(s["k"], s["v"], s["table"])
        s["ws"] = s5.PagedWorkspace.create(s["geom"])
    return s["s5"], s["geom"], s["cache"], s["ws"]


def _own_paged(s):
    s5, geom, cache, ws = _handles(s)
    s5.step5_paged_attn(geom, s["q"], cache, s["row_seq"], s["row_pos"], s["out"], ws, window=s["case"]["window"],
                        gate=s["gate"])
    return s["out"]


def _own_sparse(s):
    s5, geom, cache, ws = _handles(s)
    s5.step5_sparse_attn_paged(geom, s["q"], cache, s["row_seq"], s["row_pos"], s["sel_ids"], s["sel_count"], s["out"],
                               ws, gate=s["gate"])
    return s["out"]


def _own_plan(s):
    """The step's plan, and the roll-back of its tokens, which gives the pages back."""
    if "slots" not in s:
        import block_sparse_attention_step5_gb300 as s5

        s["s5"] = s5
        s["slots"] = s5.PagedTable(s["table"], s["held"], s["free_pages"], s["free_count"], s["case"]["page_tokens"])
        s["grown"], s["back"] = (s5.PagedRows.create(s["case"]["B"], s["N"]) for _ in range(2))
    s5 = s["s5"]
    s5.step5_paged_plan(s["slots"], s["grown"], s["lengths"], s["new"])
    s5.step5_paged_plan(s["slots"], s["back"], s["lengths"], s["none"])
    return _plan_outputs(s, *({n: getattr(r, n) for n in _ROWS} for r in (s["grown"], s["back"])))


_ROWS = ("row_seq", "row_pos", "row_start", "ends", "granted", "region_begin", "region_end")


def _plan_outputs(s, grown, back):
    out = {"grown_" + n: grown[n] for n in _ROWS}
    out.update({"back_" + n: back[n] for n in _ROWS})
    out.update(table=s["table"], held=s["held"], free_pages=s["free_pages"], free_count=s["free_count"])
    return out


# ---------------------------------------------------------------- plain forms (32 bits)

def _plain_values(s, pool, seq, tok):
    """fp32 values of tokens tok [..., L] of sequences seq [..., 1]: [..., G, L, 128]."""
    pt = s["case"]["page_tokens"]
    return pool[s["table"].long()[seq, tok // pt], :, tok % pt].float().transpose(-3, -2)


def _plain_softmax_av(q, k, v, seen):
    """q [..., G, R, 128] against k, v [..., G, L, 128], seen [..., G, R, L]: [..., G, R, 128]."""
    x = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D))
    x.masked_fill_(~seen, -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    return (x @ v) / x.sum(-1, keepdim=True)


def _plain_store(s, n, o):
    """o [rows][Hq][128] through the gate into rows n .. of the output."""
    m = o.shape[0]
    if s["gate"] is not None:
        o = o / (1.0 + (-s["gate"][n:n + m].float()).exp())[..., None]
    s["out"][n:n + m] = o.bfloat16()


def _plain_paged(s):
    c = s["case"]
    B, rows, G, hq, W = c["B"], c["rows"], c["G"], c["hq"], c["window"]
    first = s["starts"]
    lo = (first - W + 1).clamp(min=0) if W else torch.zeros_like(first)
    L = c["hi"] + rows if not W else min(c["hi"] + rows, rows + W - 1)
    tok = lo[:, None] + torch.arange(L, device=DEV)               # [B][L]
    at = tok.clamp(max=s["table"].shape[1] * c["page_tokens"] - 1)
    seq = torch.arange(B, device=DEV)[:, None]
    k, v = (_plain_values(s, s[x], seq, at) for x in "kv")        # [B][G][L][128]
    q = s["q"].float().view(B, rows, G, hq, D)
    out = torch.empty((B, rows, G * hq, D), device=DEV)
    step = max(1, (1 << 32) // (B * G * hq * L))                  # rows of a sequence whose scores fit in 16 GB
    for j in range(0, rows, step):
        m = min(step, rows - j)
        pos = first[:, None] + torch.arange(j, j + m, device=DEV)  # [B][m]
        seen = tok[:, None, :] <= pos[:, :, None]
        if W:
            seen &= tok[:, None, :] > pos[:, :, None] - W
        seen = seen[:, None, :, None, :].expand(-1, -1, -1, hq, -1).reshape(B, 1, m * hq, L)
        o = _plain_softmax_av(q[:, j:j + m].transpose(1, 2).reshape(B, G, m * hq, D), k, v, seen)
        out[:, j:j + m] = o.view(B, G, m, hq, D).transpose(1, 2).reshape(B, m, G * hq, D)
    _plain_store(s, 0, out.view(B * rows, G * hq, D))
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
        k, v = (s[x][page, g, slot].float() for x in "kv")
        q = s["q"][n:n + step].float().reshape(m, G, hq, D)
        _plain_store(s, n, _plain_softmax_av(q, k, v, seen[:, :, None, :]).reshape(m, G * hq, D))
    return s["out"]


def _before(x):
    """Sums of the elements before each one, and of all."""
    x = x.long()
    inc = x.cumsum(0)
    return inc - x, inc[-1]


def _plain_step(s, new):
    """Pages of sequences that got shorter go onto the stack of free ones, in the sequences' order; the
    pages that the others need are its top ones, handed out from the lowest on in the sequences' order,
    up to the first sequence whose need is not met; then the rows of what was granted."""
    c = s["case"]
    B, pt, N = c["B"], c["page_tokens"], s["N"]
    lengths, held = s["lengths"].long(), s["held"].long()
    start, _ = _before(new)
    fits = start + new.long() <= N
    want = (lengths + new.long() + pt - 1) // pt
    less = torch.where(fits, (held - want).clamp(min=0), 0)
    need = torch.where(fits, (want - held).clamp(min=0), 0)
    freed_before, freed = _before(less)
    have = s["free_count"].long()[0] + freed
    need_before, _ = _before(need)
    ok = fits & ((need == 0) | (need_before + need <= have))
    need = torch.where(ok, need, 0)
    need_before, taken = _before(need)
    entry = torch.arange(s["table"].shape[1], device=DEV)
    # onto the stack
    gone = (entry >= want[:, None]) & (entry < held[:, None]) & (less > 0)[:, None]
    to = torch.where(gone, s["free_count"].long()[0] + freed_before[:, None] + entry - want[:, None], s["pages"])
    stack = torch.cat((s["free_pages"], s["free_pages"][:1]))
    stack.scatter_(0, to.reshape(-1), s["table"].reshape(-1))
    # off it
    came = (entry >= held[:, None]) & (entry < (held + need)[:, None])
    at = torch.where(came, have - taken + need_before[:, None] + entry - held[:, None], 0)
    s["table"].copy_(torch.where(came, stack[at], s["table"]))
    s["free_pages"].copy_(stack[:-1])
    s["free_count"].copy_((have - taken).int())
    s["held"].copy_((held + need - less).int())
    # the rows
    granted = torch.where(ok, new.long(), 0)
    n = torch.arange(N, device=DEV)
    b = (torch.searchsorted(start, n, right=True) - 1).clamp(min=0)
    real = ok[b] & (n < (start + new.long())[b])
    ends = lengths + granted
    full = torch.cat((start, (start + new.long())[-1:])).clamp(max=N)
    return {"row_seq": torch.where(real, b, -1).int(), "row_pos": torch.where(real, lengths[b] + n - start[b], -1).int(),
            "row_start": full.int(), "ends": ends.int(), "granted": granted.int(), "region_begin": (lengths // RT).int(),
            "region_end": (ends // RT).int()}


def _plain_plan(s):
    grown = _plain_step(s, s["new"])
    return _plan_outputs(s, grown, _plain_step(s, s["none"]))


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _exact_values(s, name, b, g, tok):
    pt = s["case"]["page_tokens"]
    return s[name][s["table"][b].long()[tok // pt], g, tok % pt].double()


def _exact_gated(s, out):
    return out if s["gate"] is None else out * torch.sigmoid(s["gate"].double())[..., None]


def _exact_paged(s):
    c = s["case"]
    rows, G, hq, W = c["rows"], c["G"], c["hq"], c["window"]
    out = torch.zeros((c["B"] * rows, G, hq, D), device=DEV, dtype=torch.float64)
    qs = s["q"].reshape(-1, G, hq, D)
    for b, start in enumerate(s["starts"].tolist()):
        lo = max(0, start - W + 1) if W else 0
        tok = torch.arange(lo, start + rows, device=DEV)
        for g in range(G):
            k, v = (_exact_values(s, x, b, g, tok) for x in "kv")
            q = qs[b * rows:(b + 1) * rows, g].double()
            for j in range(0, rows, 256):
                pos = torch.arange(start + j, start + min(rows, j + 256), device=DEV)[:, None, None]
                x = torch.einsum("rhd,ld->rhl", q[j:j + 256], k) / math.sqrt(D)
                hide = (tok > pos) | (tok <= pos - W if W else False)
                x = torch.softmax(x.masked_fill(hide, -math.inf), -1)
                out[b * rows + j:b * rows + j + pos.shape[0], g] = torch.einsum("rhl,ld->rhd", x, v)
    return _exact_gated(s, out.view(-1, G * hq, D))


def _exact_sparse(s):
    c = s["case"]
    G, hq, N = c["G"], c["hq"], c["B"] * c["rows"]
    out = torch.zeros((N, G, hq, D), device=DEV, dtype=torch.float64)
    pos, seq, count = s["row_pos"].tolist(), s["row_seq"].tolist(), s["sel_count"].tolist()
    q = s["q"].reshape(N, G, hq, D).double()
    eight = torch.arange(RT, device=DEV)
    for n in range(N):
        mine = torch.arange(pos[n] // RT * RT, pos[n] + 1, device=DEV)
        for g in range(G):
            tok = torch.cat(((s["sel_ids"][n, g, :count[n][g]].long()[:, None] * RT + eight).reshape(-1), mine))
            k, v = (_exact_values(s, x, seq[n], g, tok) for x in "kv")
            out[n, g] = torch.softmax(q[n, g] @ k.T / math.sqrt(D), dim=-1) @ v
    return _exact_gated(s, out.view(N, G * hq, D))


def _exact_step(s, host, new):
    """One sequence after another, on lists."""
    c, N = s["case"], s["N"]
    B, pt = c["B"], c["page_tokens"]
    table, held, stack, lengths = host["table"], host["held"], host["stack"], host["lengths"]
    at = np.concatenate(([0], np.cumsum(new)))
    want = [-(-(lengths[b] + new[b]) // pt) for b in range(B)]
    for b in range(B):                                            # the pages given back
        if at[b + 1] <= N and want[b] < held[b]:
            stack += table[b][want[b]:held[b]]
            held[b] = want[b]
    granted, takes, left, short = [0] * B, [], len(stack), False
    for b in range(B):
        need = max(0, want[b] - held[b]) if at[b + 1] <= N else 0
        short = short or need > left
        if at[b + 1] <= N and (need == 0 or not short):
            granted[b] = new[b]
            takes.append((b, need))
            left -= need
    got = stack[left:]
    del stack[left:]
    for b, need in takes:
        for _ in range(need):
            table[b][held[b]] = got.pop(0)
            held[b] += 1
    seq, pos = [-1] * N, [-1] * N
    for b in range(B):
        for i in range(granted[b]):
            seq[at[b] + i], pos[at[b] + i] = b, lengths[b] + i
    ends = [lengths[b] + granted[b] for b in range(B)]
    return {"row_seq": seq, "row_pos": pos, "row_start": [min(int(a), N) for a in at], "ends": ends, "granted": granted,
            "region_begin": [n // RT for n in lengths], "region_end": [n // RT for n in ends]}


def _exact_plan(s):
    count = int(s["free_count"])
    host = {"table": s["table"].tolist(), "held": s["held"].tolist(), "lengths": s["lengths"].tolist(),
            "stack": s["free_pages"][:count].tolist()}
    above = s["free_pages"].tolist()[count:]                       # (what lies above the stack's top stays)
    grown = _exact_step(s, host, s["new"].tolist())
    back = _exact_step(s, host, s["none"].tolist())
    stack = host["stack"] + above
    as_int = lambda x: torch.tensor(x, device=DEV, dtype=torch.int32)
    out = {"grown_" + n: as_int(grown[n]) for n in _ROWS}
    out.update({"back_" + n: as_int(back[n]) for n in _ROWS})
    out.update(table=as_int(host["table"]), held=as_int(host["held"]), free_pages=as_int(stack),
               free_count=as_int([len(host["stack"])]))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"paged": _exact_paged, "sparse": _exact_sparse, "plan": _exact_plan}[case["op"]](s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "plan":
        # both steps: lengths, new tokens and held pages read, held, ends, granted, regions and row starts written,
        # the rows; pages moved are a few of the table's entries
        B, N = case["B"], case["N"]
        moved = B * case["most"] / 2 / case["page_tokens"]
        return {"bytes": 2 * (4 * 9 * B + 8 * N + 8 * moved), "flops": 2 * (8 * B + 2 * N)}
    B, rows, G, hq = case["B"], case["rows"], case["G"], case["hq"]
    N, Hq = B * rows, G * case["hq"]
    mid = (case["lo"] + case["hi"]) / 2
    qo = 2 * N * Hq * D * 2
    per_token = G * 2 * D * 2
    if case["op"] == "paged":
        W = case["window"]
        ends = [mid + j + 1 for j in range(rows)]
        keys = sum(min(e, W) if W else e for e in ends)
        span = mid + rows if not W else min(mid + rows, rows + W - 1)
        return {"bytes": qo + B * span * per_token, "flops": 4 * D * Hq * B * keys}
    picked = min(case["top_k"], mid / RT) * RT + RT / 2
    touched = min(rows * picked, mid + rows)
    return {"bytes": qo + B * touched * per_token + N * G * 4 * min(case["top_k"], mid / RT), "flops": 4 * D * Hq * N * picked}
