"""Attention over bf16 pages and the step's plan from their definitions, on the CPU, for the tests:
nothing here is shared with the library."""
import numpy as np
import torch

import paged_reference as R


def keys_of(p, window, ids, count):
    """The tokens that a row at position p sees."""
    if ids is None:
        return np.arange(max(0, p - window + 1) if window else 0, p + 1)
    own = p // 8
    picked = ids[:count].long().numpy()
    return np.concatenate([(picked[:, None] * 8 + np.arange(8)).reshape(-1), np.arange(own * 8, p + 1)])


def attend(q, k, v, table, row_seq, row_pos, scale, window=0, ids=None, counts=None, gate=None, bad_pages=()):
    """64-bit attention: q [N][Hq][128], pools [P][G][pt][128].  Returns (out, mass) with mass
    sum_t w_t |v_t| (tolerance()).  Tokens on table entries in bad_pages are no keys."""
    N, Hq, _ = q.shape
    G, pt = k.shape[1], k.shape[2]
    hq = Hq // G
    out = torch.zeros(q.shape, dtype=torch.float64)
    mass = torch.zeros_like(out)
    for n in range(N):
        b, p = int(row_seq[n]), int(row_pos[n])
        if b < 0:
            continue
        for g in range(G):
            toks = keys_of(p, window, None if ids is None else ids[n, g], 0 if ids is None else int(counts[n, g]))
            at = [R.place(table, b, int(t), pt) for t in toks]
            at = [a for a in at if a[0] not in bad_pages]
            if not at:
                continue
            page, slot = (torch.tensor([a[i] for a in at]) for i in range(2))
            kk, vv = k[page, g, slot].double(), v[page, g, slot].double()
            h = slice(g * hq, (g + 1) * hq)
            w = torch.softmax(q[n, h].double() @ kk.T * scale, -1)
            out[n, h], mass[n, h] = w @ vv, w @ vv.abs()
    if gate is not None:
        f = torch.sigmoid(gate.double())[..., None]
        out, mass = out * f, mass * f
    return out, mass


def shares(N, hq, B):
    """Whether rows of a sequence share its keys' tiles (the rule of the header)."""
    return N * hq >= 128 * B


def tolerance(out, mass, shared):
    """One bf16 rounding of the result is off by at most 2^-8 of it.  Before it, a weight that meets V
    is off by its own rounding, half a step of bf16, 2^-8 of it, where rows share tiles, and 2^-16 where
    it has two parts (the second half a step of what the first leaves); and by 2^-11 for the score and
    the sums: products of bf16 values are exact in fp32, an fp32 sum of 128 of them is off by less than
    2^-17 of their magnitudes' sum, below 2^5 in these tests (in units of the exponent, base 2), the
    exponential by 2^-22, the sums of weights by less than 2^-12."""
    return 2.0 ** -8 * out.abs() + ((2.0 ** -8 if shared else 2.0 ** -16) + 2.0 ** -11) * mass + 1e-30


def off(got, out, mass, shared) -> float:
    """The largest error in units of the tolerance."""
    return float(((got.double().cpu() - out).abs() / tolerance(out, mass, shared)).max())


def plan(table, held, free, num_pages, page_tokens, N, lengths, new):
    """One sequence after another on lists; table, held and free (the stack) are changed in place.  Returns
    (outputs, whether anything was out of range); see the header for the rule."""
    B, table_len = len(lengths), len(table[0])
    start, rows = [0], [max(0, n) for n in new]
    for n in rows:
        start.append(start[-1] + n)
    good, bad = [], False
    for b in range(B):
        ok = (lengths[b] >= 0 and new[b] >= 0 and lengths[b] + new[b] <= table_len * page_tokens
              and 0 <= held[b] <= table_len and start[b + 1] <= N)
        good.append(ok)
        bad = bad or not ok
    want = [-(-(lengths[b] + new[b]) // page_tokens) if good[b] else held[b] for b in range(B)]
    for b in range(B):
        if want[b] < held[b]:
            given = table[b][want[b]:held[b]]
            bad = bad or any(not 0 <= x < num_pages for x in given)
            for x in given:
                if len(free) < num_pages:
                    free.append(x)
                else:
                    bad = True
            held[b] = want[b]
    left, takes, granted, short = len(free), [], [0] * B, False
    for b in range(B):
        need = want[b] - held[b]
        if need > left:
            short = True
        if good[b] and (need <= 0 or not short):
            granted[b] = new[b]
            takes.append((b, need))
            left -= need
    taken = free[left:]
    del free[left:]
    for b, need in takes:
        for _ in range(need):
            x = taken.pop(0)
            bad = bad or not 0 <= x < num_pages
            table[b][held[b]] = x
            held[b] += 1
    seq, pos = [-1] * N, [-1] * N
    for b in range(B):
        for i in range(granted[b]):
            seq[start[b] + i], pos[start[b] + i] = b, lengths[b] + i
    ends = [lengths[b] + granted[b] for b in range(B)]
    return {"row_seq": seq, "row_pos": pos, "row_start": [min(x, N) for x in start], "ends": ends, "granted": granted,
            "region_begin": [max(x, 0) // 8 for x in lengths], "region_end": [max(x, 0) // 8 for x in ends]}, bad
