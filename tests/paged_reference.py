"""The paged KV cache's operators from their definitions, in 64 bits on the CPU, for the
tests: nothing here is shared with the library."""
import math

import numpy as np
import torch


def bf16_near(x: torch.Tensor) -> torch.Tensor:
    """64-bit values rounded once to bf16's 8 significant bits (as 64-bit values)."""
    m, e = torch.frexp(x)
    ulp = torch.exp2((e - 8).clamp(min=-133).double())
    return torch.round(x / ulp) * ulp


def e4m3_near(x: torch.Tensor) -> torch.Tensor:
    """64-bit values rounded once to e4m3 (as 64-bit values): 4 significant bits, no step
    finer than 2^-9, saturating at 448, NaN kept."""
    m, e = torch.frexp(x)
    ulp = torch.exp2((e - 4).clamp(min=-9).double())
    return (torch.round(x / ulp) * ulp).clamp(-448.0, 448.0)


def rotate(x: torch.Tensor, cos, sin, pos) -> torch.Tensor:
    """NEOX rotation of x [N][H][128] (64-bit) at positions pos, rounded to bf16."""
    if cos is None:
        return x
    h = cos.shape[1]
    c, s = cos.double()[pos][:, None], sin.double()[pos][:, None]
    a, b = x[..., :h], x[..., h:2 * h]
    return torch.cat((bf16_near(a * c - b * s), bf16_near(b * c + a * s), x[..., 2 * h:]), -1)


def place(table, b, pos, page_tokens):
    """(page, slot) of a token, or None where the table has no page for it."""
    i = pos // page_tokens
    if table is None:
        return (b, pos) if i == 0 else None
    if i >= table.shape[1]:
        return None
    return int(table[b, i]), pos % page_tokens


def needed_scale(amax: float) -> float:
    """The smallest power of two s >= 2^-126 with amax <= 448 s."""
    s = 2.0 ** -126
    while 448.0 * s < amax and s < 2.0 ** 120:
        s *= 2.0
    return s


def append_e4m3(x, codes, scales, table, row_seq, row_pos):
    """Appends rows x [N][G][128] (64-bit values) one region at a time.  codes: 64-bit values of the codes
    [P][G][page_tokens][128], scales [P][G][page_tokens / 8], both changed in place."""
    pt = codes.shape[2]
    n = 0
    while n < len(row_seq):
        b, p = int(row_seq[n]), int(row_pos[n])
        m = 1
        while (n + m < len(row_seq) and row_seq[n + m] == b and row_pos[n + m] == p + m and (p + m) % 8):
            m += 1
        if b >= 0:
            page, slot = place(table, b, p, pt)
            r, t0 = slot // 8, slot % 8
            for g in range(codes.shape[1]):
                new = x[n:n + m, g]
                mag = new.abs()[~torch.isnan(new)].clamp(max=torch.finfo(torch.bfloat16).max)
                s = needed_scale(float(mag.max()) if mag.numel() else 0.0)
                held = float(scales[page, g, r])
                if t0 and s < held:
                    s = held
                if t0 and s > held:
                    codes[page, g, 8 * r:8 * r + t0] = e4m3_near(codes[page, g, 8 * r:8 * r + t0] * (held / s))
                codes[page, g, slot:slot + m] = e4m3_near(new / s)
                scales[page, g, r] = s
        n += m


def decode(codes_u8: torch.Tensor) -> torch.Tensor:
    return codes_u8.cpu().view(torch.float8_e4m3fn).double()


def attend(q, k, v, ks, vs, table, row_seq, row_pos, scale, window=0, ids=None, counts=None, gate=None):
    """64-bit attention: q [N][Hq][128], codes' values k, v [P][G][pt][128], scales.  Returns
    (out, terms): what the errors of the weights act on (terms())."""
    N, Hq, D = q.shape
    G, pt = k.shape[1], k.shape[2]
    hq = Hq // G
    out = torch.zeros((N, Hq, D), dtype=torch.float64)
    mass = torch.zeros_like(out)
    for n in range(N):
        b, p = int(row_seq[n]), int(row_pos[n])
        if b < 0:
            continue
        for g in range(G):
            if ids is None:
                toks = np.arange(max(0, p - window + 1) if window else 0, p + 1)
            else:
                picked = ids[n, g, :int(counts[n, g])].long().numpy()
                own = p // 8
                toks = np.concatenate([(picked[:, None] * 8 + np.arange(8)).reshape(-1), np.arange(own * 8, p + 1)])
            at = [place(table, b, int(t), pt) for t in toks]
            page = torch.tensor([a[0] for a in at])
            slot = torch.tensor([a[1] for a in at])
            kk = k[page, g, slot] * ks[page, g, slot // 8].double()[:, None]
            vv = v[page, g, slot] * vs[page, g, slot // 8].double()[:, None]
            w = torch.softmax(q[n, g * hq:(g + 1) * hq].double() @ kk.T * scale, -1)
            out[n, g * hq:(g + 1) * hq] = w @ vv
            mass[n, g * hq:(g + 1) * hq] = terms(w, v[page, g, slot], vs[page, g, slot // 8].double())
    if gate is not None:
        f = torch.sigmoid(gate.double())[..., None]
        out, mass = out * f, mass * f
    return out, mass


def terms(w, codes, scales):
    """sum_t w_t |v_t| + 2^-13 max scale * sum_t |code_t| for weights w [heads][L], codes [L][128], scales [L]."""
    return w @ (codes.abs() * scales[:, None]) + 2.0 ** -13 * float(scales.max()) * codes.abs().sum(0)


def tolerance(out, mass):
    """One bf16 rounding of the result is off by at most 2^-8 of it.  Before it, a weight is
    off by at most 3 * 2^-12 of itself: 2^-11 for its rounding to the 11 bits (f16) that meet V, and
    2^-12 for its score (128 products and the exponential in fp32: scores of the tests stay below 2^6,
    an fp32 sum of 128 terms is off by less than 2^-17 of the terms' magnitudes, which are below 2^5)
    and the sums.  Small weights have a floor: they are held, times vscale over a power of two above
    every vscale and times 2^5, in three e4m3 parts 2^5 apart, the last in steps of 2^-9 at the finest,
    so a weight (against the row's largest) times its vscale is off by up to half a step,
    2^-10 * 2^-10 * 2^-5 = 2^-25 of that power of two, which is at most twice the largest vscale:
    sum_t 2^-24 max scale |code_t| = 2^-11 of the second of terms(), below 3 * 2^-12 of it."""
    return 2.0 ** -8 * out.abs() + 3 * 2.0 ** -12 * mass + 1e-30


def off(got, out, mass) -> float:
    """The largest error in units of the tolerance."""
    return float(((got.double().cpu() - out).abs() / tolerance(out, mass)).max())
