"""The paged KV cache on the GPU against its definitions in 64 bits: appending with rotation
(bf16 and e4m3), attention over the e4m3 pages, over picked regions, and a run of them together."""
import numpy as np
import pytest
import torch

import paged_reference as R
import synthetic as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def s5():
    import block_sparse_attention_step5_gb300 as s5
    s5.build()
    s5.load()
    return s5


def geometry(s5, G=4, hq=8, **over):
    return s5.Geometry.step5(num_q_heads=G * hq, num_kv_groups=G, idx_heads=4 * G, **over)


def normal(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).bfloat16()


def tables(gen, B, length, spare=3):
    """A block table over a pool of B * length + spare pages in a random order."""
    return torch.randperm(B * length + spare, generator=gen)[:B * length].int().view(B, length).contiguous()


def rows_of(*runs):
    """(row_seq, row_pos) of runs (sequence, first position, rows)."""
    seq = [b for b, p, n in runs for _ in range(n)]
    pos = [p + i for b, p, n in runs for i in range(n)]
    return torch.tensor(seq, dtype=torch.int32), torch.tensor(pos, dtype=torch.int32)


def random_pool(gen, P, G, pt, lo=-9, hi=-4):
    codes = (torch.randn((P, G, pt, 128), generator=gen) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, torch.exp2(torch.randint(lo, hi, (P, G, pt // 8), generator=gen).float())


def dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


def status(s5):
    torch.cuda.synchronize()
    return s5.step5_device_status()


# ------------------------------------------------------------------------------ append

RUNS = {
    "one": [(0, 5, 1)],
    "first": [(0, 0, 1)],
    "last_of_region": [(1, 15, 1)],
    "decode": [(0, 5, 1), (2, 8, 1), (1, 31, 1)],
    "chunk": [(0, 3, 27)],
    "chunks": [(1, 0, 8), (0, 7, 2), (-1, 0, 3), (2, 12, 20)],
    "long": [(0, 1, 200)],
}


@pytest.mark.parametrize("runs", list(RUNS))
@pytest.mark.parametrize("G, hq, pt, rot", [(4, 8, 16, 128), (1, 4, 8, 32), (8, 16, 24, 96), (2, 8, 64, 0)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_append(s5, runs, G, hq, pt, rot, e4m3):
    gen = torch.Generator().manual_seed(len(runs) * 100 + rot)
    geom = geometry(s5, G, hq)
    seq, pos = rows_of(*RUNS[runs])
    N, B, length = len(seq), 3, -(-208 // pt)
    table = tables(gen, B, length)
    P = B * length + 3
    # one projection's rows, magnitudes over many binades
    qkv = (torch.randn((N, G * (hq + 2), 128), generator=gen) *
           torch.exp2(torch.randint(-20, 12, (N, G * (hq + 2), 1), generator=gen).float())).bfloat16()
    q, k, v = qkv.split((G * hq, G, G), dim=1)
    cos, sin = S.rope_tables(length * pt, rot) if rot else (None, None)
    dq, dseq, dpos, dtab, dcos, dsin = dev(qkv, seq, pos, table, cos, sin)
    gq, gk, gv = dq.split((G * hq, G, G), dim=1)
    q_out = torch.full((N, G * hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    at = pos.long().clamp(min=0)
    want_q = R.rotate(q.double(), cos, sin, at)
    want = {"k": R.rotate(k.double(), cos, sin, at), "v": v.double()}
    real = (seq >= 0)
    if e4m3:
        pools = [random_pool(gen, P, G, pt, -12, 4) for _ in "kv"]
        (kc, ks), (vc, vs) = [tuple(x.cuda() for x in pl) for pl in pools]
        s5.step5_kv_append_e4m3(geom, gk, gv, s5.PagedCache(kc, vc, dtab, ks, vs), dseq, dpos, dcos, dsin, q=gq,
                                q_out=q_out)
    else:
        pools = [(normal(gen, P, G, pt, 128), None) for _ in "kv"]
        kc, vc = (pl[0].cuda() for pl in pools)
        s5.step5_kv_append(geom, gk, gv, s5.PagedCache(kc, vc, dtab), dseq, dpos, dcos, dsin, q=gq, q_out=q_out)
    assert status(s5) == 0
    assert torch.equal(q_out.cpu().double()[real], want_q[real])
    assert bool((q_out.cpu()[~real] == 7.0).all())
    for name, got, got_s, (base, base_s) in (("k", kc, ks if e4m3 else None, pools[0]),
                                             ("v", vc, vs if e4m3 else None, pools[1])):
        if e4m3:
            codes, scales = R.decode(base), base_s.double()
            R.append_e4m3(want[name], codes, scales, table, seq, pos)
            assert torch.equal(got_s.cpu().double(), scales), name
            assert torch.equal(R.decode(got), codes), name
        else:
            pool = base.double()
            for n in range(N):
                if seq[n] >= 0:
                    page, slot = R.place(table, int(seq[n]), int(pos[n]), pt)
                    pool[page, :, slot] = want[name][n]
            assert torch.equal(got.cpu().double(), pool), name


def test_append_e4m3_token_by_token(s5):
    """Appending tokens one at a time, the scale growing inside regions, equals the
    definition step by step; and a rolled-back position written again keeps the scale held."""
    gen = torch.Generator().manual_seed(3)
    geom = geometry(s5, 2, 4)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    kc, vc = (torch.zeros((3, 2, 8, 128), dtype=torch.uint8) for _ in "kv")
    ks, vs = (torch.full((3, 2, 1), float("nan")) for _ in "kv")
    gpu = [t.cuda() for t in (kc, vc, table, ks, vs)]
    cache = s5.PagedCache(*gpu)
    ref = [[R.decode(kc), ks.double()], [R.decode(vc), vs.double()]]
    for p in list(range(20)) + [13, 14, 16, 17]:
        x = normal(gen, 2, 1, 2, 128, scale=2.0 ** (p % 5 * 3 - 6))
        seq, pos = rows_of((0, p, 1))
        for i in range(2):
            R.append_e4m3(x[i].double(), *ref[i], table, seq, pos)
        s5.step5_kv_append_e4m3(geom, *dev(x[0], x[1]), cache, *dev(seq, pos))
        for i, (c, s) in enumerate(((gpu[0], gpu[3]), (gpu[1], gpu[4]))):
            assert torch.equal(R.decode(c), ref[i][0]), p
            assert torch.equal(s.cpu().double().nan_to_num(-1.0), ref[i][1].nan_to_num(-1.0)), p
    assert status(s5) == 0


def test_append_e4m3_special_values(s5):
    """Zero regions, the largest and smallest bf16 values, infinities (saturate) and NaN (kept; scale
    from the rest)."""
    geom = geometry(s5, 1, 4)
    x = torch.ones((40, 1, 128), dtype=torch.bfloat16)
    x[0:8] = 0.0
    x[8, 0, 3] = torch.finfo(torch.bfloat16).max
    x[16:24] = 2.0 ** -133
    x[24, 0, 5], x[25, 0, 6] = float("inf"), -float("inf")
    x[32:40] = 3.0
    x[33, 0, 7] = float("nan")
    seq, pos = rows_of((0, 0, 40))
    table = torch.zeros((1, 1), dtype=torch.int32)
    kc, vc, ks, vs = (torch.zeros((1, 1, 40, 128), dtype=torch.uint8), torch.zeros((1, 1, 40, 128), dtype=torch.uint8),
                      torch.zeros((1, 1, 5)), torch.zeros((1, 1, 5)))
    codes, scales = R.decode(kc), ks.double()
    R.append_e4m3(x.double(), codes, scales, table, seq, pos)
    gk, gv, gt, gks, gvs = dev(kc, vc, table, ks, vs)
    s5.step5_kv_append_e4m3(geom, *dev(x, x), s5.PagedCache(gk, gv, gt, gks, gvs), *dev(seq, pos))
    assert status(s5) == 0
    assert torch.equal(gks.cpu().double(), scales) and torch.equal(gvs, gks)
    assert torch.equal(torch.isnan(R.decode(gk)), torch.isnan(codes))
    assert torch.equal(R.decode(gk).nan_to_num(0.0), codes.nan_to_num(0.0))


def test_append_e4m3_beside_scales_of_another_kind(s5):
    """Scales held that are no powers of two: the new values divided by one, and the codes held multiplied by it,
    are rounded once, ties and what lies next to them among them."""
    ties = (17 + 2 * torch.arange(8)).double() / 16
    geom, G = geometry(s5, 8, 4), 8
    gen = torch.Generator().manual_seed(77)
    table = torch.zeros((1, 1), dtype=torch.int32)
    seq, pos = rows_of((0, 4, 4))
    for grows in (False, True):
        held = torch.empty(G)
        x = normal(gen, 4, G, 128, scale=1.0)
        codes = (torch.randn((1, G, 8, 128), generator=gen) * 8).to(torch.float8_e4m3fn)
        for g in range(G):
            if grows:  # held * code is next to a tie for codes of 9 / 8, 11 / 8, ...
                code = torch.tensor([9, 11, 13, 15])[g % 4].double() / 8
                held[g] = (ties[g] / code / 32).float()
                codes[0, g, :4, :64] = code.to(torch.float8_e4m3fn)
                x[0, g, 0] = 96.0  # (a scale of 1 / 4)
            else:
                held[g] = 1.75 * 2.0 ** -g if g < 4 else (2.0 ** -g / ties[g]).float()
                x[:2, g, :8] = (held[g].double() * (ties if g < 4 else ties[g])).bfloat16()
                x[:, g] = x[:, g].clamp(-float(held[g]) * 256, float(held[g]) * 256)
        want, scales = codes.double(), held.double().view(1, G, 1).clone()
        R.append_e4m3(x.double(), want, scales, table, seq, pos)
        k, v = (codes.view(torch.uint8).clone().cuda() for _ in "kv")
        ks, vs = (held.view(1, G, 1).clone().cuda() for _ in "kv")
        s5.step5_kv_append_e4m3(geom, *dev(x, x), s5.PagedCache(k, v, table.cuda(), ks, vs), *dev(seq, pos))
        assert status(s5) == 0
        for c, sc in ((k, ks), (v, vs)):
            assert torch.equal(sc.cpu().double(), scales)
            assert torch.equal(R.decode(c), want)


def test_append_refuses_rows_on_the_device(s5):
    """Rows out of range, out of order or without a page write nothing and raise the range flag."""
    geom = geometry(s5, 2, 4)
    table = torch.tensor([[1, -1], [0, 99]], dtype=torch.int32)
    x = torch.ones((1, 2, 128), dtype=torch.bfloat16).cuda()
    for b, p in ((0, 16), (0, -1), (2, 0), (-2, 0), (0, 8), (1, 15)):
        kc, vc = (torch.full((2, 2, 8, 128), 9, dtype=torch.uint8, device="cuda") for _ in "kv")
        ks, vs = (torch.full((2, 2, 1), 3.0, device="cuda") for _ in "kv")
        seq, pos = dev(*rows_of((b, p, 1)))
        s5.step5_kv_append_e4m3(geom, x, x, s5.PagedCache(kc, vc, table.cuda(), ks, vs), seq, pos)
        assert status(s5) == s5.DEV_RANGE, (b, p)
        assert bool((kc == 9).all()) and bool((vc == 9).all()) and bool((ks == 3).all()) and bool((vs == 3).all())
        kb, vb = (torch.full((2, 2, 8, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        s5.step5_kv_append(geom, x, x, s5.PagedCache(kb, vb, table.cuda()), seq, pos)
        assert status(s5) == s5.DEV_RANGE, (b, p)
        assert bool((kb == 9).all()) and bool((vb == 9).all())
    # a rope table shorter than the pages
    cos, sin = dev(*S.rope_tables(4, 32))
    seq, pos = dev(*rows_of((0, 4, 1)))
    s5.step5_kv_append(geom, x, x, s5.PagedCache(kb, vb, table.cuda()), seq, pos, cos, sin)
    assert status(s5) == s5.DEV_RANGE and bool((kb == 9).all())
    # a sequence's rows out of order
    kc, vc = (torch.full((2, 2, 8, 128), 9, dtype=torch.uint8, device="cuda") for _ in "kv")
    ks, vs = (torch.full((2, 2, 1), 3.0, device="cuda") for _ in "kv")
    seq, pos = dev(*rows_of((0, 5, 1), (0, 2, 1)))
    s5.step5_kv_append_e4m3(geom, x.expand(2, -1, -1).contiguous(), x.expand(2, -1, -1).contiguous(),
                            s5.PagedCache(kc, vc, table.cuda(), ks, vs), seq, pos)
    assert status(s5) == s5.DEV_RANGE
    assert bool((kc[1, :, 5] != 9).any()) and bool((kc[1, :, 2] == 9).all())


@pytest.mark.parametrize("B", [2, 40000])
def test_append_e4m3_flags_sequences_that_are_split(s5, B):
    """Rows of a sequence with others between them raise the range flag (here they share no region)."""
    geom = geometry(s5, 1, 4)
    table = torch.arange(4, dtype=torch.int32).repeat(B, 1).cuda()
    cache = s5.PagedCache.create(geom, 4, 64, table)
    for runs, want in (([(B - 1, 8, 1), (0, 40, 1), (B - 1, 16, 1), (0, 48, 1)], s5.DEV_RANGE),
                       ([(0, 8, 4), (-1, 0, 1), (0, 16, 1)], s5.DEV_RANGE),
                       ([(0, 0, 100), (B - 1, 128, 100), (-1, 0, 60), (0, 104, 7)], s5.DEV_RANGE),
                       ([(B - 1, 8, 1), (0, 40, 1), (-1, 0, 1), (-1, 0, 1)], 0),
                       ([(-1, 0, 1), (B - 1, 8, 100), (-1, 0, 300), (0, 120, 100), (-1, 0, 1)], 0)):
        seq, pos = rows_of(*runs)
        x = torch.ones((len(seq), 1, 128), dtype=torch.bfloat16).cuda()
        s5.step5_kv_append_e4m3(geom, x, x, cache, *dev(seq, pos))
        assert status(s5) == want, runs
    if B > 2:  # a decode batch of many sequences, in any order, and with one of them twice
        seq = torch.randperm(B, generator=torch.Generator().manual_seed(78)).int()
        pos = torch.zeros(B, dtype=torch.int32)
        cache = s5.PagedCache.create(geom, B, 16, torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1))
        x = torch.ones((B, 1, 128), dtype=torch.bfloat16).cuda()
        for twice in (False, True):
            if twice:
                seq[100], seq[-100] = seq[200], -1
                pos[100] = 8  # (in the next region)
            s5.step5_kv_append_e4m3(geom, x, x, cache, *dev(seq, pos))
            assert status(s5) == (s5.DEV_RANGE if twice else 0)


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_rotates_q_in_place(s5, e4m3):
    geom = geometry(s5, 2, 8)
    gen = torch.Generator().manual_seed(61)
    q, k, v = (normal(gen, 33, h, 128).cuda() for h in (16, 2, 2))
    cos, sin, seq, pos = dev(*S.rope_tables(64, 96), *rows_of((0, 5, 33)))
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
    call = s5.step5_kv_append_e4m3 if e4m3 else s5.step5_kv_append
    caches = [s5.PagedCache.create(geom, 8, 8, table, e4m3=e4m3) for _ in range(2)]
    out = torch.empty_like(q)
    call(geom, k, v, caches[0], seq, pos, cos, sin, q, out)
    same = q.clone()
    call(geom, k, v, caches[1], seq, pos, cos, sin, same, same)
    assert status(s5) == 0
    assert torch.equal(same, out) and not torch.equal(out, q)
    assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)


def test_append_bf16_fills_the_contiguous_caches(s5):
    """Without a table the bf16 append fills the caches that step5_sparse_attn reads: tokens
    appended one chunk at a time give the same output as caches filled by hand."""
    w = S.workload({"positions": [5003, 129], "B": 2}, seed=31)
    t = S.materialize(w, device="cuda")
    geom = s5.STEP5_GEOMETRY
    k, v = (torch.zeros_like(t[n]) for n in ("k_cache", "v_cache"))
    cache = s5.PagedCache(k, v)
    for b in range(2):
        for at in range(0, int(w.row_pos[b]) + 1, 1000):
            n = min(1000, int(w.row_pos[b]) + 1 - at)
            rows = [t[x][b, :, at:at + n].transpose(0, 1).contiguous() for x in ("k_cache", "v_cache")]
            s5.step5_kv_append(geom, *rows, cache, *dev(*rows_of((b, at, n))))
    ws = s5.Workspace.create(geom, w.N, w.r_cap)
    ids = torch.empty((2, 4, 512), dtype=torch.int32, device="cuda")
    cnt = torch.empty((2, 4), dtype=torch.int32, device="cuda")
    s5.step5_region_summarize(geom, t["idx_k"], t["idx_z"], t["cos"], t["sin"], t["sum_begin"], t["sum_end"],
                              t["summaries"], max_regions_per_seq=w.max_span)
    s5.step5_index_score_topk(geom, t["idx_q"], t["w"], t["row_seq"], t["row_pos"], t["cos"], t["sin"], t["summaries"],
                              ids, cnt, ws.tensor, t_cap=w.t_cap)
    outs = []
    for kk, vv in ((k, v), (t["k_cache"], t["v_cache"])):
        out = torch.empty((2, 32, 128), dtype=torch.bfloat16, device="cuda")
        s5.step5_sparse_attn(geom, t["q"], kk, vv, t["row_seq"], t["row_pos"], ids, cnt, out, ws.tensor)
        outs.append(out)
    assert status(s5) == 0
    assert torch.equal(*outs)


# ------------------------------------------------------------------------------ attention

class Case:
    """A pool, its table and rows at (row_seq, row_pos), and the 64-bit answer."""

    def __init__(self, s5, runs, G=4, hq=8, pt=64, seed=1, q_scale=1.5, lo=-9, hi=-4, extra=0, **geom):
        self.s5, self.gen = s5, torch.Generator().manual_seed(seed)
        self.geom = geometry(s5, G, hq, **geom)
        self.seq, self.pos = rows_of(*runs)
        self.N, B = len(self.seq), int(self.seq.max()) + 1
        length = -(-(int(self.pos.max()) + 1 + extra) // pt)
        self.table = tables(self.gen, B, length)
        P = B * length + 3
        self.k, self.ks = random_pool(self.gen, P, G, pt, lo, hi)
        self.v, self.vs = random_pool(self.gen, P, G, pt, lo, hi)
        self.q = normal(self.gen, self.N, G * hq, 128, scale=q_scale)
        self.ws = s5.PagedWorkspace.create(self.geom)
        self.ids = self.cnt = self.gate = None

    def pick(self, counts=None):
        G, top_k = self.geom.num_kv_groups, self.geom.top_k
        self.ids = torch.full((self.N, G, top_k), -1, dtype=torch.int32)
        self.cnt = torch.zeros((self.N, G), dtype=torch.int32)
        for n in range(self.N):
            own = int(self.pos[n]) // 8
            for g in range(G):
                c = min(top_k, own)
                self.ids[n, g, :c] = torch.randperm(max(own, 1), generator=self.gen)[:c].int()
                self.cnt[n, g] = c
        return self

    def cache(self):
        return self.s5.PagedCache(*dev(self.k, self.v, self.table, self.ks, self.vs))

    def run(self, window=0, cache=None, out=None):
        out = torch.full((self.N, self.geom.num_q_heads, 128), 5.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        q, seq, pos, ids, cnt, gate = dev(self.q, self.seq, self.pos, self.ids, self.cnt, self.gate)
        cache = cache or self.cache()
        if ids is None:
            self.s5.step5_paged_attn_e4m3(self.geom, q, cache, seq, pos, out, self.ws, window=window, gate=gate)
        else:
            self.s5.step5_sparse_attn_e4m3(self.geom, q, cache, seq, pos, ids, cnt, out, self.ws, gate=gate)
        return out

    def want(self, window=0):
        return R.attend(self.q.double(), R.decode(self.k), R.decode(self.v), self.ks, self.vs, self.table, self.seq,
                        self.pos, self.geom.softmax_scale, window, self.ids, self.cnt, self.gate)

    def check(self, window=0):
        got = self.run(window).cpu()
        assert status(self.s5) == 0
        out, mass = self.want(window)
        real = self.seq >= 0
        assert bool((got[~real] == 5.0).all())
        assert R.off(got[real], out[real], mass[real]) <= 1.0


SHAPES = [(4, 8, 64), (1, 16, 8), (2, 4, 24), (8, 8, 16)]
ROWS = {
    "first": [(0, 0, 1)], "region_end": [(0, 7, 1)], "region_start": [(0, 8, 1)], "tile": [(0, 127, 1)],
    "past_tile": [(0, 128, 1)], "odd": [(0, 1001, 1)], "ragged": [(3, 300, 1), (0, 1, 1), (-1, 0, 1), (2, 2047, 1), (1, 515, 1)],
    "draft": [(0, 130, 4), (1, 6, 4)], "chunk": [(0, 0, 37)], "chunk_on": [(0, 201, 50)],
    "chunks": [(1, 100, 19), (0, 0, 21), (-1, 0, 2), (2, 63, 9)],
}


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("G, hq, pt", SHAPES)
def test_paged_attention(s5, rows, G, hq, pt):
    Case(s5, ROWS[rows], G, hq, pt, seed=len(rows)).check()


@pytest.mark.parametrize("window", [1, 2, 7, 8, 9, 100, 128, 512, 5000])
@pytest.mark.parametrize("rows", ["first", "odd", "ragged", "chunk_on", "chunks"])
def test_paged_attention_window(s5, rows, window):
    Case(s5, ROWS[rows], 2, 8, 24, seed=window).check(window)


def test_windows_past_32_bits(s5):
    """A window of 2^32 + 1 tokens is every token, one of -2^32 none that is allowed."""
    c = Case(s5, [(0, 1001, 1)], 2, 8, 24, seed=80)
    assert torch.equal(c.run(2 ** 32 + 1), c.run(0))
    with pytest.raises(s5.Step5Error):
        c.run(-2 ** 32)


def test_paged_attention_scattered_rows(s5):
    """Rows of one sequence in any order, some twice, beside others."""
    c = Case(s5, [(0, 900, 1)] * 2 + [(0, 3, 1), (1, 77, 2), (0, 901, 3), (1, 12, 1), (0, 10, 1)], seed=9)
    c.check()
    c.check(64)


def test_paged_attention_long_row(s5):
    """One row of 70,001 tokens: the split of its keys over the GPU and their merge."""
    Case(s5, [(0, 70000, 1)], 1, 8, 64, seed=5).check()


@pytest.mark.parametrize("tiles", [900, 1100, 1777, 2500, 3333])
def test_paged_attention_runs_of_tiles(s5, tiles):
    """Rows whose tiles are cut at other places of their look-ahead: every CTA's run starts
    somewhere inside an item."""
    rest = tiles - 2 * (tiles // 3)
    Case(s5, [(b, 128 * n - 5, 1) for b, n in enumerate((tiles // 3, rest, tiles // 3))], 1, 4, 64, seed=tiles).check()


@pytest.mark.parametrize("n", [23, 37, 101])
def test_sparse_attention_runs_of_tiles(s5, n):
    Case(s5, [(0, 4300, n), (1, 1511, n // 2)], 2, 8, 16, seed=n).pick().check()


def test_paged_attention_gate(s5):
    for runs in ([(0, 1001, 1), (1, 9, 1)], [(0, 90, 40)]):
        c = Case(s5, runs, seed=6)
        c.gate = normal(c.gen, c.N, c.geom.num_q_heads, scale=2.0)
        c.check()


def test_paged_attention_extreme_scales(s5):
    """Scales over 60 binades, zero regions of V with the smallest scale, zero q."""
    c = Case(s5, [(0, 1200, 1), (0, 300, 20)], 2, 8, 16, seed=7)
    c.vs = torch.exp2(torch.randint(-30, 30, c.vs.shape, generator=c.gen).float())
    c.q[0, :4] = 0.0
    c.check()
    c = Case(s5, [(0, 1200, 1)], 2, 8, 16, seed=8)
    zero = torch.randint(0, 2, c.vs.shape, generator=c.gen).bool()
    c.vs[zero] = 2.0 ** -126
    c.v.view(*c.vs.shape, 8, 128)[zero] = 0
    c.check()


def test_paged_attention_peaked_scores(s5):
    """A few keys that hold nearly all weight, found late and early: the running maximum moves far."""
    for at in (3, 640, 1199):
        c = Case(s5, [(0, 1200, 1), (0, 1195, 8)], 1, 8, 16, seed=at)
        page, slot = R.place(c.table, 0, at, 16)
        best = (c.q[0, 3].float() * 40).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        c.k[page, 0, slot] = best
        c.check()


def test_paged_attention_sink(s5):
    """One key 2^14 times as heavy as each of the others, whose sum is still half of the mass."""
    c = Case(s5, [(0, 16383, 1)], 1, 8, 64, seed=2, lo=-7, hi=-6)
    c.q[:] = 0.0
    c.q[..., 0] = 1.0
    c.k[...] = 0
    page, slot = R.place(c.table, 0, 100, 64)
    c.k[page, 0, slot, 0] = torch.tensor([448.0]).to(torch.float8_e4m3fn).view(torch.uint8)[0]
    c.ks[page, 0, slot // 8] = 14 * np.log(2) / c.geom.softmax_scale / 448.0
    c.v[...] = torch.tensor([1.0]).to(torch.float8_e4m3fn).view(torch.uint8)[0]
    c.v[page, 0, slot] = 0
    c.check()


@pytest.mark.parametrize("rows", [[(0, 1002, 1)], [(0, 1002, 1), (0, 4, 1)], [(0, 300, 37)]])
@pytest.mark.parametrize("window", [0, 101])
def test_tokens_outside_never_reach_the_result(s5, rows, window):
    """NaN codes and bad scales and pages outside a row's keys change nothing."""
    c = Case(s5, rows, 2, 8, 24, seed=4, extra=200)
    base = c.run(window)
    last = int(c.pos.max())
    nan = 0x7f
    lows = [max(0, int(p) - window + 1) if window else 0 for p in c.pos]
    first = min(lows)
    for tok in range(0, c.table.shape[1] * 24):
        page, slot = R.place(c.table, 0, tok, 24)
        if tok > last or tok < first:
            c.k[page, :, slot] = nan
            c.v[page, :, slot] = nan
            r = tok // 8
            if r > last // 8 or r < first // 8:
                c.ks[page, :, slot // 8] = float("nan")
                c.vs[page, :, slot // 8] = 0.0
    used = set(c.table.flatten().tolist())
    for page in range(c.k.shape[0]):
        if page not in used:
            c.k[page], c.v[page], c.ks[page], c.vs[page] = nan, nan, float("inf"), -1.0
    for i in range(c.table.shape[1]):
        if i * 24 > last or (i + 1) * 24 <= first:
            c.table[0, i] = -7
    got = c.run(window)
    assert status(s5) == 0
    assert torch.equal(base, got)


def test_nan_of_a_later_row_stays_with_it(s5):
    """A NaN in a token's value reaches the rows that see the token and no row before it."""
    c = Case(s5, [(0, 300, 37)], 2, 8, 24, seed=14)
    base = c.run().cpu()
    page, slot = R.place(c.table, 0, 320, 24)
    c.v[page, 1, slot, 17] = 0x7f
    got = c.run().cpu()
    assert status(s5) == 0
    sees = torch.zeros(got.shape, dtype=torch.bool)
    sees[20:, 8:, 17] = True
    assert bool(torch.isnan(got[sees]).all())
    assert torch.equal(got[~sees], base[~sees])
    c = Case(s5, [(0, 300, 37)], 2, 8, 24, seed=14)
    c.k[page, 1, slot, 17] = 0x7f
    got = c.run().cpu()
    sees[20:, 8:] = True
    assert bool(torch.isnan(got[sees]).all())
    assert torch.equal(got[~sees], base[~sees])


def test_bad_pages_scales_and_rows(s5):
    """A region of the keys without a page or with a bad scale is left out and flagged; a
    row out of range gets zeros."""
    for runs in ([(0, 500, 1)], [(0, 480, 20)]):
        c = Case(s5, runs, 2, 8, 16, seed=11)
        want_seen = torch.ones(501, dtype=torch.bool)
        c.table[0, 3] = -1
        c.table[0, 9] = c.k.shape[0]
        page, slot = R.place(c.table, 0, 200, 16)
        c.ks[page, :, slot // 8] = float("inf")
        page2, slot2 = R.place(c.table, 0, 300, 16)
        c.vs[page2, :, slot2 // 8] = 0.0
        for lo, n in ((48, 16), (144, 16), (200, 8), (296, 8)):
            want_seen[lo:lo + n] = False
        got = c.run().cpu()
        assert status(s5) == s5.DEV_RANGE
        for n in range(c.N):
            p = int(c.pos[n])
            toks = torch.arange(p + 1)[want_seen[:p + 1]]
            at = [R.place(c.table, 0, int(t), 16) for t in toks]
            pg, sl = torch.tensor([a[0] for a in at]), torch.tensor([a[1] for a in at])
            for g in range(2):
                kk = R.decode(c.k)[pg, g, sl] * c.ks[pg, g, sl // 8].double()[:, None]
                codes, scales = R.decode(c.v)[pg, g, sl], c.vs[pg, g, sl // 8].double()
                x = torch.softmax(c.q[n, 8 * g:8 * g + 8].double() @ kk.T * c.geom.softmax_scale, -1)
                assert R.off(got[n, 8 * g:8 * g + 8], x @ (codes * scales[:, None]), R.terms(x, codes, scales)) <= 1.0
    c = Case(s5, [(0, 100, 1), (0, 101, 1), (0, 102, 1), (0, 103, 1)], 2, 8, 16, seed=12)
    good = c.run()
    c.pos[1], c.seq[2] = 16 * c.table.shape[1], 7
    got = c.run()
    assert status(s5) == s5.DEV_RANGE
    assert bool((got[1:3] == 0).all())
    for n in (0, 3):  # the other rows as ever, up to the order of fp32 sums
        assert float((got[n] - good[n]).float().abs().max()) <= 2.0 ** -7 * float(good[n].float().abs().max())
    # a row none of whose regions can be read
    c = Case(s5, [(0, 5, 1)], 2, 8, 16, seed=13)
    c.table[0, 0] = -1
    assert bool((c.run() == 0).all()) and status(s5) == s5.DEV_RANGE


@pytest.mark.parametrize("top_k", [1, 5, 64, 512])
@pytest.mark.parametrize("G, hq, pt", SHAPES)
def test_sparse_attention(s5, top_k, G, hq, pt):
    runs = [(2, 2000, 1), (0, 7, 1), (-1, 0, 1), (1, 0, 1), (0, 1000, 3)]
    Case(s5, runs, G, hq, pt, seed=top_k, top_k=top_k).pick().check()


def test_sparse_attention_many_rows(s5):
    """A chunk of 150 rows beyond 512 regions, all 4 groups."""
    Case(s5, [(0, 4200, 150)], seed=21).pick().check()


def test_sparse_attention_gate_and_bad_picks(s5):
    c = Case(s5, [(0, 1000, 2)], 2, 8, 16, seed=22, top_k=64).pick()
    c.gate = normal(c.gen, c.N, 16, scale=2.0)
    c.check()
    want = c.want()
    # ids at, past and below the range stand for nothing
    ids, cnt = c.ids.clone(), c.cnt.clone()
    c.cnt -= 3
    short = c.want()
    c.ids[..., 61], c.ids[..., 62], c.ids[..., 63] = 125, -1, 1 << 30
    c.cnt += 3
    got = c.run()
    assert status(s5) == s5.DEV_RANGE
    assert R.off(got, *short) <= 1.0
    c.ids, c.cnt = ids, cnt + 1000  # a count past top_k is clamped
    got = c.run()
    assert status(s5) == s5.DEV_RANGE
    assert R.off(got, *want) <= 1.0


def test_attention_is_deterministic_and_replays(s5):
    """The same inputs give the same bits, on other streams, with other calls on the
    workspace in between, and captured into graphs that share the workspace."""
    cases = [Case(s5, [(0, 9000, 1), (1, 33, 1)], seed=31), Case(s5, [(0, 5000, 1)], seed=32).pick(),
             Case(s5, [(0, 1100, 60)], seed=33)]
    caches = [c.cache() for c in cases]
    ws = cases[0].ws
    for c in cases:
        c.ws = ws
    first = [c.run(cache=m) for c, m in zip(cases, caches)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [c.run(cache=m) for c, m in zip(cases, caches)]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    graphs = []
    for c, m in zip(cases, caches):
        tensors = [t for t in dev(c.q, c.seq, c.pos, c.ids, c.cnt)]
        out = torch.zeros_like(first[0][:1]).expand(c.N, -1, -1).contiguous()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            if tensors[3] is None:
                s5.step5_paged_attn_e4m3(c.geom, tensors[0], m, tensors[1], tensors[2], out, ws)
            else:
                s5.step5_sparse_attn_e4m3(c.geom, tensors[0], m, tensors[1], tensors[2], tensors[3], tensors[4], out, ws)
        graphs.append((g, out, tensors))
    for _ in range(3):
        for g, _, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (g, out, _), a in zip(graphs, first):
        assert torch.equal(out, a)
    assert status(s5) == 0


@pytest.mark.parametrize("runs", [[(0, 900, 1)], [(0, 60000, 1)], [(0, 100, 1), (1, 200, 1)], [(0, 700, 70), (1, 3, 40)], [(0, 3000, 33)]])
def test_buffers_of_the_smallest_alignment(s5, runs):
    """q and out at addresses that are multiples of 16 bytes and no more give the same bits."""
    c = Case(s5, runs, 2, 8, 16, seed=51)
    base = c.run()
    n = base.numel()
    q, out = (torch.zeros(n + 64, dtype=torch.bfloat16, device="cuda") for _ in "qo")
    for at in (8, 24):
        qv, ov = (x[at:at + n].view(base.shape) for x in (q, out))
        assert qv.data_ptr() % 32 == 16 and ov.data_ptr() % 32 == 16
        qv.copy_(c.q)
        out.zero_()
        s5.step5_paged_attn_e4m3(c.geom, qv, c.cache(), *dev(c.seq, c.pos), ov, c.ws)
        assert status(s5) == 0
        assert torch.equal(ov, base)
        assert bool((out[:at] == 0).all()) and bool((out[at + n:] == 0).all())


@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("G, hq", [(1, 4), (2, 16)])
def test_drafts_of_long_rows(s5, G, hq, window):
    """A few rows of each of several sequences, long and short ones, one of them padding."""
    Case(s5, [(0, 9001, 4), (1, 130, 5), (-1, 0, 1), (2, 4092, 8), (3, 0, 2)], G, hq, 16, seed=52).check(window)


@pytest.mark.parametrize("G, hq, n", [(1, 4, 130), (2, 8, 70), (1, 16, 37)])
@pytest.mark.parametrize("window", [0, 40])
def test_scattered_rows_that_share_tiles(s5, G, hq, n, window):
    """Many rows of two sequences in any order, some twice, some of them padding."""
    gen = torch.Generator().manual_seed(n)
    runs = [(int(b), int(p), 1) for b, p in zip(torch.randint(-1, 2, (n,), generator=gen), torch.randint(0, 700, (n,), generator=gen))]
    Case(s5, runs + [runs[0]] + [(1, 699, 1), (0, 0, 1)], G, hq, 16, seed=n).check(window)


@pytest.mark.parametrize("G, hq, runs", [(1, 8, [(0, 20000, 16)]), (2, 16, [(0, 9000, 9), (1, 40, 9)]), (1, 4, [(0, 40000, 33)]),
                                         (4, 8, [(0, 2500, 33), (1, 5, 40)])])
def test_few_rows_shared_by_many_ctas(s5, G, hq, runs):
    Case(s5, runs, G, hq, 64, seed=len(runs) + hq).check()


def test_nan_in_a_block_of_two_sequences(s5):
    """A NaN that one sequence's rows see leaves the rows of the other in their block alone."""
    runs = [(0, 256, 9), (1, 200, 9)]
    c = Case(s5, runs, 1, 8, 16, seed=53)
    base = c.run().cpu()
    for tok, first in ((10, 0), (260, 4)):  # seen by every row of the sequence; by rows from the fifth on
        c = Case(s5, runs, 1, 8, 16, seed=53)
        page, slot = R.place(c.table, 0, tok, 16)
        c.v[page, 0, slot, 77] = 0xff
        got = c.run().cpu()
        assert status(s5) == 0
        sees = torch.zeros(got.shape, dtype=torch.bool)
        sees[first:9, :, 77] = True
        assert bool(torch.isnan(got[sees]).all())
        assert torch.equal(got[~sees], base[~sees])


def zero_values(c, toks):
    """V of tokens toks (whole regions) as appending zeros leaves it: codes 0, the smallest scale."""
    for tok in toks[::8]:
        page, slot = R.place(c.table, 0, tok, c.k.shape[2])
        c.v[page, :, slot:slot + 8] = 0
        c.vs[page, :, slot // 8] = 2.0 ** -126


@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("runs", [[(0, 300, 40)], [(0, 339, 1)]])
def test_regions_whose_values_are_zero(s5, runs, window):
    """V of zeros, which has the smallest scale: in the first tiles of a row's keys, in all of them, and beside a region
    that cannot be read."""
    for until in (128, 240):
        c = Case(s5, runs, 2, 8, 16, seed=71)
        zero_values(c, range(0, until))
        c.check(window)
    c = Case(s5, runs, 2, 8, 16, seed=71)
    zero_values(c, range(0, 352))
    assert bool((c.run(window) == 0).all()) and status(s5) == 0
    page, slot = R.place(c.table, 0, 168, 16)
    c.ks[page, :, slot // 8] = float("inf")
    assert bool((c.run(window) == 0).all()) and status(s5) == s5.DEV_RANGE


@pytest.mark.parametrize("B, n", [(1, 40), (40, 64)])
@pytest.mark.parametrize("window", [0, 200])
def test_bad_rows_in_a_block_of_good_ones(s5, B, n, window):
    """Rows out of range between rows that see whole tiles get zeros, the others what they get beside
    padding: items that many CTAs share (B 1), and whole ones (B 40)."""
    c = Case(s5, [(b, 300, n) for b in range(B)], 2, 8, 16, seed=72)
    bad = torch.zeros(c.N, dtype=torch.bool)
    bad[17::29] = True
    bad[-1] = True
    seq, pos = c.seq.clone(), c.pos.clone()
    c.seq[bad] = -1
    want = c.run(window)
    assert status(s5) == 0
    assert bool((want[bad] == 5.0).all())
    c.seq[:], c.pos[:] = seq, pos
    c.seq[bad] = B
    c.seq[17], c.pos[17] = seq[17], 16 * c.table.shape[1]
    c.seq[-1], c.pos[-1] = seq[-1], -1
    got = c.run(window)
    assert status(s5) == s5.DEV_RANGE
    assert bool((got[bad] == 0).all())
    assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("big", [2.0 ** 30, 2.0 ** 110])
def test_large_value_scales_of_unseen_regions(s5, window, big):
    """The V scale of a later token's region, or of another sequence of the block, changes nothing in the
    rows that do not see it."""
    c = Case(s5, [(0, 130, 40)], 1, 8, 16, seed=73)
    base = c.run(window)
    page, slot = R.place(c.table, 0, 160, 16)
    c.vs[page, :, slot // 8] = big
    got = c.run(window)
    assert torch.equal(got[:30], base[:30])
    c.check(window)
    for first in (0, 1):  # the sequence walked first, or second
        runs = [(0, 256, 9), (1, 200, 9)]
        c = Case(s5, runs, 1, 8, 16, seed=74)
        base = c.run(window)
        c.vs[c.table[first].long()] *= big
        got = c.run(window)
        assert status(s5) == 0
        other = c.seq != first
        assert torch.equal(got[other], base[other])
        c.check(window)


@pytest.mark.parametrize("hq, pt", [(4, 64), (8, 16), (16, 8)])
def test_windows_of_rows_that_lie_apart(s5, hq, pt):
    """What no row's window holds is not touched where the rows of a sequence that share tiles lie apart: freed
    pages and bad scales there are no errors."""
    c = Case(s5, [(0, 20, 20), (0, 900, 9), (0, 3, 1), (0, 2000, 30)], 1, hq, pt, seed=76)
    base = c.run(16)
    assert status(s5) == 0
    seen = torch.zeros(c.table.shape[1] * pt, dtype=torch.bool)
    for p in c.pos.tolist():
        seen[max(0, p - 15):p + 1] = True
    pages = seen.view(-1, pt).any(1)
    regions = seen.view(-1, 8).any(1)
    for r in (~regions).nonzero().flatten().tolist():
        page, slot = R.place(c.table, 0, 8 * r, pt)
        c.ks[page, :, slot // 8], c.vs[page, :, slot // 8] = float("nan"), -1.0
    c.table[0, ~pages] = -7
    got = c.run(16)
    assert status(s5) == 0
    assert torch.equal(got, base)
    c.table[0, int(pages.nonzero()[-1])] = -7  # (and one that a row sees is)
    c.run(16)
    assert status(s5) == s5.DEV_RANGE


@pytest.mark.parametrize("runs, low, gate", [([20000 - b for b in range(40)], -126, 0.0), ([300 + i for _ in range(40) for i in range(64)], -118, -8.0)])
def test_values_near_the_smallest(s5, runs, low, gate):
    """Values of 2^-126 times their codes keep their bits beside large row sums and small gates.  q is zero and the codes are
    positive, so that each result is the mean of its keys' values: one rounding (2^-8), sums of 20,000 positive terms in fp32
    (below 2^-9) and a gate in fp32."""
    c = Case(s5, [(0, p, 1) for p in runs], 4, 8, 64, seed=79)
    c.seq = torch.arange(40).repeat_interleave(c.N // 40).int()
    c.table = c.table.repeat(40, 1)
    c.q[:] = 0.0
    c.v &= 0x7f
    c.vs = torch.exp2(torch.randint(low, low + 3, c.vs.shape, generator=c.gen).float())
    c.gate = torch.full((c.N, 32), gate, dtype=torch.bfloat16) if gate else None
    got = c.run().cpu().double()
    assert status(s5) == 0
    v = (R.decode(c.v) * c.vs.double().repeat_interleave(8, 2)[..., None])[c.table[0].long()]  # [pages][G][64][128]
    mean = v.transpose(1, 2).reshape(-1, 4, 128).cumsum(0) / torch.arange(1, c.table.shape[1] * 64 + 1)[:, None, None]
    want = mean[c.pos.long()].repeat_interleave(8, 1) * (1.0 / (1.0 + np.exp(-gate)) if gate else 1.0)
    assert float(want.min()) > 2.0 ** -125
    assert float(((got - want).abs() / want).max()) <= 2.0 ** -8 + 2.0 ** -9


@pytest.mark.parametrize("runs", [[(0, 5, 1), (0, 900, 1)], [(b, 40 * b, 1) for b in range(60)], [(0, 300, 40)], [(b, 300, 64) for b in range(40)]])
def test_rows_without_keys_are_zero_whatever_their_gate(s5, runs):
    """NaN as the gate of a row out of range."""
    c = Case(s5, runs, 4, 8, 16, seed=81)
    c.gate = normal(c.gen, c.N, 32)
    bad = torch.zeros(c.N, dtype=torch.bool)
    bad[::7] = True
    c.gate[bad] = float("nan")
    c.pos[bad] = 16 * c.table.shape[1]
    got = c.run()
    assert status(s5) == s5.DEV_RANGE
    assert bool((got[bad] == 0).all()) and bool(torch.isfinite(got[~bad]).all())


def test_a_table_that_is_replaced(s5):
    """The cache's next call reads the table assigned to it."""
    c = Case(s5, [(0, 1001, 1), (1, 500, 1)], seed=75)
    cache = c.cache()
    c.table = c.table.flip(0).contiguous()
    cache.block_table = c.table.cuda()
    got = c.run(cache=cache).cpu()
    assert status(s5) == 0
    assert R.off(got, *c.want()) <= 1.0


def test_two_streams_at_once(s5):
    """Calls on two streams, each with its own workspace, none waiting for the other."""
    cases = [Case(s5, [(0, 30000, 1)], 2, 8, 16, seed=54), Case(s5, [(0, 1000, 300)], 2, 8, 16, seed=55),
             Case(s5, [(0, 4300, 200)], 2, 8, 16, seed=56).pick(), Case(s5, [(b, 3000, 1) for b in range(9)], 2, 8, 16, seed=57)]
    args = [(c, c.cache(), dev(c.q, c.seq, c.pos, c.ids, c.cnt)) for c in cases]
    first = [c.run(cache=m) for c, m, _ in args]
    outs = [[torch.empty_like(f) for f in first] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [s5.PagedWorkspace.create(cases[0].geom) for _ in range(2)]
    torch.cuda.synchronize()
    for turn in range(4):
        for i, (st, ws) in enumerate(zip(streams, spaces)):
            for j in range(len(args)):
                j = (j + i) % len(args)
                c, m, (q, seq, pos, ids, cnt) = args[j]
                if ids is None:
                    s5.step5_paged_attn_e4m3(c.geom, q, m, seq, pos, outs[i][j], ws, stream=st)
                else:
                    s5.step5_sparse_attn_e4m3(c.geom, q, m, seq, pos, ids, cnt, outs[i][j], ws, stream=st)
    assert status(s5) == 0
    for got in outs:
        for a, b in zip(got, first):
            assert torch.equal(a, b)


@pytest.mark.parametrize("runs, picks", [([(0, 1001, 1), (1, 70, 1)], False), ([(0, 300, 70)], False), ([(0, 1001, 2)], True)])
def test_attention_over_pools_past_32_bit_offsets(s5, runs, picks):
    """The same pages at the end of pools of more than 2^31 bytes give the same bits."""
    c = Case(s5, runs, 4, 8, 64, seed=62)
    if picks:
        c.pick()
    base = c.run()
    pages = 2 ** 31 // (4 * 64 * 128) + 50
    first = pages - c.k.shape[0]
    pools = []
    for small in (c.k, c.v, c.ks, c.vs):
        big = torch.full((pages, *small.shape[1:]), 0x7f if small.dtype == torch.uint8 else float("nan"), dtype=small.dtype, device="cuda")
        big[first:] = small.cuda()
        pools.append(big)
    k, v, ks, vs = pools
    got = c.run(cache=s5.PagedCache(k, v, (c.table + first).cuda(), ks, vs))
    assert status(s5) == 0
    assert torch.equal(got, base)


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_to_pools_past_32_bit_offsets(s5, e4m3):
    geom = geometry(s5, 4, 8)
    gen = torch.Generator().manual_seed(63)
    k, v = (normal(gen, 100, 4, 128).cuda() for _ in "kv")
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    seq, pos = dev(*rows_of((0, 60, 100)))
    call = s5.step5_kv_append_e4m3 if e4m3 else s5.step5_kv_append
    pages = 2 ** 31 // (4 * 64 * 128) + 50
    small = s5.PagedCache.create(geom, 3, 64, table, e4m3=e4m3)
    big = s5.PagedCache.create(geom, pages, 64, table + (pages - 3), e4m3=e4m3)
    for cache in (small, big):
        call(geom, k, v, cache, seq, pos)
    assert status(s5) == 0
    for name in ("k", "v") + (("k_scales", "v_scales") if e4m3 else ()):
        x = getattr(big, name)
        assert torch.equal(x[-3:], getattr(small, name)), name
        assert bool((x[:-3] == (1 if "scales" in name else 0)).all()), name


def test_workspace_needs_no_initialisation(s5):
    """A workspace full of anything gives the same bits."""
    for c in (Case(s5, [(0, 5000, 1), (1, 3, 1)], seed=58), Case(s5, [(0, 2000, 40)], seed=59), Case(s5, [(0, 5000, 3)], seed=60).pick()):
        base = c.run()
        c.ws.tensor.fill_(0xff)
        assert torch.equal(c.run(), base)
        assert status(s5) == 0


# ------------------------------------------------------------------------------ together

def test_run_together(s5):
    """Prompt chunks appended, then decode steps of the whole path over the pages: every
    step's output is the attention over the picked regions of what the cache holds, and
    near the bf16 path's on the same tokens."""
    w = S.workload({"positions": [4700, 4170], "B": 2}, seed=41)
    t = S.materialize(w, device="cuda")
    geom = s5.STEP5_GEOMETRY
    pt, length = 32, -(-4710 // 32)
    gen = torch.Generator().manual_seed(1)
    table = tables(gen, 2, length)
    cache = s5.PagedCache.create(geom, 2 * length + 3, pt, table.cuda())
    cos, sin = dev(*S.rope_tables(length * pt, 64))
    for b in range(2):
        for at in range(0, int(w.row_pos[b]), 1999):
            n = min(1999, int(w.row_pos[b]) - at)
            rows = [t[x][b, :, at:at + n].transpose(0, 1).contiguous() for x in ("k_cache", "v_cache")]
            s5.step5_kv_append_e4m3(geom, *rows, cache, *dev(*rows_of((b, at, n))), cos, sin)
    ws, pws = s5.Workspace.create(geom, 2, w.r_cap), s5.PagedWorkspace.create(geom)
    ids = torch.empty((2, 4, 512), dtype=torch.int32, device="cuda")
    cnt = torch.empty((2, 4), dtype=torch.int32, device="cuda")
    out, q_rot = (torch.empty((2, 32, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.stack([t[x][b, :, int(w.row_pos[b])] for b in range(2)]) for x in ("k_cache", "v_cache"))
    s5.decode_step_paged(geom, t, cache, ws, pws, k, v, ids, cnt, q_rot, out, w.max_span, cos, sin)
    assert status(s5) == 0
    at = torch.from_numpy(w.row_pos).long()
    assert torch.equal(q_rot.cpu().double(), R.rotate(t["q"].cpu().double(), cos.cpu(), sin.cpu(), at))
    want = R.attend(q_rot.cpu(), R.decode(cache.k), R.decode(cache.v), cache.k_scales.cpu(), cache.v_scales.cpu(),
                    table, w.row_seq, w.row_pos, geom.softmax_scale, ids=ids.cpu(), counts=cnt.cpu())
    assert R.off(out, *want) <= 1.0
    # the same step over bf16 caches: e4m3 rounds each key and value by at most 2^-4 of itself
    kb, vb = (torch.zeros_like(t[x]) for x in ("k_cache", "v_cache"))
    flat = s5.PagedCache(kb, vb)
    for b in range(2):
        n = int(w.row_pos[b]) + 1
        rows = [t[x][b, :, :n].transpose(0, 1).contiguous() for x in ("k_cache", "v_cache")]
        s5.step5_kv_append(geom, *rows, flat, *dev(*rows_of((b, 0, n))), cos, sin)
    ref = torch.empty_like(out)
    s5.step5_sparse_attn(geom, q_rot, kb, vb, t["row_seq"], t["row_pos"], ids, cnt, ref, ws.tensor)
    assert status(s5) == 0
    rel = float((out.float() - ref.float()).norm() / ref.float().norm())
    assert rel <= 2.0 ** -4
