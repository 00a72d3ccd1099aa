"""The step's plan on the GPU against the rule, one sequence after another on lists."""
import random

import pytest
import torch

import paged_bf16_reference as B16
from test_gpu_paged import s5, status  # noqa: F401

pytestmark = pytest.mark.gpu
FIELDS = ("row_seq", "row_pos", "row_start", "ends", "granted", "region_begin", "region_end")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Slots:
    """A table and its stack on the GPU and, as lists, on the host."""

    def __init__(self, s5, num_pages, pt, table_len, held, order=None, free=None):  # noqa: F811
        self.s5, self.pt, self.num_pages = s5, pt, num_pages
        order = list(range(num_pages)) if order is None else order
        self.held, self.table = list(held), [[-5] * table_len for _ in held]
        at = 0
        for b, h in enumerate(held):
            h = min(max(h, 0), table_len)
            self.table[b][:h] = order[at:at + h]
            at += h
        self.free = order[at:] if free is None else order[at:at + free]
        stack = self.free + [-9] * (num_pages - len(self.free))
        self.gpu = s5.PagedTable(i32(self.table), i32(self.held), i32(stack), i32([len(self.free)]), pt)

    def step(self, N, lengths, new, in_place=False, twice=None):
        rows = self.s5.PagedRows.create(len(lengths), N)
        for f in FIELDS:
            getattr(rows, f).fill_(77)
        dl, dn = i32(lengths), i32(new)
        if in_place:
            rows.ends = dl
        above = self.gpu.free_pages.tolist()
        self.s5.step5_paged_plan(self.gpu, rows, dl, dn)
        flagged = status(self.s5)
        want, bad = B16.plan(self.table, self.held, self.free, self.num_pages, self.pt, N, lengths, new)
        assert flagged == (1 if bad else 0)
        for f in FIELDS:
            assert getattr(rows, f).tolist() == want[f], f
        assert self.gpu.block_table.tolist() == self.table
        assert self.gpu.held.tolist() == self.held
        assert self.gpu.free_count.tolist() == [len(self.free)]
        assert self.gpu.free_pages.tolist()[:len(self.free)] == self.free
        if not in_place:
            assert dl.tolist() == lengths
        return want, above


@pytest.mark.parametrize("B, pt, N", [(1, 8, 1), (1, 64, 700), (3, 16, 64), (33, 8, 100), (600, 24, 3000), (1025, 16, 9000)])
@pytest.mark.parametrize("scarce", [False, True])
def test_steps(s5, B, pt, N, scarce):  # noqa: F811
    """Steps on end: sequences that grow, pause, shrink, end and start again, with pages to spare or not."""
    rng = random.Random(B * 10 + pt + scarce)
    table_len = -(-400 // pt)
    num = B * table_len if not scarce else max(2, B * table_len // 4)
    order = list(range(num))
    rng.shuffle(order)
    s = Slots(s5, num, pt, table_len, [0] * B, order)
    lengths = [0] * B
    for step in range(6):
        most = max(1, 2 * N // B // 2)
        new = []
        for b in range(B):
            kind = rng.random()
            if kind < 0.15:
                lengths[b] = 0                                    # the sequence is through
            elif kind < 0.3:
                lengths[b] = rng.randint(0, lengths[b])           # tokens rolled back
            cap = table_len * pt - lengths[b]
            new.append(0 if rng.random() < 0.2 else min(cap, rng.choice([1, rng.randint(0, most)])))
        want, _ = s.step(N, lengths, new, in_place=step % 2 == 1)
        lengths = want["ends"]


def test_the_rule_of_scarce_pages(s5):  # noqa: F811
    """Four free pages: the second sequence's need is not met, so the third, which one page would do, waits too, while
    the fourth, which needs none, goes on; the fifth's page comes back first and makes the need of the first two."""
    s = Slots(s5, 10, 8, 4, [0, 0, 1, 1, 0], free=4)
    want, _ = s.step(40, [0, 0, 8, 3, 0], [16, 24, 2, 4, 0])     # (46 rows: the fourth's end past 40)
    assert want["granted"] == [16, 0, 0, 0, 0] and len(s.free) == 2
    s = Slots(s5, 10, 8, 4, [0, 0, 1, 1, 0], free=4)
    want, _ = s.step(46, [0, 0, 8, 3, 0], [16, 24, 2, 4, 0])
    assert want["granted"] == [16, 0, 0, 4, 0] and len(s.free) == 2
    s = Slots(s5, 10, 8, 4, [0, 0, 0, 0, 1], free=4)
    want, _ = s.step(60, [0, 0, 0, 0, 0], [16, 24, 1, 0, 0])
    assert want["granted"] == [16, 24, 0, 0, 0] and s.free == []


def test_roll_back_restores_the_stack(s5):  # noqa: F811
    rng = random.Random(4)
    order = list(range(200))
    rng.shuffle(order)
    lengths = [rng.randint(0, 60) for _ in range(20)]
    s = Slots(s5, 200, 8, 12, [-(-n // 8) for n in lengths], order)
    stack, held = list(s.free), list(s.held)
    for _ in range(3):
        s.step(500, lengths, [rng.randint(0, 20) for _ in range(20)])
        s.step(500, lengths, [0] * 20)
        assert s.free == stack and s.held == held


def test_out_of_range(s5):  # noqa: F811
    """Sequences out of range keep their pages and are flagged; the others are planned."""
    s = Slots(s5, 64, 8, 4, [1, 1, 1, 2, 1, 1], free=20)
    s.step(64, [8, -1, 8, 40, 8, 2 ** 31 - 1], [3, 2, -4, 1, 2, 5])
    s = Slots(s5, 64, 8, 4, [1, 9, -1, 1], free=20)
    s.step(64, [8, 8, 8, 8], [3, 2, 1, 1])
    # rows past N
    s = Slots(s5, 64, 8, 4, [0, 0, 0, 0], free=20)
    s.step(10, [0, 0, 0, 0], [4, 7, 0, 3])
    s = Slots(s5, 64, 8, 4, [0, 0, 0], free=20)
    s.step(10, [0, 0, 0], [4, 2 ** 31 - 1, 3])
    # page numbers out of range are moved as they are
    s = Slots(s5, 64, 8, 4, [2, 0], order=[3, 99, -4, 5], free=2)
    s.step(20, [0, 0], [0, 24])
    # more pages given back than the stack has room for
    s = Slots(s5, 8, 8, 4, [4, 4], order=list(range(16)), free=6)
    s.step(20, [0, 0], [0, 0])
    # a count outside the stack
    for count in (-3, 99):
        s = Slots(s5, 8, 8, 4, [0], free=0 if count < 0 else 8)
        s.gpu.free_count.fill_(count)
        rows = s5.PagedRows.create(1, 4)
        s5.step5_paged_plan(s.gpu, rows, i32([0]), i32([4]))
        assert status(s5) == 1
        assert rows.granted.tolist() == [0 if count < 0 else 4] and s.gpu.free_count.tolist() == [0 if count < 0 else 7]


def test_many_sequences_and_long_ones(s5):  # noqa: F811
    rng = random.Random(1)
    s = Slots(s5, 3 * 8192, 8, 3, [0] * 8192)
    new = [rng.choice([0, 1, 1, 2, 17]) for _ in range(8192)]
    s.step(40000, [0] * 8192, new)
    s.step(40000, new, [1] * 8192)
    # one sequence of 200,000 tokens, given back at once while another takes as many
    s = Slots(s5, 40000, 8, 25000, [25000, 0])
    s.step(200001, [0, 0], [1, 200000])


def test_graph_of_steps(s5):  # noqa: F811
    """A captured step that goes on from the one before."""
    s = Slots(s5, 40, 8, 8, [0] * 4)
    rows = s5.PagedRows.create(4, 12)
    lengths, new = i32([0, 5, 0, 9]), i32([3, 1, 0, 2])
    rows.ends = lengths
    s5.step5_paged_plan(s.gpu, rows, lengths, i32([0, 0, 0, 0]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s5.step5_paged_plan(s.gpu, rows, lengths, new)
    B16.plan(s.table, s.held, s.free, 40, 8, 12, [0, 5, 0, 9], [0] * 4)
    at = [0, 5, 0, 9]
    for _ in range(9):
        graph.replay()
        want, bad = B16.plan(s.table, s.held, s.free, 40, 8, 12, at, [3, 1, 0, 2])
        at = want["ends"]
        assert not bad and rows.ends.tolist() == at and rows.row_pos.tolist() == want["row_pos"]
        assert s.gpu.block_table.tolist() == s.table and s.gpu.held.tolist() == s.held
    assert status(s5) == 0


@pytest.mark.parametrize("B, pt, N", [(3, 16, 64), (40, 8, 300), (600, 24, 3000)])
def test_the_stack_above_its_top(s5, B, pt, N):  # noqa: F811
    """Entries of the stack past the pages that lay on it and those given back stay as they were."""
    rng = random.Random(B)
    table_len = 20
    num = 3 * B * table_len
    order = list(range(num))
    rng.shuffle(order)
    lengths = [rng.randint(0, table_len * pt // 2) for _ in range(B)]
    s = Slots(s5, num, pt, table_len, [-(-n // pt) for n in lengths], order, free=B * table_len)
    s.gpu.free_pages[len(s.free):] = torch.arange(-1000, -1000 - num + len(s.free), -1, dtype=torch.int32, device="cuda")
    for _ in range(4):
        lengths = [0 if rng.random() < 0.3 else rng.randint(0, n) for n in lengths]
        new = [rng.randint(0, min(table_len * pt - n, 2 * N // B // 2)) for n in lengths]
        top, held = len(s.free), list(s.held)
        want, above = s.step(N, lengths, new)
        given = sum(max(0, a - b) for a, b in zip(held, s.held))
        assert s.gpu.free_pages.tolist()[top + given:] == above[top + given:]
        lengths = want["ends"]
