"""hpa_assign_pages against the definition, exactly: every array after every step."""
import random

import pytest
import torch

import load_balanced_split_gb300 as hpa
from oracle import paging

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


class Both:
    """A PageTable and the oracle's state, stepped together."""

    def __init__(self, P, rows, stride, max_batch, max_tokens):
        self.pt = hpa.PageTable(P, rows, stride, max_batch, max_tokens)
        self.pt.table.fill_(-7)
        self.pt.page_indices.fill_(-7)
        self.P, self.max_tokens = P, max_tokens
        self.state = ([[-7] * stride for _ in range(rows)], [0] * rows, list(range(P - 1, -1, -1)))

    def step(self, lens, new=None, rows=None, offset=None, stream=None):
        pt = self.pt
        pt.status.zero_()
        before = pt.page_indices.tolist()
        pt.assign(_i32(lens), None if new is None else _i32(new), None if rows is None else _i32(rows),
                  None if offset is None else _i32(offset))
        self.state, (indptr, ix), (slots, pos), status = paging.assign(
            lens, new, *self.state, self.P, rows, offset, None if new is None else self.max_tokens)
        table, held, free = self.state
        assert pt.status.item() == status
        assert pt.held.tolist() == held and pt.table.tolist() == table
        assert pt.free_count.item() == len(free)
        assert pt.free_pages[:len(free)].tolist() == free
        assert pt.page_indptr.tolist() == indptr
        assert pt.page_indices.tolist() == ix + before[len(ix):]
        if new is not None:
            assert pt.slots.tolist() == slots and pt.positions.tolist() == pos
        return status


@pytest.mark.parametrize("rows,stride,P,max_tokens", [(1, 1, 1, 3), (5, 4, 12, 40), (33, 20, 300, 500),
                                                      (200, 7, 500, 100), (1500, 3, 2500, 900)])
@pytest.mark.parametrize("mapped", [False, True])
def test_random_steps(rows, stride, P, max_tokens, mapped):
    rng = random.Random(rows + 7 * mapped)
    both = Both(P, rows, stride, rows, max_tokens)
    for it in range(25 if rows < 1000 else 6):
        B = rng.choice([1, rows, rng.randint(1, rows)])
        which = rng.sample(range(rows), B) if mapped else None
        lens = [rng.choice([0, 64 * rng.randint(0, stride), rng.randint(0, 64 * stride)])
                for _ in range(B)]
        new = [rng.randint(0, min(x, rng.choice([1, 3, 70, 64 * stride]))) for x in lens]
        both.step(lens, new if it % 5 else None, which,
                  [rng.randint(-5, 1000) for _ in range(B)] if it % 3 == 0 else None)


def test_pool_too_small():
    """Requests are served in order while the pages last; later ones with pages enough go on."""
    both = Both(10, 6, 8, 6, 80)
    assert both.step([64 * 4, 64 * 4, 64, 0, 0, 0], [1, 1, 1, 0, 0, 0]) == 0
    assert both.step([64 * 5, 64 * 5, 64, 1, 0, 64], [64, 1, 1, 1, 0, 1]) == paging.NO_PAGES
    assert both.step([64, 64 * 7, 64, 64 * 2, 1, 64], [1, 1, 1, 1, 1, 1]) == paging.NO_PAGES
    assert both.step([0, 64 * 8, 0, 64 * 2, 0, 0], [0, 2, 0, 1, 0, 0]) == 0


def test_long_requests():
    both = Both(9000, 3, 6000, 3, 300000)
    both.step([64 * 5000 + 1, 1, 64 * 3000 - 5], [200000, 1, 100000])
    both.step([0, 64 * 4444 + 3, 0], [0, 64 * 4000, 0])        # pages returned and taken at once
    both.step([64 * 6000, 3, 64 * 1001], [1, 0, 64])
    both.step([64 * 6000 + 1, 5, 9], [1, 0, 0])                # beyond its row of the table


def test_lengths_and_counts_out_of_range():
    """A bad request keeps its pages, the others are served."""
    both = Both(40, 6, 5, 6, 50)
    both.step([64, 100, 200, 300, 5, 9], [1, 2, 3, 4, 5, 6])
    bad = both.step([-1, 101, 201, 301, 64 * 5 + 1, 10], [0, -3, 202, 1, 1, 1])
    assert bad == paging.BAD_SEQLEN | paging.OVERFLOW
    assert both.step([1, 2, 3, 4, 5, 6], None, [0, 9, -1, 0, 2, 2]) == paging.BAD_MAP
    assert both.step([65, 65, 65], [60, 0, 65], [3, 3, 4]) == paging.BAD_MAP | paging.OVERFLOW
    both.pt.status.zero_()                                     # more tokens than there is room for
    both.pt.assign(_i32([-2 ** 31, 2 ** 31 - 1, 64]), _i32([0, 2 ** 31 - 1, 2 ** 31 - 1]))
    assert both.pt.status.item() == paging.BAD_SEQLEN | paging.OVERFLOW
    assert both.pt.held.tolist() == both.state[1] and set(both.pt.slots.tolist()) == {-1}
    both.pt.held[4] = 6                                        # a damaged count
    both.state[1][4] = 6
    assert both.step([70, 70], [1, 1], [4, 5]) == paging.BAD_MAP


@pytest.mark.parametrize("rows", [8192, 8193])
def test_rows_listed_twice_in_large_tables(rows):
    """Tables on both sides of the size up to which shared memory tells who owns a row."""
    rng = random.Random(rows)
    both = Both(6000, rows, 3, 1300, 2000)
    for B in (1300, 900, 1024):
        which = [rng.choice([rng.randrange(rows), rng.randrange(40), -1, rows]) for _ in range(B)]
        lens = [rng.randint(0, 192) for _ in range(B)]
        assert both.step(lens, [min(x, 1) for x in lens], which) == paging.BAD_MAP


def test_damaged_stack_is_reported_and_nothing_is_written_past_it():
    pt = hpa.PageTable(8, 2, 8, max_tokens=70)
    pt.assign(_i32([64 * 3, 64]), _i32([1, 1]))
    guard = pt.free_pages.clone()
    for count in (-3, 9, 1000000):
        pt.free_count.fill_(count)
        pt.status.zero_()
        pt.assign(_i32([64 * 3, 64]), _i32([0, 0]))
        assert pt.status.item() == 32 and torch.equal(pt.free_pages, guard)
        assert 0 <= pt.free_count.item() <= 8
    pt.free_count.fill_(8)          # pages both held and free: what does not fit is not pushed
    pt.status.zero_()
    pt.assign(_i32([0, 64]))
    assert pt.status.item() == 32 and pt.free_count.item() == 8
    pt.free_pages.fill_(99)         # ids out of range
    pt.status.zero_()
    pt.assign(_i32([70, 70]), _i32([70, 70]))
    assert pt.status.item() & 4
    s = pt.slots.tolist()
    assert all(-1 <= x < 8 * 64 for x in s)


def test_lists_longer_than_their_room_are_cut():
    pt = hpa.PageTable(20, 3, 8, max_tokens=4)
    ix = torch.full((9,), -7, dtype=torch.int32, device="cuda")
    hpa.hpa_assign_pages(_i32([200, 200, 200]), None, pt.table, pt.held, pt.free_pages,
                         pt.free_count, pt.page_indptr, ix[:6], None, None, pt.workspace,
                         status=pt.status)
    assert pt.status.item() == 16 and pt.page_indptr.tolist() == [0, 4, 6, 6]
    assert ix.tolist()[6:] == [-7] * 3 and ix.tolist()[:6] == [0, 1, 2, 3, 4, 5]
    pt.status.zero_()
    pt.assign(_i32([200, 200, 200]), _i32([3, 3, 3]))
    assert pt.status.item() == 16 and pt.slots.tolist() == [3 * 64 + 5, 3 * 64 + 6, 3 * 64 + 7,
                                                            7 * 64 + 5]


def test_a_step_taken_again_from_the_state_before_it():
    """held_out and free_count_out: draft tokens rejected, the same step with shorter lengths."""
    pt = hpa.PageTable(64, 4, 16, max_tokens=400)
    pt.assign(_i32([60, 128, 700, 0]))
    table, held, count = pt.table.clone(), pt.held.clone(), pt.free_count.clone()
    for lens in ([70, 0, 900, 5], [61, 129, 701, 0], [61, 129, 64, 65]):
        new_held, new_count = pt.held.clone(), torch.zeros_like(count)
        hpa.hpa_assign_pages(_i32(lens), _i32([1, 0, 1, 0]), pt.table, pt.held, pt.free_pages,
                             pt.free_count, pt.page_indptr, pt.page_indices, pt.slots, pt.positions,
                             pt.workspace, held_out=new_held, free_count_out=new_count,
                             status=pt.status)
        assert torch.equal(pt.held, held) and torch.equal(pt.free_count, count)
        ref = hpa.PageTable(64, 4, 16, max_tokens=400)
        ref.assign(_i32([60, 128, 700, 0]))
        ref.assign(_i32(lens), _i32([1, 0, 1, 0]))
        assert torch.equal(new_held, ref.held) and torch.equal(new_count, ref.free_count)
        assert torch.equal(pt.page_indptr, ref.page_indptr) and torch.equal(pt.slots, ref.slots)
        n = int(pt.page_indptr[-1])
        assert torch.equal(pt.page_indices[:n], ref.page_indices[:n])
        for r, h in enumerate(held.tolist()):
            assert torch.equal(pt.table[r, :h], table[r, :h])
    assert pt.status.item() == 0


def test_captured_and_replayed_on_a_stream():
    both = Both(400, 16, 12, 16, 64)
    pt, rng = both.pt, random.Random(5)
    lens, new, rows = (torch.zeros(16, dtype=torch.int32, device="cuda") for _ in range(3))
    state = [0] * 16
    side = torch.cuda.Stream()
    pt.assign(lens, new, rows + torch.arange(16, device="cuda", dtype=torch.int32))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pt.assign(lens, new, rows)
    for _ in range(10):
        which = rng.sample(range(16), 16)
        add = [rng.choice([0, 1, 4]) for _ in range(16)]
        state = [0 if rng.random() < 0.1 else min(x + a, 64 * 12) for x, a in zip(state, add)]
        a = [min(x, y) for x, y in zip(add, state)]
        lens.copy_(_i32(state[r] for r in which))
        new.copy_(_i32(a[r] for r in which))
        rows.copy_(_i32(which))
        graph.replay()
        torch.cuda.synchronize()
        both.state, (indptr, ix), (slots, pos), status = paging.assign(
            lens.tolist(), new.tolist(), *both.state, 400, which, None, 64)
        assert pt.held.tolist() == both.state[1] and pt.page_indptr.tolist() == indptr
        assert pt.slots.tolist() == slots and pt.positions.tolist() == pos
        assert pt.page_indices.tolist()[:len(ix)] == ix and pt.status.item() == status == 0
