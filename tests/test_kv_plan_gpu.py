"""kv_plan against a plain sequential restatement: lengths, starts, pages, the stack of free pages, slots and refusals."""
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import qmoe_mnb_matmul_gb300 as mnb  # noqa: E402

CONTENT = 7


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def plain(held, keep, new, table, stack, num_pages, page, columns, budget):
    """The same step, one sequence after the other.  `stack`: the free pages, the top last."""
    need = [-(-(k + n) // page) for k, n in zip(keep, new)]
    impossible = [n > 0 and (w > columns or k + n > 2 ** 31 - 4097) for k, n, w in zip(keep, new, need)]
    table, stack = [list(r) for r in table], list(stack)
    back = []
    for b, w in enumerate(need):
        if not impossible[b] and w < held[b]:
            back += table[b][w:held[b]]
    stack += reversed(back)
    room, asked_pages, asked_tokens = len(stack), 0, 0
    out = {"held": [], "lens": [], "start": [0], "refused": [], "slots": []}
    for b in range(len(held)):
        n, w, h = new[b], need[b], held[b]
        grow = 0 if impossible[b] else max(w - h, 0)
        if not impossible[b]:
            asked_pages += grow
            asked_tokens += n
        refused = impossible[b] or (n > 0 and ((grow > 0 and asked_pages > room) or asked_tokens > budget))
        if refused:
            n = 0
        elif grow:
            for c in range(h, w):
                table[b][c] = stack.pop()
        out["held"].append(h if impossible[b] or (refused and grow) else w)
        out["lens"].append(keep[b] + n)
        out["start"].append(out["start"][-1] + n)
        out["refused"].append(int(refused))
        for pos in range(keep[b], keep[b] + n):
            p = table[b][pos // page]
            out["slots"].append(p * page + pos % page if 0 <= p < num_pages else -1)
    return {**out, "table": table, "stack": stack}


class Pool:
    def __init__(self, held, columns, spare, page, seed=0, stride=None):
        r = random.Random(seed)
        pages = list(range(sum(held) + spare))
        r.shuffle(pages)
        self.page, self.columns, self.num = page, columns, len(pages)
        self.held, self.rows = list(held), []
        for h in held:
            self.rows.append(pages[:h] + [-7] * (columns - h))
            pages = pages[h:]
        self.stack = pages
        wide = torch.full((len(held), stride or columns), -9, dtype=torch.int32, device="cuda")
        wide[:, :columns] = i32(self.rows).view(len(held), columns)
        self.wide, self.table = wide, wide[:, :columns]
        self.free = i32(pages + [-3] * (self.num - len(pages)))
        self.held_dev, self.count = i32(held), i32([len(pages)])

    def step(self, keep, new, budget=None, inplace=False, slots=True, max_tokens=None):
        """Runs kv_plan, compares everything with plain(), and takes the new state over."""
        batch = len(self.held)
        budget = sum(new) + 3 if budget is None else budget
        want = plain(self.held, keep, new, self.rows, self.stack, self.num, self.page, self.columns,
                     budget if max_tokens is None else max_tokens)
        held_out = self.held_dev if inplace else torch.full_like(self.held_dev, -1)
        count_out = self.count if inplace else torch.full_like(self.count, -1)
        pool = mnb.kv_pool(self.held_dev, self.table, self.free, self.count, self.page, held_out=held_out,
                           free_count_out=count_out)
        keep_dev, new_dev = i32(keep), i32(new)
        lens = keep_dev if inplace else torch.full((batch,), -1, dtype=torch.int32, device="cuda")
        refused = new_dev if inplace else torch.full((batch,), -1, dtype=torch.int32, device="cuda")
        start = torch.full((batch + 1,), -1, dtype=torch.int32, device="cuda")
        free_before = self.free.clone()
        got_slots = torch.full((budget,), -77, dtype=torch.int64, device="cuda") if slots else None
        mnb.kv_plan(pool, keep_dev, new_dev, lens, start, slots=got_slots,
                    max_tokens=max_tokens if slots else budget, refused=refused)
        assert mnb.mnb_get_last_device_error() == 0
        assert held_out.tolist() == want["held"]
        assert lens.tolist() == want["lens"]
        assert start.tolist() == want["start"]
        assert refused.tolist() == want["refused"]
        assert self.table.tolist() == want["table"]
        assert (self.wide[:, self.columns:] == -9).all()
        n = int(count_out)
        assert self.free[:n].tolist() == want["stack"]
        behind = max(n, len(self.stack))  # what lies behind the stack, then and now, is left alone
        assert torch.equal(self.free[behind:], free_before[behind:])
        if slots:
            total = want["start"][-1]
            assert got_slots[:total].tolist() == want["slots"]
            assert (got_slots[total:] == -77).all()
        self.held, self.rows, self.stack = want["held"], want["table"], want["stack"]
        self.held_dev, self.count = held_out, count_out
        return want


@pytest.mark.parametrize("batch,page,columns,most,spare,inplace", [
    (1, 16, 4, 1, 0, False), (1, 16, 400, 5000, 400, True), (7, 8, 9, 20, 3, False), (64, 16, 30, 5, 40, True),
    (64, 24, 30, 100, 90, False), (257, 128, 12, 700, 300, True), (1000, 16, 60, 400, 5000, False),
    (1031, 32, 8, 3, 100, True), (1, 1, 50, 40, 60, False), (5000, 8, 4, 12, 2000, False), (8192, 8, 3, 9, 3000, True)])
def test_steps_in_a_row(batch, page, columns, most, spare, inplace):
    r = random.Random(batch * 31 + page)
    pool = Pool([r.randint(0, columns) for _ in range(batch)], columns, spare, page, seed=batch, stride=columns + batch % 3)
    for k in range(4):
        keep = [r.choice([h * page, r.randint(0, h * page), max(0, h * page - r.randint(0, 30)), 0]) for h in pool.held]
        new = [r.choice([0, 1, r.randint(0, most), r.randint(0, most)]) for _ in keep]
        total = sum(new)
        pool.step(keep, new, budget=[None, max(1, total // 2), total, total + 40000][k], inplace=inplace)


def test_a_step_that_drops_what_the_last_one_added_undoes_it():
    r = random.Random(5)
    pool = Pool([r.randint(0, 6) for _ in range(40)], 20, 300, 16)
    stack, held = list(pool.stack), list(pool.held)
    keep = [h * 16 - r.randint(0, 15) if h else 0 for h in held]
    pool.step(keep, [r.randint(0, 90) for _ in keep])
    assert pool.stack != stack
    pool.step(keep, [0] * 40)
    assert pool.stack == stack and pool.held == held


def test_refusals():
    pool = Pool([1, 2, 0, 1], 3, 2, 16)
    w = pool.step([10, 32, 0, 16], [7, 1, 17, 20])       # pages asked for: 1, 1, 2, 2; two are free
    assert w["refused"] == [0, 0, 1, 1]
    w = pool.step([17, 33, 0, 3], [1, 0, 1, 13])         # nothing free, but 13 tokens fit in the page held
    assert w["refused"] == [0, 0, 1, 0]
    w = pool.step([0, 20, 0, 16], [40, 30, 5, 0])        # row 1 is too long for the table and counts for nothing
    assert w["refused"][1] == 1
    w = pool.step(w["lens"], [1, 1, 1, 1], budget=2)     # two tokens of room
    assert w["refused"] == [0, 0, 1, 1]
    assert pool.step(w["lens"], [0, 0, 0, 0], budget=0)["refused"] == [0, 0, 0, 0]


def test_a_finished_sequence_feeds_the_others():
    pool = Pool([4, 0, 0], 8, 0, 16)
    w = pool.step([0, 0, 0], [0, 20, 30])
    assert w["refused"] == [0, 0, 0] and w["held"] == [0, 2, 2]


def test_without_slots_and_with_a_budget_below_their_length():
    pool = Pool([2, 2], 6, 8, 16)
    pool.step([30, 20], [9, 9], budget=18, slots=False)
    pool.step(pool_lens(pool, [39, 29]), [9, 9], budget=40, max_tokens=17)


def pool_lens(pool, lens):
    assert all(n <= h * pool.page for n, h in zip(lens, pool.held))
    return lens


def test_many_slots_have_a_grid_of_their_own():
    pool = Pool([0] * 30, 700, 12000, 16)
    r = random.Random(9)
    pool.step([0] * 30, [r.randint(0, 6000) for _ in range(30)])
    pool.step(pool_lens(pool, [h * 16 // 2 for h in pool.held]), [r.randint(0, 3000) for _ in range(30)], budget=20000)


def test_no_sequences():
    held = torch.zeros(0, dtype=torch.int32, device="cuda")
    table = torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    free, count, start = i32([5, 6]), i32([2]), i32([9])
    pool = mnb.kv_pool(held, table, free, count, 16)
    mnb.kv_plan(pool, held, held, held, start)
    assert start.tolist() == [0] and count.tolist() == [2]


def test_entries_outside_their_range_are_cut_and_reported():
    def run(held, keep, new, count, table, free, slots=6):
        pool = mnb.kv_pool(i32(held), table, free, i32([count]), 8, held_out=i32([0] * len(held)), free_count_out=i32([0]))
        lens, start, s = i32([0] * len(held)), i32([0] * (len(held) + 1)), torch.full((slots,), -5, device="cuda").long()
        mnb.kv_plan(pool, i32(keep), i32(new), lens, start, slots=s)
        return lens.tolist(), start.tolist(), s.tolist(), pool.tensors[4].tolist(), mnb.mnb_get_last_device_error()

    table = lambda: i32([[2, 1, -1], [3, -1, -1]])  # noqa: E731
    good = run([2, 1], [9, 8], [1, 1], 2, table(), i32([0, 4, 9, 9, 9]))
    assert good == ([10, 9], [0, 1, 2], [9, 32, -5, -5, -5, -5], [2, 2], 0)
    assert run([2, 1], [17, 8], [0, -3], 2, table(), i32([0, 4, 9, 9, 9]))[::4] == ([16, 8], CONTENT)
    assert run([2, 1], [-1, 8], [1, 0], 2, table(), i32([0, 4, 9, 9, 9]))[::4] == ([1, 8], CONTENT)
    assert run([4, 1], [24, 8], [0, 0], 2, table(), i32([0, 4, 9, 9, 9]))[3:] == ([3, 1], CONTENT)
    assert run([2, 1], [9, 8], [0, 0], 99, table(), i32([0, 4, 9, 9, 9]))[4] == CONTENT
    lens, start, slots, _, err = run([2, 1], [9, 8], [1, 1], 2, i32([[2, 50, -1], [3, -1, -1]]), i32([0, 4, 9, 9, 9]))
    assert (lens, slots[:2], err) == ([10, 9], [-1, 32], CONTENT)


def test_captured_and_replayed_on_another_stream():
    pool = Pool([2] * 9, 12, 60, 16)
    keep, new = i32([32] * 9), i32([3] * 9)
    start, slots = i32([0] * 10), torch.full((40,), -1, dtype=torch.int64, device="cuda")
    d = mnb.kv_pool(pool.held_dev, pool.table, pool.free, pool.count, 16)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        mnb.kv_plan(d, keep, new, keep, start, slots=slots)
    lens, rows, stack, held = [32] * 9, pool.rows, pool.stack, pool.held
    for n in (3, 1, 20):
        new.fill_(n)
        graph.replay()
        want = plain(held, lens, [n] * 9, rows, stack, pool.num, 16, 12, 40)
        lens, rows, stack, held = want["lens"], want["table"], want["stack"], want["held"]
        assert keep.tolist() == lens and pool.held_dev.tolist() == held and pool.table.tolist() == rows
        assert slots[:want["start"][-1]].tolist() == want["slots"]
        assert pool.free[:int(pool.count)].tolist() == stack
    assert mnb.mnb_get_last_device_error() == 0
