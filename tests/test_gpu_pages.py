"""GPU tests of the page steps of a paged cache against their definition, request by request on the
host, and of a sequence of steps, releases among them, in which no page is held twice."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def rope():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import packed_varlen_rotary_rope_amd as m
    return m


def int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def reference(ring, state, table, held, new, T, page):
    """The step of kv_pages.h; `table` (a list of lists) is written."""
    first, count = state[0] % len(ring), min(max(state[1], 0), len(ring))
    per = len(table[0]) if table else 0
    asked = used = tokens = 0
    cu, lens, after = [0], [], []
    positions, slots = [-1] * T, [-1] * T
    for s, (h, n) in enumerate(zip(held, new)):
        h0, h, n = h, max(h, 0), max(n, 0)
        start = tokens
        tokens += n
        cu.append(min(tokens, T))
        has, needs = -(-h // page), -(-(h + n) // page)
        fits = h + n < 2 ** 31 - 1 - 4096 and needs <= per
        wants = needs - has if n > 0 and fits else 0
        asked += wants
        if n > 0 and not (fits and tokens <= T and (wants == 0 or asked <= count)):
            lens.append(0)
            after.append(h0)
            continue
        for x in range(wants):
            table[s][has + x] = ring[(first + used) % len(ring)]
            used += 1
        lens.append(h + n)
        after.append(h + n if n > 0 else h0)
        for i in range(n):
            p = h + i
            number = table[s][p // page]
            positions[start + i] = p
            slots[start + i] = number * page + p % page if number >= 0 else -1
    return cu, lens, after, positions, slots, [(first + used) % len(ring), count - used], table


def compare(rope, ring, state, table, held, new, T, page):
    want = reference(ring, state, [list(r) for r in table], held, new, T, page)
    dev_table = int32(table).view(len(table), -1)
    pool = rope.PagePool(int32(ring), int32(state))
    dev_held = int32(held)
    step = rope.page_step(pool, dev_table, dev_held, int32(new), T, page)
    torch.cuda.synchronize()
    got = (step.cu_seqlens, step.kv_lens, step.held, step.positions, step.slots, step.state)
    for name, a, b in zip(step._fields[:4] + ("slots", "state"), got, want):
        assert a.tolist() == b, name
    assert dev_table.tolist() == want[6]
    assert pool.ring.tolist() == list(ring) and pool.state.tolist() == list(state) and dev_held.tolist() == list(held)


def random_step(seed, B, page, most_held, most_new, free, turned=True):
    rng = random.Random(seed)
    held = [rng.randint(0, most_held) for _ in range(B)]
    new = [rng.choice([0, 1, 1, rng.randint(0, most_new)]) for _ in range(B)]
    has = [-(-h // page) for h in held]
    per = max([1] + [-(-(h + n) // page) for h, n in zip(held, new)])
    wants = sum(-(-(h + n) // page) - a for h, n, a in zip(held, new, has))
    count = int(wants * free) if free < 1 else wants + rng.randint(0, 9)
    total = sum(has) + count + 1
    numbers = list(range(total))
    rng.shuffle(numbers)
    table, at = [], 0
    for a in has:
        table.append(numbers[at:at + a] + [-1] * (per - a))
        at += a
    first = rng.randrange(total) if turned else 0
    ring = [-5] * total
    for i in range(count):
        ring[(first + i) % total] = numbers[at + i]
    return ring, [first, count], table, held, new, sum(new), page


STEPS = [(1, 1, 16, 100, 1, 1.0), (2, 64, 16, 5000, 1, 1.0), (3, 7, 1, 20, 9, 1.0), (4, 300, 48, 900, 300, 1.0),
         (5, 1023, 8, 60, 3, 1.0), (6, 1025, 64, 500, 40, 0.6), (7, 5000, 16, 200, 5, 1.0), (8, 40, 7, 300, 3000, 0.3),
         (9, 3, 128, 0, 5000, 1.0), (10, 4097, 256, 1000, 2, 0.0), (11, 2, 16, 40000, 40000, 1.0)]


@pytest.mark.parametrize("case", STEPS, ids=str)
def test_against_the_definition(rope, case):
    print(f"[page_step] {case}", flush=True)
    compare(rope, *random_step(*case))


def test_refused_for_its_row_of_the_table_and_for_its_rows(rope):
    ring, state = [9, 8, 7, 6, 5, 4, 3], [2, 5]
    # the second needs more pages than its row has and asks for none, the others go on
    compare(rope, ring, state, [[1, -1, -1], [0, 2, -1], [-1, -1, -1]], [16, 32, 0], [20, 30, 2], 52, 16)
    # the tokens of the last two do not all lie in the rows; one without new tokens is served
    compare(rope, ring, state, [[1, -1, -1], [0, 2, -1], [-1, -1, -1], [1, -1, -1]], [16, 32, 0, 5], [2, 3, 4, 0], 8, 16)
    # rows of no sequence, negative lengths
    compare(rope, ring, state, [[1, -1], [0, 2], [-1, -1]], [16, -3, 0], [1, 5, -7], 40, 16)
    # no page is free, and two of them need none
    compare(rope, ring, [3, 0], [[1, -1], [0, -1], [2, 6]], [15, 16, 20], [1, 1, 12], 14, 16)
    # more tokens than numbers of 32 bits count
    compare(rope, ring, state, [[1, -1]] * 5, [2 ** 31 - 1, 5, 0, 2 ** 31 - 4097, 3],
            [2, 2 ** 31 - 1, 2 ** 31 - 1, 1, 2 ** 31 - 1], 30, 2 ** 30)


def test_state_of_any_contents_is_safe(rope):
    for state in ([-1, 5], [2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, -2 ** 31], [100, 3]):
        table, held = int32([[1, -1, -1]]), int32([3])
        pool = rope.PagePool(int32([4, 5, 6, -2]), int32(state))
        step = rope.page_step(pool, table, held, int32([40]), 40, 16)
        assert step.positions.numel() == 40 and -1 <= int(step.slots.min()) and int(step.slots.max()) < 7 * 16
        rope.page_release_(pool, table, held, torch.tensor([True], device=DEV), 16)
        assert 0 <= int(pool.state[0]) < 4 and 0 <= int(pool.state[1]) <= 4


def test_no_sequences_and_no_rows(rope):
    pool = rope.page_pool(4)
    e = int32([])
    step = rope.page_step(pool, torch.empty((0, 3), dtype=torch.int32, device=DEV), e, e, 5, 16)
    assert step.cu_seqlens.tolist() == [0] and step.slots.tolist() == [-1] * 5 and step.state.tolist() == [0, 4]
    step = rope.page_step(pool, int32([[2, 3]]), int32([20]), int32([0]), 0, 16)
    assert step.cu_seqlens.tolist() == [0, 0] and step.kv_lens.tolist() == [20] and step.held.tolist() == [20]
    rope.page_release_(pool, torch.empty((0, 3), dtype=torch.int32, device=DEV), e, torch.empty(0, dtype=torch.bool, device=DEV), 16)
    assert pool.state.tolist() == [0, 4]


def test_rows_of_a_wider_table(rope):
    """Rows further apart than they are long: what lies between stays as it is."""
    wide = torch.full((3, 10), 77, dtype=torch.int32, device=DEV)
    step = rope.page_step(rope.page_pool(9), wide[:, 2:6], int32([0, 0, 0]), int32([33, 1, 64]), 98, 16)
    assert wide.tolist() == [[77, 77, 0, 1, 2, 77, 77, 77, 77, 77], [77, 77, 3] + [77] * 7,
                             [77, 77, 4, 5, 6, 7, 77, 77, 77, 77]]
    assert step.state.tolist() == [8, 1]


def test_a_service(rope):
    """Requests that come, grow and end: whatever is refused, no page is held twice and none is lost."""
    rng = random.Random(5)
    B, page, per, pages = 60, 8, 12, 260
    pool, table = rope.page_pool(pages), torch.full((B, per), -1, dtype=torch.int32, device=DEV)
    held = int32([0] * B)
    refused = 0
    out = [None, None]
    for turn in range(40):
        lens = held.tolist()
        new = [rng.choice([1, 1, 0]) if h else rng.randint(0, 60) for h in lens]
        T = sum(new) + rng.randint(0, 3)
        gone = torch.tensor([h > 0 and rng.random() < 0.15 for h in lens], device=DEV)
        rope.page_release_(pool, table, held, gone, page)
        lens = held.tolist()
        new = [n if h or n != 1 else 0 for h, n in zip(lens, new)]
        step = rope.page_step(pool, table, held, int32(new), T, page)
        refused += sum(n > 0 and k == 0 for n, k in zip(new, step.kv_lens.tolist()))
        pool.state, held = step.state, step.held.clone()
        # the pages of each sequence and the free ones are all pages, each once
        rows, first, count = table.tolist(), *pool.state.tolist()
        mine = [rows[s][i] for s, h in enumerate(held.tolist()) for i in range(-(-h // page))]
        free = [pool.ring.tolist()[(first + i) % pages] for i in range(count)]
        assert sorted(mine + free) == list(range(pages)), turn
        slots = [x for x in step.slots.tolist() if x >= 0]
        assert len(set(slots)) == len(slots) and all(x // page in set(mine) for x in slots)
    assert refused > 0  # the pool was too small now and then


def test_refusals(rope):
    pool, table, held, new = rope.page_pool(8), int32([[0, -1], [1, -1]]), int32([3, 4]), int32([1, 1])
    good = rope.page_step(pool, table, held, new, 2, 16)
    with pytest.raises(TypeError):
        rope.page_step(table, table, held, new, 2, 16)
    with pytest.raises(TypeError):
        rope.page_step(pool, table.long(), held, new, 2, 16)
    with pytest.raises(TypeError):
        rope.page_step(pool, table, held.long(), new, 2, 16)
    with pytest.raises(ValueError):
        rope.page_step(pool, table[:1], held, new, 2, 16)
    with pytest.raises(ValueError):
        rope.page_step(pool, table, held[:1], new, 2, 16)
    with pytest.raises(ValueError):
        rope.page_step(pool, table[:1].expand(2, 2), held, new, 2, 16)
    for T, page in ((-1, 16), (2 ** 31, 16), (2, 0)):
        with pytest.raises(ValueError):
            rope.page_step(pool, table, held, new, T, page)
    with pytest.raises(ValueError, match="sizes"):
        rope.page_step(pool, table, held, new, 3, 16, out=good)
    with pytest.raises(ValueError, match="read"):
        rope.page_step(pool, table, good.held, new, 2, 16, out=good)
    with pytest.raises(ValueError, match="read"):
        rope.page_step(rope.PagePool(pool.ring, good.state), table, held, new, 2, 16, out=good)
    with pytest.raises(TypeError):
        rope.page_release_(pool, table, held, new, 16)
    with pytest.raises(ValueError):
        rope.PagePool(pool.ring, int32([0]))


def test_captured_steps(rope):
    """A step and the taking over of its result in a graph: every replay goes one token further."""
    B, page, T = 5, 4, 5
    pool, table, held = rope.page_pool(40), torch.full((B, 8), -1, dtype=torch.int32, device=DEV), int32([0] * B)
    new = int32([1] * B)
    out = rope.page_step(pool, table.clone(), held, new, T, page)  # its buffers

    def step():
        rope.page_step(pool, table, held, new, T, page, out=out)
        pool.state.copy_(out.state)
        held.copy_(out.held)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(2, 12):
        graph.replay()
        torch.cuda.synchronize()
        assert held.tolist() == [i] * B and out.kv_lens.tolist() == [i] * B and out.positions.tolist() == [i - 1] * B
        rows = table.tolist()
        n = -(-i // page)
        assert sorted(x for r in rows for x in r[:n]) == list(range(B * n))
        assert out.slots.tolist() == [r[(i - 1) // page] * page + (i - 1) % page for r in rows]
