"""GPU tests of the release of pages against its definition on the host: many sequences, full rings, lengths
that no sequence has."""
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


def reference(ring, state, table, held, gone, page):
    """The release of kv_pages.h, in place."""
    pages = len(ring)
    first, count = state[0] % pages, min(max(state[1], 0), pages)
    for s, g in enumerate(gone):
        if g:
            for number in table[s][:max(-(-held[s] // page), 0)]:
                if count < pages:
                    ring[(first + count) % pages] = number
                    count += 1
            held[s] = 0
    state[:] = first, count


def compare(rope, ring, state, table, held, gone, page):
    pool = rope.PagePool(int32(ring), int32(state))
    dev_table, dev_held = int32(table).view(len(table), -1), int32(held)
    rope.page_release_(pool, dev_table, dev_held, torch.tensor(gone, dtype=torch.bool, device=DEV), page)
    ring, state, held = list(ring), list(state), list(held)
    reference(ring, state, table, held, gone, page)
    assert pool.state.tolist() == state and dev_held.tolist() == held
    assert pool.ring.tolist() == ring
    assert dev_table.tolist() == [list(r) for r in table]


CASES = [  # seed, B, page, most held, share that is gone, free before, room for all
    (1, 1, 16, 100, 1.0, 0, True), (2, 64, 1, 90, 0.5, 30, True), (3, 1024, 16, 40, 0.5, 100, True),
    (4, 1025, 16, 300, 0.7, 5, True), (5, 3000, 8, 100, 1.0, 50, True), (6, 3000, 16, 400, 0.3, 0, True),
    (7, 2500, 4, 60, 0.9, 200, False), (8, 5, 16, 40000, 1.0, 10, True), (9, 5, 16, 40000, 1.0, 10, False),
    (10, 2049, 16, 50, 0.0, 40, True)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_the_definition(rope, case):
    seed, B, page, most, share, free, room = case
    print(f"[page_release] {case}", flush=True)
    rng = random.Random(seed)
    held = [rng.choice([0, rng.randint(0, most)]) for _ in range(B)]
    gone = [rng.random() < share for _ in range(B)]
    has = [-(-h // page) for h in held]
    per = max([1] + has) + 1
    numbers = list(range(max(sum(has) + free, 1)))  # a pool has a page at least
    rng.shuffle(numbers)
    total = len(numbers) if room else free + sum(has) // 3 + 1
    table, at = [], free
    for a in has:
        table.append(numbers[at:at + a] + [-1] * (per - a))
        at += a
    first = total - min(total, 3)  # the free ones and those that come back go past the ring's end
    ring = [-5] * total
    for i in range(free):
        ring[(first + i) % total] = numbers[i]
    compare(rope, ring, [first, free], table, held, gone, page)


def test_lengths_that_no_sequence_has(rope):
    """Negative ones hold nothing, ones past the table's row the row's pages, a full ring takes none."""
    table = [[4, 5], [6, 7], [8, 9], [10, 11]]
    gone = [True, True, False, True]
    for state in ([5, 2], [0, 0], [7, 8], [-1, 7], [2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, -2 ** 31]):
        first = state[0] % 2 ** 32  # as the kernel takes a place in the ring
        compare(rope, list(range(20, 28)), [first % 8, state[1]], table, [-3, 2 ** 31 - 1, 2 ** 31 - 1, 17], gone, 16)
        pool = rope.PagePool(int32(list(range(20, 28))), int32(state))
        rope.page_release_(pool, int32(table), int32([-3, 2 ** 31 - 1, 2 ** 31 - 1, 17]),
                           torch.tensor(gone, device=DEV), 16)
        assert pool.state.tolist() == [first % 8, min(max(state[1], 0) + 4, 8)]


def test_what_comes_back_is_given_again(rope):
    """3000 sequences leave and as many come: they get the pages that were free first, then those given back."""
    B, page = 3000, 16
    table = torch.full((B, 4), -1, dtype=torch.int32, device=DEV)
    pool, held = rope.page_pool(3 * B + 50), int32([0] * B)
    step = rope.page_step(pool, table, held, int32([40] * B), 40 * B, page)
    pool.state, held = step.state, step.held
    rope.page_release_(pool, table, held, torch.ones(B, dtype=torch.bool, device=DEV), page)
    assert pool.state.tolist() == [3 * B, 3 * B + 50] and not bool(held.any())
    step = rope.page_step(pool, table, held, int32([40] * B), 40 * B, page)
    want = (torch.arange(3 * B, 6 * B, device=DEV) % (3 * B + 50)).view(B, 3)
    # the ring holds the pages in the order in which they came back, which is that of the sequences
    ring = pool.ring.long()
    assert torch.equal(table[:, :3].long(), ring[want])
    assert table[:, :3].flatten().unique().numel() == 3 * B
