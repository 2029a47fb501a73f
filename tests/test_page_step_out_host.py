"""What page_step accepts to be written over, without a GPU: calls go as far as the launch, which fails for
want of a device and is recorded, so that a step whose buffers the kernel would run past, or that it reads while
it writes them, is seen to be refused before any launch."""
import pytest
import torch

import packed_varlen_rotary_rope_amd as rope
from packed_varlen_rotary_rope_amd import attention as A

B, T, PAGES = 3, 10, 8
EINVAL = -1


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def kind(t):
    return f"{str(t.dtype)[6:]}_{t.numel()}_{t.stride(0)}_{t.device}"


@pytest.fixture
def launches(monkeypatch):
    if torch.cuda.is_available():
        pytest.skip("the launches of CPU tensors here are to fail")
    seen = []

    def call(device, fn, what, *args):
        status = fn(*args, None)
        if status == EINVAL:
            raise rope.RopeError(status, what)
        seen.append(what)

    monkeypatch.setattr(A, "_gpu", lambda device: None)
    monkeypatch.setattr(A, "_call", call)
    return seen


def args():
    pool = rope.PagePool(torch.arange(PAGES, dtype=torch.int32), torch.tensor([0, PAGES], dtype=torch.int32))
    return dict(pool=pool, block_table=i32(B, 4), held=i32(B), new_lens=i32(B), T=T, page_size=16)


def buffers(**kw):
    a = dict(cu_seqlens=i32(B + 1), kv_lens=i32(B), held=i32(B), positions=i32(T), state=i32(2),
             slots=torch.zeros(T, dtype=torch.int64))
    a.update(kw)
    return rope.PageStep(**a)


def test_steps_of_the_right_sizes(launches):
    a = args()
    step = rope.page_step(**a)
    assert rope.page_step(**{**a, "held": i32(B)}, out=step) is step
    own = buffers()
    assert rope.page_step(**a, out=own) is own
    # a view into a longer buffer of the caller's, and neighbours in one
    line = i32(100)
    rope.page_step(**a, out=buffers(cu_seqlens=line[:B + 1], kv_lens=line[B + 1:2 * B + 1], state=line[40:42]))
    a["held"], a["new_lens"] = line[:B], line[:B]  # inputs may be one
    rope.page_step(**a, out=own)
    assert launches == ["kv_page_step"] * 5


@pytest.mark.parametrize("name,value", [
    ("cu_seqlens", i32(B)), ("cu_seqlens", i32(B + 2)), ("cu_seqlens", torch.zeros(B + 1, dtype=torch.int64)),
    ("cu_seqlens", i32(2 * B + 2)[::2]), ("kv_lens", i32(B - 1)), ("kv_lens", torch.zeros(B, dtype=torch.int16)),
    ("held", i32(B - 1)), ("held", torch.zeros(B, dtype=torch.int16)), ("held", i32(1).expand(B)),
    ("positions", i32(T - 1)), ("positions", torch.zeros(T, dtype=torch.int64)), ("positions", i32(1).expand(T)),
    ("state", i32(1)), ("state", i32(3)), ("state", torch.zeros(2, dtype=torch.int16)),
    ("slots", i32(T)), ("slots", torch.zeros(T - 1, dtype=torch.int64)),
    ("slots", torch.zeros(1, dtype=torch.int64).expand(T)), ("slots", torch.zeros(T, dtype=torch.int64, device="meta")),
    ("kv_lens", torch.zeros(B, dtype=torch.int32, device="meta"))], ids=lambda x: x if isinstance(x, str) else kind(x))
def test_buffers_of_other_sizes_and_kinds_are_refused(launches, name, value):
    with pytest.raises((TypeError, ValueError)):
        rope.page_step(**args(), out=buffers(**{name: value}))
    assert not launches


def test_buffers_that_are_read_or_written_twice_are_refused(launches):
    a = args()
    own = buffers()
    line = i32(B + T + 4)
    pool = a["pool"]
    for kw, out in [
            ({"held": own.kv_lens}, own), ({"held": own.held}, own), ({"new_lens": own.held}, own),
            ({"new_lens": own.kv_lens}, own), ({"new_lens": own.cu_seqlens[1:]}, own),
            ({"new_lens": own.positions[4:4 + B]}, own), ({"held": own.cu_seqlens[:B]}, own),
            ({"pool": rope.PagePool(pool.ring, own.state)}, own),
            ({"pool": rope.PagePool(own.positions, pool.state)}, own),
            ({"block_table": own.positions[:2 * B].view(B, 2)}, own),
            ({"block_table": own.slots.view(torch.int32)[:4 * B].view(B, 4)}, own),
            ({}, buffers(kv_lens=line[:B], held=line[:B])), ({}, buffers(kv_lens=line[:B], positions=line[B - 1:B - 1 + T])),
            ({}, buffers(state=a["held"][:2])), ({}, buffers(held=a["block_table"].view(-1)[9:9 + B]))]:
        with pytest.raises((ValueError, rope.RopeError)):
            rope.page_step(**{**a, **kw}, out=out)
    table = i32(2 * B * 4)
    with pytest.raises(rope.RopeError):  # a table that reaches into the lengths, without `out`
        rope.page_step(**{**a, "block_table": table.view(2 * B, 4)[::2], "held": table[17:17 + B]})
    rope.page_step(**{**a, "block_table": table.view(2 * B, 4)[::2], "held": table[20:20 + B]})
    assert launches == ["kv_page_step"]


@pytest.mark.parametrize("ring", [torch.arange(PAGES), i32(2 * PAGES)[::2], i32(0), torch.zeros(4, dtype=torch.int32, device="meta")],
                         ids=kind)
def test_a_pool_that_was_changed_is_checked_again(launches, ring):
    pool = args()["pool"]
    with pytest.raises((TypeError, ValueError)):
        pool.ring = ring
    with pytest.raises((TypeError, ValueError)):
        rope.PagePool(ring, pool.state)
    assert pool.ring.tolist() == list(range(PAGES))


@pytest.mark.parametrize("state", [i32(1), i32(3), i32(4)[::2], torch.zeros(2), torch.zeros(2, dtype=torch.int32, device="meta")],
                         ids=kind)
def test_a_state_that_is_taken_over_is_checked(launches, state):
    pool = args()["pool"]
    with pytest.raises((TypeError, ValueError)):
        pool.state = state
    assert pool.state.tolist() == [0, PAGES]
