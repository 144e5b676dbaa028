"""kv8_plan against the host's bookkeeping, request by request: equal in
every value."""
import random

import numpy as np
import pytest
import torch

from tests import batch_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nvm():
    import nvfp4_w4a16_mtp_amd as nv
    return nv


def i32(a):
    return torch.tensor(list(a), dtype=torch.int32, device="cuda")


def compare(pool, host, plan, want, rows):
    cu, lens, pos, slots, missing = want
    n = cu[-1]
    assert plan.cu_rows.tolist() == cu and plan.kv_lens.tolist() == lens
    assert plan.positions[:n].tolist() == pos and plan.slots[:n].tolist() == slots
    assert int(plan.missing) == missing
    assert pool.held.tolist() == host.held and int(pool.free_count) == len(host.free)
    assert pool.free_pages[:len(host.free)].tolist() == host.free
    table = pool.block_table.cpu().numpy()
    assert np.array_equal(table, host.table)
    held = [int(table[b, i]) for b in range(table.shape[0]) for i in range(host.held[b])]
    assert sorted(held + host.free) == list(range(host.num_pages))    # every page once


@pytest.mark.parametrize("batch,page,max_pages,pages,steps", [(1, 16, 4, 3, 12), (5, 16, 9, 40, 20), (64, 32, 20, 700, 12),
                                                             (257, 64, 6, 900, 8), (1024, 16, 5, 3000, 5), (1025, 16, 7, 4000, 5),
                                                             (3000, 128, 3, 5000, 4)])
def test_many_steps(nvm, batch, page, max_pages, pages, steps):
    """Requests that grow, fall back, end and begin, in a pool that runs short."""
    r = random.Random(batch)
    pool, host = nvm.KV8Pool.empty(pages, batch, max_pages, page), ref.Pool(pages, batch, max_pages, page)
    lens = [0] * batch
    for _ in range(steps):
        kept = [x if r.random() < 0.5 else max(0, x - r.randint(0, 5)) for x in lens]
        new = [r.randint(0, 4) if r.random() < 0.8 else r.randint(0, max_pages * page) for _ in lens]
        for b in range(batch):
            if r.random() < 0.1:
                kept[b] = new[b] = 0
        rows = sum(min(n, max_pages * page - k) for k, n in zip(kept, new)) if r.random() < 0.7 else r.randint(0, 2 * batch)
        plan = nvm.kv8_plan(pool, i32(kept), i32(new), rows)
        compare(pool, host, plan, host.plan(kept, new, rows), rows)
        lens = plan.kv_lens.tolist()


@pytest.mark.parametrize("rows", [2047, 2048, 2049, 9000])
def test_few_and_many_rows(nvm, rows):
    pool, host = nvm.KV8Pool.empty(1000, 7, 300, 32), ref.Pool(1000, 7, 300, 32)
    new = [rows // 7] * 6 + [rows - 6 * (rows // 7)]
    kept = [5, 0, 100, 31, 32, 33, 1]
    compare(pool, host, nvm.kv8_plan(pool, i32(kept), i32(new), rows), host.plan(kept, new, rows), rows)


def test_a_step_taken_back_leaves_the_stack_as_it_was(nvm):
    pool = nvm.KV8Pool.empty(200, 6, 12, 16)
    nvm.kv8_plan(pool, i32([0] * 6), i32([30, 1, 0, 64, 100, 17]), 212)
    count = int(pool.free_count)                      # (what lies above the stack is nobody's)
    state = [t.clone() for t in (pool.block_table, pool.held, pool.free_pages[:count], pool.free_count)]
    nvm.kv8_plan(pool, i32([0, 1, 0, 64, 50, 17]), i32([0, 60, 30, 4, 0, 16]), 110)
    nvm.kv8_plan(pool, i32([30, 1, 0, 64, 100, 17]), i32([0] * 6), 0)
    for a, b in zip(state, (pool.block_table, pool.held, pool.free_pages[:count], pool.free_count)):
        assert torch.equal(a, b)


def test_an_empty_pool_is_asked_again(nvm):
    pool, host = nvm.KV8Pool.empty(3, 2, 8, 16), ref.Pool(3, 2, 8, 16)
    for kept, new in (([0, 0], [40, 40]), ([40, 40], [1, 1]), ([0, 41], [0, 1]), ([0, 42], [5, 0])):
        plan = nvm.kv8_plan(pool, i32(kept), i32(new), 100)
        compare(pool, host, plan, host.plan(kept, new, 100), 100)


def test_values_that_make_no_sense(nvm):
    """Cut to their range; nothing outside the arrays is touched."""
    big = 2 ** 31 - 1
    pool = nvm.KV8Pool(torch.full((4, 3), 2, dtype=torch.int32, device="cuda"), i32([big, -5, 2, 0]), i32([7, 8, 9, 10, 11]), i32([big]), 16)
    plan = nvm.kv8_plan(pool, i32([-3, big, 20, -big]), i32([big, big, -1, 7]), 60)
    assert plan.kv_lens.tolist() == [48, 48, 20, 7] and plan.cu_rows.tolist() == [0, 48, 48, 48, 55]
    assert pool.held.tolist() == [3, 3, 2, 1] and int(plan.missing) == 0
    assert pool.free_pages.tolist() == [7, 8, 9, 10, 11] and int(pool.free_count) == 1
    assert pool.block_table.tolist() == [[2, 2, 2], [11, 10, 9], [2, 2, 2], [8, 2, 2]]
    # pages past the pool have no slots
    assert plan.slots[:48].tolist() == [2 * 16 + i % 16 for i in range(48)] and plan.slots[48:55].tolist() == [-1] * 7
    pool = nvm.KV8Pool(torch.full((1, 2), 0, dtype=torch.int32, device="cuda"), i32([2]), i32([5]), i32([-9]), 16)
    plan = nvm.kv8_plan(pool, i32([0]), i32([0]), 0)   # two pages given back to a stack of one place
    assert pool.held.tolist() == [0] and int(pool.free_count) == 1 and pool.block_table.tolist() == [[-1, -1]]


def test_rows_behind_the_last_request_and_no_outputs(nvm):
    pool = nvm.KV8Pool.empty(20, 2, 4, 16)
    out = nvm.KV8Plan(i32([9] * 3), i32([9] * 2), i32([9] * 8), torch.full((8,), 9, dtype=torch.int64, device="cuda"), i32([9]))
    nvm.kv8_plan(pool, i32([0, 0]), i32([2, 3]), 8, out=out)
    assert out.positions.tolist() == [0, 1, 0, 1, 2, 9, 9, 9] and out.slots.tolist() == [0, 1, 16, 17, 18, 9, 9, 9]
    empty = nvm.KV8Pool.empty(5, 0, 4, 16)
    plan = nvm.kv8_plan(empty, i32([]), i32([]), 3)
    assert plan.cu_rows.tolist() == [0] and int(plan.missing) == 0 and int(empty.free_count) == 5


def test_lengths_in_place_and_graph_replays(nvm):
    """kv_lens may be kept_lens; a captured plan replayed over a changing state."""
    pool, host = nvm.KV8Pool.empty(300, 40, 10, 16), ref.Pool(300, 40, 10, 16)
    kept, new = i32([0] * 40), i32([3] * 40)
    out = nvm.KV8Plan(i32([0] * 41), kept, i32([0] * 200), torch.zeros(200, dtype=torch.int64, device="cuda"), i32([0]))
    compare(pool, host, nvm.kv8_plan(pool, kept, new, 200, out=out), host.plan([0] * 40, [3] * 40, 200), 200)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        nvm.kv8_plan(pool, kept, new, 200, out=out)
    for i in range(6):
        was = kept.tolist()
        n = [(b * i) % 6 for b in range(40)]
        new.copy_(i32(n))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        compare(pool, host, out, host.plan(was, n, 200), 200)
