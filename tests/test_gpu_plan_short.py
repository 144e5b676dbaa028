"""kv8_plan where the pool runs dry, with the cache behind it, and without its row
outputs."""
import pytest
import torch

from tests import batch_ref as ref
from tests.test_gpu_plan import compare, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nvm():
    import nvfp4_w4a16_mtp_amd as nv
    return nv


def test_a_request_that_went_short_reads_its_own_tokens_alone(nvm):
    """Two requests, three pages: the second gets none until the first has ended.  With
    covered() its rows come again as new ones, and its attention has the bits of a pool of its own."""
    gen = torch.Generator().manual_seed(1)
    page, n, kvh, dim = 16, 40, 2, 64

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen) * std).to(torch.bfloat16).cuda()
    q, k, v = normal(n + 1, 4, dim), normal(n + 1, kvh, dim), normal(n + 1, kvh, dim)
    other_k, other_v = normal(n, kvh, dim, std=4.0), normal(n, kvh, dim, std=50.0)

    def attend(cache, pool, plan, rows_q, rows_k, rows_v):
        seqs = nvm.KV8Seqs(plan.cu_rows, plan.kv_lens, pool.block_table, 64)
        nvm.kv8_append(cache, seqs, rows_k, rows_v)
        return nvm.kv8_attention(rows_q, cache, seqs)
    pool, cache = nvm.KV8Pool.empty(3, 2, 4, page), nvm.KV8Cache.empty(3, kvh, dim, page)
    plan = nvm.kv8_plan(pool, i32([0, 0]), i32([n, n]), 2 * n)
    assert int(plan.missing) == 3 and plan.kv_lens.tolist() == [n, n] and plan.slots[n:].tolist() == [-1] * n
    attend(cache, pool, plan, torch.cat((q[:n], q[:n])), torch.cat((other_k, k[:n])), torch.cat((other_v, v[:n])))
    kept = pool.covered(plan.kv_lens)
    assert kept.tolist() == [n, 0] and kept.dtype is torch.int32
    # the first ends; all of the second's rows, and one more
    kept[0] = 0
    plan = nvm.kv8_plan(pool, kept, i32([0, n + 1]), n + 1)
    assert int(plan.missing) == 0 and plan.kv_lens.tolist() == [0, n + 1] and plan.positions.tolist() == list(range(n + 1))
    got = attend(cache, pool, plan, q, k, v)
    alone, own = nvm.KV8Pool.empty(3, 1, 4, page), nvm.KV8Cache.empty(3, kvh, dim, page)
    want = attend(own, alone, nvm.kv8_plan(alone, i32([0]), i32([n + 1]), n + 1), q, k, v)
    assert torch.equal(got, want)


def test_covered_cuts_to_the_pages_there_are(nvm):
    pool, host = nvm.KV8Pool.empty(7, 4, 9, 32), ref.Pool(7, 4, 9, 32)
    new = [70, 0, 33, 200]
    plan = nvm.kv8_plan(pool, i32([0] * 4), i32(new), 400)
    compare(pool, host, plan, host.plan([0] * 4, new, 400), 400)
    assert pool.covered(plan.kv_lens).tolist() == [min(x, 32 * h) for x, h in zip(new, host.held)] == [70, 0, 33, 64]
    for bad in (i32([1, 2]), torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, dtype=torch.int32)):
        with pytest.raises(ValueError):
            pool.covered(bad)


@pytest.mark.parametrize("rows", [900, 2048, 2049, 5000])
@pytest.mark.parametrize("with_positions,with_slots", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("batch", [3, 1030])
def test_without_row_outputs(nvm, rows, with_positions, with_slots, batch):
    """No positions, no slots, neither: everything else as with them."""
    pool, host = nvm.KV8Pool.empty(6000, batch, 200, 16), ref.Pool(6000, batch, 200, 16)
    new = [rows // batch] * batch
    new[0] += rows - sum(new)
    kept = [(7 * b) % 40 for b in range(batch)]
    at = torch.full((rows,), 9, dtype=torch.int32, device="cuda")
    slots = torch.full((rows,), 9, dtype=torch.int64, device="cuda")
    out = nvm.KV8Plan(i32([9] * (batch + 1)), i32([9] * batch), at if with_positions else None, slots if with_slots else None, i32([9]))
    nvm.kv8_plan(pool, i32(kept), i32(new), rows, out=out)
    want = host.plan(kept, new, rows)
    if not with_positions:
        assert at.tolist() == [9] * rows
        at = i32(want[2])
    if not with_slots:
        assert slots.tolist() == [9] * rows
        slots = torch.tensor(want[3], device="cuda")
    compare(pool, host, out._replace(positions=at, slots=slots), want, rows)
