"""moe_sort, moe_gather, moe_combine, moe_combine_grad and moe_w4a16_gemm
against their plain 64-bit forms; whole numbers equal."""
import math

import numpy as np
import pytest
import torch

from tests import batch_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nvm():
    import nvfp4_w4a16_mtp_amd as nv
    return nv


def gen(seed):
    return torch.Generator().manual_seed(seed)


def check_order(o, ids, experts):
    offsets, order, place = ref.order(ids, experts)
    assert o.offsets.tolist() == offsets.tolist()
    assert np.array_equal(o.order.cpu().numpy()[:len(order)], order)
    assert np.array_equal(o.place.cpu().numpy(), place)


@pytest.mark.parametrize("m", [1, 2, 31, 32, 33, 64, 100, 1000])
@pytest.mark.parametrize("experts,k", [(1, 1), (3, 2), (8, 8), (60, 4), (64, 6), (65, 16), (256, 8), (300, 10), (1000, 3), (1024, 16)])
def test_sort(nvm, m, experts, k):
    logits = torch.randn((m, experts), generator=gen(m + experts)).to(torch.bfloat16 if experts % 2 else torch.float32).float()
    o = nvm.moe_sort(logits.cuda(), k)
    ids, w = ref.route(logits, k)
    assert np.array_equal(o.topk_ids.cpu().numpy(), ids)
    # exp of a difference (exact to 2^-24 of it) to 2^-22, a sum of k terms and a quotient
    assert bool((np.abs(o.topk_w.double().cpu().numpy() - w) <= (2.0 ** -20 + 2.0 ** -23 * np.abs(logits.numpy()).max()) * w).all())
    check_order(o, ids, experts)


def test_sort_many_tokens(nvm):
    for m, experts, k in ((9001, 256, 8), (70000, 40, 2), (20000, 7, 7)):
        logits = torch.randn((m, experts), generator=gen(m))
        o = nvm.moe_sort(logits.cuda(), k)
        v, i = torch.sort(logits, dim=1, descending=True, stable=True)
        assert torch.equal(o.topk_ids.cpu().long(), i[:, :k])
        check = torch.sort(i[:, :k].flatten(), stable=True)
        assert torch.equal(o.order.cpu().long(), check.indices)
        assert torch.equal(o.place.cpu().long()[check.indices], torch.arange(m * k))
        assert torch.equal(o.offsets.cpu().long(), torch.searchsorted(check.values, torch.arange(experts + 1)))


def test_sort_special_logits(nvm):
    inf, big = math.inf, torch.finfo(torch.float32).max
    rows = [[0.0, -0.0, 0.0, 1.0], [-inf, -inf, 2.0, -inf], [-inf] * 4, [math.nan, 1.0, math.nan, 0.0], [math.nan] * 4,
            [inf, 1.0, inf, 0.0], [-big, -big, -big, -big], [big, -big, 0.0, big], [1e-45, 0.0, -1e-45, 0.0]]
    logits = torch.tensor(rows * 5)
    o = nvm.moe_sort(logits.cuda(), 3)
    ids, w = ref.route(logits, 3)
    assert np.array_equal(o.topk_ids.cpu().numpy(), ids)
    got = o.topk_w.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(w)) and np.nanmax(np.abs(got - w)) <= 2.0 ** -20
    check_order(o, ids, 4)


@pytest.mark.parametrize("m", [5, 40, 3000])
def test_sort_given_ids(nvm, m):
    """Any numbers: the same expert twice in a token, some outside, all of one."""
    g = gen(m)
    for ids in (torch.randint(-2, 12, (m, 6), generator=g), torch.full((m, 6), 3), torch.full((m, 6), -1), torch.full((m, 6), 10),
                torch.randint(-2 ** 31, 2 ** 31 - 1, (m, 6), generator=g)):
        ids = ids.to(torch.int32)
        dev = ids.cuda()
        o = nvm.moe_sort(None, topk_ids=dev, experts=10)
        assert torch.equal(dev.cpu(), ids) and o.topk_w is None
        check_order(o, ids.numpy(), 10)


def test_sort_of_nothing(nvm):
    o = nvm.moe_sort(torch.zeros((0, 8), device="cuda"), 2)
    assert o.offsets.tolist() == [0] * 9
    x = nvm.moe_gather(torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda"), o)
    assert x.shape == (0, 64) and nvm.moe_combine(x, o).shape == (0, 64)


def case(nv, m, experts, k, hidden, seed, dtype, left_out=False):
    g = gen(seed)
    o = nv.moe_sort(torch.randn((m, experts), generator=g).cuda(), k)
    if left_out:
        ids = torch.where(torch.rand((m, k), generator=g).cuda() < 0.3, -1, o.topk_ids).to(torch.int32)
        ids[0] = -1
        o = nv.moe_sort(None, topk_ids=ids, experts=experts)._replace(topk_w=o.topk_w)
    ys = torch.randn((m * k, hidden), generator=g).to(dtype).cuda()
    return o, ys


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,experts,k,hidden", [(1, 4, 1, 8), (3, 4, 2, 24), (37, 20, 8, 2048), (130, 300, 16, 136), (700, 64, 6, 1000)])
def test_gather_and_back(nvm, m, experts, k, hidden, dtype):
    for left_out in (False, True):
        o, ys = case(nvm, m, experts, k, hidden, 3, dtype, left_out)
        place = o.place.cpu().long()
        x = torch.randn((m, hidden), generator=gen(4)).to(dtype).cuda()
        out = torch.full((m * k, hidden), 5.0, dtype=dtype, device="cuda")
        nvm.moe_gather(x, o, out=out)
        used = place >= 0
        want = torch.full((m * k, hidden), 5.0, dtype=dtype)
        want[place[used]] = x.cpu().repeat_interleave(k, 0)[used]
        assert torch.equal(out.cpu(), want)
        for weighted in (True, False):
            w = o.topk_w.double().cpu().flatten() if weighted else torch.ones(m * k, dtype=torch.float64)
            w = torch.where(used, w, 0.0)
            terms = (ys.double().cpu()[place.clamp(min=0)] * w[:, None]).unflatten(0, (m, k))
            y64, size = terms.sum(1), terms.abs().sum(1)
            for out_dtype in (torch.bfloat16, torch.float32):
                y = nvm.moe_combine(ys, o, weighted=weighted, out_dtype=out_dtype)
                half = torch.finfo(out_dtype).eps / 2
                assert bool(((y.double().cpu() - y64).abs() <= half * y64.abs() + (k + 1) * 2.0 ** -23 * size).all())


@pytest.mark.parametrize("ys_type", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dy_type", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,experts,k,hidden", [(1, 4, 1, 8), (3, 20, 9, 264), (65, 64, 8, 2048), (40, 300, 16, 4104)])
def test_gradient(nvm, m, experts, k, hidden, ys_type, dy_type):
    for left_out in (False, True):
        o, ys = case(nvm, m, experts, k, hidden, 5, ys_type, left_out)
        place = o.place.cpu().long()
        used = place >= 0
        dy = torch.randn((m, hidden), generator=gen(6)).to(dy_type).cuda()
        keep = torch.full_like(ys, 3.0)
        dys, dw = nvm.moe_combine_grad(dy, ys, o, dys=keep)
        w = o.topk_w.double().cpu().flatten()
        pair = dy.double().cpu().repeat_interleave(k, 0)
        want = torch.full((m * k, hidden), 3.0, dtype=torch.float64)
        want[place[used]] = (pair * w[:, None])[used]
        assert bool(((dys.double().cpu() - want).abs() <= (torch.finfo(ys_type).eps / 2 + 2.0 ** -24) * want.abs()).all())
        terms = torch.where(used[:, None], ys.double().cpu()[place.clamp(min=0)] * pair, 0.0)
        assert bool(((dw.double().cpu().flatten() - terms.sum(1)).abs() <= (hidden + 2) * 2.0 ** -24 * terms.abs().sum(1)).all())
        # in place, and without weights
        same, dw2 = nvm.moe_combine_grad(dy, ys.clone(), o, weighted=False)
        pairs = pair.to(ys_type)
        assert torch.equal(same.cpu()[place[used]], pairs[used]) and torch.equal(dw2, dw)
        again = ys.clone()
        nvm.moe_combine_grad(dy, again, o, dys=again, dw=dw2)
        assert torch.equal(again.cpu()[place[used]], dys.cpu()[place[used]]) and torch.equal(dw2, dw)


def test_gradient_against_differences(nvm):
    """A loss over moe_gather and moe_combine, both gradients against central differences (fp32,
    powers of two for the steps: a bilinear form has no other error than the sums')."""
    m, experts, k, hidden = 6, 5, 3, 16
    o, ys = case(nvm, m, experts, k, hidden, 7, torch.float32)
    c = torch.randn((m, hidden), generator=gen(8)).cuda()
    loss = lambda rows, w: float((nvm.moe_combine(rows, o._replace(topk_w=w)).double() * c.double()).sum())
    dys, dw = nvm.moe_combine_grad(c, ys, o)
    g = gen(9)
    for _ in range(5):
        d = torch.randint(-4, 5, ys.shape, generator=g).float().cuda()
        diff = (loss(ys + d, o.topk_w) - loss(ys - d, o.topk_w)) / 2
        assert abs(diff - float((dys.double() * d.double()).sum())) <= 1e-4 * (1 + abs(diff))
        d = torch.randint(-4, 5, dw.shape, generator=g).float().cuda()
        diff = (loss(ys, o.topk_w + d) - loss(ys, o.topk_w - d)) / 2
        assert abs(diff - float((dw.double() * d.double()).sum())) <= 1e-4 * (1 + abs(diff))
    x = torch.randn((m, hidden), generator=g).cuda()
    back = nvm.moe_combine(nvm.moe_gather(x, o), o, weighted=False)      # k copies of every row
    assert bool(((back - k * x).abs() <= 2.0 ** -21 * (k * x).abs()).all())


def experts_of(nv, e, hidden, inter, seed):
    g = gen(seed)

    def one(rows, cols):
        c = torch.randint(0, 256, (e, rows, cols // 2), generator=g, dtype=torch.uint8)
        s = torch.randint(0x28, 0x40, (e, rows, cols // 16), generator=g, dtype=torch.uint8)
        s[:, :, ::5] = 0
        f = torch.zeros((e, 4))
        f[:, 0] = 0.4 * cols ** -0.5 * (0.5 + torch.rand(e, generator=g))
        return c, s, f
    w = [one(inter, hidden), one(inter, hidden), one(hidden, inter)]
    dev = nv.NVFP4Experts(*(t.cuda() for p in w for t in p))
    return dev, [ref.weight_values(p) for p in w]


def check_ffn(nv, x, logits, k, dev, vals, **kw):
    for out_dtype in (torch.float32, torch.bfloat16):
        y, ids, w = nv.moe_w4a16_gemm(x, logits.cuda(), k, dev, out_dtype=out_dtype, **kw)
        rids, rw = ref.route(logits, k)
        assert np.array_equal(ids.cpu().numpy(), rids)
        want, bound = ref.experts_ffn(x, rids, rw, *vals)
        half = torch.finfo(out_dtype).eps / 2
        err = (y.double().cpu() - want).abs()
        assert bool((err <= bound + half * (want.abs() + bound) + 1e-37).all()), float((err / (bound + half * want.abs() + 1e-37)).max())
    return y


@pytest.mark.parametrize("m", [1, 7, 16, 17, 40, 100, 333])
@pytest.mark.parametrize("e,k,hidden,inter", [(1, 1, 32, 32), (4, 2, 96, 160), (16, 4, 544, 96), (40, 8, 256, 544), (6, 3, 1056, 64)])
def test_experts(nvm, m, e, k, hidden, inter):
    dev, vals = experts_of(nvm, e, hidden, inter, 11)
    x = torch.randn((m, hidden), generator=gen(m)).to(torch.bfloat16).cuda()
    logits = torch.randn((m, e), generator=gen(m + 1)) + torch.linspace(0, 2, e)
    check_ffn(nvm, x, logits, k, dev, vals)


@pytest.mark.parametrize("m", [130, 400, 900])
def test_experts_uneven(nvm, m):
    """One expert takes nearly all tokens, some none: full and ragged tiles of every height."""
    dev, vals = experts_of(nvm, 5, 192, 224, 12)
    x = torch.randn((m, 192), generator=gen(1)).to(torch.bfloat16).cuda()
    logits = torch.randn((m, 5), generator=gen(2))
    logits[:, 3] += 8.0
    logits[:, 1] = -50.0
    check_ffn(nvm, x, logits, 2, dev, vals)


def test_experts_equal_the_decode_call(nvm):
    """Up to 8 rows: moe_w4a16_gemv's results up to the order of its sums and the rounding of an
    activation next to a border."""
    dev, vals = experts_of(nvm, 32, 512, 256, 13)
    for m in (1, 4, 8):
        x = torch.randn((m, 512), generator=gen(m)).to(torch.bfloat16).cuda()
        logits = torch.randn((m, 32), generator=gen(m + 9))
        a = nvm.moe_w4a16_gemv(x, logits.cuda(), 4, dev)
        b = nvm.moe_w4a16_gemm(x, logits.cuda(), 4, dev)
        assert torch.equal(a[1], b[1]) and bool(((a[2] - b[2]).abs() <= 2.0 ** -21).all())
        rids, rw = ref.route(logits, 4)
        _, bound = ref.experts_ffn(x, rids, rw, *vals)
        assert bool(((a[0].double() - b[0].double()).abs().cpu() <= 2 * bound + 1e-6).all())


def test_experts_of_nothing_and_same_bits(nvm):
    dev, _ = experts_of(nvm, 8, 64, 64, 14)
    y, ids, w = nvm.moe_w4a16_gemm(torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((0, 8), device="cuda"), 2, dev)
    assert y.shape == (0, 64) and ids.shape == (0, 2)
    x = torch.randn((300, 64), generator=gen(1)).to(torch.bfloat16).cuda()
    logits = torch.randn((300, 8), generator=gen(2)).cuda()
    first = nvm.moe_w4a16_gemm(x, logits, 2, dev)[0]
    ws = nvm.moe_gemm_workspace(300, 2, dev, "cuda")
    for _ in range(5):
        ws.random_(0, 256)
        assert torch.equal(nvm.moe_w4a16_gemm(x, logits, 2, dev, workspace=ws)[0], first)


def test_a_token_with_values_that_are_not_finite_keeps_to_itself(nvm):
    dev, _ = experts_of(nvm, 6, 128, 96, 15)
    for m in (20, 500):
        x = torch.randn((m, 128), generator=gen(3)).to(torch.bfloat16).cuda()
        logits = torch.randn((m, 6), generator=gen(4)).cuda()
        clean = nvm.moe_w4a16_gemm(x, logits, 2, dev)[0]
        x[7, 5] = math.nan
        x[11] = math.inf
        y = nvm.moe_w4a16_gemm(x, logits, 2, dev)[0]
        rest = [i for i in range(m) if i not in (7, 11)]
        assert torch.equal(y[rest], clean[rest]) and not bool(torch.isfinite(y[7]).all())


def test_streams_and_graph_replays(nvm):
    dev, _ = experts_of(nvm, 24, 256, 128, 16)
    x = torch.randn((70, 256), generator=gen(5)).to(torch.bfloat16).cuda()
    logits = torch.randn((70, 24), generator=gen(6)).cuda()
    ws = [nvm.moe_gemm_workspace(70, 4, dev, "cuda") for _ in range(2)]
    want = nvm.moe_w4a16_gemm(x, logits, 4, dev)[0]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for s, w in zip(streams, ws):
        with torch.cuda.stream(s):
            outs.append([nvm.moe_w4a16_gemm(x, logits, 4, dev, workspace=w)[0] for _ in range(4)])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for a in outs for o in a)
    y, ids, tw = torch.empty_like(want), torch.empty((70, 4), dtype=torch.int32, device="cuda"), torch.empty((70, 4), device="cuda")
    o = nvm.MoeOrder.empty(70, 4, 24, "cuda")
    sws, xs, back = nvm.moe_sort_workspace(70, 4, 24, "cuda"), torch.empty((280, 256), dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=streams[0]):
        nvm.moe_w4a16_gemm(x, logits, 4, dev, workspace=ws[0], out=y, topk_ids=ids, topk_w=tw)
        nvm.moe_sort(logits, 4, workspace=sws, out=o)
        nvm.moe_gather(x, o, out=xs)
        nvm.moe_combine(xs, o, out=back)
    for i in range(4):
        logits.copy_(torch.randn((70, 24), generator=gen(20 + i)))
        want = nvm.moe_w4a16_gemm(x, logits, 4, dev)
        so = nvm.moe_sort(logits, 4)
        wb = nvm.moe_combine(nvm.moe_gather(x, so), so)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(ids, want[1]) and torch.equal(o.place, so.place) and torch.equal(back, wb)
