"""prompt_attention against its plain 64-bit form, within a bound derived per
output, and where it can go wrong: lengths, dims, masks, values, streams."""
import math

import pytest
import torch

from tests import batch_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nvm():
    import nvfp4_w4a16_mtp_amd as nv
    return nv


def normal(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(torch.bfloat16).cuda()


def cu_of(ns):
    return torch.tensor([0] + [sum(ns[:i + 1]) for i in range(len(ns))], dtype=torch.int32, device="cuda")


def check(nv, ns, hq, hk, dk, dv, window=0, sinks=0, scale=None, seed=0, std=1.0, poke=None, max_rows=None, **kw):
    gen = torch.Generator().manual_seed(seed)
    rows = sum(ns)
    q, k, v = normal(gen, rows, hq, dk, std=std), normal(gen, rows, hk, dk, std=std), normal(gen, rows, hk, dv)
    if poke:
        poke(q, k, v)
    y = nv.prompt_attention(q, k, v, cu_of(ns), max_rows or max(ns), scale=scale, window=window, sinks=sinks, **kw)
    o, b = ref.attention(q, k, v, ns, dk ** -0.5 if scale is None else scale, window, sinks)
    err = (y.double() - o).abs()
    assert bool((err <= b).all()), (float((err / b).max()), ns[:8], hq, hk, dk, dv, window, sinks)
    return q, k, v, y


@pytest.mark.parametrize("hq,hk,dk,dv", [(4, 2, 64, 64), (8, 2, 128, 128), (2, 2, 192, 128), (3, 1, 192, 192), (4, 1, 256, 256),
                                         (8, 8, 8, 8), (5, 1, 80, 80), (2, 1, 232, 104), (16, 2, 40, 248), (2, 1, 136, 64)])
@pytest.mark.parametrize("ns", [[1], [2, 1], [63, 64, 65], [127, 0, 128, 129], [300, 5]])
def test_dims_and_lengths(nvm, hq, hk, dk, dv, ns):
    check(nvm, ns, hq, hk, dk, dv)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 0), (64, 64), (65, 200), (128, 5), (200, 1), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("hq,hk,dk,dv", [(2, 1, 128, 128), (2, 2, 192, 128), (2, 1, 256, 256)])
def test_windows_and_sinks(nvm, hq, hk, dk, dv, window, sinks):
    check(nvm, [390, 64, 1], hq, hk, dk, dv, window, sinks)


@pytest.mark.parametrize("count", [63, 64, 65, 130, 700])
def test_many_sequences(nvm, count):
    check(nvm, [(7 * i * i) % 150 for i in range(count)] + [3], 2, 1, 64, 64)


@pytest.mark.parametrize("hq,hk,dk,dv", [(8, 1, 64, 64), (2, 1, 128, 128), (1, 1, 256, 256)])
def test_long(nvm, hq, hk, dk, dv):
    check(nvm, [2500, 1100], hq, hk, dk, dv)
    check(nvm, [3000], hq, hk, dk, dv, window=700, sinks=9)


@pytest.mark.parametrize("scale", [-0.1, 1.0, 1e-30, -3.0])
def test_scales(nvm, scale):
    check(nvm, [200, 70], 4, 2, 64, 64, scale=scale)


def test_scale_zero_is_a_plain_mean(nvm):
    q, k, v, y = check(nvm, [150, 3], 2, 1, 128, 128, scale=0.0)
    mean = torch.cumsum(v[:150].double(), 0) / torch.arange(1, 151, device="cuda")[:, None, None]
    assert bool(((y[:150].double() - mean).abs() <= 2.0 ** -6 * (1 + mean.abs())).all())


def test_strided_heads_and_padded_output(nvm):
    """q, k and v inside one projection's rows, head by head memory, wider output rows."""
    gen = torch.Generator().manual_seed(5)
    ns = [100, 41]
    qkv = normal(gen, 141, 8, 64)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    wide = torch.full((141, 6 * 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 64:320].unflatten(1, (4, 64))
    nvm.prompt_attention(q, k, v, cu_of(ns), 100, out=out)
    same = nvm.prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), cu_of(ns), 100)
    assert torch.equal(out, same)
    assert bool((wide[:, :64] == 7).all()) and bool((wide[:, 320:] == 7).all())
    byhead = torch.empty((4, 141, 64), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    byhead.copy_(q)
    assert torch.equal(nvm.prompt_attention(byhead, k, v, cu_of(ns), 100), same)


def test_rows_outside_the_sequences(nvm):
    """Rows before, between and behind, past max_rows, and ranges that make no sense."""
    gen = torch.Generator().manual_seed(6)
    q, k, v = normal(gen, 300, 2, 128), normal(gen, 300, 1, 128), normal(gen, 300, 1, 128)

    def run(cu, max_rows):
        out = torch.full((300, 2, 128), 9.0, dtype=torch.bfloat16, device="cuda")
        nvm.prompt_attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), max_rows, out=out)
        return out
    whole = run([10, 200], 300)
    assert bool((whole[:10] == 9).all()) and bool((whole[200:] == 9).all())
    part = run([10, 200], 70)
    assert torch.equal(part[10:80], whole[10:80]) and bool((part[80:] == 9).all())
    assert torch.equal(run([10, 200, 200, 200], 300), whole)
    bad = run([-50, 10, 5, 400], 300)                 # 0..10, none, 5..300
    assert torch.equal(bad[5:300], run([5, 300], 300)[5:300])
    assert bool((run([290, 20], 300) == 9).all())
    out = torch.full((300, 2, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    for args in (([0, 300], 0), ([0], 300)):
        nvm.prompt_attention(q, k, v, torch.tensor(args[0], dtype=torch.int32, device="cuda"), args[1], out=out)
    assert bool((out == 9).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("hq,hk,dk,dv", [(2, 1, 64, 64), (2, 1, 128, 128), (2, 1, 80, 40), (1, 1, 192, 128), (1, 1, 256, 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_what_a_row_does_not_see_never_reaches_it(nvm, bad, hq, hk, dk, dv, window, sinks):
    """Values that are not finite in k and v of one token, and in the rows of other sequences."""
    gen = torch.Generator().manual_seed(7)
    ns = [230, 90]
    q, k, v = normal(gen, 320, hq, dk), normal(gen, 320, hk, dk), normal(gen, 320, hk, dv)
    clean = nvm.prompt_attention(q, k, v, cu_of(ns), 230, window=window, sinks=sinks)
    t = 133
    ok = ref.sees(230, window, sinks)[:, t].cuda()
    for which in (k, v):
        was = which[t].clone()
        which[t, :, 1] = bad
        y = nvm.prompt_attention(q, k, v, cu_of(ns), 230, window=window, sinks=sinks)
        which[t] = was
        hidden = torch.cat((~ok, torch.ones(90, dtype=torch.bool, device="cuda")))
        assert torch.equal(y[hidden], clean[hidden])
        if which is v:
            seen = y[:230][ok]
            assert bool((seen[:, :, 1].isnan() if math.isnan(bad) else seen[:, :, 1] == bad).all())
            other = [d for d in range(dv) if d != 1]
            assert torch.equal(seen[:, :, other], clean[:230][ok][:, :, other])
        elif math.isnan(bad):
            assert bool(y[:230][ok].isnan().all())


def test_largest_values_average(nvm):
    """Sums of the largest finite values stay in range; a hidden infinity beside them too."""
    gen = torch.Generator().manual_seed(8)
    q, k = normal(gen, 200, 2, 128), normal(gen, 200, 1, 128)
    v = torch.full((200, 1, 128), torch.finfo(torch.bfloat16).max, dtype=torch.bfloat16, device="cuda")
    y = nvm.prompt_attention(q, k, v, cu_of([200]), 200)
    assert bool((y == v[0, 0, 0]).all())
    v[150] = math.inf
    y = nvm.prompt_attention(q, k, v, cu_of([200]), 200)
    assert bool((y[:150] == v[0, 0, 0]).all()) and bool((y[150:] == math.inf).all())


@pytest.mark.parametrize("q_exp,k_exp,scale", [(0, 0, 1e9), (0, 0, -1e20), (40, 20, 1.0), (60, 60, 1e-30), (0, 0, 1e38)])
def test_large_scales_and_scores(nvm, q_exp, k_exp, scale):
    """One-hot rows: every score is exact (signs of one element), so the row's best tokens share the weight."""
    gen = torch.Generator().manual_seed(9)
    n = 150
    q, k = torch.zeros(n, 1, 64), torch.zeros(n, 1, 64)
    q[:, 0, 0] = 2.0 ** q_exp
    k[:, 0, 0] = torch.randint(1, 5, (n,), generator=gen).float() * 2.0 ** k_exp
    v = normal(gen, n, 1, 64)
    y = nvm.prompt_attention(q.bfloat16().cuda(), k.bfloat16().cuda(), v, cu_of([n]), n, scale=scale)
    s = (k[:, 0, 0].double() * math.copysign(1.0, scale))
    for i in range(n):
        best = (s[:i + 1] == s[:i + 1].max()).nonzero()[:, 0].cuda()
        o = v[best, 0].double().mean(dim=0)
        assert bool(((y[i, 0].double() - o).abs() <= 2.0 ** -7 * v[best, 0].double().abs().amax(0) + 1e-30).all()), i


def test_reference_moves(nvm):
    """Scores that climb, fall and jump over many tiles."""
    def climb(q, k, v):
        k[:, :, 0] = torch.linspace(-60, 60, k.shape[0]).bfloat16().cuda()[:, None]
        q[:, :, 0] = 8.0
    def fall(q, k, v):
        k[:, :, 0] = torch.linspace(60, -60, k.shape[0]).bfloat16().cuda()[:, None]
        q[:, :, 0] = 8.0
    def jump(q, k, v):
        k[::97] *= 30.0
    for poke in (climb, fall, jump):
        check(nvm, [700], 2, 1, 128, 128, poke=poke)
        check(nvm, [700], 2, 1, 64, 64, poke=poke, window=100, sinks=2)


def test_streams_and_graph_replays(nvm):
    gen = torch.Generator().manual_seed(10)
    ns = [260, 33, 129]
    q, k, v = normal(gen, sum(ns), 4, 128), normal(gen, sum(ns), 2, 128), normal(gen, sum(ns), 2, 128)
    cu = cu_of(ns)
    eager = nvm.prompt_attention(q, k, v, cu, 260)
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = torch.empty_like(eager), torch.empty_like(eager)
    for s, o in ((side, a), (other, b)):
        with torch.cuda.stream(s):
            for _ in range(5):
                nvm.prompt_attention(q, k, v, cu, 260, out=o)
    torch.cuda.synchronize()
    assert torch.equal(a, eager) and torch.equal(b, eager)
    out = torch.empty_like(eager)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        nvm.prompt_attention(q, k, v, cu, 260, out=out)
    for i in range(4):
        q.copy_(normal(gen, *q.shape))
        want = nvm.prompt_attention(q, k, v, cu, 260)
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_offsets_past_32_bits(nvm):
    """Rows beyond 2^31 elements of one buffer."""
    stride, n = 1 << 22, 600
    buf = torch.zeros(n * stride, dtype=torch.bfloat16, device="cuda")
    rows = buf.view(n, stride)
    gen = torch.Generator().manual_seed(11)
    q, k, v = normal(gen, n, 2, 64), normal(gen, n, 1, 64), normal(gen, n, 1, 64)
    far = [rows[:, i * 128:i * 128 + x.shape[1] * 64].unflatten(1, (x.shape[1], 64)) for i, x in enumerate((q, k, v))]
    for d, x in zip(far, (q, k, v)):
        d.copy_(x)
    cu = cu_of([500, 100])
    assert torch.equal(nvm.prompt_attention(*far, cu, 500), nvm.prompt_attention(q, k, v, cu, 500))
