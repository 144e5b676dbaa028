"""Rotary positions, the paged 8-bit KV cache and attention over it against
their plain 64-bit forms (tests/kv_ref.py)."""
import numpy as np
import pytest
import torch

from tests import kv_ref as ref

pytestmark = pytest.mark.gpu


def nvm():
    import nvfp4_w4a16_mtp_amd as nv
    return nv


def bf(x):
    return torch.from_numpy(np.float32(x)).cuda().to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def normal(rng, shape, std=1.0):
    return ref.bf16(rng.normal(0, std, shape))


def device_cache(c):
    def up(x):
        return torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return nvm().KV8Cache(up(c.k), up(c.ks), up(c.v.transpose(0, 1, 3, 2)), up(c.vs))


def same_cache(dev, c, what=""):
    assert np.array_equal(dev.k_scales.cpu().numpy(), c.ks), what
    assert np.array_equal(dev.v_scales.cpu().numpy(), c.vs), what
    for got, want in ((dev.k_codes.cpu().numpy(), c.k), (dev.v_codes.cpu().numpy().transpose(0, 1, 3, 2), c.v)):
        nan = (want & 0x7F) == 0x7F                    # a NaN's sign is not specified
        assert np.array_equal(got[~nan], want[~nan]) and np.all((got[nan] & 0x7F) == 0x7F), what


def batch(rng, ns, lens, P, spare=3):
    """cu_rows, block table in random page order, pool size."""
    need = [max(1, -(-x // P)) for x in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.zeros((len(ns), max(need)), np.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c
    return np.concatenate([[0], np.cumsum(ns)]).astype(np.int32), table, pages


def seqs(cu, lens, table, max_rows, **kw):
    return nvm().KV8Seqs(i32(cu), i32(lens), i32(table), max_rows=max_rows, **kw)


# ------------------------------------------------------------------- rope
@pytest.mark.parametrize("rows,hq,hk,dim,rot,inter", [(1, 1, 1, 64, 64, False), (5, 16, 2, 256, 64, False), (33, 3, 1, 128, 128, True),
                                                      (7, 4, 4, 80, 48, True), (300, 8, 2, 128, 96, False), (2, 5, 1, 24, 16, True)])
def test_rope(rows, hq, hk, dim, rot, inter):
    nv = nvm()
    rng = np.random.default_rng(rows)
    q, k = normal(rng, (rows, hq, dim)), normal(rng, (rows, hk, dim))
    pos = rng.integers(-5, 1 << 20, rows).astype(np.int32)
    pos[0] = 2147483647 if rows > 1 else 0
    freq = 1e6 ** (-np.arange(0, rot, 2) / rot)
    outs = nv.rope_qk(bf(q), bf(k), i32(pos), torch.from_numpy(freq).cuda(), interleaved=inter, mscale=1.25)
    for x, got in ((q, outs[0]), (k, outs[1])):
        want = ref.rotate(x, pos, freq, rot, inter, 1.25)
        # one rounding to bf16 through fp32, and the angle's own rounding: p * f in
        # fp64 is off by 2^-52 relative on each side, the sums by a few 2^-53
        size = np.abs(x).max() * 1.25 * 2
        tol = (2.0 ** -8 + 2.0 ** -23) * np.abs(want) + size * (np.abs(pos.astype(float)).max() * 2.0 ** -50 + 1e-12)
        assert np.all(np.abs(f64(got) - want) <= tol)
        assert np.array_equal(f64(got)[..., rot:], x[..., rot:])


def test_rope_strided_in_place_and_single():
    nv = nvm()
    rng = np.random.default_rng(5)
    freq = torch.from_numpy(1e4 ** (-np.arange(0, 64, 2) / 64)).cuda()
    pos = i32([3, 99, 1000])
    wide = bf(rng.normal(0, 1, (3, 4, 256)))          # per head: q (128) | gate (128)
    q = wide[:, :, :128]
    want, none = nv.rope_qk(q, None, pos, freq)
    assert none is None
    keep = wide.clone()
    got, _ = nv.rope_qk(q, None, pos, freq, q_out=q)
    assert got.data_ptr() == wide.data_ptr() and torch.equal(got, want)
    assert torch.equal(wide[:, :, 128:], keep[:, :, 128:])
    # k alone, into a strided output with canaries around
    buf = torch.full((3, 6, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    nv.rope_qk(None, keep[:, :, :128], pos, freq, k_out=buf[:, 1:5])
    assert torch.equal(buf[:, 1:5], want) and bool((buf[:, 0] == 7).all()) and bool((buf[:, 5] == 7).all())
    empty = nv.rope_qk(q[:0], q[:0], pos[:0], freq)
    assert empty[0].shape[0] == 0


# ------------------------------------------------------------------ cache
@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("dim,heads", [(64, 1), (128, 3), (192, 2), (256, 2)])
def test_append_and_read(P, dim, heads):
    nv = nvm()
    rng = np.random.default_rng(P + dim)
    ns = [1, 5, 0, P, 2 * P + 3, 3, 1]
    lens = [1, 5 + 3 * P - 2, P + 7, P, 4 * P + 1, 3 + P, 2 * P]
    cu, table, pages = batch(rng, ns, lens, P)
    host = ref.Cache(pages, heads, P, dim, rng)
    host.ks[table[1, 2]] = 60                        # a continued page whose scale grows by far
    dev = device_cache(host)
    rows = sum(ns)
    k, v = normal(rng, (rows, heads, dim), 3.0), normal(rng, (rows, heads, dim), 0.01)
    k[rows - 1] = 0.0
    s = seqs(cu, lens, table, max(ns))
    for _ in range(2):                               # the same rows again give the same pages
        nv.kv8_append(dev, s, bf(k), bf(v))
        host.append(table, cu, lens, k, v)
        same_cache(dev, host)
    # read back more than was written
    back = [min(x, n + 20) for n, x in zip(ns, lens)]
    cub = np.concatenate([[0], np.cumsum(back)])
    got = nv.kv8_read(dev, seqs(cub, lens, table, max(back)), rows=int(cub[-1]))
    for b in range(len(ns)):
        want = host.values(table, b, lens[b])
        for g, w in zip(got, want):
            assert np.array_equal(f64(g)[cub[b]:cub[b + 1]], w.transpose(1, 0, 2)[lens[b] - back[b]:])
    # one of the two, strided
    buf = torch.full((int(cub[-1]) + 1, heads + 1, dim), 3.0, dtype=torch.bfloat16, device="cuda")
    nv.kv8_read(dev, seqs(cub, lens, table, max(back)), v_out=buf[:-1, 1:])
    assert torch.equal(buf[:-1, 1:], got[1]) and bool((buf[:, 0] == 3).all()) and bool((buf[-1] == 3).all())
    nv.kv8_read(dev, seqs(cub, lens, table, max(back)), k_out=buf[:-1, 1:])
    assert torch.equal(buf[:-1, 1:], got[0])


def test_append_token_by_token_and_rollback():
    nv = nvm()
    rng = np.random.default_rng(11)
    host = ref.Cache(6, 2, 16, 128, rng)
    dev = device_cache(host)
    table = np.array([[3, 0, 5]], np.int32)
    length = 0
    for step in range(40):
        n = int(rng.integers(1, 4))
        if step % 5 == 4:
            length = max(0, length - 3)              # drafts that fell
        if length + n > 48:
            break
        length += n
        k, v = (normal(rng, (n, 2, 128), 2.0 ** float(rng.integers(-8, 8))) for _ in range(2))
        nv.kv8_append(dev, seqs([0, n], [length], table, n), bf(k), bf(v))
        host.append(table, [0, n], [length], k, v)
        same_cache(dev, host, f"step {step}")


def test_append_special_values():
    nv = nvm()
    rng = np.random.default_rng(12)
    host = ref.Cache(4, 1, 16, 64, rng)
    dev = device_cache(host)
    table = np.array([[0], [1], [2]], np.int32)
    k = normal(rng, (24, 1, 64))
    k[0, 0, :4] = [np.inf, -np.inf, np.nan, 5.0]      # infinities saturate at the scale of the finite values
    k[8:16] = 0.0                                     # a page of zeros
    k[16:24] = normal(rng, (8, 1, 64), 1e38)
    k[17, 0, 0] = 3.3895313892515355e38               # the largest bf16
    v = k * 1.0
    v[16:24] = 2.0 ** -130 * rng.integers(-8, 8, (8, 1, 64))   # bf16 subnormals
    args = ([0, 8, 16, 24], [8, 8, 8])
    nv.kv8_append(dev, seqs(args[0], args[1], table, 8), bf(k), bf(v))
    host.append(table, *args, k, v)
    same_cache(dev, host)
    assert host.ks[1, 0] == 127 + ref.MIN_EXP
    # a NaN that is re-rounded to a grown scale stays a NaN
    big = np.full((1, 1, 64), 1000.0)
    nv.kv8_append(dev, seqs([0, 1, 1, 1], [9, 8, 8], table, 1), bf(big), bf(big))
    host.append(table, [0, 1, 1, 1], [9, 8, 8], big, big)
    same_cache(dev, host)


def test_attention_largest_window():
    """A window of the largest int32 is no window, also for rows that begin
    before the first token."""
    nv = nvm()
    rng = np.random.default_rng(29)
    host = ref.Cache(12, 2, 16, 64, rng)
    dev = device_cache(host)
    table = rng.permutation(12)[:10].reshape(2, 5).astype(np.int32)
    cu, lens = [0, 12, 92], [3, 70]                   # 9 and 10 rows before the first token
    q = normal(rng, (92, 4, 64))
    for rows in (12, 92):                             # one row tile, and several
        n = cu[:2] if rows == 12 else cu
        b = len(n) - 1
        want, bound, _ = ref.attention(q[:rows], host, table[:b], n, lens[:b], 0.125)
        for window in (2 ** 31 - 1, 2 ** 31 - 6, 0):
            got = f64(nv.kv8_attention(bf(q[:rows]), dev, seqs(n, lens[:b], table[:b], 80), scale=0.125, window=window))
            assert np.all(np.abs(got - want) <= bound), (rows, window)


def test_scales_that_bfloat16_cannot_hold():
    """Values up to the largest bf16: no code is infinite, and hidden tokens of
    such a page (all larger than the visible ones) reach no row."""
    nv = nvm()
    rng = np.random.default_rng(28)
    host = ref.Cache(4, 2, 16, 64, rng)
    dev = device_cache(host)
    table = np.array([[2, 1]], np.int32)
    k, v = normal(rng, (20, 2, 64)), normal(rng, (20, 2, 64))
    v[10:] = 3.3895313892515355e38 * rng.choice([-1.0, 1.0], (10, 2, 64))
    nv.kv8_append(dev, seqs([0, 20], [20], table, 20), bf(k), bf(v))
    host.append(table, [0, 20], [20], k, v)
    same_cache(dev, host)
    assert host.vs.max() == 127 + ref.MAX_EXP
    _, back = nv.kv8_read(dev, seqs([0, 20], [20], table, 20), rows=20)
    assert torch.isfinite(back).all()
    q = normal(rng, (3, 4, 64))
    for byte in (None, 247, 255):                     # and bytes that only a caller can write
        if byte is not None:
            dev.v_scales[2] = byte
            host.vs[2] = byte
        for length in (10, 3):                        # tokens 10 .. hold the large ones
            want, bound, _ = ref.attention(q, host, table, [0, 3], [length], 0.125)
            got = f64(nv.kv8_attention(bf(q), dev, seqs([0, 3], [length], table, 3), scale=0.125))
            assert np.all(np.abs(got - want) <= bound), (byte, length)


def test_append_bounds():
    """Rows at negative positions, page ids out of range, more rows than
    max_rows, row ranges past the rows: bounded, the rest unharmed."""
    nv = nvm()
    rng = np.random.default_rng(13)
    host = ref.Cache(5, 2, 16, 64, rng)
    table = np.array([[1, -1], [2, 99], [4, 0], [3, 0]], np.int32)
    lens = [20, 30, 4, 1000]
    cu = [0, 8, 20, 26, 500]                          # the third sequence: 6 rows, 4 tokens; the last: past the rows
    rows = 30
    k, v = normal(rng, (rows, 2, 64)), normal(rng, (rows, 2, 64))
    dev = device_cache(host)
    nv.kv8_append(dev, seqs(cu, lens, table, 12), bf(k), bf(v))
    host.append(table, cu, lens, k, v, max_rows=12)
    same_cache(dev, host)
    out = torch.full((rows, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    nv.kv8_read(dev, seqs(cu, lens, table, 12), k_out=out)
    got = f64(out)
    assert np.all(got[20:22] == 0)                    # negative positions
    for b in (0, 1, 2, 3):
        kk, _, ok = host.values(table, b, min(lens[b], 32))
        n = min(cu[b + 1], rows) - cu[b]
        L = min(lens[b], 32)
        for i in range(n):
            t = L - n + i
            if t >= 0:
                assert np.array_equal(got[cu[b] + i], kk[:, t] if ok[t] else np.zeros((2, 64))), (b, i)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot,P", [(64, 64, 16), (256, 64, 16), (128, 96, 64), (192, 192, 128), (256, 256, 128)])
def test_fused_equals_the_two_calls(inter, dim, rot, P):
    nv = nvm()
    rng = np.random.default_rng(dim + rot)
    ns, lens = [3, 1, P + 5, 0, 2], [100, 1, 2 * P + 9, 5, 100 + P]
    cu, table, pages = batch(rng, ns, lens, P)
    rows, hq, hk = sum(ns), 6, 2
    host = ref.Cache(pages, hk, P, dim, rng)
    one, two = device_cache(host), device_cache(host)
    freq = torch.from_numpy(1e6 ** (-np.arange(0, rot, 2) / rot)).cuda()
    gated = bf(rng.normal(0, 1, (rows, hq, 2 * dim)))
    q, k, v = gated[:, :, :dim], bf(rng.normal(0, 1, (rows, hk, dim))), bf(rng.normal(0, 1, (rows, hk, dim)))
    s = seqs(cu, lens, table, max(ns))
    pos = np.concatenate([np.arange(x - n, x) for n, x in zip(ns, lens)])
    q2, k2 = nv.rope_qk(q, k, i32(pos), freq, interleaved=inter, mscale=1.1)
    nv.kv8_append(two, s, k2, v)
    q1 = nv.rope_kv8_append(one, s, q, k, v, freq, interleaved=inter, mscale=1.1)
    assert torch.equal(q1, q2)
    for a, b in zip((one.k_codes, one.k_scales, one.v_codes, one.v_scales), (two.k_codes, two.k_scales, two.v_codes, two.v_scales)):
        assert torch.equal(a, b)
    nv.rope_kv8_append(two, s, q, k, v, freq, interleaved=inter, mscale=1.1, q_out=q)
    assert torch.equal(q, q2)
    third = device_cache(host)
    assert nv.rope_kv8_append(third, s, None, k, v, freq, interleaved=inter, mscale=1.1) is None
    assert torch.equal(third.k_codes, one.k_codes)


def test_fused_leaves_rows_outside_the_sequences():
    nv = nvm()
    rng = np.random.default_rng(14)
    host = ref.Cache(3, 2, 16, 64, rng)
    dev = device_cache(host)
    q, k, v = (bf(rng.normal(0, 1, (6, h, 64))) for h in (4, 2, 2))
    freq = torch.from_numpy(1e4 ** (-np.arange(0, 64, 2) / 64)).cuda()
    q_out = torch.full_like(q, 3.0)
    nv.rope_kv8_append(dev, seqs([1, 3, 4], [2, 20], np.array([[0, 1], [1, 2]]), 2), q, k, v, freq, q_out=q_out)
    assert bool((q_out[0] == 3).all()) and bool((q_out[4:] == 3).all()) and not bool((q_out[1:4] == 3).all())
    want, _ = nv.rope_qk(q[1:4], None, i32([0, 1, 19]), freq)
    assert torch.equal(q_out[1:4], want)


# -------------------------------------------------------------- attention
def check_attention(rng, ns, lens, P, hq, hk, dim, window=0, sinks=0, scale=None, std=1.0, poke=None, **kw):
    nv = nvm()
    cu, table, pages = batch(rng, ns, lens, P)
    host = ref.Cache(pages, hk, P, dim, rng)
    rows = sum(ns)
    q = normal(rng, (rows + 2, hq, dim), std)
    if poke is not None:
        poke(host, table, q)
    dev = device_cache(host)
    scale = dim ** -0.5 if scale is None else scale
    want, bound, owned = ref.attention(q, host, table, cu, lens, scale, window, sinks)
    out = torch.full((rows + 2, hq, dim), 5.0, dtype=torch.bfloat16, device="cuda")
    s = seqs(cu, lens, table, max(max(ns), 1), **kw)
    ws = nv.kv8_attention_workspace(dev, s, hq, rows + 2)
    nv.kv8_attention(bf(q), dev, s, scale=scale, window=window, sinks=sinks, workspace=ws, out=out)
    got = f64(out)
    assert np.all(got[~owned] == 5.0), "rows outside the sequences"
    g, w, t = got[owned], want[owned], bound[owned]
    nan = np.isnan(w)
    assert np.array_equal(np.isnan(g), nan), f"NaN at {np.argwhere(np.isnan(g) != nan)[:4]}"
    bad = ~nan & ~(np.abs(g - w) <= t)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, first {np.argwhere(bad)[0]}, {g[bad][0]} for {w[bad][0]}, {t[bad][0]}"
    again = out.clone()
    nv.kv8_attention(bf(q), dev, s, scale=scale, window=window, sinks=sinks, workspace=ws, out=out)
    assert torch.equal(torch.nan_to_num(out, 77.0), torch.nan_to_num(again, 77.0)), "a second call on the workspace differs"
    return got


SHAPES = [(16, 2, 256), (8, 1, 128), (12, 4, 64), (9, 3, 192), (5, 5, 64), (32, 2, 128), (7, 1, 256)]


@pytest.mark.parametrize("hq,hk,dim", SHAPES)
@pytest.mark.parametrize("P", [16, 64])
def test_attention_decode(hq, hk, dim, P):
    rng = np.random.default_rng(hq + dim + P)
    check_attention(rng, [1] * 6, [1, 63, 64, 65, 200, 1300], P, hq, hk, dim)


@pytest.mark.parametrize("hq,hk,dim", SHAPES)
@pytest.mark.parametrize("P", [16, 32, 128])
def test_attention_several_rows(hq, hk, dim, P):
    rng = np.random.default_rng(hq + dim + P)
    check_attention(rng, [3, 0, 5, 1, 2, 8], [3, 40, 129, 1, 700, 64], P, hq, hk, dim)


@pytest.mark.parametrize("hq,hk,dim", [(16, 2, 256), (4, 4, 64), (6, 2, 128), (3, 1, 192)])
def test_attention_prompt(hq, hk, dim):
    rng = np.random.default_rng(dim)
    check_attention(rng, [130, 1, 67], [130, 300, 200], 16, hq, hk, dim)


@pytest.mark.parametrize("hq,hk,dim,ns", [(16, 2, 256, [5, 6, 1]), (16, 2, 128, [6, 5, 2]), (12, 2, 192, [8, 6, 1]), (16, 2, 192, [8, 7, 1]),
                                          (16, 2, 64, [5, 1, 6]), (16, 2, 256, [8, 7, 2])])
@pytest.mark.parametrize("P", [16, 128])
def test_attention_three_and_four_row_tiles(hq, hk, dim, ns, P):
    """33 to 64 rows a kv head, keys split over workgroups and not."""
    rng = np.random.default_rng(hq + dim + P)
    check_attention(rng, ns, [700, 1300, 130], P, hq, hk, dim)
    check_attention(rng, ns, [9, 6, 3000], P, hq, hk, dim, window=200, sinks=3)


@pytest.mark.parametrize("count", [64, 65, 257, 300, 1024, 1025])
@pytest.mark.parametrize("hq,dim,most", [(16, 64, 1), (8, 128, 4), (16, 64, 3), (4, 192, 2), (16, 256, 2)])
def test_attention_many_sequences(count, hq, dim, most):
    """Sequences in several wavefronts' and several rounds' prefix sums, and more
    than share their steps evenly; some without rows or without tokens."""
    rng = np.random.default_rng(count + dim + most)
    ns = rng.integers(0, most + 1, count)
    ns[-1] = most
    lens = np.where(rng.random(count) < 0.1, 0, rng.integers(1, 200, count))
    lens[count // 3], lens[-1] = 1500, 700
    check_attention(rng, [int(n) for n in ns], [int(x) for x in lens], 16, hq, 1, dim)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("n", [1, 20, 40])
def test_attention_wide_block_table(dim, n):
    """A block table of so many steps that they are not shared evenly: keys in
    pieces, one to three row tiles."""
    nv = nvm()
    rng = np.random.default_rng(dim + n)
    heads = 512 if dim <= 128 else 256
    length = 300
    host = ref.Cache(4, heads, 128, dim, rng)
    table = np.array([[2, 0, 3]], np.int32)
    wide = torch.zeros((1, (1 << 30) // heads), dtype=torch.int32, device="cuda")
    wide[:, :3] = i32(table)
    q = normal(rng, (n, heads, dim))
    want, bound, _ = ref.attention(q, host, table, [0, n], [length], dim ** -0.5)
    s = nv.KV8Seqs(i32([0, n]), i32([length]), wide, max_rows=n, max_kv_len=length)
    got = f64(nv.kv8_attention(bf(q), device_cache(host), s))
    assert np.all(np.abs(got - want) <= bound)


@pytest.mark.parametrize("hq,hk,dim", [(16, 2, 256), (8, 1, 128)])
def test_attention_prompt_chunk_beside_decode_rows(hq, hk, dim):
    rng = np.random.default_rng(dim)
    check_attention(rng, [1, 150, 1, 0, 2, 1], [3000, 400, 1, 9, 129, 800], 16, hq, hk, dim)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (17, 3), (64, 64), (100, 65), (128, 4), (5000, 4), (300, 1000)])
def test_attention_window(window, sinks):
    rng = np.random.default_rng(window + sinks)
    check_attention(rng, [1, 2, 5, 40, 1], [1, 66, 500, 400, 1025], 32, 8, 2, 128, window=window, sinks=sinks)
    check_attention(rng, [1, 3], [900, 130], 16, 16, 2, 256, window=window, sinks=sinks)


def test_attention_long_and_split():
    rng = np.random.default_rng(21)
    check_attention(rng, [1], [9001], 16, 8, 1, 128)
    check_attention(rng, [2, 1], [7000, 10], 128, 16, 2, 256, max_kv_len=7000)
    check_attention(rng, [1, 1], [3000, 2999], 64, 4, 4, 64, max_kv_len=100)      # a bound that is too small


def test_attention_rows_that_see_nothing():
    """Length zero, more rows than tokens, pages out of range."""
    rng = np.random.default_rng(22)

    def poke(host, table, q):
        table[2, 0] = -1
        table[3, 0] = 10 ** 6
        table[3, 1] = -7
        table[4, 1] = 2 ** 31 - 1
    got = check_attention(rng, [2, 5, 3, 1, 2], [0, 3, 16, 32, 48], 16, 4, 2, 64, poke=poke)
    assert np.all(got[0:2] == 0) and np.all(got[2:4] == 0) and np.all(got[7:11] == 0)
    check_attention(rng, [1, 1], [0, 0], 16, 4, 2, 64)


@pytest.mark.parametrize("hq,hk,dim,ns", [(8, 2, 64, [4, 1, 9]), (16, 2, 256, [2, 1, 4]), (6, 2, 128, [70, 1, 40])])
def test_attention_nan_where_it_is_not_seen(hq, hk, dim, ns):
    """NaN codes in stale tokens, in the causal future and outside the window
    reach no row; a visible one reaches exactly its row's (K) or dim's (V)
    results."""
    rng = np.random.default_rng(dim)
    lens = [n + 60 for n in ns]

    def poke(host, table, q):
        P = host.tokens
        for b, x in enumerate(lens):
            page, off = table[b, x // P if x % P else x // P - 1], x % P
            if x % P:
                host.k[page, :, off:] = 0x7F         # behind the sequence
                host.v[page, :, off:] = 0xFF
            last = x - 1
            host.k[table[b, last // P], 0, last % P] = 0x7F          # the last token: the earlier rows do not see it
            host.v[table[b, last // P], 0, last % P, 5:9] = 0x7F
        host.v[table[0, 0], :, 2] = 0x7F             # before the window
        host.v[table[1, 2], 1, 3, 11] = 0x7F         # in sight
        q[1, 0, 0] = np.nan
        q[2, 1, 3] = np.inf
    check_attention(rng, ns, lens, 16, hq, hk, dim, window=50, sinks=1, poke=poke)
    check_attention(rng, ns, lens, 16, hq, hk, dim, poke=lambda h, t, q: [poke(h, t, q), h.v.__setitem__((t[0, 0], slice(None), 2), 1)])


def test_attention_extreme_values():
    """Scores far apart, scale bytes at the ends of their range."""
    rng = np.random.default_rng(23)
    check_attention(rng, [1, 3], [130, 500], 16, 8, 2, 128, scale=3.0, std=4.0)
    check_attention(rng, [1, 3], [130, 500], 16, 8, 2, 128, scale=-0.5)
    check_attention(rng, [2], [100], 16, 8, 2, 128, scale=0.0)

    def poke(host, table, q):
        host.vs[:] = rng.choice([0, 1, 90, 127, 150], host.vs.shape)
        host.ks[:] = rng.choice([0, 20, 118, 119], host.ks.shape)
    check_attention(rng, [1, 3], [130, 500], 16, 8, 2, 128, poke=poke)


def check_exact_scores(rng, ns, lens, hq, hk, dim, scale, q_exp=0, k_exp=0):
    """Scores that are whole numbers times 2^(q_exp + k_exp), exact in fp32, and so
    far apart under the scale that only a row's largest count: the mean of v over
    those.  Their weights are exactly 1; fp32 sums of up to L terms are off by (L +
    64) 2^-24 each, the result by its rounding to bf16."""
    nv = nvm()
    cu, table, pages = batch(rng, ns, lens, 16)
    host = ref.Cache(pages, hk, 16, dim, rng)
    host.k[:] = ref.e4m3_encode(rng.integers(-2, 3, host.k.shape))
    host.ks[:] = 127 + k_exp
    q = rng.integers(-2, 3, (sum(ns), hq, dim)) * 2.0 ** q_exp
    want, _, _ = ref.attention(q, host, table, cu, lens, scale)
    got = f64(nv.kv8_attention(bf(q), device_cache(host), seqs(cu, lens, table, max(ns)), scale=scale))
    top = max(np.abs(host.values(table, b, lens[b])[1]).max() for b in range(len(ns)))
    tol = 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * 2 * (max(lens) + 64) * 2.0 ** -24 * top
    assert np.isfinite(got).all() and np.all(np.abs(got - want) <= tol), (scale, np.argwhere(~(np.abs(got - want) <= tol))[:3])


@pytest.mark.parametrize("scale", [1e3, 1e9, -1e9, 1e30, -2e38])
@pytest.mark.parametrize("hq,hk,dim,ns,lens", [(8, 1, 128, [1, 3], [1, 1500]), (16, 2, 256, [5, 1], [700, 130]), (6, 2, 64, [70, 2], [300, 129])])
def test_attention_large_scales(scale, hq, hk, dim, ns, lens):
    check_exact_scores(np.random.default_rng(31), ns, lens, hq, hk, dim, scale)


@pytest.mark.parametrize("q_exp,k_exp,scale", [(40, 0, None), (20, 20, None), (57, 57, None), (57, 57, -0.5), (50, 57, 1e6), (57, 50, 1e30)])
def test_attention_large_scores(q_exp, k_exp, scale):
    """Scores up to 2^124 under ordinary scales, and under scales that take the
    product past fp32's range."""
    for hq, hk, dim, ns, lens in ((8, 1, 128, [1, 3], [65, 1500]), (4, 2, 256, [40, 1], [400, 2000])):
        check_exact_scores(np.random.default_rng(32), ns, lens, hq, hk, dim, dim ** -0.5 if scale is None else scale, q_exp, k_exp)


@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-60, 1e-44, -1e-40, 3e-38])
def test_attention_scales_near_zero(scale):
    """A scale of zero is a plain mean whatever the scores; one among the
    subnormals counts as it is (1e-60 is zero in fp32)."""
    nv = nvm()
    rng = np.random.default_rng(33)
    for hq, hk, dim, ns, lens in ((8, 1, 128, [1, 3], [65, 1500]), (4, 2, 256, [40, 1], [400, 300])):
        cu, table, pages = batch(rng, ns, lens, 16)
        host = ref.Cache(pages, hk, 16, dim, rng)
        host.k[:] = ref.e4m3_encode(rng.integers(-2, 3, host.k.shape))
        host.ks[:] = 127 + 58
        q = rng.integers(-2, 3, (sum(ns), hq, dim)) * 2.0 ** 58          # scores up to 2^126
        want, bound, _ = ref.attention(q, host, table, cu, lens, float(np.float32(scale)))
        got = f64(nv.kv8_attention(bf(q), device_cache(host), seqs(cu, lens, table, max(ns)), scale=scale))
        assert np.all(np.abs(got - want) <= bound), scale
    # zero times what is not finite is NaN, in its row and head alone
    host.k[table[0, 0], 0, 3, 1] = 0x7F
    q[40, 3, 5] = np.inf
    want, bound, _ = ref.attention(q, host, table, cu, lens, 0.0)
    got = f64(nv.kv8_attention(bf(q), device_cache(host), seqs(cu, lens, table, max(ns)), scale=0.0))
    nan = np.isnan(want)
    assert nan.any() and np.array_equal(np.isnan(got), nan) and np.all(np.abs(got - want)[~nan] <= bound[~nan])


@pytest.mark.parametrize("hq,hk,dim,ns,lens", [(8, 1, 128, [1, 3], [2, 1500]), (16, 2, 256, [1], [9001]), (16, 2, 256, [5, 6], [700, 40]),
                                               (4, 2, 64, [100, 2], [300, 129])])
@pytest.mark.parametrize("flat", [False, True])
def test_attention_large_values_in_sight(hq, hk, dim, ns, lens, flat):
    """V up to the largest value the cache holds, of one sign, in every page or
    in some: an average of finite values is finite."""
    def poke(host, table, q):
        if flat:
            q[:] = 0.0
        host.v[:] = host.v & 0x7F
        host.vs[:] = 246
    rng = np.random.default_rng(34)
    got = check_attention(rng, ns, lens, 16, hq, hk, dim, poke=poke)
    assert np.isfinite(got).all() and np.abs(got).max() > 1e37

    def late(host, table, q):                         # small values, then large ones, then small ones
        if flat:
            q[:] = 0.0
        host.vs[table[:, table.shape[1] // 2]] = 246
        host.vs[table[0, -1]] = 208
    check_attention(rng, ns, lens, 16, hq, hk, dim, poke=late)

    def hidden(host, table, q):                       # large values that a window hides: the small ones keep their precision
        host.vs[table[:, 0]] = 246
    check_attention(rng, ns, lens, 16, hq, hk, dim, window=20, poke=hidden)


def test_attention_largest_value_of_many():
    """Equal keys, every visible value the largest: the average is that value."""
    nv = nvm()
    rng = np.random.default_rng(35)
    for rows, length in ((1, 20000), (2, 3), (300, 1000)):
        cu, table, pages = batch(rng, [rows], [length], 64)
        host = ref.Cache(pages, 2, 64, 128, rng)
        host.k[:], host.v[:], host.vs[:] = 0x38, 0x7E, 246
        q = normal(rng, (rows, 8, 128))
        got = f64(nv.kv8_attention(bf(q), device_cache(host), seqs(cu, [length], table, rows)))
        want = 448.0 * 2.0 ** 119
        # equal weights cancel up to fp32 sums of up to `length` terms
        seen = (np.arange(rows) + length - rows >= 0)
        assert np.all(np.abs(got[seen] - want) <= want * (2.0 ** -8 + 2 * (length + 64) * 2.0 ** -24)), (rows, length)


def test_host_integers_past_32_bits_are_refused():
    """None is cut to its low bits: a window of 2^32 is not no window."""
    nv = nvm()
    rng = np.random.default_rng(36)
    dev = device_cache(ref.Cache(2, 1, 16, 64, rng))
    q = bf(rng.normal(0, 1, (1, 1, 64)))
    args = (i32([0, 1]), i32([20]), i32([[0, 1]]))
    s = nv.KV8Seqs(*args, max_rows=1)
    for v in (1 << 32, (1 << 32) + 1, 1 << 31, -(1 << 31) - 1):
        for kw in (dict(window=v), dict(window=5, sinks=v)):
            with pytest.raises(ValueError):
                nv.kv8_attention(q, dev, s, **kw)
        for kw in (dict(max_rows=v), dict(max_rows=1, max_kv_len=v)):
            with pytest.raises(ValueError):
                nv.KV8Seqs(*args, **kw)
        with pytest.raises(ValueError):
            nv.kv8_attention_workspace(dev, s, v, 1)
        with pytest.raises(ValueError):
            nv.kv8_attention_workspace(dev, s, 1, v)
        with pytest.raises(ValueError):
            nv.verify_workspace(v, 1, 10, "cuda")
        with pytest.raises(ValueError):
            nv.verify_drafts(torch.zeros((1, 10), device="cuda"), i32([0, 1]), i32([0]), torch.zeros(1, device="cuda"),
                             torch.zeros(1, device="cuda"), v)


def test_attention_strided_rows():
    nv = nvm()
    rng = np.random.default_rng(24)
    ns, lens = [2, 1], [50, 77]
    cu, table, pages = batch(rng, ns, lens, 16)
    host = ref.Cache(pages, 2, 16, 128, rng)
    dev = device_cache(host)
    wide = bf(rng.normal(0, 1, (3, 8, 256)))
    s = seqs(cu, lens, table, 2)
    want = nv.kv8_attention(wide[:, :, :128].contiguous(), dev, s)
    buf = torch.full((3, 10, 128), 2.0, dtype=torch.bfloat16, device="cuda")
    nv.kv8_attention(wide[:, :, :128], dev, s, out=buf[:, 1:9])
    assert torch.equal(buf[:, 1:9], want) and bool((buf[:, [0, 9]] == 2).all())


def test_attention_shared_pages_and_two_streams_at_once():
    """Sequences that share the pages of a common beginning; two calls on two
    streams with workspaces of their own."""
    nv = nvm()
    rng = np.random.default_rng(27)
    host = ref.Cache(20, 2, 16, 256, rng)
    dev = device_cache(host)
    table = np.array([[4, 9, 9, 7, 1], [4, 9, 9, 3, 2], [4, 9, 9, 3, 2]], np.int32)   # one page twice as well
    cu, lens = [0, 2, 3, 5], [70, 66, 80]
    q = normal(rng, (5, 16, 256))
    want, bound, _ = ref.attention(q, host, table, cu, lens, 1 / 16)
    s, qd = seqs(cu, lens, table, 2), bf(q)
    one = nv.kv8_attention(qd, dev, s)
    assert np.all(np.abs(f64(one) - want) <= bound)
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [nv.kv8_attention_workspace(dev, s, 16, 5) for _ in streams]
    outs = [torch.zeros_like(one) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, ws, out in zip(streams, wss, outs):
            with torch.cuda.stream(st):
                nv.kv8_attention(qd, dev, s, workspace=ws, out=out)
    torch.cuda.synchronize()
    assert all(torch.equal(o, one) for o in outs)


def test_cache_past_two_gigabytes():
    """Pages whose code offsets pass 2^31 and 2^32 bytes."""
    nv = nvm()
    rng = np.random.default_rng(25)
    hk, P, dim = 4, 64, 256                           # 64 KiB a page for K
    pages = (1 << 32) // (hk * P * dim) + 9
    dev = nv.KV8Cache.empty(pages, hk, dim, P)
    table = np.array([[pages - 1, 3, pages // 2 + 1, pages - 5]], np.int32)
    n = 200
    k, v = normal(rng, (n, hk, dim)), normal(rng, (n, hk, dim))
    s = seqs([0, n], [n], table, n)
    nv.kv8_append(dev, s, bf(k), bf(v))
    small = ref.Cache(4, hk, P, dim)
    near = np.array([[0, 1, 2, 3]], np.int32)
    small.append(near, [0, n], [n], k, v)
    got = nv.kv8_read(dev, s, rows=n)
    for g, w in zip(got, small.values(near, 0, n)):
        assert np.array_equal(f64(g), w.transpose(1, 0, 2))
    q = normal(rng, (2, 8, dim))
    want, bound, _ = ref.attention(q, small, near, [0, 2], [n], dim ** -0.5)
    out = nv.kv8_attention(bf(q), dev, seqs([0, 2], [n], table, 2))
    assert np.all(np.abs(f64(out) - want) <= bound)


def test_streams_and_graph_replays():
    """On a side stream, captured: every replay equals the eager result, with
    eager work between replays and lengths that change on the device."""
    nv = nvm()
    rng = np.random.default_rng(26)
    hk, hq, dim, P, B, n = 2, 16, 256, 16, 3, 2
    table = rng.permutation(3 * 40).reshape(3, 40).astype(np.int32)
    host = ref.Cache(3 * 40, hk, P, dim, rng)
    dev = device_cache(host)
    start = dev.k_codes.clone(), dev.k_scales.clone(), dev.v_codes.clone(), dev.v_scales.clone()
    q, k, v = (bf(rng.normal(0, 1, (B * n, h, dim))) for h in (hq, hk, hk))
    freq = torch.from_numpy(1e6 ** (-np.arange(0, 64, 2) / 64)).cuda()
    lens = i32([50, 600, 17])
    s = nv.KV8Seqs(i32([0, 2, 4, 6]), lens, i32(table), max_rows=n)
    q_out, out = torch.empty_like(q), torch.empty_like(q)
    kb, vb = (torch.empty((B * n, hk, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = nv.kv8_attention_workspace(dev, s, hq, B * n)

    def step():
        nv.rope_kv8_append(dev, s, q, k, v, freq, q_out=q_out)
        nv.kv8_attention(q_out, dev, s, workspace=ws, out=out)
        nv.kv8_read(dev, s, k_out=kb, v_out=vb)

    def reset():
        for t, o in zip((dev.k_codes, dev.k_scales, dev.v_codes, dev.v_scales), start):
            t.copy_(o)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    cases = [[50, 600, 17], [52, 640, 2], [3, 199, 400], [2, 2, 2]]
    eager = []
    for x in cases:
        reset()
        lens.copy_(i32(x))
        step()
        torch.cuda.synchronize()
        eager.append([t.clone() for t in (q_out, out, kb, vb)])
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
        with torch.cuda.graph(g, stream=side):
            step()
    torch.cuda.synchronize()
    for rep in range(2):
        for x, want in zip(cases, eager):
            reset()
            lens.copy_(i32(x))
            for t in (q_out, out, kb, vb):
                t.zero_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip((q_out, out, kb, vb), want):
                assert torch.equal(a, b), (rep, x)
            with torch.cuda.stream(side):
                step()
            torch.cuda.synchronize()
