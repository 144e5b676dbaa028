"""CPU: the plain forms against facts of the formats, the frequency tables
against closed forms, and the refusals of the attention and verification calls
(host checks, nothing is launched)."""
import ctypes
import os

import numpy as np
import pytest
import torch

from tests import kv_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "nvfp4_w4a16_mtp_amd", "libnvfp4_mtp.so")
built = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built (run __graft_entry__.build())")


def test_e4m3_table_and_rounding():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref.E4M3, equal_nan=True)
    x = np.concatenate([np.random.default_rng(0).normal(0, s, 20000) for s in (1e-3, 0.02, 1.0, 100.0)])
    x = np.concatenate([x, (ref._GRID[1:] + ref._GRID[:-1]) / 2, -(ref._GRID[1:] + ref._GRID[:-1]) / 2]).clip(-448, 448)
    x = np.float32(x).astype(np.float64)
    want = torch.from_numpy(np.float32(x)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_encode(x), want)
    assert np.array_equal(ref.e4m3_encode([449.0, -1e30, np.inf, 0.0, -0.0]), [0x7E, 0xFE, 0x7E, 0, 0x80])


def test_scale_exponent_is_the_smallest():
    for amax in (448.0, np.nextafter(448.0, 1e9), 449.0, 1.75, 1.75 * 1.01, 3.3e38, 1e-20, 5e-324, 0.0):
        e = ref.scale_exp(amax)
        assert amax <= 448.0 * 2.0 ** e
        assert e == ref.MIN_EXP or amax > 448.0 * 2.0 ** (e - 1)


def test_bf16_rounding():
    x = np.random.default_rng(1).normal(0, 3, 4096)
    assert np.array_equal(ref.bf16(x), torch.from_numpy(np.float32(x)).to(torch.bfloat16).double().numpy())


def test_append_continues_and_restarts_pages():
    rng = np.random.default_rng(2)
    c = ref.Cache(4, 1, 16, 64)
    table = np.array([[2, 1]])
    x = ref.bf16(rng.normal(0, 1, (20, 1, 64)))
    whole = c.clone()
    whole.append(table, [0, 20], [20], x, x)
    steps = c.clone()
    for i in range(20):
        steps.append(table, [0, 1], [i + 1], x[i:i + 1], x[i:i + 1])
    # powers of two: re-rounding a code to a larger scale changes subnormals alone
    assert np.array_equal(whole.ks, steps.ks)
    a, b = whole.values(table, 0, 20)[0], steps.values(table, 0, 20)[0]
    step = 2.0 ** (whole.ks[[2, 1]].max() - 127.0 - 9)
    assert np.abs(a - b).max() <= step and (a != b).mean() < 0.05
    # a page that is written from its first token forgets its old scale
    steps.append(table, [0, 16], [16], x[:16] * 2.0 ** -10, x[:16] * 2.0 ** -10)
    assert steps.ks[2, 0] == whole.ks[2, 0] - 10


def test_rotation_is_orthogonal_and_relative():
    rng = np.random.default_rng(3)
    x, y = rng.normal(0, 1, (1, 1, 32)), rng.normal(0, 1, (1, 1, 32))
    f = 10000.0 ** (-np.arange(0, 32, 2) / 32)
    for inter in (False, True):
        dots = [float((ref.rotate(x, [p + 7], f, 32, inter) * ref.rotate(y, [p], f, 32, inter)).sum()) for p in (0, 5, 1000)]
        assert np.allclose(dots, dots[0], rtol=1e-9)


def test_rope_frequencies():
    import nvfp4_w4a16_mtp_amd as nv
    f, m = nv.rope_frequencies(64, 1e7, device="cpu")
    assert f.dtype == torch.float64 and m == 1.0 and f[0] == 1.0
    assert np.allclose(f.numpy(), 1e7 ** (-np.arange(0, 64, 2) / 64), rtol=1e-14)
    g, m = nv.rope_frequencies(64, 1e7, scaling="linear", factor=4.0, device="cpu")
    assert np.allclose(g.numpy() * 4, f.numpy()) and m == 1.0
    g, _ = nv.rope_frequencies(64, 1e4, scaling="base", factor=8.0, device="cpu")
    h, _ = nv.rope_frequencies(64, 1e4, device="cpu")
    assert g[0] == 1.0 and np.isclose(float(h[-1] / g[-1]), 8.0)      # the slowest pair is stretched by factor
    g, m = nv.rope_frequencies(128, 1e4, scaling="by_parts", factor=8.0, original_len=4096, device="cpu")
    h, _ = nv.rope_frequencies(128, 1e4, device="cpu")
    turns = 4096 * h / (2 * np.pi)
    ratio = (h / g).numpy()
    assert np.all(ratio[turns.numpy() > 32] == 1.0) and np.allclose(ratio[turns.numpy() < 1], 8.0)
    assert np.all(np.diff(ratio) >= -1e-12) and np.isclose(m, 1 + 0.1 * np.log(8))
    for bad in (dict(rot_dim=24), dict(rot_dim=64, base=0.0), dict(rot_dim=64, factor=0.5), dict(rot_dim=64, scaling="x")):
        with pytest.raises(ValueError):
            nv.rope_frequencies(device="cpu", **bad)


def test_verify_keeps_the_target_distribution():
    """Drawn over many random numbers, accepted-or-drawn tokens follow p."""
    rng = np.random.default_rng(4)
    vocab, n = 5, 6000
    p, q = rng.normal(0, 1, vocab), rng.normal(0, 1, vocab)
    pq = [np.exp(x) / np.exp(x).sum() for x in (p, q)]
    for outright in (False, True):
        count = np.zeros(vocab)
        for _ in range(n):
            d = int(np.argmax(q)) if outright else int(rng.choice(vocab, p=pq[1]))
            _, tokens, _, _ = ref.verify(np.stack([p, p]), [0, 2], [d, 0], rng.random(2), rng.random(1),
                                         draft=None if outright else np.stack([q, q]))
            count[tokens[0]] += 1
        # five standard deviations of a binomial share
        assert np.all(np.abs(count / n - pq[0]) < 5 * np.sqrt(pq[0] * (1 - pq[0]) / n))


# ---------------------------------------------------------------- refusals
A = ctypes.c_void_p(4096)


def _cache(nv, **kw):
    d = dict(k_codes=4096, k_scales=4096, v_codes=4096, v_scales=4096, num_pages=8, page_tokens=16, kv_heads=2, head_dim=64)
    d.update(kw)
    return nv._KV8Cache(*[d[n] for n, _ in nv._KV8Cache._fields_])


def _seqs(nv, **kw):
    d = dict(cu_rows=4096, kv_lens=4096, block_table=4096, batch=2, rows=4, max_rows=2, max_pages=4, max_kv_len=0)
    d.update(kw)
    return nv._KV8Seqs(*[d[n] for n, _ in nv._KV8Seqs._fields_])


def _rows(nv, **kw):
    d = dict(data=4096, row_stride=128, head_stride=64, heads=2, dim=64)
    d.update(kw)
    return nv._HeadRows(*[d[n] for n, _ in nv._HeadRows._fields_])


BAD_CACHE = [(dict(k_codes=0), -1), (dict(v_scales=0), -1), (dict(num_pages=0), -2), (dict(page_tokens=24), -2),
             (dict(page_tokens=256), -2), (dict(head_dim=96), -2), (dict(head_dim=320), -2), (dict(kv_heads=0), -2),
             (dict(k_codes=4104), -3), (dict(v_codes=4097), -3)]
BAD_SEQS = [(dict(cu_rows=0), -1), (dict(kv_lens=0), -1), (dict(block_table=0), -1), (dict(batch=-1), -2),
            (dict(rows=-1), -2), (dict(max_rows=0), -2), (dict(max_pages=0), -2), (dict(max_kv_len=-1), -2),
            (dict(kv_lens=4098), -3)]
BAD_ROWS = [(dict(data=0), -1), (dict(heads=0), -2), (dict(dim=60), -2), (dict(row_stride=-128), -2), (dict(row_stride=100), -2),
            (dict(head_stride=56), -2), (dict(data=4104), -3)]


@built
@pytest.mark.parametrize("call", ["append", "rope_append", "read", "attention"])
def test_cache_calls_refuse(call):
    import nvfp4_w4a16_mtp_amd as nv
    L = nv.lib()
    B = ctypes.byref
    rope = nv._Rope(4096, 32, 0, 1.0)

    def go(c, s, r, rp=rope):
        if call == "append":
            return L.kv8_append(B(c), B(s), B(r), B(_rows(nv)), None)
        if call == "rope_append":
            return L.rope_kv8_append(B(c), B(s), B(rp), B(_rows(nv)), B(_rows(nv)), B(r), B(_rows(nv)), None)
        if call == "read":
            return L.kv8_read(B(c), B(s), B(r), B(_rows(nv)), None)
        return L.kv8_attention(B(r), B(c), B(s), 0.125, 0, 0, A, 128, A, 1 << 30, None)

    for bad, rc in BAD_CACHE:
        assert go(_cache(nv, **bad), _seqs(nv), _rows(nv)) == rc, bad
    for bad, rc in BAD_SEQS:
        assert go(_cache(nv), _seqs(nv, **bad), _rows(nv)) == rc, bad
    for bad, rc in BAD_ROWS:
        assert go(_cache(nv), _seqs(nv), _rows(nv, **bad)) == rc, bad
    wrong_dim = _rows(nv, dim=128, head_stride=128, row_stride=256)
    assert go(_cache(nv), _seqs(nv), wrong_dim) == -2
    assert go(_cache(nv), _seqs(nv), _rows(nv, heads=3)) == -2 and nv.lib().nvfp4_mtp_last_error()
    # nothing to do: no pointer is looked at
    for empty in (dict(batch=0), dict(rows=0)):
        none = _seqs(nv, cu_rows=0, kv_lens=0, block_table=0, **empty)
        assert go(_cache(nv), none, _rows(nv, data=0)) == 0


@built
def test_other_refusals():
    import nvfp4_w4a16_mtp_amd as nv
    L = nv.lib()
    B = ctypes.byref
    c, s, r = _cache(nv), _seqs(nv), _rows(nv)
    # rope
    for bad, rc in ((dict(inv_freq=0), -1), (dict(rot_dim=24), -2), (dict(rot_dim=80), -2), (dict(rot_dim=0), -2),
                    (dict(inv_freq=4100), -3)):
        d = dict(inv_freq=4096, rot_dim=32, interleaved=0, mscale=1.0)
        d.update(bad)
        rp = nv._Rope(d["inv_freq"], d["rot_dim"], d["interleaved"], d["mscale"])
        assert L.rope_qk(B(r), B(r), None, None, 4, A, B(rp), None) == rc, bad
        assert L.rope_kv8_append(B(c), B(s), B(rp), None, None, B(r), B(r), None) == rc, bad
    rp = nv._Rope(4096, 32, 0, 1.0)
    assert L.rope_qk(None, None, None, None, 4, A, B(rp), None) == -1
    assert L.rope_qk(B(r), None, None, None, 4, A, B(rp), None) == -1
    assert L.rope_qk(B(r), B(r), None, None, 4, None, B(rp), None) == -1
    assert L.rope_qk(B(r), B(r), None, None, -1, A, B(rp), None) == -2
    assert L.rope_qk(B(r), B(_rows(nv, heads=3)), None, None, 4, A, B(rp), None) == -2
    assert L.rope_qk(B(r), B(_rows(nv, row_stride=256)), None, None, 4, A, B(rp), None) == -2
    assert L.rope_qk(B(r), B(r), B(_rows(nv, dim=32)), B(_rows(nv, dim=32)), 4, A, B(rp), None) == -2
    assert L.rope_qk(B(r), B(r), None, None, 4, ctypes.c_void_p(4098), B(rp), None) == -3
    assert L.kv8_read(B(c), B(s), None, None, None) == -1
    # outputs whose rows overlap (4 rows of 2 heads of 64): one row for all, rows
    # within heads, heads within rows
    for strides in (dict(row_stride=0), dict(row_stride=64), dict(row_stride=64, head_stride=128), dict(row_stride=120)):
        o = _rows(nv, **strides)
        assert L.rope_qk(B(r), B(_rows(nv, data=1 << 20, **strides)), None, None, 4, A, B(rp), None) == -2, strides
        assert L.rope_qk(None, None, B(o), B(o), 4, A, B(rp), None) == -2, strides
        assert L.rope_kv8_append(B(c), B(s), B(rp), B(r), B(_rows(nv, data=1 << 20, **strides)), B(r), B(r), None) == -2, strides
        assert L.kv8_read(B(c), B(s), B(o), None, None) == -2 and L.kv8_read(B(c), B(s), B(r), B(o), None) == -2, strides
    # attention
    q3 = _rows(nv, heads=3, row_stride=192)
    assert L.kv8_attention(B(q3), B(c), B(s), 0.1, 0, 0, A, 192, A, 1 << 30, None) == -2
    ok = (B(r), B(c), B(s))
    assert L.kv8_attention(*ok, 0.1, -1, 0, A, 128, A, 1 << 30, None) == -1
    assert L.kv8_attention(*ok, 0.1, 0, -1, A, 128, A, 1 << 30, None) == -1
    assert L.kv8_attention(*ok, float("nan"), 0, 0, A, 128, A, 1 << 30, None) == -1
    for scale in (float("inf"), 3e38, -3e38):         # times log2(e) past fp32
        assert L.kv8_attention(*ok, scale, 0, 0, A, 128, A, 1 << 30, None) == -1
    assert L.kv8_attention(*ok, 0.1, 0, 0, None, 128, A, 1 << 30, None) == -1
    assert L.kv8_attention(*ok, 0.1, 0, 0, A, 120, A, 1 << 30, None) == -2
    assert L.kv8_attention(*ok, 0.1, 0, 0, ctypes.c_void_p(4104), 128, A, 1 << 30, None) == -3
    need = L.kv8_attention_workspace_bytes(B(c), B(s), 2)
    assert need >= 256 and L.kv8_attention(*ok, 0.1, 0, 0, A, 128, A, need - 1, None) == -4
    assert L.kv8_attention(*ok, 0.1, 0, 0, A, 128, None, need, None) == -4
    assert L.kv8_attention(*ok, 0.1, 0, 0, A, 128, ctypes.c_void_p(4096 + 16), need, None) == -3
    assert L.kv8_attention_workspace_bytes(B(c), B(s), 3) == 0
    # verification
    def ver(logits=A, dt=0, stride=100, vocab=100, draft=None, dstride=0, cu=A, batch=2, rows=4, max_rows=3, ids=A, temp=None,
            ua=A, us=A, lens=None, acc=A, tok=A, nxt=A, olens=None, ws=A, nb=1 << 30):
        return L.verify_drafts(logits, dt, stride, vocab, draft, dstride, cu, batch, rows, max_rows, ids, temp, ua, us, lens, acc,
                               tok, nxt, olens, ws, nb, None)
    for kw, rc in ((dict(logits=None), -1), (dict(cu=None), -1), (dict(ids=None), -1), (dict(ua=None), -1), (dict(us=None), -1),
                   (dict(acc=None), -1), (dict(tok=None), -1), (dict(nxt=None), -1), (dict(lens=A), -1), (dict(olens=A), -1),
                   (dict(dt=2), -1), (dict(vocab=0), -2), (dict(vocab=(1 << 24) + 1, stride=1 << 25), -2), (dict(max_rows=0), -2),
                   (dict(max_rows=65), -2), (dict(batch=-1), -2), (dict(rows=-1), -2), (dict(stride=99), -2),
                   (dict(draft=A, dstride=99), -2), (dict(logits=ctypes.c_void_p(4098)), -3),
                   (dict(ids=ctypes.c_void_p(4097)), -3), (dict(ws=None), -4), (dict(nb=16), -4),
                   (dict(ws=ctypes.c_void_p(4104)), -3)):
        assert ver(**kw) == rc, kw
    assert ver(batch=0, logits=None, cu=None) == 0
    assert L.verify_drafts_workspace_bytes(2, 65, 100, 0) == 0


@built
def test_grids_past_32_bits_of_threads_are_refused():
    """By the host's own check, before anything is launched."""
    import nvfp4_w4a16_mtp_amd as nv
    L = nv.lib()
    B = ctypes.byref
    big = 2 ** 31 - 1
    c, s, r, rp = _cache(nv), _seqs(nv, batch=big, rows=big, max_rows=64), _rows(nv), nv._Rope(4096, 32, 0, 1.0)
    one = _rows(nv, heads=1)
    assert L.rope_qk(B(one), B(one), None, None, big, A, B(rp), None) == -5 and b"too large" in L.nvfp4_mtp_last_error()
    for rows in (big, (1 << 23)):                     # past 2^31 workgroups, and past 2^32 threads alone
        s = _seqs(nv, batch=rows, rows=rows, max_rows=2)
        assert L.kv8_append(B(c), B(s), B(r), B(r), None) == -5, rows
        assert L.rope_kv8_append(B(c), B(s), B(rp), B(r), B(r), B(r), B(r), None) == -5, rows
        assert L.kv8_read(B(c), B(s), B(r), B(r), None) == -5, rows
        assert L.kv8_attention(B(r), B(c), B(s), 0.125, 0, 0, A, 128, A, 1 << 62, None) == -5, rows
    assert L.verify_drafts(A, 0, 151936, 151936, None, 0, A, 1 << 14, 1 << 14, 64, A, None, A, A, None, A, A, A, None, A, 1 << 62, None) == -5


def test_frequencies_refuse():
    import nvfp4_w4a16_mtp_amd as nv
    for kw in (dict(rot_dim=24), dict(rot_dim=0), dict(rot_dim=32, base=0.0), dict(rot_dim=32, factor=0.5),
               dict(rot_dim=32, scaling="other"), dict(rot_dim=32, scaling="by_parts", low_turns=4.0, high_turns=4.0)):
        with pytest.raises(ValueError):
            nv.rope_frequencies(device="cpu", **kw)


def test_frequencies_refuse_what_is_not_finite():
    import nvfp4_w4a16_mtp_amd as nv
    inf, nan = float("inf"), float("nan")
    for kw in (dict(base=inf), dict(base=nan), dict(factor=inf, scaling="linear"), dict(factor=nan, scaling="base"),
               dict(scaling="by_parts", original_len=0), dict(scaling="by_parts", original_len=nan),
               dict(scaling="by_parts", high_turns=inf), dict(scaling="by_parts", low_turns=-inf), dict(scaling="by_parts", low_turns=nan)):
        with pytest.raises(ValueError):
            nv.rope_frequencies(32, device="cpu", **kw)
    for factor in (1e8, 1e300):                       # the stretched base is past fp64's range
        with pytest.raises(ValueError):
            nv.rope_frequencies(32, 1e300, scaling="base", factor=factor, device="cpu")
    f, _ = nv.rope_frequencies(32, 1e290, scaling="base", factor=1e8, device="cpu")
    assert torch.isfinite(f).all()


@built
def test_bindings_refuse_host_tensors_and_types():
    import nvfp4_w4a16_mtp_amd as nv
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nv.rope_qk(x, None, torch.zeros(2, dtype=torch.int32), torch.zeros(16, dtype=torch.float64))
    with pytest.raises(ValueError):
        nv.KV8Cache.empty(4, 2, 64, device="cpu").desc()
    with pytest.raises(ValueError):
        nv.verify_drafts(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                         torch.zeros(2), torch.zeros(1), 2)
