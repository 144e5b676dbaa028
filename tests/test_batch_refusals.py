"""What the batch and prompt calls refuse, on the host, before anything is
launched (no GPU needed)."""
import ctypes
import os

import pytest
import torch

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_w4a16_mtp_amd", "libnvfp4_mtp.so")
built = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built (run __graft_entry__.build())")
A = ctypes.c_void_p(4096)
OFF = ctypes.c_void_p(4098)
BIG = 2 ** 31 - 1


def rows(nv, data=4096, row_stride=128, head_stride=64, heads=2, dim=64):
    return nv._HeadRows(data, row_stride, head_stride, heads, dim)


@built
def test_prompt_attention():
    import nvfp4_w4a16_mtp_amd as nv
    L, B = nv.lib(), ctypes.byref

    def call(q=None, k=None, v=None, cu=A, batch=2, n=10, max_rows=5, scale=0.1, window=0, sinks=0, out=A, stride=128):
        q, k, v = (rows(nv) if x is None else x for x in (q, k, v))
        return L.prompt_attention(B(q), B(k), B(v), cu, batch, n, max_rows, scale, window, sinks, out, stride, None)
    r = lambda **kw: rows(nv, **kw)
    for kw, rc in ((dict(batch=-1), -2), (dict(n=-1), -2), (dict(max_rows=-1), -2), (dict(window=-1), -1), (dict(sinks=-1), -1),
                   (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(scale=3e38), -1),
                   (dict(cu=None), -1), (dict(out=None), -1), (dict(cu=OFF), -3), (dict(out=ctypes.c_void_p(4104)), -3),
                   (dict(q=r(data=None)), -1), (dict(k=r(data=4104)), -3), (dict(q=r(heads=3, row_stride=192), stride=192), -2),
                   (dict(v=r(heads=1)), -2), (dict(q=r(dim=56)), -2), (dict(q=r(dim=60)), -2), (dict(k=r(head_stride=56)), -2),
                   (dict(q=r(dim=264, head_stride=264, row_stride=528), k=r(dim=264, head_stride=264, row_stride=528)), -5),
                   (dict(v=r(dim=264, head_stride=264, row_stride=528), stride=528), -5),
                   (dict(k=r(row_stride=1 << 23)), -5), (dict(v=r(row_stride=1 << 40)), -5), (dict(stride=120), -2), (dict(stride=132), -2),
                   (dict(batch=BIG, n=BIG, max_rows=BIG), -5)):
        assert call(**kw) == rc, kw
    assert call(batch=0, cu=None, out=None) == 0 and call(n=0, out=None) == 0 and call(max_rows=0, cu=None) == 0


@built
def test_plan():
    import nvfp4_w4a16_mtp_amd as nv
    L, B = nv.lib(), ctypes.byref

    def call(table=4096, held=4096, free=4096, count=4096, batch=3, max_pages=4, num_pages=9, page=16, kept=A, new=A, n=8, cu=A,
             lens=A, pos=A, slots=A, missing=A):
        p = nv._KV8Pool(table, held, free, count, batch, max_pages, num_pages, page)
        return L.kv8_plan(B(p), kept, new, n, cu, lens, pos, slots, missing, None)
    for kw, rc in ((dict(table=None), -1), (dict(held=None), -1), (dict(free=None), -1), (dict(count=None), -1), (dict(kept=None), -1),
                   (dict(new=None), -1), (dict(cu=None), -1), (dict(lens=None), -1), (dict(missing=None), -1),
                   (dict(page=8), -2), (dict(page=48), -2), (dict(page=0), -2), (dict(batch=-1), -2), (dict(max_pages=0), -2),
                   (dict(num_pages=0), -2), (dict(n=-1), -2), (dict(held=4098), -3), (dict(kept=OFF), -3), (dict(pos=OFF), -3),
                   (dict(slots=ctypes.c_void_p(4100)), -3), (dict(missing=OFF), -3)):
        assert call(**kw) == rc, kw
    assert L.kv8_plan(None, A, A, 8, A, A, A, A, A, None) == -1


@built
def test_sorted_tokens():
    import nvfp4_w4a16_mtp_amd as nv
    L = nv.lib()

    def sort(logits=A, m=40, e=8, k=2, ids=A, w=A, offsets=A, order=A, place=A, ws=A, nb=1 << 20):
        return L.moe_sort(logits, m, e, k, ids, w, offsets, order, place, ws, nb, None)
    for kw, rc in ((dict(m=-1), -2), (dict(e=0), -2), (dict(e=1025), -2), (dict(k=0), -2), (dict(k=9), -2), (dict(e=64, k=17), -2),
                   (dict(m=1 << 23), -5), (dict(ids=None), -1), (dict(w=None), -1), (dict(offsets=None), -1), (dict(order=None), -1),
                   (dict(place=None), -1), (dict(logits=OFF), -3), (dict(ids=OFF), -3), (dict(ws=OFF), -3), (dict(ws=None), -4), (dict(nb=8), -4)):
        assert sort(**kw) == rc, kw
    assert L.moe_sort_workspace_bytes(40, 8, 9) == 0 and L.moe_sort_workspace_bytes(40, 8, 2) >= 256

    def gather(x=A, dt=1, m=4, h=64, k=2, place=A, out=A):
        return L.moe_gather(x, dt, m, h, k, place, out, None)

    def combine(ys=A, dt=1, m=4, h=64, k=2, place=A, w=A, y=A, ydt=1):
        return L.moe_combine(ys, dt, m, h, k, place, w, y, ydt, None)

    def grad(dy=A, ddt=1, ys=A, dt=1, m=4, h=64, k=2, place=A, w=A, dys=A, dw=A):
        return L.moe_combine_grad(dy, ddt, ys, dt, m, h, k, place, w, dys, dw, None)
    common = ((dict(dt=2), -1), (dict(m=-1), -2), (dict(h=0), -2), (dict(h=60), -2), (dict(k=0), -2), (dict(k=17), -2),
              (dict(m=1 << 23), -5), (dict(place=None), -1), (dict(place=OFF), -3))
    for f, extra in ((gather, ((dict(x=None), -1), (dict(out=None), -1), (dict(x=ctypes.c_void_p(4104)), -3), (dict(out=OFF), -3))),
                     (combine, ((dict(ys=None), -1), (dict(y=None), -1), (dict(ydt=-1), -1), (dict(ys=OFF), -3), (dict(y=OFF), -3), (dict(w=OFF), -3))),
                     (grad, ((dict(dy=None), -1), (dict(ys=None), -1), (dict(dys=None), -1), (dict(dw=None), -1), (dict(ddt=7), -1),
                             (dict(dy=OFF), -3), (dict(ys=OFF), -3), (dict(dys=OFF), -3), (dict(dw=OFF), -3), (dict(w=OFF), -3)))):
        for kw, rc in common + extra:
            assert f(**kw) == rc, (f.__name__, kw)
        assert f(m=0) == 0


@built
def test_experts():
    import nvfp4_w4a16_mtp_amd as nv
    L, B = nv.lib(), ctypes.byref

    def call(m=20, k=2, e=8, hidden=64, inter=96, ptr=4096, x=A, logits=A, y=A, dt=0, ids=A, w=A, ws=A, nb=1 << 30):
        d = nv._MoeWeights(e, hidden, inter, *([ptr] * 9))
        return L.moe_w4a16_gemm(x, m, logits, k, B(d), y, dt, ids, w, ws, nb, None)
    for kw, rc in ((dict(m=-1), -2), (dict(k=0), -2), (dict(k=9), -2), (dict(e=0), -2), (dict(e=2000), -2), (dict(hidden=48), -2),
                   (dict(inter=0), -2), (dict(m=1 << 23), -5), (dict(ptr=None), -1), (dict(ptr=4104), -3), (dict(x=None), -1),
                   (dict(logits=None), -1), (dict(y=None), -1), (dict(ids=None), -1), (dict(w=None), -1), (dict(dt=2), -1),
                   (dict(x=ctypes.c_void_p(4104)), -3), (dict(y=OFF), -3), (dict(ids=OFF), -3), (dict(ws=None), -4), (dict(nb=100), -4),
                   (dict(ws=ctypes.c_void_p(4096 + 16)), -3)):
        assert call(**kw) == rc, kw
    assert call(m=0) == 0
    d = nv._MoeWeights(8, 64, 96, *([4096] * 9))
    assert L.moe_w4a16_gemm_workspace_bytes(20, 9, B(d)) == 0 and L.moe_w4a16_gemm_workspace_bytes(20, 2, None) == 0
    need = L.moe_w4a16_gemm_workspace_bytes(20, 2, B(d))
    assert call(nb=need - 1) == -4


@built
def test_bindings_refuse():
    import nvfp4_w4a16_mtp_amd as nv
    i32 = torch.zeros(3, dtype=torch.int32)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nv.prompt_attention(x, x, x, i32, 2)
    with pytest.raises(ValueError):
        nv.KV8Pool.empty(4, 2, 3, device="cpu")
    with pytest.raises(ValueError):
        nv.moe_sort(torch.zeros(2, 8), 2)
    with pytest.raises(ValueError):
        nv.moe_sort(None)
    o = nv.MoeOrder.empty(2, 2, 4, "cpu")
    rows = torch.zeros(2, 8)
    for f in (lambda: nv.moe_gather(rows, o), lambda: nv.moe_combine(torch.zeros(4, 8), o), lambda: nv.moe_combine_grad(rows, rows, o)):
        with pytest.raises(ValueError):
            f()
    for args in ((2 ** 31, 2, 8), (4, 2 ** 31, 8), (4, 2, 2 ** 32 + 8)):
        with pytest.raises(ValueError):
            nv.moe_sort_workspace(*args, "cpu")
    with pytest.raises(nv.NVFP4Error):
        nv.moe_sort_workspace(4, 9, 8, "cpu")
