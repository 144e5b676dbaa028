"""verify_drafts against its plain 64-bit form, and a run of draft step,
target step and verification together."""
import numpy as np
import pytest
import torch

from tests import kv_ref as ref

pytestmark = pytest.mark.gpu


def nvm():
    import nvfp4_w4a16_mtp_amd as nv
    return nv


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def f32(a):
    return torch.tensor(np.asarray(a, np.float32), device="cuda")


def check(logits, cu, ids, ua, us, temp=None, draft=None, lens=None, max_rows=8, dtype=torch.float32, pad=0):
    nv = nvm()
    rows, vocab = logits.shape

    def dev(x):
        t = torch.full((rows, vocab + pad), float("nan"), dtype=dtype, device="cuda")[:, :vocab]
        t.copy_(torch.from_numpy(np.float32(x)))
        return t
    tl = dev(logits)
    td = dev(draft) if draft is not None else None
    want = ref.verify(tl.double().cpu().numpy(), cu, ids, np.float32(ua), np.float32(us),
                      None if temp is None else np.float32(temp), None if td is None else td.double().cpu().numpy(), lens, max_rows)
    got = nv.verify_drafts(tl, i32(cu), i32(ids), f32(ua), f32(us), max_rows,
                           temperature=None if temp is None else f32(temp), draft_logits=td,
                           kv_lens=None if lens is None else i32(lens),
                           out=None if lens is not None else nv.Verified(i32(np.zeros(len(cu) - 1)), i32(np.full(rows, -999)),
                                                                         i32(np.zeros(len(cu) - 1)), None))
    for name, g, w in zip(("accepted", "tokens", "next", "kv_lens"), got, want):
        if w is None:
            assert g is None
            continue
        g, w = g.cpu().numpy(), np.asarray(w)
        if name == "tokens":
            keep = w != -999
            g, w = g[keep], w[keep]
        assert np.array_equal(g, w), (name, g, w)
    return want


def make(rng, ns, vocab, peak=4.0, agree=0.7):
    """Target logits, draft logits near them, drafts, random numbers."""
    cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int64)
    rows = int(cu[-1])
    logits = rng.normal(0, peak, (rows, vocab))
    draft = logits + rng.normal(0, agree, (rows, vocab))
    ids = np.array([int(np.argmax(draft[r] + rng.gumbel(0, 1, vocab))) for r in range(rows)]) if rows else np.zeros(0, int)
    return cu, logits, draft, ids, rng.random(rows), rng.random(len(ns))


@pytest.mark.parametrize("vocab", [1, 2, 7, 1000, 2048, 4097, 33000, 151936])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sampled", [False, True])
def test_verify(vocab, dtype, sampled):
    rng = np.random.default_rng(vocab)
    ns = [1, 4, 0, 2, 8, 3]
    cu, logits, draft, ids, ua, us = make(rng, ns, vocab, peak=3.0 if vocab < 5000 else 6.0)
    out = check(logits, cu, ids, ua, us, temp=[0.7, 1.0, 1.0, 2.0, 0.9, 0.0], draft=draft if sampled else None,
                lens=[100, 200, 5, 7, 8, 9], dtype=dtype, pad=3 if vocab in (7, 4097) else 0)
    assert out[2][2] == -1 and out[0][2] == 0 and out[3][2] == 5


@pytest.mark.parametrize("sampled", [False, True])
def test_verify_many_sequences(sampled):
    rng = np.random.default_rng(3)
    ns = [int(x) for x in rng.integers(1, 7, 200)]
    cu, logits, draft, ids, ua, us = make(rng, ns, 3001, peak=2.0, agree=0.4)
    out = check(logits, cu, ids, ua, us, draft=draft if sampled else None, lens=rng.integers(10, 1000, 200))
    # both outcomes occur.  An outright draft stands with its own p, on average sum p^2
    # = e^(peak^2) / vocab = 0.018 here, so only a few of the 499 do
    assert 0 < out[0].sum() < sum(ns) - len(ns)


@pytest.mark.parametrize("sampled", [False, True])
def test_verify_border_random_numbers(sampled):
    """u = 0 and the largest fp32 below 1, flat and peaked rows, equal models."""
    rng = np.random.default_rng(4)
    top = float(np.float32(1) - np.float32(2.0 ** -24))
    for vocab in (5, 3000):
        cu, logits, draft, ids, _, _ = make(rng, [3] * 8, vocab)
        logits[0:6] = 0.25                            # flat
        logits[6:9, :] = -50.0
        logits[6:9, vocab // 2] = 60.0                # one token has all the mass
        ids[6:9] = vocab // 2
        draft[12:18] = logits[12:18]                  # equal models
        logits[18:21, ::2] = -np.inf                  # half the tokens masked out
        for ua in (0.0, top):
            for us in (0.0, 0.5, top):
                check(logits, cu, ids, np.full(24, ua), np.full(8, us), draft=draft if sampled else None)


@pytest.mark.parametrize("batch", [1, 80])
def test_verify_first_draw_behind_masked_chunks(batch):
    """u_sample = 0 with nothing but the fallen draft in the first chunks."""
    vocab, live = 20000, [14000, 14001, 19999]
    logits = np.full((2 * batch, vocab), -np.inf)
    logits[:, live] = 1.0
    logits[::2, 17] = 1.5
    cu, ids = np.arange(0, 2 * batch + 1, 2), np.full(2 * batch, 17)
    out = check(logits, cu, ids, np.full(2 * batch, 0.999), np.zeros(batch))
    assert np.all(out[0] == 0) and np.all(out[2] == 14000)


@pytest.mark.parametrize("sampled", [False, True])
def test_verify_rows_without_a_softmax(sampled):
    """NaN, +inf, nothing above -inf: the greedy scan; ids out of range fall."""
    rng = np.random.default_rng(5)
    vocab = 5000
    cu, logits, draft, ids, ua, us = make(rng, [2] * 9, vocab)
    ua[:] = 0.0
    logits[0, 17] = np.nan
    ids[0] = ref.first_max(logits[0])
    logits[2, [4000, 9]] = np.inf
    ids[2] = 9
    logits[4] = -np.inf
    ids[4] = 0
    logits[6] = np.nan
    ids[6] = 3
    logits[9] = -np.inf                               # a last row
    ids[10], ids[12] = -1, vocab
    draft[14] = np.nan                                # the draft's row has no softmax: an outright draft
    draft[16] = -np.inf
    ua[14], ua[16] = 0.999, 0.999
    logits[14, ids[14]] = -np.inf
    out = check(logits, cu, ids, ua, us, draft=draft if sampled else None)
    assert out[0][0] == 1 and out[0][1] == 1 and out[0][2] == 1 and out[0][3] == 0 and out[0][5] == 0 and out[0][6] == 0


@pytest.mark.parametrize("sampled", [False, True])
@pytest.mark.parametrize("vocab,batch", [(3000, 3), (20011, 60)])
def test_verify_far_from_zero(vocab, batch, sampled):
    """Logits with a large common offset, tokens masked with the type's lowest
    value, temperatures at the ends of fp32."""
    rng = np.random.default_rng(vocab)
    cu, logits, draft, ids, ua, us = make(rng, [3] * batch, vocab, peak=3.0)
    logits, draft = np.round(logits * 64) / 64 + 30000.0, np.round(draft * 64) / 64 + 30000.0
    lowest = float(np.finfo(np.float32).min)
    for r in range(0, len(ids), 4):
        mask = rng.random(vocab) < 0.9
        mask[ids[r]] = False
        logits[r, mask], draft[r, mask] = lowest, lowest
    temp = rng.choice([0.3, 1.0, 1.7], batch)
    temp[:3] = [1e-38, 3e38, 0.02]
    check(logits, cu, ids, ua * 0.3, us, temp=temp, draft=draft if sampled else None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab,batch", [(3000, 3), (20011, 60)])
def test_verify_logits_further_apart_than_fp32_holds(vocab, batch, dtype):
    """Finite logits at both ends of fp32 under temperatures that let both count:
    a sum without the lower ones would be about half, and random numbers 1.3 times
    p(d) would let drafts stand."""
    rng = np.random.default_rng(vocab + 1)
    rows = 3 * batch
    logits = np.where(rng.random((rows, vocab)) < 0.1, 3.3e38, -3.3e38) * rng.uniform(0.9, 1.0, (rows, vocab))
    logits = torch.from_numpy(np.float32(logits)).to(dtype).double().numpy()
    ids = logits.argmax(1)
    temp = np.float32(rng.choice([2.5e38, 3e38, 3.4e38], batch))
    p = np.array([1 / ref.softmax(logits[r], float(temp[r // 3]))[1] for r in range(rows)])
    ua = p * np.where(np.arange(rows) % 3 == 0, 0.7, 1.3)
    out = check(logits, np.arange(0, rows + 1, 3), ids, ua, rng.random(batch), temp=temp, dtype=dtype)
    assert np.all(out[0] == 1)


def test_verify_temperatures():
    rng = np.random.default_rng(6)
    cu, logits, draft, ids, ua, us = make(rng, [3] * 8, 2000)
    logits[0] = logits[0].round()                     # ties among greedy maxima
    logits[3, [5, 900]] = 99.0
    ids[3] = 5
    logits[6, [5, 900]] = 99.0
    ids[6] = 900
    for d in (None, draft):
        out = check(logits, cu, ids, ua, us, temp=[0.0, 0.0, -1.0, np.inf, np.nan, 1e-30, 100.0, 0.3], draft=d)
        assert out[0][1] >= 1 and out[0][2] == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sampled", [False, True])
@pytest.mark.parametrize("batch,vocab,most", [(56, 151936, 4), (300, 33003, 3)])
def test_verify_large_batches(batch, vocab, most, sampled, dtype):
    """Rows and sequences enough that a wavefront takes a chunk alone, in the first
    pass and in the second."""
    rng = np.random.default_rng(batch)
    ns = [int(x) for x in rng.integers(1, most + 1, batch)]
    ns[batch // 2] = 0
    cu, logits, draft, ids, ua, us = make(rng, ns, vocab, peak=4.0)
    temp = rng.choice([0.4, 0.7, 1.0, 0.0], batch)
    out = check(logits, cu, ids, ua * 0.5, us, temp=temp, draft=draft if sampled else None, lens=rng.integers(10, 1000, batch), dtype=dtype)
    assert 0 < out[0].sum() < sum(ns) - batch


def check_next_to_the_border(batch, vocab, sampled, dtype, of_draft):
    """u_accept 2^-17 to 2^-22 of it below, at and above min(p(d) / q(d), 0.999).
    Drafts: the target's first choices, or the draft model's."""
    rng = np.random.default_rng(vocab)
    cu, logits, draft, ids, ua, us = make(rng, [2] * batch, vocab, peak=2.0)
    ids = (draft if of_draft else logits).argmax(1)
    temp = np.float32(rng.uniform(0.5, 1.5, batch))

    def seen(x):
        return torch.from_numpy(np.float32(x)).to(dtype).double().numpy()
    ua = np.zeros(2 * batch, np.float32)
    want = []
    for b in range(batch):
        (e, total), d = ref.softmax(seen(logits[2 * b]), float(temp[b])), ids[2 * b]
        border = e[d] / total
        if sampled:
            e, total = ref.softmax(seen(draft[2 * b]), float(temp[b]))
            border /= e[d] / total
        near = np.float32(min(border, 0.999) * (1 + [0.0, 1.0, -1.0][b % 3] * 2.0 ** -rng.integers(17, 23)))
        # the oracle's and the kernel's fp64 sums are off by less than 1e-11 relative
        while abs(float(near) / border - 1) < 1e-10:
            near = np.nextafter(near, np.float32(0))
        ua[2 * b] = near
        want.append(int(float(near) < border))
    out = check(logits, cu, ids, ua, us, temp=temp, draft=draft if sampled else None, dtype=dtype)
    assert np.array_equal(out[0], want)
    return want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sampled", [False, True])
@pytest.mark.parametrize("batch,vocab", [(6, 5000), (70, 20011), (300, 33003)])
def test_verify_random_numbers_next_to_the_border(batch, vocab, sampled, dtype):
    """Closer to the border than fp32 sums can tell."""
    want = check_next_to_the_border(batch, vocab, sampled, dtype, False)
    if not sampled:                                   # (a draft model that finds them less likely: they stand)
        assert 0 < sum(want) < batch


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,vocab", [(70, 20011), (300, 33003)])
def test_verify_sampled_random_numbers_next_to_the_border(batch, vocab, dtype):
    want = check_next_to_the_border(batch, vocab, True, dtype, True)
    assert 0 < sum(want) < batch


def test_verify_rows_bounds_and_aliasing():
    nv = nvm()
    rng = np.random.default_rng(7)
    cu, logits, draft, ids, ua, us = make(rng, [5, 9, 1], 700)
    check(logits, cu, ids, ua, us, max_rows=4, lens=[50, 60, 70])    # longer sequences are cut to max_rows
    lens = i32([50, 60, 70])
    args = (f32(logits), i32(cu), i32(ids), f32(ua), f32(us), 9)
    want = nv.verify_drafts(*args, kv_lens=i32([50, 60, 70]))
    out = nv.Verified(want.accepted.clone(), want.tokens.clone(), want.next.clone(), lens)
    nv.verify_drafts(*args, kv_lens=lens, out=out)
    assert torch.equal(lens, want.kv_lens)
    # row ranges past the rows are cut
    got = nv.verify_drafts(f32(logits), i32([0, 5, 14, 400]), i32(ids), f32(ua), f32(us), 9)
    assert torch.equal(got.accepted, want.accepted) and torch.equal(got.tokens, want.tokens)


def test_verify_graph_replays():
    nv = nvm()
    rng = np.random.default_rng(8)
    ns = [4, 2, 5]
    sets = [make(rng, ns, 20000) for _ in range(3)]
    bufs = [f32(sets[0][1]), i32(sets[0][3]), f32(sets[0][4]), f32(sets[0][5]), f32(sets[0][2])]
    cu, lens = i32(sets[0][0]), i32([30, 40, 50])
    for sampled in (False, True):
        ws = nv.verify_workspace(5, 3, 20000, "cuda", sampled=sampled)
        out = nv.verify_drafts(bufs[0], cu, bufs[1], bufs[2], bufs[3], 5, kv_lens=lens, workspace=ws,
                               draft_logits=bufs[4] if sampled else None)

        def step():
            nv.verify_drafts(bufs[0], cu, bufs[1], bufs[2], bufs[3], 5, kv_lens=lens, workspace=ws, out=out,
                             draft_logits=bufs[4] if sampled else None)

        def load(x):
            for t, a in zip(bufs, (x[1], x[3], x[4], x[5], x[2])):
                t.copy_(torch.from_numpy(np.asarray(a)).to(t.dtype))
        eager = []
        for x in sets:
            load(x)
            step()
            torch.cuda.synchronize()
            eager.append([t.clone() for t in out])
        side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            with torch.cuda.graph(g, stream=side):
                step()
        torch.cuda.synchronize()
        for rep in range(2):
            for x, want in zip(sets, eager):
                load(x)
                for t in out:
                    t.zero_()
                torch.cuda.synchronize()
                g.replay()
                torch.cuda.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(out, want)), (sampled, rep)
                with torch.cuda.stream(side):
                    step()
                torch.cuda.synchronize()


@pytest.mark.parametrize("sampled", [False, True])
def test_verify_longest_sequences(sampled):
    """64 rows, the bound; drafts that mostly stand."""
    rng = np.random.default_rng(11)
    ns = [64, 33, 1, 64]
    cu, logits, draft, ids, ua, us = make(rng, ns, 1500)
    ids = logits.argmax(1)
    logits[np.arange(len(ids)), ids] += 20.0
    draft[np.arange(len(ids)), ids] += 19.0
    ids[40] = (ids[40] + 1) % 1500
    out = check(logits, cu, ids, ua * 0.9, us, draft=draft if sampled else None, lens=[70, 40, 9, 64], max_rows=64)
    # (a sampled draft that neither model finds likely stands or falls with u)
    assert list(out[0][1:]) == [32, 0, 63] and (sampled or out[0][0] == 40)


def test_verify_nothing_to_verify():
    """No rows at all, and sequences that are all empty."""
    nv = nvm()
    for rows in (0, 3):
        logits = torch.zeros((rows, 50), device="cuda")
        tokens = torch.full((rows,), 9, dtype=torch.int32, device="cuda")
        out = nv.Verified(i32([7, 7]), tokens, i32([7, 7]), i32([7, 7]))
        nv.verify_drafts(logits, i32([0, 0, 0]), i32(np.zeros(rows)), f32(np.zeros(rows)), f32([0.5, 0.5]), 4, kv_lens=i32([3, 0]), out=out)
        assert out.accepted.tolist() == [0, 0] and out.next.tolist() == [-1, -1] and out.kv_lens.tolist() == [3, 0]
        assert bool((tokens == 9).all())


@pytest.mark.parametrize("sampled", [False, True])
def test_verify_two_streams_at_once_and_replays_of_large_batches(sampled):
    """Two calls on two streams with workspaces of their own, and a captured one
    replayed between eager ones."""
    nv = nvm()
    sets = [make(np.random.default_rng(s), [3] * 70, 20011) for s in (12, 13)]
    streams, calls, wants = [torch.cuda.Stream() for _ in sets], [], []
    for cu, logits, draft, ids, ua, us in sets:
        args = (f32(logits), i32(cu), i32(ids), f32(ua * 0.5), f32(us), 3)
        kw = dict(draft_logits=f32(draft) if sampled else None, kv_lens=i32(np.full(70, 40)),
                  workspace=nv.verify_workspace(3, 70, 20011, "cuda", sampled=sampled))
        wants.append([t.clone() for t in nv.verify_drafts(*args, **kw)])
        out = nv.Verified(*(torch.zeros_like(t) for t in wants[-1]))
        calls.append(lambda args=args, kw=kw, out=out: nv.verify_drafts(*args, out=out, **kw))
    assert not torch.equal(wants[0][1], wants[1][1])
    torch.cuda.synchronize()
    for _ in range(10):
        outs = []
        for st, call in zip(streams, calls):
            with torch.cuda.stream(st):
                outs.append(call())
    torch.cuda.synchronize()
    for out, want in zip(outs, wants):
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(streams[0]):
        with torch.cuda.graph(g, stream=streams[0]):
            calls[0]()
    for _ in range(3):
        for t in outs[0]:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[0], wants[0]))
        calls[1]()
        torch.cuda.synchronize()


def test_rounds_of_speculation():
    """Rounds as they are used: the target's rows (last token and drafts) go
    through q|k|v, the fused rotation and append, attention and o; the logits'
    verification gives the cache lengths of the next round, on the device.  The
    cache and the attention follow the plain forms round by round."""
    from tests import synth
    from tests.gpu_util import dev_bf16
    nv = nvm()
    rng = np.random.default_rng(9)
    H, hq, hk, dim, P, B, drafts, vocab = 512, 4, 2, 64, 16, 3, 3, 600
    wq, wk, wv, wo, wh = (nv.nvfp4_quantize(dev_bf16(synth.weight_bf16(i, n, k)))
                          for i, (n, k) in enumerate([(hq * dim, H), (hk * dim, H), (hk * dim, H), (H, hq * dim), (vocab, H)]))
    n = drafts + 1
    rows = B * n
    table = rng.permutation(B * 8).reshape(B, 8).astype(np.int32)
    host = ref.Cache(B * 8, hk, P, dim)
    cache = nv.KV8Cache.empty(B * 8, hk, dim, P)
    freq, mscale = nv.rope_frequencies(32, 1e4)
    cu = np.arange(0, rows + 1, n).astype(np.int32)
    kv_lens = i32([0, 0, 0])
    host_lens = np.zeros(B, np.int64)
    for rnd in range(6):
        x = dev_bf16(synth.acts_bf16(100 + rnd, rows, H))
        kv_lens += n
        host_lens += n
        s = nv.KV8Seqs(i32(cu), kv_lens, i32(table), max_rows=n)
        q, k, v = (torch.cat([nv.w4a16_gemv(x[i:i + 8], w, out_dtype=torch.bfloat16) for i in range(0, rows, 8)])
                   .view(rows, -1, dim) for w in (wq, wk, wv))
        qr = nv.rope_kv8_append(cache, s, q, k, v, freq, mscale=mscale)
        o = nv.kv8_attention(qr, cache, s)
        pos = np.concatenate([np.arange(z - n, z) for z in host_lens])
        kr = ref.bf16(ref.rotate(k.double().cpu().numpy(), pos, freq.cpu().numpy(), 32))
        host.append(table, cu, host_lens, kr, v.double().cpu().numpy())
        assert np.array_equal(cache.k_codes.cpu().numpy(), host.k) and np.array_equal(cache.k_scales.cpu().numpy(), host.ks)
        assert np.array_equal(cache.v_codes.cpu().numpy().transpose(0, 1, 3, 2), host.v)
        want, bound, _ = ref.attention(qr.double().cpu().numpy(), host, table, cu, host_lens, dim ** -0.5)
        assert np.all(np.abs(o.double().cpu().numpy() - want) <= bound)
        y = torch.cat([nv.w4a16_gemv(o.view(rows, -1)[i:i + 8], wo, out_dtype=torch.bfloat16) for i in range(0, rows, 8)])
        logits = torch.cat([nv.w4a16_gemv((x + y)[i:i + 8].contiguous(), wh) for i in range(0, rows, 8)])
        ids = logits.argmax(1).to(torch.int32)
        ids[torch.arange(rows, device="cuda") % 5 == rnd % 5] = 7     # some drafts are poor
        ua, us = torch.rand(rows, device="cuda") * 0.05, torch.rand(B, device="cuda")
        got = nv.verify_drafts(logits, i32(cu), ids, ua, us, n, temperature=f32([0.4, 0.0, 0.5]), kv_lens=kv_lens)
        ref_out = ref.verify(logits.double().cpu().numpy(), cu, ids.cpu().numpy(), ua.cpu().numpy(), us.cpu().numpy(),
                             np.float32([0.4, 0.0, 0.5]), lens=host_lens)
        for g, w in zip(got, ref_out):
            assert np.array_equal(g.cpu().numpy(), w)
        kv_lens = got.kv_lens
        host_lens = ref_out[3].astype(np.int64)
    assert host_lens.min() >= 6 and host_lens.max() <= 6 * n
