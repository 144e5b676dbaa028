"""The batch and prompt operators together, as a server runs a draft step: a
plan of the pool, rotation and append, attention over the prompts from their
own rows and from the cache, the experts, verification, and the next plan."""
import pytest
import torch

from tests import batch_ref as ref
from tests.test_gpu_moe_sorted import experts_of

pytestmark = pytest.mark.gpu


def test_prompts_then_a_verification_step():
    import nvfp4_w4a16_mtp_amd as nv
    g = torch.Generator().manual_seed(1)
    batch, hq, hk, dim, page, hidden, vocab = 5, 4, 2, 64, 16, 256, 500
    def normal(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    pool = nv.KV8Pool.empty(120, batch, 24, page)
    cache = nv.KV8Cache.empty(120, hk, dim, page)
    freq, mscale = nv.rope_frequencies(32)
    w = [nv.nvfp4_quantize(normal(n, k)) for n, k in ((dim * (hq + 2 * hk), hidden), (hidden, hq * dim), (8, hidden))]
    experts, vals = experts_of(nv, 8, hidden, 128, 2)

    def layer(x, plan, max_rows, prompts):
        """One layer over a planned batch's rows: (attention, experts' output)."""
        rows = x.shape[0]
        qkv = nv.w4a16_gemm_m128(x, w[0], out_dtype=torch.bfloat16).view(rows, hq + 2 * hk, dim)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        seqs = nv.KV8Seqs(plan.cu_rows, plan.kv_lens, pool.block_table, max_rows)
        q2, k2 = nv.rope_qk(q, k, plan.positions, freq, mscale=mscale)
        fused = nv.rope_kv8_append(cache, seqs, q, k, v, freq, mscale=mscale)
        assert torch.equal(fused, q2)
        cached = nv.kv8_attention(q2, cache, seqs)
        att = nv.prompt_attention(q2, k2, v, plan.cu_rows, max_rows) if prompts else cached
        if prompts:
            # on the cache's own values the two calls are one attention, each within its bound
            kq, vq = nv.kv8_read(cache, seqs, rows)
            same = nv.prompt_attention(q2, kq, vq, plan.cu_rows, max_rows)
            want, bound = ref.attention(q2, kq, vq, plan.cu_rows.diff().tolist(), dim ** -0.5)
            assert bool(((same.double() - cached.double()).abs() <= 2 * bound).all())
            want, bound = ref.attention(q2, k2, v, plan.cu_rows.diff().tolist(), dim ** -0.5)
            assert bool(((att.double() - want).abs() <= bound).all())
        h = nv.w4a16_gemm_m128(att.flatten(1), w[1], out_dtype=torch.bfloat16)
        logits = nv.w4a16_gemm_m128(h, w[2])
        y, ids, tw = nv.moe_w4a16_gemm(h, logits, 2, experts)
        # the same through the separate calls, with the experts in 64 bits between
        o = nv.moe_sort(logits, 2)
        assert torch.equal(o.topk_ids, ids) and torch.equal(o.topk_w, tw)
        xs = nv.moe_gather(h, o)
        off = o.offsets.tolist()
        ys = torch.zeros((rows * 2, hidden))
        for e in range(8):
            r = xs[off[e]:off[e + 1]].double().cpu()
            a = torch.nn.functional.silu(r @ vals[0][e].t()) * (r @ vals[1][e].t())
            ys[off[e]:off[e + 1]] = (a @ vals[2][e].t()).float()
        y2 = nv.moe_combine(ys.cuda(), o)
        want, bound = ref.experts_ffn(h, ids.cpu().numpy(), tw.double().cpu().numpy(), *vals)
        assert bool(((y.double().cpu() - want).abs() <= bound + 2.0 ** -23 * want.abs()).all())
        assert bool(((y2.double().cpu() - want).abs() <= bound + 2.0 ** -22 * want.abs() + 1e-6).all())
        return y

    # prompts
    n = [70, 1, 130, 16, 33]
    plan = nv.kv8_plan(pool, i32([0] * batch), i32(n), sum(n))
    assert int(plan.missing) == 0 and plan.slots.min() >= 0 and len(set(plan.slots.tolist())) == sum(n)
    layer(normal(sum(n), hidden), plan, max(n), True)
    # three drafts and their token each, verified; one request ends
    lens, rows = plan.kv_lens, 4 * batch
    plan = nv.kv8_plan(pool, lens, i32([4] * batch), rows)
    assert plan.kv_lens.tolist() == [a + 4 for a in n]
    layer(normal(rows, hidden), plan, 4, False)
    logits = torch.randn((rows, vocab), generator=g).cuda()
    drafts = logits.argmax(1).to(torch.int32)
    drafts[1] = (drafts[1] + 1) % vocab               # request 0 keeps one draft
    v = nv.verify_drafts(logits, plan.cu_rows, drafts, torch.zeros(rows, device="cuda"), torch.zeros(batch, device="cuda"), 4,
                         temperature=torch.zeros(batch, device="cuda"), kv_lens=plan.kv_lens)
    assert v.accepted.tolist() == [1, 3, 3, 3, 3]
    kept = v.kv_lens.clone()
    assert kept.tolist() == [n[0] + 2] + [a + 4 for a in n[1:]]
    kept[3] = 0
    new = i32([4, 4, 4, 0, 4])
    before = int(pool.free_count)
    plan = nv.kv8_plan(pool, kept, new, 16)
    want = [-(-x // page) for x in plan.kv_lens.tolist()]
    assert pool.held.tolist() == want and int(pool.free_count) == 120 - sum(want) and want[3] == 0 and int(pool.free_count) >= before - 4
    layer(normal(16, hidden), plan, 4, False)
