"""Performance cases of the operators that run a draft step for whole batches
and prompts: the plan of a step (block tables, positions and slots from request
lengths), attention over whole packed prompts, tokens sorted by expert and back
(with the gradient of the way back), and the expert FFN over sorted tokens.

`run` computes a case in plain torch operations, or, with `own` set, with the
library's kernels.  `exact` gives the same outputs from the definitions in
64 bits.

Packed batches: sequence b owns the rows cu_rows[b] .. cu_rows[b + 1].  Sorted
tokens: the pair t * top_k + j (token t's j-th expert) stands at place[pair],
pairs in the order of their experts and, within one, of their own numbers;
expert e's rows are offsets[e] .. offsets[e + 1] and order[place] is the pair.
"""
import math
import random

import numpy as np
import torch

own = False


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the plan of a verification step for 64 users (1 to 4 rows each, a few
        # of them finished, a few new with short prompts), and the plan that
        # follows it, where the rows have fallen and the old requests hold
        # their pages again
        dict(name="plan_decode", op="plan", batch=64, new_lo=1, new_hi=4, kept_hi=9000, prompt_hi=200, turnover=0.1, page=16,
             pool=1.2, seed=1),
        # the same for a large server's step: 700 users, of whom a tenth bring
        # prompts of up to 4000 tokens
        dict(name="plan_prompts", op="plan", batch=700, new_lo=1, new_hi=6, kept_hi=30000, prompt_hi=4000, turnover=0.2, page=64,
             pool=1.2, seed=2),
        # one user's prompt at the head's own shape (16 + 2 heads of 256)
        dict(name="prompt_one", op="attn", batch=1, rows_lo=700, rows_hi=700, seed=3, q_heads=16, kv_heads=2, dk=256, dv=256,
             window=0, sinks=0),
        # a packed batch of prompts, from a word to a long document
        dict(name="prompt_packed", op="attn", batch=24, rows_lo=1, rows_hi=4500, seed=4, q_heads=32, kv_heads=8, dk=128, dv=128,
             window=0, sinks=0),
        # one long document at the head's own shape
        dict(name="prompt_long", op="attn", batch=1, rows_lo=12001, rows_hi=12001, seed=5, q_heads=16, kv_heads=2, dk=256, dv=256,
             window=0, sinks=0),
        # documents through a sliding-window layer with sinks, with keys of 192
        # (128 and the 64 rotated ones) and values of 128, a key head a query head
        dict(name="prompt_window", op="attn", batch=3, rows_lo=3000, rows_hi=7000, seed=6, q_heads=16, kv_heads=16, dk=192, dv=128,
             window=2048, sinks=4),
        # the tokens of a verification step (24 users, 4 rows) to 256 experts
        dict(name="sort_batch", op="sort", rows=96, experts=256, top_k=8, hidden=2048, ties=True),
        # a prompt's tokens to 256 experts
        dict(name="sort_prompt", op="sort", rows=8191, experts=256, top_k=8, hidden=2048, ties=False),
        # the experts' rows of a prompt back to its tokens
        dict(name="back_prompt", op="back", rows=8191, experts=256, top_k=8, hidden=2048),
        # the gradient of that way back, at the widest hidden size
        dict(name="back_grad", op="grad", rows=2000, experts=256, top_k=8, hidden=7168),
        # the expert FFN of a verification step: 40 rows, nearly every expert's
        # weights are read for one or two of them
        dict(name="experts_batch", op="experts", rows=40, experts=256, top_k=8, hidden=2048, inter=512),
        # the expert FFN of a prompt
        dict(name="experts_prompt", op="experts", rows=4096, experts=256, top_k=8, hidden=2048, inter=512),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "attn", "attn", "sort", "back", "grad", "experts", "experts"])
    seed = rng.randrange(1 << 20)
    if op == "plan":
        lo = rng.randint(0, 3)
        return dict(op="plan", batch=_log_int(rng, 1, 700), new_lo=lo, new_hi=lo + rng.randint(0, 5), kept_hi=_log_int(rng, 10, 20000),
                    prompt_hi=_log_int(rng, 1, 3000), turnover=rng.choice([0.0, 0.05, 0.2]), page=rng.choice([16, 32, 64, 128]),
                    pool=rng.choice([0.9, 1.05, 1.5]), seed=seed)
    if op == "attn":
        heads, kv, dk, dv = rng.choice([(16, 2, 256, 256), (32, 8, 128, 128), (8, 1, 128, 128), (12, 4, 64, 64), (24, 3, 192, 192),
                                        (5, 5, 64, 64), (16, 16, 192, 128), (8, 2, 80, 80), (6, 3, 232, 104), (16, 4, 96, 96)])
        window = rng.choice([0, 0, _log_int(rng, 8, 4000)])
        batch = _log_int(rng, 1, 60)
        hi = _log_int(rng, 2, 9000)
        # no more pairs than the longest listed case, nor more rows than a batch holds
        hi = max(1, min(hi, int(9000 / math.sqrt(batch * heads * (dk + dv) / 8192.0)), 120000 // batch))
        return dict(op="attn", batch=batch, rows_lo=rng.choice([0, 1, max(1, hi // 2)]), rows_hi=hi, seed=seed, q_heads=heads,
                    kv_heads=kv, dk=dk, dv=dv, window=window, sinks=rng.choice([0, 4, 70]) if window else 0)
    experts = rng.choice([256, 256, 8, 60, 128, 512, _log_int(rng, 2, 1000)])
    top_k = min(experts, rng.choice([1, 2, 4, 6, 8, 8, 10]))
    if op == "sort":
        return dict(op="sort", rows=_log_int(rng, 1, 7000), experts=experts, top_k=top_k, hidden=8 * _log_int(rng, 8, 256),
                    ties=rng.random() < 0.5)
    if op in ("back", "grad"):
        return dict(op=op, rows=_log_int(rng, 1, 2000 if op == "grad" else 7000), experts=experts, top_k=min(top_k, 8),
                    hidden=8 * _log_int(rng, 8, 256))
    hidden, inter = 32 * rng.randint(8, 64), 32 * rng.randint(4, 16)
    experts = min(experts, 256)
    return dict(op="experts", rows=_log_int(rng, 1, 3500), experts=experts, top_k=min(top_k, 8, experts), hidden=hidden, inter=inter)


# the requests of a plan, on the host: kept and new tokens, pages held before
def _requests(case):
    r = random.Random(case["seed"] * 7919 + 13)
    kept, new, held = [], [], []
    for _ in range(case["batch"]):
        k = r.randint(1, case["kept_hi"])
        n = r.randint(case["new_lo"], case["new_hi"])
        h = -(-k // case["page"])
        x = r.random()
        if x < case["turnover"] / 2:          # finished: its pages go back
            k = n = 0
        elif x < case["turnover"]:            # new, with a prompt
            k, h, n = 0, 0, r.randint(1, case["prompt_hi"])
        elif x < case["turnover"] + 0.2:      # drafts that fell: a page or two too many
            h += r.randint(0, 2)
        kept.append(k)
        new.append(n)
        held.append(h)
    return kept, new, held


def _lengths(case):
    r = random.Random(case["seed"] * 104729 + 7)
    lo, hi = case["rows_lo"], case["rows_hi"]
    n = []
    for _ in range(case["batch"]):
        # as many short prompts as long ones
        n.append(r.randint(lo, hi) if lo > hi // 4 else min(hi, lo - 1 + _log_int(r, 1, max(1, hi - lo + 1))))
    n[-1] = hi
    return n


def _pairs(n, window, sinks):
    """(row, key) pairs that are seen in a prompt of n rows."""
    if window == 0 or n <= window:
        return n * (n + 1) // 2
    pairs = window * (window + 1) // 2 + (n - window) * window
    for s in range(sinks):                    # sink s is outside the windows of the rows from s + window on
        pairs += max(0, n - s - window)
    return pairs


def work(case):
    op = case["op"]
    if op == "plan":
        kept, new, held = _requests(case)
        rows = sum(new)
        need = [-(-(a + b) // case["page"]) for a, b in zip(kept, new)]
        moved = sum(abs(a - b) for a, b in zip(need, held))
        # lengths in and out, positions and slots, the rows' pages and the pages that move, twice
        return dict(bytes=case["batch"] * 2 * 4 * 6 + rows * 12 + sum(-(-x // case["page"]) + 1 for x in new) * 4 + moved * 2 * 8,
                    flops=0)
    if op == "attn":
        n = _lengths(case)
        pairs, rows = sum(_pairs(x, case["window"], case["sinks"]) for x in n), sum(n)
        h, kv, dk, dv = case["q_heads"], case["kv_heads"], case["dk"], case["dv"]
        return dict(bytes=rows * (h + kv) * (dk + dv) * 2, flops=pairs * h * 2 * (dk + dv))
    m, e, k, hid = case["rows"], case["experts"], case["top_k"], case["hidden"]
    if op == "sort":
        return dict(bytes=m * e * 4 + m * k * 16 + e * 4 + m * hid * 2 * (k + 1), flops=m * e * k)
    if op == "back":
        return dict(bytes=m * hid * 2 * (k + 1) + m * k * 8, flops=2 * m * k * hid)
    if op == "grad":
        return dict(bytes=m * hid * 2 * (2 * k + 1) + m * k * 12, flops=3 * m * k * hid)
    i = case["inter"]
    used = e * (1.0 - (1.0 - k / e) ** m)     # experts that some token chooses, evenly spread
    return dict(bytes=used * 3 * i * hid * 0.5625 + m * hid * 4 + m * e * 4 + m * k * 8, flops=6 * m * k * i * hid)


# ------------------------------------------------------------------ inputs
def _dev():
    return torch.device("cuda")


def _i32(a):
    return torch.tensor(a, dtype=torch.int32, device=_dev())


def _cu(n):
    return _i32([0] + [int(x) for x in np.cumsum(n)])


def prepare(case, seed):
    gen = torch.Generator(device=_dev())
    gen.manual_seed(seed)
    op = case["op"]

    def rand(shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(shape, generator=gen, device=_dev()) * std).to(dtype)

    if own:
        import nvfp4_w4a16_mtp_amd as nv
    if op == "plan":
        kept, new, held = _requests(case)
        p = case["page"]
        need = [-(-(a + b) // p) for a, b in zip(kept, new)]
        width = max(1, max(need + held))
        total = int(max(sum(held), sum(need)) * case["pool"]) + 1
        total = max(total, sum(held))
        order = np.random.default_rng(seed).permutation(total).astype(np.int32)
        table = np.full((len(kept), width), -1, np.int32)
        at = 0
        for b, c in enumerate(held):
            table[b, :c] = order[at:at + c]
            at += c
        free = np.full(total, -1, np.int32)
        free[:total - at] = order[at:]
        st = dict(case=case, kept=_i32(kept), new=_i32(new), rows=sum(new), table=torch.from_numpy(table).to(_dev()),
                  held=_i32(held), free=torch.from_numpy(free).to(_dev()), count=_i32([total - at]),
                  before=_i32([h * p for h in held]), none=_i32([0] * len(kept)))
        if own:
            st["nv"] = nv
            st["pool"] = nv.KV8Pool(st["table"], st["held"], st["free"], st["count"], p)
        return st
    if op == "attn":
        n = _lengths(case)
        rows, h, kv, dk, dv = sum(n), case["q_heads"], case["kv_heads"], case["dk"], case["dv"]
        if dk == dv:
            # q, k and v as one projection writes them, a token's heads in a row
            qkv = rand((rows, h + 2 * kv, dk))
            q, k, v = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
        else:
            q, k, v = rand((rows, h, dk)), rand((rows, kv, dk)), rand((rows, kv, dv))
        st = dict(case=case, n=n, cu=_cu(n), q=q, k=k, v=v, scale=dk ** -0.5)
        if own:
            st.update(nv=nv, out=torch.empty((rows, h, dv), dtype=torch.bfloat16, device=_dev()))
        return st
    m, e, k, hid = case["rows"], case["experts"], case["top_k"], case["hidden"]
    # experts are not equally liked
    logits = torch.randn((m, e), generator=gen, device=_dev()) * 1.5 + torch.randn((e,), generator=gen, device=_dev()) * 0.5
    if case.get("ties"):
        logits = logits.to(torch.bfloat16).float()
    st = dict(case=case, logits=logits.contiguous())
    if op in ("sort", "experts"):
        st["x"] = rand((m, hid))
    if op in ("back", "grad"):
        ids, w, _ = _route(logits, k)
        st.update(ids=ids, w=w, order=_order(ids, e), ys=rand((m * k, hid)))
        if op == "grad":
            st["dy"] = rand((m, hid), std=0.1)
    if op == "experts":
        i = case["inter"]
        count = torch.bincount(_route(logits, k)[0].flatten().long(), minlength=e)
        st["cap"] = int(count.max())

        def weight(rows, cols):
            # codes and block scales of weights with a standard deviation of about cols^-0.5
            c = torch.randint(0, 256, (e, rows, cols // 2), generator=gen, device=_dev(), dtype=torch.uint8)
            s = torch.randint(0x30, 0x40, (e, rows, cols // 16), generator=gen, device=_dev(), dtype=torch.uint8)
            g = torch.zeros((e, 4), dtype=torch.float32, device=_dev())
            g[:, 0] = 0.3 * cols ** -0.5 * (0.8 + 0.4 * torch.rand((e,), generator=gen, device=_dev()))
            return c, s, g

        st.update(gate=weight(i, hid), up=weight(i, hid), down=weight(hid, i))
    if own:
        st["nv"] = nv
        dev = _dev()
        if op == "sort":
            st.update(buffers=nv.MoeOrder.empty(m, k, e, dev), ws=nv.moe_sort_workspace(m, k, e, dev),
                      xs=torch.zeros((m * k, hid), dtype=torch.bfloat16, device=dev))
        elif op == "back":
            offsets, order, place = st["order"]
            st.update(sorted=nv.MoeOrder(st["ids"], st["w"], offsets, order, place),
                      y=torch.empty((m, hid), dtype=torch.bfloat16, device=dev))
        elif op == "grad":
            offsets, order, place = st["order"]
            st.update(sorted=nv.MoeOrder(st["ids"], st["w"], offsets, order, place),
                      dys=torch.empty_like(st["ys"]), dw=torch.empty((m, k), dtype=torch.float32, device=dev))
        else:
            st["weights"] = nv.NVFP4Experts(*st["gate"], *st["up"], *st["down"])
            st.update(ws=nv.moe_gemm_workspace(m, k, st["weights"], dev), y=torch.empty((m, hid), dtype=torch.bfloat16, device=dev),
                      ids=torch.empty((m, k), dtype=torch.int32, device=dev), w=torch.empty((m, k), dtype=torch.float32, device=dev))
    return st


# --------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return dict(plan=_own_plan, attn=_own_attn, sort=_own_sort, back=_own_back, grad=_own_grad, experts=_own_experts)[op](st)
    return dict(plan=_plain_plan, attn=_plain_attn, sort=_plain_sort, back=_plain_back, grad=_plain_grad,
                experts=_plain_experts)[op](st)


def _own_plan(st):
    nv, pool = st["nv"], st["pool"]
    a = nv.kv8_plan(pool, st["kept"], st["new"], st["rows"])
    b = nv.kv8_plan(pool, st["before"], st["none"], 0)
    return dict(cu=a.cu_rows, lens=a.kv_lens, positions=a.positions, slots=a.slots, missing=a.missing,
                lens_after=b.kv_lens, missing_after=b.missing, table=pool.block_table, held=pool.held, free=pool.free_pages,
                count=pool.free_count)


def _own_attn(st):
    c = st["case"]
    return st["nv"].prompt_attention(st["q"], st["k"], st["v"], st["cu"], max_rows=c["rows_hi"], scale=st["scale"],
                                     window=c["window"], sinks=c["sinks"], out=st["out"])


def _own_sort(st):
    nv = st["nv"]
    o = nv.moe_sort(st["logits"], st["case"]["top_k"], workspace=st["ws"], out=st["buffers"])
    xs = nv.moe_gather(st["x"], o, out=st["xs"])
    return o.topk_ids, o.topk_w, o.offsets, o.order, o.place, xs


def _own_back(st):
    return st["nv"].moe_combine(st["ys"], st["sorted"], out=st["y"])


def _own_grad(st):
    return st["nv"].moe_combine_grad(st["dy"], st["ys"], st["sorted"], dys=st["dys"], dw=st["dw"])


def _own_experts(st):
    return st["nv"].moe_w4a16_gemm(st["x"], st["logits"], st["case"]["top_k"], st["weights"], workspace=st["ws"], out=st["y"],
                                   topk_ids=st["ids"], topk_w=st["w"])


# ------------------------------------------------------------- plain torch
def _plan_once(table, held, free, count, kept, new, rows, page):
    """One plan: (cu, lens, positions, slots, missing, table, held, free, count)."""
    batch, width = table.shape
    cap = width * page
    k = kept.long().clamp(0, cap)
    n = torch.minimum(new.long().clamp(min=0), cap - k)
    cu = torch.cat((torch.zeros(1, dtype=torch.long, device=_dev()), torch.cumsum(n, 0))).clamp(max=rows)
    lens = k + cu[1:] - cu[:-1]
    need = (lens + page - 1) // page
    h = held.long()
    col = torch.arange(width, device=_dev())[None, :]
    table = table.long()
    # pages given back, the first of them on top
    gone = (col >= need[:, None]) & (col < h[:, None])
    given = gone.flatten().cumsum(0).reshape(batch, width) - 1
    g = gone.sum()
    top = count.long()[0] + g
    free = torch.cat((free.long(), torch.zeros(1, dtype=torch.long, device=_dev())))    # (a place for what is not pushed)
    free = free.scatter(0, torch.where(gone, top - 1 - given, free.numel() - 1).flatten(), table.flatten())[:-1]
    # pages taken from the top
    wanted = (col >= h[:, None]) & (col < need[:, None])
    taken = wanted.flatten().cumsum(0).reshape(batch, width) - 1
    got = wanted & (taken < top)
    page_of = free[(top - 1 - taken).clamp(0, free.numel() - 1)]
    table = torch.where(got, page_of, torch.where(gone | (wanted & ~got), -1, table))
    w = wanted.sum()
    count = top - torch.minimum(w, top)
    held = torch.minimum(h, need) + got.sum(dim=1)
    row = torch.arange(rows, device=_dev())
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True).clamp(max=batch - 1)
    pos = k[seq] + row - cu[seq]
    at = table[seq, (pos // page).clamp(0, width - 1)]
    slots = torch.where(at >= 0, at * page + pos % page, -1)
    i32 = torch.int32
    return (cu.to(i32), lens.to(i32), pos.to(i32), slots, (w - torch.minimum(w, top)).to(i32).reshape(1), table.to(i32), held.to(i32),
            free.to(i32), count.to(i32).reshape(1))


def _plain_plan(st):
    page = st["case"]["page"]
    a = _plan_once(st["table"], st["held"], st["free"], st["count"], st["kept"], st["new"], st["rows"], page)
    b = _plan_once(a[5], a[6], a[7], a[8], st["before"], st["none"], 0, page)
    return dict(cu=a[0], lens=a[1], positions=a[2], slots=a[3], missing=a[4], lens_after=b[1], missing_after=b[4], table=b[5],
                held=b[6], free=b[7], count=b[8])


def _plain_attn(st):
    c = st["case"]
    h, g = c["kv_heads"], c["q_heads"] // c["kv_heads"]
    at, outs = 0, []
    for n in (x for x in st["n"] if x):
        q = st["q"][at:at + n].float().unflatten(1, (h, g)).permute(1, 2, 0, 3).flatten(1, 2)      # [h][g * n][dk]
        k = st["k"][at:at + n].float().permute(1, 2, 0).contiguous()
        v = st["v"][at:at + n].float().transpose(0, 1).contiguous()
        s = torch.matmul(q, k) * st["scale"]
        t, pos = torch.arange(n, device=_dev())[None, :], torch.arange(n, device=_dev())[:, None]
        see = t <= pos
        if c["window"]:
            see &= (t > pos - c["window"]) | (t < c["sinks"])
        s = s.unflatten(1, (g, n)).masked_fill_(~see, float("-inf"))
        s = s.sub_(s.amax(dim=-1, keepdim=True)).exp_()
        s = s.div_(s.sum(dim=-1, keepdim=True)).flatten(1, 2)
        outs.append(torch.matmul(s, v).unflatten(1, (g, n)).permute(2, 0, 1, 3).flatten(1, 2))
        at += n
    return torch.cat(outs).to(torch.bfloat16)


def _route(logits, k):
    """Experts by descending logit, the lower one first among equals; weights:
    softmax over the chosen logits, in 64 bits and rounded."""
    v, i = torch.sort(logits, dim=1, descending=True, stable=True)
    v = v[:, :k].double()
    w = torch.exp(v - v[:, :1])
    return i[:, :k].to(torch.int32).contiguous(), (w / w.sum(dim=1, keepdim=True)).float().contiguous(), None


def _order(ids, experts):
    """(offsets, order, place) of the pairs sorted by expert."""
    flat = ids.flatten().long()
    key, order = torch.sort(flat, stable=True)
    place = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device=_dev()))
    offsets = torch.searchsorted(key, torch.arange(experts + 1, device=_dev()))
    return offsets.to(torch.int32), order.to(torch.int32), place.to(torch.int32)


def _plain_sort(st):
    k = st["case"]["top_k"]
    ids, w, _ = _route(st["logits"], k)
    offsets, order, place = _order(ids, st["case"]["experts"])
    return ids, w, offsets, order, place, st["x"][order.long() // k]


def _plain_back(st):
    m, k = st["w"].shape
    rows = st["ys"][st["order"][2].long()].float().unflatten(0, (m, k))
    return (rows * st["w"][:, :, None]).sum(dim=1).to(torch.bfloat16)


def _plain_grad(st):
    m, k = st["w"].shape
    order, place = st["order"][1].long(), st["order"][2].long()
    dys = st["dy"].float()[order // k] * st["w"].flatten()[order][:, None]
    dw = (st["ys"][place].float().unflatten(0, (m, k)) * st["dy"].float()[:, None, :]).sum(dim=2)
    return dys.to(torch.bfloat16), dw


def _dequantize(codes, scales, glob):
    """fp32 values of [e][rows][cols / 2] codes: E2M1 * E4M3 * the matrix's factor."""
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float32, device=_dev())
    w = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), dim=-1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float() * glob[:, None, None, 0]
    return w.unflatten(-1, (-1, 16)).mul_(s[..., None]).flatten(-2)


def _plain_experts(st):
    c = st["case"]
    e, k, cap = c["experts"], c["top_k"], st["cap"]
    ids, w, _ = _route(st["logits"], k)
    offsets, order, place = _order(ids, e)
    order, place, flat = order.long(), place.long(), ids.flatten().long()
    # every expert's rows side by side, as many as the fullest has
    at = flat[order] * cap + torch.arange(order.numel(), device=_dev()) - offsets.long()[flat[order]]
    xs = torch.zeros((e * cap, c["hidden"]), dtype=torch.float32, device=_dev())
    xs[at] = st["x"].float()[order // k]
    xs = xs.unflatten(0, (e, cap))
    g = torch.bmm(xs, _dequantize(*st["gate"]).transpose(1, 2))
    u = torch.bmm(xs, _dequantize(*st["up"]).transpose(1, 2))
    a = (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16).float()       # the activations are bf16 rows by definition
    d = torch.bmm(a, _dequantize(*st["down"]).transpose(1, 2)).flatten(0, 1)
    y = (d[at][place].unflatten(0, (-1, k)) * w[:, :, None]).sum(dim=1)
    return y.to(torch.bfloat16), ids, w


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """The outputs of `run` from the definitions, in 64 bits: sequence by
    sequence, expert by expert."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "plan":
        return None                           # whole numbers alone
    return dict(attn=_exact_attn, sort=_exact_sort, back=_exact_back, grad=_exact_grad, experts=_exact_experts)[case["op"]](st)


def _exact_attn(st):
    """Query head by query head, a part of the rows at a time."""
    c = st["case"]
    g = c["q_heads"] // c["kv_heads"]
    rows = st["q"].shape[0]
    out = torch.zeros((rows, c["q_heads"], c["dv"]), dtype=torch.float64, device=_dev())
    at = 0
    for n in st["n"]:
        for h in range(c["kv_heads"]):
            k, v = st["k"][at:at + n, h].double(), st["v"][at:at + n, h].double()
            for i in range(0, n, 512):
                j = min(n, i + 512)
                lo = max(0, i - c["window"] + 1) if c["window"] and c["sinks"] == 0 else 0
                t, pos = torch.arange(lo, j, device=_dev()), torch.arange(i, j, device=_dev())[:, None]
                hide = t > pos
                if c["window"]:
                    hide |= (t <= pos - c["window"]) & (t >= c["sinks"])
                q = st["q"][at + i:at + j, h * g:(h + 1) * g].double()
                s = torch.tensordot(q, k[lo:j], dims=([2], [1])) * st["scale"]
                s.masked_fill_(hide[:, None, :], float("-inf"))
                s = torch.exp(s - torch.logsumexp(s, dim=-1, keepdim=True))
                out[at + i:at + j, h * g:(h + 1) * g] = torch.tensordot(s, v[lo:j], dims=([2], [0]))
        at += n
    return out


def _choose(logits, k):
    """The k first experts of every token, one after the other."""
    left = logits.double().clone()
    ids, vals = [], []
    number = torch.arange(logits.shape[1], device=_dev())
    for _ in range(k):
        best = left.amax(dim=1, keepdim=True)
        i = torch.where(left == best, number, logits.shape[1]).amin(dim=1)
        ids.append(i)
        vals.append(best[:, 0])
        left.scatter_(1, i[:, None], float("-inf"))
    ids, vals = torch.stack(ids, 1), torch.stack(vals, 1)
    return ids, torch.exp(vals - torch.logsumexp(vals, dim=1, keepdim=True))


def _exact_sort(st):
    c = st["case"]
    k, e = c["top_k"], c["experts"]
    ids, w = _choose(st["logits"], k)
    pairs = torch.cat([torch.nonzero(ids.flatten() == i).flatten() for i in range(e)])
    counts = torch.stack([(ids == i).sum() for i in range(e)])
    place = torch.zeros_like(pairs)
    place[pairs] = torch.arange(pairs.numel(), device=_dev())
    offsets = torch.cat((torch.zeros(1, dtype=torch.long, device=_dev()), counts.cumsum(0)))
    return ids.int(), w, offsets.int(), pairs.int(), place.int(), st["x"].double()[torch.div(pairs, k, rounding_mode="floor")]


def _exact_back(st):
    m, k = st["w"].shape
    y = torch.zeros((m, st["ys"].shape[1]), dtype=torch.float64, device=_dev())
    place = st["order"][2].long().reshape(m, k)
    for j in range(k):
        y += st["w"][:, j:j + 1].double() * st["ys"][place[:, j]].double()
    return y


def _exact_grad(st):
    m, k = st["w"].shape
    place = st["order"][2].long().reshape(m, k)
    dys = torch.zeros(st["ys"].shape, dtype=torch.float64, device=_dev())
    dw = torch.zeros((m, k), dtype=torch.float64, device=_dev())
    dy = st["dy"].double()
    for j in range(k):
        dys[place[:, j]] = dy * st["w"][:, j:j + 1].double()
        dw[:, j] = torch.einsum("td,td->t", dy, st["ys"][place[:, j]].double())
    return dys, dw


def _value(codes, scales, glob):
    """64-bit values of one matrix from its bits."""
    out = []
    for c in (codes & 15, codes >> 4):
        c = c.double()
        mag = torch.remainder(c, 8)
        e, m = torch.div(mag, 2, rounding_mode="floor"), torch.remainder(mag, 2)
        mag = torch.where(e == 0, 0.5 * m, torch.exp2(e - 1) * (1 + 0.5 * m))
        out.append(torch.where(c >= 8, -mag, mag))
    w = torch.stack(out, dim=2).reshape(codes.shape[0], -1)
    s = scales.double()
    e, m = torch.div(s, 8, rounding_mode="floor"), torch.remainder(s, 8)
    s = torch.where(e == 0, m * 2.0 ** -9, torch.exp2(e - 7) * (1 + m / 8))
    return w * torch.repeat_interleave(s, 16, dim=1) * glob[0].double()


def _exact_experts(st):
    c = st["case"]
    ids, w = _choose(st["logits"], c["top_k"])
    y = torch.zeros(st["x"].shape, dtype=torch.float64, device=_dev())
    for i in range(c["experts"]):
        token, j = torch.nonzero(ids == i, as_tuple=True)
        if token.numel() == 0:
            continue
        x = st["x"][token].double()
        g = torch.mm(x, _value(*(p[i] for p in st["gate"])).t())
        u = torch.mm(x, _value(*(p[i] for p in st["up"])).t())
        a = (g * torch.sigmoid(g) * u).to(torch.bfloat16).double()       # bf16 rows by definition
        y.index_add_(0, token, torch.mm(a, _value(*(p[i] for p in st["down"])).t()) * w[token, j][:, None])
    return y, ids.int(), w
