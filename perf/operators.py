"""Performance cases of the draft step's attention operators and of draft
verification: rotary positions, the paged 8-bit KV cache (append, read back),
attention over it, and the verification of drafted tokens.

`run` computes a case in plain torch operations, or, with `own` set, with the
library's kernels.  `exact` gives the same outputs from the definitions in
64 bits.

The cache of a case: E4M3 codes with one power-of-two scale per (page, head),
byte b standing for 2^(b - 127); K pages are [tokens][head_dim], V pages
[head_dim][tokens].  Every batch is ragged: sequence b owns the rows
cu_rows[b] .. cu_rows[b + 1], the last tokens of its kv_lens[b] tokens.
"""
import math
import random

import numpy as np
import torch

own = False

FP8 = torch.float8_e4m3fn
MIN_EXP = -110          # smallest exponent of a page's scale


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the q and k rows of a prompt chunk: 32 + 8 heads of 128, rotated in
        # interleaved pairs over the whole head, positions scaled for a context
        # eight times the trained one
        dict(name="rope_prompt", op="rope", rows=6001, q_heads=32, k_heads=8, dim=128, rot=128, interleaved=True,
             base=10000.0, factor=8.0, first=20000),
        # one decode step's q and k at the head's own shape (16 + 2 heads of
        # 256, the first 64 rotated in halves), far into long contexts
        dict(name="rope_decode", op="rope", rows=64, q_heads=16, k_heads=2, dim=256, rot=64, interleaved=False,
             base=1e7, factor=1.0, first=150000),
        # 64 sequences append the rows of a verification step (1 to 4 tokens),
        # rotation included, into pages of 16 tokens that are partly filled
        dict(name="append_decode", op="append", rope=True, batch=64, rows_lo=1, rows_hi=4, len_lo=300, len_hi=9000, seed=1,
             q_heads=16, kv_heads=2, dim=256, rot=64, page=16),
        # three prompts of unequal length are written into an empty cache and
        # read back (the prompt pass of an 8-head layer)
        dict(name="append_prompt", op="append", rope=False, batch=3, rows_lo=4000, rows_hi=12000, len_lo=0, len_hi=0, seed=2,
             q_heads=0, kv_heads=8, dim=128, rot=0, page=64),
        # a single user's draft step: one token against a short context; the
        # time is latency
        dict(name="attn_one_token", op="attn", batch=1, rows_lo=1, rows_hi=1, len_lo=1500, len_hi=1500, seed=3, q_heads=16,
             kv_heads=2, dim=256, page=16, window=0, sinks=0),
        # one draft token for each of 32 users, contexts from 2 K to 30 K
        dict(name="attn_draft_batch", op="attn", batch=32, rows_lo=1, rows_hi=1, len_lo=2000, len_hi=30000, seed=4, q_heads=16,
             kv_heads=2, dim=256, page=16, window=0, sinks=0),
        # the target's verification step: 3 to 6 rows for each of 16 users
        dict(name="attn_verify", op="attn", batch=16, rows_lo=3, rows_hi=6, len_lo=6000, len_hi=16000, seed=5, q_heads=16,
             kv_heads=2, dim=256, page=16, window=0, sinks=0),
        # a sliding-window layer with sinks: long contexts, of which the last
        # 4096 tokens and the first 4 are read
        dict(name="attn_window", op="attn", batch=48, rows_lo=1, rows_hi=2, len_lo=9000, len_hi=100000, seed=6, q_heads=32,
             kv_heads=8, dim=128, page=64, window=4096, sinks=4),
        # two prompt chunks attend to themselves and to what was cached before
        dict(name="attn_prompt", op="attn", batch=2, rows_lo=1100, rows_hi=2048, len_lo=5000, len_hi=9000, seed=7, q_heads=16,
             kv_heads=2, dim=256, page=16, window=0, sinks=0),
        # three drafts of one user and the target's four rows of logits
        dict(name="verify_one", op="verify", batch=1, rows_lo=4, rows_hi=4, seed=8, vocab=151936, bf16=True, sampled=False,
             greedy=False),
        # 2 to 7 drafts of 64 users, the drafts being the draft head's argmax
        dict(name="verify_batch", op="verify", batch=64, rows_lo=3, rows_hi=8, seed=9, vocab=151936, bf16=True, sampled=False,
             greedy=False),
        # drafts that were sampled from the draft's own distribution
        dict(name="verify_sampled", op="verify", batch=24, rows_lo=2, rows_hi=6, seed=10, vocab=129280, bf16=False, sampled=True,
             greedy=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "attn", "attn", "attn", "verify", "verify"])
    seed = rng.randrange(1 << 20)
    heads, kv, dim = rng.choice([(16, 2, 256), (32, 8, 128), (8, 1, 128), (12, 4, 64), (24, 3, 192), (5, 5, 64), (32, 4, 256)])
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        rot = 2 * rng.randint(4, dim // 16) * 8 if rng.random() < 0.5 else dim
        rot = min(rot, dim)
        return dict(op="rope", rows=_log_int(rng, 1, 4000), q_heads=heads, k_heads=kv, dim=dim, rot=rot,
                    interleaved=rng.random() < 0.5, base=rng.choice([1e4, 5e5, 1e7]), factor=rng.choice([1.0, 1.0, 4.0, 32.0]),
                    first=_log_int(rng, 1, 1000000))
    if op == "append":
        if rng.random() < 0.5:
            lo = rng.randint(1, 4)
            return dict(op="append", rope=True, batch=_log_int(rng, 1, 96), rows_lo=lo, rows_hi=lo + rng.randint(0, 4), len_lo=1,
                        len_hi=_log_int(rng, 2, 6000), seed=seed, q_heads=heads, kv_heads=kv, dim=dim,
                        rot=rng.choice([dim, dim // 2]), page=page)
        hi = _log_int(rng, 20, 6000)
        return dict(op="append", rope=rng.random() < 0.5, batch=rng.randint(1, 4), rows_lo=max(1, hi // 3), rows_hi=hi, len_lo=0,
                    len_hi=rng.choice([0, 700]), seed=seed, q_heads=heads, kv_heads=kv, dim=dim, rot=dim // 2, page=page)
    if op == "attn":
        window = rng.choice([0, 0, _log_int(rng, 16, 8000)])
        sinks = rng.choice([0, 4, 17]) if window else 0
        if rng.random() < 0.75:
            batch = _log_int(rng, 1, 40)
            hi = max(2, min(_log_int(rng, 30, 30000), 400000 // batch))
            lo = rng.randint(1, 4)
            return dict(op="attn", batch=batch, rows_lo=lo, rows_hi=lo + rng.randint(0, 4), len_lo=max(1, hi // 10), len_hi=hi,
                        seed=seed, q_heads=heads, kv_heads=kv, dim=dim, page=page, window=window, sinks=sinks)
        hi = _log_int(rng, 40, 1500)
        heads, kv = (24, 2) if heads > 24 else (heads, kv)
        return dict(op="attn", batch=rng.randint(1, 3), rows_lo=max(1, hi // 2), rows_hi=hi, len_lo=hi, len_hi=hi + rng.randint(0, 4000),
                    seed=seed, q_heads=heads, kv_heads=kv, dim=dim, page=page, window=window, sinks=sinks)
    sampled = rng.random() < 0.5
    lo = rng.randint(1, 5)
    return dict(op="verify", batch=_log_int(rng, 1, 24 if sampled else 48), rows_lo=lo, rows_hi=lo + rng.randint(0, 3), seed=seed,
                vocab=rng.choice([_log_int(rng, 100, 130000), 32000, 129280, 50257]), bf16=rng.random() < 0.6, sampled=sampled,
                greedy=rng.random() < 0.25)


def _ragged(case):
    """Row counts and total lengths of the case's sequences."""
    r = random.Random(case["seed"] * 7919 + 13)
    n = [r.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["batch"])]
    if case["batch"] > 1:
        n[-1] = case["rows_hi"]
    if case["op"] == "append":
        lens = [c + r.randint(case["len_lo"], case["len_hi"]) for c in n]
    elif case["op"] == "attn":
        lens = [max(c, r.randint(case["len_lo"], case["len_hi"])) for c in n]
    else:
        lens = [c + r.randint(0, 5000) for c in n]
    return n, lens


def _visible(case, n, length):
    """(keys read, (row, key) pairs) of one sequence."""
    w, s = case["window"], case["sinks"]
    pairs, first = 0, length
    for i in range(n):
        pos = length - n + i
        if w == 0 or pos + 1 <= w:
            pairs += pos + 1
            first = 0
        else:
            a = pos + 1 - w
            pairs += w + min(s, a)
            first = min(first, a)
    keys = length - first + (min(s, first) if w else 0)
    return keys, pairs


def work(case):
    op = case["op"]
    if op == "rope":
        e = case["rows"] * (case["q_heads"] + case["k_heads"])
        return dict(bytes=e * case["dim"] * 4 + case["rows"] * 4 + case["rot"] * 4, flops=e * case["rot"] * 3)
    n, lens = _ragged(case)
    rows = sum(n)
    if op == "append":
        h, d, p = case["kv_heads"], case["dim"], case["page"]
        kept, read = _held(n, lens, p)
        # new rows in, codes out; codes read back, values out; older codes of the
        # continued pages are among those read back
        b = rows * h * d * 2 * (2 + 1) + read * h * d * 2 * (1 + 2)
        f = rows * h * d * 2 * 2
        if case["rope"]:
            b += rows * case["q_heads"] * d * 4
            f += rows * (case["q_heads"] + h) * case["rot"] * 3
        return dict(bytes=b, flops=f)
    if op == "attn":
        keys = pairs = 0
        for a, b in zip(n, lens):
            k, p = _visible(case, a, b)
            keys, pairs = keys + k, pairs + p
        return dict(bytes=keys * case["kv_heads"] * case["dim"] * 2 + rows * case["q_heads"] * case["dim"] * 4,
                    flops=pairs * case["q_heads"] * case["dim"] * 4)
    logits = rows * case["vocab"] * (2 if case["bf16"] else 4)
    if case["sampled"]:
        logits += (rows - len(n)) * case["vocab"] * (2 if case["bf16"] else 4)
    return dict(bytes=logits + rows * 16 + len(n) * 24, flops=rows * case["vocab"] * 4)


def _held(n, lens, page):
    """(tokens before the new ones in the pages they go to, tokens read back:
    those and the new ones)."""
    kept = [(b - a) % page for a, b in zip(n, lens)]
    return sum(kept), sum(kept) + sum(n)


# ------------------------------------------------------------------ inputs
def _dev():
    return torch.device("cuda")


def _i32(a):
    return torch.tensor(a, dtype=torch.int32, device=_dev())


def _cu(n):
    return _i32([0] + list(np.cumsum(n)))


def _pages(case, lens, seed):
    """A block table whose pages lie in random order in a pool with a few
    unused ones, and the pool's size."""
    p = case["page"]
    need = [-(-x // p) for x in lens]
    width = max(1, max(need))
    total = sum(need) + 5
    order = np.random.default_rng(seed).permutation(total)
    table = np.zeros((len(lens), width), np.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c
    return torch.from_numpy(table).to(_dev()), total


def _pow2(e, dtype=torch.float32):
    """2^e, exactly (0 below the smallest normal number)."""
    if dtype == torch.float64:
        return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)
    return ((e.to(torch.int32) + 127).clamp(min=0) << 23).view(torch.float32)


def _scale_exp(amax):
    """Smallest exponent e >= MIN_EXP with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, x = torch.frexp(amax.float())
    e = torch.where(m <= 0.875, x - 9, x - 8).to(torch.int32)
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)


def _fill_cache(case, total, gen):
    """A filled pool: rows of unequal size, quantised per page and head."""
    h, d, p = case["kv_heads"], case["dim"], case["page"]
    out = []
    for what in range(2):
        chan = torch.exp(0.5 * torch.randn((h, 1, d), generator=gen, device=_dev()))
        codes = torch.empty((total, h, p, d), dtype=torch.uint8, device=_dev())
        scales = torch.empty((total, h), dtype=torch.uint8, device=_dev())
        step = max(1, (1 << 27) // (h * p * d))
        for i in range(0, total, step):
            j = min(total, i + step)
            x = torch.randn((j - i, h, p, d), generator=gen, device=_dev()) * chan
            x = x.to(torch.bfloat16).float()
            e = _scale_exp(x.abs().amax(dim=(2, 3)))
            codes[i:j] = (x * _pow2(-e)[:, :, None, None]).to(FP8).view(torch.uint8)
            scales[i:j] = (e + 127).to(torch.uint8)
        if what == 1:
            codes = codes.transpose(2, 3).contiguous()
        out += [codes, scales]
    return dict(k_codes=out[0], k_scales=out[1], v_codes=out[2], v_scales=out[3])


def _rope_table(case):
    """Angles per position (radians, 64 bits) and the factor of the rotated
    values.  A factor above 1 stretches the wavelengths that a 4096-token
    context does not finish, by parts."""
    rot = case["rot"]
    f = case.get("base", 1e7) ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    factor = case.get("factor", 1.0)
    if factor == 1.0:
        return f, 1.0
    turns = 4096.0 * f / (2.0 * np.pi)
    keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
    return f * (keep + (1.0 - keep) / factor), 0.1 * math.log(factor) + 1.0


def prepare(case, seed):
    gen = torch.Generator(device=_dev())
    gen.manual_seed(seed)
    op = case["op"]

    def rand(shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(shape, generator=gen, device=_dev()) * std).to(dtype)

    if op == "rope":
        t, d = case["rows"], case["dim"]
        f, mscale = _rope_table(case)
        pos = torch.arange(t, device=_dev(), dtype=torch.int32) + case["first"]
        st = dict(case=case, q=rand((t, case["q_heads"], d)), k=rand((t, case["k_heads"], d)), pos=pos,
                  freq=torch.from_numpy(f).to(_dev()), mscale=mscale)
        if own:
            import nvfp4_w4a16_mtp_amd as nv
            st.update(nv=nv, q_out=torch.empty_like(st["q"]), k_out=torch.empty_like(st["k"]))
        return st
    n, lens = _ragged(case)
    rows = sum(n)
    if op in ("append", "attn"):
        table, total = _pages(case, lens, seed)
        st = dict(case=case, n=n, lens=lens, cu=_cu(n), kv_lens=_i32(lens), table=table, **_fill_cache(case, total, gen))
        d, h = case["dim"], case["kv_heads"]
        if op == "attn":
            st.update(q=rand((rows, case["q_heads"], d)), scale=d ** -0.5)
        else:
            st.update(k=rand((rows, h, d), std=1.5), v=rand((rows, h, d), std=1.5))
            _, st["read_rows"] = _held(n, lens, case["page"])
            back = [(b - a) % case["page"] + a for a, b in zip(n, lens)]
            st.update(back=back, cu_back=_cu(back))
            if case["rope"]:
                f, _ = _rope_table(case)
                st.update(q=rand((rows, case["q_heads"], d)), freq=torch.from_numpy(f).to(_dev()))
        if own:
            import nvfp4_w4a16_mtp_amd as nv
            cache = nv.KV8Cache(st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"])
            seqs = nv.KV8Seqs(st["cu"], st["kv_lens"], st["table"], max_rows=max(n), max_kv_len=max(lens))
            st.update(nv=nv, cache=cache, seqs=seqs)
            if op == "attn":
                st.update(out=torch.empty_like(st["q"]), ws=nv.kv8_attention_workspace(cache, seqs, case["q_heads"], rows))
            else:
                st.update(seqs_back=nv.KV8Seqs(st["cu_back"], st["kv_lens"], st["table"], max_rows=max(st["back"]),
                                               max_kv_len=max(lens)),
                          k_back=rand((st["read_rows"], h, d)), v_back=rand((st["read_rows"], h, d)))
                if case["rope"]:
                    st["q_out"] = torch.empty_like(st["q"])
        return st
    # verification: peaked target rows, drafts that the draft model finds likely
    v, b = case["vocab"], case["batch"]
    dt = torch.bfloat16 if case["bf16"] else torch.float32
    logits = torch.empty((rows, v), dtype=dt, device=_dev())
    draft = torch.empty((rows, v), dtype=dt, device=_dev()) if case["sampled"] else None
    ids = torch.empty(rows, dtype=torch.int32, device=_dev())
    u = torch.rand((rows + b,), generator=gen, device=_dev(), dtype=torch.float32)
    temp = 0.5 + torch.rand((b,), generator=gen, device=_dev(), dtype=torch.float32)
    if case["greedy"]:
        temp[::2] = 0.0
    step = max(1, (1 << 27) // v)
    for i in range(0, rows, step):
        j = min(rows, i + step)
        x = torch.randn((j - i, v), generator=gen, device=_dev()) * 2.5
        hot = torch.randint(0, v, (j - i, 3), generator=gen, device=_dev())
        x.scatter_(1, hot, torch.randn((j - i, 3), generator=gen, device=_dev()) + 14.0)
        y = x + 0.7 * torch.randn((j - i, v), generator=gen, device=_dev())
        logits[i:j] = x.to(dt)
        if case["sampled"]:
            draft[i:j] = y.to(dt)
            g = -torch.log(-torch.log(torch.rand((j - i, v), generator=gen, device=_dev(), dtype=torch.float64)
                                      .clamp_(1e-300, 1 - 1e-16)))
            ids[i:j] = (draft[i:j].double() + g).argmax(dim=1).to(torch.int32)
        else:
            ids[i:j] = y.argmax(dim=1).to(torch.int32)
    st = dict(case=case, n=n, lens=lens, cu=_cu(n), kv_lens=_i32(lens), logits=logits, draft=draft, ids=ids,
              u_accept=u[:rows].contiguous(), u_sample=u[rows:].contiguous(), temp=temp)
    if own:
        import nvfp4_w4a16_mtp_amd as nv
        st.update(nv=nv, ws=nv.verify_workspace(max(n), b, v, _dev(), sampled=case["sampled"]))
    return st


# --------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return dict(rope=_own_rope, append=_own_append, attn=_own_attn, verify=_own_verify)[op](st)
    return dict(rope=_plain_rope, append=_plain_append, attn=_plain_attn, verify=_plain_verify)[op](st)


def _own_rope(st):
    return st["nv"].rope_qk(st["q"], st["k"], st["pos"], st["freq"], interleaved=st["case"]["interleaved"],
                            mscale=st["mscale"], q_out=st["q_out"], k_out=st["k_out"])


def _own_append(st):
    nv = st["nv"]
    if st["case"]["rope"]:
        q = nv.rope_kv8_append(st["cache"], st["seqs"], st["q"], st["k"], st["v"], st["freq"], q_out=st["q_out"])
        k, v = nv.kv8_read(st["cache"], st["seqs_back"], k_out=st["k_back"], v_out=st["v_back"])
        return q, k, v
    nv.kv8_append(st["cache"], st["seqs"], st["k"], st["v"])
    return nv.kv8_read(st["cache"], st["seqs_back"], k_out=st["k_back"], v_out=st["v_back"])


def _own_attn(st):
    c = st["case"]
    return st["nv"].kv8_attention(st["q"], st["cache"], st["seqs"], scale=st["scale"], window=c["window"], sinks=c["sinks"],
                                  workspace=st["ws"], out=st["out"])


def _own_verify(st):
    r = st["nv"].verify_drafts(st["logits"], st["cu"], st["ids"], st["u_accept"], st["u_sample"], max_rows=max(st["n"]),
                               temperature=st["temp"], draft_logits=st["draft"], kv_lens=st["kv_lens"], workspace=st["ws"])
    return r.accepted, r.tokens, r.next, r.kv_lens


# ------------------------------------------------------------- plain torch
def _rotate(x, angle, rot, interleaved, mscale):
    """x [rows][heads][dim] rotated, in 64 bits (angles of far positions lose
    their meaning in 32, and values next to a rounding border move the code
    of an 8-bit cache)."""
    cos, sin = (torch.cos(angle) * mscale)[:, None, :], (torch.sin(angle) * mscale)[:, None, :]
    y = x.double()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((turned, y[..., rot:]), dim=-1).to(x.dtype)


def _plain_rope(st):
    c = st["case"]
    angle = st["pos"].double()[:, None] * st["freq"][None, :]
    return tuple(_rotate(st[k], angle, c["rot"], c["interleaved"], st["mscale"]) for k in ("q", "k"))


def _plain_append(st):
    c, p = st["case"], st["case"]["page"]
    n, lens = st["n"], st["lens"]
    cu, kv_lens = st["cu"].long(), st["kv_lens"].long()
    counts = [(b - 1) // p - (b - a) // p + 1 for a, b in zip(n, lens)]
    items = sum(counts)
    cnt = torch.tensor(counts, device=_dev())
    seq = torch.repeat_interleave(torch.arange(len(n), device=_dev()), cnt, output_size=items)
    start = kv_lens - (cu[1:] - cu[:-1])
    first = torch.cumsum(cnt, 0) - cnt
    idx = start[seq] // p + torch.arange(items, device=_dev()) - first[seq]
    page = st["table"].long()[seq, idx]
    pos = idx[:, None] * p + torch.arange(p, device=_dev())[None, :]
    new = (pos >= start[seq][:, None]) & (pos < kv_lens[seq][:, None])
    old = pos < start[seq][:, None]
    src = (cu[seq][:, None] + pos - start[seq][:, None]).clamp(0, st["k"].shape[0] - 1)
    k = st["k"]
    outs = []
    if c["rope"]:
        row_pos = torch.repeat_interleave(start - cu[:-1], torch.tensor(n, device=_dev()), output_size=sum(n)) \
            + torch.arange(sum(n), device=_dev())
        angle = row_pos.double()[:, None] * st["freq"][None, :]
        k = _rotate(k, angle, c["rot"], False, 1.0)
        outs.append(_rotate(st["q"], angle, c["rot"], False, 1.0))
    for x, codes, scales, turned in ((k, st["k_codes"], st["k_scales"], False), (st["v"], st["v_codes"], st["v_scales"], True)):
        held = codes[page].view(FP8).float()                      # [items][heads][page][dim]
        if turned:
            held = held.transpose(2, 3)
        e_old = scales[page].to(torch.int32) - 127
        fresh = x.float()[src].permute(0, 2, 1, 3)                # [items][heads][page][dim]
        e = _scale_exp(fresh.abs().masked_fill(~new[:, None, :, None], 0.0).amax(dim=(2, 3)))
        e = torch.where(old[:, :1], torch.maximum(e, e_old), e)
        put = torch.where(new[:, None, :, None], fresh * _pow2(-e)[:, :, None, None],
                          held * _pow2(e_old - e)[:, :, None, None])
        back = put.clamp(-448.0, 448.0).to(FP8).float() * _pow2(e)[:, :, None, None]
        keep = (new | old).flatten().nonzero_static(size=st["read_rows"]).flatten()
        outs.append(back.permute(0, 2, 1, 3).flatten(0, 1)[keep].to(torch.bfloat16))
    return tuple(outs)


def _gather(codes, scales, pages, length, turned, dtype):
    x = codes[pages].view(FP8).to(dtype)
    if turned:
        x = x.transpose(2, 3)
    x = x * _pow2(scales[pages].to(torch.int32) - 127, dtype)[:, :, None, None]
    return x.permute(1, 0, 2, 3).flatten(1, 2)[:, :length]        # [heads][length][dim]


def _plain_attn(st, dtype=torch.float32):
    c, p = st["case"], st["case"]["page"]
    h, g = c["kv_heads"], c["q_heads"] // c["kv_heads"]
    at, outs = 0, []
    for b, (n, length) in enumerate(zip(st["n"], st["lens"])):
        pages = st["table"][b, :-(-length // p)].long()
        k = _gather(st["k_codes"], st["k_scales"], pages, length, False, dtype)
        v = _gather(st["v_codes"], st["v_scales"], pages, length, True, dtype)
        q = st["q"][at:at + n].to(dtype).unflatten(1, (h, g)).permute(1, 2, 0, 3).flatten(1, 2)   # [h][g * n][d]
        s = torch.matmul(q, k.transpose(1, 2)) * st["scale"]
        t = torch.arange(length, device=_dev())[None, :]
        pos = torch.arange(length - n, length, device=_dev())[:, None]
        see = t <= pos
        if c["window"]:
            see &= (t > pos - c["window"]) | (t < c["sinks"])
        s = s.unflatten(1, (g, n)).masked_fill(~see, float("-inf"))
        s = torch.exp(s - s.amax(dim=-1, keepdim=True))
        s = (s / s.sum(dim=-1, keepdim=True)).flatten(1, 2)
        o = torch.matmul(s, v)
        outs.append(o.unflatten(1, (g, n)).permute(2, 0, 1, 3).flatten(1, 2))
        at += n
    return torch.cat(outs).to(torch.bfloat16 if dtype == torch.float32 else dtype)


def _plain_verify(st):
    """Softmax and running sums in 64 bits: a draw next to a border of the
    running sum has to fall on the same side."""
    rows, v = st["logits"].shape
    n, b = st["n"], len(st["n"])
    cu = st["cu"].long()
    row = torch.arange(rows, device=_dev())
    seq = torch.repeat_interleave(torch.arange(b, device=_dev()), cu[1:] - cu[:-1], output_size=rows)
    temp = st["temp"].double()
    t = torch.where(temp > 0, temp, torch.ones_like(temp))[seq][:, None]

    def probs(x):
        x = x.double() / t
        x = torch.exp(x - x.amax(dim=1, keepdim=True))
        return x / x.sum(dim=1, keepdim=True)

    p = probs(st["logits"])
    top = st["logits"].float().argmax(dim=1)
    ids = st["ids"].long()
    pd = p.gather(1, ids[:, None])[:, 0]
    q = probs(st["draft"]) if st["draft"] is not None else None
    qd = q.gather(1, ids[:, None])[:, 0] if q is not None else 1.0
    ok = torch.where(temp[seq] > 0, st["u_accept"].double() * qd < pd, top == ids)
    last = row == cu[1:][seq] - 1
    stop = ~ok | last
    # first stopping row of each sequence
    at = torch.full((b,), rows, device=_dev()).scatter_reduce(0, seq, torch.where(stop, row, torch.full_like(row, rows)), "amin")
    accepted = at - cu[:-1]
    w = p[at]
    bonus = at == cu[1:] - 1
    if q is not None:
        rest = (w - q[at]).clamp(min=0.0)
    else:
        rest = w.scatter(1, ids[at][:, None], 0.0)
    w = torch.where(bonus[:, None], w, rest)
    c = torch.cumsum(w, dim=1)
    tok = (c > st["u_sample"].double()[:, None] * c[:, -1:]).to(torch.uint8).argmax(dim=1)
    tok = torch.where(temp > 0, tok, top[at]).to(torch.int32)
    tokens = torch.where(row < at[seq], st["ids"], torch.where(row == at[seq], tok[seq], torch.full_like(st["ids"], -1)))
    kept = st["kv_lens"] - torch.tensor(n, dtype=torch.int32, device=_dev()) + accepted.to(torch.int32) + 1
    return accepted.to(torch.int32), tokens, tok, kept


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """The outputs of `run` from the definitions, in 64 bits: row by row and
    sequence by sequence."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return dict(rope=_exact_rope, append=_exact_append, attn=_exact_attn, verify=_exact_verify)[case["op"]](st)


def _turn(x, pos, freq, rot, interleaved, mscale):
    """Rotation as a product with the complex number mscale * e^(i p f)."""
    z = torch.polar(torch.full((len(pos), rot // 2), mscale, dtype=torch.float64, device=x.device),
                    torch.outer(pos.double(), freq))[:, None, :]
    y = x.double().clone()
    if interleaved:
        pair = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], rot // 2, 2).contiguous()) * z
        y[..., :rot] = torch.view_as_real(pair).flatten(-2)
    else:
        pair = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * z
        y[..., :rot // 2], y[..., rot // 2:rot] = pair.real, pair.imag
    return y


def _exact_rope(st):
    c = st["case"]
    return tuple(_turn(st[k], st["pos"], st["freq"], c["rot"], c["interleaved"], st["mscale"]) for k in ("q", "k"))


def _nearest_e4m3(x):
    """Nearest value of the E4M3 grid (3 bits after the leading one, smallest
    step 2^-9, largest 448), ties to the even step."""
    _, ex = torch.frexp(x.abs().clamp(min=2.0 ** -6))
    step = _pow2(ex - 4, torch.float64)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_append(st):
    c, p = st["case"], st["case"]["page"]
    q, ks, vs = [], [], []
    at = 0
    grid = torch.arange(256, dtype=torch.uint8, device=_dev()).view(FP8).double()
    for b, (n, length) in enumerate(zip(st["n"], st["lens"])):
        start = length - n
        k, v = st["k"][at:at + n].double(), st["v"][at:at + n].double()
        if c["rope"]:
            pos = torch.arange(start, length, device=_dev())
            # the rotated k is a bf16 row before it is quantised
            k = _turn(st["k"][at:at + n], pos, st["freq"], c["rot"], False, 1.0).to(torch.bfloat16).double()
            q.append(_turn(st["q"][at:at + n], pos, st["freq"], c["rot"], False, 1.0))
        first = start // p
        pages = st["table"][b, first:(length - 1) // p + 1].long()
        off = start - first * p
        m = len(pages)
        for x, codes, scales, turned, to in ((k, st["k_codes"], st["k_scales"], False, ks), (v, st["v_codes"], st["v_scales"], True, vs)):
            old = grid[codes[pages[:1]].long()][0]                # the first page alone holds older tokens
            old = (old.transpose(1, 2) if turned else old)[:, :off]                              # [heads][off][dim]
            e_old = scales[pages[:1]].long()[0] - 127
            full = torch.zeros((m * p, *x.shape[1:]), dtype=torch.float64, device=_dev())
            full[off:off + n] = x
            amax = full.abs().unflatten(0, (m, p)).amax(dim=(1, 3))
            e = torch.ceil(torch.log2(amax.clamp(min=1e-60) / 448.0) - 1e-9).long()
            e = torch.where(amax > 448.0 * _pow2(e, torch.float64), e + 1, e).clamp(min=MIN_EXP)
            e = torch.where(amax <= 448.0 * _pow2(e - 1, torch.float64), e - 1, e).clamp(min=MIN_EXP)
            if off:
                e[0] = torch.maximum(e[0], e_old)
            s = _pow2(e, torch.float64)
            new = _nearest_e4m3(full.unflatten(0, (m, p)) / s[:, None, :, None]) * s[:, None, :, None]
            if off:
                so = _pow2(e_old - e[0], torch.float64)
                new[0, :off] = (_nearest_e4m3(old * so[:, None, None]) * s[0][:, None, None]).transpose(0, 1)
            to.append(new.flatten(0, 1)[:off + n])
        at += n
    out = (torch.cat(ks), torch.cat(vs))
    return (torch.cat(q), *out) if c["rope"] else out


def _exact_attn(st):
    """Query head by query head, the visible keys alone."""
    c, p = st["case"], st["case"]["page"]
    g = c["q_heads"] // c["kv_heads"]
    grid = torch.arange(256, dtype=torch.uint8, device=_dev()).view(FP8).double()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=_dev())
    at = 0
    for b, (n, length) in enumerate(zip(st["n"], st["lens"])):
        pages = st["table"][b, :-(-length // p)].long()
        for h in range(c["kv_heads"]):
            ks = _pow2(st["k_scales"][pages, h].long() - 127, torch.float64)
            vs = _pow2(st["v_scales"][pages, h].long() - 127, torch.float64)
            k = (grid[st["k_codes"][pages, h].int()] * ks[:, None, None]).flatten(0, 1)[:length]
            v = (grid[st["v_codes"][pages, h].int()] * vs[:, None, None]).transpose(1, 2).flatten(0, 1)[:length]
            t = torch.arange(length, device=_dev())
            for i in range(0, n, 256):
                j = min(n, i + 256)
                pos = torch.arange(length - n + i, length - n + j, device=_dev())[:, None]
                hide = t > pos
                if c["window"]:
                    hide |= (t <= pos - c["window"]) & (t >= c["sinks"])
                q = st["q"][at + i:at + j, h * g:(h + 1) * g].double()
                s = torch.tensordot(q, k, dims=([2], [1])) * st["scale"]
                s.masked_fill_(hide[:, None, :], float("-inf"))
                s = torch.exp(s - torch.logsumexp(s, dim=-1, keepdim=True))
                out[at + i:at + j, h * g:(h + 1) * g] = torch.tensordot(s, v, dims=([2], [0]))
        at += n
    return out


def _exact_verify(st):
    at = 0
    accepted, tokens, nxt, kept = [], [], [], []
    ids, ua, us = st["ids"].tolist(), st["u_accept"].tolist(), st["u_sample"].tolist()
    temp = st["temp"].tolist()
    for b, n in enumerate(st["n"]):
        acc, tok = 0, None
        for i in range(n):
            row, last = at + i, i == n - 1
            x = st["logits"][row].double()
            if temp[b] == 0.0:
                best = int(torch.nonzero(x == x.max())[0])
                if last or best != ids[row]:
                    tok = best
                    break
                acc += 1
                continue
            p = torch.exp(x / temp[b] - torch.logsumexp(x / temp[b], dim=0))
            q = torch.zeros_like(p)
            if st["draft"] is not None:
                y = st["draft"][row].double() / temp[b]
                q = torch.exp(y - torch.logsumexp(y, dim=0))
            else:
                q[ids[row]] = 1.0
            if not last and ua[row] * float(q[ids[row]]) < float(p[ids[row]]):
                acc += 1
                continue
            w = p if last else (p - q).clamp(min=0.0)
            run_sum = torch.cumsum(w, dim=0)
            tok = int(torch.searchsorted(run_sum, us[b] * float(run_sum[-1]), right=True))
            break
        accepted.append(acc)
        nxt.append(tok)
        tokens += ids[at:at + acc] + [tok] + [-1] * (n - acc - 1)
        kept.append(st["lens"][b] - n + acc + 1)
        at += n
    return tuple(torch.tensor(a, dtype=torch.int32) for a in (accepted, tokens, nxt, kept))
