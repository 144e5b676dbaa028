"""Plain 64-bit forms of the batch and prompt operators, for their tests:
page plans, attention over packed prompts, routing and sorted rows."""
import math

import numpy as np
import torch


# ---------------------------------------------------------------- page plans
class Pool:
    """The host's bookkeeping of a page pool, request by request."""

    def __init__(self, num_pages, batch, max_pages, page):
        self.table = np.full((batch, max_pages), -1, np.int32)
        self.held = [0] * batch
        self.free = list(range(num_pages - 1, -1, -1))        # the top is last
        self.num_pages, self.page = num_pages, page

    def plan(self, kept, new, rows):
        batch, width = self.table.shape
        cap, p = width * self.page, self.page
        cu, lens, need, left = [0], [], [], rows
        for k, n in zip(kept, new):
            k = min(max(k, 0), cap)
            n = min(max(n, 0), cap - k, left)
            left -= n
            cu.append(cu[-1] + n)
            lens.append(k + n)
            need.append(-(-(k + n) // p))
        gone = [(b, i) for b in range(batch) for i in range(need[b], self.held[b])]
        for b, i in reversed(gone):
            self.free.append(int(self.table[b, i]))
            self.table[b, i] = -1
        missing = 0
        for b in range(batch):
            had = self.held[b]
            self.held[b] = min(had, need[b])
            for i in range(had, need[b]):
                if self.free:
                    self.table[b, i] = self.free.pop()
                    self.held[b] += 1
                else:
                    self.table[b, i] = -1
                    missing += 1
        pos, slots = [], []
        for b in range(batch):
            n = cu[b + 1] - cu[b]
            for i in range(n):
                t = lens[b] - n + i
                pg = int(self.table[b, t // p])
                pos.append(t)
                slots.append(pg * p + t % p if 0 <= pg < self.num_pages else -1)
        return cu, lens, pos, slots, missing


# ----------------------------------------------------------------- attention
def sees(n, window, sinks):
    t = torch.arange(n)
    ok = t[None, :] <= t[:, None]
    if window > 0:
        ok &= (t[None, :] > t[:, None] - window) | (t[None, :] < sinks)
    return ok


def attention(q, k, v, ns, scale, window=0, sinks=0):
    """(out, bound) in 64 bits on q's device.  The bound counts: weights rounded to bf16
    (2^-8 each, and their sum of the same), scores in fp32 (a sum of dk products, each
    partial sum off by 2^-24 of the largest the row's scores can be, and as much again for the
    reference), 2^x to 2^-22, and the result's own rounding (2^-8)."""
    rows, hq, dk = q.shape
    g = hq // k.shape[1]
    out = torch.zeros((rows, hq, v.shape[2]), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    at = 0
    for n in ns:
        if n == 0:
            continue
        ok = sees(n, window, sinks).to(q.device)
        for h in range(hq):
            qh, kh, vh = (x[at:at + n, y].double() for x, y in ((q, h), (k, h // g), (v, h // g)))
            s = torch.mm(qh, kh.t()) * scale
            s = s.masked_fill(~ok, -math.inf)
            p = torch.softmax(s, dim=1)
            o = torch.mm(p, vh)
            size = torch.mm(qh.abs(), kh.abs().t()).amax(dim=1, keepdim=True) * abs(scale)
            eps = 2.0 ** -8 * (1 + 2.0 ** -8) + 2.0 ** -22 + 3 * (dk + 2) * 2.0 ** -24 * size
            spread = torch.mm(p, vh.abs()) + o.abs()          # >= sum p |v - o|
            out[at:at + n, h] = o
            bound[at:at + n, h] = 2.0 ** -8 * o.abs() + (1 + 2.0 ** -7) * eps * spread + 1e-38
        at += n
    return out, bound


# ------------------------------------------------------------------- experts
def route(logits, k):
    """ids and 64-bit weights of float logits [m][experts]."""
    x = logits.double().cpu().numpy()
    ids = np.zeros((x.shape[0], k), np.int64)
    for t in range(x.shape[0]):
        key = [(-math.inf if math.isnan(v) else v) for v in x[t]]
        nan = [math.isnan(v) for v in x[t]]
        ids[t] = sorted(range(x.shape[1]), key=lambda e: (nan[e], -key[e], e))[:k]
    v = np.take_along_axis(x, ids, 1)
    with np.errstate(all="ignore"):
        w = np.exp(v - v[:, :1])
        w = w / w.sum(axis=1, keepdims=True)
    return ids, w


def order(ids, experts):
    """(offsets, order, place) of ids [m][k]; those outside [0, experts) left out."""
    flat = np.asarray(ids).reshape(-1)
    ok = [p for p in range(flat.size) if 0 <= flat[p] < experts]
    seq = sorted(ok, key=lambda p: (flat[p], p))
    place = np.full(flat.size, -1, np.int64)
    place[seq] = np.arange(len(seq))
    offsets = np.concatenate(([0], np.cumsum(np.bincount(flat[ok], minlength=experts)))) if ok else np.zeros(experts + 1)
    return offsets.astype(np.int64), np.asarray(seq, np.int64), place


def weight_values(w):
    """64-bit values of (codes, scales, glob) with codes [rows][cols / 2]."""
    codes, scales, glob = (x.cpu() for x in w)
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).long()
    v = lut[c & 7] * torch.where(c >= 8, -1.0, 1.0)
    return v * torch.repeat_interleave(scales.view(torch.float8_e4m3fn).double(), 16, dim=-1) * glob[..., 0].double()[..., None, None]


def experts_ffn(x, ids, w, gate, up, down):
    """(y, bound) in 64 bits: activations left unrounded here, so that the bound counts
    their rounding (2^-8 of each), the fp32 sums' errors (a sum of n terms: n 2^-24 of
    the terms' magnitudes) through the activation, and nothing of the output's rounding."""
    m, hid = x.shape
    x = x.double().cpu()
    y, bound = torch.zeros((m, hid), dtype=torch.float64), torch.zeros((m, hid), dtype=torch.float64)
    inter = gate.shape[1]
    for e in range(gate.shape[0]):
        t, j = np.nonzero(ids == e)
        if t.size == 0:
            continue
        xe = x[t]
        g, u = xe @ gate[e].t(), xe @ up[e].t()
        eg, eu = ((hid + 2) * 2.0 ** -24 * (xe.abs() @ b.abs().t()) for b in (gate[e], up[e]))
        sg = torch.sigmoid(g)
        a = g * sg * u
        # |silu'| < 1.1
        ea = 2.0 ** -8 * a.abs() + 1.01 * (1.1 * eg * u.abs() + (g * sg).abs() * eu + 1.1 * eg * eu) + 2.0 ** -21 * a.abs()
        ww = torch.from_numpy(w[t, j])[:, None]
        d = a @ down[e].t()
        ed = ea @ down[e].abs().t() + (inter + 2) * 2.0 ** -24 * ((a.abs() + ea) @ down[e].abs().t())
        tt = torch.from_numpy(t)
        y.index_add_(0, tt, d * ww)
        bound.index_add_(0, tt, (ed + 2.0 ** -20 * d.abs()) * ww)
    return y, bound
