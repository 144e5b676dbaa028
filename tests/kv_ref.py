"""Plain 64-bit forms (numpy) of the draft step's attention operators and of
draft verification, for the tests: definitions only, no sharing with the HIP
path."""
import math

import numpy as np

MIN_EXP, MAX_EXP = -110, 119     # of a page's scale; 448 * 2^119 is finite in bf16
E4M3 = np.array([(-1.0 if b & 128 else 1.0) * ((b & 7) * 2.0 ** -9 if (b >> 3) & 15 == 0 else
                                               (1 + (b & 7) / 8) * 2.0 ** (((b >> 3) & 15) - 7)) for b in range(256)])
E4M3[[0x7F, 0xFF]] = np.nan
_GRID = E4M3[:0x7F]


def bf16(x):
    """float64 values rounded to the nearest bf16 (through fp32, as a kernel's
    fp32 result is)."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    r = np.where(np.isnan(np.asarray(x, np.float32)), np.uint32(0x7FC00000), r)
    return r.view(np.float32).astype(np.float64)


def e4m3_encode(x):
    """Nearest E4M3 code, ties to the even code, saturating; NaN -> 0x7F with
    the sign unspecified (0x7F here)."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.searchsorted(_GRID, a, side="left").clip(0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _GRID[lo], _GRID[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(_GRID[hi] == a, hi, code).astype(np.uint8)
    code = code | np.where(np.signbit(x), np.uint8(0x80), np.uint8(0))
    return np.where(np.isnan(x), np.uint8(0x7F), code).astype(np.uint8)


def scale_exp(amax):
    """Smallest exponent >= MIN_EXP with amax <= 448 * 2^e."""
    if amax == 0:
        return MIN_EXP
    e = math.frexp(amax)[1] - 9
    if amax > 448.0 * 2.0 ** e:
        e += 1
    return max(e, MIN_EXP)


def scale_of(byte):
    return 2.0 ** (min(int(byte) - 127, MAX_EXP))


class Cache:
    """Host copy of a paged cache; K and V pages [pages][heads][tokens][dim]."""

    def __init__(self, pages, heads, tokens, dim, rng=None):
        self.tokens = tokens
        shape = (pages, heads, tokens, dim)
        if rng is None:
            self.k, self.v = np.zeros(shape, np.uint8), np.zeros(shape, np.uint8)
            self.ks, self.vs = np.zeros(shape[:2], np.uint8), np.zeros(shape[:2], np.uint8)
        else:
            # stale content: any finite code, plausible scales
            self.k, self.v = (rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2))
            for c in (self.k, self.v):
                c[(c & 0x7F) == 0x7F] = 0x11
            self.ks, self.vs = (rng.integers(117, 124, shape[:2]).astype(np.uint8) for _ in range(2))

    def clone(self):
        c = Cache.__new__(Cache)
        c.tokens = self.tokens
        c.k, c.v, c.ks, c.vs = (x.copy() for x in (self.k, self.v, self.ks, self.vs))
        return c

    def append(self, table, cu, lens, k, v, max_rows=None):
        """k, v float64 [rows][heads][dim] (bf16 values)."""
        P, pages = self.tokens, self.k.shape[0]
        cap = table.shape[1] * P
        for b in range(len(lens)):
            r0 = min(max(int(cu[b]), 0), len(k))
            full = min(max(int(cu[b + 1]), r0), len(k)) - r0
            n = full if max_rows is None else min(full, max_rows)
            length = min(max(int(lens[b]), 0), cap)
            shift = length - full
            for first in range(max(shift, 0) // P * P, max(shift + n, 0), P):
                page = int(table[b, first // P])
                if not 0 <= page < pages:
                    continue
                o0, o1 = max(shift - first, 0), min(shift + n - first, P)
                if o1 <= o0:
                    continue
                rows = slice(r0 + first + o0 - shift, r0 + first + o1 - shift)
                for x, codes, scales in ((k, self.k, self.ks), (v, self.v, self.vs)):
                    for h in range(codes.shape[1]):
                        new = x[rows, h]
                        fin = np.abs(new[np.isfinite(new)])
                        e = min(scale_exp(fin.max() if fin.size else 0.0), MAX_EXP)
                        if o0 > 0:
                            s = scale_of(scales[page, h])
                            e = max(e, min(int(scales[page, h]) - 127, MAX_EXP))
                            if s != 2.0 ** e:
                                old = codes[page, h, :o0]
                                re = e4m3_encode(E4M3[old] * (s / 2.0 ** e))
                                codes[page, h, :o0] = np.where((old & 0x7F) == 0x7F, old, re)
                        codes[page, h, o0:o1] = e4m3_encode(new / 2.0 ** e)
                        scales[page, h] = e + 127

    def values(self, table, b, length, heads_first=True):
        """(k, v) float64 [heads][length][dim] and which tokens have a page."""
        P = self.tokens
        ks, vs, ok = [], [], []
        for t in range(0, length, P):
            page = int(table[b, t // P])
            inside = 0 <= page < self.k.shape[0]
            pg = page if inside else 0
            sk = np.array([scale_of(x) for x in self.ks[pg]])[:, None, None]
            sv = np.array([scale_of(x) for x in self.vs[pg]])[:, None, None]
            ks.append(E4M3[self.k[pg]] * sk)
            vs.append(E4M3[self.v[pg]] * sv)
            ok += [inside] * P
        if not ks:
            z = np.zeros((self.k.shape[1], 0, self.k.shape[3]))
            return z, z, np.zeros(0, bool)
        return np.concatenate(ks, 1)[:, :length], np.concatenate(vs, 1)[:, :length], np.array(ok[:length])


def attention(q, cache, table, cu, lens, scale, window=0, sinks=0):
    """(out, bound) float64 [rows][q_heads][dim]: bound is what the kernel's
    arithmetic may be off by before... including its last rounding.

    With u = 2^-24 and A = sum p |v| (softmax p): fp32 scores are off by ds <=
    (D + 4) u scale sum |q||k| plus two products (2 u |s|), so a weight by a
    factor 1 + 2 ds + 2^-21 (exp2, its argument in fp32: |s| u more); weights
    are rounded to bf16 (2^-8); sums of up to L terms in fp32 add (L + 64) u for
    numerator and denominator each; the result is rounded to bf16 (2^-8)."""
    u = 2.0 ** -24
    rows, hq, d = q.shape
    out, bound = np.zeros_like(q), np.zeros_like(q)
    owned = np.zeros(rows, bool)
    heads = cache.k.shape[1]
    g = hq // heads
    cap = table.shape[1] * cache.tokens
    for b in range(len(lens)):
        r0 = min(max(int(cu[b]), 0), rows)
        n = min(max(int(cu[b + 1]), r0), rows) - r0
        length = min(max(int(lens[b]), 0), cap)
        k, v, ok = cache.values(table, b, length)
        t = np.arange(length)
        for i in range(n):
            owned[r0 + i] = True
            pos = length - n + i
            see = (t <= pos) & ok
            if window:
                see &= (t > pos - window) | (t < sinks)
            if not see.any():
                continue
            for h in range(hq):
                kk, vv = k[h // g][see], v[h // g][see]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = kk @ q[r0 + i, h] * scale
                    p = np.exp(s - s.max())
                    p = p / p.sum()
                    out[r0 + i, h] = p @ vv
                    a = p @ np.abs(vv)
                    ds = ((d + 4) * u * abs(scale) * (np.abs(kk) @ np.abs(q[r0 + i, h])) + 6 * u * np.abs(s)).max()
                    bound[r0 + i, h] = 2.0 ** -8 * np.abs(out[r0 + i, h]) + (1 + 2.0 ** -8) * a * (
                        2.0 ** -8 + 4 * ds + 2.0 ** -20 + 2 * (len(p) + 64) * u) + 1e-30
    return out, bound, owned


def rotate(x, pos, freq, rot, interleaved=False, mscale=1.0):
    """x float64 [rows][heads][dim] rotated (not rounded)."""
    y = x.copy()
    ang = np.asarray(pos, np.float64)[:, None] * freq[None, :]
    c, s = (np.cos(ang) * mscale)[:, None, :], (np.sin(ang) * mscale)[:, None, :]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, a * s + b * c
    return y


def first_max(x):
    """Index of the ascending strict-greater scan: NaN never wins, 0 if nothing
    exceeds -inf."""
    best, at = -np.inf, 0
    for i in np.flatnonzero(x > -np.inf):
        if x[i] > best:
            best, at = x[i], int(i)
    return at


def softmax(x, t):
    """exp(x / t) up to a factor and its sum, or None where there is no finite
    sum.  (Equal logits give equal exact terms, so a draw at an exact border of
    their running sum is exact too; terms divided by the sum would not be.)"""
    if np.isnan(x).any() or np.isposinf(x).any() or not (x > -np.inf).any():
        return None
    e = np.exp((x - x.max()) / t)
    return e, e.sum()


def verify(logits, cu, ids, ua, us, temp=None, draft=None, lens=None, max_rows=64):
    rows, vocab = logits.shape
    batch = len(cu) - 1
    acc, nxt = np.zeros(batch, np.int32), np.full(batch, -1, np.int32)
    tokens = np.full(rows, -999, np.int32)
    kept = None if lens is None else np.array(lens, np.int32)
    for b in range(batch):
        r0, full = int(cu[b]), int(cu[b + 1] - cu[b])
        n = min(full, max_rows)
        if n == 0:
            continue
        t = 1.0 if temp is None else float(temp[b])
        greedy = not (t > 0 and math.isfinite(t))
        for i in range(n):
            r, last = r0 + i, i == n - 1
            x = logits[r].astype(np.float64)
            p = None if greedy else softmax(x, t)
            d = int(ids[r])
            inside = 0 <= d < vocab
            if p is None:
                best = first_max(x)
                if not last and d == best:
                    continue
                tok = best
                break
            q = softmax(draft[r].astype(np.float64), t) if draft is not None and not last else None
            outright = q is None
            if outright:
                q = np.zeros(vocab)
                if inside:
                    q[d] = 1.0
            else:
                q = q[0] / q[1]
            p, total = p
            if not last and inside and float(ua[r]) * q[d] < p[d] / total:
                continue
            w = p.copy()
            if not last and outright and inside:
                w[d] = 0.0
            elif not last and not outright:
                w = np.maximum(p / total - q, 0.0)
            if not w.sum() > 0:
                w = p
            c = np.cumsum(w)
            hits = np.flatnonzero(c > float(us[b]) * c[-1])
            tok = int(hits[0]) if len(hits) else int(np.flatnonzero(w > 0)[-1])
            break
        acc[b], nxt[b] = i, tok
        tokens[r0:r0 + n] = -1
        tokens[r0:r0 + i] = ids[r0:r0 + i]
        tokens[r0 + i] = tok
        if kept is not None:
            kept[b] = lens[b] - full + i + 1
    return acc, tokens, nxt, kept
