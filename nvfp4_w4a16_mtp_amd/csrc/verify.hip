// verify_drafts: acceptance of drafted tokens and the token after them
// (definition in nvfp4_mtp.h).
//
// A first pass over the logits gives for every chunk of a row its maximum, the sum of
// exp((l - max) / T) and, for greedy sequences, its first maximum's index.  Then one of
// two plans (verify_plan):
// - few rows of outright drafts, two launches: fp64 sums, without the draft's own
//   term; the second launch decides and draws from them and reads only the drafts'
//   logits and the chunk that holds the drawn token again;
// - else four: the decision; a second pass over the drawn rows (and the draft model's)
//   for the fp64 sums of what is drawn from; the draw and its chunk.  The first pass of
//   many outright drafts has fp32 sums, and a test too close for those is made again
//   with the row's fp64 sum.
// A row without a softmax is read again for its first maximum.  Bytes bound it for many
// rows, launches and dependent loads for few.
//
// Why fp64 where a token is drawn.  It is where a running sum over the vocabulary passes
// u * total.  A relative error e of the sums moves every one of V borders, so a
// draw changes with a probability up to about V * e: a few per cent in fp32 (V =
// 150000), 1e-7 with the exponential below.  gfx950 runs fp64 FMAs at the fp32
// rate, but its fp64 conversions, roundings and ldexp at a quarter of it: the
// exponential is 14 full-rate fp64 operations, one conversion and two integer
// operations.
#include "common.hpp"

namespace nvfp4 {

struct VerifyArgs {
    const void *logits, *draft;
    int64_t stride, dstride;
    int vocab, batch, rows, max_rows;
    const int32_t *cu, *ids;
    const float *temp, *ua, *us;
    const int32_t *lens;
    int32_t *accepted, *tokens, *next, *out_lens;
    int chunks;             // of a row, kChunk elements each
    struct VPart *part;     // [batch][max_rows][1 or 2][chunks]
    bool exact;             // the partials' sums are fp64
    bool second;            // k_verify_decide and k_verify_rest run
    double *rest;           // [batch][chunks]: sums of what is drawn from (second)
    struct Decision *decided;   // [batch] (second)
};

constexpr int kChunk = 2048;

struct VPart {
    double sum;             // of exp((l - max) / T) over the chunk (fp64 sums of outright
                            // drafts: without the draft's own term)
    float max;
    int idx;                // of the first maximum (-1: nothing above -inf); greedy sequences alone
};

// 2^(d c) for d c in [-1022, 0]: d c = n + r with n an integer (the sum with 1.5 *
// 2^52 holds it in its low bits), |r| <= 1/2, and 2^r = 1 + r P(r) with a
// near-minimax P of degree 7, relative error 8.2e-13 (equal logits give equal terms,
// the maximum exactly 1).  n is added to the exponent field.
__device__ __forceinline__ double exp2_neg(double d, double c) {
    const double t = __builtin_fma(d, c, 6755399441055744.0);
    const double r = __builtin_fma(d, c, -(t - 6755399441055744.0));
    double p = 1.3178936296684062e-06;
    p = __builtin_fma(p, r, 1.5309156251773027e-05);
    p = __builtin_fma(p, r, 0.0001540382545029347);
    p = __builtin_fma(p, r, 0.001333345486025463);
    p = __builtin_fma(p, r, 0.009618128616138841);
    p = __builtin_fma(p, r, 0.05550410935266539);
    p = __builtin_fma(p, r, 0.24022650698110554);
    p = __builtin_fma(p, r, 0.6931471805482123);
    p = __builtin_fma(p, r, 1.0);
    const uint64_t u = __builtin_bit_cast(uint64_t, p);
    const uint32_t hi = (uint32_t)(u >> 32) + ((uint32_t)__builtin_bit_cast(uint64_t, t) << 20);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | (uint32_t)u);
}
// The same without exact zeros: terms far below the maximum, of -inf and of NaN
// become 2^-1000, nothing beside the maximum's 1.  low = -1000 / c.
__device__ __forceinline__ double term_above(float l, float max, double low, double c) {
    return exp2_neg(fmax((double)l - (double)max, low), c);
}
// exp((l - max) / T), c = log2(e) / T: 0 far below the maximum (and for l =
// -inf), NaN for NaN.
__device__ __forceinline__ double term(float l, float max, double c) {
    const double d = (double)l - (double)max, y = d * c;
    const double e = exp2_neg(y > -1020.0 ? d : 0.0, c);
    return y > -1020.0 ? e : (y != y ? y : 0.0);
}

template <bool BF16>
__device__ __forceinline__ float logit(const void *base, int64_t at) {
    if (BF16) return bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(base)[at]);
    return reinterpret_cast<const float *>(base)[at];
}

struct VSeq {
    int r0, n, full;        // first row, rows considered, rows
};
__device__ __forceinline__ VSeq verify_seq(const VerifyArgs &a, int b) {
    VSeq q;
    const int lo = a.cu[b], hi = a.cu[b + 1];
    q.r0 = min(max(lo, 0), a.rows);
    q.full = min(max(hi, q.r0), a.rows) - q.r0;
    q.n = min(q.full, a.max_rows);
    return q;
}
// log2(e) / T, or 0 for greedy.
__device__ __forceinline__ double inv_temp(const VerifyArgs &a, int b) {
    const float t = a.temp ? a.temp[b] : 1.0f;
    return t > 0.0f && t < INFINITY ? 1.44269504088896340736 / (double)t : 0.0;
}

// A maximum with the lowest index among equals; NaN never wins.
__device__ __forceinline__ void take_max(float &bv, int &bi, float v, int i) {
    if (v > bv || (v == bv && i >= 0 && (unsigned)i < (unsigned)bi)) {
        bv = v;
        bi = i;
    }
}
__device__ __forceinline__ double shfl_xor_f64(double v, int m) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __shfl_xor((int)(uint32_t)u, m, 64), hi = __shfl_xor((int)(uint32_t)(u >> 32), m, 64);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double shfl_up_f64(double v, int d) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __shfl_up((int)(uint32_t)u, d, 64), hi = __shfl_up((int)(uint32_t)(u >> 32), d, 64);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Elements e0 .. e0 + N - 1 of a row (-inf from `end` on); `vec`: rows are 16-byte
// aligned and e0 * element size a multiple of the N elements' bytes or 16.
template <bool BF16, int N>
__device__ __forceinline__ void load_logits(const void *base, int64_t row, int e0, int end, bool vec, float (&x)[N]) {
    if (vec && e0 + N <= end) {
        if (BF16) {
            const uint16_t *p = reinterpret_cast<const uint16_t *>(base) + row + e0;
            uint32_t w[N / 2];
            if (N == 4) {
                const uint2 v = *reinterpret_cast<const uint2 *>(p);
                w[0] = v.x;
                w[1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < N / 8; ++i) {
                    const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
                    w[4 * i] = v.x;
                    w[4 * i + 1] = v.y;
                    w[4 * i + 2] = v.z;
                    w[4 * i + 3] = v.w;
                }
            }
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        } else {
            const float4 *p = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(base) + row + e0);
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {
                const float4 v = p[i];
                x[4 * i] = v.x;
                x[4 * i + 1] = v.y;
                x[4 * i + 2] = v.z;
                x[4 * i + 3] = v.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = e0 + i < end ? logit<BF16>(base, row + e0 + i) : -INFINITY;
    }
}

// ------------------------------------------------------ partials of chunks --
constexpr int kVThreads = 256;

// A chunk is taken by WAVES wavefronts, kChunk / (64 * WAVES) elements a lane in
// groups of 16 bytes.  WAVES = 1: no barriers, the loads of a workgroup's four
// chunks overlap with each other's sums (many rows).  WAVES = 4: a quarter of the
// terms per lane (few rows, where one chunk's time counts).  EXACT: fp64 terms.
// Else fp32 ones (v_exp_f32): the whole is off by less than 1e-5 (2^-22 of arguments
// up to 40, 32 fp32 additions), which decides every draft but those next to
// the border (see decide), and the drawn row is summed again.
template <bool BF16, int WAVES, bool EXACT>
__global__ __launch_bounds__(kVThreads) void k_verify_stats(VerifyArgs a, int kinds, bool vec) {
    constexpr int E = BF16 ? 8 : 4, PER = kChunk / (64 * WAVES), G = PER / E, T = 64 * WAVES;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int blocks = WAVES == 1 ? (a.chunks + 3) / 4 : a.chunks;
    int w = blockIdx.x / blocks;
    const int chunk = WAVES == 1 ? (blockIdx.x - w * blocks) * 4 + wave : blockIdx.x - w * blocks;
    const int kind = kinds == 2 ? w & 1 : 0;          // 0 target, 1 draft
    if (kinds == 2) w >>= 1;
    const int b = w / a.max_rows, i = w - b * a.max_rows;
    const VSeq q = verify_seq(a, b);
    if (i >= q.n || (kind == 1 && i == q.n - 1) || chunk >= a.chunks) return;
    const int tid = WAVES == 1 ? lane : (int)threadIdx.x, c0 = chunk * kChunk, c1 = min(c0 + kChunk, a.vocab);
    const void *base = kind ? a.draft : a.logits;
    const int64_t row = (int64_t)(q.r0 + i) * (kind ? a.dstride : a.stride);
    float x[G][E];
#pragma unroll
    for (int g = 0; g < G; ++g) load_logits<BF16, E>(base, row, c0 + (g * T + tid) * E, c1, vec, x[g]);
    const double it = inv_temp(a, b);
    const int id = EXACT && kinds == 1 && i < q.n - 1 ? a.ids[q.r0 + i] : -1;
    float mx = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < E; ++j) {
            mx = fmaxf(mx, x[g][j]);
            if (EXACT) nan |= x[g][j] != x[g][j];     // (an fp32 sum becomes NaN by itself)
        }
    const float own = mx;
    nan = EXACT && __any(nan);
    for (int m = 1; m < 64; m <<= 1) mx = fmaxf(mx, __shfl_xor(mx, m, 64));
    __shared__ float smax[4];
    __shared__ bool snan[4];
    __shared__ int sidx[4];
    __shared__ double ssum[4];
    if (WAVES > 1) {
        if (lane == 0) {
            smax[wave] = mx;
            snan[wave] = nan;
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < WAVES; ++v) {
            mx = fmaxf(mx, smax[v]);
            nan |= snan[v];
        }
    }
    // greedy: the first index that has the maximum
    int mi = 0x7FFFFFFF;
    if (!(it > 0.0)) {
        if (own == mx && mx > -INFINITY)
#pragma unroll
            for (int g = G - 1; g >= 0; --g)
#pragma unroll
                for (int j = E - 1; j >= 0; --j) mi = x[g][j] == mx ? c0 + (g * T + tid) * E + j : mi;
        for (int m = 1; m < 64; m <<= 1) mi = min(mi, __shfl_xor(mi, m, 64));
    }
    double sum = 0.0;
    if (it > 0.0) {
        if (id >= c0 && id < c1) {
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int j = 0; j < E; ++j)
                    if (c0 + (g * T + tid) * E + j == id) x[g][j] = -INFINITY;
        }
        const float ref = mx == -INFINITY ? 0.0f : mx;
        if (EXACT) {
            const double low = -1000.0 / it;          // (a NaN is noted)
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int j = 0; j < E; ++j) sum += term_above(x[g][j], ref, low, it);
        } else {
            // (finite logits can be 6.8e38 apart, which temperatures near that make count:
            // half the difference, exact, times 2 c)
            float c = (float)fmin(it, 3.0e38);
            const float h = c < 0x1p-100f ? 0.5f : 1.0f, shift = -ref * h;
            c /= h;
            float part = 0.0f;
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int j = 0; j < E; ++j) part += __builtin_amdgcn_exp2f(__builtin_fmaf(x[g][j], h, shift) * c);
            sum = part;
        }
        for (int m = 1; m < 64; m <<= 1) sum += shfl_xor_f64(sum, m);
    }
    if (WAVES > 1) {
        if (lane == 0) {
            ssum[wave] = sum;
            sidx[wave] = mi;
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < WAVES; ++v) mi = min(mi, sidx[v]);
        sum = 0.0;
#pragma unroll
        for (int v = 0; v < WAVES; ++v) sum += ssum[v];
    }
    if (tid == 0) {
        VPart p;
        // (nothing but terms far below, the excluded draft the only one: no weight)
        p.sum = nan || sum != sum ? NAN : mx > -INFINITY && sum > 0x1p-900 ? sum : 0.0;
        p.max = mx;
        p.idx = mx > -INFINITY && !(it > 0.0) ? mi : -1;
        a.part[((int64_t)(b * a.max_rows + i) * kinds + kind) * a.chunks + chunk] = p;
    }
}

// ---------------------------------------------------------------- decision --
// A whole row from its chunks (a wavefront; every lane gets the result).
struct VRow {
    double sum;
    float max;
    int idx;
    // a softmax exists: some mass, no NaN, no +inf
    __device__ __forceinline__ bool finite() const { return sum > 0.0 && sum < 1e300; }
};
__device__ __forceinline__ VRow join_chunks(const VPart *p, int chunks, double it, int lane) {
    VRow r{0.0, -INFINITY, -1};
    const VPart mine = p[min(lane, chunks - 1)];       // of the first 64 chunks
    if (lane < chunks) take_max(r.max, r.idx, mine.max, mine.idx);
    for (int c = lane + 64; c < chunks; c += 64) take_max(r.max, r.idx, p[c].max, p[c].idx);
    for (int m = 1; m < 64; m <<= 1) take_max(r.max, r.idx, __shfl_xor(r.max, m, 64), __shfl_xor(r.idx, m, 64));
    if (it > 0.0 && r.max > -INFINITY && r.max < INFINITY) {
        if (lane < chunks) r.sum = mine.sum * term(mine.max, r.max, it);
        for (int c = lane + 64; c < chunks; c += 64) r.sum += p[c].sum * term(p[c].max, r.max, it);
        for (int m = 1; m < 64; m <<= 1) r.sum += shfl_xor_f64(r.sum, m);
    }
    return r;
}

enum { kGreedy = 0, kFromP = 1, kWithout = 2, kRest = 3 };   // how the token is drawn

struct Decision {
    int row, draft, mode, best;      // stopping row (of the sequence), its draft, mode, its first maximum
    float pmax, qmax;
    double psum, qsum;
};

constexpr int kMaxRows = 64;
constexpr int kDecideThreads = 512;

// The sum of a whole row in fp64, by the whole workgroup.
template <bool BF16>
__device__ __forceinline__ double row_sum(const VerifyArgs &a, int64_t row, float max, double it) {
    __shared__ double part[kDecideThreads / 64];
    double sum = 0.0;
#pragma unroll 4
    for (int e = threadIdx.x; e < a.vocab; e += kDecideThreads) sum += term(logit<BF16>(a.logits, row * a.stride + e), max, it);
    for (int m = 1; m < 64; m <<= 1) sum += shfl_xor_f64(sum, m);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = 0.0;
    for (int i = 0; i < kDecideThreads / 64; ++i) sum += part[i];
    return sum;
}

// The first index of a row's maximum by the whole workgroup (0: nothing above -inf).
template <bool BF16>
__device__ __forceinline__ int row_first_max(const VerifyArgs &a, int64_t row) {
    __shared__ float pmax[kDecideThreads / 64];
    __shared__ int pidx[kDecideThreads / 64];
    float mx = -INFINITY;
    int mi = -1;
#pragma unroll 4
    for (int e = threadIdx.x; e < a.vocab; e += kDecideThreads) take_max(mx, mi, logit<BF16>(a.logits, row * a.stride + e), e);
    if (mx == -INFINITY) mi = -1;
    for (int m = 1; m < 64; m <<= 1) take_max(mx, mi, __shfl_xor(mx, m, 64), __shfl_xor(mi, m, 64));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        pmax[threadIdx.x >> 6] = mx;
        pidx[threadIdx.x >> 6] = mi;
    }
    __syncthreads();
    mx = -INFINITY;
    mi = -1;
    for (int i = 0; i < kDecideThreads / 64; ++i) take_max(mx, mi, pmax[i], pidx[i]);
    return mx > -INFINITY ? mi : 0;
}

// One workgroup of kDecideThreads: where sequence b stops and how its token is
// drawn.  The test u q(d) < p(d) is u wq sum_p < wd sum_q with the drafts' terms wd,
// wq; with fp32 sums a test whose sides agree to 2^-16 is made again with the row's
// fp64 sum.
template <bool BF16>
__device__ __forceinline__ void decide(const VerifyArgs &a, int b, const VSeq &q, double it, int kinds, Decision &d) {
    __shared__ VRow sp[kMaxRows], sq[kMaxRows];
    __shared__ double swd[kMaxRows];
    __shared__ float sua[kMaxRows];
    __shared__ int sstop[kMaxRows], sid[kMaxRows];    // 2: too close to tell, 3: no softmax
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (int i = wave; i < q.n; i += kDecideThreads / 64) {
        const VPart *p = a.part + ((int64_t)(b * a.max_rows + i) * kinds) * a.chunks;
        const bool last = i == q.n - 1;
        const int64_t row = q.r0 + i;
        const int id = last ? -1 : a.ids[row];
        const bool in = id >= 0 && id < a.vocab;
        const float ld = in ? logit<BF16>(a.logits, row * a.stride + id) : 0.0f;
        const float lq = in && kinds == 2 ? logit<BF16>(a.draft, row * a.dstride + id) : 0.0f;
        const float ua = last ? 0.0f : a.ua[row];
        VRow rp = join_chunks(p, a.chunks, it, lane);
        VRow rq{0.0, -INFINITY, -1};
        double wd = 0.0;                              // the draft's term of the sum
        int stop = 1;
        if (!last) {
            if (in && it > 0.0 && rp.max > -INFINITY && rp.max < INFINITY) {
                wd = term(ld, rp.max, it);
                if (kinds == 1 && a.exact) rp.sum += wd;
            }
            if (kinds == 2) rq = join_chunks(p + a.chunks, a.chunks, it, lane);
            if (!(it > 0.0)) {
                stop = id != max(rp.idx, 0);
            } else if (!rp.finite()) {
                stop = 3;
            } else if (in) {
                double lhs = (double)ua * rp.sum, rhs = wd;
                if (kinds == 2 && rq.finite()) {
                    lhs *= term(lq, rq.max, it);
                    rhs *= rq.sum;
                }
                stop = !(lhs < rhs);
                if (!a.exact && fabs(lhs - rhs) <= rhs * 0x1p-16) stop = 2;
            }
        }
        if (lane == 0) {
            sp[i] = rp;
            sq[i] = rq;
            swd[i] = wd;
            sua[i] = ua;
            sid[i] = id;
            sstop[i] = stop;
        }
    }
    __syncthreads();
    int at = 0, best = 0;
    for (;; ++at) {                                   // the last row always stops
        int stop = sstop[at];
        best = max(sp[at].idx, 0);
        if (stop == 3 || (at == q.n - 1 && it > 0.0 && !sp[at].finite())) {
            best = row_first_max<BF16>(a, q.r0 + at);
            stop = at == q.n - 1 || sid[at] != best;
        }
        if (stop == 2) stop = !((double)sua[at] * row_sum<BF16>(a, q.r0 + at, sp[at].max, it) < swd[at]);
        if (stop) break;
    }
    const bool last = at == q.n - 1;
    const VRow rp = sp[at], rq = sq[at];
    d.row = at;
    d.draft = sid[at];
    d.best = best;
    d.pmax = rp.max;
    d.psum = rp.sum;
    d.qmax = rq.max;
    d.qsum = rq.sum;
    if (!(it > 0.0) || !rp.finite())
        d.mode = kGreedy;
    else if (last)
        d.mode = kFromP;
    else if (kinds == 2 && rq.finite())
        d.mode = kRest;
    else
        d.mode = d.draft >= 0 && d.draft < a.vocab ? kWithout : kFromP;
    __syncthreads();
}

// Weights of a thread's N elements e0 .. under the decision (0 from `end` on).
template <bool BF16, int N>
__device__ __forceinline__ void weights(const VerifyArgs &a, const Decision &d, int mode, int64_t row, int e0, int end,
                                        double it, bool vec, double (&w)[N]) {
    float x[N];
    load_logits<BF16, N>(a.logits, row * a.stride, e0, end, vec, x);
    if (mode == kRest) {
        float y[N];
        load_logits<BF16, N>(a.draft, row * a.dstride, e0, end, vec, y);
        const double ip = 1.0 / d.psum, iq = 1.0 / d.qsum;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const double r = term(x[i], d.pmax, it) * ip - term(y[i], d.qmax, it) * iq;
            w[i] = e0 + i < end && r > 0.0 ? r : 0.0;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = mode == kWithout && e0 + i == d.draft ? 0.0 : term(x[i], d.pmax, it);
    }
}

template <bool BF16>
__global__ __launch_bounds__(kDecideThreads) void k_verify_decide(VerifyArgs a, int kinds) {
    const int b = blockIdx.x;
    const VSeq q = verify_seq(a, b);
    if (q.n == 0) return;
    Decision d;
    decide<BF16>(a, b, q, inv_temp(a, b), kinds, d);
    if (threadIdx.x == 0) a.decided[b] = d;
}

// Per chunk (WAVES wavefronts, steps of 512 elements) the fp64 sums of what is drawn
// from: max(p - q, 0), or p, or p without the draft.  Two wavefronts a chunk where one
// leaves the SIMDs less than four deep (24 sequences' pairs of fp32 rows of 129280: 47.6
// us the whole call with one, 45.9 with two, 46.1 with four; 64 sequences' bf16 rows of
// 151936: 53.2, 54.0, 53.8).
template <bool BF16, int WAVES>
__global__ __launch_bounds__(kVThreads) void k_verify_rest(VerifyArgs a, bool vec) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, blocks = (a.chunks * WAVES + 3) / 4;
    const int b = blockIdx.x / blocks, chunk = ((blockIdx.x - b * blocks) * 4 + wave) / WAVES, part = wave % WAVES;
    const VSeq q = verify_seq(a, b);
    if (q.n == 0) return;
    const Decision d = a.decided[b];
    if (d.mode == kGreedy) return;
    const double it = inv_temp(a, b);
    // (past the last chunk: the last one again, not stored)
    const int c0 = min(chunk, a.chunks - 1) * kChunk, c1 = min(c0 + kChunk, a.vocab);
    const int64_t row = q.r0 + d.row;
    const double low = -1000.0 / it;
    const double ip = 1.0 / d.psum, iq = 1.0 / d.qsum;
    double sum = 0.0;
#pragma unroll 2
    for (int k = 0; k < kChunk / 512 / WAVES; ++k) {
        const int e0 = c0 + (k * WAVES + part) * 512 + lane * 8;
        float x[8];
        load_logits<BF16, 8>(a.logits, row * a.stride, e0, c1, vec, x);
        if (d.mode == kRest) {
            float y[8];
            load_logits<BF16, 8>(a.draft, row * a.dstride, e0, c1, vec, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const double r = term_above(x[i], d.pmax, low, it) * ip - term_above(y[i], d.qmax, low, it) * iq;
                sum += r > 0.0 ? r : 0.0;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum += term_above(d.mode == kWithout && e0 + i == d.draft ? -INFINITY : x[i], d.pmax, low, it);
        }
    }
    for (int m = 1; m < 64; m <<= 1) sum += shfl_xor_f64(sum, m);
    if (WAVES > 1) {
        __shared__ double sums[4];
        if (lane == 0) sums[wave] = sum;
        __syncthreads();
#pragma unroll
        for (int i = 1; i < WAVES; ++i) sum += sums[(wave + i) & 3];
    }
    // a chunk of nothing but terms far below holds no weight
    if (lane == 0 && part == 0 && chunk < a.chunks) a.rest[(int64_t)b * a.chunks + chunk] = sum > 0x1p-900 ? sum : 0.0;
}

__device__ __forceinline__ double lane_f64(double v, int l) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __shfl((int)(uint32_t)u, l, 64), hi = __shfl((int)(uint32_t)(u >> 32), l, 64);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// One workgroup per sequence: the decision, the draw, the outputs.
template <bool BF16, bool SECOND>
__global__ __launch_bounds__(kDecideThreads) void k_verify_pick(VerifyArgs a, int kinds, bool vec) {
    constexpr int N = kChunk / kDecideThreads;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const VSeq q = verify_seq(a, b);
    if (q.n == 0) {
        if (tid == 0) {
            a.accepted[b] = 0;
            a.next[b] = -1;
            if (a.out_lens) a.out_lens[b] = a.lens[b];
        }
        return;
    }
    const double it = inv_temp(a, b);
    Decision d;
    if (SECOND)
        d = a.decided[b];
    else
        decide<BF16>(a, b, q, it, kinds, d);
    __shared__ int schunk, smode, shit[kDecideThreads / 64], slast[kDecideThreads / 64];
    __shared__ double starget, wsum[kDecideThreads / 64];
    int token = d.mode == kWithout ? d.draft : d.best;   // (kWithout: should nothing else have weight)
    if (d.mode != kGreedy) {
        const VPart *part = a.part + ((int64_t)(b * a.max_rows + d.row) * kinds) * a.chunks;
        const double *rest = a.rest + (int64_t)b * a.chunks;
        if (wave == 0) {
            // chunk weights, their running sum, and the chunk that passes u * total
            // (the partials of outright drafts are already without the draft)
            int mode = d.mode;
            bool again = SECOND;
            auto chunk_weight = [&](int c) {
                if (c >= a.chunks) return 0.0;
                if (again) return rest[c];
                return part[c].max > -INFINITY ? part[c].sum * term(part[c].max, d.pmax, it) : 0.0;
            };
            double mine = chunk_weight(lane), total = mine;
            for (int c = lane + 64; c < a.chunks; c += 64) total += chunk_weight(c);
            for (int m = 1; m < 64; m <<= 1) total += shfl_xor_f64(total, m);
            if (mode == kRest && !(total > 0.0)) {    // p and q are equal: draw from p
                mode = kFromP;
                again = false;
                total = d.psum;
                mine = chunk_weight(lane);
            }
            const double target = (double)a.us[b] * total;
            double before = 0.0, from = 0.0, live_from = 0.0;
            int hit = -1, live = -1;                  // the chunk found; the last one with weight
            for (int c0 = 0; c0 < a.chunks && hit < 0; c0 += 64) {
                const double own = c0 == 0 ? mine : chunk_weight(c0 + lane);
                double run = own;
                for (int s = 1; s < 64; s <<= 1) {
                    const double o = shfl_up_f64(run, s);
                    if (lane >= s) run += o;
                }
                const uint64_t pass = __ballot(before + run > target && own > 0.0), some = __ballot(own > 0.0);
                const double excl = before + run - own;
                if (pass) {
                    hit = c0 + __builtin_ctzll(pass);
                    from = lane_f64(excl, hit - c0);
                }
                if (some) {
                    live = c0 + 63 - __builtin_clzll(some);
                    live_from = lane_f64(excl, live - c0);
                }
                before = lane_f64(before + run, 63);
            }
            if (hit < 0) {                            // rounding at the very end
                hit = live;
                from = live_from;
            }
            if (lane == 0) {
                schunk = hit;
                starget = target - from;
                smode = mode;
            }
        }
        __syncthreads();
        const int chunk = schunk;
        if (chunk >= 0) {
            // the chunk again: N elements a thread, their running sum
            const double target = starget;
            const int c0 = chunk * kChunk, c1 = min(c0 + kChunk, a.vocab), e0 = c0 + tid * N;
            double w[N], own = 0.0;
            weights<BF16, N>(a, d, smode, q.r0 + d.row, e0, c1, it, vec, w);
            int last = -1;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                own += w[i];
                last = w[i] > 0.0 ? e0 + i : last;
            }
            double run = own;
            for (int s = 1; s < 64; s <<= 1) {
                const double o = shfl_up_f64(run, s);
                if (lane >= s) run += o;
            }
            if (lane == 63) wsum[wave] = run;
            __syncthreads();
            double sum = run - own;
            for (int i = 0; i < wave; ++i) sum += wsum[i];
            int at = -1;                              // the first element that passes the target
            if (sum + own > target && own > 0.0) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    sum += w[i];
                    at = at < 0 && w[i] > 0.0 && sum > target ? e0 + i : at;
                }
            }
            // of the lowest lane that has one; the last element with weight of the
            // highest lane
            const uint64_t hits = __ballot(at >= 0), live = __ballot(last >= 0);
            const int hit = hits ? __shfl(at, __builtin_ctzll(hits), 64) : -1;
            const int end = live ? __shfl(last, 63 - __builtin_clzll(live), 64) : -1;
            if (lane == 0) {
                shit[wave] = hit;
                slast[wave] = end;
            }
            __syncthreads();
            int fall = -1, found = -1;
            for (int i = 0; i < kDecideThreads / 64; ++i) {
                found = found < 0 ? shit[i] : found;
                fall = slast[i] >= 0 ? slast[i] : fall;
            }
            token = found >= 0 ? found : (fall >= 0 ? fall : token);
        }
    }
    for (int i = tid; i < q.n; i += kDecideThreads)
        a.tokens[q.r0 + i] = i < d.row ? a.ids[q.r0 + i] : (i == d.row ? token : -1);
    if (tid == 0) {
        a.accepted[b] = d.row;
        a.next[b] = token;
        if (a.out_lens) a.out_lens[b] = a.lens[b] - q.full + d.row + 1;
    }
}

struct VerifyPlan {
    int chunks;
    bool exact, second, many;
    size_t part, ws;
};

static VerifyPlan verify_plan(int batch, int max_rows, int vocab, bool draft) {
    VerifyPlan p;
    const int64_t rows = (int64_t)batch * max_rows * (draft ? 2 : 1);
    p.chunks = (vocab + kChunk - 1) / kChunk;
    // a wavefront a chunk once they fill the device's SIMDs four deep
    p.many = rows * p.chunks >= (int64_t)num_cus() * 16;
    // Outright drafts of many rows: fp32 partials and a second pass over the drawn
    // rows (337 rows of 151936: 63 us against 68 with fp64 partials of every row); of
    // few: fp64 partials, no second pass (4 rows: 15.7 us with two launches).
    p.exact = draft || !p.many;
    p.second = draft || !p.exact;
    p.part = (size_t)rows * p.chunks * sizeof(VPart);
    p.ws = p.part + (p.second ? (size_t)batch * (p.chunks * sizeof(double) + sizeof(Decision)) : 0);
    return p;
}

template <bool BF16>
static void launch_verify(const VerifyArgs &a, bool many, bool draft, bool vec, hipStream_t s) {
    const int kinds = draft ? 2 : 1;
    const int64_t rows = (int64_t)a.batch * a.max_rows * kinds;
    const dim3 grid((unsigned)(rows * (many ? (a.chunks + 3) / 4 : a.chunks)));
    if (!many)
        hipLaunchKernelGGL((k_verify_stats<BF16, 4, true>), grid, dim3(kVThreads), 0, s, a, kinds, vec);
    else if (a.exact)
        hipLaunchKernelGGL((k_verify_stats<BF16, 1, true>), grid, dim3(kVThreads), 0, s, a, kinds, vec);
    else
        hipLaunchKernelGGL((k_verify_stats<BF16, 1, false>), grid, dim3(kVThreads), 0, s, a, kinds, vec);
    if (a.second) {
        hipLaunchKernelGGL((k_verify_decide<BF16>), dim3((unsigned)a.batch), dim3(kDecideThreads), 0, s, a, kinds);
        if (a.batch * a.chunks < num_cus() * 16)
            hipLaunchKernelGGL((k_verify_rest<BF16, 2>), dim3((unsigned)(a.batch * ((a.chunks * 2 + 3) / 4))), dim3(kVThreads), 0, s, a, vec);
        else
            hipLaunchKernelGGL((k_verify_rest<BF16, 1>), dim3((unsigned)(a.batch * ((a.chunks + 3) / 4))), dim3(kVThreads), 0, s, a, vec);
    }
    if (a.second)
        hipLaunchKernelGGL((k_verify_pick<BF16, true>), dim3((unsigned)a.batch), dim3(kDecideThreads), 0, s, a, kinds, vec);
    else
        hipLaunchKernelGGL((k_verify_pick<BF16, false>), dim3((unsigned)a.batch), dim3(kDecideThreads), 0, s, a, kinds, vec);
}

}  // namespace nvfp4

using namespace nvfp4;

static int verify_shape(int batch, int max_rows, int vocab, const char *who) {
    if (batch < 0 || max_rows < 1 || max_rows > kMaxRows || vocab < 1 || vocab > (1 << 24))
        return fail(NVFP4_ERR_SHAPE, "%s: need batch >= 0, max_rows in 1..%d, vocab in 1..2^24 (batch=%d max_rows=%d vocab=%d)",
                    who, kMaxRows, batch, max_rows, vocab);
    return NVFP4_OK;
}

extern "C" size_t verify_drafts_workspace_bytes(int32_t batch, int32_t max_rows, int32_t vocab, int32_t with_draft_logits) {
    if (verify_shape(batch, max_rows, vocab, "verify_drafts_workspace_bytes")) return 0;
    return verify_plan(batch, max_rows, vocab, with_draft_logits != 0).ws + 16;
}

extern "C" int verify_drafts(const void *logits, int32_t logits_dtype, int64_t row_stride, int32_t vocab,
                             const void *draft_logits, int64_t draft_stride, const int32_t *cu_rows, int32_t batch,
                             int32_t rows, int32_t max_rows, const int32_t *draft_ids, const float *temperature,
                             const float *u_accept, const float *u_sample, const int32_t *kv_lens, int32_t *out_accepted,
                             int32_t *out_tokens, int32_t *out_next, int32_t *out_kv_lens, void *workspace,
                             size_t ws_bytes, void *stream) {
    const char *who = "verify_drafts";
    if (int rc = verify_shape(batch, max_rows, vocab, who)) return rc;
    if (rows < 0) return fail(NVFP4_ERR_SHAPE, "%s: rows=%d < 0", who, rows);
    if (logits_dtype != NVFP4_OUT_F32 && logits_dtype != NVFP4_OUT_BF16)
        return fail(NVFP4_ERR_ARG, "%s: unknown logits_dtype %d", who, logits_dtype);
    if (batch == 0) return ok();
    if (!cu_rows || !out_accepted || !out_next || (rows > 0 && (!logits || !draft_ids || !u_accept || !u_sample || !out_tokens)))
        return fail(NVFP4_ERR_ARG, "%s: NULL logits, cu_rows, draft_ids, u_accept, u_sample or output", who);
    if ((kv_lens == nullptr) != (out_kv_lens == nullptr))
        return fail(NVFP4_ERR_ARG, "%s: kv_lens and out_kv_lens go together", who);
    if (row_stride < vocab || (draft_logits && draft_stride < vocab))
        return fail(NVFP4_ERR_SHAPE, "%s: a row stride (%lld, %lld) is below vocab=%d", who, (long long)row_stride,
                    (long long)draft_stride, vocab);
    const bool bf16 = logits_dtype == NVFP4_OUT_BF16;
    const uintptr_t el = bf16 ? 2 : 4;
    if (!aligned(logits, el) || !aligned(draft_logits, el))
        return fail(NVFP4_ERR_ALIGN, "%s: logits not aligned to their element", who);
    for (const void *p : {(const void *)cu_rows, (const void *)draft_ids, (const void *)temperature, (const void *)u_accept,
                          (const void *)u_sample, (const void *)kv_lens, (const void *)out_accepted, (const void *)out_tokens,
                          (const void *)out_next, (const void *)out_kv_lens})
        if (!aligned(p, 4)) return fail(NVFP4_ERR_ALIGN, "%s: an int32 or fp32 array is not 4-byte aligned", who);
    const VerifyPlan p = verify_plan(batch, max_rows, vocab, draft_logits != nullptr);
    if (!workspace || ws_bytes < p.ws + 16)
        return fail(NVFP4_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", who, workspace ? ws_bytes : 0, p.ws + 16);
    if (!aligned(workspace, 16)) return fail(NVFP4_ERR_ALIGN, "%s: workspace not 16-byte aligned", who);
    if (!grid_fits((int64_t)batch * max_rows * (draft_logits ? 2 : 1) * (p.many ? (p.chunks + 3) / 4 : p.chunks), kVThreads))
        return fail(NVFP4_ERR_UNSUPPORTED, "%s: grid too large", who);
    VerifyArgs a;
    a.logits = logits;
    a.draft = draft_logits;
    a.stride = row_stride;
    a.dstride = draft_stride;
    a.vocab = vocab;
    a.batch = batch;
    a.rows = rows;
    a.max_rows = max_rows;
    a.cu = cu_rows;
    a.ids = draft_ids;
    a.temp = temperature;
    a.ua = u_accept;
    a.us = u_sample;
    a.lens = kv_lens;
    a.accepted = out_accepted;
    a.tokens = out_tokens;
    a.next = out_next;
    a.out_lens = out_kv_lens;
    a.chunks = p.chunks;
    a.exact = p.exact;
    a.second = p.second;
    a.part = static_cast<VPart *>(workspace);
    a.rest = reinterpret_cast<double *>(static_cast<char *>(workspace) + p.part);
    a.decided = reinterpret_cast<Decision *>(a.rest + (size_t)batch * p.chunks);
    const bool vec = aligned(logits, 16) && row_stride * el % 16 == 0 &&
                     (!draft_logits || (aligned(draft_logits, 16) && draft_stride * el % 16 == 0));
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (bf16)
        launch_verify<true>(a, p.many, draft_logits != nullptr, vec, s);
    else
        launch_verify<false>(a, p.many, draft_logits != nullptr, vec, s);
    return check_launch(who);
}
