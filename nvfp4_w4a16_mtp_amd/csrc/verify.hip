// verify_drafts: acceptance of drafted tokens and the token after them
// (definition in nvfp4_mtp.h).
//
// The logits are read once: a chunk of a row gives its maximum, the sum of
// exp((l - max) / T) and its first maximum's index.  Everything after that works
// on those partials, and only the one chunk that holds the drawn token is read
// again.  Bytes bound it for many rows, launches and dependent loads for few.
//
// Why fp64.  The drawn token is where a running sum over the vocabulary passes
// u * total.  A relative error e of the sums moves every one of V borders, so a
// draw changes with a probability up to about V * e: a few per cent in fp32 (V =
// 150000), 1e-9 in fp64.  gfx950 runs fp64 FMAs at the fp32 rate, so the
// exponentials (about 20 FMAs each) stay near the time the bytes take.
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
    int chunk, chunks;
    struct VPart *part;     // [batch][max_rows][1 or 2][chunks]
    double *rest;           // [batch][chunks]: sums of max(p - q, 0)
};

struct VPart {
    double sum;             // of exp((l - max) / T) over the chunk; without the draft's own
                            // term where the draft is outright
    float max;
    int idx;                // of the first maximum (-1: nothing above -inf)
};

// exp(x), x <= 0 (or NaN): relative error about 1e-14.
__device__ __forceinline__ double exp_neg(double x) {
    x = x < -800.0 ? -800.0 : x;
    const double n = __builtin_rint(x * 1.44269504088896340736);
    const double r = __builtin_fma(n, -0.69314718055994530942, x);   // |r| <= 0.347
    double p = 1.0 / 39916800.0;                                     // Taylor to r^11
    p = __builtin_fma(p, r, 1.0 / 3628800.0);
    p = __builtin_fma(p, r, 1.0 / 362880.0);
    p = __builtin_fma(p, r, 1.0 / 40320.0);
    p = __builtin_fma(p, r, 1.0 / 5040.0);
    p = __builtin_fma(p, r, 1.0 / 720.0);
    p = __builtin_fma(p, r, 1.0 / 120.0);
    p = __builtin_fma(p, r, 1.0 / 24.0);
    p = __builtin_fma(p, r, 1.0 / 6.0);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return __builtin_ldexp(p, (int)n);
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
// 1 / T, or 0 for greedy.
__device__ __forceinline__ double inv_temp(const VerifyArgs &a, int b) {
    const float t = a.temp ? a.temp[b] : 1.0f;
    return t > 0.0f ? 1.0 / (double)t : 0.0;
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

// ------------------------------------------------------ partials of chunks --
constexpr int kVThreads = 256;

// PER elements a thread in groups of E (16 bytes); VEC: rows are 16-byte
// aligned.
template <bool BF16, int PER, bool VEC>
__global__ __launch_bounds__(kVThreads) void k_verify_stats(VerifyArgs a, int kinds) {
    constexpr int E = BF16 ? 8 : 4;
    const int chunk = blockIdx.x % a.chunks;
    int w = blockIdx.x / a.chunks;
    const int kind = w % kinds;                       // 0 target, 1 draft
    w /= kinds;
    const int i = w % a.max_rows, b = w / a.max_rows;
    const VSeq q = verify_seq(a, b);
    if (i >= q.n || (kind == 1 && i == q.n - 1)) return;
    const double it = inv_temp(a, b);
    const int tid = threadIdx.x, c0 = chunk * a.chunk, c1 = min(c0 + a.chunk, a.vocab);
    const void *base = kind ? a.draft : a.logits;
    const int64_t row = (int64_t)(q.r0 + i) * (kind ? a.dstride : a.stride);
    float x[PER];
#pragma unroll
    for (int g = 0; g < PER / E; ++g) {
        const int e0 = c0 + (g * kVThreads + tid) * E;
        if (VEC && e0 + E <= c1) {
            if (BF16) {
                const uint4 v = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(base) + row + e0);
                const uint32_t p[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < E; ++j) x[g * E + j] = bf16_bits_to_f32(j & 1 ? p[j / 2] >> 16 : p[j / 2] & 0xFFFFu);
            } else {
                const float4 v = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(base) + row + e0);
                x[g * E] = v.x;
                x[g * E + 1] = v.y;
                x[g * E + 2] = v.z;
                x[g * E + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < E; ++j) x[g * E + j] = e0 + j < c1 ? logit<BF16>(base, row + e0 + j) : -INFINITY;
        }
    }
    float mx = -INFINITY;
    int mi = -1;
#pragma unroll
    for (int g = 0; g < PER / E; ++g)
#pragma unroll
        for (int j = 0; j < E; ++j)
            if (x[g * E + j] > mx) {
                mx = x[g * E + j];
                mi = c0 + (g * kVThreads + tid) * E + j;
            }
    for (int m = 1; m < 64; m <<= 1) take_max(mx, mi, __shfl_xor(mx, m, 64), __shfl_xor(mi, m, 64));
    __shared__ float smax[kVThreads / 64];
    __shared__ int sidx[kVThreads / 64];
    __shared__ double ssum[kVThreads / 64];
    if ((tid & 63) == 0) {
        smax[tid >> 6] = mx;
        sidx[tid >> 6] = mi;
    }
    __syncthreads();
    mx = smax[0];
    mi = sidx[0];
    for (int v = 1; v < kVThreads / 64; ++v) take_max(mx, mi, smax[v], sidx[v]);
    double sum = 0.0;
    if (it > 0.0) {
        const float ref = mx == -INFINITY ? 0.0f : mx;
        if (kinds == 1 && i < q.n - 1) {
            const int id = a.ids[q.r0 + i];
#pragma unroll
            for (int g = 0; g < PER / E; ++g)
#pragma unroll
                for (int j = 0; j < E; ++j)
                    if (c0 + (g * kVThreads + tid) * E + j == id) x[g * E + j] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) sum += exp_neg(((double)x[j] - (double)ref) * it);
        for (int m = 1; m < 64; m <<= 1) sum += shfl_xor_f64(sum, m);
        if ((tid & 63) == 0) ssum[tid >> 6] = sum;
        __syncthreads();
        sum = ssum[0];
        for (int v = 1; v < kVThreads / 64; ++v) sum += ssum[v];
    }
    if (tid == 0) {
        VPart p;
        p.sum = sum;
        p.max = mx;
        p.idx = mi;
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
    for (int c = lane; c < chunks; c += 64) take_max(r.max, r.idx, p[c].max, p[c].idx);
    for (int m = 1; m < 64; m <<= 1) take_max(r.max, r.idx, __shfl_xor(r.max, m, 64), __shfl_xor(r.idx, m, 64));
    if (it > 0.0 && r.max > -INFINITY && r.max < INFINITY) {
        for (int c = lane; c < chunks; c += 64) {
            const double s = p[c].sum;
            if (p[c].max > -INFINITY || !(s == 0.0)) r.sum += s * exp_neg(((double)p[c].max - (double)r.max) * it);
        }
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

// One workgroup of kDecideThreads: where sequence b stops and how its token is
// drawn.
template <bool BF16>
__device__ __forceinline__ void decide(const VerifyArgs &a, int b, const VSeq &q, double it, int kinds, Decision &d) {
    __shared__ VRow sp[kMaxRows], sq[kMaxRows];
    __shared__ int sstop[kMaxRows];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (int i = wave; i < q.n; i += kDecideThreads / 64) {
        const VPart *p = a.part + ((int64_t)(b * a.max_rows + i) * kinds) * a.chunks;
        VRow rp = join_chunks(p, a.chunks, it, lane);
        VRow rq{0.0, -INFINITY, -1};
        const bool last = i == q.n - 1;
        int stop = 1;
        if (!last) {
            const int64_t row = q.r0 + i;
            const int id = a.ids[row];
            const bool in = id >= 0 && id < a.vocab;
            double wd = 0.0;                          // the draft's term of the sum
            if (in && it > 0.0 && rp.max > -INFINITY && rp.max < INFINITY) {
                wd = exp_neg(((double)logit<BF16>(a.logits, row * a.stride + id) - (double)rp.max) * it);
                if (kinds == 1) rp.sum += wd;
            }
            if (kinds == 2) rq = join_chunks(p + a.chunks, a.chunks, it, lane);
            if (!(it > 0.0) || !rp.finite()) {
                stop = id != max(rp.idx, 0);
            } else if (in) {
                const double pd = wd / rp.sum;
                double qd = 1.0;
                if (kinds == 2 && rq.finite())
                    qd = exp_neg(((double)logit<BF16>(a.draft, row * a.dstride + id) - (double)rq.max) * it) / rq.sum;
                stop = !((double)a.ua[row] * qd < pd);
            }
        }
        if (lane == 0) {
            sp[i] = rp;
            sq[i] = rq;
            sstop[i] = stop;
        }
    }
    __syncthreads();
    int at = 0;
    while (!sstop[at]) ++at;                          // the last row always stops
    const bool last = at == q.n - 1;
    const VRow rp = sp[at], rq = sq[at];
    d.row = at;
    d.draft = last ? -1 : a.ids[q.r0 + at];
    d.best = max(rp.idx, 0);
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

// Weight of token e under the decision.
template <bool BF16>
__device__ __forceinline__ double weight(const VerifyArgs &a, const Decision &d, int mode, int64_t prow, int64_t qrow, int e,
                                         double it) {
    if (mode == kWithout && e == d.draft) return 0.0;
    const double p = exp_neg(((double)logit<BF16>(a.logits, prow + e) - (double)d.pmax) * it);
    if (mode != kRest) return p;
    const double r = p / d.psum - exp_neg(((double)logit<BF16>(a.draft, qrow + e) - (double)d.qmax) * it) / d.qsum;
    return r > 0.0 ? r : 0.0;
}

// Sums per chunk of what is drawn from after a fallen draft (draft logits
// given): max(p - q, 0), or p without the draft where q has no finite sum.
template <bool BF16>
__global__ __launch_bounds__(kDecideThreads) void k_verify_rest(VerifyArgs a) {
    const int chunk = blockIdx.x % a.chunks, b = blockIdx.x / a.chunks;
    const VSeq q = verify_seq(a, b);
    if (q.n == 0) return;
    const double it = inv_temp(a, b);
    Decision d;
    decide<BF16>(a, b, q, it, 2, d);
    if (d.mode != kRest && d.mode != kWithout) return;
    const int64_t row = q.r0 + d.row;
    const int c0 = chunk * a.chunk, c1 = min(c0 + a.chunk, a.vocab);
    double sum = 0.0;
    for (int e = c0 + (int)threadIdx.x; e < c1; e += kDecideThreads)
        sum += weight<BF16>(a, d, d.mode, row * a.stride, row * a.dstride, e, it);
    for (int m = 1; m < 64; m <<= 1) sum += shfl_xor_f64(sum, m);
    __shared__ double ssum[kDecideThreads / 64];
    if ((threadIdx.x & 63) == 0) ssum[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kDecideThreads / 64; ++i) sum += ssum[i];
        a.rest[(int64_t)b * a.chunks + chunk] = sum;
    }
}

// One workgroup per sequence: the decision, the draw, the outputs.
template <bool BF16>
__global__ __launch_bounds__(kDecideThreads) void k_verify_pick(VerifyArgs a, int kinds) {
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
    decide<BF16>(a, b, q, it, kinds, d);
    __shared__ int schunk, stoken;
    __shared__ double starget;
    int token = d.best;
    if (d.mode != kGreedy) {
        const VPart *part = a.part + ((int64_t)(b * a.max_rows + d.row) * kinds) * a.chunks;
        const double *rest = a.rest + (int64_t)b * a.chunks;
        const int64_t prow = (int64_t)(q.r0 + d.row) * a.stride, qrow = (int64_t)(q.r0 + d.row) * a.dstride;
        int mode = d.mode;
        if (wave == 0) {
            // chunk weights, their running sum, and the chunk that passes u * total
            // (outright drafts: the partial sums are already without the draft)
            auto chunk_weight = [&](int c, int m) {
                if (c >= a.chunks) return 0.0;
                if (m == kRest || (m == kWithout && kinds == 2)) return rest[c];
                return part[c].max > -INFINITY ? part[c].sum * exp_neg(((double)part[c].max - (double)d.pmax) * it) : 0.0;
            };
            double total = 0.0;
            for (int c = lane; c < a.chunks; c += 64) total += chunk_weight(c, mode);
            for (int m = 1; m < 64; m <<= 1) total += shfl_xor_f64(total, m);
            if (mode == kRest && !(total > 0.0)) {    // p and q are equal: draw from p
                mode = kFromP;
                total = d.psum;
            }
            const double target = (double)a.us[b] * total;
            double before = 0.0, best_before = 0.0;
            int hit = -1, live = -1;                  // the chunk found; the last one with weight
            double live_before = 0.0;
            for (int c0 = 0; c0 < a.chunks && hit < 0; c0 += 64) {
                const double own = chunk_weight(c0 + lane, mode);
                double run = own;
                for (int s = 1; s < 64; s <<= 1) {
                    const double o = shfl_up_f64(run, s);
                    if (lane >= s) run += o;
                }
                const uint64_t pass = __ballot(before + run > target && own > 0.0), some = __ballot(own > 0.0);
                const double excl = before + run - own;
                auto lane_value = [&](double v, int l) {
                    const uint64_t u = __builtin_bit_cast(uint64_t, v);
                    const uint32_t lo = __shfl((int)(uint32_t)u, l, 64), hi = __shfl((int)(uint32_t)(u >> 32), l, 64);
                    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
                };
                if (pass) {
                    const int l = __builtin_ctzll(pass);
                    hit = c0 + l;
                    best_before = lane_value(excl, l);
                }
                if (some) {
                    const int l = 63 - __builtin_clzll(some);
                    live = c0 + l;
                    live_before = lane_value(excl, l);
                }
                before = lane_value(before + run, 63);
            }
            if (hit < 0) {                            // rounding at the very end
                hit = live;
                best_before = live_before;
            }
            if (lane == 0) {
                schunk = hit;
                starget = target - best_before;
                stoken = mode;
            }
        }
        __syncthreads();
        mode = stoken;
        const int chunk = schunk;
        const double target = starget;
        __syncthreads();
        if (chunk >= 0) {
            // scan of the chunk: contiguous elements per thread
            const int c0 = chunk * a.chunk, c1 = min(c0 + a.chunk, a.vocab);
            const int per = (a.chunk + kDecideThreads - 1) / kDecideThreads;
            const int e0 = c0 + tid * per, e1 = min(e0 + per, c1);
            double own = 0.0;
            int last = -1;
            for (int e = e0; e < e1; ++e) {
                const double v = weight<BF16>(a, d, mode, prow, qrow, e, it);
                own += v;
                if (v > 0.0) last = e;
            }
            double run = own;
            for (int s = 1; s < 64; s <<= 1) {
                const double o = shfl_up_f64(run, s);
                if (lane >= s) run += o;
            }
            __shared__ double wsum[kDecideThreads / 64];
            __shared__ int first_hit, last_live;
            if (lane == 63) wsum[wave] = run;
            if (tid == 0) {
                first_hit = 0x7FFFFFFF;
                last_live = -1;
            }
            __syncthreads();
            double before = run - own;
            for (int i = 0; i < wave; ++i) before += wsum[i];
            if (last >= 0) atomicMax(&last_live, last);
            if (before + own > target && own > 0.0) {
                double s = before;
                for (int e = e0; e < e1; ++e) {
                    const double v = weight<BF16>(a, d, mode, prow, qrow, e, it);
                    s += v;
                    if (v > 0.0 && s > target) {
                        atomicMin(&first_hit, e);
                        break;
                    }
                }
            }
            __syncthreads();
            token = first_hit != 0x7FFFFFFF ? first_hit : (last_live >= 0 ? last_live : d.best);
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
    int per, chunk, chunks;
    size_t part, ws;
};

// Elements a chunk: the largest of 1024..8192 that still gives the device four
// workgroups a CU.
static VerifyPlan verify_plan(int batch, int max_rows, int vocab, bool draft) {
    VerifyPlan p;
    const int64_t rows = (int64_t)batch * max_rows;
    p.per = 32;
    while (p.per > 8 && rows * ((vocab + kVThreads * p.per - 1) / (kVThreads * p.per)) < (int64_t)num_cus() * 4) p.per /= 2;
    p.chunk = kVThreads * p.per;
    p.chunks = (vocab + p.chunk - 1) / p.chunk;
    p.part = (size_t)rows * (draft ? 2 : 1) * p.chunks * sizeof(VPart);
    p.ws = p.part + (draft ? (size_t)batch * p.chunks * sizeof(double) : 0);
    return p;
}

template <bool BF16, int PER>
static void launch_stats(const VerifyArgs &a, int kinds, bool vec, hipStream_t s) {
    const unsigned grid = (unsigned)((int64_t)a.batch * a.max_rows * kinds * a.chunks);
    if (vec)
        hipLaunchKernelGGL((k_verify_stats<BF16, PER, true>), dim3(grid), dim3(kVThreads), 0, s, a, kinds);
    else
        hipLaunchKernelGGL((k_verify_stats<BF16, PER, false>), dim3(grid), dim3(kVThreads), 0, s, a, kinds);
}

template <bool BF16>
static void launch_verify(const VerifyArgs &a, int per, bool draft, bool vec, hipStream_t s) {
    const int kinds = draft ? 2 : 1;
    switch (per) {
        case 8: launch_stats<BF16, 8>(a, kinds, vec, s); break;
        case 16: launch_stats<BF16, 16>(a, kinds, vec, s); break;
        default: launch_stats<BF16, 32>(a, kinds, vec, s); break;
    }
    if (draft)
        hipLaunchKernelGGL((k_verify_rest<BF16>), dim3((unsigned)(a.batch * a.chunks)), dim3(kDecideThreads), 0, s, a);
    hipLaunchKernelGGL((k_verify_pick<BF16>), dim3((unsigned)a.batch), dim3(kDecideThreads), 0, s, a, kinds);
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
    if ((int64_t)batch * max_rows * 2 * p.chunks > 2147483647LL) return fail(NVFP4_ERR_UNSUPPORTED, "%s: grid too large", who);
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
    a.chunk = p.chunk;
    a.chunks = p.chunks;
    a.part = static_cast<VPart *>(workspace);
    a.rest = reinterpret_cast<double *>(static_cast<char *>(workspace) + p.part);
    const bool vec = aligned(logits, 16) && row_stride * el % 16 == 0 &&
                     (!draft_logits || (aligned(draft_logits, 16) && draft_stride * el % 16 == 0));
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (bf16)
        launch_verify<true>(a, p.per, draft_logits != nullptr, vec, s);
    else
        launch_verify<false>(a, p.per, draft_logits != nullptr, vec, s);
    return check_launch(who);
}
