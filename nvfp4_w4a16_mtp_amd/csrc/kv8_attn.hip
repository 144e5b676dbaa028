// kv8_attention: softmax attention over the paged 8-bit cache (definition in
// nvfp4_mtp.h).
//
// For each row (a query head of one token): o = sum_t p_t v_t / sum_t p_t with
// p_t = exp(scale q.k_t - m), one pass over the keys with a running reference m
// and sum (both fp32).  Must read: 2 * head_dim bytes a visible token and kv
// head; must compute: 4 * head_dim flop a visible (row, key) pair.
//
// A workgroup of four wavefronts takes 16 * RT rows of one (sequence, kv head) and
// walks their keys in steps of 128 tokens, with v_mfma_f32_16x16x32_bf16:
//   S^T = K Q^T    A = K (16 tokens), B = Q^T (16 rows); wavefront w computes the
//                  scores of tokens 32 w .. 32 w + 31 for every row;
//   O^T = V^T P^T  A = V^T (16 dims), B = P^T; wavefront w owns a quarter of the
//                  dims for every row, over all 128 tokens.
// So every K and V byte is loaded and converted (E4M3 -> bf16, exact) by one
// wavefront only, straight from memory into matrix operands: K rows as 16
// contiguous bytes a lane (the k order inside a 64-element chunk is permuted the
// same way in Q), V columns as 16 tokens of one dim, contiguous in the
// transposed page.  A 16-token block lies in one page, and the conversion applies
// the page's power-of-two scale for nothing.  Only Q (in operand order), P and the
// row statistics pass through LDS.  A lane's column is a row of queries in both
// products, so rescaling is a per-lane scalar.
//
// The reference m is common to the four wavefronts and moves only when some score
// exceeds it by more than kSlack (2^kSlack in the weights): the usual step needs
// no exchange of maxima, just one barrier for P (double buffered).  Weights up to
// 2^kSlack cost no precision (bf16 and fp32 keep it relative; for range see kLargeV).
// m is a score before scaling and a weight 2^((s - m) scale), so that the row's maximum
// has the weight 1 whatever its size.  (The rounded product m scale subtracted from s scale
// in one fma leaves half an ulp of it in every exponent, 2^7 from 2^31 on: infinite or
// vanishing rows.  It takes one instruction less a score: prompt chunks 374 us, 382 so.)
//
// P is rounded to bf16 (2^-8 relative at most) for the matrix cores, and the row's
// sum is of the rounded values: a row with one large weight comes out exact.  Against
// 64 bits the relative error (root mean square) is 0.0020 to 0.0023, and 0.0017 with
// fp32 weights, which is the result's own rounding; weights in two bf16 parts would
// double the second product.
#include <type_traits>

#include "kv8.hpp"

namespace nvfp4 {

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

constexpr int kStep = 128;        // tokens a step
constexpr float kSlack = 6.0f;

// A sum of up to 2^31 weights of up to 2^kSlack each, times V, stays below 2^128 while
// the pages' exponents are at most 80.  From the first larger one on, a row tile's
// weights and sums are 2^-kLow of what they would be (its averages come out the same;
// terms below 2^-86 may be lost then).
constexpr uint32_t kLargeV = 80 + 127;
constexpr float kLow = 40.0f, kLowFactor = 0x1p-40f;

// x / d for 0 <= x < 2^31 by a multiplication with a host-made reciprocal: with l =
// ceil(log2 d), m = floor(2^32 (2^l - d) / d) + 1 and t the high word of m x, the
// quotient is (t + (x - t) / 2) >> (l - 1).
struct FastDiv {
    uint32_t d, mul, sh;
    __device__ __forceinline__ int div(int x) const {
        if (sh == 0) return x;                        // d = 1
        const uint32_t t = __umulhi(mul, (uint32_t)x);
        return (int)((t + (((uint32_t)x - t) >> 1)) >> (sh - 1));
    }
};
static FastDiv fast_div(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    return FastDiv{d, (uint32_t)(((1ull << 32) * ((1ull << l) - d)) / d + 1), l};
}

struct AttnArgs {
    HeadRows q;
    KV8 c;
    Seqs s;
    float scale;            // |scale| * log2(e), 1 for a scale of 0
    bool negate, zero;      // scale < 0, scale == 0
    int window, sinks;
    uint16_t *out;
    int64_t out_stride;
    FastDiv group;          // q heads per kv head
    int row_tiles;          // row tiles of a sequence at most
    int splits;             // pieces of a row tile's keys (uneven grid)
    int32_t *before;        // [kMaxShared + 1] steps of the sequences before b, for k_attn_join
    float *part;            // partial results, two slots of RT row tiles a workgroup
};

// A value that is the same in every lane, into a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Maximum and sum over the four lane groups (lanes l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float groups_max(float v) {
    u32x2 a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a.x), __uint_as_float(a.y));
    a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(a.x), __uint_as_float(a.y));
}
__device__ __forceinline__ float groups_sum(float v) {
    u32x2 a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a.x) + __uint_as_float(a.y);
    a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(a.x) + __uint_as_float(a.y);
}

// Eight E4M3 codes times a power of two -> an MFMA operand (exact; the
// conversion applies the exponent of its scale operand).
__device__ __forceinline__ bf16x8 bf16x8_of(uint32_t a, uint32_t b, float scale) {
    union {
        bf16x2 h[4];
        bf16x8 v;
    } u;
    u.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false);
    u.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true);
    u.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false);
    u.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true);
    return u.v;
}

// Bit 7 of every byte that is an E4M3 NaN (0x7F or 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
// Those bytes cleared, and those bytes as E4M3 ones (0x38), all others 0.
__device__ __forceinline__ uint32_t without_nan(uint32_t w) {
    const uint32_t n = nan_bytes(w);
    return w & ~((n - (n >> 7)) | n);
}
__device__ __forceinline__ uint32_t nan_ones(uint32_t w) { return (nan_bytes(w) >> 7) * 0x38u; }

// The key range of one row tile as a list of steps: those of the sinks, then
// those from the window's first token on.
struct Keys {
    int end;          // tokens >= end are seen by no row
    int sink_steps, lo_step, count;
    __device__ __forceinline__ int step(int v) const { return v < sink_steps ? v : lo_step + v - sink_steps; }
};
__device__ __forceinline__ Keys key_range(int pos_lo, int pos_hi, int window, int sinks) {
    Keys k;
    k.end = max(pos_hi + 1, 0);
    // (rows at negative positions see nothing; their window could pass 32 bits)
    k.lo_step = window > 0 ? max(max(pos_lo, 0) - window + 1, 0) / kStep : 0;
    const int steps = (k.end + kStep - 1) / kStep;
    k.sink_steps = window > 0 ? min((min(sinks, k.end) + kStep - 1) / kStep, k.lo_step) : 0;
    k.count = k.end > 0 ? k.sink_steps + steps - k.lo_step : 0;
    return k;
}

// Floats of one partial result: 16 rows x D averages (C layout; a sum could pass
// fp32's range), 16 maxima, 16 sums of weights.
template <int D>
constexpr int part_floats() { return 16 * D + 32; }

// Four dims of one row.
__device__ __forceinline__ void store_out(uint16_t *at, f32x4 v) {
    *reinterpret_cast<uint2 *>(at) = make_uint2(f32_to_bf16_bits(v[0]) | (f32_to_bf16_bits(v[1]) << 16),
                                                f32_to_bf16_bits(v[2]) | (f32_to_bf16_bits(v[3]) << 16));
}

// P in LDS: a row of 128 weights and 16 bytes of padding (the 16 lanes of a
// 16-byte read fall on different banks).
constexpr int kPRow = kStep + 8;

template <int D, int RT>
struct Shared {
    uint16_t p[2][16 * RT][kPRow];
    bf16x8 q[RT][D / 64][2][64];       // in operand order: [chunk][half][lane]
    float m[4][16 * RT];
    int flag[2][4];
};

// Steps of sequence b when one row tile holds its rows: at least one if it has
// rows (a row that sees nothing is still written), and kSetup for what a workgroup
// spends before its first step (the loads of ids, Q, K and V in turn).
constexpr int kSetup = 2;
__device__ __forceinline__ int seq_steps(const AttnArgs &a, const Seq &sq) {
    const int rows = min(sq.n, a.s.max_rows) * (int)a.group.d;
    if (rows == 0) return 0;
    const int shift = sq.len - sq.n;
    return max(key_range(shift, shift + a.group.div(rows - 1), a.window, a.sinks).count, 1) + kSetup;
}

constexpr int kMaxShared = 1024;   // sequences of a batch in even shares at most

// Prefix sums of the sequences' steps into before[0 .. batch] (LDS).
__device__ __forceinline__ void count_steps(const AttnArgs &a, int *before, int *waves) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int base = 0;
    if (tid == 0) before[0] = 0;
    for (int b0 = 0; b0 < a.s.batch; b0 += 256) {
        const int b = b0 + tid;
        int run = b < a.s.batch ? seq_steps(a, load_seq(a.s, b, a.c.lp)) : 0;
        const int n = min(a.s.batch - b0, 64);
        for (int d = 1; d < n; d <<= 1) {
            const int o = __shfl_up(run, d, 64);
            if (lane >= d) run += o;
        }
        if (b0 + 64 < a.s.batch) {                    // more than one wavefront's sequences
            if (lane == 63) waves[wave] = run;
            __syncthreads();
            for (int i = 0; i < wave; ++i) run += waves[i];
        }
        if (b < a.s.batch) before[b + 1] = base + run;
        if (b0 + 256 < a.s.batch) {
            base += waves[0] + waves[1] + waves[2] + waves[3];
            __syncthreads();
        }
    }
    __syncthreads();
}

// Pieces in consecutive workgroups first .. first + count - 1; piece k is in slot
// 0 of its workgroup except, perhaps, the first.
struct Pieces {
    int first, count, first_slot;
    __device__ __forceinline__ int at(int k) const { return (first + k) * 2 + (k == 0 ? first_slot : 0); }
};

// Even shares of `total` steps: the first total % shares workgroups have one
// more.
struct Shares {
    int q, rem;
    __device__ __forceinline__ Shares(int total, int grid) {
        const int shares = max(min(grid, total), 1);  // none of them empty
        q = total / shares;
        rem = total - q * shares;
    }
    __device__ __forceinline__ int begin(int i) const { return i * q + min(i, rem); }
    __device__ __forceinline__ int owner(int u) const {
        const int big = rem * (q + 1);
        return u < big ? u / (q + 1) : rem + (u - big) / q;
    }
    // of a pair whose n steps begin at u
    __device__ __forceinline__ Pieces pieces(int u, int n) const {
        const int first = owner(u);
        return Pieces{first, owner(u + n - 1) - first + 1, begin(first) < u ? 1 : 0};
    }
};

// Workgroups a CU holds at once (a wavefront of each on every SIMD): enough loads in
// flight, and no more shares than that.  One row each of 32 sequences, D = 256: 100 us
// with 2, 106 with 3; windowed decode, D = 128: 101 with 2, 92 with 3, 96 with 4.
constexpr int groups_per_cu(int d, int rt) { return rt >= 3 || d >= 192 ? 2 : d == 128 ? 3 : 4; }

// One workgroup: a share of the steps.  EVEN: the steps of all (sequence, kv head)
// pairs in order are cut into equal shares, so that every workgroup reads the same
// number of keys however ragged the batch is (one row tile a sequence).  Else: 16 *
// RT rows of one pair and one of `splits` pieces of their keys.  Where a pair's (a
// row tile's) keys are spread over workgroups, each leaves a partial result in the
// workspace, and k_attn_join adds them up in piece order.  (Joined by the last
// workgroup to arrive instead, through device-scope accesses: 114 against 111 us for
// one row each of 32 sequences, 102 against 80 us with 3 to 6 rows of 16.)
template <int D, int RT, bool EVEN>
__global__ __launch_bounds__(256, D == 128 && RT == 1 ? 4 : groups_per_cu(D, RT)) void k_attn(AttnArgs a) {
    constexpr int C = D / 64, DW = D / 64;            // 64-element chunks; 16-dim tiles of a wavefront
    __shared__ Shared<D, RT> sh;
    __shared__ int before[EVEN ? kMaxShared + 1 : 1], wave_sum[4];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int r = lane & 15, g = lane >> 4;
    const int64_t page_bytes = (int64_t)D << a.c.lp;
    const int pmask = (1 << a.c.lp) - 1;

    int u = 0, u1 = 1;
    Shares share(1, 1);
    if (EVEN) {
        count_steps(a, before, wave_sum);
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i <= a.s.batch; i += 256) a.before[i] = before[i];
        const int total = uniform(before[a.s.batch]) * a.c.heads;
        if ((int)blockIdx.x >= total) return;
        share = Shares(total, gridDim.x);
        u = share.begin(blockIdx.x);
        u1 = share.begin(blockIdx.x + 1);
    }
    do {
    int b, h, rtile, v0, v1, slot;
    Pieces pieces;
    Seq sq;
    if (!EVEN) {
        const int split = blockIdx.x % a.splits;
        int w = blockIdx.x / a.splits;
        rtile = a.row_tiles - 1 - w % a.row_tiles;    // the longest key ranges first
        w /= a.row_tiles;
        h = w % a.c.heads;
        b = w / a.c.heads;
        sq = load_seq(a.s, b, a.c.lp);
        pieces = Pieces{(int)blockIdx.x - split, a.splits, 0};
        slot = 0;
        v0 = split;                                   // the piece; its steps follow below
        v1 = 0;
        u = u1;
    } else {
        int lo = 0, hi = a.s.batch;                   // before[lo] * heads <= u < before[hi] * heads
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (uniform(before[mid]) * a.c.heads <= u) lo = mid; else hi = mid;
        }
        b = lo;
        sq = load_seq(a.s, b, a.c.lp);
        const int steps = uniform(before[b + 1]) - uniform(before[b]), in = u - uniform(before[b]) * a.c.heads;
        h = in / steps;
        rtile = 0;
        v0 = in - h * steps;
        v1 = min(steps, v0 + (u1 - u));
        pieces = share.pieces(u - v0 + kSetup, steps - kSetup);
        u += v1 - v0;
        v0 = max(v0 - kSetup, 0);
        v1 -= kSetup;
        if (v1 <= v0) continue;                       // the setup alone: the next workgroup has the first step
        slot = v0 == 0 ? pieces.first_slot : 0;
    }
    sq = Seq{uniform(sq.r0), uniform(sq.n), uniform(sq.len)};
    const int rows = min(sq.n, a.s.max_rows) * (int)a.group.d, row0 = rtile * 16 * RT;
    if (!EVEN && row0 >= rows) return;
    const int shift = sq.len - sq.n;
    const int pos_lo = shift + a.group.div(row0), pos_hi = shift + a.group.div(min(row0 + 16 * RT, rows) - 1);
    const Keys keys = key_range(pos_lo, pos_hi, a.window, a.sinks);
    if (!EVEN) {
        const int per = (keys.count + a.splits - 1) / a.splits;
        v0 *= per;
        v1 = v0 + per;
    }
    v1 = min(v1, keys.count);
    const int last_page = max(keys.end - 1, 0) >> a.c.lp;
    const int32_t *table = a.s.table + (int64_t)b * a.s.max_pages;

    auto valid = [&](int id) { return id >= 0 && id < a.c.pages; };
    // ids of the pages of the wavefront's two K blocks and of the lane's two V blocks
    struct Ids {
        int k[2], v[2];
    };
    auto load_ids = [&](int step) {
        Ids id;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            id.k[j] = table[min((step * kStep + 32 * wave + 16 * j) >> a.c.lp, last_page)];
            id.v[j] = table[min((step * kStep + 64 * j + 16 * g) >> a.c.lp, last_page)];
        }
        return id;
    };
    uint4 kf[2][C], vf[2][DW];
    uint32_t sk[2], sv[2];
    auto load_k = [&](const Ids &id) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t at = (int64_t)(valid(id.k[j]) ? id.k[j] : 0) * a.c.heads + h;
            const uint8_t *p = a.c.k + at * page_bytes + ((32 * wave + 16 * j) & pmask) * D;
#pragma unroll
            for (int c = 0; c < C; ++c) kf[j][c] = *reinterpret_cast<const uint4 *>(p + r * D + 16 * g + c * 64);
            sk[j] = a.c.ks[at];
        }
    };
    auto load_v = [&](const Ids &id) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t at = (int64_t)(valid(id.v[j]) ? id.v[j] : 0) * a.c.heads + h;
            sv[j] = a.c.vs[at];
            const uint8_t *p = a.c.v + at * page_bytes + ((wave * DW * 16 + r) << a.c.lp) + ((64 * j + 16 * g) & pmask);
#pragma unroll
            for (int dt = 0; dt < DW; ++dt) vf[j][dt] = *reinterpret_cast<const uint4 *>(p + ((dt * 16) << a.c.lp));
        }
    };

    int pos[RT];
    f32x4 o[RT][DW];
    float m[RT], l[RT];
    uint32_t poison[RT];              // bit 4 dt + i: o[rt][dt][i] is NaN
    float low = 0.0f;                 // or kLow
    int step = 0, next = 0;
    Ids id{}, nid{};
    if (v0 < v1) {
        step = keys.step(v0);
        id = load_ids(step);
        next = keys.step(min(v0 + 1, v1 - 1));
        nid = load_ids(next);
    }
    // Q into LDS (each wavefront a part); a scale below zero is its magnitude on the
    // negated q, a scale of zero is any other on q = 0 (what is not finite stays: NaN)
    constexpr int QN = (RT * C * 2 + 3) / 4;
    uint4 qv[QN];
#pragma unroll
    for (int k = 0; k < QN; ++k) {
        const int f = k * 4 + wave, rt = f / (C * 2), ce = f % (C * 2);
        const int row = min(row0 + min(rt, RT - 1) * 16 + r, rows - 1), i = a.group.div(row);
        qv[k] = *reinterpret_cast<const uint4 *>(a.q.data + (int64_t)(sq.r0 + i) * a.q.row +
                                                 (int64_t)(h * (int)a.group.d + row - i * (int)a.group.d) * a.q.head + 16 * g +
                                                 32 * ce - 24 * (ce & 1));
    }
    if (v0 < v1) {
        load_k(id);
        load_v(id);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        pos[rt] = max(shift + a.group.div(min(row0 + rt * 16 + r, rows - 1)), -1);
        m[rt] = -INFINITY;
        l[rt] = 0.0f;
        poison[rt] = 0u;
#pragma unroll
        for (int dt = 0; dt < DW; ++dt) o[rt][dt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    if (EVEN) __syncthreads();                        // the previous piece's reads of sh are over
#pragma unroll
    for (int k = 0; k < QN; ++k) {
        const int f = k * 4 + wave;
        const uint32_t flip = a.negate ? 0x80008000u : 0u;
        auto prepared = [&](uint32_t w) {
            if (a.zero) return ((w & 0x7F80u) == 0x7F80u ? w & 0xFFFFu : 0u) | ((w & 0x7F800000u) == 0x7F800000u ? w & 0xFFFF0000u : 0u);
            return w ^ flip;
        };
        if (f < RT * C * 2)
            (&sh.q[0][0][0][0])[f * 64 + lane] =
                __builtin_bit_cast(bf16x8, make_uint4(prepared(qv[k].x), prepared(qv[k].y), prepared(qv[k].z), prepared(qv[k].w)));
    }
    __syncthreads();

    auto sees = [&](int t, int p) { return (t <= p) & ((a.window == 0) | (t > p - a.window) | (t < a.sinks)); };
    // (wavefront, row tile) maxima of the step's scores
    auto row_max = [&](const f32x4 (&s)[RT][2], int rt) {
        float mx = s[rt][0][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) mx = fmaxf(mx, s[rt][i >> 2][i & 3]);
        return groups_max(mx);
    };
    // Weights of the wavefront's tokens under the present reference into LDS, and
    // their sums as rounded.
    auto write_p = [&](int buf, const f32x4 (&s)[RT][2], float (&sum)[RT]) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const float ref = m[rt] == -INFINITY ? 0.0f : m[rt];
            sum[rt] = 0.0f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                bf16x2 p[2];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    p[i >> 1][i & 1] = static_cast<__bf16>(__builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][j][i] - ref, a.scale, -low)));
                sum[rt] = dot2(p[0], as_bf16x2(0x3F803F80u), sum[rt]);
                sum[rt] = dot2(p[1], as_bf16x2(0x3F803F80u), sum[rt]);
                *reinterpret_cast<uint2 *>(&sh.p[buf][rt * 16 + r][32 * wave + 16 * j + 4 * g]) =
                    make_uint2(__builtin_bit_cast(uint32_t, p[0]), __builtin_bit_cast(uint32_t, p[1]));
            }
        }
    };

    {
        for (int v = v0; v < v1; ++v) {
            const int buf = (v - v0) & 1, cur = step;
            const bool kv_ok = __all(valid(id.k[0]) && valid(id.k[1]) && valid(id.v[0]) && valid(id.v[1]));
            const bool k_ok[2] = {valid(id.k[0]), valid(id.k[1])};
            const float fk[2] = {kv8_scale(sk[0]), kv8_scale(sk[1])};
            f32x4 s[RT][2];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) s[rt][0] = s[rt][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            // Half a chunk at a time: the next half's Q reads and conversions run beside
            // the products of this one (two prompt chunks 400 us with a chunk's reads and
            // conversions before its products, 364 so, both with one instruction less a
            // weight than now; one row each of 32 sequences 100.7 and 97.0).
            bf16x8 kc[2][2], qq[2][RT];
            auto half = [&](int i, bf16x8 (&k)[2]) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 w = kf[j][i >> 1];
                    k[j] = i & 1 ? bf16x8_of(w.z, w.w, fk[j]) : bf16x8_of(w.x, w.y, fk[j]);
                }
            };
            auto read_q = [&](int i, bf16x8 (&q)[RT]) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) q[rt] = sh.q[rt][i >> 1][i & 1][lane];
            };
            constexpr bool kAhead = RT < 4 || !EVEN;  // (else the reads ahead spill: 16 x 8 rows of D = 256, 78 us; 73 so)
            if (kAhead) read_q(0, qq[0]);
            half(0, kc[0]);
#pragma unroll
            for (int i = 0; i < 2 * C; ++i) {
                if (kAhead && i + 1 < 2 * C) read_q(i + 1, qq[(i + 1) & 1]);
                if (!kAhead) read_q(i, qq[i & 1]);
                __builtin_amdgcn_sched_barrier(0);
                if (i + 1 < 2 * C) half(i + 1, kc[(i + 1) & 1]);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    s[rt][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kc[i & 1][0], qq[i & 1][rt], s[rt][0], 0, 0, 0);
                    s[rt][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kc[i & 1][1], qq[i & 1][rt], s[rt][1], 0, 0, 0);
                }
                if (RT < 4) {                         // (one product, then its share of the conversions)
#pragma unroll
                    for (int k = 0; k < 2 * RT; ++k) {
                        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x2, (8 + 2 * RT - 1) / (2 * RT), 0);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            // the next step's K and scales, then the ids after it (past the last
            // step the last one is loaded again)
            step = next;
            const Ids vid = nid;
            load_k(nid);
            next = keys.step(min(v + 2, v1 - 1));
            nid = load_ids(next);
            __builtin_amdgcn_sched_barrier(0);
            const int t0 = cur * kStep;
            const bool whole = kv_ok && t0 + kStep - 1 <= pos_lo &&
                               (a.window == 0 || t0 > pos_hi - a.window || t0 + kStep <= a.sinks);
            bool need = false;
            float mx[RT], sum[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                if (!whole) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            s[rt][j][i] = k_ok[j] & sees(t0 + 32 * wave + 16 * j + 4 * g + i, pos[rt]) ? s[rt][j][i] : -INFINITY;
                }
                mx[rt] = row_max(s, rt);
                need |= (mx[rt] - m[rt]) * a.scale > kSlack;
            }
            bool move = v == v0;                      // no reference yet
            if (!move) {
                need = __any(need);
                write_p(buf, s, sum);
                if (lane == 0) sh.flag[buf][wave] = need;
                __syncthreads();
                move = sh.flag[buf][0] | sh.flag[buf][1] | sh.flag[buf][2] | sh.flag[buf][3];
            }
            if (move) {
                // move the reference to the present maximum, in every wavefront alike
                if (lane < 16)
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) sh.m[wave][rt * 16 + r] = mx[rt];
                __syncthreads();
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    float mn = m[rt];
#pragma unroll
                    for (int k = 0; k < 4; ++k) mn = fmaxf(mn, sh.m[k][rt * 16 + r]);
                    const float alpha = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m[rt] - mn) * a.scale);
                    l[rt] *= alpha;
#pragma unroll
                    for (int dt = 0; dt < DW; ++dt) o[rt][dt] *= alpha;
                    m[rt] = mn;
                }
                write_p(buf, s, sum);
                __syncthreads();
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) l[rt] += sum[rt];
            const float fv[2] = {kv8_scale(sv[0]), kv8_scale(sv[1])};
            // (every wavefront has all of the step's scales of V)
            if (low == 0.0f && __any(max(sv[0], sv[1]) > kLargeV)) {
                low = kLow;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    l[rt] *= kLowFactor;
#pragma unroll
                    for (int dt = 0; dt < DW; ++dt) o[rt][dt] *= kLowFactor;
                }
                // and the wavefront's weights of this step
#pragma unroll 1
                for (int k = 0; k < 2 * RT; ++k) {
                    uint16_t *p = &sh.p[buf][(k >> 1) * 16 + r][32 * wave + 16 * (k & 1) + 4 * g];
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = (uint16_t)f32_to_bf16_bits(bf16_bits_to_f32(p[i]) * kLowFactor);
                }
                __syncthreads();
            }
            if (!whole) {
                // A token that some row does not see may hold a NaN in V that the row
                // must not get (0 * NaN is NaN): such codes are counted per (dim, row)
                // over the tokens the row sees, and left out of the product.
                uint32_t any = 0;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int dt = 0; dt < DW; ++dt)
                        any |= nan_bytes(vf[j][dt].x) | nan_bytes(vf[j][dt].y) | nan_bytes(vf[j][dt].z) | nan_bytes(vf[j][dt].w);
                if (__any(any != 0)) {
                    // a rare path, kept small: the codes are read again, eight tokens
                    // of 16 dims at a time
#pragma unroll 1
                    for (int k = 0; k < DW * 4; ++k) {
                        const int dt = k >> 2, at = 64 * (k >> 1 & 1) + 16 * g, e8 = 8 * (k & 1);
                        const int page = k & 2 ? id.v[1] : id.v[0];
                        const bool ok = valid(page);
                        const uint2 c = *reinterpret_cast<const uint2 *>(
                            a.c.v + ((int64_t)(ok ? page : 0) * a.c.heads + h) * page_bytes +
                            (((wave * DW + dt) * 16 + r) << a.c.lp) + (at & pmask) + e8);
                        const bf16x8 ones = bf16x8_of(nan_ones(c.x), nan_ones(c.y), 1.0f);
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) {
                            union {
                                uint32_t w[4];
                                bf16x8 v;
                            } u;
#pragma unroll
                            for (int i = 0; i < 8; i += 2) {
                                const int t = t0 + at + e8 + i;
                                u.w[i / 2] = (ok & sees(t, pos[rt]) ? 0x3F80u : 0u) | (ok & sees(t + 1, pos[rt]) ? 0x3F800000u : 0u);
                            }
                            const f32x4 n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, u.v, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
                            for (int i = 0; i < 4; ++i) poison[rt] |= n[i] > 0.0f ? 1u << (4 * dt + i) : 0u;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int dt = 0; dt < DW; ++dt)
                            vf[j][dt] = make_uint4(without_nan(vf[j][dt].x), without_nan(vf[j][dt].y), without_nan(vf[j][dt].z),
                                                   without_nan(vf[j][dt].w));
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    bf16x8 pv[RT];
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
                        pv[rt] = *reinterpret_cast<const bf16x8 *>(&sh.p[buf][rt * 16 + r][64 * j + 16 * g + 8 * e]);
#pragma unroll
                    for (int dt = 0; dt < DW; ++dt) {
                        const bf16x8 vv = e ? bf16x8_of(vf[j][dt].z, vf[j][dt].w, fv[j]) : bf16x8_of(vf[j][dt].x, vf[j][dt].y, fv[j]);
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
                            o[rt][dt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vv, pv[rt], o[rt][dt], 0, 0, 0);
                    }
                }
            id = vid;
            load_v(id);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // the rows' sums over the wavefronts; each wavefront holds its dims whole
    __syncthreads();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const float lw = groups_sum(l[rt]);
        if (lane < 16) sh.m[wave][rt * 16 + r] = lw;
    }
    __syncthreads();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        l[rt] = (sh.m[0][rt * 16 + r] + sh.m[1][rt * 16 + r]) + (sh.m[2][rt * 16 + r] + sh.m[3][rt * 16 + r]);
#pragma unroll
        for (int dt = 0; dt < DW; ++dt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (poison[rt] >> (4 * dt + i) & 1u) o[rt][dt][i] = NAN;
    }
    auto part_at = [&](int at, int rt) { return a.part + ((int64_t)at * RT + rt) * part_floats<D>(); };
    if (pieces.count > 1) {                           // k_attn_join does the rest
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            if (row0 + rt * 16 + r >= rows) continue;
            float *p = part_at(blockIdx.x * 2 + slot, rt);
            const float inv = l[rt] == 0.0f ? 0.0f : 1.0f / l[rt];
#pragma unroll
            for (int dt = 0; dt < DW; ++dt) *reinterpret_cast<f32x4 *>(p + (wave * DW + dt) * 256 + lane * 4) = o[rt][dt] * inv;
            if (threadIdx.x < 16)
                *reinterpret_cast<float2 *>(p + 16 * D + 2 * r) = make_float2(m[rt], low == 0.0f ? l[rt] : l[rt] * (1.0f / kLowFactor));
        }
        continue;
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int row = row0 + rt * 16 + r, i = a.group.div(min(row, rows - 1)), hq = h * (int)a.group.d + row - i * (int)a.group.d;
        const float inv = l[rt] == 0.0f ? 0.0f : 1.0f / l[rt];
        if (row < rows) {
            uint16_t *dst = a.out + (int64_t)(sq.r0 + i) * a.out_stride + (int64_t)hq * D + wave * DW * 16 + 4 * g;
#pragma unroll
            for (int dt = 0; dt < DW; ++dt) store_out(dst + dt * 16, o[rt][dt] * inv);
        }
    }
    } while (EVEN && u < u1);
}

// Joins the pieces of 16 rows: one wavefront per 16 dims.
template <int D, int RT, bool EVEN>
__global__ __launch_bounds__(64) void k_attn_join(AttnArgs a, int grid) {
    const int dt = blockIdx.x % (D / 16), lane = threadIdx.x, r = lane & 15;
    const int w = blockIdx.x / (D / 16), rt = w % RT, tile = w / RT;
    const int unit = tile / a.row_tiles, h = unit % a.c.heads, b = unit / a.c.heads;
    const Seq sq = load_seq(a.s, b, a.c.lp);
    Pieces pieces{tile * a.splits, a.splits, 0};
    if (EVEN) {
        const int b0 = a.before[b], steps = a.before[b + 1] - b0, total = a.before[a.s.batch] * a.c.heads;
        if (steps == 0) return;
        pieces = Shares(total, grid).pieces(b0 * a.c.heads + h * steps + kSetup, steps - kSetup);
        if (pieces.count == 1) return;                // written by its workgroup
    }
    const int rows = min(sq.n, a.s.max_rows) * (int)a.group.d;
    const int row = ((a.row_tiles - 1 - tile % a.row_tiles) * RT + rt) * 16 + r;
    if (row >= rows) return;
    float mx = -INFINITY, sum = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    // n pieces at a time, their loads in flight together; o stays an average
    auto add = [&](auto n) {
        constexpr int N = decltype(n)::value;
        for (int k0 = 0; k0 < pieces.count; k0 += N) {
            float2 ml[N];
            f32x4 v[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float *p = a.part + ((int64_t)pieces.at(min(k0 + k, pieces.count - 1)) * RT + rt) * part_floats<D>();
                ml[k] = *reinterpret_cast<const float2 *>(p + 16 * D + 2 * r);
                v[k] = *reinterpret_cast<const f32x4 *>(p + dt * 256 + lane * 4);
            }
            __builtin_amdgcn_sched_barrier(0);
            float mn = mx;
#pragma unroll
            for (int k = 0; k < N; ++k) mn = fmaxf(mn, ml[k].x);
            const float ref = mn == -INFINITY ? 0.0f : mn, old = sum * __builtin_amdgcn_exp2f((mx - ref) * a.scale);
            sum = old;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                ml[k].y = k0 + k < pieces.count ? ml[k].y * __builtin_amdgcn_exp2f((ml[k].x - ref) * a.scale) : 0.0f;
                sum += ml[k].y;
            }
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            o *= old * inv;
#pragma unroll
            for (int k = 0; k < N; ++k) o += v[k] * (ml[k].y * inv);
            mx = mn;
        }
    };
    // (one token over 1500 keys, 12 pieces: 12.6 us eight at a time, 11.9 sixteen; a
    // windowed batch, two or three pieces: 91.7 and 93.0)
    if (pieces.count <= 4)
        add(std::integral_constant<int, 4>{});
    else
        add(std::integral_constant<int, 16>{});
    const int i = a.group.div(row), hq = h * (int)a.group.d + row - i * (int)a.group.d;
    store_out(a.out + (int64_t)(sq.r0 + i) * a.out_stride + (int64_t)hq * D + dt * 16 + 4 * (lane >> 4),
              o);
}

struct AttnPlan {
    int rt, row_tiles, splits;
    bool even;
    int64_t blocks, join_blocks;
    size_t ws;
};

constexpr size_t kHeader = 4352;                   // before
static_assert((kMaxShared + 1) * sizeof(int32_t) <= kHeader, "before fits its place");

template <int D>
static const void *attn_kernel(int rt, bool even) {
    if (even)
        return rt == 1 ? reinterpret_cast<const void *>(k_attn<D, 1, true>)
                       : rt == 2 ? reinterpret_cast<const void *>(k_attn<D, 2, true>) : rt == 3 ? reinterpret_cast<const void *>(k_attn<D, 3, true>) : reinterpret_cast<const void *>(k_attn<D, 4, true>);
    return rt == 1 ? reinterpret_cast<const void *>(k_attn<D, 1, false>)
                   : rt == 2 ? reinterpret_cast<const void *>(k_attn<D, 2, false>) : rt == 3 ? reinterpret_cast<const void *>(k_attn<D, 3, false>) : reinterpret_cast<const void *>(k_attn<D, 4, false>);
}
static const void *attn_kernel(int dim, int rt, bool even) {
    return dim == 64 ? attn_kernel<64>(rt, even)
                     : dim == 128 ? attn_kernel<128>(rt, even) : dim == 192 ? attn_kernel<192>(rt, even) : attn_kernel<256>(rt, even);
}

static AttnPlan attn_plan(const nvfp4_kv8_cache *c, const nvfp4_kv8_seqs *s, int q_heads) {
    AttnPlan p{};
    const int max_rows = s->max_rows < s->rows ? s->max_rows : s->rows;
    const int64_t rows = (int64_t)max_rows * (q_heads / c->kv_heads);
    p.rt = rows <= 16 ? 1 : rows <= 32 ? 2 : rows <= 48 ? 3 : 4;
    p.row_tiles = (int)((rows + 16 * p.rt - 1) / (16 * p.rt));
    const int64_t units = (int64_t)s->batch * c->kv_heads * p.row_tiles;
    const int64_t cap = (int64_t)s->max_pages * c->page_tokens;
    const int64_t len = s->max_kv_len > 0 && s->max_kv_len < cap ? s->max_kv_len : cap;
    const int64_t steps = (len + kStep - 1) / kStep;
    // even shares keep the step count in 32 bits
    p.even = p.row_tiles == 1 && s->batch <= kMaxShared && units * ((cap + kStep - 1) / kStep + 1 + kSetup) < (1LL << 30);
    const int fit = blocks_per_cu(attn_kernel(c->head_dim, p.rt, p.even), 256, 0), want_cu = groups_per_cu(c->head_dim, p.rt);
    const int64_t slots = (int64_t)num_cus() * (fit < want_cu ? fit : want_cu);
    p.splits = 1;
    bool pieces;
    if (p.even) {
        // one workgroup a slot of the device, or a step
        p.blocks = slots < units * (steps + kSetup) ? slots : units * (steps + kSetup);
        pieces = true;
    } else {
        int64_t want = units < slots ? (slots + units - 1) / units : 1;   // less than 2 * slots workgroups
        want = want < steps ? want : steps;
        p.splits = (int)(want < 1 ? 1 : want);
        p.blocks = units * p.splits;
        pieces = p.splits > 1;
    }
    p.join_blocks = pieces ? units * p.rt * (c->head_dim / 16) : 0;
    p.ws = kHeader + (pieces ? (size_t)(p.blocks * 2 * p.rt) * (16 * c->head_dim + 32) * sizeof(float) : 0);
    return p;
}

template <int D, int RT, bool EVEN>
static void launch_attn(const AttnPlan &p, const AttnArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((k_attn<D, RT, EVEN>), dim3((unsigned)p.blocks), dim3(256), 0, s, a);
    if (p.join_blocks > 0)
        hipLaunchKernelGGL((k_attn_join<D, RT, EVEN>), dim3((unsigned)p.join_blocks), dim3(64), 0, s, a, (int)p.blocks);
}
template <int D>
static void launch_attn(const AttnPlan &p, const AttnArgs &a, hipStream_t s) {
    if (p.even) {
        if (p.rt == 1) launch_attn<D, 1, true>(p, a, s);
        else if (p.rt == 2) launch_attn<D, 2, true>(p, a, s);
        else if (p.rt == 3) launch_attn<D, 3, true>(p, a, s);
        else launch_attn<D, 4, true>(p, a, s);
    } else {
        if (p.rt == 1) launch_attn<D, 1, false>(p, a, s);
        else if (p.rt == 2) launch_attn<D, 2, false>(p, a, s);
        else if (p.rt == 3) launch_attn<D, 3, false>(p, a, s);
        else launch_attn<D, 4, false>(p, a, s);
    }
}

}  // namespace nvfp4

using namespace nvfp4;

static int attn_check(const nvfp4_kv8_cache *cache, const nvfp4_kv8_seqs *seqs, int q_heads, const char *who) {
    if (int rc = validate_kv8_cache(cache, who)) return rc;
    if (int rc = validate_kv8_seqs(seqs, who)) return rc;
    if (q_heads < 1 || q_heads % cache->kv_heads)
        return fail(NVFP4_ERR_SHAPE, "%s: q_heads=%d is not a multiple of kv_heads=%d", who, q_heads, cache->kv_heads);
    return NVFP4_OK;
}

extern "C" size_t kv8_attention_workspace_bytes(const nvfp4_kv8_cache *cache, const nvfp4_kv8_seqs *seqs, int32_t q_heads) {
    if (attn_check(cache, seqs, q_heads, "kv8_attention_workspace_bytes")) return 0;
    if (seqs->batch == 0 || seqs->rows == 0) return kHeader;
    return attn_plan(cache, seqs, q_heads).ws;
}

extern "C" int kv8_attention(const nvfp4_head_rows *q, const nvfp4_kv8_cache *cache, const nvfp4_kv8_seqs *seqs, float scale,
                             int32_t window, int32_t sinks, uint16_t *out, int64_t out_row_stride, void *workspace,
                             size_t ws_bytes, void *stream) {
    const char *who = "kv8_attention";
    if (int rc = validate_kv8_cache(cache, who)) return rc;
    if (int rc = validate_kv8_seqs(seqs, who)) return rc;
    if (seqs->batch == 0 || seqs->rows == 0) return ok();
    if (int rc = validate_head_rows(q, who, "q")) return rc;
    if (int rc = attn_check(cache, seqs, q->heads, who)) return rc;
    if (q->dim != cache->head_dim) return fail(NVFP4_ERR_SHAPE, "%s: q has dim %d, the cache %d", who, q->dim, cache->head_dim);
    if (window < 0 || sinks < 0) return fail(NVFP4_ERR_ARG, "%s: window=%d or sinks=%d < 0", who, window, sinks);
    const float scale2 = __builtin_fabsf(scale) * 1.44269504088896340736f;   // for 2^x
    if (!__builtin_isfinite(scale2)) return fail(NVFP4_ERR_ARG, "%s: scale * log2(e) is not finite", who);
    if (!out) return fail(NVFP4_ERR_ARG, "%s: NULL out", who);
    if (!aligned(out, 16)) return fail(NVFP4_ERR_ALIGN, "%s: out not 16-byte aligned", who);
    if (out_row_stride % 8 || out_row_stride < (int64_t)q->heads * q->dim)
        return fail(NVFP4_ERR_SHAPE, "%s: out_row_stride=%lld must be a multiple of 8 and >= q_heads * head_dim", who,
                    (long long)out_row_stride);
    if ((int64_t)seqs->max_rows * (q->heads / cache->kv_heads) >= (1LL << 30))
        return fail(NVFP4_ERR_UNSUPPORTED, "%s: max_rows=%d rows of %d query heads a kv head are too many", who, seqs->max_rows,
                    q->heads / cache->kv_heads);
    const AttnPlan p = attn_plan(cache, seqs, q->heads);
    if (!grid_fits(p.blocks, 256) || !grid_fits(p.join_blocks, 64)) return fail(NVFP4_ERR_UNSUPPORTED, "%s: grid too large", who);
    if (!workspace || ws_bytes < p.ws)
        return fail(NVFP4_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", who, workspace ? ws_bytes : 0, p.ws);
    if (!aligned(workspace, 256)) return fail(NVFP4_ERR_ALIGN, "%s: workspace not 256-byte aligned", who);
    AttnArgs a;
    a.q = view(q);
    a.c = view(cache);
    a.s = view(seqs);
    // (a hidden token's score of -inf times a scale of 0 would be NaN)
    a.scale = scale == 0.0f ? 1.0f : scale2;
    a.negate = scale < 0.0f;
    a.zero = scale == 0.0f;
    a.window = window;
    a.sinks = sinks;
    a.out = out;
    a.out_stride = out_row_stride;
    a.group = fast_div((uint32_t)(q->heads / cache->kv_heads));
    a.row_tiles = p.row_tiles;
    a.splits = p.splits;
    a.before = static_cast<int32_t *>(workspace);
    a.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + kHeader);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    switch (cache->head_dim) {
        case 64: launch_attn<64>(p, a, s); break;
        case 128: launch_attn<128>(p, a, s); break;
        case 192: launch_attn<192>(p, a, s); break;
        default: launch_attn<256>(p, a, s); break;
    }
    return check_launch(who);
}
