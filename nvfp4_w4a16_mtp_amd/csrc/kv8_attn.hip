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
// 2^kSlack cost nothing: bf16 and fp32 keep their relative precision.
//
// P is rounded to bf16 (2^-8 relative at most) for the matrix cores, and the row's
// sum is of the rounded values: a row with one large weight comes out exact.
#include "kv8.hpp"

namespace nvfp4 {

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

constexpr int kStep = 128;        // tokens a step
constexpr float kSlack = 6.0f;

struct AttnArgs {
    HeadRows q;
    KV8 c;
    Seqs s;
    float scale;            // |scale| * log2(e)
    bool negate;            // scale < 0
    int window, sinks;
    uint16_t *out;
    int64_t out_stride;
    int group;              // q heads per kv head
    int row_tiles;          // row tiles of a sequence at most
    int splits;             // pieces of the key range
    float *part;            // partial results (splits > 1)
};

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

// The same value, computed anew where it is used.
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

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
    k.lo_step = window > 0 ? max(pos_lo - window + 1, 0) / kStep : 0;
    const int steps = (k.end + kStep - 1) / kStep;
    k.sink_steps = window > 0 ? min((min(sinks, k.end) + kStep - 1) / kStep, k.lo_step) : 0;
    k.count = k.end > 0 ? k.sink_steps + steps - k.lo_step : 0;
    return k;
}

// Floats of one partial result: 16 rows x D sums (C layout), 16 maxima, 16 sums.
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

// One workgroup: 16 * RT rows of one (sequence, kv head), one piece of their
// keys.
template <int D, int RT>
__global__ __launch_bounds__(256, (RT == 4 ? 2 : D * RT <= 256 ? 4 - (D * RT > 128) : 2)) void k_attn(AttnArgs a) {
    constexpr int C = D / 64, DW = D / 64;            // 64-element chunks; 16-dim tiles of a wavefront
    __shared__ Shared<D, RT> sh;
    const int split = blockIdx.x % a.splits;
    int w = blockIdx.x / a.splits;
    const int rtile = a.row_tiles - 1 - w % a.row_tiles;   // the longest key ranges first
    w /= a.row_tiles;
    const int h = w % a.c.heads, b = w / a.c.heads;
    const Seq sq = load_seq(a.s, b, a.c.lp);
    const int rows = min(sq.n, a.s.max_rows) * a.group, row0 = rtile * 16 * RT;
    if (row0 >= rows) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int r = lane & 15, g = lane >> 4;
    const int shift = sq.len - sq.n;
    const int pos_lo = shift + row0 / a.group, pos_hi = shift + (min(row0 + 16 * RT, rows) - 1) / a.group;
    const Keys keys = key_range(pos_lo, pos_hi, a.window, a.sinks);
    const int last_page = max(keys.end - 1, 0) >> a.c.lp;
    const int per = (keys.count + a.splits - 1) / a.splits;
    const int v0 = split * per, v1 = min(v0 + per, keys.count);
    const int32_t *table = a.s.table + (int64_t)b * a.s.max_pages;
    const int64_t page_bytes = (int64_t)D << a.c.lp;
    const int pmask = (1 << a.c.lp) - 1;

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
    auto load_k = [&](int step, const Ids &id) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t at = (int64_t)(valid(id.k[j]) ? id.k[j] : 0) * a.c.heads + h;
            const uint8_t *p = a.c.k + at * page_bytes + (((32 * wave + 16 * j) & pmask) + r) * D + 16 * g;
#pragma unroll
            for (int c = 0; c < C; ++c) kf[j][c] = *reinterpret_cast<const uint4 *>(p + c * 64);
            sk[j] = a.c.ks[at];
        }
    };
    auto load_v = [&](int step, const Ids &id) {
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
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int row = min(row0 + rt * 16 + r, rows - 1);
        const int i = row / a.group;
        pos[rt] = shift + i;
        m[rt] = -INFINITY;
        l[rt] = 0.0f;
        poison[rt] = 0u;
        const uint16_t *src = a.q.data + (int64_t)(sq.r0 + i) * a.q.row + (int64_t)(h * a.group + row % a.group) * a.q.head + 16 * g;
        // a scale below zero is its magnitude on the negated q
        const uint32_t flip = a.negate ? 0x80008000u : 0u;
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (((rt * C + c) & 3) == wave)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint4 v = *reinterpret_cast<const uint4 *>(src + 64 * c + 8 * e);
                    v.x ^= flip;
                    v.y ^= flip;
                    v.z ^= flip;
                    v.w ^= flip;
                    sh.q[rt][c][e][lane] = __builtin_bit_cast(bf16x8, v);
                }
#pragma unroll
        for (int dt = 0; dt < DW; ++dt) o[rt][dt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __syncthreads();

    auto sees = [&](int t, int p) { return t <= p && (a.window == 0 || t > p - a.window || t < a.sinks); };
    // (wavefront, row tile) maxima of the step's scores
    auto row_max = [&](const f32x4 (&s)[RT][2], int rt) {
        float mx = s[rt][0][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) mx = fmaxf(mx, s[rt][i >> 2][i & 3]);
        return groups_max(mx) * a.scale;
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
                    p[i >> 1][i & 1] = static_cast<__bf16>(__builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][j][i], a.scale, -ref)));
                sum[rt] = dot2(p[0], as_bf16x2(0x3F803F80u), sum[rt]);
                sum[rt] = dot2(p[1], as_bf16x2(0x3F803F80u), sum[rt]);
                *reinterpret_cast<uint2 *>(&sh.p[buf][rt * 16 + r][32 * wave + 16 * j + 4 * g]) =
                    make_uint2(__builtin_bit_cast(uint32_t, p[0]), __builtin_bit_cast(uint32_t, p[1]));
            }
        }
    };

    if (v0 < v1) {
        int step = keys.step(v0);
        Ids id = load_ids(step);
        load_k(step, id);
        load_v(step, id);
        int next = keys.step(min(v0 + 1, v1 - 1));
        Ids nid = load_ids(next);
        for (int v = v0; v < v1; ++v) {
            const int buf = (v - v0) & 1, cur = step;
            const bool kv_ok = __all(valid(id.k[0]) && valid(id.k[1]) && valid(id.v[0]) && valid(id.v[1]));
            const bool k_ok[2] = {valid(id.k[0]), valid(id.k[1])}, v_ok[2] = {valid(id.v[0]), valid(id.v[1])};
            const float fk[2] = {kv8_scale(sk[0]), kv8_scale(sk[1])};
            f32x4 s[RT][2];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) s[rt][0] = s[rt][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const bf16x8 k0[2] = {bf16x8_of(kf[0][c].x, kf[0][c].y, fk[0]), bf16x8_of(kf[0][c].z, kf[0][c].w, fk[0])};
                const bf16x8 k1[2] = {bf16x8_of(kf[1][c].x, kf[1][c].y, fk[1]), bf16x8_of(kf[1][c].z, kf[1][c].w, fk[1])};
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const bf16x8 qq = sh.q[rt][c][e][lane];
                        s[rt][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0[e], qq, s[rt][0], 0, 0, 0);
                        s[rt][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1[e], qq, s[rt][1], 0, 0, 0);
                    }
                __builtin_amdgcn_sched_barrier(0);
            }
            // the next step's K and scales, then the ids after it (past the last
            // step the last one is loaded again)
            step = next;
            const Ids vid = nid;
            load_k(step, nid);
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
                            if (!(k_ok[j] && sees(t0 + 32 * wave + 16 * j + 4 * g + i, pos[rt]))) s[rt][j][i] = -INFINITY;
                }
                mx[rt] = row_max(s, rt);
                need |= mx[rt] > m[rt] + kSlack;
            }
            need = __any(need);
            write_p(buf, s, sum);
            if (lane == 0) sh.flag[buf][wave] = need;
            __syncthreads();
            if (sh.flag[buf][0] | sh.flag[buf][1] | sh.flag[buf][2] | sh.flag[buf][3]) {
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
                    const float alpha = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[rt] - mn);
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
                    // a rare path: opaque() keeps its values from being computed ahead, or
                    // kept, for all tiles, which cost the loop 80 registers
#pragma unroll
                    for (int dt = 0; dt < DW; ++dt)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                uint32_t &lo = e ? vf[j][dt].z : vf[j][dt].x, &hi = e ? vf[j][dt].w : vf[j][dt].y;
                                lo = opaque(lo);
                                hi = opaque(hi);
                                const bf16x8 ones = bf16x8_of(nan_ones(lo), nan_ones(hi), 1.0f);
                                lo = opaque(without_nan(lo));
                                hi = opaque(without_nan(hi));
#pragma unroll
                                for (int rt = 0; rt < RT; ++rt) {
                                    const int t = (int)opaque(t0 + 64 * j + 16 * g + 8 * e);
                                    union {
                                        uint32_t w[4];
                                        bf16x8 v;
                                    } u;
#pragma unroll
                                    for (int i = 0; i < 8; i += 2)
                                        u.w[i / 2] = (v_ok[j] && sees(t + i, pos[rt]) ? 0x3F80u : 0u) |
                                                     (v_ok[j] && sees(t + i + 1, pos[rt]) ? 0x3F800000u : 0u);
                                    const f32x4 n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, u.v, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
                                    for (int i = 0; i < 4; ++i) poison[rt] |= n[i] > 0.0f ? 1u << (4 * dt + i) : 0u;
                                    poison[rt] = opaque(poison[rt]);
                                }
                            }
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
            load_v(step, id);
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
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) sum += sh.m[k][rt * 16 + r];
#pragma unroll
        for (int dt = 0; dt < DW; ++dt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (poison[rt] >> (4 * dt + i) & 1u) o[rt][dt][i] = NAN;
        if (a.splits > 1) {
            float *part = a.part + (((((int64_t)b * a.c.heads + h) * a.row_tiles + rtile) * RT + rt) * a.splits + split) * part_floats<D>();
#pragma unroll
            for (int dt = 0; dt < DW; ++dt) *reinterpret_cast<f32x4 *>(part + (wave * DW + dt) * 256 + lane * 4) = o[rt][dt];
            if (threadIdx.x < 16) {
                part[16 * D + r] = m[rt];
                part[16 * D + 16 + r] = sum;
            }
        } else {
            const int row = row0 + rt * 16 + r, i = row / a.group, hq = h * a.group + row % a.group;
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            if (row < rows) {
                uint16_t *dst = a.out + (int64_t)(sq.r0 + i) * a.out_stride + (int64_t)hq * D + wave * DW * 16 + 4 * g;
#pragma unroll
                for (int dt = 0; dt < DW; ++dt) store_out(dst + dt * 16, o[rt][dt] * inv);
            }
        }
    }
}

// Joins the pieces of 16 rows: one wavefront per 16 dims.
template <int D>
__global__ __launch_bounds__(64) void k_attn_join(AttnArgs a, int sub_tiles) {
    const int dt = blockIdx.x % (D / 16), lane = threadIdx.x, r = lane & 15;
    int w = blockIdx.x / (D / 16);
    const int st = w % sub_tiles;
    const int unit = w / sub_tiles, h = unit % a.c.heads, b = unit / a.c.heads;
    const Seq sq = load_seq(a.s, b, a.c.lp);
    const int rows = min(sq.n, a.s.max_rows) * a.group;
    if (st * 16 >= rows) return;
    const float *part = a.part + (int64_t)w * a.splits * part_floats<D>();
    float mx = -INFINITY;
    for (int s = 0; s < a.splits; ++s) mx = fmaxf(mx, part[(int64_t)s * part_floats<D>() + 16 * D + r]);
    const float ref = mx == -INFINITY ? 0.0f : mx;
    float sum = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < a.splits; ++s) {
        const float *p = part + (int64_t)s * part_floats<D>();
        const float f = __builtin_amdgcn_exp2f(p[16 * D + r] - ref);
        sum += p[16 * D + 16 + r] * f;
        o += *reinterpret_cast<const f32x4 *>(p + dt * 256 + lane * 4) * f;
    }
    const int row = st * 16 + r;
    if (row >= rows) return;
    const int i = row / a.group, hq = h * a.group + row % a.group;
    store_out(a.out + (int64_t)(sq.r0 + i) * a.out_stride + (int64_t)hq * D + dt * 16 + 4 * (lane >> 4),
              o * (sum == 0.0f ? 0.0f : 1.0f / sum));
}

struct AttnPlan {
    int rt, row_tiles, splits;
    int64_t blocks;
    size_t ws;
};

static AttnPlan attn_plan(const nvfp4_kv8_cache *c, const nvfp4_kv8_seqs *s, int q_heads) {
    AttnPlan p{};
    const int max_rows = s->max_rows < s->rows ? s->max_rows : s->rows;
    const int64_t rows = (int64_t)max_rows * (q_heads / c->kv_heads);
    p.rt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    p.row_tiles = (int)((rows + 16 * p.rt - 1) / (16 * p.rt));
    const int64_t units = (int64_t)s->batch * c->kv_heads * p.row_tiles;
    const int64_t cap = (int64_t)s->max_pages * c->page_tokens;
    const int64_t len = s->max_kv_len > 0 && s->max_kv_len < cap ? s->max_kv_len : cap;
    const int64_t steps = (len + kStep - 1) / kStep;
    int64_t want = ((int64_t)num_cus() * (p.rt == 1 ? 4 : 2) + units - 1) / units;
    want = want < steps ? want : steps;
    p.splits = (int)(want < 1 ? 1 : want);
    p.blocks = units * p.splits;
    p.ws = p.splits > 1 ? (size_t)(units * p.rt * p.splits) * (16 * c->head_dim + 32) * sizeof(float) : 0;
    return p;
}

template <int D>
static void launch_attn(const AttnPlan &p, const AttnArgs &a, int batch, hipStream_t s) {
    if (p.rt == 1)
        hipLaunchKernelGGL((k_attn<D, 1>), dim3((unsigned)p.blocks), dim3(256), 0, s, a);
    else if (p.rt == 2)
        hipLaunchKernelGGL((k_attn<D, 2>), dim3((unsigned)p.blocks), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((k_attn<D, 4>), dim3((unsigned)p.blocks), dim3(256), 0, s, a);
    if (p.splits > 1)
        hipLaunchKernelGGL(k_attn_join<D>, dim3((unsigned)(batch * a.c.heads * p.row_tiles * p.rt * (D / 16))), dim3(64), 0, s,
                           a, p.row_tiles * p.rt);
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
    if (seqs->batch == 0 || seqs->rows == 0) return 256;
    return 256 + attn_plan(cache, seqs, q_heads).ws;
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
    if (!__builtin_isfinite(scale)) return fail(NVFP4_ERR_ARG, "%s: scale is not finite", who);
    if (!out) return fail(NVFP4_ERR_ARG, "%s: NULL out", who);
    if (!aligned(out, 16)) return fail(NVFP4_ERR_ALIGN, "%s: out not 16-byte aligned", who);
    if (out_row_stride % 8 || out_row_stride < (int64_t)q->heads * q->dim)
        return fail(NVFP4_ERR_SHAPE, "%s: out_row_stride=%lld must be a multiple of 8 and >= q_heads * head_dim", who,
                    (long long)out_row_stride);
    const AttnPlan p = attn_plan(cache, seqs, q->heads);
    if (p.blocks > 2147483647LL) return fail(NVFP4_ERR_UNSUPPORTED, "%s: grid too large", who);
    if (!workspace || ws_bytes < 256 + p.ws)
        return fail(NVFP4_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", who, workspace ? ws_bytes : 0, 256 + p.ws);
    if (!aligned(workspace, 256)) return fail(NVFP4_ERR_ALIGN, "%s: workspace not 256-byte aligned", who);
    AttnArgs a;
    a.q = view(q);
    a.c = view(cache);
    a.s = view(seqs);
    // at least the smallest normal number: a hidden score of -inf stays -inf, and any
    // finite score times it is 0 to exp2
    a.scale = __builtin_fmaxf(__builtin_fabsf(scale) * 1.44269504088896340736f, 1.17549435e-38f);
    a.negate = scale < 0.0f;
    a.window = window;
    a.sinks = sinks;
    a.out = out;
    a.out_stride = out_row_stride;
    a.group = q->heads / cache->kv_heads;
    a.row_tiles = p.row_tiles;
    a.splits = p.splits;
    a.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + 256);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    switch (cache->head_dim) {
        case 64: launch_attn<64>(p, a, seqs->batch, s); break;
        case 128: launch_attn<128>(p, a, seqs->batch, s); break;
        case 192: launch_attn<192>(p, a, seqs->batch, s); break;
        default: launch_attn<256>(p, a, seqs->batch, s); break;
    }
    return check_launch(who);
}
