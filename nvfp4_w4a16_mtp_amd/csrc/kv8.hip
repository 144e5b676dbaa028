// Rotary positions and the paged 8-bit KV cache: rope_qk, kv8_append,
// rope_kv8_append, kv8_read.  Definitions in nvfp4_mtp.h.
//
// Everything here moves each row once and computes little, so memory traffic
// (long prompts) or launch and dependent-load latency (decode) bounds it.
//
// Rotation.  The angle is p * f in fp64: at p = 1e6 an fp32 product is off by
// up to 0.03 rad.  It is held in turns (f / 2 pi), reduced to [-1/8, 1/8] turn
// by a rint, and sine and cosine are Taylor sums in fp64 (cut below 2e-14).
// The rotation itself is fp64 too: its result is rounded to bf16 and, for the
// cache, to three mantissa bits, and an fp32 sum next to a rounding border
// would move a code by a whole step against the definition.  gfx950 runs fp64
// FMAs at the fp32 rate, so a prompt's rotation stays under its memory time.
//
// Append.  One workgroup owns one (page, head) of K or of V: the scale of a
// page needs the maximum over every token the call writes to it, and a grown
// scale re-rounds the page's older codes, so no two workgroups may share a
// page.  A thread's unit is a cell of 4 tokens x 8 elements: 16-byte loads, 8-byte
// K stores, and dword V stores of 4 tokens (V is transposed in its page).  The
// workgroup has a thread for every cell of the page (64 to 1024), so the rows stay
// in registers between the maximum and the encoding.  Rotated k elements pass
// through LDS, each pair turned once (turned where a cell needs them, the code of
// the unrolled angles, 50 to 180 KB, took longer to fetch than to run: 14 us
// instead of 8 for 64 sequences of 1 to 4 rows).
#include "kv8.hpp"

namespace nvfp4 {

struct Rope {
    const double *inv_freq;
    int rot, inter;
    float mscale;
};

// sin and cos of pos * f radians.
__device__ __forceinline__ void sincos_pos(double pos, double f, double &s, double &c) {
    const double turns = pos * (f * 0.15915494309189533577);   // 1 / (2 pi)
    const double y = (turns - __builtin_rint(turns)) * 4.0;     // quarter turns, [-2, 2]
    const double n = __builtin_rint(y);
    const double r = (y - n) * 1.57079632679489661923;          // [-pi/4, pi/4]
    const double r2 = r * r;
    double ps = -1.0 / 1307674368000.0, pc = 1.0 / 20922789888000.0;   // -1/15!, 1/16!
    ps = __builtin_fma(ps, r2, 1.0 / 6227020800.0);
    ps = __builtin_fma(ps, r2, -1.0 / 39916800.0);
    ps = __builtin_fma(ps, r2, 1.0 / 362880.0);
    ps = __builtin_fma(ps, r2, -1.0 / 5040.0);
    ps = __builtin_fma(ps, r2, 1.0 / 120.0);
    ps = __builtin_fma(ps, r2, -1.0 / 6.0);
    ps = __builtin_fma(ps * r2, r, r);
    pc = __builtin_fma(pc, r2, -1.0 / 87178291200.0);
    pc = __builtin_fma(pc, r2, 1.0 / 479001600.0);
    pc = __builtin_fma(pc, r2, -1.0 / 3628800.0);
    pc = __builtin_fma(pc, r2, 1.0 / 40320.0);
    pc = __builtin_fma(pc, r2, -1.0 / 720.0);
    pc = __builtin_fma(pc, r2, 1.0 / 24.0);
    pc = __builtin_fma(pc, r2, -0.5);
    pc = __builtin_fma(pc, r2, 1.0);
    const int q = (int)n;                                       // -2 .. 2
    const double a = (q & 1) ? pc : ps, b = (q & 1) ? ps : pc;
    s = (q & 2) ? -a : a;                                       // quadrants 2, 3 (and -2, -1)
    c = ((q + 1) & 2) ? -b : b;                                 // quadrants 1, 2 (and -2, -3)
}

__device__ __forceinline__ uint32_t pack_bf16(double a, double b) {
    return f32_to_bf16_bits((float)a) | (f32_to_bf16_bits((float)b) << 16);
}

// Eight bf16 pairs (x[i], y[i]) turned in place; x and y are packed octets of
// the half layout, or x and y the two octets of 8 interleaved pairs.
struct Turn8 {
    double s[8], c[8];
    __device__ __forceinline__ void load(const Rope &rp, double pos, int pair0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sincos_pos(pos, rp.inv_freq[pair0 + i], s[i], c[i]);
            s[i] *= rp.mscale;
            c[i] *= rp.mscale;
        }
    }
    __device__ __forceinline__ void apply_half(uint4 &x, uint4 &y) const {
        uint32_t *px = reinterpret_cast<uint32_t *>(&x), *py = reinterpret_cast<uint32_t *>(&y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double x0 = bf16_bits_to_f32(px[i] & 0xFFFFu), x1 = bf16_bits_to_f32(px[i] >> 16);
            const double y0 = bf16_bits_to_f32(py[i] & 0xFFFFu), y1 = bf16_bits_to_f32(py[i] >> 16);
            px[i] = pack_bf16(x0 * c[2 * i] - y0 * s[2 * i], x1 * c[2 * i + 1] - y1 * s[2 * i + 1]);
            py[i] = pack_bf16(x0 * s[2 * i] + y0 * c[2 * i], x1 * s[2 * i + 1] + y1 * c[2 * i + 1]);
        }
    }
    __device__ __forceinline__ void apply(uint4 &x, uint4 &y, bool inter) const {
        if (inter) {
            apply_inter<0>(x);
            apply_inter<4>(y);
        } else {
            apply_half(x, y);
        }
    }
    // pairs OFF .. OFF + 3 on one octet
    template <int OFF>
    __device__ __forceinline__ void apply_inter(uint4 &x) const {
        uint32_t *px = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double a = bf16_bits_to_f32(px[i] & 0xFFFFu), b = bf16_bits_to_f32(px[i] >> 16);
            px[i] = pack_bf16(a * c[OFF + i] - b * s[OFF + i], a * s[OFF + i] + b * c[OFF + i]);
        }
    }
};

// ------------------------------------------------------------------- rope --
// Unit u of a row: u < rot / 16 turns 16 elements of each of the heads
// [h0, h1); later units copy 8 elements each (only when out is not in).
struct RopeTask {
    HeadRows in, out;
    int heads;
};

constexpr int kHeads = 2;   // heads whose loads are in flight together

__device__ __forceinline__ void rope_unit(const RopeTask &t, const Rope &rp, int64_t row, int u, int h0, int h1,
                                          double pos) {
    const int turns = rp.rot >> 4;
    const uint16_t *src = t.in.data + row * t.in.row;
    uint16_t *dst = t.out.data + row * t.out.row;
    if (u >= turns) {
        const int d = rp.rot + (u - turns) * 8;
        for (int h = h0; h < h1; ++h)
            *reinterpret_cast<uint4 *>(dst + h * t.out.head + d) =
                *reinterpret_cast<const uint4 *>(src + h * t.in.head + d);
        return;
    }
    Turn8 w;
    w.load(rp, pos, u * 8);
    const int d0 = rp.inter ? u * 16 : u * 8, d1 = rp.inter ? d0 + 8 : d0 + (rp.rot >> 1);
    // the loads of kHeads heads at a time (past the last one, the last again)
    for (int h = h0; h < h1; h += kHeads) {
        uint4 x[kHeads], y[kHeads];
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
            const uint16_t *at = src + (int64_t)min(h + k, h1 - 1) * t.in.head;
            x[k] = *reinterpret_cast<const uint4 *>(at + d0);
            y[k] = *reinterpret_cast<const uint4 *>(at + d1);
        }
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
            if (h + k >= h1) break;
            w.apply(x[k], y[k], rp.inter);
            uint16_t *at = dst + (int64_t)(h + k) * t.out.head;
            *reinterpret_cast<uint4 *>(at + d0) = x[k];
            *reinterpret_cast<uint4 *>(at + d1) = y[k];
        }
    }
}

// blockIdx.y: a group of heads of q, then of k.
__global__ __launch_bounds__(256) void k_rope(RopeTask q, RopeTask k, Rope rp, const int32_t *__restrict__ pos,
                                             int rows, int uq, int uk, int per, int qgroups) {
    const bool is_q = (int)blockIdx.y < qgroups;
    const RopeTask &t = is_q ? q : k;
    const int units = is_q ? uq : uk;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = i / units;
    if (row >= rows) return;
    const int u = (int)(i - row * units);
    const int h0 = ((int)blockIdx.y - (is_q ? 0 : qgroups)) * per;
    rope_unit(t, rp, row, u, h0, min(h0 + per, t.heads), (double)pos[row]);
}

// ----------------------------------------------------------------- append --
// Two floats -> two E4M3 codes in half SEL of `into`: nearest, ties to even,
// saturating; NaN stays NaN (both comparisons are false).
template <bool HI>
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t into, float a, float b) {
    a = a > 448.0f ? 448.0f : (a < -448.0f ? -448.0f : a);
    b = b > 448.0f ? 448.0f : (b < -448.0f ? -448.0f : b);
    return __builtin_amdgcn_cvt_pk_fp8_f32(a, b, into, HI);
}
// Two packed bf16 pairs times 2^-e -> four codes.
__device__ __forceinline__ uint32_t encode4(uint32_t lo, uint32_t hi, int e) {
    const uint32_t v = e4m3_pair<false>(0u, __builtin_ldexpf(bf16_bits_to_f32(lo & 0xFFFFu), -e),
                                        __builtin_ldexpf(bf16_bits_to_f32(lo >> 16), -e));
    return e4m3_pair<true>(v, __builtin_ldexpf(bf16_bits_to_f32(hi & 0xFFFFu), -e),
                           __builtin_ldexpf(bf16_bits_to_f32(hi >> 16), -e));
}
// Four codes re-rounded to a scale 2^up times as large.
__device__ __forceinline__ uint32_t requant4(uint32_t w, int up) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    uint32_t o = e4m3_pair<false>(0u, __builtin_ldexpf(a.x, -up), __builtin_ldexpf(a.y, -up));
    return e4m3_pair<true>(o, __builtin_ldexpf(b.x, -up), __builtin_ldexpf(b.y, -up));
}

// Largest finite |bf16| of a packed pair, as bits.
__device__ __forceinline__ uint32_t finite_max(uint32_t mx, uint32_t pair) {
    const uint32_t a = pair & 0x7FFFu, b = (pair >> 16) & 0x7FFFu;
    mx = max(mx, a < 0x7F80u ? a : 0u);
    return max(mx, b < 0x7F80u ? b : 0u);
}

struct AppendArgs {
    KV8 c;
    Seqs s;
    HeadRows kin, vin;
    Rope rp;            // rot == 0: no rotation
    RopeTask q;         // heads == 0: no q
    int dim, items;     // pages a sequence's rows can touch
    int kv_blocks;      // blocks of the cache part; q blocks follow
    int q_units, q_per, q_groups;
};

constexpr int kMinExp = -110;

// Smallest e >= kMinExp with amax <= 448 * 2^e, or kMaxExp; amax = 1.m * 2^(x - 127)
// as bf16 bits (448 = 1.75 * 2^8).
__device__ __forceinline__ int scale_exp(uint32_t bits) {
    const int e = (int)(bits >> 7) - 135 + ((bits & 0x7Fu) > 0x60u);
    return min(max(e, kMinExp), kMaxExp);
}

// ROPE: the k rows are rotated (dynamic LDS: page_tokens * rot bf16).
template <bool ROPE>
__global__ __launch_bounds__(1024) void k_append(AppendArgs a) {
    extern __shared__ uint4 turned[];                 // [token of the page][rot / 8]
    const int bid = blockIdx.x, tid = threadIdx.x, threads = blockDim.x;
    if (ROPE && bid >= a.kv_blocks) {
        // q rows: thread = (unit, row of the sequence, sequence)
        const int qb = bid - a.kv_blocks, group = qb % a.q_groups;
        const int64_t i = (int64_t)(qb / a.q_groups) * threads + tid;
        const int64_t r = i / a.q_units;
        const int b = (int)(r / a.s.max_rows), j = (int)(r % a.s.max_rows);
        if (b >= a.s.batch) return;
        const Seq sq = load_seq(a.s, b, a.c.lp);
        if (j >= sq.n) return;
        rope_unit(a.q, a.rp, sq.r0 + j, (int)(i - r * a.q_units), group * a.q_per,
                  min(group * a.q_per + a.q_per, a.q.heads), (double)(sq.len - sq.n + j));
        return;
    }
    const int hk = bid % (2 * a.c.heads), w = bid / (2 * a.c.heads);
    const bool is_v = hk >= a.c.heads;
    const int h = is_v ? hk - a.c.heads : hk;
    const int b = w / a.items, item = w % a.items;
    const Seq sq = load_seq(a.s, b, a.c.lp);
    const int n = min(sq.n, a.s.max_rows);
    const int P = 1 << a.c.lp;
    const int shift = sq.len - sq.n;                 // position of the first row (may be negative)
    const int start = max(shift, 0), end = shift + n;
    const int idx = (start >> a.c.lp) + item;
    if (end <= 0 || (int64_t)idx << a.c.lp >= end) return;
    const int page = a.s.table[(int64_t)b * a.s.max_pages + idx];
    if (page < 0 || page >= a.c.pages) return;
    uint8_t *scale = (is_v ? a.c.vs : a.c.ks) + (int64_t)page * a.c.heads + h;
    const int e_old = kv8_exp(*scale);
    const int p0 = idx << a.c.lp;
    const int o0 = max(start - p0, 0), o1 = min(end - p0, P);
    const int oct = a.dim >> 3;
    const HeadRows &in = is_v ? a.vin : a.kin;
    // row of token p0: rows run with the positions
    const uint16_t *src = in.data + ((int64_t)sq.r0 + p0 - shift) * in.row + h * in.head;
    const bool rotate = ROPE && !is_v;
    const int turns = rotate ? a.rp.rot >> 4 : 0;     // units of 8 pairs
    if (rotate) {
        for (int i = tid; i < (o1 - o0) * turns; i += threads) {
            const int t = o0 + i / turns, u = i % turns;
            const int d0 = a.rp.inter ? u * 2 : u, d1 = a.rp.inter ? d0 + 1 : d0 + turns;   // octets
            const uint4 *row = reinterpret_cast<const uint4 *>(src + (int64_t)t * in.row);
            uint4 x = row[d0], y = row[d1];
            Turn8 turn;
            turn.load(a.rp, (double)(p0 + t), u * 8);
            turn.apply(x, y, a.rp.inter);
            turned[t * 2 * turns + d0] = x;
            turned[t * 2 * turns + d1] = y;
        }
        __syncthreads();
    }
    // cells: K octet fastest (row loads and stores run along the row); V quad
    // fastest (its stores run along the tokens)
    const int quads = P >> 2;
    const int quad = is_v ? tid & (quads - 1) : tid / oct, o = is_v ? tid >> (a.c.lp - 2) : tid - quad * oct;
    const int t0 = quad * 4;
    const bool cell = o < oct && quad < quads;
    uint4 x[4];
    uint32_t mx = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int t = t0 + j;
        x[j] = make_uint4(0, 0, 0, 0);
        if (cell && t >= o0 && t < o1)
            x[j] = o < 2 * turns ? turned[t * 2 * turns + o] : reinterpret_cast<const uint4 *>(src + (int64_t)t * in.row)[o];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        mx = finite_max(mx, x[j].x);
        mx = finite_max(mx, x[j].y);
        mx = finite_max(mx, x[j].z);
        mx = finite_max(mx, x[j].w);
    }
    __shared__ uint32_t wmax[16];
    for (int off = 32; off > 0; off >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, off, 64));
    if ((tid & 63) == 0) wmax[tid >> 6] = mx;
    __syncthreads();                                  // every thread has read the old scale
    for (int i = 0; i < threads >> 6; ++i) mx = max(mx, wmax[i]);
    int e = scale_exp(mx);
    const bool older = o0 > 0;
    if (older) e = max(e, e_old);
    const int up = older ? e - e_old : 0;
    if (tid == 0) *scale = (uint8_t)(e + 127);
    if (!cell || t0 >= o1 || (t0 + 4 <= o0 && up == 0)) return;
    uint8_t *dst = (is_v ? a.c.v : a.c.k) + ((int64_t)page * a.c.heads + h) * ((int64_t)a.dim << a.c.lp);
    uint32_t code[4][2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        code[j][0] = encode4(x[j].x, x[j].y, e);
        code[j][1] = encode4(x[j].z, x[j].w, e);
    }
    if (!is_v) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = t0 + j;
            uint2 *at = reinterpret_cast<uint2 *>(dst + (int64_t)t * a.dim + o * 8);
            if (t >= o0 && t < o1) {
                *at = make_uint2(code[j][0], code[j][1]);
            } else if (t < o0 && up > 0) {
                const uint2 old = *at;
                *at = make_uint2(requant4(old.x, up), requant4(old.y, up));
            }
        }
        return;
    }
    // V: element d of the four tokens is one dword; merged with what the page holds
    // where only some of them are new
    uint32_t fresh = 0, held = 0;                     // bytes that are new, and that hold older tokens
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        fresh |= (t0 + j >= o0 && t0 + j < o1) ? 0xFFu << (8 * j) : 0u;
        held |= (t0 + j < o0) ? 0xFFu << (8 * j) : 0u;
    }
    uint32_t *at = reinterpret_cast<uint32_t *>(dst + (((int64_t)o * 8) << a.c.lp) + t0);
    const int step = P >> 2;                          // dwords from one dim to the next
    uint32_t old[8];
#pragma unroll
    for (int d = 0; d < 8; ++d) old[d] = fresh != 0xFFFFFFFFu ? at[d * step] : 0u;
    if (up > 0) {
#pragma unroll
        for (int d = 0; d < 8; ++d) old[d] = (requant4(old[d], up) & held) | (old[d] & ~held);
    }
#pragma unroll
    for (int h2 = 0; h2 < 2; ++h2) {
        // 4 x 4 bytes transposed: two rounds of byte merges
        const uint32_t a0 = code[0][h2], a1 = code[1][h2], a2 = code[2][h2], a3 = code[3][h2];
        const uint32_t lo01 = __builtin_amdgcn_perm(a1, a0, 0x05010400u), hi01 = __builtin_amdgcn_perm(a1, a0, 0x07030602u);
        const uint32_t lo23 = __builtin_amdgcn_perm(a3, a2, 0x05010400u), hi23 = __builtin_amdgcn_perm(a3, a2, 0x07030602u);
        const uint32_t v[4] = {__builtin_amdgcn_perm(lo23, lo01, 0x05040100u), __builtin_amdgcn_perm(lo23, lo01, 0x07060302u),
                               __builtin_amdgcn_perm(hi23, hi01, 0x05040100u), __builtin_amdgcn_perm(hi23, hi01, 0x07060302u)};
#pragma unroll
        for (int d = 0; d < 4; ++d) at[(h2 * 4 + d) * step] = (v[d] & fresh) | (old[h2 * 4 + d] & ~fresh);
    }
}

// ------------------------------------------------------------------- read --
// One workgroup per (page of a sequence, head) of K or V; cells as in append.
struct ReadArgs {
    KV8 c;
    Seqs s;
    HeadRows kout, vout;
    int dim, items;
    int lists;          // 2: K and V, 1: one of them
};

__device__ __forceinline__ uint2 bf16x4_of(uint32_t w, int e) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    return make_uint2(f32_to_bf16_bits(__builtin_ldexpf(a.x, e)) | (f32_to_bf16_bits(__builtin_ldexpf(a.y, e)) << 16),
                      f32_to_bf16_bits(__builtin_ldexpf(b.x, e)) | (f32_to_bf16_bits(__builtin_ldexpf(b.y, e)) << 16));
}

__global__ __launch_bounds__(256) void k_kv8_read(ReadArgs a) {
    const int tid = threadIdx.x;
    const int hk = blockIdx.x % (a.lists * a.c.heads), w = blockIdx.x / (a.lists * a.c.heads);
    const bool is_v = hk >= a.c.heads || a.kout.data == nullptr;
    const int h = hk % a.c.heads;
    const int b = w / a.items, item = w % a.items;
    const Seq sq = load_seq(a.s, b, a.c.lp);
    const int n = min(sq.n, a.s.max_rows);
    const int P = 1 << a.c.lp, shift = sq.len - sq.n;
    const HeadRows &out = is_v ? a.vout : a.kout;
    const int oct = a.dim >> 3, quads = P >> 2, cells = quads * oct;
    // rows at negative positions are zero rows (the first item writes them)
    if (item == 0 && shift < 0) {
        const int lim = min(-shift, n);
        for (int i = tid; i < lim * oct; i += 256)
            *reinterpret_cast<uint4 *>(out.data + ((int64_t)sq.r0 + i / oct) * out.row + h * out.head + (i % oct) * 8) =
                make_uint4(0, 0, 0, 0);
    }
    const int start = max(shift, 0), end = shift + n;
    const int idx = (start >> a.c.lp) + item;
    if (end <= 0 || (int64_t)idx << a.c.lp >= end) return;
    const int page = a.s.table[(int64_t)b * a.s.max_pages + idx];
    const bool in = page >= 0 && page < a.c.pages;
    const int p0 = idx << a.c.lp;
    const int o0 = max(start - p0, 0), o1 = min(end - p0, P);
    const int64_t pg = in ? page : 0;
    const int e = kv8_exp((is_v ? a.c.vs : a.c.ks)[pg * a.c.heads + h]);
    const uint8_t *src = (is_v ? a.c.v : a.c.k) + (pg * a.c.heads + h) * ((int64_t)a.dim << a.c.lp);
    uint16_t *dst = out.data + ((int64_t)sq.r0 + p0 - shift) * out.row + h * out.head;
    for (int cell = tid; cell < cells; cell += 256) {
        const int quad = cell / oct, o = cell % oct, t0 = quad * 4;
        if (t0 >= o1 || t0 + 4 <= o0) continue;
        uint32_t word[4][2];                          // [token][half of the octet]
        if (!is_v) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint2 v = *reinterpret_cast<const uint2 *>(src + (int64_t)(t0 + j) * a.dim + o * 8);
                word[j][0] = v.x;
                word[j][1] = v.y;
            }
        } else {
            uint32_t d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = *reinterpret_cast<const uint32_t *>(src + (((int64_t)o * 8 + i) << a.c.lp) + t0);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t v = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) v |= ((d[4 * q + i] >> (8 * j)) & 0xFFu) << (8 * i);
                    word[j][q] = v;
                }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = t0 + j;
            if (t < o0 || t >= o1) continue;
            const uint2 lo = bf16x4_of(word[j][0], e), hi = bf16x4_of(word[j][1], e);
            *reinterpret_cast<uint4 *>(dst + (int64_t)t * out.row + o * 8) =
                in ? make_uint4(lo.x, lo.y, hi.x, hi.y) : make_uint4(0, 0, 0, 0);
        }
    }
}

// ------------------------------------------------------------ host checks --
int validate_head_rows(const nvfp4_head_rows *r, const char *who, const char *what) {
    if (!r || !r->data) return fail(NVFP4_ERR_ARG, "%s: %s is NULL", who, what);
    if (r->heads < 1 || r->dim < 8 || r->dim % 8)
        return fail(NVFP4_ERR_SHAPE, "%s: %s has heads=%d dim=%d (need heads >= 1, dim a multiple of 8)", who, what,
                    r->heads, r->dim);
    if (r->row_stride < 0 || r->row_stride % 8 || r->head_stride % 8 || r->head_stride < r->dim)
        return fail(NVFP4_ERR_SHAPE, "%s: %s has row_stride=%lld head_stride=%lld (need multiples of 8, row_stride >= 0, "
                    "head_stride >= dim)", who, what, (long long)r->row_stride, (long long)r->head_stride);
    if (!aligned(r->data, 16)) return fail(NVFP4_ERR_ALIGN, "%s: %s not 16-byte aligned", who, what);
    return NVFP4_OK;
}

// Outputs: no two of `rows` rows' heads share an element.
static int validate_apart(const nvfp4_head_rows *r, int64_t rows, const char *who, const char *what) {
    if (rows <= 1 || r->row_stride >= (r->heads - 1) * r->head_stride + r->dim ||
        (r->row_stride >= r->dim && r->head_stride >= (rows - 1) * r->row_stride + r->dim))
        return NVFP4_OK;
    return fail(NVFP4_ERR_SHAPE, "%s: rows of %s overlap (row_stride=%lld, head_stride=%lld)", who, what,
                (long long)r->row_stride, (long long)r->head_stride);
}

int validate_kv8_cache(const nvfp4_kv8_cache *c, const char *who) {
    if (!c || !c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales)
        return fail(NVFP4_ERR_ARG, "%s: NULL cache descriptor or pointer", who);
    if (c->num_pages < 1 || c->kv_heads < 1 || c->kv_heads > 65535)
        return fail(NVFP4_ERR_SHAPE, "%s: cache has num_pages=%d kv_heads=%d", who, c->num_pages, c->kv_heads);
    if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
        return fail(NVFP4_ERR_SHAPE, "%s: page_tokens=%d is not 16, 32, 64 or 128", who, c->page_tokens);
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 192 && c->head_dim != 256)
        return fail(NVFP4_ERR_SHAPE, "%s: head_dim=%d is not 64, 128, 192 or 256", who, c->head_dim);
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16))
        return fail(NVFP4_ERR_ALIGN, "%s: cache codes not 16-byte aligned", who);
    return NVFP4_OK;
}

int validate_kv8_seqs(const nvfp4_kv8_seqs *s, const char *who) {
    if (!s) return fail(NVFP4_ERR_ARG, "%s: seqs descriptor is NULL", who);
    if (s->batch < 0 || s->rows < 0 || s->max_rows < 0 || s->max_pages < 0 || s->max_kv_len < 0)
        return fail(NVFP4_ERR_SHAPE, "%s: negative batch=%d rows=%d max_rows=%d max_pages=%d or max_kv_len=%d", who,
                    s->batch, s->rows, s->max_rows, s->max_pages, s->max_kv_len);
    if (s->batch == 0 || s->rows == 0) return NVFP4_OK;   // nothing is read
    if (s->max_rows < 1 || s->max_pages < 1)
        return fail(NVFP4_ERR_SHAPE, "%s: max_rows=%d and max_pages=%d must be positive", who, s->max_rows, s->max_pages);
    if (!s->cu_rows || !s->kv_lens || !s->block_table) return fail(NVFP4_ERR_ARG, "%s: NULL cu_rows, kv_lens or block_table", who);
    if (!aligned(s->cu_rows, 4) || !aligned(s->kv_lens, 4) || !aligned(s->block_table, 4))
        return fail(NVFP4_ERR_ALIGN, "%s: cu_rows, kv_lens and block_table need 4-byte alignment", who);
    return NVFP4_OK;
}

static int validate_rope(const nvfp4_rope *r, int dim, const char *who) {
    if (!r || !r->inv_freq) return fail(NVFP4_ERR_ARG, "%s: NULL rope descriptor or inv_freq", who);
    if (r->rot_dim < 16 || r->rot_dim % 16 || r->rot_dim > dim)
        return fail(NVFP4_ERR_SHAPE, "%s: rot_dim=%d must be a multiple of 16 in 16..%d", who, r->rot_dim, dim);
    if (!aligned(r->inv_freq, 8)) return fail(NVFP4_ERR_ALIGN, "%s: inv_freq not 8-byte aligned", who);
    return NVFP4_OK;
}

// One of the two rope pairs: both NULL (heads = 0) or both valid and alike.
static int rope_pair(const nvfp4_head_rows *in, const nvfp4_head_rows *out, int64_t rows, const char *who,
                     const char *what, RopeTask &t) {
    t = RopeTask{HeadRows{nullptr, 0, 0}, HeadRows{nullptr, 0, 0}, 0};
    if (!in && !out) return NVFP4_OK;
    if (int rc = validate_head_rows(in, who, what)) return rc;
    if (int rc = validate_head_rows(out, who, what)) return rc;
    if (int rc = validate_apart(out, rows, who, what)) return rc;
    if (in->heads != out->heads || in->dim != out->dim)
        return fail(NVFP4_ERR_SHAPE, "%s: %s and its output have different heads or dim", who, what);
    if (in->data == out->data && (in->row_stride != out->row_stride || in->head_stride != out->head_stride))
        return fail(NVFP4_ERR_SHAPE, "%s: %s rotated in place needs equal strides", who, what);
    t = RopeTask{view(in), view(out), in->heads};
    return NVFP4_OK;
}

static int rope_units(const RopeTask &t, int dim, int rot) {
    return rot / 16 + (t.in.data == t.out.data ? 0 : (dim - rot) / 8);
}

// Heads a thread turns with one set of angles: as many as leave the device about
// four workgroups per CU, four at most (the angles are most of the arithmetic, but
// fewer heads keep more loads in flight: 6001 rows of 32 + 8 heads of 128, 33.3 us
// with seven heads a thread, 29.9 with four).
static int heads_per_thread(int64_t threads_per_head, int heads) {
    const int64_t want = (int64_t)num_cus() * 4 * 256;
    int64_t per = threads_per_head * heads / want;
    per = per < 1 ? 1 : per;
    return (int)(per < 4 ? per : 4);
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" int rope_qk(const nvfp4_head_rows *q, const nvfp4_head_rows *q_out, const nvfp4_head_rows *k,
                       const nvfp4_head_rows *k_out, int32_t rows, const int32_t *positions, const nvfp4_rope *rope,
                       void *stream) {
    const char *who = "rope_qk";
    if (!q && !q_out && !k && !k_out) return fail(NVFP4_ERR_ARG, "%s: neither q nor k", who);
    if (rows < 0) return fail(NVFP4_ERR_SHAPE, "%s: rows=%d < 0", who, rows);
    if (rows == 0) return ok();
    RopeTask tq, tk;
    if (int rc = rope_pair(q, q_out, rows, who, "q", tq)) return rc;
    if (int rc = rope_pair(k, k_out, rows, who, "k", tk)) return rc;
    const int dim = q ? q->dim : k->dim;
    if (q && k && q->dim != k->dim) return fail(NVFP4_ERR_SHAPE, "%s: q and k have different dim", who);
    if (int rc = validate_rope(rope, dim, who)) return rc;
    if (!positions) return fail(NVFP4_ERR_ARG, "%s: NULL positions", who);
    if (!aligned(positions, 4)) return fail(NVFP4_ERR_ALIGN, "%s: positions not 4-byte aligned", who);
    const int uq = rope_units(tq, dim, rope->rot_dim), uk = rope_units(tk, dim, rope->rot_dim);
    const int units = uq > uk ? uq : uk;
    const int per = heads_per_thread((int64_t)rows * units, tq.heads + tk.heads);
    const int qg = (tq.heads + per - 1) / per, kg = (tk.heads + per - 1) / per;
    const int64_t blocks = ((int64_t)rows * units + 255) / 256;
    if (!grid_fits(blocks, 256) || qg + kg > 65535) return fail(NVFP4_ERR_UNSUPPORTED, "%s: grid too large", who);
    const Rope rp{rope->inv_freq, rope->rot_dim, rope->interleaved != 0, rope->mscale};
    hipLaunchKernelGGL(k_rope, dim3((unsigned)blocks, qg + kg), dim3(256), 0, reinterpret_cast<hipStream_t>(stream), tq,
                       tk, rp, positions, rows, uq > 0 ? uq : 1, uk > 0 ? uk : 1, per, qg);
    return check_launch(who);
}

static int append(const char *who, const nvfp4_kv8_cache *cache, const nvfp4_kv8_seqs *seqs, const nvfp4_rope *rope,
                  const nvfp4_head_rows *q, const nvfp4_head_rows *q_out, const nvfp4_head_rows *k,
                  const nvfp4_head_rows *v, void *stream) {
    if (int rc = validate_kv8_cache(cache, who)) return rc;
    if (int rc = validate_kv8_seqs(seqs, who)) return rc;
    if (seqs->batch == 0 || seqs->rows == 0) return ok();
    if (int rc = validate_head_rows(k, who, "k")) return rc;
    if (int rc = validate_head_rows(v, who, "v")) return rc;
    for (const nvfp4_head_rows *r : {k, v})
        if (r->heads != cache->kv_heads || r->dim != cache->head_dim)
            return fail(NVFP4_ERR_SHAPE, "%s: k and v need the cache's kv_heads=%d and head_dim=%d", who, cache->kv_heads,
                        cache->head_dim);
    RopeTask tq;
    if (int rc = rope_pair(q, q_out, seqs->rows, who, "q", tq)) return rc;
    if (q && q->dim != cache->head_dim) return fail(NVFP4_ERR_SHAPE, "%s: q has dim %d, the cache %d", who, q->dim, cache->head_dim);
    const int P = cache->page_tokens;
    const int max_rows = seqs->max_rows < seqs->rows ? seqs->max_rows : seqs->rows;
    AppendArgs a;
    a.c = view(cache);
    a.s = view(seqs);
    a.s.max_rows = max_rows;
    a.kin = view(k);
    a.vin = view(v);
    a.rp = rope ? Rope{rope->inv_freq, rope->rot_dim, rope->interleaved != 0, rope->mscale} : Rope{nullptr, 0, 0, 1.0f};
    a.q = tq;
    a.dim = cache->head_dim;
    a.items = (int)(((int64_t)max_rows + 2 * P - 2) / P);
    const int64_t kv_blocks = (int64_t)seqs->batch * a.items * 2 * cache->kv_heads;
    a.q_units = a.q_per = a.q_groups = 1;
    const int cells = P / 4 * (a.dim / 8);            // 32 .. 1024
    const int threads = (cells + 63) / 64 * 64;
    int64_t blocks = kv_blocks;
    if (tq.heads > 0) {
        a.q_units = rope_units(tq, a.dim, a.rp.rot);
        const int64_t units = (int64_t)seqs->batch * max_rows * a.q_units;
        a.q_per = heads_per_thread(units, tq.heads);
        a.q_groups = (tq.heads + a.q_per - 1) / a.q_per;
        blocks += (units + threads - 1) / threads * a.q_groups;
    }
    if (!grid_fits(blocks, threads)) return fail(NVFP4_ERR_UNSUPPORTED, "%s: grid too large", who);
    a.kv_blocks = (int)kv_blocks;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (rope) {
        const size_t lds = (size_t)P * a.rp.rot * 2;  // at most 64 KiB, and 64 bytes of the kernel's own
        if (int rc = allow_lds(reinterpret_cast<const void *>(k_append<true>), lds + 64, who)) return rc;
        hipLaunchKernelGGL(k_append<true>, dim3((unsigned)blocks), dim3(threads), lds, s, a);
    } else {
        hipLaunchKernelGGL(k_append<false>, dim3((unsigned)blocks), dim3(threads), 0, s, a);
    }
    return check_launch(who);
}

extern "C" int kv8_append(const nvfp4_kv8_cache *cache, const nvfp4_kv8_seqs *seqs, const nvfp4_head_rows *k,
                          const nvfp4_head_rows *v, void *stream) {
    return append("kv8_append", cache, seqs, nullptr, nullptr, nullptr, k, v, stream);
}

extern "C" int rope_kv8_append(const nvfp4_kv8_cache *cache, const nvfp4_kv8_seqs *seqs, const nvfp4_rope *rope,
                               const nvfp4_head_rows *q, const nvfp4_head_rows *q_out, const nvfp4_head_rows *k,
                               const nvfp4_head_rows *v, void *stream) {
    if (int rc = validate_kv8_cache(cache, "rope_kv8_append")) return rc;
    if (int rc = validate_rope(rope, cache->head_dim, "rope_kv8_append")) return rc;
    return append("rope_kv8_append", cache, seqs, rope, q, q_out, k, v, stream);
}

extern "C" int kv8_read(const nvfp4_kv8_cache *cache, const nvfp4_kv8_seqs *seqs, const nvfp4_head_rows *k_out,
                        const nvfp4_head_rows *v_out, void *stream) {
    const char *who = "kv8_read";
    if (int rc = validate_kv8_cache(cache, who)) return rc;
    if (int rc = validate_kv8_seqs(seqs, who)) return rc;
    if (seqs->batch == 0 || seqs->rows == 0) return ok();
    if (!k_out && !v_out) return fail(NVFP4_ERR_ARG, "%s: neither k_out nor v_out", who);
    for (const nvfp4_head_rows *r : {k_out, v_out}) {
        if (!r) continue;
        if (int rc = validate_head_rows(r, who, r == k_out ? "k_out" : "v_out")) return rc;
        if (int rc = validate_apart(r, seqs->rows, who, r == k_out ? "k_out" : "v_out")) return rc;
        if (r->heads != cache->kv_heads || r->dim != cache->head_dim)
            return fail(NVFP4_ERR_SHAPE, "%s: outputs need the cache's kv_heads=%d and head_dim=%d", who, cache->kv_heads,
                        cache->head_dim);
    }
    const int P = cache->page_tokens;
    const int max_rows = seqs->max_rows < seqs->rows ? seqs->max_rows : seqs->rows;
    ReadArgs a;
    a.c = view(cache);
    a.s = view(seqs);
    a.s.max_rows = max_rows;
    a.kout = view(k_out);
    a.vout = view(v_out);
    a.dim = cache->head_dim;
    a.items = (int)(((int64_t)max_rows + 2 * P - 2) / P);
    a.lists = k_out && v_out ? 2 : 1;
    const int64_t blocks = (int64_t)seqs->batch * a.items * a.lists * cache->kv_heads;
    if (!grid_fits(blocks, 256)) return fail(NVFP4_ERR_UNSUPPORTED, "%s: grid too large", who);
    hipLaunchKernelGGL(k_kv8_read, dim3((unsigned)blocks), dim3(256), 0, reinterpret_cast<hipStream_t>(stream), a);
    return check_launch(who);
}
