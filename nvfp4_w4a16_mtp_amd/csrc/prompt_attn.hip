// prompt_attention: causal softmax attention over whole packed prompts
// (definition in nvfp4_mtp.h).
//
// For each row: o = sum_t p_t v_t / sum_t p_t with p_t = 2^((q.k_t - m) scale'), one pass
// over the keys with a running reference m and sum (fp32).  Must compute 2 (dk + dv) flop
// a visible (row, key) pair and query head; the bytes (q, k, v and the result once) are
// nothing beside that for long prompts.
//
// A workgroup of four wavefronts takes 128 rows of one query head, a wavefront 32 of them
// with all dims of their sums in registers, and walks the keys in tiles of 64 tokens with
// v_mfma_f32_32x32x16_bf16:
//   S^T = K Q^T    A = K (32 tokens), B = Q^T (32 rows, in registers throughout);
//   O^T = V^T P^T  A = V^T (32 dims), B = P^T.
// A lane's column is a row of queries in both products, and S^T comes out of the first in
// a lane order that is the second's operand order up to a permutation of the tokens; V is
// read in the same permutation (transposing LDS reads), so P never leaves its registers.
// Tiles go from memory straight into LDS (double buffered, swizzled at the source so that
// reads have few bank conflicts: none counted at 128 and 256 dims, 37% of the LDS cycles at 192,
// where the swizzle has eight places), each fragment is read a few products ahead.
//  - The first product accumulates onto -m, so a weight is one multiplication and 2^x, and the
//    reference moves only where a row's score exceeds it by kPromptSlack (2^6 in the weights).
//  - The weights of 16 tokens are made beside the products of the 16 before: exponentials run
//    on the vector units while the matrix cores are busy (12001 rows, 16 + 2 heads of 256:
//    2257 us with no read-ahead, 1552 with it, 1323 so; the next tile's scores beside this
//    one's weights 1238 us there, but 64 more registers: packed prompts of 128 dims 506 us
//    against 404).
//  - 64-token tiles: 32-token ones with four stages spill or pay the barrier twice (128 dims:
//    506 us).  Two workgroups a CU where registers and LDS allow (dims up to 192 x 128: windowed
//    prompts 465 us with one, 325 so); 192 x 192 and 256 x 256 have one wavefront a SIMD.
//  - 24 prompts of up to 4500 rows, 32 + 8 heads of 128: 404 us, 880 TFLOP/s; 12001 rows of
//    256 dims: 1323 us, 893 TFLOP/s (an 8192^3 product reaches 1222).  With everything but the
//    products and barriers left out the latter takes 915 us.  What bounds it: one wavefront a
//    SIMD with little to cover the waits between its two products (matrix cores busy 38%); at
//    128 dims matrix cores busy 47%, vector issue 51%.
// Long prompts' tiles first: the keys of a row tile grow with its number.  All tiles of a query
// head go to one XCD, whose L2 then holds that head's keys.
#include <type_traits>

#include "kv8.hpp"

namespace nvfp4 {

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(16))) float f32x16;

// Excess of a scaled score over the reference that moves it: weights up to 2^6 cost no precision.
constexpr float kPromptSlack = 6.0f;

// Exponent of the weights' factor in a third pass: sums of up to 2^31 weights of up to
// 2^kPromptSlack, times values of up to 2^128, stay below 2^128.
constexpr float kLow = 40.0f;

struct PromptArgs {
    HeadRows q, k, v;
    const int32_t *cu;
    int batch, rows, max_rows;
    float scale;            // |scale| * log2(e), 1 for a scale of 0
    bool negate, zero;      // scale < 0, scale == 0
    int window, sinks;
    int heads, group;       // q heads, q heads a kv head
    int dk, dv;
    int per_xcd;            // heads / 8, or 0 where 8 does not divide them
    uint16_t *out;
    int64_t out_stride;
};

__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

__device__ __forceinline__ bool not_finite(uint32_t bf16) { return (bf16 & 0x7F80u) == 0x7F80u; }
// ... of the two in a word.
__device__ __forceinline__ bool any_not_finite(uint32_t two) { return not_finite(two) || not_finite(two >> 16); }
// Two bf16 values, and to each the other word's where that is not finite.
__device__ __forceinline__ uint32_t add_not_finite(uint32_t to, uint32_t v) {
    const float lo = bf16_bits_to_f32(to & 0xFFFFu) + bf16_bits_to_f32(v & 0xFFFFu), hi = bf16_bits_to_f32(to >> 16) + bf16_bits_to_f32(v >> 16);
    return (not_finite(v) ? f32_to_bf16_bits(lo) : to & 0xFFFFu) | (not_finite(v >> 16) ? f32_to_bf16_bits(hi) << 16 : to & 0xFFFF0000u);
}

// Rows of sequence b, cut to the call's bounds.
__device__ __forceinline__ int2 prompt_rows(const PromptArgs &a, int b) {
    const int lo = min(max(a.cu[b], 0), a.rows);
    const int n = min(max(a.cu[b + 1], lo), a.rows) - lo;
    return make_int2(lo, min(n, a.max_rows));
}

// The item-th row tile of R rows: its sequence and its number there, or false.
// Up to 64 sequences: all sequences' last tiles first, as a tile's keys grow with
// its number.  More: sequence by sequence, the last tile first.
template <int R>
__device__ __forceinline__ bool find_tile(const PromptArgs &a, int item, int lane, int &b, int &tile, int2 &sq) {
    if (a.batch <= 64) {
        const int2 mine = lane < a.batch ? prompt_rows(a, lane) : make_int2(0, 0);
        const int nt = (mine.y + R - 1) / R;
        int lo = -1, hi = (min(a.max_rows, a.rows) + R - 1) / R;    // tiles at or above lo: more than item; above hi: none
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (wave_sum(max(nt - mid, 0)) > item) lo = mid; else hi = mid;
        }
        if (lo < 0) return false;
        tile = lo;
        const int rank = item - wave_sum(max(nt - lo - 1, 0));
        uint64_t mask = __ballot(nt > lo);
        for (int i = 0; i < rank; ++i) mask &= mask - 1;
        b = __ffsll((unsigned long long)mask) - 1;
        sq = make_int2(__builtin_amdgcn_readlane(mine.x, b), __builtin_amdgcn_readlane(mine.y, b));
        return true;
    }
    int before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        const int2 mine = b0 + lane < a.batch ? prompt_rows(a, b0 + lane) : make_int2(0, 0);
        const int nt = (mine.y + R - 1) / R;
        int run = nt;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(run, d, 64);
            if (lane >= d) run += o;
        }
        const uint64_t mask = __ballot(before + run > item);
        if (mask) {
            const int l = __ffsll((unsigned long long)mask) - 1;
            b = b0 + l;
            tile = before + __builtin_amdgcn_readlane(run, l) - 1 - item;
            sq = make_int2(__builtin_amdgcn_readlane(mine.x, l), __builtin_amdgcn_readlane(mine.y, l));
            return true;
        }
        before += __builtin_amdgcn_readlane(run, 63);
    }
    return false;
}

// Tiles of KT tokens that some row of [lo, hi] sees: those of the sinks, then those
// from the window's first token on.
template <int KT>
struct PromptKeys {
    int sink_tiles, lo_tile, count;
    __device__ __forceinline__ PromptKeys(int lo, int hi, int window, int sinks) {
        lo_tile = window > 0 ? max(lo - window + 1, 0) / KT : 0;
        const int tiles = hi / KT + 1;
        sink_tiles = window > 0 ? min((int)(((int64_t)min(sinks, hi + 1) + KT - 1) / KT), lo_tile) : 0;
        count = sink_tiles + tiles - lo_tile;
    }
    __device__ __forceinline__ int tile(int i) const { return i < sink_tiles ? i : lo_tile + i - sink_tiles; }
};

// 16-byte chunks of a K row in LDS change places by the row's number, so that a read
// of one chunk of 16 (8) rows meets all banks; 64-byte parts of a V row do, so that a
// transposing read of one part of four rows does.
template <int D>
__device__ __forceinline__ int swizzle_k(int c, int row) { return c ^ (row & (D % 128 ? 7 : 15)); }
template <int D>
__device__ __forceinline__ int swizzle_v(int c, int row) { return c ^ ((D % 128 ? (row >> 1) & 1 : row & 3) << 2); }

__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}
// The value, unknown to the compiler: what is made from it in a loop stays there
// (hoisted, the addresses of a tile's reads take more registers than there are).
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

// (m0 among the clobbers is a reserved register, of which the compiler warns)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16 bytes a lane from `from` + at[lane] to LDS address `to` + 16 * lane (from, to: the same
// in every lane; lanes that are switched off load nothing).  In assembly, as the
// compiler would wait for it before any later read of LDS; the caller waits
// (wait_loads) before the barrier that hands the tile over.  The compiler does not see the
// load either, and the base is often the result of a v_readfirstlane just before: such a
// register may be read as an address after five wait states (s_mov, s_nop 3), m0 after one.
__device__ __forceinline__ void load_lds(const void *from, uint32_t at, uint32_t to) {
    const uint64_t f = reinterpret_cast<uint64_t>(from);
    const uint64_t base = (uint64_t)(uint32_t)scalar((int)(f >> 32)) << 32 | (uint32_t)scalar((int)f);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(scalar((int)to)), "v"(at), "s"(base)
                 : "memory", "m0");
}
// ... from an address of each lane's own.
__device__ __forceinline__ void load_lds_wide(const void *from, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(scalar((int)to)), "v"(from) : "memory", "m0");
}
#pragma clang diagnostic pop
// Waits for this wavefront's loads.
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// Source of the chunks that pad a K row.
__device__ const uint4 kZeroChunk = {0, 0, 0, 0};

// The loads of a tile of KT rows of D elements by WAVES wavefronts: 64 chunks an
// instruction, chunk o of the tile's LDS by lane o % 64.  Instruction i + P loads what i
// does, `rows` rows further on.
template <int D, int KT, int WAVES, bool V>
struct TileLoad {
    static constexpr int CH = D / 8, N = KT * CH / 64 / WAVES, P = D % 128 == 64 && D > 64 ? 3 : !V && D == 256 ? 2 : 1;
    static constexpr int rows = P * 64 * WAVES / CH;
    static_assert(N % P == 0 && P * 64 * WAVES % CH == 0 && (V || rows % (D % 128 ? 8 : 16) == 0) && rows % 4 == 0, "the pattern repeats");
    const uint16_t *base;
    int64_t stride;
    uint32_t at[P], row[P];
    bool in[P], pad;
    __device__ __forceinline__ TileLoad(const uint16_t *first, int64_t row_stride, int dim, int wave, int lane)
        : base(first), stride(row_stride), pad(!V && dim < D) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int o = (i * WAVES + wave) * 64 + lane;
            row[i] = o / CH;
            int c = V ? swizzle_v<D>(o % CH, row[i]) : swizzle_k<D>(o % CH, row[i]);
            in[i] = 8 * c < dim;
            if (!in[i]) c = 0;
            at[i] = row[i] * (uint32_t)(2 * row_stride) + 16 * c;
        }
    }
    __device__ __forceinline__ bool whole(int t0, int n) const { return t0 + KT <= n && !pad; }
    // Load i of a whole tile from `from`.
    __device__ __forceinline__ void one(int i, uint32_t tile, const uint16_t *from, int wave) const {
        load_lds(from + (i / P) * rows * stride, at[i % P], tile + (i * WAVES + wave) * 1024);
    }
    // Always N loads a wavefront.  V's padding is its first elements again (its columns
    // are dropped), K's is zero.
    __device__ __forceinline__ void load(uint32_t tile, int t0, int n, int wave) const {
        const uint16_t *from = base + t0 * stride;
        if (whole(t0, n)) {
#pragma unroll
            for (int i = 0; i < N; ++i) one(i, tile, from, wave);
        } else {                                      // rows past the end: the last one
            const uint32_t last = opaque(n - 1 - t0);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t r = row[i % P] + (i / P) * rows;
                const uint32_t o = at[i % P] + (min(r, last) - row[i % P]) * (uint32_t)(2 * stride);
                load_lds_wide(in[i % P] || V ? (const void *)((const char *)from + o) : &kZeroChunk, tile + (i * WAVES + wave) * 1024);
            }
        }
    }
};

// LDS: two tiles of K, two of V.
constexpr int kStages = 2;
template <int DK, int DV, int KT>
constexpr int prompt_lds() { return kStages * KT * (DK + DV) * 2; }

template <int DK, int DV, int WAVES, int KT, int EU>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(EU))) void k_prompt(PromptArgs a) {
    constexpr int R = 32 * WAVES;                     // rows a workgroup
    constexpr int KB = KT / 32, DB = DV / 32;         // 32-token blocks, 32-dim blocks
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    constexpr int kTile = KT * DK * 2, vTile = KT * DV * 2;     // bytes
    const uint32_t k_lds = lds_address(smem), v_lds = k_lds + kStages * kTile;
    const int wave = scalar(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;

    int head, item;
    if (a.per_xcd > 0) {
        const int j = blockIdx.x >> 3;
        head = (blockIdx.x & 7) * a.per_xcd + j % a.per_xcd;
        item = j / a.per_xcd;
    } else {
        head = blockIdx.x % a.heads;
        item = blockIdx.x / a.heads;
    }
    int b, tile;
    int2 sq;
    if (!find_tile<R>(a, item, lane, b, tile, sq)) return;
    const int n = scalar(sq.y), r0 = scalar(sq.x), row0 = scalar(tile) * R;
    const int kvh = head / a.group;
    const uint16_t *kbase = a.k.data + (int64_t)r0 * a.k.row + (int64_t)kvh * a.k.head;
    const uint16_t *vbase = a.v.data + (int64_t)r0 * a.v.row + (int64_t)kvh * a.v.head;
    const PromptKeys<KT> keys(row0, min(row0 + R, n) - 1, a.window, a.sinks);

    const TileLoad<DK, KT, WAVES, false> lk(kbase, a.k.row, a.dk, wave, lane);
    const TileLoad<DV, KT, WAVES, true> lv(vbase, a.v.row, a.dv, wave, lane);
    // Tile i lies in place i % kStages.
    constexpr int kLoads = lk.N + lv.N;
    auto load = [&](int i) {
        const int t0 = keys.tile(i) * KT;
        lk.load(k_lds + (i & (kStages - 1)) * kTile, t0, n, wave);
        lv.load(v_lds + (i & (kStages - 1)) * vTile, t0, n, wave);
    };
    auto load_first = [&] {
        // (a zero that the compiler does not know: it would make the first tiles'
        // addresses once and keep them)
        const int first = scalar((int)opaque(0u));
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i)
            if (first + i < keys.count) load(first + i);
    };
    load_first();

    // the wavefront's rows: column block `wave` of the tile
    const int pos = row0 + 32 * wave + col;
    bf16x8 q[DK / 16];
    const uint16_t *qrow = a.q.data + (int64_t)(r0 + min(pos, n - 1)) * a.q.row + (int64_t)head * a.q.head + 8 * half;
#pragma unroll
    for (int c = 0; c < DK / 16; ++c) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (16 * c + 8 * half < a.dk) w = *reinterpret_cast<const uint4 *>(qrow + 16 * c);
        const uint32_t flip = a.negate ? 0x80008000u : 0u;
        q[c] = __builtin_bit_cast(bf16x8, make_uint4(w.x ^ flip, w.y ^ flip, w.z ^ flip, w.w ^ flip));
    }
    if (a.zero) {                                     // (what is not finite stays: NaN)
#pragma unroll
        for (int c = 0; c < DK / 16; ++c) {
            uint4 w = __builtin_bit_cast(uint4, q[c]);
            auto only_odd = [](uint32_t x) { return (not_finite(x & 0xFFFFu) ? x & 0xFFFFu : 0u) | (not_finite(x >> 16) ? x & 0xFFFF0000u : 0u); };
            q[c] = __builtin_bit_cast(bf16x8, make_uint4(only_odd(w.x), only_odd(w.y), only_odd(w.z), only_odd(w.w)));
        }
    }
    auto sees = [&](int t) { return (t <= pos) & ((a.window == 0) | (t > pos - a.window) | (t < a.sinks)); };

    // The lane's place in a tile of K (row col, chunk half) and of V (row 4 half + lane
    // % 16 / 4, its 8 bytes of the group's 32): the swizzle makes other chunks and parts an exclusive
    // or with a constant.
    const int vrow = 4 * half + ((lane & 15) >> 2);
    const uint32_t k_at = k_lds + col * (2 * DK) + 16 * swizzle_k<DK>(half, col);
    const uint32_t v_at = v_lds + vrow * (2 * DV) + 16 * swizzle_v<DV>(2 * (col >> 4) + ((lane & 3) >> 1), vrow) + 8 * (lane & 1);

    f32x16 o[DB];
    float m, l;                                       // l: this lane's half of the tokens
    f32x16 minus_m;
    bool done = pos >= n;

    for (int pass = 0;; ++pass) {
    const bool slow = pass > 0;
    m = l = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) minus_m[i] = 0.0f;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
    const int w_lo = row0 + 32 * wave, w_hi = w_lo + 31;
    constexpr int CS = DK / 16, kAhead = EU == 1 ? 3 : 2, kVAhead = EU == 1 ? 5 : 4;        // fragments read ahead of their products
    const float bias = pass > 1 ? -kLow : 0.0f;
    f32x16 s[KB];
    bf16x8 p[KB][2], vf[kVAhead + 1];
    // four weights under the present reference, and their sum as rounded
    auto weigh = [&](int qd) {
        const int j = qd / 4, g = qd % 4;
        bf16x2 w[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i >> 1][i & 1] = static_cast<__bf16>(__builtin_amdgcn_exp2f(__builtin_fmaf(s[j][4 * g + i], a.scale, bias)));
            p[j][g >> 1][4 * (g & 1) + i] = w[i >> 1][i & 1];
        }
        l = dot2(w[0], as_bf16x2(0x3F803F80u), l);
        l = dot2(w[1], as_bf16x2(0x3F803F80u), l);
    };
    // Scores of tile `it` less the reference, with the first reads of V and, where LOADS,
    // tile `it` + kStages - 1 on its way into LDS between the products.
    auto score = [&](auto loads, int it, auto read_v) {
        constexpr bool LOADS = decltype(loads)::value;
        const int to = (it + kStages - 1) & (kStages - 1);
        const uint32_t k_to = k_lds + to * kTile, v_to = v_lds + to * vTile;
        const int64_t t_to = LOADS ? keys.tile(it + kStages - 1) * KT : 0;
        const uint16_t *k_from = lk.base + t_to * lk.stride, *v_from = lv.base + t_to * lv.stride;
        const uint32_t at = opaque(k_at + (it & (kStages - 1)) * kTile);
        bf16x8 kf[kAhead + 1][KB];
        auto read_k = [&](int c) {
            constexpr int W = DK % 128 ? 4 : 8;       // steps whose chunks the swizzle mixes
#pragma unroll
            for (int j = 0; j < KB; ++j)
                kf[c % (kAhead + 1)][j] = *reinterpret_cast<const __attribute__((address_space(3))) bf16x8 *>(
                    (at ^ ((c % W) << 5)) + (c / W) * (32 * W) + 32 * j * (2 * DK));
        };
#pragma unroll
        for (int c = 0; c < kAhead; ++c) read_k(c);
#pragma unroll
        for (int c = 0; c < CS; ++c) {
            if (c + kAhead < CS) read_k(c + kAhead);
            if (c >= CS - 2) {
#pragma unroll
                for (int i = 0; i < kVAhead; ++i)
                    if (i % 2 == c - (CS - 2)) read_v(i);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (LOADS) {
#pragma unroll
                for (int i = c * kLoads / CS; i < (c + 1) * kLoads / CS; ++i) {
                    if (i < lk.N) lk.one(i, k_to, k_from, wave);
                    else lv.one(i - lk.N, v_to, v_from, wave);
                }
            }
#pragma unroll
            for (int j = 0; j < KB; ++j)
                s[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[c % (kAhead + 1)][j], q[c], c == 0 ? minus_m : s[j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto mask = [&](int t0) {
        if (t0 + KT - 1 <= w_lo && (a.window == 0 || t0 > w_hi - a.window || t0 + KT <= a.sinks)) return;
        const int base = (int)opaque(t0 + 4 * half), window = a.window > 0 ? min(a.window, 0x7FFFF000) : 0x7FFFF000, sink = a.sinks - base;
        const int here = pos - base, low = here - window;
#pragma unroll
        for (int j = 0; j < KB; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int t = 32 * j + 8 * (i >> 2) + (i & 3);     // the token less base
                s[j][i] = (t <= here) & ((t > low) | (t < sink)) ? s[j][i] : -INFINITY;
            }
    };
    // Moves the reference to the row's maximum where scores exceed it by too much, or
    // where there is none yet.
    auto refer = [&] {
        float mx = s[0][0];
#pragma unroll
        for (int i = 1; i < 16 * KB; ++i) mx = fmaxf(mx, s[i >> 4][i & 15]);
        u32x2 sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(mx), __float_as_uint(mx), false, false);
        mx = fmaxf(__uint_as_float(sw.x), __uint_as_float(sw.y));
        if (!__any(mx * a.scale > kPromptSlack || l == 0.0f)) return;
        // (a half may hold no weight yet: the row has one if either does)
        sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
        const bool fresh = __uint_as_float(sw.x) == 0.0f && __uint_as_float(sw.y) == 0.0f;
        // (a row that needs no move stays as it is, whatever its neighbours do)
        const float up = mx * a.scale > kPromptSlack || (fresh && mx > -INFINITY) ? mx : 0.0f;
        const float alpha = fresh ? 1.0f : __builtin_amdgcn_exp2f(-up * a.scale);
        m += up;
        l *= alpha;
#pragma unroll
        for (int d = 0; d < DB; ++d) o[d] *= alpha;
#pragma unroll
        for (int j = 0; j < KB; ++j) s[j] -= up;
#pragma unroll
        for (int i = 0; i < 16; ++i) minus_m[i] = -m;
    };
    for (int it = scalar((int)opaque(0u)); it < keys.count; ++it) {
        const int t0 = keys.tile(it) * KT;
        wait_loads();
        __syncthreads();                              // and every wavefront is done with the tile before
        const bool next = it + kStages - 1 < keys.count, fast = next && t0 <= w_hi && lk.whole(keys.tile(it + kStages - 1) * KT, n);
        if (next && !fast) load(it + kStages - 1);
        if (slow) {                                   // V without what is not finite (0 * NaN is NaN)
            for (int i = threadIdx.x; i < KT * DV / 2; i += 64 * WAVES) {
                uint32_t &w = reinterpret_cast<uint32_t *>(smem + kStages * kTile + (it & (kStages - 1)) * vTile)[i];
                w = (not_finite(w & 0xFFFFu) ? 0u : w & 0xFFFFu) | (not_finite(w >> 16) ? 0u : w & 0xFFFF0000u);
            }
            __syncthreads();
        }
        if (t0 > w_hi) continue;                      // (no barrier below)
        // token 32 j + 16 e + 8 (i / 4) + 4 half + i % 4 is element i of the product's
        // operands: the order in which S comes out.  Fragment i: j, e, d = i / DB / 2,
        // i / DB % 2, i % DB.
        const uint32_t vat = opaque(v_at + (it & (kStages - 1)) * vTile);
        auto read_v = [&](int i) {
            const int d = i % DB, e = i / DB % 2, j = i / DB / 2;
            union {
                s16x4 h[2];
                bf16x8 v;
            } u;
            constexpr int W = DV % 128 ? 2 : 4;       // parts that the swizzle mixes
#pragma unroll
            for (int z = 0; z < 2; ++z)
                u.h[z] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<__attribute__((address_space(3))) s16x4 *>(
                    (vat ^ ((d % W) << 6)) + (d / W) * (64 * W) + (32 * j + 16 * e + 8 * z) * (2 * DV)));
            vf[i % (kVAhead + 1)] = u.v;
        };
        if (fast) score(std::true_type{}, it, read_v);
        else score(std::false_type{}, it, read_v);
        mask(t0);
        refer();
        // The weights of 16 tokens beside the products of the 16 before: exponentials on the
        // vector units while the matrix cores are busy.
#pragma unroll
        for (int qd = 0; qd < 2; ++qd) weigh(qd);
        __builtin_amdgcn_sched_barrier(0);
        constexpr int PS = 2 * KB * DB;
#pragma unroll
        for (int i = 0; i < PS; ++i) {
            if (i + kVAhead < PS) read_v(i + kVAhead);
            __builtin_amdgcn_sched_barrier(0);
            const int group = i / DB, d = i % DB;
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[i % (kVAhead + 1)], p[group / 2][group % 2], o[d], 0, 0, 0);
            if (group + 1 < 2 * KB) {
#pragma unroll
                for (int z = d * 2 / DB; z < (d + 1) * 2 / DB; ++z) weigh(2 * (group + 1) + z);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // A value that is not finite may come from a token that its row does not see, from one that
    // it does (as infinity times a weight of 0, too), or from a sum past fp32's range: such rows
    // once more without the former two, and if that does not help with smaller weights.  The
    // others are done.
    float far = 0.0f;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) far = __builtin_fmaf(o[d][i], 0.0f, far);
    u32x2 sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(far), __float_as_uint(far), false, false);
    const bool odd = !(__uint_as_float(sw.x) + __uint_as_float(sw.y) == 0.0f);      // (0 * NaN and 0 * inf are NaN)
    const bool write = !done && (!odd || pass == 2);
    done |= write;
    sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
    // (a row sees itself: without a weight all its scores are -inf, and 0 * inf is NaN)
    const float inv = 1.0f / (__uint_as_float(sw.x) + __uint_as_float(sw.y));
    uint16_t *dst = a.out + (int64_t)(r0 + pos) * a.out_stride + (int64_t)head * a.dv + 4 * half;
    if (write) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int at = 32 * d + 8 * g;
                if (at >= a.dv) continue;
                float x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = o[d][4 * g + i] * inv;
                *reinterpret_cast<uint2 *>(dst + at) = make_uint2(f32_to_bf16_bits(x[0]) | (f32_to_bf16_bits(x[1]) << 16),
                                                                  f32_to_bf16_bits(x[2]) | (f32_to_bf16_bits(x[3]) << 16));
            }
    }
    if (slow) {
        // The values that were left out, to the rows that see them, whatever their weights: in
        // memory, where this lane has just written (the sums take all registers).
        static_assert(KT == 64, "a token a lane");
        for (int it = 0; it < keys.count; ++it) {
            const int t0 = keys.tile(it) * KT;
            if (t0 > w_hi) continue;
            bool bad = false;
            if (t0 + lane < n) {
                const uint16_t *vt = vbase + (int64_t)(t0 + lane) * a.v.row;
#pragma unroll 4
                for (int d = 0; d < a.dv; d += 8) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(vt + d);
                    bad = bad || any_not_finite(v.x) || any_not_finite(v.y) || any_not_finite(v.z) || any_not_finite(v.w);
                }
            }
            for (uint64_t tokens = __ballot(bad); tokens; tokens &= tokens - 1) {
                const int t = t0 + __builtin_ctzll(tokens);
                const uint16_t *vt = vbase + (int64_t)t * a.v.row + 4 * half;
                if (!write || !sees(t)) continue;
                for (int d = 0; d < a.dv; d += 8) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(vt + d);
                    if (!any_not_finite(v.x) && !any_not_finite(v.y)) continue;
                    uint2 x = *reinterpret_cast<const uint2 *>(dst + d);
                    x.x = add_not_finite(x.x, v.x);
                    x.y = add_not_finite(x.y, v.y);
                    *reinterpret_cast<uint2 *>(dst + d) = x;
                }
            }
        }
    }
    // (__syncthreads_or would take static LDS, with which two 192 x 128 workgroups miss a CU)
    int *flag = reinterpret_cast<int *>(smem);
    __syncthreads();
    if (threadIdx.x == 0) *flag = 0;
    __syncthreads();
    if (!done) *flag = 1;
    __syncthreads();
    if (*flag == 0) break;
    __syncthreads();
    load_first();
    }
}

template <int DK, int DV, int WAVES, int KT, int EU>
static int launch_prompt(const PromptArgs &a, hipStream_t s, const char *who) {
    constexpr int R = 32 * WAVES;
    const size_t lds = prompt_lds<DK, DV, KT>();
    const void *fn = reinterpret_cast<const void *>(k_prompt<DK, DV, WAVES, KT, EU>);
    if (int rc = allow_lds(fn, lds, who)) return rc;
    // sum over b of ceil(n_b / R)
    const int64_t most = a.max_rows < a.rows ? a.max_rows : a.rows;
    int64_t items = (a.rows + (int64_t)a.batch * (R - 1)) / R;
    const int64_t other = (int64_t)a.batch * ((most + R - 1) / R);
    if (other < items) items = other;
    const int64_t blocks = items * a.heads;
    if (!grid_fits(blocks, 64 * WAVES)) return fail(NVFP4_ERR_UNSUPPORTED, "%s: grid too large", who);
    hipLaunchKernelGGL((k_prompt<DK, DV, WAVES, KT, EU>), dim3((unsigned)blocks), dim3(64 * WAVES), lds, s, a);
    return check_launch(who);
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" int prompt_attention(const nvfp4_head_rows *q, const nvfp4_head_rows *k, const nvfp4_head_rows *v,
                                const int32_t *cu_rows, int32_t batch, int32_t rows, int32_t max_rows, float scale,
                                int32_t window, int32_t sinks, uint16_t *out, int64_t out_row_stride, void *stream) {
    const char *who = "prompt_attention";
    if (batch < 0 || rows < 0 || max_rows < 0)
        return fail(NVFP4_ERR_SHAPE, "%s: batch=%d, rows=%d or max_rows=%d < 0", who, batch, rows, max_rows);
    if (window < 0 || sinks < 0) return fail(NVFP4_ERR_ARG, "%s: window=%d or sinks=%d < 0", who, window, sinks);
    const float scale2 = __builtin_fabsf(scale) * 1.44269504088896340736f;   // for 2^x
    if (!__builtin_isfinite(scale2)) return fail(NVFP4_ERR_ARG, "%s: scale * log2(e) is not finite", who);
    if (batch == 0 || rows == 0 || max_rows == 0) return ok();
    if (int rc = validate_head_rows(q, who, "q")) return rc;
    if (int rc = validate_head_rows(k, who, "k")) return rc;
    if (int rc = validate_head_rows(v, who, "v")) return rc;
    if (q->heads % k->heads || k->heads != v->heads)
        return fail(NVFP4_ERR_SHAPE, "%s: %d q heads, %d k heads and %d v heads: k's and v's must be one number that divides q's", who,
                    q->heads, k->heads, v->heads);
    if (q->dim != k->dim) return fail(NVFP4_ERR_SHAPE, "%s: q has dim %d, k %d", who, q->dim, k->dim);
    if (q->dim % 8 || v->dim % 8 || q->dim > 256 || v->dim > 256)
        return fail(NVFP4_ERR_UNSUPPORTED, "%s: dims %d and %d must be multiples of 8 up to 256", who, q->dim, v->dim);
    // (a tile's rows are addressed in 32 bits)
    if (k->row_stride >= (1 << 23) || v->row_stride >= (1 << 23))
        return fail(NVFP4_ERR_UNSUPPORTED, "%s: row strides of k and v must be below 2^23", who);
    if (!cu_rows || !out) return fail(NVFP4_ERR_ARG, "%s: NULL cu_rows or out", who);
    if (!aligned(cu_rows, 4) || !aligned(out, 16)) return fail(NVFP4_ERR_ALIGN, "%s: cu_rows not 4-byte or out not 16-byte aligned", who);
    if (out_row_stride % 8 || out_row_stride < (int64_t)q->heads * v->dim)
        return fail(NVFP4_ERR_SHAPE, "%s: out_row_stride=%lld must be a multiple of 8 and >= q_heads * v's dim", who,
                    (long long)out_row_stride);
    PromptArgs a;
    a.q = view(q);
    a.k = view(k);
    a.v = view(v);
    a.cu = cu_rows;
    a.batch = batch;
    a.rows = rows;
    a.max_rows = max_rows;
    // (a hidden token's score of -inf times a scale of 0 would be NaN)
    a.scale = scale == 0.0f ? 1.0f : scale2;
    a.negate = scale < 0.0f;
    a.zero = scale == 0.0f;
    a.window = window;
    a.sinks = sinks;
    a.heads = q->heads;
    a.group = q->heads / k->heads;
    a.dk = q->dim;
    a.dv = v->dim;
    a.per_xcd = q->heads % 8 ? 0 : q->heads / 8;
    a.out = out;
    a.out_stride = out_row_stride;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const int dk = q->dim, dv = v->dim;
    // the smallest tile that holds the dims; others are padded with zeros
    if (dk <= 64 && dv <= 64) return launch_prompt<64, 64, 4, 64, 2>(a, s, who);
    if (dk <= 128 && dv <= 128) return launch_prompt<128, 128, 4, 64, 2>(a, s, who);
    if (dk <= 192 && dv <= 128) return launch_prompt<192, 128, 4, 64, 2>(a, s, who);
    if (dk <= 192 && dv <= 192) return launch_prompt<192, 192, 4, 64, 1>(a, s, who);
    return launch_prompt<256, 256, 4, 64, 1>(a, s, who);
}
