// kv8_attention: softmax attention over the paged 8-bit cache (definition in
// nvfp4_mtp.h).
//
// For each row (a query head of one token): o = sum_t p_t v_t / sum_t p_t with
// p_t = exp(scale q.k_t - m), one pass over the keys with the running maximum m
// and sum (both fp32).  Must read: 2 * head_dim bytes a visible token and kv
// head; must compute: 4 * head_dim flop a visible (row, key) pair.
//
// Layout of one wavefront's step: 64 tokens x 16 rows.
//   S^T = K Q^T   v_mfma_f32_16x16x32_bf16, A = K (16 tokens), B = Q^T (16 rows)
//   O^T = V^T P^T the same, A = V^T (16 dims), B = P^T
// so a lane owns one row (its C column) in both products: the row's maximum,
// sum and rescaling are per-lane scalars.  The C layout gives lane group g the
// A rows 4g..4g+3; A row r of token tile t is taken to be token 16 (r / 4) + 4 t +
// r % 4, so group g ends up with the scores of tokens 16 g .. 16 g + 15, which is
// also the k slice that group g supplies to the second product: P goes from one
// product to the other in registers, and a group's 16 tokens lie in one page
// (pages hold 16 tokens or more), so the page's K scale is one factor per lane
// on its scores and its V scale one on its weights.  K rows are read as 16
// contiguous bytes a lane (the k order inside a 64-element chunk is permuted the
// same way in Q), V columns as 16 tokens of one dim, 16 contiguous bytes of the
// transposed page: both operands go from memory to the matrix cores through two
// registers' conversion (E4M3 -> bf16 is exact) with no LDS.
//
// P is rounded to bf16 (2^-9 relative, unbiased) for the matrix cores; its sum
// is of the unrounded values.
#include "kv8.hpp"

namespace nvfp4 {

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

constexpr int kTile = 64;   // tokens a wavefront step

struct AttnArgs {
    HeadRows q;
    KV8 c;
    Seqs s;
    float scale;            // times log2(e)
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

// Eight E4M3 codes -> an MFMA operand (exact).
__device__ __forceinline__ bf16x8 bf16x8_of(uint32_t a, uint32_t b) {
    union {
        bf16x2 h[4];
        bf16x8 v;
    } u;
    u.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
    u.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
    u.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
    u.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
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

// The key range of one row tile as a list of 64-token tiles: the sink tiles,
// then the tiles from the window's first token on.
struct Keys {
    int end;          // tokens >= end are seen by no row
    int sink_tiles, lo_tile, count;
    __device__ __forceinline__ int tile(int v) const { return v < sink_tiles ? v : lo_tile + v - sink_tiles; }
};
__device__ __forceinline__ Keys key_range(int pos_lo, int pos_hi, int window, int sinks) {
    Keys k;
    k.end = max(pos_hi + 1, 0);
    k.lo_tile = window > 0 ? max(pos_lo - window + 1, 0) / kTile : 0;
    const int tiles = (k.end + kTile - 1) / kTile;
    k.sink_tiles = window > 0 ? min((min(sinks, k.end) + kTile - 1) / kTile, k.lo_tile) : 0;
    k.count = k.end > 0 ? k.sink_tiles + tiles - k.lo_tile : 0;
    return k;
}

// Page ids of the lane's K tokens and of its group's tokens in one tile.
struct PageIds {
    int k, v;
};

template <int D, int RT>
struct Wave {
    static constexpr int C = D / 64, DT = D / 16;
    bf16x8 q[RT][C][2];
    f32x4 o[RT][DT];
    float m[RT], l[RT];
    int pos[RT];
    uint4 kf[4][C], vf[DT];
    float ks, vs;
    bool page_ok;

    const AttnArgs &a;
    const int32_t *table;
    int h, lane, last_page;
    Keys keys;

    __device__ __forceinline__ Wave(const AttnArgs &args) : a(args) {}

    __device__ __forceinline__ PageIds load_ids(int tile) const {
        const int t = tile * kTile, kg = (lane & 15) >> 2, vg = lane >> 4;
        return PageIds{table[min((t + 16 * kg) >> a.c.lp, last_page)], table[min((t + 16 * vg) >> a.c.lp, last_page)]};
    }
    __device__ __forceinline__ bool id_ok(int id) const { return id >= 0 && id < a.c.pages; }
    __device__ __forceinline__ void load_k(int tile, PageIds id) {
        const int r = lane & 15, t = tile * kTile + 16 * (r >> 2), off = (t & ((1 << a.c.lp) - 1)) + (r & 3);
        const uint8_t *p = a.c.k + ((int64_t)(id_ok(id.k) ? id.k : 0) * a.c.heads + h) * ((int64_t)D << a.c.lp) +
                           off * D + 16 * (lane >> 4);
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int c = 0; c < C; ++c) kf[tt][c] = *reinterpret_cast<const uint4 *>(p + tt * 4 * D + c * 64);
    }
    __device__ __forceinline__ void load_v(int tile, PageIds id) {
        const int t = tile * kTile + 16 * (lane >> 4), off = t & ((1 << a.c.lp) - 1);
        const uint8_t *p = a.c.v + ((int64_t)(id_ok(id.v) ? id.v : 0) * a.c.heads + h) * ((int64_t)D << a.c.lp) +
                           ((lane & 15) << a.c.lp) + off;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) vf[dt] = *reinterpret_cast<const uint4 *>(p + ((dt * 16) << a.c.lp));
    }
    __device__ __forceinline__ void load_scales(PageIds id, uint32_t &sk, uint32_t &sv) const {
        const int64_t at = (int64_t)(id_ok(id.v) ? id.v : 0) * a.c.heads + h;
        sk = a.c.ks[at];
        sv = a.c.vs[at];
    }

    __device__ __forceinline__ void scores(f32x4 (&s)[RT][4]) const {
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) s[rt][tt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const bf16x8 lo = bf16x8_of(kf[tt][c].x, kf[tt][c].y), hi = bf16x8_of(kf[tt][c].z, kf[tt][c].w);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    s[rt][tt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, q[rt][c][0], s[rt][tt], 0, 0, 0);
                    s[rt][tt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, q[rt][c][1], s[rt][tt], 0, 0, 0);
                }
            }
        }
    }
    __device__ __forceinline__ bool sees(int t, int p) const {
        return page_ok && t <= p && (a.window == 0 || t > p - a.window || t < a.sinks);
    }
    // Scores -> weights (times the page's V scale) in bf16; running maximum and
    // sum, and the accumulators' rescaling when a maximum grew.
    template <bool MASK>
    __device__ __forceinline__ void softmax(int tile, f32x4 (&s)[RT][4], bf16x8 (&p)[RT][2]) {
        const float f = a.scale * ks;
        const int t0 = tile * kTile + 16 * (lane >> 4);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float mx = -INFINITY;
#pragma unroll
            for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = s[rt][tt][i] * f;
                    if (MASK) v = sees(t0 + 4 * tt + i, pos[rt]) ? v : -INFINITY;
                    s[rt][tt][i] = v;
                    mx = fmaxf(mx, v);
                }
            const float mn = fmaxf(m[rt], groups_max(mx));
            const float ref = mn == -INFINITY ? 0.0f : mn;
            if (__any(mn > m[rt])) {
                const float alpha = __builtin_amdgcn_exp2f(m[rt] - ref);
                l[rt] *= alpha;
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) o[rt][dt] *= alpha;
                m[rt] = mn;
            }
            float sum = 0.0f;
            union {
                __bf16 e[16];
                bf16x8 v[2];
            } u;
#pragma unroll
            for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float w = __builtin_amdgcn_exp2f(s[rt][tt][i] - ref);
                    sum += w;
                    u.e[4 * tt + i] = static_cast<__bf16>(w * vs);
                }
            l[rt] += sum;
            p[rt][0] = u.v[0];
            p[rt][1] = u.v[1];
        }
    }
    __device__ __forceinline__ void weigh(const bf16x8 (&p)[RT][2]) {
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
            const bf16x8 lo = bf16x8_of(vf[dt].x, vf[dt].y), hi = bf16x8_of(vf[dt].z, vf[dt].w);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                o[rt][dt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, p[rt][0], o[rt][dt], 0, 0, 0);
                o[rt][dt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, p[rt][1], o[rt][dt], 0, 0, 0);
            }
        }
    }
    // A tile that some row sees only in part may hold a NaN in V that the row
    // must not get (0 * NaN is NaN): such codes are counted per (dim, row) over
    // the tokens the row sees, and left out of the product.
    __device__ __forceinline__ void weigh_masked(int tile, const bf16x8 (&p)[RT][2]) {
        uint32_t any = 0;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) any |= nan_bytes(vf[dt].x) | nan_bytes(vf[dt].y) | nan_bytes(vf[dt].z) | nan_bytes(vf[dt].w);
        if (__any(any != 0)) {
            const int t0 = tile * kTile + 16 * (lane >> 4);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                union {
                    __bf16 e[16];
                    bf16x8 v[2];
                } u;
#pragma unroll
                for (int j = 0; j < 16; ++j) u.e[j] = static_cast<__bf16>(sees(t0 + j, pos[rt]) ? 1.0f : 0.0f);
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) {
                    f32x4 n = {0.0f, 0.0f, 0.0f, 0.0f};
                    n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16x8_of(nan_ones(vf[dt].x), nan_ones(vf[dt].y)), u.v[0], n, 0, 0, 0);
                    n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16x8_of(nan_ones(vf[dt].z), nan_ones(vf[dt].w)), u.v[1], n, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[rt][dt][i] = n[i] > 0.0f ? NAN : o[rt][dt][i];
                }
            }
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
                vf[dt] = make_uint4(without_nan(vf[dt].x), without_nan(vf[dt].y), without_nan(vf[dt].z), without_nan(vf[dt].w));
        }
        weigh(p);
    }
};

// Floats of one partial result: 16 rows x D sums (C layout), 16 maxima, 16 sums.
template <int D>
constexpr int part_floats() { return 16 * D + 32; }

// Writes rows of C layout values: lane (g, r) holds dims 16 dt + 4 g + i of
// row `row`.
__device__ __forceinline__ void store_out(uint16_t *at, f32x4 v) {
    *reinterpret_cast<uint2 *>(at) = make_uint2(f32_to_bf16_bits(v[0]) | (f32_to_bf16_bits(v[1]) << 16),
                                                f32_to_bf16_bits(v[2]) | (f32_to_bf16_bits(v[3]) << 16));
}

// One workgroup: 16 * RT rows of one (sequence, kv head), one piece of their
// keys; its four wavefronts take every fourth tile and join through LDS.
template <int D, int RT>
__global__ __launch_bounds__(256) void k_attn(AttnArgs a) {
    constexpr int C = D / 64, DT = D / 16;
    const int split = blockIdx.x % a.splits;
    int w = blockIdx.x / a.splits;
    const int rtile = w % a.row_tiles;
    w /= a.row_tiles;
    const int h = w % a.c.heads, b = w / a.c.heads;
    const Seq sq = load_seq(a.s, b, a.c.lp);
    const int rows = min(sq.n, a.s.max_rows) * a.group, row0 = rtile * 16 * RT;
    if (row0 >= rows) return;
    const int wave = threadIdx.x >> 6;
    const int shift = sq.len - sq.n;

    Wave<D, RT> x(a);
    x.lane = threadIdx.x & 63;
    x.h = h;
    x.table = a.s.table + (int64_t)b * a.s.max_pages;
    x.keys = key_range(shift + row0 / a.group, shift + (min(row0 + 16 * RT, rows) - 1) / a.group, a.window, a.sinks);
    x.last_page = max(x.keys.end - 1, 0) >> a.c.lp;
    const int per = (x.keys.count + a.splits - 1) / a.splits;
    const int v0 = split * per, v1 = min(v0 + per, x.keys.count);
    const int pos_lo = shift + row0 / a.group, pos_hi = x.keys.end - 1;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int row = min(row0 + rt * 16 + (x.lane & 15), rows - 1);
        const int i = row / a.group;
        x.pos[rt] = shift + i;
        x.m[rt] = -INFINITY;
        x.l[rt] = 0.0f;
        const uint16_t *src = a.q.data + (int64_t)(sq.r0 + i) * a.q.row + (int64_t)(h * a.group + row % a.group) * a.q.head +
                              16 * (x.lane >> 4);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            x.q[rt][c][0] = *reinterpret_cast<const bf16x8 *>(src + 64 * c);
            x.q[rt][c][1] = *reinterpret_cast<const bf16x8 *>(src + 64 * c + 8);
        }
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) x.o[rt][dt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    int v = v0 + wave;
    if (v < v1) {
        int tile = x.keys.tile(v);
        PageIds id = x.load_ids(tile);
        x.load_k(tile, id);
        x.load_v(tile, id);
        uint32_t sk, sv;
        x.load_scales(id, sk, sv);
        bool ok = x.id_ok(id.v);
        int next = x.keys.tile(min(v + 4, v1 - 1));
        PageIds nid = x.load_ids(next);
        for (; v < v1; v += 4) {
            f32x4 s[RT][4];
            bf16x8 p[RT][2];
            x.ks = kv8_scale(sk);
            x.vs = kv8_scale(sv);
            x.page_ok = ok;
            const int cur = tile;
            x.scores(s);
            // the next tile's K and scales, then the ids after it (past the
            // last tile the last one is loaded again)
            tile = next;
            id = nid;
            x.load_k(tile, id);
            x.load_scales(id, sk, sv);
            ok = x.id_ok(id.v);
            next = x.keys.tile(min(v + 8, v1 - 1));
            nid = x.load_ids(next);
            __builtin_amdgcn_sched_barrier(0);
            const int t0 = cur * kTile;
            const bool whole = t0 + kTile - 1 <= pos_lo && (a.window == 0 || t0 > pos_hi - a.window || t0 + kTile <= a.sinks) &&
                               !__any(!x.page_ok);
            if (whole) {
                x.template softmax<false>(cur, s, p);
                x.weigh(p);
            } else {
                x.template softmax<true>(cur, s, p);
                x.weigh_masked(cur, p);
            }
            x.load_v(tile, id);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // join the four wavefronts: the common maximum, then each wavefront sums a
    // quarter of the dims
    __shared__ float sm[4][16], sl[4][16];
    __shared__ f32x4 so[3][DT][64];
    const int r = x.lane & 15;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const float lw = groups_sum(x.l[rt]);
        if (rt > 0) __syncthreads();
        if (x.lane < 16) {
            sm[wave][r] = x.m[rt];
            sl[wave][r] = lw;
        }
        __syncthreads();
        float mx = sm[0][r];
        for (int i = 1; i < 4; ++i) mx = fmaxf(mx, sm[i][r]);
        const float ref = mx == -INFINITY ? 0.0f : mx;
        float sum = 0.0f;
        for (int i = 0; i < 4; ++i) sum += sl[i][r] * __builtin_amdgcn_exp2f(sm[i][r] - ref);
        const float f = __builtin_amdgcn_exp2f(x.m[rt] - ref);
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
            x.o[rt][dt] *= f;
            const int owner = dt & 3;
            if (owner != wave) so[wave - (wave > owner)][dt][x.lane] = x.o[rt][dt];
        }
        __syncthreads();
        const int row = row0 + rt * 16 + r, i = row / a.group, hq = h * a.group + row % a.group;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        uint16_t *dst = a.out + (int64_t)(sq.r0 + i) * a.out_stride + (int64_t)hq * D + 4 * (x.lane >> 4);
        float *part = a.part + (int64_t)(((((int64_t)b * a.c.heads + h) * a.row_tiles + rtile) * RT + rt) * a.splits + split) *
                                   part_floats<D>();
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
            if ((dt & 3) != wave) continue;
            f32x4 t = x.o[rt][dt];
            for (int k = 0; k < 3; ++k) t += so[k][dt][x.lane];
            if (a.splits > 1) {
                *reinterpret_cast<f32x4 *>(part + dt * 256 + x.lane * 4) = t;
            } else if (row < rows) {
                store_out(dst + dt * 16, t * inv);
            }
        }
        if (a.splits > 1 && threadIdx.x < 16) {
            part[16 * D + r] = mx;
            part[16 * D + 16 + r] = sum;
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
    p.rt = rows <= 16 ? 1 : 2;
    p.row_tiles = (int)((rows + 16 * p.rt - 1) / (16 * p.rt));
    const int64_t units = (int64_t)s->batch * c->kv_heads * p.row_tiles;
    const int64_t cap = (int64_t)s->max_pages * c->page_tokens;
    const int64_t len = s->max_kv_len > 0 && s->max_kv_len < cap ? s->max_kv_len : cap;
    const int64_t tiles = (len + kTile - 1) / kTile;
    int64_t want = ((int64_t)num_cus() * 2 + units - 1) / units;
    want = want < tiles / 4 ? want : tiles / 4;
    p.splits = (int)(want < 1 ? 1 : want);
    p.blocks = units * p.splits;
    p.ws = p.splits > 1 ? (size_t)(units * p.rt * p.splits) * (16 * c->head_dim + 32) * sizeof(float) : 0;
    return p;
}

template <int D>
static void launch_attn(const AttnPlan &p, const AttnArgs &a, int batch, hipStream_t s) {
    if (p.rt == 1)
        hipLaunchKernelGGL((k_attn<D, 1>), dim3((unsigned)p.blocks), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((k_attn<D, 2>), dim3((unsigned)p.blocks), dim3(256), 0, s, a);
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
    a.scale = scale * 1.44269504088896340736f;
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
