// moe_w4a16_gemm: the routed-expert FFN of moe_w4a16_gemv for any number of rows
// (definition in nvfp4_mtp.h).
//
// The (token, slot) pairs are sorted by expert (moe_sort.hip), which also leaves a
// list of row tiles, none across two experts.  Two W4A16 products over those tiles:
// gate and up together, reading the tokens' rows through the sorted order, with
// a = bf16(silu(g) u) in the epilogue; then down over the sorted rows of a, in fp32.
// A last launch adds each token's rows with their weights, in slot order.
#include "moe_sort.hpp"

namespace nvfp4 {

constexpr int kMoeBM = 128, kMoeBN = 128, kMoeBK = 64;

// As the prompt GEMM's: 16-byte chunk c of a 128-byte row r at place c ^ (r % 8).
__device__ __forceinline__ int moe_off(int r, int c) { return r * 128 + 16 * (c ^ (r & 7)); }

template <int SEL>
__device__ __forceinline__ uint32_t moe_dq2(uint32_t word, float sf) {
    typedef __attribute__((ext_vector_type(2))) float f32x2;
    const f32x2 f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, SEL);
    const uint32_t lo = __float_as_uint(f.x * sf), hi = __float_as_uint(f.y * sf);
    return __builtin_amdgcn_perm(hi, lo, 0x07060302u);   // upper halves: exact bf16
}

struct MoeGemmArgs {
    const MoeTile *tiles;
    const int32_t *tile_count, *offsets, *order;
    int top_k, cols;              // column tiles
    int n, k;                     // output columns (of one expert), products
    const uint16_t *x;            // [m][k] through order, or [pairs][k]
    const uint8_t *codes[2], *scales[2];
    const nvfp4_global *global[2];
    void *y;                      // bf16 [pairs][n] or fp32 [pairs][n]
};

// One row tile (128 rows of one expert) by 128 weight rows, dequantized on the way into LDS
// as in the prompt GEMM, whose 128-row rate it reaches (4096 rows of top-8 of 256 experts:
// 393 tiles, 65% full, gate and up 291 us on average and 268 at least, 725 and 787 TFLOP/s
// counting whole tiles).  Measured against the latter there: 64-row tiles 314 us, 256-row tiles 359, 128-k steps 314, four
// wavefronts a SIMD 392 (they spill), the weights of four steps asked for at once 294, a row
// tile's columns on one XCD 268.  GATE_UP: 64 rows of
// gate and the same 64 of up, in turn by 16, so that a wavefront has both of an output.
template <bool GATE_UP>
__global__ __launch_bounds__(256) void k_moe_gemm(MoeGemmArgs a) {
    constexpr int BM = kMoeBM, WM = 2, WN = 2;                  // wavefronts along rows and columns
    constexpr int MI = BM / 16 / WM, NJ = kMoeBN / 16 / WN;
    constexpr int XQ = BM * 8 / 256;                            // 16-byte chunks of x a thread
    __shared__ __attribute__((aligned(16))) uint8_t lds_a[BM * 128];
    __shared__ __attribute__((aligned(16))) uint8_t lds_b[kMoeBN * 128];
    const int th = threadIdx.x, lane = th & 63, wave = th >> 6;
    const int wm = wave / WN, wn = wave % WN;
    const int t = blockIdx.x / a.cols, nt = blockIdx.x % a.cols;
    if (t >= *a.tile_count) return;
    const MoeTile tile = a.tiles[t];
    const int e = tile.expert, row0 = tile.row, rows = min(a.offsets[e + 1] - row0, BM);
    const int n0 = nt * (GATE_UP ? 64 : 128);

    // staging: chunk th % 8 of the rows th / 8 + 32 q of x; half a weight row
    const int xch = th & 7;
    const uint16_t *xp[XQ];
    bool xin[XQ];
#pragma unroll
    for (int q = 0; q < XQ; ++q) {
        const int r = (th >> 3) + 32 * q;
        xin[q] = r < rows;
        const int s = row0 + (xin[q] ? r : 0);
        xp[q] = a.x + (int64_t)(GATE_UP ? a.order[s] / a.top_k : s) * a.k + 8 * xch;
    }
    const int brow = th >> 1, bpart = th & 1;
    const int which = GATE_UP ? (brow >> 4) & 1 : 0;
    const int wrow = GATE_UP ? n0 + 16 * (brow >> 5) + (brow & 15) : n0 + brow;
    const bool wval = wrow < a.n;
    const int64_t wat = (int64_t)e * a.n + (wval ? wrow : 0);
    const uint8_t *crow = a.codes[which] + wat * (a.k >> 1), *srow = a.scales[which] + wat * (a.k >> 4);

    uint4 xr[XQ], cr;
    uint32_t sr;
    auto load_step = [&](int k0) {
        const bool kin = k0 + 8 * xch < a.k;
#pragma unroll
        for (int q = 0; q < XQ; ++q) xr[q] = xin[q] && kin ? *reinterpret_cast<const uint4 *>(xp[q] + k0) : make_uint4(0, 0, 0, 0);
        const int kb = k0 + 32 * bpart;
        cr = make_uint4(0, 0, 0, 0);
        sr = 0;
        if (wval && kb < a.k) {
            cr = *reinterpret_cast<const uint4 *>(crow + (kb >> 1));
            sr = *reinterpret_cast<const uint16_t *>(srow + (kb >> 4));
        }
    };
    f32x4 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // 16-row blocks WM i + wm of the tile; those past its rows are left out
    const int blocks = (rows + 15) / 16, mi = (blocks - wm + WM - 1) / WM;
    load_step(0);
    for (int k0 = 0; k0 < a.k; k0 += kMoeBK) {
        __syncthreads();
#pragma unroll
        for (int q = 0; q < XQ; ++q)
            *reinterpret_cast<uint4 *>(lds_a + moe_off((th >> 3) + 32 * q, xch)) = xr[q];
        typedef __attribute__((ext_vector_type(2))) float f32x2;
        const f32x2 sf = __builtin_amdgcn_cvt_pk_f32_fp8((int)sr, false);
        const uint32_t w[4] = {cr.x, cr.y, cr.z, cr.w};
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const float f = d >= 2 ? sf.y : sf.x;
            *reinterpret_cast<uint4 *>(lds_b + moe_off(brow, 4 * bpart + d)) =
                make_uint4(moe_dq2<0>(w[d], f), moe_dq2<1>(w[d], f), moe_dq2<2>(w[d], f), moe_dq2<3>(w[d], f));
        }
        __syncthreads();
        if (k0 + kMoeBK < a.k) load_step(k0 + kMoeBK);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const int kc = 4 * ks + (lane >> 4);
            bf16x8 bf[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j) bf[j] = *reinterpret_cast<const bf16x8 *>(lds_b + moe_off(16 * (NJ * wn + j) + (lane & 15), kc));
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                if (i >= mi) break;
                const bf16x8 af = *reinterpret_cast<const bf16x8 *>(lds_a + moe_off(16 * (WM * i + wm) + (lane & 15), kc));
#pragma unroll
                for (int j = 0; j < NJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af, bf[j], acc[i][j], 0, 0, 0);
            }
        }
    }
    const float dec0 = a.global[0][e].dec, dec1 = GATE_UP ? a.global[1][e].dec : 0.0f;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 16 * (WM * i + wm) + 4 * (lane >> 4) + r;
            if (row >= rows) continue;
            const int64_t at = (int64_t)(row0 + row) * a.n;
#pragma unroll
            for (int j = 0; j < NJ; j += GATE_UP ? 2 : 1) {
                if (GATE_UP) {
                    const int col = n0 + 16 * ((NJ * wn + j) >> 1) + (lane & 15);
                    const float g = acc[i][j][r] * dec0, u = acc[i][j + 1][r] * dec1;
                    if (col < a.n) static_cast<uint16_t *>(a.y)[at + col] = (uint16_t)f32_to_bf16_bits(g / (1.0f + expf(-g)) * u);
                } else {
                    const int col = n0 + 16 * (NJ * wn + j) + (lane & 15);
                    if (col < a.n) static_cast<float *>(a.y)[at + col] = acc[i][j][r] * dec0;
                }
            }
        }
}

// The same for tiles of few rows, whose time is the weights': 16 MT rows of one expert by
// 64 columns of gate and up (128 of down), a wavefront's 32 weight rows straight from
// memory into matrix operands.  A lane holds 32 consecutive codes of one weight row, so
// that an instruction reads 64 bytes of each of 16 rows and four cover whole lines (with
// the 64-k steps of k_moe_gemm, 32 bytes at a time, the lines and their scales were
// fetched three times over: 40 rows' gate and up 104 us).  The products take the k of a
// 128-k step in the order that follows from that, and x is read from LDS in the same one.
// The next 512 k of weights are on their way during the products of the present ones.
constexpr int kRowsK = 512, kRowsPitch = kRowsK * 2 + 16;      // bytes of an LDS row of x

template <int MT, bool GATE_UP>
__global__ __launch_bounds__(256) void k_moe_rows(MoeGemmArgs a) {
    constexpr int BM = 16 * MT, XQ = BM * (kRowsK / 8) / 256;   // 16-byte chunks of x a thread
    __shared__ __attribute__((aligned(16))) uint8_t lds[BM * kRowsPitch];
    const int th = threadIdx.x, lane = th & 63, wave = th >> 6, col = lane & 15, g = lane >> 4;
    const int t = blockIdx.x / a.cols, nt = blockIdx.x % a.cols;
    if (t >= *a.tile_count) return;
    const MoeTile tile = a.tiles[t];
    const int e = tile.expert, row0 = tile.row, rows = min(a.offsets[e + 1] - row0, BM);
    // weight rows of the wavefront's two blocks of 16: gate and up, or two of down
    const int n0 = nt * (GATE_UP ? 64 : 128) + wave * (GATE_UP ? 16 : 32);
    const uint8_t *crow[2], *srow[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int n = n0 + (GATE_UP ? 0 : 16 * b) + col, which = GATE_UP ? b : 0;
        const int64_t at = (int64_t)e * a.n + min(n, a.n - 1);
        crow[b] = a.codes[which] + at * (a.k >> 1) + 16 * g;
        srow[b] = a.scales[which] + at * (a.k >> 4) + 2 * g;
    }
    // x: chunk th % 64 of the rows th / 64 + 4 q; past the tile's rows zeros
    const int xch = th & 63;
    const uint16_t *xp[XQ];
#pragma unroll
    for (int q = 0; q < XQ; ++q) {
        const int r = (th >> 6) + 4 * q;
        xp[q] = nullptr;
        if (r < rows) xp[q] = a.x + (int64_t)(GATE_UP ? a.order[row0 + r] / a.top_k : row0 + r) * a.k + 8 * xch;
    }
    uint4 xr[XQ], cr[2][4];
    uint32_t sr[2][4];
    auto load_x = [&](int k0) {
#pragma unroll
        for (int q = 0; q < XQ; ++q)
            xr[q] = xp[q] && k0 + 8 * xch < a.k ? *reinterpret_cast<const uint4 *>(xp[q] + k0) : make_uint4(0, 0, 0, 0);
    };
    auto load_w = [&](int k0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = k0 + 128 * i + 32 * g < a.k;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                cr[b][i] = make_uint4(0, 0, 0, 0);
                sr[b][i] = 0;
                if (in) {
                    cr[b][i] = *reinterpret_cast<const uint4 *>(crow[b] + (k0 >> 1) + 64 * i);
                    sr[b][i] = *reinterpret_cast<const uint16_t *>(srow[b] + (k0 >> 4) + 8 * i);
                }
            }
        }
    };
    f32x4 acc[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    load_x(0);
    load_w(0);
    for (int k0 = 0; k0 < a.k; k0 += kRowsK) {
        __syncthreads();
#pragma unroll
        for (int q = 0; q < XQ; ++q) *reinterpret_cast<uint4 *>(lds + ((th >> 6) + 4 * q) * kRowsPitch + 16 * xch) = xr[q];
        __syncthreads();
        uint4 c[2][4];
        uint32_t sc[2][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                c[b][i] = cr[b][i];
                sc[b][i] = sr[b][i];
            }
        if (k0 + kRowsK < a.k) {
            load_x(k0 + kRowsK);
            load_w(k0 + kRowsK);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            typedef __attribute__((ext_vector_type(2))) float f32x2;
            f32x2 sf[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) sf[b] = __builtin_amdgcn_cvt_pk_f32_fp8((int)sc[b][i], false);
#pragma unroll
            for (int u = 0; u < 4; ++u) {             // eight codes of the lane's 32
                bf16x8 w[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const uint32_t word = u == 0 ? c[b][i].x : u == 1 ? c[b][i].y : u == 2 ? c[b][i].z : c[b][i].w;
                    const float f = u >= 2 ? sf[b].y : sf[b].x;
                    w[b] = __builtin_bit_cast(bf16x8, make_uint4(moe_dq2<0>(word, f), moe_dq2<1>(word, f), moe_dq2<2>(word, f), moe_dq2<3>(word, f)));
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const bf16x8 x = *reinterpret_cast<const bf16x8 *>(lds + (16 * m + col) * kRowsPitch + 2 * (128 * i + 32 * g + 8 * u));
                    acc[m][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w[0], acc[m][0], 0, 0, 0);
                    acc[m][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w[1], acc[m][1], 0, 0, 0);
                }
            }
        }
    }
    const float dec0 = a.global[0][e].dec, dec1 = GATE_UP ? a.global[1][e].dec : dec0;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 16 * m + 4 * g + r;
            if (row >= rows) continue;
            const int64_t at = (int64_t)(row0 + row) * a.n;
            if (GATE_UP) {
                const float gate = acc[m][0][r] * dec0, up = acc[m][1][r] * dec1;
                if (n0 + col < a.n) static_cast<uint16_t *>(a.y)[at + n0 + col] = (uint16_t)f32_to_bf16_bits(gate / (1.0f + expf(-gate)) * up);
            } else {
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    if (n0 + 16 * b + col < a.n) static_cast<float *>(a.y)[at + n0 + 16 * b + col] = acc[m][b][r] * dec0;
            }
        }
}

struct MoeGemmLayout {
    size_t hist, offsets, order, place, count, tiles, act, down, bytes;
    int bm;
    int64_t max_tiles;
};
static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

static MoeGemmLayout moe_gemm_layout(int m, int top_k, const nvfp4_moe_weights *e) {
    MoeGemmLayout l;
    const int64_t pairs = (int64_t)m * top_k, E = e->num_experts;
    const int64_t avg = pairs / E;
    // A tile costs its weights once however few rows it has, and a row past the last tile
    // another one.  The whole call at top-8 of 256, hidden 2048, with tiles of 16, 32 and 128
    // rows, us (rows an expert: inter 512; inter 1024):
    //     1: 106 121 150; 196 215 277       8: 161 184 228; 279 307 414
    //    12: 173 189 233; 303 314 422      16: 204 194 238; 360 321 433
    //    32: 311 265 265; 581 456 472      48: 419 352 295; 777 596 530
    //   128: 970 752 505; 1821 1287 838
    // (k_moe_rows with 64 rows, one wavefront a SIMD, lost to one of them everywhere: 32 rows
    // an expert 358 and 633, 48 407 and 702.)
    l.bm = avg <= 12 ? 16 : avg <= 32 ? 32 : kMoeBM;
    // sum over the experts of ceil(n_e / bm)
    l.max_tiles = pairs / l.bm + (pairs < E ? pairs : E);
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t was = at;
        at += up256(n);
        return was;
    };
    l.hist = take(moe_sort_hist_bytes(m, (int)E));
    l.offsets = take((E + 1) * 4);
    l.order = take(pairs * 4);
    l.place = take(pairs * 4);
    l.count = take(4);
    l.tiles = take(l.max_tiles * sizeof(MoeTile));
    l.act = take(pairs * e->inter * 2);
    l.down = take(pairs * e->hidden * 4);
    l.bytes = at;
    return l;
}

template <bool GATE_UP>
static void launch_moe_gemm(int bm, int64_t blocks, const MoeGemmArgs &a, hipStream_t s) {
    const dim3 g((unsigned)blocks), b(256);
    if (bm == 16) hipLaunchKernelGGL((k_moe_rows<1, GATE_UP>), g, b, 0, s, a);
    else if (bm == 32) hipLaunchKernelGGL((k_moe_rows<2, GATE_UP>), g, b, 0, s, a);
    else hipLaunchKernelGGL((k_moe_gemm<GATE_UP>), g, b, 0, s, a);
}

static int check_experts(const nvfp4_moe_weights *e, const char *who) {
    if (!e) return fail(NVFP4_ERR_ARG, "%s: NULL experts", who);
    if (e->hidden < 32 || e->hidden % 32 || e->inter < 32 || e->inter % 32)
        return fail(NVFP4_ERR_SHAPE, "%s: hidden=%d and inter=%d must be positive multiples of 32", who, e->hidden, e->inter);
    return NVFP4_OK;
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" size_t moe_w4a16_gemm_workspace_bytes(int32_t m, int32_t top_k, const nvfp4_moe_weights *e) {
    const char *who = "moe_w4a16_gemm_workspace_bytes";
    if (check_experts(e, who) || check_moe_sizes(m, e->num_experts, top_k, who)) return 0;
    return moe_gemm_layout(m, top_k, e).bytes;
}

extern "C" int moe_w4a16_gemm(const uint16_t *x_bf16, int32_t m, const float *router_logits, int32_t top_k, const nvfp4_moe_weights *e,
                              void *y, int32_t y_dtype, int32_t *topk_ids, float *topk_w, void *workspace, size_t ws_bytes,
                              void *stream) {
    const char *who = "moe_w4a16_gemm";
    if (int rc = check_experts(e, who)) return rc;
    if (int rc = check_moe_sizes(m, e->num_experts, top_k, who)) return rc;
    if (y_dtype != NVFP4_OUT_F32 && y_dtype != NVFP4_OUT_BF16) return fail(NVFP4_ERR_ARG, "%s: unknown y_dtype %d", who, y_dtype);
    if (m == 0) return ok();
    if (!x_bf16 || !router_logits || !y || !topk_ids || !topk_w) return fail(NVFP4_ERR_ARG, "%s: NULL pointer", who);
    const uint8_t *w[6] = {e->gate_codes, e->up_codes, e->down_codes, e->gate_scales, e->up_scales, e->down_scales};
    const nvfp4_global *g[3] = {e->gate_global, e->up_global, e->down_global};
    for (int i = 0; i < 6; ++i) {
        if (!w[i]) return fail(NVFP4_ERR_ARG, "%s: NULL codes or scales", who);
        if (!aligned(w[i], i < 3 ? 16 : 2)) return fail(NVFP4_ERR_ALIGN, "%s: codes not 16-byte or scales not 2-byte aligned", who);
    }
    for (int i = 0; i < 3; ++i)
        if (!g[i] || !aligned(g[i], 4)) return fail(g[i] ? NVFP4_ERR_ALIGN : NVFP4_ERR_ARG, "%s: a global is NULL or not 4-byte aligned", who);
    if (!aligned(x_bf16, 16) || !aligned(y, 16) || !aligned(router_logits, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4))
        return fail(NVFP4_ERR_ALIGN, "%s: x or y not 16-byte aligned, or another pointer not 4-byte", who);
    const MoeGemmLayout l = moe_gemm_layout(m, top_k, e);
    if (!workspace || ws_bytes < l.bytes)
        return fail(NVFP4_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", who, workspace ? ws_bytes : 0, l.bytes);
    if (!aligned(workspace, 256)) return fail(NVFP4_ERR_ALIGN, "%s: workspace not 256-byte aligned", who);
    const int gcols = (e->inter + 63) / 64, dcols = (e->hidden + 127) / 128;
    if (!grid_fits(l.max_tiles * gcols, 256) || !grid_fits(l.max_tiles * dcols, 256))
        return fail(NVFP4_ERR_UNSUPPORTED, "%s: grid too large", who);
    char *ws = static_cast<char *>(workspace);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    SortArgs so{};
    so.logits = router_logits;
    so.m = m;
    so.experts = e->num_experts;
    so.top_k = top_k;
    so.ids = topk_ids;
    so.w = topk_w;
    so.offsets = reinterpret_cast<int32_t *>(ws + l.offsets);
    so.order = reinterpret_cast<int32_t *>(ws + l.order);
    so.place = reinterpret_cast<int32_t *>(ws + l.place);
    so.hist = reinterpret_cast<int32_t *>(ws + l.hist);
    so.tiles = reinterpret_cast<MoeTile *>(ws + l.tiles);
    so.tile_count = reinterpret_cast<int32_t *>(ws + l.count);
    so.tile_rows = l.bm;
    launch_moe_sort(so, s);
    MoeGemmArgs a{};
    a.tiles = so.tiles;
    a.tile_count = so.tile_count;
    a.offsets = so.offsets;
    a.order = so.order;
    a.top_k = top_k;
    a.cols = gcols;
    a.n = e->inter;
    a.k = e->hidden;
    a.x = x_bf16;
    for (int i = 0; i < 2; ++i) {
        a.codes[i] = w[i];
        a.scales[i] = w[3 + i];
        a.global[i] = g[i];
    }
    a.y = ws + l.act;
    launch_moe_gemm<true>(l.bm, l.max_tiles * gcols, a, s);
    a.cols = dcols;
    a.n = e->hidden;
    a.k = e->inter;
    a.x = reinterpret_cast<const uint16_t *>(ws + l.act);
    a.codes[0] = w[2];
    a.scales[0] = w[5];
    a.global[0] = g[2];
    a.y = ws + l.down;
    launch_moe_gemm<false>(l.bm, l.max_tiles * dcols, a, s);
    launch_moe_combine(ws + l.down, false, m, e->hidden, top_k, so.place, topk_w, y, y_dtype == NVFP4_OUT_BF16, s);
    return check_launch(who);
}
