// Tokens sorted by expert and back: top-k routing with a stable counting sort of the
// (token, slot) pairs, rows out to their sorted places, weighted rows back, and the
// gradient of the way back (definitions in nvfp4_mtp.h).
//
// Sort: counts of every block's tokens, then places from the counts of all blocks; ranks
// within a block from ballots, so that the order does not depend on timing.  8191 tokens of
// 256 experts, top-8: 11 us to route and count (bound by the selections' instructions: some 600
// a token), 8 us to place.  Blocks of 16 tokens: 12 and 11 us, of 64: 17 and 7.
// Rows out, back and the gradient move every byte once (a large copy reaches 5.1 TB/s): 8191
// tokens of 2048 to eight places 51 us, 5.9 TB/s, and back 57 us, 5.2; the gradient of 2000
// tokens of 7168, 104 us, 4.7.
#include "moe_sort.hpp"

namespace nvfp4 {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kCountBlocks = 256, kPlaceBlocks = 2;

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    return max(max(a, b), max(c, d));
}

// Ascending with the float, -0 as +0; NaN 1, so that it comes after -inf; 0 is nothing.
__device__ __forceinline__ uint32_t order_key(float f) {
    if (f != f) return 1u;
    const uint32_t u = __float_as_uint(f == 0.0f ? 0.0f : f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return k == 1u ? NAN : __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// One token's top_k experts by one wavefront: lane j gets the j-th.  Lane l holds
// experts [l PER, (l + 1) PER), the larger logit first and the lower number first among
// equals, so that the lowest lane whose head is the maximum has the lowest expert.
template <int PER>
__device__ __forceinline__ void choose(const float *lg, int experts, int top_k, int lane, float &my_v, int &my_i) {
    uint32_t v[PER];
    int id[PER];
    float f[PER];
    if (PER % 4 == 0 && experts % 4 == 0 && (reinterpret_cast<uintptr_t>(lg) & 15) == 0) {
#pragma unroll
        for (int j = 0; j < PER; j += 4) {
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (lane * PER + j < experts) x = *reinterpret_cast<const float4 *>(lg + lane * PER + j);
            f[j] = x.x;
            f[j + 1 < PER ? j + 1 : 0] = x.y;
            f[j + 2 < PER ? j + 2 : 0] = x.z;
            f[j + 3 < PER ? j + 3 : 0] = x.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < PER; ++j) f[j] = lane * PER + j < experts ? lg[lane * PER + j] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        id[j] = lane * PER + j;
        v[j] = id[j] < experts ? order_key(f[j]) : 0u;
    }
#pragma unroll
    for (int r = 0; r < PER; ++r)                     // (odd and even neighbours in turn; equals keep their order)
#pragma unroll
        for (int j = r & 1; j + 1 < PER; j += 2) {
            const bool sw = v[j + 1] > v[j];
            const uint32_t tv = v[j];
            const int ti = id[j];
            v[j] = sw ? v[j + 1] : v[j];
            id[j] = sw ? id[j + 1] : id[j];
            v[j + 1] = sw ? tv : v[j + 1];
            id[j + 1] = sw ? ti : id[j + 1];
        }
    uint32_t mine = 0;
    my_i = 0;
    for (int s = 0; s < top_k; ++s) {                 // (top_k <= experts: some head is not 0)
        const uint32_t mx = wave_max_u32(v[0]);
        const int wl = (int)__builtin_ctzll(__ballot(v[0] == mx));
        const int wid = __builtin_amdgcn_readlane(id[0], wl);
        if (lane == s) {
            mine = mx;
            my_i = wid;
        }
        const bool pop = lane == wl;
#pragma unroll
        for (int j = 0; j + 1 < PER; ++j) {
            v[j] = pop ? v[j + 1] : v[j];
            id[j] = pop ? id[j + 1] : id[j];
        }
        v[PER - 1] = pop ? 0u : v[PER - 1];
    }
    my_v = key_value(mine);
}

// ... and their weights, softmax over the chosen logits; into memory, and counted.
template <int PER>
__device__ __forceinline__ void route(const SortArgs &a, int t, int lane, int *hist) {
    float v;
    int i;
    choose<PER>(a.logits + (int64_t)t * a.experts, a.experts, a.top_k, lane, v, i);
    const float top = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 0));
    const float e = lane < a.top_k ? expf(v - top) : 0.0f;
    float sum = row16_sum(e);                         // (top_k <= 16: the first lanes)
    sum = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(sum)));
    if (lane < a.top_k) {
        a.ids[(int64_t)t * a.top_k + lane] = i;
        a.w[(int64_t)t * a.top_k + lane] = e / sum;
        atomicAdd(&hist[i], 1);
    }
}

// Tokens [t0, t1): routed, or their given experts counted, into hist (LDS).
__device__ __forceinline__ void route_block(const SortArgs &a, int t0, int t1, int *hist) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < a.experts; e += kSortThreads) hist[e] = 0;
    __syncthreads();
    if (a.logits) {
        const int per = (a.experts + 63) / 64;
        for (int t = t0 + wave; t < t1; t += kSortWaves) {
            if (per <= 1) route<1>(a, t, lane, hist);
            else if (per <= 2) route<2>(a, t, lane, hist);
            else if (per <= 4) route<4>(a, t, lane, hist);
            else if (per <= 8) route<8>(a, t, lane, hist);
            else route<16>(a, t, lane, hist);
        }
    } else {
        for (int64_t p = (int64_t)t0 * a.top_k + tid; p < (int64_t)t1 * a.top_k; p += kSortThreads) {
            const int i = a.ids[p];
            if (i >= 0 && i < a.experts) atomicAdd(&hist[i], 1);
        }
    }
    __syncthreads();
}

__global__ __launch_bounds__(kSortThreads) void k_sort_count(SortArgs a) {
    __shared__ int hist[kMaxExperts];
    const int t0 = blockIdx.x * a.per_block;
    route_block(a, t0, min(t0 + a.per_block, a.m), hist);
    // (counts of two experts a word: 2^23 pairs over kCountBlocks blocks fit 16 bits)
    const int words = (a.experts + 1) / 2;
    for (int c = threadIdx.x; c < words; c += kSortThreads)
        a.hist[(int64_t)blockIdx.x * words + c] = hist[2 * c] | (2 * c + 1 < a.experts ? hist[2 * c + 1] << 16 : 0);
}

// Exclusive prefix sum over the workgroup's threads.
__device__ __forceinline__ int scan_threads(int v, int *waves) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int run = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(run, d, 64);
        if (lane >= d) run += o;
    }
    if (lane == 63) waves[wave] = run;
    __syncthreads();
    for (int i = 0; i < wave; ++i) run += waves[i];
    __syncthreads();
    return run - v;
}

// Places of the pairs of tokens [t0, t1).  Thread e has expert e's rows in all (count)
// and in the blocks before (before); first: this block also writes what is of the whole
// call.  A round takes 1024 pairs: a wavefront finds the equals among its 64 (a ballot
// a bit of the number), and counts per wavefront give the rank among the round's.
__device__ __forceinline__ void place_block(const SortArgs &a, int t0, int t1, int count, int before, bool first) {
    __shared__ int base[kMaxExperts], waves[kSortWaves];
    __shared__ uint16_t cnt[kSortWaves][kMaxExperts];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int start = scan_threads(tid < a.experts ? count : 0, waves);
    base[tid] = start + before;
    if (first) {
        if (tid < a.experts) a.offsets[tid] = start;
        if (tid == a.experts - 1) a.offsets[a.experts] = start + count;
        if (a.tiles) {
            const int n = tid < a.experts ? (count + a.tile_rows - 1) / a.tile_rows : 0;
            const int at = scan_threads(n, waves);
            for (int i = 0; i < n; ++i) a.tiles[at + i] = MoeTile{tid, start + i * a.tile_rows};
            if (tid == kSortThreads - 1) *a.tile_count = at + n;
        }
    }
    for (int w = 0; w < kSortWaves; ++w)
        if (tid < a.experts) cnt[w][tid] = 0;
    const int64_t p1 = (int64_t)t1 * a.top_k;
    int bits = 1;
    while ((1 << bits) < a.experts) ++bits;
    for (int64_t p0 = (int64_t)t0 * a.top_k; p0 < p1; p0 += kSortThreads) {
        __syncthreads();
        const int64_t p = p0 + tid;
        int id = p < p1 ? a.ids[p] : -1;
        const bool ok = id >= 0 && id < a.experts;
        uint64_t same = __ballot(ok);
        for (int i = 0; i < bits; ++i) {
            const uint64_t ones = __ballot(id >> i & 1);
            same &= id >> i & 1 ? ones : ~ones;
        }
        const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
        if (ok && rank == 0) cnt[wave][id] = (uint16_t)__builtin_popcountll(same);
        __syncthreads();
        if (ok) {
            int at = base[id] + rank;
            for (int w = 0; w < wave; ++w) at += cnt[w][id];
            a.place[p] = at;
            a.order[at] = (int)p;
        } else if (p < p1) {
            a.place[p] = -1;
        }
        if (p0 + kSortThreads < p1) {
            __syncthreads();
            if (tid < a.experts) {
                int add = 0;
                for (int w = 0; w < kSortWaves; ++w) {
                    add += cnt[w][tid];
                    cnt[w][tid] = 0;
                }
                base[tid] += add;
            }
        }
    }
}

// A block places the pairs of kPlaceBlocks counting blocks.  The counts of all blocks are
// summed by all threads, a word (two experts) of every (1024 / words)-th block each.
__global__ __launch_bounds__(kSortThreads) void k_sort_place(SortArgs a, int blocks) {
    __shared__ int all[kMaxExperts], before[kMaxExperts];
    const int tid = threadIdx.x, words = (a.experts + 1) / 2, groups = kSortThreads / words;
    all[tid] = before[tid] = 0;
    __syncthreads();
    const int c = tid % words, first = (int)blockIdx.x * kPlaceBlocks;
    if (tid < groups * words) {
        int n0 = 0, n1 = 0, b0 = 0, b1 = 0;
#pragma unroll 8
        for (int b = tid / words; b < blocks; b += groups) {
            const uint32_t h = (uint32_t)a.hist[(int64_t)b * words + c];
            n0 += h & 0xFFFFu;
            n1 += h >> 16;
            b0 += b < first ? h & 0xFFFFu : 0;
            b1 += b < first ? h >> 16 : 0;
        }
        atomicAdd(&all[2 * c], n0);
        atomicAdd(&before[2 * c], b0);
        if (2 * c + 1 < a.experts) {
            atomicAdd(&all[2 * c + 1], n1);
            atomicAdd(&before[2 * c + 1], b1);
        }
    }
    __syncthreads();
    const int64_t t0 = (int64_t)first * a.per_block, t1 = t0 + (int64_t)kPlaceBlocks * a.per_block;
    place_block(a, (int)t0, (int)min(t1, (int64_t)a.m), all[tid], before[tid], blockIdx.x == 0);
}

// Few tokens: all of it in one workgroup.
__global__ __launch_bounds__(kSortThreads) void k_sort_one(SortArgs a) {
    __shared__ int hist[kMaxExperts];
    route_block(a, 0, a.m, hist);
    place_block(a, 0, a.m, threadIdx.x < a.experts ? hist[threadIdx.x] : 0, 0, true);
}

// Tokens sorted by one workgroup, in one launch: 8 tokens of 256 experts 6.4 us (two launches
// 8.0), 16 7.8 (9.4), 24 9.0 (9.5), 32 11.1 (9.8).
constexpr int kOneTokens = 24;

// A token a wavefront, until that makes more than kCountBlocks blocks, whose counts every
// placing block reads.
static int sort_per_block(int m) {
    const int per = (m + kCountBlocks - 1) / kCountBlocks;
    return per < kSortWaves ? kSortWaves : per;
}

size_t moe_sort_hist_bytes(int m, int experts) {
    if (m <= kOneTokens) return 0;
    const int per = sort_per_block(m);
    return (size_t)((m + per - 1) / per) * ((experts + 1) / 2) * sizeof(int32_t);
}

void launch_moe_sort(SortArgs a, hipStream_t s) {
    if (a.m <= kOneTokens) {
        hipLaunchKernelGGL(k_sort_one, dim3(1), dim3(kSortThreads), 0, s, a);
        return;
    }
    a.per_block = sort_per_block(a.m);
    const int blocks = (a.m + a.per_block - 1) / a.per_block;
    hipLaunchKernelGGL(k_sort_count, dim3(blocks), dim3(kSortThreads), 0, s, a);
    hipLaunchKernelGGL(k_sort_place, dim3((blocks + kPlaceBlocks - 1) / kPlaceBlocks), dim3(kSortThreads), 0, s, a, blocks);
}

// ------------------------------------------------------------- rows out and back
// Item (token, 16-byte chunk of its row): read once, written to its top_k places.
// (a place outside the pairs is passed over, here and below)
__global__ __launch_bounds__(256) void k_moe_gather(const uint4 *__restrict__ x, int64_t items, int chunks, int top_k, uint32_t pairs,
                                                    const int32_t *__restrict__ place, uint4 *__restrict__ out) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / chunks;
        const int c = (int)(i - t * chunks);
        const uint4 v = x[i];
        for (int j = 0; j < top_k; ++j) {
            const uint32_t p = (uint32_t)place[t * top_k + j];
            if (p < pairs) out[(int64_t)p * chunks + c] = v;
        }
    }
}

// Eight consecutive elements as fp32, and back.
template <bool BF16>
struct Row8;
template <>
struct Row8<true> {
    static __device__ __forceinline__ void load(const void *p, int64_t at, float (&v)[8]) {
        const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ void store(void *p, int64_t at, const float (&v)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = f32_to_bf16_bits(v[2 * i]) | (f32_to_bf16_bits(v[2 * i + 1]) << 16);
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <>
struct Row8<false> {
    static __device__ __forceinline__ void load(const void *p, int64_t at, float (&v)[8]) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
        const float4 a = q[0], b = q[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    static __device__ __forceinline__ void store(void *p, int64_t at, const float (&v)[8]) {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
};

// y = sum over the slots, in slot order, of w * the pair's row; fp32 sums.
template <bool YS, bool Y>
__global__ __launch_bounds__(256) void k_moe_combine(const void *__restrict__ ys, int64_t items, int chunks, int top_k, uint32_t pairs,
                                                     const int32_t *__restrict__ place, const float *__restrict__ w,
                                                     void *__restrict__ y) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / chunks;
        const int c = (int)(i - t * chunks);
        float acc[8] = {};
#pragma unroll 4
        for (int j = 0; j < top_k; ++j) {
            const uint32_t p = (uint32_t)place[t * top_k + j];
            if (p >= pairs) continue;
            const float f = w ? w[t * top_k + j] : 1.0f;
            float v[8];
            Row8<YS>::load(ys, ((int64_t)p * chunks + c) * 8, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = __builtin_fmaf(f, v[e], acc[e]);
        }
        Row8<Y>::store(y, i * 8, acc);
    }
}

// One workgroup a token: dys rows w * dy, and dw = <ys row, dy>.  dys may be ys.
template <bool YS, bool Y, int K>
__global__ __launch_bounds__(256) void k_moe_combine_grad(const void *__restrict__ dy, const void *ys, int m, int chunks,
                                                          int top_k, const int32_t *__restrict__ place, const float *__restrict__ w,
                                                          void *dys, float *__restrict__ dw) {
    __shared__ float part[4][K];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t t = blockIdx.x;
    const uint32_t pairs = (uint32_t)m * (uint32_t)top_k;
    uint32_t p[K];
    float f[K], acc[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        p[j] = j < top_k ? (uint32_t)place[t * top_k + j] : pairs;
        f[j] = j < top_k && w ? w[t * top_k + j] : 1.0f;
        acc[j] = 0.0f;
    }
    for (int c = tid; c < chunks; c += 256) {
        float g[8];
        Row8<Y>::load(dy, (t * chunks + c) * 8, g);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (p[j] >= pairs) continue;
            float v[8];
            const int64_t at = ((int64_t)p[j] * chunks + c) * 8;
            Row8<YS>::load(ys, at, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[j] = __builtin_fmaf(v[e], g[e], acc[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = f[j] * g[e];
            Row8<YS>::store(dys, at, v);
        }
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
        float s = acc[j];
#pragma unroll
        for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d, 64);
        if (lane == 0) part[wave][j] = s;
    }
    __syncthreads();
    if (tid < top_k) dw[t * top_k + tid] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
}

static unsigned row_blocks(int64_t items) {
    const int64_t want = (items + 255) / 256, cap = (int64_t)num_cus() * 32;
    return (unsigned)(want < cap ? want : cap);
}

void launch_moe_combine(const void *ys, bool ys_bf16, int m, int hidden, int top_k, const int32_t *place, const float *w,
                        void *y, bool y_bf16, hipStream_t s) {
    const int chunks = hidden / 8;
    const int64_t items = (int64_t)m * chunks;
    const uint32_t pairs = (uint32_t)m * (uint32_t)top_k;
    const dim3 grid(row_blocks(items)), block(256);
    if (ys_bf16 && y_bf16) hipLaunchKernelGGL((k_moe_combine<true, true>), grid, block, 0, s, ys, items, chunks, top_k, pairs, place, w, y);
    else if (ys_bf16) hipLaunchKernelGGL((k_moe_combine<true, false>), grid, block, 0, s, ys, items, chunks, top_k, pairs, place, w, y);
    else if (y_bf16) hipLaunchKernelGGL((k_moe_combine<false, true>), grid, block, 0, s, ys, items, chunks, top_k, pairs, place, w, y);
    else hipLaunchKernelGGL((k_moe_combine<false, false>), grid, block, 0, s, ys, items, chunks, top_k, pairs, place, w, y);
}

template <bool YS, bool Y>
static void launch_grad(const void *dy, const void *ys, int m, int chunks, int top_k, const int32_t *place, const float *w,
                        void *dys, float *dw, hipStream_t s) {
    if (top_k <= 8) hipLaunchKernelGGL((k_moe_combine_grad<YS, Y, 8>), dim3(m), dim3(256), 0, s, dy, ys, m, chunks, top_k, place, w, dys, dw);
    else hipLaunchKernelGGL((k_moe_combine_grad<YS, Y, 16>), dim3(m), dim3(256), 0, s, dy, ys, m, chunks, top_k, place, w, dys, dw);
}

int check_moe_sizes(int m, int experts, int top_k, const char *who) {
    if (m < 0 || experts < 1 || experts > kMaxExperts)
        return fail(NVFP4_ERR_SHAPE, "%s: m=%d (need >= 0) or num_experts=%d (need 1..%d)", who, m, experts, kMaxExperts);
    if (top_k < 1 || top_k > kMaxTopK || top_k > experts)
        return fail(NVFP4_ERR_SHAPE, "%s: top_k=%d (need 1..min(num_experts, %d))", who, top_k, kMaxTopK);
    if ((int64_t)m * top_k > (1 << 23)) return fail(NVFP4_ERR_UNSUPPORTED, "%s: %d x %d pairs are too many", who, m, top_k);
    return NVFP4_OK;
}

static int check_rows(int m, int hidden, int top_k, const char *who) {
    if (m < 0 || hidden < 8 || hidden % 8) return fail(NVFP4_ERR_SHAPE, "%s: m=%d hidden=%d (need hidden a multiple of 8)", who, m, hidden);
    if (top_k < 1 || top_k > kMaxTopK) return fail(NVFP4_ERR_SHAPE, "%s: top_k=%d (need 1..%d)", who, top_k, kMaxTopK);
    if ((int64_t)m * top_k > (1 << 23)) return fail(NVFP4_ERR_UNSUPPORTED, "%s: %d x %d pairs are too many", who, m, top_k);
    return NVFP4_OK;
}

static int check_dtype(int dtype, const char *who, const char *what) {
    if (dtype != NVFP4_OUT_F32 && dtype != NVFP4_OUT_BF16) return fail(NVFP4_ERR_ARG, "%s: unknown %s %d", who, what, dtype);
    return NVFP4_OK;
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" size_t moe_sort_workspace_bytes(int32_t m, int32_t num_experts, int32_t top_k) {
    if (check_moe_sizes(m, num_experts, top_k, "moe_sort_workspace_bytes")) return 0;
    const size_t n = moe_sort_hist_bytes(m, num_experts);
    return n > 256 ? n : 256;
}

extern "C" int moe_sort(const float *router_logits, int32_t m, int32_t num_experts, int32_t top_k, int32_t *topk_ids, float *topk_w,
                        int32_t *offsets, int32_t *order, int32_t *place, void *workspace, size_t ws_bytes, void *stream) {
    const char *who = "moe_sort";
    if (int rc = check_moe_sizes(m, num_experts, top_k, who)) return rc;
    if (!offsets || (m > 0 && (!topk_ids || !order || !place || (router_logits && !topk_w))))
        return fail(NVFP4_ERR_ARG, "%s: NULL pointer", who);
    const void *all[] = {router_logits, topk_ids, topk_w, offsets, order, place, workspace};
    for (const void *x : all)
        if (!aligned(x, 4)) return fail(NVFP4_ERR_ALIGN, "%s: a pointer is not 4-byte aligned", who);
    const size_t need = moe_sort_hist_bytes(m, num_experts);
    if (need && (!workspace || ws_bytes < need))
        return fail(NVFP4_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", who, workspace ? ws_bytes : 0, need);
    SortArgs a{};
    a.logits = router_logits;
    a.m = m;
    a.experts = num_experts;
    a.top_k = top_k;
    a.ids = topk_ids;
    a.w = topk_w;
    a.offsets = offsets;
    a.order = order;
    a.place = place;
    a.hist = static_cast<int32_t *>(workspace);
    launch_moe_sort(a, reinterpret_cast<hipStream_t>(stream));
    return check_launch(who);
}

extern "C" int moe_gather(const void *x, int32_t x_dtype, int32_t m, int32_t hidden, int32_t top_k, const int32_t *place, void *out,
                          void *stream) {
    const char *who = "moe_gather";
    if (int rc = check_dtype(x_dtype, who, "x_dtype")) return rc;
    if (int rc = check_rows(m, hidden, top_k, who)) return rc;
    if (m == 0) return ok();
    if (!x || !place || !out) return fail(NVFP4_ERR_ARG, "%s: NULL pointer", who);
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(place, 4))
        return fail(NVFP4_ERR_ALIGN, "%s: x or out not 16-byte aligned, or place not 4-byte", who);
    const int chunks = hidden / 8 * (x_dtype == NVFP4_OUT_F32 ? 2 : 1);
    const int64_t items = (int64_t)m * chunks;
    hipLaunchKernelGGL(k_moe_gather, dim3(row_blocks(items)), dim3(256), 0, reinterpret_cast<hipStream_t>(stream),
                       static_cast<const uint4 *>(x), items, chunks, top_k, (uint32_t)m * (uint32_t)top_k, place, static_cast<uint4 *>(out));
    return check_launch(who);
}

extern "C" int moe_combine(const void *ys, int32_t ys_dtype, int32_t m, int32_t hidden, int32_t top_k, const int32_t *place,
                           const float *topk_w, void *y, int32_t y_dtype, void *stream) {
    const char *who = "moe_combine";
    if (int rc = check_dtype(ys_dtype, who, "ys_dtype")) return rc;
    if (int rc = check_dtype(y_dtype, who, "y_dtype")) return rc;
    if (int rc = check_rows(m, hidden, top_k, who)) return rc;
    if (m == 0) return ok();
    if (!ys || !place || !y) return fail(NVFP4_ERR_ARG, "%s: NULL pointer", who);
    if (!aligned(ys, 16) || !aligned(y, 16) || !aligned(place, 4) || !aligned(topk_w, 4))
        return fail(NVFP4_ERR_ALIGN, "%s: ys or y not 16-byte aligned, or place or topk_w not 4-byte", who);
    launch_moe_combine(ys, ys_dtype == NVFP4_OUT_BF16, m, hidden, top_k, place, topk_w, y, y_dtype == NVFP4_OUT_BF16,
                       reinterpret_cast<hipStream_t>(stream));
    return check_launch(who);
}

extern "C" int moe_combine_grad(const void *dy, int32_t dy_dtype, const void *ys, int32_t ys_dtype, int32_t m, int32_t hidden,
                                int32_t top_k, const int32_t *place, const float *topk_w, void *dys, float *dw, void *stream) {
    const char *who = "moe_combine_grad";
    if (int rc = check_dtype(ys_dtype, who, "ys_dtype")) return rc;
    if (int rc = check_dtype(dy_dtype, who, "dy_dtype")) return rc;
    if (int rc = check_rows(m, hidden, top_k, who)) return rc;
    if (m == 0) return ok();
    if (!dy || !ys || !place || !dys || !dw) return fail(NVFP4_ERR_ARG, "%s: NULL pointer", who);
    if (!aligned(dy, 16) || !aligned(ys, 16) || !aligned(dys, 16) || !aligned(place, 4) || !aligned(topk_w, 4) || !aligned(dw, 4))
        return fail(NVFP4_ERR_ALIGN, "%s: dy, ys or dys not 16-byte aligned, or place, topk_w or dw not 4-byte", who);
    if (!grid_fits(m, 256)) return fail(NVFP4_ERR_UNSUPPORTED, "%s: grid too large", who);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const int chunks = hidden / 8;
    const bool yb = ys_dtype == NVFP4_OUT_BF16, db = dy_dtype == NVFP4_OUT_BF16;
    if (yb && db) launch_grad<true, true>(dy, ys, m, chunks, top_k, place, topk_w, dys, dw, s);
    else if (yb) launch_grad<true, false>(dy, ys, m, chunks, top_k, place, topk_w, dys, dw, s);
    else if (db) launch_grad<false, true>(dy, ys, m, chunks, top_k, place, topk_w, dys, dw, s);
    else launch_grad<false, false>(dy, ys, m, chunks, top_k, place, topk_w, dys, dw, s);
    return check_launch(who);
}
