// Shared pieces of the 8-bit KV cache operators: device views of the host
// descriptors and the host-side checks.
#pragma once

#include "common.hpp"

namespace nvfp4 {

typedef __attribute__((ext_vector_type(2))) float f32x2;

// Rows of heads; strides in elements.
struct HeadRows {
    uint16_t *data;
    int64_t row, head;
};

struct KV8 {
    uint8_t *k, *ks, *v, *vs;
    int pages, heads;
    int lp;   // log2(page_tokens)
};

struct Seqs {
    const int32_t *cu, *lens, *table;
    int batch, rows, max_rows, max_pages;
};

// One sequence's rows and length, bounded as the header says.
struct Seq {
    int r0, n, len;
};
__device__ __forceinline__ Seq load_seq(const Seqs &s, int b, int lp) {
    Seq q;
    const int a = s.cu[b], z = s.cu[b + 1];
    q.r0 = min(max(a, 0), s.rows);
    q.n = min(max(z, q.r0), s.rows) - q.r0;
    const int64_t cap = (int64_t)s.max_pages << lp;
    q.len = (int)min((int64_t)max(s.lens[b], 0), min(cap, (int64_t)0x7FFFFF00));
    return q;
}

// Scale byte -> exponent of its power of two, at most 2^119: a larger one would make
// codes infinite in bf16, and a hidden token's infinity times its weight of 0 is NaN.
constexpr int kMaxExp = 119;
__device__ __forceinline__ int kv8_exp(uint32_t b) { return (int)min(b, kMaxExp + 127u) - 127; }
// ... -> a float with that exponent field, the scale operand of a conversion.
__device__ __forceinline__ float kv8_scale(uint32_t b) { return __uint_as_float(min(b, kMaxExp + 127u) << 23); }

inline HeadRows view(const nvfp4_head_rows *r) {
    return r ? HeadRows{r->data, r->row_stride, r->head_stride} : HeadRows{nullptr, 0, 0};
}
inline KV8 view(const nvfp4_kv8_cache *c) {
    return KV8{c->k_codes, c->k_scales, c->v_codes, c->v_scales, c->num_pages, c->kv_heads,
               __builtin_ctz((unsigned)c->page_tokens)};
}
inline Seqs view(const nvfp4_kv8_seqs *s) {
    return Seqs{s->cu_rows, s->kv_lens, s->block_table, s->batch, s->rows, s->max_rows, s->max_pages};
}

int validate_head_rows(const nvfp4_head_rows *r, const char *who, const char *what);
int validate_kv8_cache(const nvfp4_kv8_cache *c, const char *who);
int validate_kv8_seqs(const nvfp4_kv8_seqs *s, const char *who);

}  // namespace nvfp4
