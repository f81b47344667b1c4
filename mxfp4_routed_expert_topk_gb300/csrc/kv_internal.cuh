// Internal declarations of the serving operators: the paged key/value cache, the
// attention over it, and draft verification.
#pragma once

#include "moe_internal.cuh"

namespace moe {

constexpr int kMaxLen = 1 << 30;  // tokens of a sequence

// Device-side view of a paged cache (layout in moe.h).
struct KvView {
    uint8_t *base;
    uint64_t page_rec;   // bytes of a page's record (all layers)
    uint64_t layer_rec;  // bytes of one layer in it
    uint64_t off_scale;  // scales in a layer's record = 2 * heads * page * dim
    int n_pages, n_layers, heads, dim, page;

    __device__ uint8_t *layer_at(int p, int layer) const {
        return base + (uint64_t)p * page_rec + (uint64_t)layer * layer_rec;
    }
    // codes of (page, layer, side, head): [page][dim] bytes
    __device__ uint8_t *codes(int p, int layer, int side, int head) const {
        return layer_at(p, layer) + (uint64_t)(side * heads + head) * (uint64_t)(page * dim);
    }
    __device__ float *scale(int p, int layer, int side, int head) const {
        return reinterpret_cast<float *>(layer_at(p, layer) + off_scale) + side * heads + head;
    }
};

// Four E4M3 codes -> fp32 (exact).
__device__ __forceinline__ void e4m3x4_to_float(uint32_t c, float (&f)[4]) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
    const float2 x = __half22float2(*reinterpret_cast<__half2 *>(&lo));
    const float2 y = __half22float2(*reinterpret_cast<__half2 *>(&hi));
    f[0] = x.x;
    f[1] = x.y;
    f[2] = y.x;
    f[3] = y.y;
}

// Two values -> two E4M3 codes (round to nearest even, saturating at +-448, NaN kept);
// the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2_rn(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4_rn(float a, float b, float c, float d) {
    return e4m3x2_rn(a, b) | (e4m3x2_rn(c, d) << 16);
}

struct KvAppendArgs {
    KvView kv;
    int layer;
    const uint16_t *k, *v;
    size_t ldk, ldv;
    int rows;
    const int32_t *cu_rows, *start, *page_table;
    int table_width, seqs;
    StatusWord *st;
    int units;  // (side, head) pairs a block takes (set by the launch)
};
cudaError_t launch_kv_append(KvAppendArgs a, cudaStream_t st);

struct KvAttentionArgs {
    KvView kv;
    int layer;
    const uint16_t *q;
    size_t ldq;
    int rows, heads_q;
    const int32_t *cu_rows, *kv_len, *page_table;
    int table_width, seqs, max_rows;
    float scale;
    uint16_t *out;
    size_t ldo;
    float *lse;
    StatusWord *st;
};
cudaError_t kv_attention_workspace_bytes(const KvView &kv, int max_rows, int heads_q, size_t *bytes);
cudaError_t launch_kv_attention(const KvAttentionArgs &a, void *ws, cudaStream_t st);
cudaError_t set_wait_limit_kv_attention(uint64_t ns);

struct VerifyArgs {
    const void *p, *q;  // (greedy: p = the logits)
    size_t ldp, ldq;
    int bf16;           // element type: 0 fp32, 1 bf16
    int rows, vocab;
    const int32_t *tokens, *cu_rows;
    int seqs;
    const float *u_accept, *u_sample;
    int32_t *accepted, *next;
    StatusWord *st;
};
size_t verify_workspace_bytes(int seqs, int rows);
cudaError_t launch_verify_sampled(const VerifyArgs &a, void *ws, cudaStream_t st);
cudaError_t launch_verify_greedy(const VerifyArgs &a, void *ws, cudaStream_t st);

// Rows [lo, hi) of sequence b, checked against the call's row count: false (an empty
// range) if they are not an ascending pair within 0..rows.
__device__ __forceinline__ bool seq_rows(const int32_t *cu_rows, int b, int rows, int &lo, int &hi) {
    lo = cu_rows[b];
    hi = cu_rows[b + 1];
    if (lo >= 0 && lo <= hi && hi <= rows) return true;
    lo = hi = 0;
    return false;
}

}  // namespace moe

struct moe_kv {
    moe::KvView v;
};
