// Cache attention of sequences that share prefixes: a prompt that several continuations are sampled
// from, or a document that many requests ask about.
//
// Every row of a group sees all of its prefix, so a row's result is
//
//   o = (2^(e1 - m) o1 + 2^(e2 - m) o2) / (2^(e1 - m) + 2^(e2 - m)),  m = max(e1, e2)
//
// with o1, o2 its attention over the prefix and over the sequence's own tokens and e1, e2 the base-2
// logarithms of their sums.  The first is one problem per group, with all of the group's rows in
// row tiles that read the prefix once for up to 128 of them; the second is one per sequence.  Both are
// the cache attention's kernels with other lengths and tables.
#include <algorithm>

#include "kv_attention_few.cuh"
#include "kv_attention_rows.cuh"

namespace moe {
namespace {

constexpr int kMergeWarps = 8;

// A warp per (row, query head).
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) kv_attention_merge_kernel(const KvAttentionArgs k, const float *half,
                                                                               const float *half_lse) {
    const int lane = threadIdx.x & 31;
    const int64_t pairs = (int64_t)k.rows * k.heads_q;
    const int64_t at = (int64_t)blockIdx.x * kMergeWarps + threadIdx.x / 32;
    if (at >= pairs) return;
    const int row = (int)(at / k.heads_q), head = (int)(at - (int64_t)row * k.heads_q);
    if (row < k.cu_rows[0] || row >= k.cu_rows[k.seqs]) return;  // no sequence takes it
    constexpr int V = D / 32;
    float x[2][V], e[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const float *o = half + (size_t)(i * pairs + at) * D + lane * V;
        e[i] = half_lse[i * pairs + at];
#pragma unroll
        for (int j = 0; j < V; j++) x[i][j] = o[j];
    }
    // (a half that saw nothing has 0 and -infinity; NaN stays)
    const float m = fmaxf(e[0], e[1]);
    const float w0 = e[0] == -INFINITY ? 0.f : ex2(e[0] - m), w1 = e[1] == -INFINITY ? 0.f : ex2(e[1] - m);
    const float l = w0 + w1, inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t *out = k.out + (size_t)row * k.ldo + (size_t)head * D + lane * V;
#pragma unroll
    for (int j = 0; j < V; j++)
        out[j] = __bfloat16_as_ushort(__float2bfloat16((fmaf(x[0][j], w0, x[1][j] * w1)) * inv));
    if (k.lse != nullptr && lane == 0) k.lse[at] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
}

cudaError_t run(const AttnSetup &s, cudaStream_t st) {
    if (s.a.rpt > kFewRows) return launch_rows<true>(s.tm, s.a, s.sms, s.smem_max, st);
    return launch_few_of<true>(s.tm, s.a, s.sms, s.smem_max, st);
}

}  // namespace

cudaError_t set_wait_limit_kv_attention_shared(uint64_t ns) { return set_wait_limit_here(ns); }

cudaError_t kv_attention_shared_workspace_bytes(const KvView &kv, int rows, int max_rows, int max_group_rows, int heads_q,
                                                size_t *bytes) {
    size_t own = 0, prefix = 0;
    cudaError_t e = part_bytes(kv, max_rows, heads_q, &own);
    if (e == cudaSuccess) e = part_bytes(kv, max_group_rows, heads_q, &prefix);
    *bytes = sizeof(StatusWord) + std::max(own, prefix) + (size_t)2 * rows * heads_q * (kv.dim + 1) * sizeof(float);
    return e;
}

cudaError_t launch_kv_attention_shared(const KvAttentionArgs &k, const int32_t *cu_groups, const int32_t *prefix_len,
                                       int groups, int max_group_rows, void *ws, cudaStream_t st) {
    AttnSetup s;
    cudaError_t e = set_up(k, ws, s);
    if (e != cudaSuccess) return e;
    size_t own = 0, prefix = 0;
    if ((e = part_bytes(k.kv, k.max_rows, k.heads_q, &own)) != cudaSuccess) return e;
    if ((e = part_bytes(k.kv, max_group_rows, k.heads_q, &prefix)) != cudaSuccess) return e;
    const size_t pairs = (size_t)k.rows * k.heads_q;
    float *half = reinterpret_cast<float *>((char *)ws + sizeof(StatusWord) + std::max(own, prefix));
    float *half_lse = half + 2 * pairs * k.kv.dim;
    s.a.cu_groups = cu_groups;
    s.a.prefix_len = prefix_len;
    s.a.groups = groups;
    TraceScope trace_scope("kv_attention_shared", st);
    for (int i = 0; i < 2; i++) {
        AttnSetup t = s;
        t.a.prefix = i == 0;
        t.a.k.max_rows = i == 0 ? max_group_rows : k.max_rows;
        t.a.half = half + i * pairs * k.kv.dim;
        t.a.half_lse = half_lse + i * pairs;
        if ((e = set_tiles(t.a, i == 0 ? groups : k.seqs)) != cudaSuccess) return e;
        if ((e = run(t, st)) != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)((pairs + kMergeWarps - 1) / kMergeWarps)), block(32 * kMergeWarps);
    if (k.kv.dim == 128)
        kv_attention_merge_kernel<128><<<grid, block, 0, st>>>(k, half, half_lse);
    else
        kv_attention_merge_kernel<64><<<grid, block, 0, st>>>(k, half, half_lse);
    return cudaGetLastError();
}

}  // namespace moe
