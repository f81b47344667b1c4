// Attention of a few rows per sequence over the paged 8-bit key/value cache.
//
// Simple form: one block per (row, query head); its four warps take every fourth token,
// each keeps a running maximum, sum and output (lanes over the head's values), and the
// four are joined at the end.
#include "kv_internal.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) kv_attention_kernel(const KvAttentionArgs a) {
    constexpr int V = D / 32;  // values per lane
    __shared__ int s_seq;
    __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
    const int r = blockIdx.x, hq = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int head = hq / (a.heads_q / a.kv.heads);
    if (threadIdx.x == 0) s_seq = a.seqs;
    __syncthreads();
    for (int b = threadIdx.x; b < a.seqs; b += blockDim.x) {
        int lo, hi;
        if (!seq_rows(a.cu_rows, b, a.rows, lo, hi) && r == 0 && hq == 0) set_status(a.st, MOE_ERR_BAD_PAGE, 1);
        if (r >= lo && r < hi) atomicMin(&s_seq, b);
    }
    __syncthreads();
    const int b = s_seq;
    if (b == a.seqs) return;
    const int lo = a.cu_rows[b], n = a.cu_rows[b + 1] - lo;
    int len = max(a.kv_len[b], 0);
    if (n > a.max_rows || (int64_t)len > (int64_t)a.table_width * a.kv.page) {
        if (threadIdx.x == 0) set_status(a.st, MOE_ERR_BAD_PAGE, 2);
        if (r - lo >= a.max_rows) return;
        len = (int)min((int64_t)len, (int64_t)a.table_width * a.kv.page);
    }
    const int see = min(len, max(0, len - n + (r - lo) + 1));  // tokens 0 .. see-1
    float q[V], o[V], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < V; i++) {
        q[i] = bf16_bits_to_float(a.q[(size_t)r * a.ldq + (size_t)hq * D + lane * V + i]) * a.scale;
        o[i] = 0.f;
    }
    for (int t = warp; t < see; t += kWarps) {
        const int page = a.page_table[(size_t)b * a.table_width + t / a.kv.page], slot = t % a.kv.page;
        if (page < 0 || page >= a.kv.n_pages) {
            if (lane == 0) set_status(a.st, MOE_ERR_BAD_PAGE, 3);
            continue;
        }
        const uint8_t *k = a.kv.codes(page, a.layer, 0, head) + slot * D + lane * V;
        const uint8_t *v = a.kv.codes(page, a.layer, 1, head) + slot * D + lane * V;
        float x = 0.f, f[4];
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < V; i++) c |= (uint32_t)k[i] << (8 * i);
        e4m3x4_to_float(c, f);
#pragma unroll
        for (int i = 0; i < V; i++) x += q[i] * f[i];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        x *= *a.kv.scale(page, a.layer, 0, head);
        const float mn = fmaxf(m, x), keep = m == -INFINITY ? 0.f : expf(m - mn), p = expf(x - mn);
        const float pv = p * *a.kv.scale(page, a.layer, 1, head);
        c = 0;
#pragma unroll
        for (int i = 0; i < V; i++) c |= (uint32_t)v[i] << (8 * i);
        e4m3x4_to_float(c, f);
#pragma unroll
        for (int i = 0; i < V; i++) o[i] = o[i] * keep + pv * f[i];
        l = l * keep + p;
        m = mn;
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < V; i++) s_o[warp][lane * V + i] = o[i];
    __syncthreads();
    float mm = -INFINITY, ll = 0.f;
    for (int w = 0; w < kWarps; w++) mm = fmaxf(mm, s_m[w]);
    for (int w = 0; w < kWarps; w++) ll += s_l[w] == 0.f ? 0.f : s_l[w] * expf(s_m[w] - mm);
    for (int d = threadIdx.x; d < D; d += blockDim.x) {
        float y = 0.f;
        for (int w = 0; w < kWarps; w++) y += s_l[w] == 0.f ? 0.f : s_o[w][d] * expf(s_m[w] - mm);
        y = see == 0 ? 0.f : y / ll;
        a.out[(size_t)r * a.ldo + (size_t)hq * D + d] = __bfloat16_as_ushort(__float2bfloat16(y));
    }
    if (a.lse != nullptr && threadIdx.x == 0)
        a.lse[(size_t)r * a.heads_q + hq] = see == 0 ? -INFINITY : mm + logf(ll);
}

}  // namespace

cudaError_t kv_attention_workspace_bytes(const KvView &, int, int, size_t *bytes) {
    *bytes = sizeof(StatusWord);
    return cudaSuccess;
}

cudaError_t launch_kv_attention(const KvAttentionArgs &a, void *, cudaStream_t st) {
    const dim3 grid((unsigned)a.rows, (unsigned)a.heads_q);
    TraceScope trace_scope("kv_attention", st);
    if (a.kv.dim == 64)
        kv_attention_kernel<64><<<grid, 32 * kWarps, 0, st>>>(a);
    else
        kv_attention_kernel<128><<<grid, 32 * kWarps, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
