// Verification of drafted tokens: acceptance in whole numbers, the next token by the
// inverse of the cumulative weights (sampled), or by the arg max (greedy).
//
// Simple form: one block of 1024 threads per sequence.
#include "kv_internal.cuh"

namespace moe {
namespace {

constexpr int kThreads = 1024;
constexpr int kGrid = 38;       // probabilities are whole multiples of 2^-38
constexpr int kUniform = 24;    // uniforms are whole multiples of 2^-24

template <bool BF16>
__device__ __forceinline__ float load_value(const void *p, size_t i) {
    return BF16 ? bf16_bits_to_float(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}

// floor(2^38 min(max(p, 0), 1)), NaN: 0.
__device__ __forceinline__ uint64_t whole(float p) {
    return __float2ull_rz(fminf(fmaxf(p, 0.f), 1.f) * 274877906944.f);
}

__device__ __forceinline__ uint64_t whole_uniform(float u) {
    return (uint64_t)__float2uint_rz(fminf(fmaxf(u, 0.f), 0.99999994f) * 16777216.f);
}

// Weight of token i at the row that decides: P - Q (cut at 0), or P alone (q null), or 0
// at `drop`.
template <bool BF16>
__device__ __forceinline__ uint64_t weight(const void *p, const void *q, int64_t drop, size_t i) {
    const uint64_t x = whole(load_value<BF16>(p, i));
    if (q != nullptr) {
        const uint64_t y = whole(load_value<BF16>(q, i));
        return x > y ? x - y : 0;
    }
    return (int64_t)i == drop ? 0 : x;
}

template <typename T>
__device__ T block_scan(T v, T *total) {
    __shared__ T sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
    for (int d = 1; d < 32; d <<= 1) {
        const T o = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += o;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    T all = 0;
    for (int w = 0; w < kThreads / 32; w++) {
        if (w < warp) x += sums[w];
        all += sums[w];
    }
    *total = all;
    return x - v;  // exclusive
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) verify_sampled_kernel(const VerifyArgs a) {
    __shared__ int s_row, s_token;
    constexpr size_t kSize = BF16 ? 2 : 4;
    const int b = blockIdx.x, tid = threadIdx.x;
    int lo, hi;
    const bool ok = seq_rows(a.cu_rows, b, a.rows, lo, hi);
    if (!ok || lo == hi) {
        if (tid == 0) {
            if (!ok) set_status(a.st, MOE_ERR_BAD_PAGE, 1);
            a.accepted[b] = 0;
            a.next[b] = -1;
        }
        return;
    }
    if (tid == 0) {
        int r = lo;
        for (; r < hi - 1; r++) {
            const int d = a.tokens[r + 1];
            if (d < 0 || d >= a.vocab) break;
            const uint64_t P = whole(load_value<BF16>(a.p, (size_t)r * a.ldp + d));
            const uint64_t Q = a.q ? whole(load_value<BF16>(a.q, (size_t)r * a.ldq + d)) : 1ull << kGrid;
            if (whole_uniform(a.u_accept[r]) * Q >= P << kUniform) break;
        }
        s_row = r;
        s_token = -1;
    }
    __syncthreads();
    const int r = s_row;
    const char *p = static_cast<const char *>(a.p) + (size_t)r * a.ldp * kSize;
    const char *q = a.q && r < hi - 1 ? static_cast<const char *>(a.q) + (size_t)r * a.ldq * kSize : nullptr;
    int64_t drop = a.q == nullptr && r < hi - 1 ? a.tokens[r + 1] : -1;
    const int per = (a.vocab + kThreads - 1) / kThreads;
    const int i0 = min(tid * per, a.vocab), i1 = min(i0 + per, a.vocab);
    for (int pass = 0; pass < 2; pass++) {
        uint64_t mine = 0, total;
        for (int i = i0; i < i1; i++) mine += weight<BF16>(p, q, drop, i);
        uint64_t at = block_scan<uint64_t>(mine, &total);
        if (total == 0) {  // nothing is left of the target: all of it
            q = nullptr;
            drop = -1;
            continue;
        }
        const uint64_t m = whole_uniform(a.u_sample[b]);
        const uint64_t aim = (total >> kUniform) * m + (((total & ((1ull << kUniform) - 1)) * m) >> kUniform);
        if (aim >= at && aim < at + mine) {
            for (int i = i0; i < i1; i++) {
                at += weight<BF16>(p, q, drop, i);
                if (at > aim) {
                    s_token = i;
                    break;
                }
            }
        }
        break;
    }
    __syncthreads();
    if (tid == 0) {
        a.accepted[b] = r - lo;
        a.next[b] = s_token;
    }
}

// A logit's place in the order (0: NaN, which is never the largest), then the lower index.
__device__ __forceinline__ uint64_t order_key(float x, int i) {
    if (!(x == x)) return 0;
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 equals +0
    const uint32_t o = (u & 0x80000000u) ? ~u : u | 0x80000000u;
    return (uint64_t)o << 32 | (0xffffffffu - (uint32_t)i);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) verify_greedy_kernel(const VerifyArgs a) {
    __shared__ unsigned long long s_best;
    const int b = blockIdx.x, tid = threadIdx.x;
    int lo, hi;
    const bool ok = seq_rows(a.cu_rows, b, a.rows, lo, hi);
    if (!ok || lo == hi) {
        if (tid == 0) {
            if (!ok) set_status(a.st, MOE_ERR_BAD_PAGE, 1);
            a.accepted[b] = 0;
            a.next[b] = -1;
        }
        return;
    }
    int r = lo, best = -1;
    for (; r < hi; r++) {
        if (tid == 0) s_best = 0;
        __syncthreads();
        uint64_t key = 0;
        for (int i = tid; i < a.vocab; i += kThreads)
            key = max(key, order_key(load_value<BF16>(a.p, (size_t)r * a.ldp + i), i));
        atomicMax(&s_best, (unsigned long long)key);
        __syncthreads();
        best = s_best == 0 ? -1 : (int)(0xffffffffu - (uint32_t)s_best);
        __syncthreads();
        if (r == hi - 1 || a.tokens[r + 1] != best || best < 0) break;
    }
    if (tid == 0) {
        a.accepted[b] = r - lo;
        a.next[b] = best;
    }
}

}  // namespace

size_t verify_workspace_bytes(int, int) { return sizeof(StatusWord); }

cudaError_t launch_verify_sampled(const VerifyArgs &a, void *, cudaStream_t st) {
    if (a.seqs == 0) return cudaSuccess;
    TraceScope trace_scope("verify_sampled", st);
    if (a.bf16)
        verify_sampled_kernel<true><<<a.seqs, kThreads, 0, st>>>(a);
    else
        verify_sampled_kernel<false><<<a.seqs, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_verify_greedy(const VerifyArgs &a, void *, cudaStream_t st) {
    if (a.seqs == 0) return cudaSuccess;
    TraceScope trace_scope("verify_greedy", st);
    if (a.bf16)
        verify_greedy_kernel<true><<<a.seqs, kThreads, 0, st>>>(a);
    else
        verify_greedy_kernel<false><<<a.seqs, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
