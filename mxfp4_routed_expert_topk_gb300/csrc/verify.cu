// Verification of drafted tokens: acceptance in whole numbers, the next token by the
// inverse of the cumulative weights (sampled), or by the arg max (greedy).
//
// Both read rows of up to 2^20 values once.  With the data in L2 the chain of dependent accesses
// before and after that read is most of the time: one sequence of 5 rows of 32001 values takes
// 6.5 us, 64 of 9 rows of 131071 (47 MB in all) 19 us, 96 of 5 rows of 65536 16-bit ones without
// draft probabilities 12 us; greedy, 8 of 17 rows of 131072 16-bit values 7 us (5.2 TB/s).
//
// Sampled: a cluster of CTAs per sequence.  Every CTA finds the deciding row by itself (a lane
// per draft: two gathers, a whole-number comparison, a vote), so nothing is exchanged for it;
// then each warp sums the weights of its own consecutive part of that row, the CTAs' sums are
// exchanged through distributed shared memory, and the CTA that has the drawn point divides the
// part of the warp that holds it among all its warps and scans it again (it is in L1 / L2; by
// the one warp alone it took 4 us more).  Weights are whole numbers of 38 bits, so the sums are
// exact in any order and the result is the definition's, bit for bit.
//
// Greedy: a cluster per row finds its arg max (all rows at once: waiting for a row's verdict
// would cost more than the rows after a mismatch), then a warp per sequence compares.
#include <algorithm>

#include "vocab_row.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
// The deciding row of sequence rows [lo, hi): the first whose draft is not accepted, or the
// last (one warp; uniform result).
template <bool BF16>
__device__ __forceinline__ int deciding_row(const VerifyArgs &a, int lo, int hi, int lane) {
    constexpr int kSize = BF16 ? 2 : 4;
    for (int r0 = lo; r0 < hi - 1; r0 += 32) {
        const int r = r0 + lane;
        bool ok = true;
        if (r < hi - 1) {
            const int d = a.tokens[r + 1];
            const uint64_t m = whole_uniform(a.u_accept[r]);
            uint64_t P = 0, Q = 1ull << kGrid;
            if (d >= 0 && d < a.vocab) {
                auto get = [&](const void *base, size_t ld) {
                    const uint8_t *at = static_cast<const uint8_t *>(base) + ((size_t)r * ld + d) * kSize;
                    return whole(BF16 ? bf16_bits_to_float(__ldg(reinterpret_cast<const uint16_t *>(at)))
                                      : __ldg(reinterpret_cast<const float *>(at)));
                };
                P = get(a.p, a.ldp);
                if (a.q != nullptr) Q = get(a.q, a.ldq);
            }
            ok = m * Q < P << kUniform;
        }
        const uint32_t bad = __ballot_sync(0xffffffffu, !ok);
        if (bad != 0u) return r0 + __ffs((int)bad) - 1;
    }
    return hi - 1;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) verify_sampled_kernel(const VerifyArgs a) {
    constexpr int kVec = Row<BF16>::kVec;
    __shared__ int s_row;
    __shared__ uint64_t s_warp[2][kWarps];
    __shared__ uint64_t s_cta[2][kMaxCluster];  // [round][rank]: every CTA's sum
    const uint32_t rank = cluster_ctarank(), ranks = cluster_nctarank();
    const int b = (int)(blockIdx.x / ranks), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int lo, hi;
    const bool ok = seq_rows(a.cu_rows, b, a.rows, lo, hi);
    if (!ok || lo == hi) {  // the whole cluster alike
        if (rank == 0 && tid == 0) {
            if (!ok) set_status(a.st, MOE_ERR_BAD_PAGE, 1);
            a.accepted[b] = 0;
            a.next[b] = -1;
        }
        return;
    }
    cluster_arrive();  // waited for before the first remote store: by then every CTA has started
    if (warp == 0) {
        const int r = deciding_row<BF16>(a, lo, hi, lane);
        if (lane == 0) s_row = r;
    }
    __syncthreads();
    const int r = s_row;
    const bool rejected = r < hi - 1;
    const Row<BF16> P(a.p, (size_t)r * a.ldp, a.vocab);
    const Row<BF16> Q(a.q, a.q != nullptr ? (size_t)r * a.ldq : 0, a.vocab);
    bool minus = a.q != nullptr && rejected;           // weights P - Q
    int drop = a.q == nullptr && rejected ? a.tokens[r + 1] : -1;  // (outside the vocabulary: none)
    const bool together = Q.lead == P.lead;            // both rows' vectors hold the same indices
    const int vectors = P.vectors();
    const int per = (vectors + (int)ranks * kWarps - 1) / ((int)ranks * kWarps);  // vectors per warp
    const int v0 = min(((int)rank * kWarps + warp) * per, vectors), v1 = min(v0 + per, vectors);

    // the weights of vector v
    auto weights = [&](int v, uint64_t (&w)[kVec]) {
        float x[kVec], y[kVec];
        P.load(v, 0.f, x);
        if (minus) {
            if (together) {
                Q.load(v, 0.f, y);
            } else {
                const int i0 = P.first(v);
#pragma unroll
                for (int k = 0; k < kVec; k++) y[k] = i0 + k >= 0 && i0 + k < a.vocab ? Q.at(i0 + k) : 0.f;
            }
        }
        if (minus) {
#pragma unroll
            for (int k = 0; k < kVec; k++) {
                const int64_t d = (int64_t)(whole_raw(x[k]) - whole_raw(y[k]));
                w[k] = d > 0 ? (uint64_t)d : 0;
            }
        } else {
#pragma unroll
            for (int k = 0; k < kVec; k++) w[k] = whole(x[k]);
        }
        const uint32_t at = (uint32_t)(drop - P.first(v));
        if (drop >= 0 && at < (uint32_t)kVec) {
#pragma unroll
            for (int k = 0; k < kVec; k++)
                if (at == (uint32_t)k) w[k] = 0;
        }
    };

    // the weights of vectors [v, end), by one warp
    auto sum_of = [&](int v, int end) {
        uint64_t sum = 0;
#pragma unroll 2
        for (v += lane; v < end; v += 32) {
            uint64_t w[kVec];
            weights(v, w);
#pragma unroll
            for (int k = 0; k < kVec; k++) sum += w[k];
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        return sum;
    };

    for (int round = 0; round < 2; round++) {
        const uint64_t sum = sum_of(v0, v1);
        if (lane == 0) s_warp[0][warp] = sum;
        __syncthreads();
        uint64_t cta = 0;
#pragma unroll
        for (int w = 0; w < kWarps; w++) cta += s_warp[0][w];
        if (round == 0) cluster_wait();
        // every CTA writes its sum into all (nothing is read remotely, so none waits to exit)
        if (tid < (int)ranks) store_cluster_u64(&s_cta[round][rank], (uint32_t)tid, cta);
        cluster_sync();
        uint64_t total = 0, before = 0;  // all weights; what the CTAs before this one hold
        for (uint32_t k = 0; k < ranks; k++) {
            if (k < rank) before += s_cta[round][k];
            total += s_cta[round][k];
        }
        if (total == 0) {
            if (round == 0 && (minus || drop >= 0)) {  // nothing is left: all of the target
                minus = false;
                drop = -1;
                continue;
            }
            if (rank == 0 && tid == 0) a.next[b] = -1;
            break;
        }
        const uint64_t m = whole_uniform(a.u_sample[b]);
        const uint64_t aim = (total >> kUniform) * m + (((total & ((1ull << kUniform) - 1)) * m) >> kUniform);
        if (aim < before || aim >= before + cta) break;  // in another CTA's part
        // the warp whose part holds the point; the CTA's warps divide that part
        int w = 0;
        for (; w < kWarps - 1 && aim >= before + s_warp[0][w]; w++) before += s_warp[0][w];
        const int a0 = min(((int)rank * kWarps + w) * per, vectors), a1 = min(a0 + per, vectors);
        const int sub = (a1 - a0 + kWarps - 1) / kWarps, b0 = min(a0 + warp * sub, a1), b1 = min(b0 + sub, a1);
        const uint64_t part = sum_of(b0, b1);
        if (lane == 0) s_warp[1][warp] = part;
        __syncthreads();
        for (int k = 0; k < warp; k++) before += s_warp[1][k];
        if (aim >= before && aim < before + part) {
            uint64_t at = before;
            for (int v = b0; v < b1; v += 32) {
                uint64_t w[kVec], mine = 0;
                if (v + lane < b1) {
                    weights(v + lane, w);
#pragma unroll
                    for (int k = 0; k < kVec; k++) mine += w[k];
                }
                uint64_t upto = mine;  // inclusive over the lanes
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint64_t o = __shfl_up_sync(0xffffffffu, upto, d);
                    if (lane >= d) upto += o;
                }
                if (aim >= at + upto - mine && aim < at + upto) {
                    uint64_t c = at + upto - mine;
                    int found = -1;
#pragma unroll
                    for (int k = 0; k < kVec; k++) {
                        c += w[k];
                        if (found < 0 && c > aim) found = P.first(v + lane) + k;
                    }
                    a.next[b] = found;
                }
                at += __shfl_sync(0xffffffffu, upto, 31);
                if (at > aim) break;
            }
        }
        break;
    }
    if (rank == 0 && tid == 0) a.accepted[b] = r - lo;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) arg_max_kernel(const VerifyArgs a, int32_t *best) {
    constexpr int kVec = Row<BF16>::kVec;
    __shared__ uint64_t s_warp[kWarps];
    __shared__ uint64_t s_cta[kMaxCluster];  // rank 0's: every CTA's best
    const uint32_t rank = cluster_ctarank(), ranks = cluster_nctarank();
    const int r = (int)(blockIdx.x / ranks), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    cluster_arrive();  // waited for before the remote store: by then every CTA has started
    griddep_launch_dependents();
    const Row<BF16> X(a.p, (size_t)r * a.ldp, a.vocab);
    const int vectors = X.vectors();
    // The largest value of each vector (NaN is passed over) and the first vector that has it;
    // vectors ascend in each thread, so only a larger one replaces.  Its place is looked up at the
    // end: 1.5 instructions a value in place of 5.
    float top = __uint_as_float(0x7fc00000u);  // none
    int best_v = -1;
#pragma unroll 4
    for (int v = (int)rank * kThreads + tid; v < vectors; v += (int)ranks * kThreads) {
        const float m = X.largest(v);
        if (!(m <= top) && m == m) {
            top = m;
            best_v = v;
        }
    }
    int at = -1;
    if (best_v >= 0) {
        float x[kVec];
        X.load(best_v, __uint_as_float(0x7fc00000u), x);
#pragma unroll
        for (int k = kVec - 1; k >= 0; k--)
            if (x[k] == top) at = X.first(best_v) + k;
    }
    uint64_t key = order_key(top, at);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, d));
    if (lane == 0) s_warp[warp] = key;
    __syncthreads();
    cluster_wait();
    if (warp == 0) {
        key = lane < kWarps ? s_warp[lane] : 0;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, d));
        if (lane == 0) store_cluster_u64(&s_cta[rank], 0, key);
    }
    cluster_sync();
    if (rank == 0 && tid == 0) {
        for (uint32_t k = 0; k < ranks; k++) key = max(key, s_cta[k]);
        best[r] = key == 0 ? -1 : (int)(0xffffffffu - (uint32_t)key);
    }
}

// A warp per sequence: the drafts that equal the rows' arg max.
__global__ void __launch_bounds__(128) greedy_verdict_kernel(const VerifyArgs a, const int32_t *best) {
    griddep_wait();
    const int b = (int)(blockIdx.x * 4 + threadIdx.x / 32), lane = threadIdx.x & 31;
    if (b >= a.seqs) return;
    int lo, hi;
    const bool ok = seq_rows(a.cu_rows, b, a.rows, lo, hi);
    if (!ok && lane == 0) set_status(a.st, MOE_ERR_BAD_PAGE, 1);
    int r = hi - 1;
    for (int r0 = lo; r0 < hi - 1; r0 += 32) {
        const int k = r0 + lane;
        const bool bad = k < hi - 1 && (best[k] < 0 || best[k] != a.tokens[k + 1]);
        const uint32_t m = __ballot_sync(0xffffffffu, bad);
        if (m != 0u) {
            r = r0 + __ffs((int)m) - 1;
            break;
        }
    }
    if (lane == 0) {
        a.accepted[b] = lo < hi ? r - lo : 0;
        a.next[b] = lo < hi ? best[r] : -1;
    }
}

PerDevice g_sms(0);

// CTAs per cluster for `units` clusters: as many as fit the device at once (two CTAs of 512
// threads per SM), 8 at most (the portable size).  With cold caches, 1 / 2 / 4 / 8 CTAs: 64
// sequences (131071 values) 64 / 39 / 31 / 33 us; 96 (65536 16-bit values) 23 / 19 / 23 / 27;
// 136 rows' arg max (131072 16-bit values) 23 / 19 / 21 / 25; one sequence 23 / 17 / 15 / 13.
int cluster_size(int units, int sms) {
    int c = kMaxCluster;
    while (c > 1 && (int64_t)units * c > 2 * (int64_t)sms) c /= 2;
    return c;
}

}  // namespace

// The status word, then each row's arg max (greedy).
size_t verify_workspace_bytes(int, int rows) { return sizeof(StatusWord) + align_up((size_t)rows * sizeof(int32_t), 256); }

cudaError_t launch_verify_sampled(const VerifyArgs &a, void *, cudaStream_t st) {
    if (a.seqs == 0) return cudaSuccess;
    int sms = 0;
    const cudaError_t e = device_attr(cudaDevAttrMultiProcessorCount, g_sms, &sms);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = cluster_config(attr, a.seqs, cluster_size(a.seqs, sms), kThreads, st);
    TraceScope trace_scope("verify_sampled", st);
    return a.bf16 ? cudaLaunchKernelEx(&cfg, verify_sampled_kernel<true>, a)
                  : cudaLaunchKernelEx(&cfg, verify_sampled_kernel<false>, a);
}

cudaError_t launch_verify_greedy(const VerifyArgs &a, void *ws, cudaStream_t st) {
    if (a.seqs == 0) return cudaSuccess;
    int sms = 0;
    cudaError_t e = device_attr(cudaDevAttrMultiProcessorCount, g_sms, &sms);
    if (e != cudaSuccess) return e;
    int32_t *best = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + sizeof(StatusWord));
    TraceScope trace_scope("verify_greedy", st);
    if (a.rows > 0) {
        cudaLaunchAttribute attr[1];
        const cudaLaunchConfig_t cfg = cluster_config(attr, a.rows, cluster_size(a.rows, sms), kThreads, st);
        e = a.bf16 ? cudaLaunchKernelEx(&cfg, arg_max_kernel<true>, a, best)
                   : cudaLaunchKernelEx(&cfg, arg_max_kernel<false>, a, best);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(greedy_verdict_kernel, dim3((unsigned)((a.seqs + 3) / 4)), dim3(128), 0, st, a,
                      (const int32_t *)best);
}

}  // namespace moe
