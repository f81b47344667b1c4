// Sampling from logits: temperature, top-k, top-p, min-p, and a draw from a given uniform number; or
// the distribution that they leave.
//
// Tokens stand in the order of falling logit, then rising index; every cut keeps a beginning of that
// order (min-p apart, which looks at a weight alone).  Weights are whole numbers of 38 bits, so sums
// are exact in any order and the result is the definition's, bit for bit.
#include <algorithm>

#include "vocab_row.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kList = 1024;     // tokens that are ranked one by one
constexpr float kReach = 39.f;  // weights of 2^-39 and less are 0
constexpr float kBinsPerOctave = 52.5f;

// What rank 0 tells the cluster.
struct Word {
    uint64_t a, b, c, d;
};

struct Smem {
    uint32_t cnt[kBins];
    uint64_t sum[kBins];
    uint32_t all_cnt[kBins];  // rank 0's: of the whole row, by bin of the logit
    uint64_t all_sum[kBins];
    uint64_t key[kList], weight[kList], gkey[kList], gweight[kList];
    uint64_t cta[2][kMaxCluster];
    uint64_t warp[2][kWarps];
    Word word;
    uint32_t wcnt[kWarps];
    uint64_t wsum[kWarps];
    int n;
};

template <typename T>
__device__ __forceinline__ T ld_cluster(const T *mine, uint32_t rank) {
    T v;
    if constexpr (sizeof(T) == 8)
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(mapa_shared(mine, rank)) : "memory");
    else
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(mine, rank)) : "memory");
    return v;
}

// The weight of a row's logits: 2^y in steps of their own, each rounded to fp32 (a product and a sum
// apart), so that any machine gets the same; the polynomial is 2^f's closest of the fifth degree
// with 1 at 0 (relative error 2^-23.4, 2^-22.3 as computed).
struct Weigh {
    float m, c;
    __device__ __forceinline__ float octaves(float x) const { return x == m ? 0.f : __fmul_rn(__fsub_rn(x, m), c); }
    __device__ __forceinline__ static uint64_t weight(float y) {
        if (!(y > -kReach)) return 0;  // (NaN too)
        const float n = rintf(y), f = __fsub_rn(y, n);
        float e = 0x1.5bba14p-10f;
        e = __fadd_rn(__fmul_rn(e, f), 0x1.3cea88p-7f);
        e = __fadd_rn(__fmul_rn(e, f), 0x1.c6b752p-5f);
        e = __fadd_rn(__fmul_rn(e, f), 0x1.ebf9bcp-3f);
        e = __fadd_rn(__fmul_rn(e, f), 0x1.62e42ap-1f);
        e = __fadd_rn(__fmul_rn(e, f), 1.f);
        return whole(__int_as_float(__float_as_int(e) + ((int)n << 23)));
    }
    __device__ __forceinline__ uint64_t operator()(float x) const { return weight(octaves(x)); }
    __device__ __forceinline__ static int bin(float y) { return min((int)(-y * kBinsPerOctave), kBins - 1); }
};

__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}

// The first 24 bits of a number in 0 .. 1 as a whole number (`none` for NaN).
__device__ __forceinline__ uint64_t first_bits(float v, uint64_t none) {
    return v == v ? (uint64_t)(__saturatef(v) * 16777216.f) : none;
}
// total m / 2^24, rounded down, or up.
__device__ __forceinline__ uint64_t share_of(uint64_t total, uint64_t m, bool up) {
    constexpr uint64_t kMask = (1ull << kUniform) - 1;
    return (total >> kUniform) * m + (((total & kMask) * m + (up ? kMask : 0)) >> kUniform);
}

// The digits of an order key by which a bin is divided: 11, 11 and 10 bits of the logit, then 11 and
// 9 of the index.
__device__ __forceinline__ int digit_shift(int level) { return level == 1 ? 53 : level == 2 ? 42 : level == 3 ? 32 : level == 4 ? 9 : 0; }
__device__ __forceinline__ int digit_bits(int level) { return level == 3 ? 10 : level == 5 ? 9 : 11; }

template <bool BF16, bool PROBS>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
    constexpr int kVec = Row<BF16>::kVec;
    extern __shared__ __align__(16) unsigned char raw[];
    Smem &s = *reinterpret_cast<Smem *>(raw);
    const uint32_t rank = cluster_ctarank(), ranks = cluster_nctarank();
    const int r = (int)(blockIdx.x / ranks), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    cluster_arrive();  // waited for before the first remote store: by then every CTA has started
    const Row<BF16> X(a.x, (size_t)r * a.ld, a.vocab);
    const int vectors = X.vectors();
    const float kNone = __uint_as_float(0x7fc00000u);

    // the first token of the order
    uint64_t top = 0;
    for (int v = (int)rank * kThreads + tid; v < vectors; v += (int)ranks * kThreads) {
        float x[kVec];
        X.load(v, kNone, x);
#pragma unroll
        for (int k = 0; k < kVec; k++)
            if (x[k] > -INFINITY) top = max(top, order_key(x[k], X.first(v) + k));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (lane == 0) s.warp[0][warp] = top;
    __syncthreads();
    for (int w = 0; w < kWarps; w++) top = max(top, s.warp[0][w]);
    cluster_wait();
    if (tid < (int)ranks) store_cluster_u64(&s.cta[0][rank], (uint32_t)tid, top);
    cluster_sync();
    for (uint32_t k = 0; k < ranks; k++) top = max(top, s.cta[0][k]);

    const float T = a.temperature[r];
    uint16_t *out16 = static_cast<uint16_t *>(a.probs) + (size_t)r * a.ldp;
    float *out32 = static_cast<float *>(a.probs) + (size_t)r * a.ldp;
    auto put = [&](int i, float p) {
        if (BF16)
            out16[i] = __bfloat16_as_ushort(__float2bfloat16(p));
        else
            out32[i] = p;
    };
    if (top == 0 || !(T > 0.f)) {  // nothing to draw from, or nothing to draw
        const int first = top == 0 ? -1 : (int)(0xffffffffu - (uint32_t)top);
        if (PROBS) {
            for (int i = (int)rank * kThreads + tid; i < a.vocab; i += (int)ranks * kThreads) put(i, i == first ? 1.f : 0.f);
        } else if (rank == 0 && tid == 0) {
            a.next[r] = first;
        }
        return;
    }
    const Weigh W{key_value(top), fminf(__fdiv_rn(0x1.715476p+0f, T), 3.4028235e38f)};
    const int k = a.top_k != nullptr ? a.top_k[r] : 0;
    const uint64_t part = a.top_p != nullptr ? max(first_bits(a.top_p[r], 1ull << kUniform), (uint64_t)1) : 1ull << kUniform;
    const uint64_t least = a.min_p != nullptr ? first_bits(a.min_p[r], 0) << (kGrid - kUniform) : 0;

    // f(logit's octaves, index) for this CTA's part of the row
    auto each = [&](auto f) {
        for (int v = (int)rank * kThreads + tid; v < vectors; v += (int)ranks * kThreads) {
            float x[kVec];
            X.load(v, kNone, x);
#pragma unroll
            for (int j = 0; j < kVec; j++) {
                const float y = W.octaves(x[j]);
                if (y > -kReach) f(x[j], y, X.first(v) + j);
            }
        }
    };
    auto clear = [&] {
        for (int i = tid; i < kBins; i += kThreads) s.cnt[i] = 0, s.sum[i] = 0;
        if (tid == 0) s.n = 0;
        __syncthreads();
    };
    auto tell = [&](Word w) {  // (one thread of rank 0)
        for (uint32_t q = 0; q < ranks; q++) {
            store_cluster_u64(&s.word.a, q, w.a);
            store_cluster_u64(&s.word.b, q, w.b);
            store_cluster_u64(&s.word.c, q, w.c);
            store_cluster_u64(&s.word.d, q, w.d);
        }
    };
    // rank 0: the cluster's bins into `cnt`, `sum`
    auto merge = [&](uint32_t *cnt, uint64_t *sum) {
        for (int i = tid; i < kBins; i += kThreads) {
            uint32_t c = 0;
            uint64_t w = 0;
            for (uint32_t q = 0; q < ranks; q++) c += ld_cluster(s.cnt + i, q), w += ld_cluster(s.sum + i, q);
            cnt[i] = c;
            sum[i] = w;
        }
        __syncthreads();
    };
    // rank 0: the bin in which the tokens, or their weights, reach `target`; told as (bin, tokens
    // before it, weights before it, tokens in it)
    auto choose = [&](const uint32_t *cnt, const uint64_t *sum, bool weights, uint64_t target, uint64_t c0, uint64_t w0) {
        constexpr int kPer = kBins / kThreads;
        uint32_t c = 0;
        uint64_t w = 0;
        for (int i = 0; i < kPer; i++) c += cnt[tid * kPer + i], w += sum[tid * kPer + i];
        uint32_t uc = c;
        uint64_t uw = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t oc = __shfl_up_sync(0xffffffffu, uc, d);
            const uint64_t ow = __shfl_up_sync(0xffffffffu, uw, d);
            if (lane >= d) uc += oc, uw += ow;
        }
        if (lane == 31) s.wcnt[warp] = uc, s.wsum[warp] = uw;
        __syncthreads();
        for (int q = 0; q < warp; q++) uc += s.wcnt[q], uw += s.wsum[q];
        uint64_t bc = c0 + uc - c, bw = w0 + uw - w;
        for (int i = 0; i < kPer; i++) {
            const uint32_t cc = cnt[tid * kPer + i];
            const uint64_t ww = sum[tid * kPer + i];
            const uint64_t before = weights ? bw : bc, here = weights ? ww : cc;
            if (before < target && target <= before + here) tell(Word{(uint64_t)(tid * kPer + i), bc, bw, cc});
            bc += cc;
            bw += ww;
        }
    };
    // The token at which tokens, or weights, reach `target` in the order: its key, and the weights up
    // to and with it.
    auto find = [&](bool weights, uint64_t target, uint64_t &upto) -> uint64_t {
        if (rank == 0) choose(s.all_cnt, s.all_sum, weights, target, 0, 0);
        cluster_sync();
        Word w = s.word;
        const int bin = (int)w.a;
        uint64_t prefix = 0;
        int level = 0;
        auto in = [&](float y, uint64_t key) {
            return Weigh::bin(y) == bin && (level == 0 || (key >> digit_shift(level)) == prefix);
        };
        while (w.d > kList) {
            clear();
            const int shift = digit_shift(level + 1), mask = (1 << digit_bits(level + 1)) - 1;
            each([&](float x, float y, int i) {
                const uint64_t key = order_key(x, i);
                if (!in(y, key)) return;
                const int d = mask - (int)(key >> shift & mask);
                atomicAdd(s.cnt + d, 1u);
                atomicAdd((unsigned long long *)(s.sum + d), (unsigned long long)Weigh::weight(y));
            });
            cluster_sync();
            if (rank == 0) {
                merge(s.cnt, s.sum);
                choose(s.cnt, s.sum, weights, target, w.b, w.c);
            }
            cluster_sync();
            w = s.word;
            level++;
            // (between the logit's digits and the index's stand constant bits)
            const uint64_t d = (uint64_t)mask - w.a;
            if (level == 4)
                prefix = (prefix << 23) | (0xfffull << 11) | d;
            else
                prefix = (prefix << digit_bits(level)) | d;
        }
        if (tid == 0) s.n = 0;
        __syncthreads();
        each([&](float x, float y, int i) {
            const uint64_t key = order_key(x, i);
            if (!in(y, key)) return;
            const int at = atomicAdd(&s.n, 1);
            s.key[at] = key;
            s.weight[at] = Weigh::weight(y);
        });
        cluster_sync();
        if (rank == 0) {
            int n = 0;
            for (uint32_t q = 0; q < ranks; q++) {
                const int nq = (int)ld_cluster((const uint32_t *)&s.n, q);
                for (int i = tid; i < nq; i += kThreads) {
                    s.gkey[n + i] = ld_cluster(s.key + i, q);
                    s.gweight[n + i] = ld_cluster(s.weight + i, q);
                }
                n += nq;
            }
            __syncthreads();
            for (int i = tid; i < n; i += kThreads) {
                const uint64_t mine = s.gkey[i];
                uint64_t c = w.b, sum = w.c;
                for (int j = 0; j < n; j++)
                    if (s.gkey[j] > mine) c++, sum += s.gweight[j];
                const uint64_t before = weights ? sum : c, here = weights ? s.gweight[i] : 1;
                if (before < target && target <= before + here) tell(Word{mine, sum + s.gweight[i], 0, 0});
            }
        }
        cluster_sync();
        upto = s.word.b;
        return s.word.a;
    };

    uint64_t cut = 0;  // tokens below this key are not kept
    const bool by_count = k > 0 && k < a.vocab, by_share = part < 1ull << kUniform;
    if (by_count || by_share) {
        clear();
        each([&](float, float y, int) {
            const int b = Weigh::bin(y);
            atomicAdd(s.cnt + b, 1u);
            atomicAdd((unsigned long long *)(s.sum + b), (unsigned long long)Weigh::weight(y));
        });
        cluster_sync();
        if (rank == 0) {
            merge(s.all_cnt, s.all_sum);
            uint32_t c = 0;
            uint64_t w = 0;
            for (int i = tid; i < kBins; i += kThreads) c += s.all_cnt[i], w += s.all_sum[i];
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) c += __shfl_xor_sync(0xffffffffu, c, d), w += __shfl_xor_sync(0xffffffffu, w, d);
            if (lane == 0) s.wcnt[warp] = c, s.wsum[warp] = w;
            __syncthreads();
            if (tid == 0) {
                c = 0, w = 0;
                for (int q = 0; q < kWarps; q++) c += s.wcnt[q], w += s.wsum[q];
                tell(Word{c, w, 0, 0});
            }
            __syncthreads();
        }
        cluster_sync();
        const uint64_t live = s.word.a;
        uint64_t total = s.word.b;
        cluster_sync();  // (the word is read)
        if (by_count && (uint64_t)k < live) cut = find(false, (uint64_t)k, total);
        if (by_share) {
            uint64_t upto;
            cluster_sync();
            cut = find(true, share_of(total, part, true), upto);
        }
    }

    // the kept weights of vector v
    auto kept = [&](int v, uint64_t (&w)[kVec]) {
        float x[kVec];
        X.load(v, kNone, x);
#pragma unroll
        for (int j = 0; j < kVec; j++) {
            w[j] = W(x[j]);
            if (w[j] < least || order_key(x[j], X.first(v) + j) < cut) w[j] = 0;
        }
    };
    auto sum_of = [&](int v, int end) {
        uint64_t sum = 0;
        for (v += lane; v < end; v += 32) {
            uint64_t w[kVec];
            kept(v, w);
#pragma unroll
            for (int j = 0; j < kVec; j++) sum += w[j];
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        return sum;
    };
    const int per = (vectors + (int)ranks * kWarps - 1) / ((int)ranks * kWarps);  // vectors per warp
    const int v0 = min(((int)rank * kWarps + warp) * per, vectors), v1 = min(v0 + per, vectors);
    const uint64_t sum = sum_of(v0, v1);
    __syncthreads();
    if (lane == 0) s.warp[0][warp] = sum;
    __syncthreads();
    uint64_t cta = 0;
    for (int w = 0; w < kWarps; w++) cta += s.warp[0][w];
    if (tid < (int)ranks) store_cluster_u64(&s.cta[1][rank], (uint32_t)tid, cta);
    cluster_sync();
    uint64_t total = 0, before = 0;
    for (uint32_t q = 0; q < ranks; q++) {
        if (q < rank) before += s.cta[1][q];
        total += s.cta[1][q];
    }
    if (PROBS) {
        const float all = __ull2float_rn(total);
        for (int v = v0 + lane; v < v1; v += 32) {
            uint64_t w[kVec];
            kept(v, w);
#pragma unroll
            for (int j = 0; j < kVec; j++) {
                const int i = X.first(v) + j;
                if (i >= 0 && i < a.vocab) put(i, __fdiv_rn(__ull2float_rn(w[j]), all));
            }
        }
        return;
    }
    const uint64_t aim = share_of(total, whole_uniform(a.u[r]), false);
    if (aim < before || aim >= before + cta) return;  // in another CTA's part
    int w = 0;
    for (; w < kWarps - 1 && aim >= before + s.warp[0][w]; w++) before += s.warp[0][w];
    if (warp != w) return;
    for (int v = v0; v < v1; v += 32) {
        uint64_t x[kVec], mine = 0;
        if (v + lane < v1) {
            kept(v + lane, x);
#pragma unroll
            for (int j = 0; j < kVec; j++) mine += x[j];
        }
        uint64_t upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint64_t o = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += o;
        }
        if (aim >= before + upto - mine && aim < before + upto) {
            uint64_t c = before + upto - mine;
            int found = -1;
#pragma unroll
            for (int j = 0; j < kVec; j++) {
                c += x[j];
                if (found < 0 && c > aim) found = X.first(v + lane) + j;
            }
            a.next[r] = found;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
        if (before > aim) break;
    }
}

PerDevice g_sms(0);

int cluster_size(int rows, int sms) {
    int c = kMaxCluster;
    while (c > 1 && (int64_t)rows * c > 2 * (int64_t)sms) c /= 2;
    return c;
}

template <bool BF16, bool PROBS>
cudaError_t launch(const SampleArgs &a, cudaStream_t st) {
    static PerDevice smem_set(0);
    int sms = 0;
    cudaError_t e = device_attr(cudaDevAttrMultiProcessorCount, g_sms, &sms);
    if (e != cudaSuccess) return e;
    if ((e = ensure_dynamic_smem(sample_kernel<BF16, PROBS>, sizeof(Smem), smem_set)) != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = cluster_config(attr, a.rows, cluster_size(a.rows, sms), kThreads, st);
    cfg.dynamicSmemBytes = sizeof(Smem);
    return cudaLaunchKernelEx(&cfg, sample_kernel<BF16, PROBS>, a);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    TraceScope trace_scope(a.probs != nullptr ? "sample_probs" : "sample", st);
    if (a.probs != nullptr) return a.bf16 ? launch<true, true>(a, st) : launch<false, true>(a, st);
    return a.bf16 ? launch<true, false>(a, st) : launch<false, false>(a, st);
}

}  // namespace moe
