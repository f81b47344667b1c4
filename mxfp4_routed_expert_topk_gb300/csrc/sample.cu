// Sampling from logits: temperature, top-k, top-p, min-p, and a draw from a given uniform number; or
// the distribution that they leave.
//
// Tokens stand in the order of falling logit, then rising index; every cut keeps a beginning of that
// order (min-p apart, which looks at a weight alone).  Weights are whole numbers of 38 bits, so sums
// are exact in any order and the result is the definition's, bit for bit, whichever way it is found.
//
// A cluster of CTAs per row, which is read once from HBM for its largest value and again from L2 for what
// else its settings ask for.  What costs is instructions, and the cluster's barriers where there are few
// rows: a weight is 13 of them (pairs of values in f32x2 arithmetic), an addition to a histogram in shared
// memory takes as long.  So:
//   - top-k of up to 1024: the largest of each part of a thread's values go into a histogram; the bin at
//     which they reach k bounds the k-th largest value from below, and the few tokens above it go to rank
//     0's list, are put in order there, and all else is done on the list;
//   - top-p: one pass sums the weights exactly; one adds them up by bins of the logit in 32 bits, for the
//     values that can matter; from that follow one or two bins in which the cut must lie; one pass sums the
//     weights above those exactly and puts what lies in them on the list; the cut is found there, and the
//     part of the row that has the drawn point is searched;
//   - where the list does not hold them (thousands of equal logits) or a larger top-k is asked for, the cut
//     is found digit by digit in exact histograms.
//
// Measured on the device: one row of 32001 values 5 (its largest), 10 (top-k of 1), 11 (50), 19 (1000), 24 to 29 us
// (top-p alone); 256 rows of 131072, settings mixed, 127 us, where rows of top-p alone (a twelfth) take 110 each
// and those with a top-k 38 to 54, many under way together; distributions of 96 rows of 131071, top-p alone, 108 us
// (31 and 29 % of the ALU and FMA pipes, 39 % of the issue slots; waits for loads are the commonest stall).  Not better
// (each against the kernel as it then was): copying a row's vectors ahead into shared memory, 96 rows 123 us
// against 110; four vectors' loads in flight per thread 113 against 110, with their arithmetic unrolled 187
// against 134; listing the largest 1024 first for top-p alone 150 against 130; functions called in place of
// inlined 137 against 114.
#include <algorithm>

#include "vocab_row.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kList = 2048;      // tokens that rank 0 sorts
constexpr int kSmallK = 1024;    // top-k that goes by the threads' largest values
constexpr int kFew = 128;        // tokens that are placed by comparing each with all
constexpr int kSubs = 4;         // parts of a thread's values whose largest are looked at
constexpr int kBins = 2048;      // of counts, or of weights in 32 bits; 16 per octave at temperature 1 for the largest
constexpr int kExact = 1024;     // of counts and weights in 64 bits
constexpr float kReach = 39.f;   // weights of 2^-39 and less are 0
constexpr float kNone = -INFINITY;

// What rank 0 tells the cluster.
struct Word {
    uint64_t a, b, c, d;
};

struct Smem {
    union {
        struct {
            uint32_t bin[kBins];
        } fast;
        struct {
            uint64_t sum[kExact];
            uint32_t cnt[kExact];
        } exact;
    };
    union {
        uint64_t stage[kList];  // a CTA's own tokens for the list; rank 0: the list's weights
        uint32_t merged[kBins]; // rank 0's: the cluster's bins
        struct {
            uint64_t sum[kExact];
            uint32_t cnt[kExact];
        } both;
    };
    uint64_t list[kList];       // rank 0's: keys
    uint64_t cta[3][kMaxCluster];
    uint64_t key[kMaxCluster];  // every CTA's first token of the order
    uint64_t warp[kWarps];
    uint64_t wscan[kWarps];
    uint32_t wcnt[kWarps];
    uint32_t low[kMaxCluster];  // every CTA's bound
    float bound;
    Word word;
    int n, total, base;  // tokens staged here, and in all CTAs; where this one's stand among those
};

__device__ __forceinline__ uint32_t ld_cluster(const uint32_t *mine, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(mine, rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t ld_cluster(const uint64_t *mine, uint32_t rank) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(mapa_shared(mine, rank)) : "memory");
    return v;
}
__device__ __forceinline__ void store_cluster_u32(uint32_t *mine, uint32_t rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(mine, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ int add_cluster(int *mine, uint32_t rank, int v) {
    int old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(mapa_shared(mine, rank)), "r"(v) : "memory");
    return old;
}

// ------------------------------------------------------------------ weights
// Two values at a time; every operation is rounded by itself.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t fma2_rz(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t both(float v) { return pack2(v, v); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The weight of a row's logits: 2^y by a polynomial for the fraction, 2^f's closest of the fifth
// degree with 1 at 0 (relative error 2^-23.4, 2^-22.3 as computed).
struct Weigh {
    float m, c;  // the row's largest, log2(e) / temperature
    // The logits as (x - m) c, at least -60, whose weight is 0, as -infinity's and NaN's is.
    __device__ __forceinline__ void octaves(float x0, float x1, float &y0, float &y1) const {
        unpack2(mul2(add2(pack2(x0, x1), both(-m)), both(c)), y0, y1);
        y0 = fmaxf(y0, -60.f);
        y1 = fmaxf(y1, -60.f);
    }
    __device__ __forceinline__ float octaves(float x) const { return fmaxf(__fmul_rn(__fsub_rn(x, m), c), -60.f); }
    // RN(RN(e f) + c).  (A mul.rn.f32x2 and the add.rn.f32x2 after it are put together into one fma, which
    // rounds once; two fma are not.)
    __device__ __forceinline__ static uint64_t step(uint64_t e, uint64_t f, float c) {
        return fma2(fma2(e, f, both(-0.f)), both(1.f), both(c));
    }
    // floor(2^38 2^y): its upper 15 or 16 and its lower 23 bits, each with the bits of 2^23 added to it.
    // (The whole parts of 2^15 p and of 2^23 times the rest appear in the mantissas of sums with
    // 2^23 that are rounded towards zero.)
    __device__ __forceinline__ static void parts(float y0, float y1, uint32_t (&hi)[2], uint32_t (&lo)[2]) {
        const uint64_t y = pack2(y0, y1), magic = both(12582912.f);
        const uint64_t t = add2(y, magic);  // the nearest whole number, in the low bits
        const uint64_t f = fma2(add2(t, both(-12582912.f)), both(-1.f), y);
        uint64_t e = both(0x1.5bba14p-10f);
        e = step(e, f, 0x1.3cea88p-7f);
        e = step(e, f, 0x1.c6b752p-5f);
        e = step(e, f, 0x1.ebf9bcp-3f);
        e = step(e, f, 0x1.62e42ap-1f);
        e = step(e, f, 1.f);
        float e0, e1, t0, t1;
        unpack2(e, e0, e1);
        unpack2(t, t0, t1);
        const uint64_t p = pack2(__uint_as_float(__float_as_uint(e0) + (__float_as_uint(t0) << 23)),
                                 __uint_as_float(__float_as_uint(e1) + (__float_as_uint(t1) << 23)));
        const uint64_t k15 = both(32768.f), k23 = both(8388608.f);
        const uint64_t h = fma2_rz(p, k15, k23);
        const uint64_t rest = fma2(p, k15, fma2(h, both(-1.f), k23));  // exact
        const uint64_t l = fma2_rz(rest, k23, k23);
        hi[0] = (uint32_t)h;
        hi[1] = (uint32_t)(h >> 32);
        lo[0] = (uint32_t)l;
        lo[1] = (uint32_t)(l >> 32);
    }
    __device__ __forceinline__ static uint64_t join(uint32_t hi, uint32_t lo) {
        return ((uint64_t)hi << 23) + lo - kRaw;
    }
    __device__ __forceinline__ static uint64_t weight(float y) {
        uint32_t hi[2], lo[2];
        parts(y, y, hi, lo);
        return join(hi[0], lo[0]);
    }
    __device__ __forceinline__ uint64_t operator()(float x) const { return weight(octaves(x)); }
};

__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ int key_index(uint64_t key) { return (int)(0xffffffffu - (uint32_t)key); }

// The first 24 bits of a number in 0 .. 1 as a whole number (`none` for NaN).
__device__ __forceinline__ uint64_t first_bits(float v, uint64_t none) {
    return v == v ? (uint64_t)(__saturatef(v) * 16777216.f) : none;
}
// total m / 2^24, rounded down, or up.
__device__ __forceinline__ uint64_t share_of(uint64_t total, uint64_t m, bool up) {
    constexpr uint64_t kMask = (1ull << kUniform) - 1;
    return (total >> kUniform) * m + (((total & kMask) * m + (up ? kMask : 0)) >> kUniform);
}

// The digits of an order key by which the exact search divides: 10, 10, 10 and 2 bits of the logit, then
// twice 10 of the index.
__device__ __forceinline__ int digit_shift(int level) { return level < 3 ? 54 - 10 * level : level == 3 ? 32 : level == 4 ? 10 : 0; }
__device__ __forceinline__ int digit_bits(int level) { return level == 3 ? 2 : 10; }

// ------------------------------------------------------- a row, by a cluster
template <bool BF16, bool PROBS>
struct Sampler {
    static constexpr int kVec = Row<BF16, PROBS>::kVec;
    const SampleArgs &a;
    Smem &s;
    const uint32_t rank, ranks;
    const int tid, lane, warp, row;
    const Row<BF16, PROBS> X;  // (the probabilities may be written over the logits)
    int v0, v1;     // this warp's vectors
    bool infinite;  // the row's largest is +infinity: those are 0, everything else -infinity
    Weigh W;

    __device__ __forceinline__ Sampler(const SampleArgs &a_, Smem &s_, int row_)
        : a(a_), s(s_), rank(cluster_ctarank()), ranks(cluster_nctarank()), tid((int)threadIdx.x), lane(tid & 31),
          warp(tid >> 5), row(row_), X(a_.x, (size_t)row * a_.ld, a_.vocab), infinite(false) {
        const int vectors = X.vectors(), per = (vectors + (int)ranks * kWarps - 1) / ((int)ranks * kWarps);
        v0 = min(((int)rank * kWarps + warp) * per, vectors);
        v1 = min(v0 + per, vectors);
    }
    __device__ __forceinline__ bool first() const { return rank == 0; }
    // This thread's first vector where the CTAs' warps take 32 each in turn.
    __device__ __forceinline__ int turn() const { return (warp * (int)ranks + (int)rank) * 32 + lane; }

    __device__ __forceinline__ void load(int v, float (&x)[kVec]) const {
        X.load(v, kNone, x);
        if (infinite) {
#pragma unroll
            for (int j = 0; j < kVec; j++) x[j] = x[j] == INFINITY ? 0.f : kNone;
        }
    }
    // f(vector, its octaves) for this warp's part.
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
#pragma unroll 2
        for (int v = v0 + lane; v < v1; v += 32) {
            float x[kVec], y[kVec];
            load(v, x);
#pragma unroll
            for (int j = 0; j < kVec; j += 2) W.octaves(x[j], x[j + 1], y[j], y[j + 1]);
            f(v, x, y);
        }
    }
    __device__ __forceinline__ void tell(Word w) const {  // (one thread of rank 0)
        for (uint32_t q = 0; q < ranks; q++) {
            store_cluster_u64(&s.word.a, q, w.a);
            store_cluster_u64(&s.word.b, q, w.b);
            store_cluster_u64(&s.word.c, q, w.c);
            store_cluster_u64(&s.word.d, q, w.d);
        }
    }
    __device__ __forceinline__ uint64_t key_of(float x, int i) const { return order_key(x, i); }

    // Sum of the CTAs' values (each thread's own), in all of them; `before`: of the CTAs before this one,
    // `cta`: of this one.  Leaves the warps' sums in s.warp.  A round's slot may be stored to again once a
    // barrier of the cluster stands between: sums that follow one another take different rounds, as the later
    // one's own barrier then frees the earlier one's slot.
    __device__ __forceinline__ uint64_t add_up(uint64_t v, int round, uint64_t &before, uint64_t &cta) const {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        __syncthreads();
        if (lane == 0) s.warp[warp] = v;
        __syncthreads();
        cta = 0;
#pragma unroll
        for (int w = 0; w < kWarps; w++) cta += s.warp[w];
        if (tid < (int)ranks) store_cluster_u64(&s.cta[round][rank], (uint32_t)tid, cta);
        cluster_sync();
        uint64_t total = 0;
        before = 0;
        for (uint32_t q = 0; q < ranks; q++) {
            if (q < rank) before += s.cta[round][q];
            total += s.cta[round][q];
        }
        return total;
    }

    // ------------------------------------------------------------- the list
    __device__ __forceinline__ void stage(float x, int i) const {
        const int at = atomicAdd(&s.n, 1);
        if (at < kList) s.stage[at] = key_of(x, i);
    }
    // Every CTA's staged tokens -> rank 0's list; how many there are (more than kList: not all are on
    // it).  s.n and s.total are 0 in every CTA before the first one is staged.
    __device__ __forceinline__ int collect() const {
        __syncthreads();
        if (tid < (int)ranks) {  // (every CTA is told: rank 0 may be gone before another asks it)
            const int base = add_cluster(&s.total, (uint32_t)tid, s.n);
            if (tid == 0) s.base = base;
        }
        __syncthreads();
        const int n = min(s.n, kList), base = s.base;
        for (int i = tid; i < n && base + i < kList; i += kThreads) store_cluster_u64(&s.list[base + i], 0, s.stage[i]);
        cluster_sync();
        return s.total;
    }
    // Rank 0: a list of n values sorted to fall; the places up to the next power of two are 0.
    __device__ __forceinline__ void sort(uint64_t *v, int n) const {
        int size = 32;
        while (size < n) size *= 2;
        for (int i = n + tid; i < size; i += kThreads) v[i] = 0;
        __syncthreads();
        for (int k = 2; k <= size; k *= 2) {
            for (int j = k / 2; j > 0; j /= 2) {
                for (int p = tid; p < size / 2; p += kThreads) {
                    const int i = 2 * p - (p & (j - 1)), o = i + j;
                    const uint64_t x = v[i], y = v[o];
                    if ((x < y) == ((i & k) == 0)) v[i] = y, v[o] = x;
                }
                __syncthreads();
            }
        }
    }
    // Rank 0: the list's n keys sorted to fall, by bins that rise as the keys fall (bin(key) in 0 .. kBins -
    // 1): a place in the bin's stretch of the list for each, then its place among those.  Where many
    // share a bin, by comparing and exchanging.
    template <typename F>
    __device__ __forceinline__ void sort_by(int n, F bin) const {
        constexpr int kPer = kList / kThreads, kPerBin = kBins / kThreads;
        for (int i = tid; i < kBins / 4; i += kThreads) reinterpret_cast<uint4 *>(s.fast.bin)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        uint64_t key[kPer];
        int at[kPer];
        uint32_t place[kPer];
        bool crowded = false;
#pragma unroll
        for (int j = 0; j < kPer; j++) {
            const int i = tid + j * kThreads;
            if (i >= n) continue;
            key[j] = s.list[i];
            at[j] = bin(key[j]);
            place[j] = atomicAdd(s.fast.bin + at[j], 1u);
            crowded |= place[j] >= 64;
        }
        if (__syncthreads_or(crowded)) return sort(s.list, n);
        uint32_t c = 0, cnt[kPerBin];
#pragma unroll
        for (int i = 0; i < kPerBin; i++) cnt[i] = s.fast.bin[tid * kPerBin + i], c += cnt[i];
        uint32_t upto = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += o;
        }
        if (lane == 31) s.wcnt[warp] = upto;
        __syncthreads();
        upto -= c;
        for (int w = 0; w < warp; w++) upto += s.wcnt[w];
#pragma unroll
        for (int i = 0; i < kPerBin; i++) {
            s.fast.bin[tid * kPerBin + i] = upto;
            upto += cnt[i];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kPer; j++)
            if (tid + j * kThreads < n) s.stage[s.fast.bin[at[j]] + place[j]] = key[j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kPer; j++) {
            if (tid + j * kThreads >= n) continue;
            const int first = (int)s.fast.bin[at[j]], end = at[j] + 1 < kBins ? (int)s.fast.bin[at[j] + 1] : n;
            int p = first;
            for (int i = first; i < end; i++) p += s.stage[i] > key[j] ? 1 : 0;
            s.list[p] = key[j];
        }
        __syncthreads();
    }
    // ... of a list whose octaves lie between -from and -to
    __device__ __forceinline__ void sort_list(int n, float from, float to) const {
        const float scale = (float)kBins / fmaxf(to - from, 0x1p-10f);
        sort_by(n, [&](uint64_t key) {
            return max(0, min((int)((-W.octaves(key_value(key)) - from) * scale), kBins - 1));
        });
    }
    // Rank 0: running sums of f(i), i < n, in place of the values: out[i] = f(0) + .. + f(i).
    template <typename F>
    __device__ __forceinline__ void scan(uint64_t *out, int n, F f) const {
        constexpr int kPer = kList / kThreads;
        uint64_t v[kPer], sum = 0;
        for (int i = 0; i < kPer; i++) {
            const int at = tid * kPer + i;
            sum += at < n ? f(at) : 0;
            v[i] = sum;
        }
        uint64_t upto = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint64_t o = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += o;
        }
        __syncthreads();
        if (lane == 31) s.wscan[warp] = upto;
        __syncthreads();
        upto -= sum;
        for (int w = 0; w < warp; w++) upto += s.wscan[w];
        for (int i = 0; i < kPer; i++)
            if (tid * kPer + i < n) out[tid * kPer + i] = upto + v[i];
        __syncthreads();
    }
    __device__ __forceinline__ uint64_t listed(int i) const {
        const float x = key_value(s.list[i]);
        return W(x);
    }

    // ------------------------------------------------------------ output
    __device__ __forceinline__ void put(int i, float p) const {
        if (BF16)
            (static_cast<uint16_t *>(a.probs) + (size_t)row * a.ldp)[i] = __bfloat16_as_ushort(__float2bfloat16(p));
        else
            (static_cast<float *>(a.probs) + (size_t)row * a.ldp)[i] = p;
    }
    // Zeros in this CTA's part of the row.
    __device__ __forceinline__ void clear_row() const {
        const int per = (a.vocab + (int)ranks - 1) / (int)ranks;
        const int i0 = min((int)rank * per, a.vocab), i1 = min(i0 + per, a.vocab);
        constexpr int kSize = BF16 ? 2 : 4;
        uint8_t *p = static_cast<uint8_t *>(a.probs) + ((size_t)row * a.ldp + i0) * kSize;
        uint8_t *end = p + (size_t)(i1 - i0) * kSize;
        uint8_t *q = (uint8_t *)(((uintptr_t)p + 15) & ~(uintptr_t)15), *qe = (uint8_t *)((uintptr_t)end & ~(uintptr_t)15);
        if (q > qe) q = qe = end;
        for (uint8_t *t = p + tid * kSize; t < q; t += kThreads * kSize) zero(t);
        for (uint8_t *t = q + tid * 16; t < qe; t += kThreads * 16) *reinterpret_cast<uint4 *>(t) = make_uint4(0, 0, 0, 0);
        for (uint8_t *t = qe + tid * kSize; t < end; t += kThreads * kSize) zero(t);
    }
    __device__ __forceinline__ static void zero(uint8_t *t) {
        if (BF16)
            *reinterpret_cast<uint16_t *>(t) = 0;
        else
            *reinterpret_cast<uint32_t *>(t) = 0;
    }

    // All that may be kept is on rank 0's list, n tokens of it: the cuts, and the draw or the
    // probabilities.  lim: what the weights before a kept one are below; 0: by `part` of the first k.  to: the
    // list's octaves are above -to.
    __device__ __forceinline__ void finish(int n, bool by_count, int k, uint64_t part, uint64_t lim, uint64_t least,
                                           float to) const {
        if (PROBS) {
            clear_row();
            cluster_sync();
        }
        if (!first()) return;
        if (n <= kFew) return finish_few(n, by_count ? k : n, part, lim, least);
        sort_list(n, 0.f, to);
        if (by_count) n = min(n, k);
        uint64_t *upto = s.stage;
        scan(upto, n, [&](int i) { return listed(i); });
        if (lim == 0) lim = share_of(upto[n - 1], part, true);
        auto kept = [&](int i) -> uint64_t {
            const uint64_t before = i > 0 ? upto[i - 1] : 0, w = upto[i] - before;
            return before < lim && w >= least ? w : 0;
        };
        if (PROBS) {
            uint64_t sum = 0;
            for (int i = tid; i < n; i += kThreads) sum += kept(i);
            sum = cta_sum(sum);
            const float all = __ull2float_rn(sum);
            for (int i = tid; i < n; i += kThreads) {
                const uint64_t w = kept(i);
                if (w != 0) put(key_index(s.list[i]), __fdiv_rn(__ull2float_rn(w), all));
            }
            return;
        }
        // the kept ones by index: (2^20 - 1 - index, weight)
        constexpr int kPer = kList / kThreads;
        uint64_t mine[kPer];
        for (int j = 0; j < kPer; j++) {
            const int i = tid + j * kThreads;
            const uint64_t w = i < n ? kept(i) : 0;
            mine[j] = w == 0 ? 0 : (uint64_t)(0xfffff - key_index(s.list[i])) << 39 | w;
        }
        if (tid == 0) s.n = 0;
        __syncthreads();
        for (int j = 0; j < kPer; j++)
            if (mine[j] != 0) s.list[atomicAdd(&s.n, 1)] = mine[j];
        __syncthreads();
        n = s.n;
        const int shift = max(0, 32 - __clz(a.vocab) - 11);
        sort_by(n, [&](uint64_t key) { return (0xfffff - (int)(key >> 39)) >> shift; });
        constexpr uint64_t kWeight = (1ull << 39) - 1;
        scan(upto, n, [&](int i) { return s.list[i] & kWeight; });
        const uint64_t aim = share_of(upto[n - 1], whole_uniform(a.u[row]), false);
        for (int i = tid; i < n; i += kThreads)
            if (upto[i] > aim && (i == 0 || upto[i - 1] <= aim)) a.next[row] = 0xfffff - (int)(s.list[i] >> 39);
    }
    // Of at most kFew listed tokens, thread 2 i and 2 i + 1's: its key and weight (0 behind the last), and how
    // many stand before it and what they weigh.  Leaves the keys and weights in pairs in s.stage.
    __device__ __forceinline__ void compare(int n, uint64_t &key, uint64_t &w, int &rank_, uint64_t &before) const {
        static_assert(2 * kFew <= kThreads && 2 * kFew <= kList, "two threads a token");
        ulonglong2 *pair = reinterpret_cast<ulonglong2 *>(s.stage);
        const int i = tid >> 1;
        key = w = before = 0;
        rank_ = 0;
        if (i < n) {
            key = s.list[i];
            w = W(key_value(key));
            if ((tid & 1) == 0) pair[i] = make_ulonglong2(key, w);
        }
        __syncthreads();
        if (i - (lane >> 1) < n) {  // (whole warps)
            for (int j = tid & 1; j < n; j += 2) {
                const ulonglong2 o = pair[j];
                if (o.x > key) {
                    before += o.y;
                    rank_++;
                }
            }
        }
        before += __shfl_xor_sync(0xffffffffu, before, 1);
        rank_ += __shfl_xor_sync(0xffffffffu, rank_, 1);
    }
    // The same for at most kFew tokens: each is compared with all, by two threads.
    __device__ __forceinline__ void finish_few(int n, int k, uint64_t part, uint64_t lim, uint64_t least) const {
        ulonglong2 *pair = reinterpret_cast<ulonglong2 *>(s.stage);
        const int i = tid >> 1;
        uint64_t key, w, before;
        int rank_;
        compare(n, key, w, rank_, before);
        const bool mine = i < n && rank_ < k;
        if (lim == 0) lim = share_of(cta_sum(mine && (tid & 1) == 0 ? w : 0), part, true);
        if (!mine || before >= lim || w < least) w = 0;
        const uint64_t total = cta_sum((tid & 1) == 0 ? w : 0);
        const int index = key_index(key);
        if (PROBS) {
            if (w != 0 && (tid & 1) == 0) put(index, __fdiv_rn(__ull2float_rn(w), __ull2float_rn(total)));
            return;
        }
        if (i < n && (tid & 1) == 0) pair[i] = make_ulonglong2(key, w);  // (all have read it: sums lie between)
        __syncthreads();
        before = 0;  // of lower indices
        if (i - (lane >> 1) < n) {
            for (int j = tid & 1; j < n; j += 2) {
                const ulonglong2 o = pair[j];
                if (key_index(o.x) < index) before += o.y;
            }
        }
        before += __shfl_xor_sync(0xffffffffu, before, 1);
        const uint64_t aim = share_of(total, whole_uniform(a.u[row]), false);
        if (w != 0 && (tid & 1) == 0 && before <= aim && aim < before + w) a.next[row] = index;
    }
    __device__ __forceinline__ uint64_t cta_sum(uint64_t v) const {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        __syncthreads();
        if (lane == 0) s.warp[warp] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int w = 0; w < kWarps; w++) v += s.warp[w];
        return v;
    }

    // ------------------------------------------------------- counts by bins
    __device__ __forceinline__ void clear_bins() const {
        for (int i = tid; i < kBins / 4; i += kThreads) reinterpret_cast<uint4 *>(s.fast.bin)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }
    __device__ __forceinline__ void clear_counts() const {
        if (tid == 0) s.n = s.total = 0;
        cluster_sync();  // (other CTAs add to s.total)
    }
    // A bound that k values of this CTA do not fall below, from the largest of each part of the
    // threads' values, or from all of them; -infinity if those do not tell.  `top`: the largest.
    __device__ __forceinline__ float bound_of(const float (&tops)[kSubs], float top, int k, bool all) const {
        constexpr float kPerUnit = 16.f * 1.442695f;
        if (tid == 0) s.bound = kNone;
        auto count = [&](float x) {
            if (!(x > kNone)) return;
            const float d = (top - x) * kPerUnit;
            if (!(d >= (float)kBins)) atomicAdd(s.fast.bin + (int)d, 1u);  // (NaN, of infinities: 0)
        };
        if (all) {
            for (int v = turn(); v < X.vectors(); v += (int)ranks * kThreads) {
                float x[kVec];
                X.load(v, kNone, x);
#pragma unroll
                for (int j = 0; j < kVec; j++) count(x[j]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kSubs; i++) count(tops[i]);
        }
        __syncthreads();
        constexpr int kPer = kBins / kThreads;
        uint32_t c = 0, cnt[kPer];
#pragma unroll
        for (int i = 0; i < kPer; i++) cnt[i] = s.fast.bin[tid * kPer + i], c += cnt[i];
        uint32_t upto = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += o;
        }
        if (lane == 31) s.wcnt[warp] = upto;
        __syncthreads();
        upto -= c;
        for (int w = 0; w < warp; w++) upto += s.wcnt[w];
        for (int i = 0; i < kPer; i++) {
            if (upto < (uint32_t)k && upto + cnt[i] >= (uint32_t)k) {
                const float below = (float)(tid * kPer + i + 1) / kPerUnit;
                s.bound = top == INFINITY ? top : top - below - (fabsf(top) + below) * 0x1p-20f;  // (whatever was rounded)
            }
            upto += cnt[i];
        }
        __syncthreads();
        return s.bound;
    }
    // The cluster's bins -> rank 0, each CTA a part of them.
    __device__ __forceinline__ void merge_bins() const {
        cluster_sync();
        const int per = (kBins + (int)ranks - 1) / (int)ranks, end = min((int)(rank + 1) * per, kBins);
        for (int i = (int)rank * per + tid; i < end; i += kThreads) {
            uint32_t c = 0;
            for (uint32_t q = 0; q < ranks; q++) c += ld_cluster(s.fast.bin + i, q);
            store_cluster_u32(s.merged + i, 0, c);
        }
        cluster_sync();
    }

    // A value's bin, as the whole number that u = place(y) is 2^23 more than.
    __device__ __forceinline__ static float place(float y, float scale) { return __fmaf_rz(-y, scale, 8388608.f); }

    // The bins [b0, b1] in which the weights reach `target` of `total`, for the values from `least_y` on: from the
    // weights in units of total / 2^31, rounded, so that sums are off by half the vocabulary at most.
    __device__ __forceinline__ void share_bins(float scale, float least_y, uint64_t target, uint64_t total, int &b0, int &b1) const {
        const float all = (float)total * 0x1p-38f, up = 31.f - log2f(all);
        each([&](int, const float(&)[kVec], const float (&y)[kVec]) {
#pragma unroll
            for (int j = 0; j < kVec; j++)
                if (y[j] >= least_y)
                    atomicAdd(s.fast.bin + (__float_as_uint(place(y[j], scale)) & (kBins - 1)), (uint32_t)__float2int_rn(ex2(y[j] + up)));
        });
        merge_bins();
        if (first()) {
            constexpr int kPer = kBins / kThreads;
            // (half a unit a value; the exponentials are off by a part in 2^20, and two roundings of 2^-23 of
            // 31; the sums and shares by 2^-22)
            const uint32_t slack = (uint32_t)a.vocab / 2 + (1u << 13);
            const uint32_t want = (uint32_t)__float2int_rn((float)target / (float)total * 0x1p31f * 0.9999999f);
            const uint32_t may = want > slack ? want - slack : 1, must = want + slack;
            uint32_t c = 0, cnt[kPer];
#pragma unroll
            for (int i = 0; i < kPer; i++) cnt[i] = s.merged[tid * kPer + i], c += cnt[i];
            uint32_t upto = c;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += o;
            }
            if (lane == 31) s.wcnt[warp] = upto;
            __syncthreads();
            upto -= c;
            for (int w = 0; w < warp; w++) upto += s.wcnt[w];
            for (int i = 0; i < kPer; i++) {
                const uint32_t next = upto + cnt[i];
                if (upto < may && next >= may)
                    for (uint32_t q = 0; q < ranks; q++) store_cluster_u64(&s.word.a, q, (uint64_t)(tid * kPer + i));
                if ((upto < must && next >= must) || (next < must && tid * kPer + i == kBins - 1))
                    for (uint32_t q = 0; q < ranks; q++) store_cluster_u64(&s.word.b, q, (uint64_t)(tid * kPer + i));
                upto = next;
            }
        }
        cluster_sync();
        b0 = (int)s.word.a;
        b1 = (int)s.word.b;
    }

    // ------------------------------------------- exact search, digit by digit
    // Rank 0: the token of a list whose octaves lie between -from and -to at which tokens, or weights, reach
    // `target`, c0 and w0 of them being before the list: told with the weights up to and with it (0: none).
    __device__ __forceinline__ void resolve(int n, float from, float to, bool weights, uint64_t c0, uint64_t w0,
                                            uint64_t target) const {
        if (tid == 0) tell(Word{0, 0, 0, 0});
        auto look = [&](uint64_t key, uint64_t rank_, uint64_t before, uint64_t w) {
            const bool is = weights ? w0 + before < target && target <= w0 + before + w : c0 + rank_ + 1 == target;
            if (is) tell(Word{key, w0 + before + w, 0, 0});
        };
        if (n <= kFew) {
            uint64_t key, w, before;
            int rank_;
            compare(n, key, w, rank_, before);  // (a barrier in it stands between the tellings)
            if ((tid & 1) == 0 && (tid >> 1) < n) look(key, (uint64_t)rank_, before, w);
            return;
        }
        sort_list(n, from, to);
        uint64_t *upto = s.stage;
        scan(upto, n, [&](int i) { return listed(i); });
        for (int i = tid; i < n; i += kThreads) {
            const uint64_t before = i > 0 ? upto[i - 1] : 0;
            look(s.list[i], (uint64_t)i, before, upto[i] - before);
        }
    }

    // The token at which tokens, or weights, reach `target` in the order: its key, and the weights up to
    // and with it.
    __device__ __noinline__ uint64_t search(bool weights, uint64_t target, uint64_t &upto) const {
        uint64_t prefix = 0, c0 = 0, w0 = 0;
#pragma unroll 1
        for (int level = 0; level < 6; level++) {
            const int shift = digit_shift(level), mask = (1 << digit_bits(level)) - 1;
            // the digits so far (between the logit's and the index's stand constant bits)
            const int above = level == 0 ? 64 : digit_shift(level - 1);
            auto in = [&](uint64_t key) { return level == 0 || key >> above == prefix; };
            cluster_sync();  // the word is read, and the bins
            for (int i = tid; i < kExact; i += kThreads) s.exact.cnt[i] = 0, s.exact.sum[i] = 0;
            __syncthreads();
            each([&](int v, const float (&x)[kVec], const float (&y)[kVec]) {
#pragma unroll
                for (int j = 0; j < kVec; j++) {
                    if (!(y[j] > -kReach)) continue;
                    const uint64_t key = key_of(x[j], X.first(v) + j);
                    if (!in(key)) continue;
                    const int d = mask - (int)(key >> shift & mask);
                    atomicAdd(s.exact.cnt + d, 1u);
                    atomicAdd((unsigned long long *)(s.exact.sum + d), (unsigned long long)Weigh::weight(y[j]));
                }
            });
            cluster_sync();
            // each CTA adds up a part of the bins, for rank 0
            const int per = (kExact + (int)ranks - 1) / (int)ranks, end = min((int)(rank + 1) * per, kExact);
            for (int i = (int)rank * per + tid; i < end; i += kThreads) {
                uint32_t c = 0;
                uint64_t w = 0;
                for (uint32_t q = 0; q < ranks; q++) c += ld_cluster(s.exact.cnt + i, q), w += ld_cluster(s.exact.sum + i, q);
                store_cluster_u64(&s.both.sum[i], 0, w);
                store_cluster_u32(&s.both.cnt[i], 0, c);
            }
            cluster_sync();
            if (first()) {
                constexpr int kPer = kExact / kThreads;
                uint32_t c = 0;
                uint64_t w = 0;
                for (int i = 0; i < kPer; i++) c += s.both.cnt[tid * kPer + i], w += s.both.sum[tid * kPer + i];
                uint32_t uc = c;
                uint64_t uw = w;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t oc = __shfl_up_sync(0xffffffffu, uc, d);
                    const uint64_t ow = __shfl_up_sync(0xffffffffu, uw, d);
                    if (lane >= d) uc += oc, uw += ow;
                }
                if (lane == 31) s.wcnt[warp] = uc, s.wscan[warp] = uw;
                __syncthreads();
                for (int q = 0; q < warp; q++) uc += s.wcnt[q], uw += s.wscan[q];
                uint64_t bc = c0 + uc - c, bw = w0 + uw - w;
                for (int i = 0; i < kPer; i++) {
                    const uint32_t cnt = s.both.cnt[tid * kPer + i];
                    const uint64_t sum = s.both.sum[tid * kPer + i];
                    const uint64_t before = weights ? bw : bc, here = weights ? sum : cnt;
                    if (before < target && target <= before + here) tell(Word{(uint64_t)(tid * kPer + i), bc, bw, cnt});
                    bc += cnt;
                    bw += sum;
                }
            }
            cluster_sync();
            const uint64_t d = (uint64_t)mask - s.word.a;
            prefix = level == 4 ? (prefix << 22) | (0xfffull << 10) | d : (prefix << digit_bits(level)) | d;
            c0 = s.word.b;
            w0 = s.word.c;
            if (s.word.d <= kList) {  // the rest on the list
                clear_counts();
                each([&](int v, const float (&x)[kVec], const float (&y)[kVec]) {
#pragma unroll
                    for (int j = 0; j < kVec; j++)
                        if (y[j] > -kReach) {
                            const uint64_t key = key_of(x[j], X.first(v) + j);
                            if (key >> shift == prefix) stage(x[j], X.first(v) + j);
                        }
                });
                const int n = collect();
                if (first()) {
                    resolve(n, 0.f, kReach, weights, c0, w0, target);
                }
                cluster_sync();
                break;
            }
        }
        upto = s.word.b;
        return s.word.a;
    }

    // -------------------------------------------------------------- the row
    __device__ __forceinline__ void run() {
        cluster_arrive();  // waited for before the first remote store: by then every CTA has started
        // the first token of the order: the largest value of each vector, and the first vector that has it
        // (vectors rise in each thread); NaN is passed over
        const int k = a.top_k != nullptr ? a.top_k[row] : 0;
        const bool by_count = k > 0 && k < a.vocab, lead = by_count && k <= kSmallK && a.vocab > kList;
        float top = kNone, tops[kSubs];
        int top_v = -1;
        // (here the CTAs and the parts of a thread take turns, so that each has its share of the large values
        // wherever in the vocabulary they lie)
        const int step = (int)ranks * kThreads, from = turn();
#pragma unroll
        for (int i = 0; i < kSubs; i++) tops[i] = kNone;
#pragma unroll 2
        for (int v = from; v < X.vectors(); v += kSubs * step) {
            float m[kSubs];
#pragma unroll
            for (int i = 0; i < kSubs; i++) m[i] = v + i * step < X.vectors() ? X.largest(v + i * step) : kNone;
#pragma unroll
            for (int i = 0; i < kSubs; i++) {
                tops[i] = fmaxf(tops[i], m[i]);
                if (m[i] > top) {
                    top = m[i];
                    top_v = v + i * step;
                }
            }
        }
        uint64_t key = 0;
        if (top_v >= 0) {
            float x[kVec];
            X.load(top_v, kNone, x);
#pragma unroll
            for (int j = kVec - 1; j >= 0; j--)
                if (x[j] == top) key = order_key(x[j], X.first(top_v) + j);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, d));
        if (lane == 0) s.warp[warp] = key;
        clear_bins();
        for (int w = 0; w < kWarps; w++) key = max(key, s.warp[w]);
        const float bound = lead ? bound_of(tops, key != 0 ? key_value(key) : 0.f, (k + (int)ranks - 1) / (int)ranks,
                                          // (too few vectors for their largest to tell a small list)
                                          a.vocab < 4 * kVec * k)
                               : kNone;
        cluster_wait();
        if (tid < (int)ranks) {
            store_cluster_u64(s.key + rank, (uint32_t)tid, key);  // (a place of its own: a sum may follow at once)
            store_cluster_u32(&s.low[rank], (uint32_t)tid, __float_as_uint(bound));
        }
        cluster_sync();
        float low = INFINITY;
        for (uint32_t q = 0; q < ranks; q++) {
            key = max(key, s.key[q]);
            low = fminf(low, __uint_as_float(s.low[q]));
        }

        const float T = a.temperature[row];
        if (key == 0 || !(T > 0.f)) {  // nothing to draw from, or nothing to draw
            if (PROBS) {
                clear_row();
                cluster_sync();
                if (first() && tid == 0 && key != 0) put(key_index(key), 1.f);
            } else if (first() && tid == 0) {
                a.next[row] = key == 0 ? -1 : key_index(key);
            }
            return;
        }
        const float low_ = low;  // (before infinities are put in place)
        W.m = key_value(key);
        W.c = fminf(__fdiv_rn(0x1.715476p+0f, T), 3.4028235e38f);
        infinite = W.m == INFINITY;
        if (infinite) {
            W.m = 0.f;
            low = low == INFINITY ? 0.f : kNone;
        }
        const uint64_t part = a.top_p != nullptr ? max(first_bits(a.top_p[row], 1ull << kUniform), (uint64_t)1) : 1ull << kUniform;
        const uint64_t least = a.min_p != nullptr ? first_bits(a.min_p[row], 0) << (kGrid - kUniform) : 0;
        const bool by_share = part < 1ull << kUniform;

        uint64_t cut = 0, before, cta;  // tokens below this key are not kept
        if (by_count || by_share) {
            bool found = false;
            if (a.vocab <= kList || low > kNone) {
                // the tokens from `low` on, among which the first k are (a small vocabulary: all)
                clear_counts();
#pragma unroll 4
                for (int v = from; v < X.vectors(); v += step) {
                    if (!(X.largest(v) >= low_)) continue;
                    float x[kVec];
                    load(v, x);
#pragma unroll
                    for (int j = 0; j < kVec; j++)
                        if (x[j] >= low && x[j] > kNone) stage(x[j], X.first(v) + j);
                }
                const int n = collect();
                if (n <= kList) return finish(n, by_count, k, part, 0, least, fminf(-W.octaves(low), kReach));
            } else if (!by_count) {
                uint64_t sum = 0;
                each([&](int, const float(&)[kVec], const float (&y)[kVec]) { sum += weights_of(y); });
                const uint64_t total = add_up(sum, 1, before, cta), target = share_of(total, part, true);
                // What weighs less than (total - target) / vocab comes after the cut, as all of it together
                // weighs less than what is not kept.
                const float least_y = fmaxf(log2f((float)(total - target) / (float)a.vocab) - 38.01f, 0.1f - kReach);
                const float scale = (float)kBins / fmaxf(-least_y, 0x1p-10f) * 0.9999f;
                int b0, b1;
                clear_bins();
                share_bins(scale, least_y, target, total, b0, b1);
                clear_counts();
                // (so few can weigh as much as the last bin's end that all of them go on the list)
                const bool whole_list = (float)total <= 0.99f * (float)kList * exp2f(38.f - (float)(b1 + 1) / scale);
                const float from = 8388608.f + (float)(whole_list ? 0 : b0), to = 8388608.f + (float)(b1 + 1);
                uint64_t above = 0;
                each([&](int v, const float (&x)[kVec], const float (&y)[kVec]) {
                    float z[kVec];
                    bool any = false;
#pragma unroll
                    for (int j = 0; j < kVec; j++) {
                        const float u = place(y[j], scale);
                        const bool before_ = u < from;
                        if (!before_ && u < to && y[j] >= least_y) stage(x[j], X.first(v) + j);
                        z[j] = before_ ? y[j] : -60.f;
                        any |= before_;
                    }
                    if (any) above += weights_of(z);
                });
                const uint64_t sum_above = add_up(above, 0, before, cta);
                const int n = collect();
                if (n <= kList && n > 0) {
                    if (whole_list) return finish(n, false, 0, 0, target, least, (float)(b1 + 1) / scale);
                    if (first()) {
                        resolve(n, (float)b0 / scale, (float)(b1 + 1) / scale, true, 0, sum_above, target);
                    }
                    cluster_sync();
                    cut = s.word.a;
                    found = cut != 0;
                    if (found && least == 0) {
                        // the kept weights by parts: those above the bins, and the list's
                        if (first())
                            for (int i = tid; i < n; i += kThreads) add_listed(s.list[i], cut);
                        else
                            for (int i = tid; i < s.n; i += kThreads) add_listed(s.stage[i], cut);
                        __syncthreads();
                        return draw(cut, 0, true);
                    }
                }
            }
            if (!found) {
                uint64_t live = 0, sum = 0;
                each([&](int, const float(&)[kVec], const float (&y)[kVec]) {
#pragma unroll
                    for (int j = 0; j < kVec; j++) live += y[j] > -kReach ? 1 : 0;
                    sum += weights_of(y);
                });
                live = add_up(live, 0, before, cta);
                uint64_t total = add_up(sum, 1, before, cta), upto;
                if (by_count && (uint64_t)k < live) cut = search(false, (uint64_t)k, total);
                if (by_share) cut = search(true, share_of(total, part, true), upto);
            }
        }
        draw(cut, least, false);
    }
    // A listed token's weight, if it is kept and of this CTA's part, to its warp's sum.
    __device__ __forceinline__ void add_listed(uint64_t key, uint64_t cut) const {
        const int per = (X.vectors() + (int)ranks * kWarps - 1) / ((int)ranks * kWarps);
        const int w = (key_index(key) + X.lead) / kVec / per - (int)rank * kWarps;
        if (key >= cut && w >= 0 && w < kWarps)
            atomicAdd((unsigned long long *)(s.warp + w), (unsigned long long)W(key_value(key)));
    }

    // ------------------------------------------------- kept weights by parts
    __device__ __forceinline__ static uint64_t weights_of(const float (&y)[kVec]) {
        uint32_t h = 0, l = 0;  // (sums of 8 upper and lower bits at most, without the bits of 2^23)
#pragma unroll
        for (int j = 0; j < kVec; j += 2) {
            uint32_t hi[2], lo[2];
            Weigh::parts(y[j], y[j + 1], hi, lo);
            h += hi[0] + hi[1];
            l += lo[0] + lo[1];
        }
        h -= kVec * 0x4b000000u;
        l -= kVec * 0x4b000000u;
        return ((uint64_t)h << 23) + l;
    }
    // The octaves of vector v's values that stand before or at the cut (of others: -60).
    __device__ __forceinline__ void before_cut(int v, uint64_t cut, float (&y)[kVec]) const {
        float x[kVec];
        load(v, x);
        const float cx = cut != 0 ? key_value(cut) : kNone;
        const int last = cut != 0 ? key_index(cut) - X.first(v) : kVec;  // (of values that equal the cut's)
#pragma unroll
        for (int j = 0; j < kVec; j++) x[j] = x[j] > cx || (x[j] == cx && j <= last) ? x[j] : kNone;
#pragma unroll
        for (int j = 0; j < kVec; j += 2) W.octaves(x[j], x[j + 1], y[j], y[j + 1]);
    }
    // The weights of vector v that stand before or at the cut and weigh at least `least`.
    __device__ __forceinline__ void kept(int v, uint64_t cut, uint64_t least, uint64_t (&w)[kVec]) const {
        float y[kVec];
        before_cut(v, cut, y);
#pragma unroll
        for (int j = 0; j < kVec; j += 2) {
            uint32_t hi[2], lo[2];
            Weigh::parts(y[j], y[j + 1], hi, lo);
#pragma unroll
            for (int i = 0; i < 2; i++) {
                w[j + i] = Weigh::join(hi[i], lo[i]);
                if (w[j + i] < least) w[j + i] = 0;
            }
        }
    }
    // The probabilities of vector v: its kept weights by their sum, the reciprocal of which is r.
    __device__ __forceinline__ void put_vector(int v, uint64_t cut, float least, float all, float r) const {
        float y[kVec], p[kVec];
        before_cut(v, cut, y);
#pragma unroll
        for (int j = 0; j < kVec; j += 2) {
            uint32_t hi[2], lo[2];
            Weigh::parts(y[j], y[j + 1], hi, lo);
#pragma unroll
            for (int i = 0; i < 2; i++) {
                // (24 significant bits at most: exact)
                float w = fmaf(__uint_as_float(hi[i]) - 8388608.f, 8388608.f, __uint_as_float(lo[i]) - 8388608.f);
                w = w < least ? 0.f : w;
                // Markstein's division: with the rounded reciprocal, one step from the rounded product gives
                // the rounded quotient
                const float q = __fmul_rn(w, r);
                p[j + i] = fmaf(fmaf(-q, all, w), r, q);
            }
        }
        const int i0 = X.first(v);
        constexpr int kSize = BF16 ? 2 : 4;
        uint8_t *to = static_cast<uint8_t *>(a.probs) + ((ptrdiff_t)((size_t)row * a.ldp) + i0) * kSize;
        if (X.whole_vector(v) && ((uintptr_t)to & 15u) == 0) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                if constexpr (BF16) {
                    const __nv_bfloat162 z = __floats2bfloat162_rn(p[2 * k], p[2 * k + 1]);
                    u[k] = *reinterpret_cast<const uint32_t *>(&z);
                } else {
                    u[k] = __float_as_uint(p[k]);
                }
            }
            *reinterpret_cast<uint4 *>(to) = make_uint4(u[0], u[1], u[2], u[3]);
        } else {
#pragma unroll
            for (int j = 0; j < kVec; j++)
                if (i0 + j >= 0 && i0 + j < a.vocab) put(i0 + j, p[j]);
        }
    }
    __device__ __forceinline__ uint64_t kept_sum(int v, int end, uint64_t cut, uint64_t least) const {
        uint64_t sum = 0;
#pragma unroll 2
        for (; v < end; v += 32) {
            uint64_t w[kVec];
            kept(v, cut, least, w);
#pragma unroll
            for (int j = 0; j < kVec; j++) sum += w[j];
        }
        return sum;
    }
    // The draw (or the probabilities) from the kept weights; `known`: the warps' sums of them are in s.warp.
    __device__ __forceinline__ void draw(uint64_t cut, uint64_t least, bool known) const {
        uint64_t before, cta;
        const uint64_t mine = known ? (lane == 0 ? s.warp[warp] : 0) : kept_sum(v0 + lane, v1, cut, least);
        const uint64_t total = add_up(mine, 2, before, cta);
        if (PROBS) {
            const float all = __ull2float_rn(total), inv = __fdiv_rn(1.f, all), at_least = (float)least;
#pragma unroll 2
            for (int v = v0 + lane; v < v1; v += 32) put_vector(v, cut, at_least, all, inv);
            return;
        }
        const uint64_t aim = share_of(total, whole_uniform(a.u[row]), false);
        if (aim < before || aim >= before + cta) return;  // in another CTA's part
        // the warp whose part holds the point; the CTA's warps divide that part
        int w = 0;
        for (; w < kWarps - 1 && aim >= before + s.warp[w]; w++) before += s.warp[w];
        const int per = (X.vectors() + (int)ranks * kWarps - 1) / ((int)ranks * kWarps);
        const int a0 = min(((int)rank * kWarps + w) * per, X.vectors()), a1 = min(a0 + per, X.vectors());
        const int sub = (a1 - a0 + kWarps - 1) / kWarps, b0 = min(a0 + warp * sub, a1), b1 = min(b0 + sub, a1);
        uint64_t sum = kept_sum(b0 + lane, b1, cut, least);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        __syncthreads();
        if (lane == 0) s.warp[warp] = sum;
        __syncthreads();
        for (int q = 0; q < warp; q++) before += s.warp[q];
        if (aim < before || aim >= before + sum) return;
        for (int v = b0; v < b1; v += 32) {
            uint64_t x[kVec], mine = 0;
            if (v + lane < b1) {
                kept(v + lane, cut, least, x);
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
                a.next[row] = found;
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
            if (before > aim) break;
        }
    }
};

// The row that cluster `unit` takes where not all are under way at once: first those whose share of the
// weights is asked for without a top-k, which take two to three times as long.  (256 rows of 131072, a twelfth
// of them such: 127 us, in their order 148.)
__device__ __forceinline__ int row_of(const SampleArgs &a, Smem &s, int unit) {
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int slow = 0, mine = -1;  // slow rows so far
    for (int round = 0; round < 2; round++) {
        const int all = slow;  // (in the second round)
        slow = 0;
        for (int r0 = 0; r0 < a.rows; r0 += kThreads) {
            const int r = r0 + tid;
            bool f = false;
            if (r < a.rows && a.temperature[r] > 0.f && a.top_p[r] < 1.f) {
                const int k = a.top_k != nullptr ? a.top_k[r] : 0;
                f = !(k > 0 && k <= kSmallK);
            }
            const uint32_t m = __ballot_sync(0xffffffffu, f);
            __syncthreads();
            if (lane == 0) s.wcnt[warp] = (uint32_t)__popc(m);
            __syncthreads();
            int before = slow + __popc(m & ((1u << lane) - 1u));
            for (int w = 0; w < kWarps; w++) {
                if (w < warp) before += (int)s.wcnt[w];
                slow += (int)s.wcnt[w];
            }
            if (round == 1 && r < a.rows && unit == (f ? before : all + r - before)) mine = r;
        }
    }
    if (mine >= 0) s.n = mine;
    __syncthreads();
    mine = s.n;
    __syncthreads();
    return mine;
}

template <bool BF16, bool PROBS>
__global__ void __launch_bounds__(kThreads, 4) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    Smem &s = *reinterpret_cast<Smem *>(raw);
    const int unit = (int)(blockIdx.x / cluster_nctarank());
    Sampler<BF16, PROBS>(a, s, a.in_order ? unit : row_of(a, s, unit)).run();
}

PerDevice g_sms(0);

// CTAs per row: as many as fit the device at once (4 CTAs of an SM), or more, so that the rows under way
// stay in L2 (256 rows of 131072: 127 us with 4, 199 with 2); 8 at most (the portable size).
int cluster_size(int rows, size_t row_bytes, int sms) {
    const int64_t slots = 4 * (int64_t)sms;
    int c = (int)std::min<int64_t>(kMaxCluster, std::max<int64_t>(1, slots / rows));
    while (c < kMaxCluster && std::min<int64_t>(rows, slots / c) * (int64_t)row_bytes > (80 << 20)) c++;
    return c;
}

template <bool BF16, bool PROBS>
cudaError_t launch(SampleArgs a, cudaStream_t st) {
    static PerDevice smem_set(0);
    int sms = 0;
    cudaError_t e = device_attr(cudaDevAttrMultiProcessorCount, g_sms, &sms);
    if (e != cudaSuccess) return e;
    if ((e = ensure_dynamic_smem(sample_kernel<BF16, PROBS>, sizeof(Smem), smem_set)) != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    const int c = cluster_size(a.rows, (size_t)a.vocab * (BF16 ? 2 : 4), sms);
    a.in_order = a.top_p == nullptr || a.vocab <= kList || (int64_t)a.rows * c <= 4 * (int64_t)sms || a.rows > 16 * kThreads;
    cudaLaunchConfig_t cfg = cluster_config(attr, a.rows, c, kThreads, st);
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
