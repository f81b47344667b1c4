// Rows of a vocabulary's probabilities or logits, as draft verification and sampling read them: in
// vectors of 16 bytes, from any address; and the whole numbers that both are defined in.
#pragma once

#include "kv_internal.cuh"
#include "sm100_tensor.cuh"

namespace moe {
namespace {

constexpr int kGrid = 38;       // probabilities are whole multiples of 2^-38
constexpr int kUniform = 24;    // uniforms are whole multiples of 2^-24

// floor(2^38 min(max(p, 0), 1)) + kRaw, NaN: as 0.  The whole part of 2^15 p and that of 2^23
// times the rest appear in the mantissas of sums with 2^23 that are rounded towards zero: six
// instructions at full rate, where a conversion to 64-bit integers alone takes twice their time.
constexpr uint64_t kRaw = (0x4b000000ull << 23) + 0x4b000000ull;
__device__ __forceinline__ uint64_t whole_raw(float p) {
    const float x = __saturatef(p);
    const float hi = __fmaf_rz(x, 32768.f, 8388608.f);
    const float rest = fmaf(x, 32768.f, 8388608.f - hi);  // exact
    const float lo = __fmaf_rz(rest, 8388608.f, 8388608.f);
    return ((uint64_t)__float_as_uint(hi) << 23) + __float_as_uint(lo);
}
__device__ __forceinline__ uint64_t whole(float p) { return whole_raw(p) - kRaw; }

__device__ __forceinline__ uint64_t whole_uniform(float u) {
    return (uint64_t)__float2uint_rz(fminf(fmaxf(u, 0.f), 0.99999994f) * 16777216.f);
}

// Larger of two pairs of bf16 values, each by itself; NaN only if both are.
__device__ __forceinline__ uint32_t max2_bf16(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A row of n values, cut into vectors of 16 bytes on 16-byte boundaries: vector 0 is the
// (possibly partial) one that holds the row's first value.  WRITTEN: the kernel writes to the row, too, so
// that its loads may not go the way that is for constant memory.
template <bool BF16, bool WRITTEN = false>
struct Row {
    static constexpr int kVec = BF16 ? 8 : 4;
    static constexpr int kSize = BF16 ? 2 : 4;
    const uint8_t *p;  // the first value
    int n, lead;       // values; places of vector 0 before the first value

    __device__ __forceinline__ Row(const void *base, size_t at, int n_) : n(n_) {
        p = static_cast<const uint8_t *>(base) + at * kSize;
        lead = (int)(((uintptr_t)p & 15u) / kSize);
    }
    __device__ __forceinline__ int vectors() const { return (n + lead + kVec - 1) / kVec; }
    __device__ __forceinline__ int first(int v) const { return v * kVec - lead; }  // index of its first place
    __device__ __forceinline__ bool whole_vector(int v) const { return first(v) >= 0 && first(v) + kVec <= n; }
    __device__ __forceinline__ float at(int i) const {
        return BF16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t *>(p)[i]) : reinterpret_cast<const float *>(p)[i];
    }
    __device__ __forceinline__ uint4 load16(int i) const {  // from value i on
        const uint4 *q = reinterpret_cast<const uint4 *>(p + (ptrdiff_t)i * kSize);
        return WRITTEN ? __ldcg(q) : __ldg(q);
    }
    // largest value of vector v (NaN if it has none)
    __device__ __forceinline__ float largest(int v) const {
        if constexpr (BF16) {
            const int i0 = first(v);
            if (i0 >= 0 && i0 + kVec <= n) {
                const uint4 u = load16(i0);
                const uint32_t m = max2_bf16(max2_bf16(u.x, u.y), max2_bf16(u.z, u.w));
                return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
            }
        }
        float x[kVec], m;
        load(v, __uint_as_float(0x7fc00000u), x);
        m = x[0];
#pragma unroll
        for (int k = 1; k < kVec; k++) m = fmaxf(m, x[k]);
        return m;
    }
    // the values of vector v (`none` outside the row)
    __device__ __forceinline__ void load(int v, float none, float (&x)[kVec]) const {
        const int i0 = first(v);
        if (i0 >= 0 && i0 + kVec <= n) {
            const uint4 u = load16(i0);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; k++) {
                if constexpr (BF16) {
                    x[2 * k] = __uint_as_float(w[k] << 16);
                    x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
                } else {
                    x[k] = __uint_as_float(w[k]);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < kVec; k++) x[k] = i0 + k >= 0 && i0 + k < n ? at(i0 + k) : none;
        }
    }
};

__device__ __forceinline__ void store_cluster_u64(uint64_t *mine, uint32_t rank, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(mine, rank)), "l"(v) : "memory");
}

// A value's place in the order (0: nothing), then the lower index.
__device__ __forceinline__ uint64_t order_key(float x, int i) {
    if (i < 0) return 0;
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 equals +0
    const uint32_t o = (u & 0x80000000u) ? ~u : u | 0x80000000u;
    return (uint64_t)o << 32 | (0xffffffffu - (uint32_t)i);
}

// A launch of `units` clusters of `c` CTAs.
inline cudaLaunchConfig_t cluster_config(cudaLaunchAttribute *attr, int units, int c, int threads, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(units * c));
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

}  // namespace
}  // namespace moe
