// Appending rows to the paged 8-bit key/value cache.
//
// One block takes one (page, side, head) that new rows land in: the page's largest new
// magnitude gives the scale, a power of two, so re-scaling what the page already holds
// only moves E4M3 exponents.  Each new value is read once into registers, reduced, then
// rounded and written: 2 bytes read and 1 written per value, nothing else.
//
// What bounds it is HBM for prompts, as long as a value costs few instructions: 6 prompts of up
// to 8191 rows, 8 heads of 128, take 38 us at 247 MB (6.5 TB/s); with infinities sorted out at
// every value and a division in place of the exact inverse they took 96.  A decoded batch (64
// rows) is one chain of dependent loads (offsets, page, values) and takes 5 us.
#include <algorithm>

#include "kv_internal.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;

// Tokens of the chunk (one page of one sequence) that block x works on.
struct Chunk {
    int seq, row, page_slot, first, count;  // first row in k/v; table column; slot in the page; tokens
};

// Rows of sequence b and its first token, cut to the table's room.
__device__ __forceinline__ bool append_range(const KvAppendArgs &a, int b, int &lo, int &n, int &start) {
    int hi;
    bool ok = seq_rows(a.cu_rows, b, a.rows, lo, hi);
    start = a.start[b];
    n = hi - lo;
    if (n == 0) return ok;  // an idle sequence may start anywhere
    if (start < 0) {
        n = 0;
        return false;
    }
    const int64_t room = min((int64_t)a.table_width * a.kv.page, (int64_t)kMaxLen) - start;
    if ((int64_t)n > room) {
        n = room > 0 ? (int)room : 0;
        ok = false;
    }
    return ok;
}

__device__ __forceinline__ int chunks_of(int n, int start, int page) {
    return n == 0 ? 0 : (start + n - 1) / page - start / page + 1;
}

// Chunk x: the sequences' chunk counts are summed by the whole block.
__device__ bool find_chunk(const KvAppendArgs &a, int x, int chunks, Chunk &c) {
    __shared__ int warp_sum[kThreads / 32];
    __shared__ Chunk found;
    __shared__ int have;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.seqs + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, a.seqs), b1 = min(b0 + per, a.seqs);
    if (tid == 0) have = 0;
    int mine = 0;
    bool ok = true;
    for (int b = b0; b < b1; b++) {
        int lo, n, start;
        ok &= append_range(a, b, lo, n, start);
        mine += chunks_of(n, start, a.kv.page);
    }
    if (!ok && blockIdx.x == 0) set_status(a.st, MOE_ERR_BAD_PAGE, 1);
    int pre = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, pre, d);
        if (lane >= d) pre += o;
    }
    if (lane == 31) warp_sum[warp] = pre;
    __syncthreads();
    for (int w = 0; w < warp; w++) pre += warp_sum[w];
    // more chunks than blocks: row ranges that overlap
    if (tid == kThreads - 1 && pre > chunks && blockIdx.x == 0)
        set_status(a.st, MOE_ERR_BAD_PAGE, 2);
    int at = pre - mine;
    if (x >= at && x < pre) {
        for (int b = b0; b < b1; b++) {
            int lo, n, start;
            append_range(a, b, lo, n, start);
            const int m = chunks_of(n, start, a.kv.page);
            if (x < at + m) {
                const int slot = start / a.kv.page + (x - at);
                const int t0 = max(start, slot * a.kv.page), t1 = min(start + n, (slot + 1) * a.kv.page);
                found.seq = b;
                found.row = lo + t0 - start;
                found.page_slot = slot;
                found.first = t0 - slot * a.kv.page;
                found.count = t1 - t0;
                have = 1;
                break;
            }
            at += m;
        }
    }
    __syncthreads();
    c = found;
    return have != 0;
}

// 2^s as a float, s in [-126, 127].
__device__ __forceinline__ float pow2(int s) { return __uint_as_float((uint32_t)(s + 127) << 23); }

// Exponent of the scale for a largest magnitude given as bf16 bits (finite): the
// smallest s >= -126 with amax <= 448 * 2^s, 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exp(uint32_t amax) {
    const int e = (int)(amax >> 7) - 127 - 8 + ((amax & 0x7fu) > 0x60u ? 1 : 0);
    return max(e, -126);
}

// Largest magnitude (bf16 bits) of a lane's values.  FINITE leaves infinities and NaN out, which
// takes three times the instructions and is only needed where there are some.
template <int IT, bool FINITE>
__device__ __forceinline__ uint32_t largest(const uint4 (&x)[IT]) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < IT; i++) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const uint32_t m = w[k] & 0x7fff7fffu;
            amax = __vmaxu2(amax, FINITE ? m & ~__vcmpgeu2(m, 0x7f807f80u) : m);
        }
    }
    return max(amax & 0xffffu, amax >> 16);
}

// IT: 16-byte vectors of values a thread holds (page * D / 8 / kThreads).
template <int IT, int D>
__global__ void __launch_bounds__(kThreads, IT == 16 ? 4 : IT == 8 ? 9 : 12) kv_append_kernel(const KvAppendArgs a) {
    constexpr int kVec = D / 8, kStep = kThreads / kVec;  // vectors of a token; tokens the block covers at once
    // heads, then sides, then chunks: neighbouring blocks read and write neighbouring memory
    const int tid = threadIdx.x, units = 2 * a.kv.heads, per = (units + a.units - 1) / a.units;
    const int x0 = (int)blockIdx.x / per, u0 = ((int)blockIdx.x - x0 * per) * a.units;
    Chunk c;
    if (!find_chunk(a, x0, (int)gridDim.x / per, c)) return;
    const int page = a.page_table[(size_t)c.seq * a.table_width + c.page_slot];
    __shared__ uint32_t warp_max[2][2][kThreads / 32];
    const int tok = tid / kVec, col = tid % kVec;
#pragma unroll 1
    for (int u = u0; u < min(u0 + a.units, units); u++) {
        const int side = u >= a.kv.heads, head = side ? u - a.kv.heads : u;
        // the new values, loaded while the page's number is still on its way
        const size_t ld = side ? a.ldv : a.ldk;
        const uint16_t *src = (side ? a.v : a.k) + (size_t)(c.row + tok) * ld + (size_t)head * D + col * 8;
        uint4 x[IT];
#pragma unroll
        for (int i = 0; i < IT; i++) {
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (tok + i * kStep < c.count) x[i] = ldg_stream16(src + (size_t)(i * kStep) * ld);
        }
        if (page < 0 || page >= a.kv.n_pages) {
            if (tid == 0) set_status(a.st, MOE_ERR_BAD_PAGE, 3);
            return;
        }
        uint8_t *dst = a.kv.codes(page, a.layer, side, head);
        float *scale = a.kv.scale(page, a.layer, side, head);
        const float old = c.first > 0 ? *scale : 0.f;

        uint32_t amax = __reduce_max_sync(0xffffffffu, largest<IT, false>(x));
        if ((tid & 31) == 0) warp_max[u & 1][0][tid >> 5] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; w++) amax = max(amax, warp_max[u & 1][0][w]);
        if (amax >= 0x7f80u) {
            amax = __reduce_max_sync(0xffffffffu, largest<IT, true>(x));
            if ((tid & 31) == 0) warp_max[u & 1][1][tid >> 5] = amax;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kThreads / 32; w++) amax = max(amax, warp_max[u & 1][1][w]);
        }

        const float fresh = pow2(scale_exp(amax));
        const float now = c.first > 0 ? fmaxf(old, fresh) : fresh;
        // the kept tokens follow the new scale
        if (c.first > 0 && now != old) {
            const float f = __fdiv_rn(old, now);
#pragma unroll 1
            for (int j = tid; j < c.first * D / 16; j += kThreads) {
                uint4 q = reinterpret_cast<uint4 *>(dst)[j];
                uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    float v[4];
                    e4m3x4_to_float(w[k], v);
                    w[k] = e4m3x4_rn(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
                }
                reinterpret_cast<uint4 *>(dst)[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        // A power of two has an exact inverse; a scale that a caller set may be none, and is divided by.
        const uint32_t bits = __float_as_uint(now);
        const bool two = (bits & 0x7fffffu) == 0u && (bits >> 23) >= 1u && (bits >> 23) <= 253u;
        const float inv = __uint_as_float(0x7f000000u - bits);
        uint8_t *to = dst + (size_t)(c.first + tok) * D + col * 8;
        auto store = [&](auto scaled) {
#pragma unroll
            for (int i = 0; i < IT; i++) {
                if (tok + i * kStep >= c.count) break;
                const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                uint32_t q[2];
#pragma unroll
                for (int k = 0; k < 2; k++)
                    q[k] = e4m3x4_rn(scaled(__uint_as_float(w[2 * k] << 16)), scaled(__uint_as_float(w[2 * k] & 0xffff0000u)),
                                     scaled(__uint_as_float(w[2 * k + 1] << 16)),
                                     scaled(__uint_as_float(w[2 * k + 1] & 0xffff0000u)));
                *reinterpret_cast<uint2 *>(to + i * (kStep * D)) = make_uint2(q[0], q[1]);
            }
        };
        if (two)
            store([&](float v) { return v * inv; });
        else
            store([&](float v) { return __fdiv_rn(v, now); });
        if (tid == 0) *scale = now;
    }
}

}  // namespace

cudaError_t launch_kv_append(KvAppendArgs a, cudaStream_t st) {
    // chunks: at most one per row, and at most rows / page + 2 per sequence with rows
    const int64_t bound = (int64_t)a.rows / a.kv.page + 2 * (int64_t)std::min(a.seqs, a.rows);
    // A block takes several (side, head) pairs one after the other where its page is small and
    // there are blocks enough all the same (27 per SM): finding the chunk is most of a small
    // block's time.  24.5 M values in pages of 16: 62 us, with a block each 83; pages of 32: 54
    // and 60.  With few blocks one pair each is right: their time is one chain of loads.
    a.units = 1;
    const int64_t chunks = std::min<int64_t>(a.rows, bound);
    while (a.kv.page * a.kv.dim * a.units < 8192 && chunks * 2 * a.kv.heads > 4096 * (int64_t)a.units) a.units *= 2;
    const int64_t blocks = chunks * ((2 * a.kv.heads + a.units - 1) / a.units);
    if (blocks > 0x7fffffff) return cudaErrorNotSupported;
    const dim3 grid((unsigned)blocks);
    TraceScope trace_scope("kv_append", st);
    auto launch = [&](auto wide, auto narrow) {
        a.kv.dim == 128 ? wide<<<grid, kThreads, 0, st>>>(a) : narrow<<<grid, kThreads, 0, st>>>(a);
    };
    switch (a.kv.page) {
        case 16: launch(kv_append_kernel<2, 128>, kv_append_kernel<1, 64>); break;
        case 32: launch(kv_append_kernel<4, 128>, kv_append_kernel<2, 64>); break;
        case 64: launch(kv_append_kernel<8, 128>, kv_append_kernel<4, 64>); break;
        case 128: launch(kv_append_kernel<16, 128>, kv_append_kernel<8, 64>); break;
        default: return cudaErrorNotSupported;
    }
    return cudaGetLastError();
}

}  // namespace moe
