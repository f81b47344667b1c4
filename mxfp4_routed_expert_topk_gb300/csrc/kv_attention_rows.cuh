// Cache attention, the form for row tiles of more than 16 rows (a verification batch's rows
// times the query heads of a key/value head, or a prompt's).
//
// Rows lie along M: S = Q K^T (M = 128 rows, N = 128 tokens, both operands K-major) and
// O = P V (M = 128 rows, N = head_dim, K = 128 tokens; P is the A operand in TMEM, V is read
// N-major).  The TMEM lane of a score is its row, so a row's maximum and sum need no exchange
// between lanes and its reference is one register; the pages' key scales and the logarithm of
// their value scales are constants of a run of 16 tokens and go into the exponent's multiply-
// add, so that the exponential is the weight with its value scale; a run's sum times 2^-(that
// logarithm) is what it adds to the row's sum.  Where that logarithm is so far below the row's
// others that the exponential would leave fp32's range while the sum needs it, both take a larger
// one (the weight, below E4M3's range, becomes 0 all the same).  Weights replace the scores they
// came from in TMEM.
//
// What bounds it is instruction issue and latency: 128 x 128 scores a tile at about 8
// instructions each are about 1000 clocks of all four schedulers, next to 1400 that the tile's
// 32 KB take from HBM and 1024 of the tensor pipe; a tile takes 2500.  So the work is split by
// role: softmax warpgroups take tiles in turn (a thread per row) over two or three score buffers,
// so that the next scores are ready when a warpgroup comes for them, one more warpgroup joins
// each tile's output with the running one as soon as it is there, and a warp of its own prepares
// the tiles' constants.  Registers go to the warpgroups by need (setmaxnreg).  17 rows in each of
// 4 sequences of up to 131072 tokens (7 query heads of 8 x 128) take 318 us: 0.49 of the HBM and
// 0.42 of the bf16 rate (313 with one reference for a tile's value scales, which was wrong); with
// the constants in the softmax warps 331, and without the joining warpgroup and the third score
// buffer 438, both before that.
//
// Row tiles of up to 64 (32) rows stand two (four) times in the 128 places, and each copy takes a
// half (quarter) of every tile's tokens: its weights for the others are zero, and the copies'
// outputs are added up at the end of the unit.  That halves (quarters) the softmax warps' work;
// the joining warpgroup is then the slowest (1700 clocks a tile), so the softmax warps load the
// queries.  24 sequences of 8192, when they came: 3 rows 136 -> 116 us (now 112), 9 rows 148 -> 136;
// heads of 64, 4 rows 76 -> 55 (now 54), 8 rows 79 -> 65.  The choice is made where the kernel is launched.
//
// Not better: weights as one fp16 part with V's tile converted to fp16 in shared memory (4 x 17:
// 346 us with two softmax warpgroups, 352 with three, where two parts took 338).
#pragma once

#include <algorithm>

#include "kv_attention.cuh"

namespace moe {
namespace {

constexpr int kGroups = 2;                     // softmax warpgroups
constexpr int kRing = 8;                       // tiles whose references and sums are kept
constexpr int kJoinWarp = kFirstSoft + 4 * kGroups;
constexpr int kSoft = 128 * kGroups + 128;     // with the joining warpgroup
constexpr int kThreads = 32 * kFirstSoft + kSoft;
constexpr int kRows = 128;
// Registers of a thread: at launch, then by role; the sum over the warpgroups is no more than
// what the launch allocated (512 x 128).
constexpr int kRegsIssue = 80, kRegsSoft = 120, kRegsJoin = 192;
static_assert(kRegsIssue + kGroups * kRegsSoft + kRegsJoin <= 4 * 128 && kThreads == 512, "register split");
constexpr int kBarAll = 7, kBarJoin = 1;

constexpr int kMaxStages = 8;  // per ring
constexpr int kSegs = 4;       // ring of segments

// Shared memory, in bytes.
struct CommonSmem {
    uint32_t k, v, q, scales, seg, split, rows, bars, misc, total;
    __host__ __device__ CommonSmem(int dim, int rows_, int nk, int nv) {
        uint32_t o = 0;
        k = o;      o += (uint32_t)nk * kTokens * dim;
        v = o;      o += (uint32_t)nv * kTokens * dim;
        q = o;      o += 4u * (uint32_t)rows_ * dim;                     // [2 buffers][2 parts][rows][dim]
        scales = o; o += (uint32_t)kMaxStages * 2u * kMaxSlots * 4u;     // per value stage: keys', values'
        seg = o;    o += (uint32_t)kSegs * (uint32_t)sizeof(SharedSeg);
        split = o;  o += 2u * (uint32_t)sizeof(SharedSeg);                 // units shared with other CTAs
        rows = o;   o += 2u * (uint32_t)rows_ * (uint32_t)sizeof(RowInfo);
        bars = o;   o += (4u * kMaxStages + 29u + kMaxStages) * 8u;
        o = (o + 15u) & ~15u;
        misc = o;   o += 512u;
        total = o;
    }
};

// Barriers, by index.
struct Bars {
    uint64_t *b;
    __device__ uint64_t *k_full(int s) const { return b + s; }
    __device__ uint64_t *k_empty(int s) const { return b + kMaxStages + s; }
    __device__ uint64_t *v_full(int s) const { return b + 2 * kMaxStages + s; }
    __device__ uint64_t *v_empty(int s) const { return b + 3 * kMaxStages + s; }
    __device__ uint64_t *q_full(int s) const { return b + 4 * kMaxStages + s; }
    __device__ uint64_t *q_empty(int s) const { return b + 4 * kMaxStages + 2 + s; }
    __device__ uint64_t *s_full(int s) const { return b + 4 * kMaxStages + 4 + s; }   // scores in TMEM
    __device__ uint64_t *p_ready(int s) const { return b + 4 * kMaxStages + 8 + s; }  // weights written, scores read
    __device__ uint64_t *o_full(int s) const { return b + 4 * kMaxStages + 12 + s; }  // outputs in TMEM
    __device__ uint64_t *o_empty(int s) const { return b + 4 * kMaxStages + 16 + s; }
    __device__ uint64_t *mma_done() const { return b + 4 * kMaxStages + 20; }
    __device__ uint64_t *seg_full(int s) const { return b + 4 * kMaxStages + 21 + s; }
    __device__ uint64_t *seg_empty(int s) const { return b + 4 * kMaxStages + 25 + s; }
    __device__ uint64_t *c_full(int s) const { return b + 4 * kMaxStages + 29 + s; }  // a value stage's constants
};

// One side's copies (SIDE 0: keys, 1: values and scales); P: page size (a constant, as the
// warp's time per tile counts).
template <int D, int SIDE, int P, bool SHARED>
__device__ __forceinline__ void copy_pages(const AttnArgs &a, const CUtensorMap *tm, unsigned char *smem,
                                           const CommonSmem &L, const Bars &B, int *abort_flag) {
    constexpr uint32_t kTile = kTokens * D;
    const int n = SIDE ? a.nv : a.nk;
    unsigned char *ring = smem + (SIDE ? L.v : L.k);
    const uint32_t elected = elect_one();
    Ring R;
    Pages<P, SHARED> pg;
    int issued = 0;
    bool run = true;
#pragma unroll 1
    for (int seg = 0; run; seg++) {
        const int ss = seg % kSegs;
        if (!warp_wait(B.seg_full(ss), (uint32_t)(seg / kSegs) & 1u, 0xa60u + SIDE, abort_flag)) break;
        const SegOf<SHARED> *sg = reinterpret_cast<const SegOf<SHARED> *>(smem + L.seg) + ss;
        const int count = sg->count, head = sg->head;
        if (count == 0) break;
        const int y = (SIDE * a.k.kv.heads + head) * P;
        pg.start(a, *sg);
        __syncwarp();
        if (elected) mbar_arrive(B.seg_empty(ss));
#pragma unroll 1
        for (int t = 0; t < count; t++) {
            uint64_t *full = SIDE ? B.v_full(R.s) : B.k_full(R.s);
            if (!(run = warp_wait(SIDE ? B.v_empty(R.s) : B.k_empty(R.s), R.ph ^ 1u, 0xa00u + 16 * SIDE + R.s, abort_flag)))
                break;
            pg.template copy<D>(tm, ring + (uint32_t)R.s * kTile, y, full, elected);
            if constexpr (SIDE == 1)
                pg.copy_scales(a, head, reinterpret_cast<float *>(smem + L.scales) + R.s * 2 * kMaxSlots, full);
            pg.next_tile();
            issued++;
            R.next(n);
        }
    }
    // nothing may be in flight when the CTA exits
    if ((threadIdx.x & 31) == 0) {
        for (int i = max(0, issued - n); i < issued; i++)
            drain(SIDE ? B.v_full(i % n) : B.k_full(i % n), (uint32_t)(i / n) & 1u, abort_flag);
    }
    __syncwarp();
}

template <int D, int SIDE, bool SHARED>
__device__ __forceinline__ void copy_role(const AttnArgs &a, const CUtensorMap *tm, unsigned char *smem,
                                          const CommonSmem &L, const Bars &B, int *abort_flag) {
    switch (a.k.kv.page) {
        case 16: return copy_pages<D, SIDE, 16, SHARED>(a, tm, smem, L, B, abort_flag);
        case 32: return copy_pages<D, SIDE, 32, SHARED>(a, tm, smem, L, B, abort_flag);
        case 64: return copy_pages<D, SIDE, 64, SHARED>(a, tm, smem, L, B, abort_flag);
        case 128: return copy_pages<D, SIDE, 128, SHARED>(a, tm, smem, L, B, abort_flag);
    }
}

struct RowsSmem {
    CommonSmem c;
    uint32_t ml, chunk, nan, merge = 0, mlc = 0, total;
    __host__ __device__ RowsSmem(int dim, int nk, int nv, int copies) : c(dim, kRows, nk, nv) {
        uint32_t o = (c.total + 127u) & ~127u;
        ml = o;    o += (uint32_t)kRing * kRows * 8u;  // [tile][row] (reference, sum)
        nan = o;   o += (uint32_t)kRing * 4u * 4u;  // [tile][warp] tokens whose values hold partial NaN
        if (copies > 1) {
            merge = o; o += 3u * 32u * 36u * 4u; // [warp of the copies but the first][lane][32 + 4] values of the head
            mlc = o;   o += kRows * 8u;          // [place] (reference, sum)
        }
        o = (o + 15u) & ~15u;
        // [value stage][page] (key scale, log2 of the value scale as references take it and as it is, its inverse)
        chunk = o; o += (uint32_t)nv * kMaxSlots * 16u;
        total = o;
    }
};

// The larger of two values; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A pair of weights as E4M3 parts: the value to 4 significant bits, and what is left.
__device__ __forceinline__ void split2(uint64_t x, float &h0, float &h1, float &l0, float &l1) {
    float x0, x1;
    unpack2(x, x0, x1);
    h0 = part_hi(x0);
    h1 = part_hi(x1);
    unpack2(fma2(pack2(h0, h1), pack2(-1.f, -1.f), x), l0, l1);
}

template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Publishes the worker's segments, then one with count 0, and the constants of each tile's
// pages (lane j has page j), which are then no part of the softmax warps' time (400 clocks of
// 5400 a tile).  A tile's constants stand beside its value stage: nothing more says that their
// place is free.
template <bool SHARED>
__device__ __forceinline__ void segment_role(const AttnArgs &a, unsigned char *smem, const RowsSmem &F, const Bars &B,
                                             const Start<SHARED> &start, int *abort_flag) {
    const int lane = threadIdx.x & 31, slots = kTokens / a.k.kv.page;
    SegOf<SHARED> *ring = reinterpret_cast<SegOf<SHARED> *>(smem + F.c.seg);
    const float *scales = reinterpret_cast<const float *>(smem + F.c.scales);
    float4 *chunk = reinterpret_cast<float4 *>(smem + F.chunk);
    Walk<SHARED> W(a, start);
    Watch eye = lane == 0 ? Watch{B.seg_empty(0), kSegs, 0, 1u} : Watch{B.v_full(0), a.nv, 0, 0u};
    int published = 0, known = 0, u = 0;  // segments, their tiles; tiles whose constants are there
    bool ended = false;
    uint64_t idle = 0;
#pragma unroll 1
    while (!ended || u < known) {
        const uint32_t m = __ballot_sync(0xffffffffu, lane < 2 && eye.ready());
        const bool publish = !ended && (m & 1u) != 0u, constants = u < known && (m & 2u) != 0u;
        if (constants && !publish) {
            const int vb = u % a.nv;
            const float *sc = scales + vb * 2 * kMaxSlots;
            __syncwarp();  // (lane 1 has seen the copies land)
            // (a loop of one turn: as straight code the compiler copies this into the polling loop, and
            // all roles feel it: 4 x 17 rows 354 us, so 323)
#pragma unroll 1
            for (int j = lane; j < slots; j += 32) {
                const float vs = sc[kMaxSlots + j], v = fabsf(vs) < INFINITY ? lg2(vs) : kNan;
                chunk[vb * kMaxSlots + j] = make_float4(sc[j] * a.scale2, fmaxf(v, kLowScale), v, ex2(-v));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(B.c_full(vb));
            u++;
            if (lane == 1) eye.next();
        } else if (publish) {
            const SegOf<SHARED> g = W.next();
            if (lane == 0) {
                ring[published % kSegs] = g;
                mbar_arrive(B.seg_full(published % kSegs));
                eye.next();
            }
            __syncwarp();
            published++;
            known += g.count;
            ended = g.count == 0;
            if (!ended) prefetch_queries(a, g);
        } else {
            if (__any_sync(0xffffffffu, expired(idle, 0xe10u, abort_flag))) return;
            continue;
        }
        idle = 0;
    }
}

// Warp w's part (of nw) of segment s's queries, once the segment is there and its buffers are
// free (`must`: waits for that).  False if they are not.
template <int D, int COPIES, bool SHARED>
__device__ __forceinline__ bool segment_queries(const AttnArgs &a, unsigned char *smem, const CommonSmem &L, const Bars &B,
                                                int s, int w, int nw, bool must, int *abort_flag) {
    uint64_t *full = B.seg_full(s % kSegs), *empty = B.q_empty(s & 1);
    const uint32_t pf = (uint32_t)(s / kSegs) & 1u, pe = ((uint32_t)(s >> 1) & 1u) ^ 1u;
    if (must) {
        if (!warp_wait(full, pf, 0xe20u, abort_flag) || !warp_wait(empty, pe, 0xe00u, abort_flag)) return false;
    } else if (!__all_sync(0xffffffffu, mbar_test(full, pf) && mbar_test(empty, pe))) {
        return false;
    }
    const SegOf<SHARED> &g = reinterpret_cast<const SegOf<SHARED> *>(smem + L.seg)[s % kSegs];
    if (g.count > 0)
        load_queries<D, kRows, SHARED, COPIES>(a, reinterpret_cast<RowInfo *>(smem + L.rows) + (s & 1) * kRows,
                                          smem + L.q + (uint32_t)(s & 1) * (2u * kRows * D), g, w, nw);
    if ((threadIdx.x & 31) == 0) mbar_arrive(B.q_full(s & 1));
    return true;
}

template <int D, int COPIES, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_rows_kernel(const __grid_constant__ CUtensorMap tm,
                                                                         const AttnArgs a) {
    constexpr uint32_t kTile = kTokens * D;
    constexpr uint32_t kSwz = D == 128 ? kSwizzle128B : kSwizzle64B;
    constexpr uint32_t kGroup8 = 8 * D;
    // score and output buffers: what TMEM's 512 columns hold
    constexpr int kSBufs = D == 128 && COPIES > 1 ? 2 : 3, kOBufs = D == 128 && COPIES == 1 ? 1 : 2;
    static_assert(kSBufs * kTokens + kOBufs * D <= 512 && kSBufs + kOBufs <= kRing, "buffers");
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = (unsigned char *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const RowsSmem F(D, a.nk, a.nv, COPIES);
    const CommonSmem &L = F.c;
    const Bars B{reinterpret_cast<uint64_t *>(smem + L.bars)};
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + L.misc);
    uint32_t *tmem_slot = misc;
    int *abort_flag = reinterpret_cast<int *>(misc + 1);
    int *n_shared = reinterpret_cast<int *>(misc + 2), *go = reinterpret_cast<int *>(misc + 3);
    int64_t *sums = reinterpret_cast<int64_t *>(misc + 8);
    Start<SHARED> *start = reinterpret_cast<Start<SHARED> *>(misc + 64);
    static_assert(kThreads / 32 * 12 <= 56 * 4 && sizeof(Start<SHARED>) <= 64 * 4, "misc");
    StatusWord *st = a.k.st;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const Line line = cut_line<kThreads, 1, SHARED>(a, sums, start);
    if ((int)blockIdx.x >= line.workers) return;  // the whole CTA: nothing set up yet
    if (tid == 0) {
        for (int s = 0; s < a.nk; s++) {
            mbar_init(B.k_full(s), 1);
            mbar_init(B.k_empty(s), 1);
        }
        for (int s = 0; s < a.nv; s++) {
            mbar_init(B.v_full(s), 1 + kTokens / a.k.kv.page);
            mbar_init(B.v_empty(s), 1);
            mbar_init(B.c_full(s), 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(B.q_full(b), COPIES == 1 ? 4 : 4 * kGroups);  // the warps that load queries
            mbar_init(B.q_empty(b), kSoft / 32);
        }
        for (int b = 0; b < kSBufs; b++) {
            mbar_init(B.s_full(b), 1);
            mbar_init(B.p_ready(b), 4);
        }
        for (int b = 0; b < kOBufs; b++) {
            mbar_init(B.o_full(b), 1);
            mbar_init(B.o_empty(b), 4);
        }
        for (int b = 0; b < kSegs; b++) {
            mbar_init(B.seg_full(b), 1);
            mbar_init(B.seg_empty(b), 2 + kSoft / 32);  // the copying warps, and the softmax
        }
        mbar_init(B.mma_done(), 1);
        *abort_flag = 0;
        *n_shared = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;        // scores, then weights: buffers of 128 columns
    const uint32_t tmem_o = tmem + kSBufs * kTokens;

    if (warp < kFirstSoft) {
        regs_dec<kRegsIssue>();
        if (warp == 0) {
            copy_role<D, 0, SHARED>(a, &tm, smem, L, B, abort_flag);
        } else if (warp == 2) {
            copy_role<D, 1, SHARED>(a, &tm, smem, L, B, abort_flag);
        } else if (warp == 1) {
            // ------------------------------------------------------ MMA issue
            const uint32_t id_s = idesc_f8(kRows, kTokens, false, false), id_o = idesc_f8(kRows, D, false, true);
            const uint64_t kd = smem_desc(smem_u32(smem + L.k), 16, kGroup8, kSwz);
            const uint64_t vd = smem_desc(smem_u32(smem + L.v), kGroup8, kGroup8, kSwz);
            const uint64_t qd = smem_desc(smem_u32(smem + L.q), 16, kGroup8, kSwz);
            int ks = 0, vs = 0;  // stages
            int ns = 0, np = 0, seg = 0, seg_end = 0, qb = 0;  // scores / outputs issued
            int bs = 0, bp = 0, bo = 0;                        // and their buffers
            bool last = false;                                 // seg_end is the share's end
            const uint32_t elected = elect_one();
            // Whichever is ready: the outputs of tile np, the scores of tile ns (over the weights of
            // tile ns - kSBufs, whose outputs have been issued; with the segment's queries).  Lanes 0 to 4
            // look at one barrier each; a vote makes the outcome uniform, which keeps the descriptors
            // in uniform registers.
            Watch eye = lane == 0   ? Watch{B.p_ready(0), kSBufs, 0, 0u}
                        : lane == 1 ? Watch{B.v_full(0), a.nv, 0, 0u}
                        : lane == 2 ? Watch{B.o_empty(0), kOBufs, 0, 1u}
                        : lane == 3 ? Watch{B.k_full(0), a.nk, 0, 0u}
                                    : Watch{B.q_full(0), 2, 0, 0u};
            uint64_t idle = 0;  // since when nothing has been ready
            while (!(last && np == seg_end)) {
                const uint32_t m = __ballot_sync(0xffffffffu, lane < 5 && eye.ready());
                const bool out = np < ns && (m & 7u) == 7u;
                if (ns == seg_end && !last && (m & 16u) != 0u) {  // the next segment's queries are there
                    __syncwarp();  // what one lane has seen holds for all (a vote orders no memory)
                    const volatile SegOf<SHARED> *sg =
                        reinterpret_cast<const volatile SegOf<SHARED> *>(smem + L.seg) + seg % kSegs;
                    const int count = __shfl_sync(0xffffffffu, sg->count, 0);
                    qb = seg & 1;
                    seg_end += count;
                    last = __any_sync(0xffffffffu, count == 0);
                    seg++;
                    if (lane == 4) eye.next();
                }
                const bool scores = ns < seg_end && ns < np + (out ? 1 : 0) + kSBufs && (m & 8u) != 0u;
                if (!out && !scores) {
                    if (__any_sync(0xffffffffu, expired(idle, 0xb00u, abort_flag))) break;
                    continue;
                }
                idle = 0;
                __syncwarp();
                tc_fence_after();
                if (out) {
                    const uint64_t va = vd + (uint64_t)((uint32_t)vs * kTile >> 4);
                    const uint32_t p = tmem + (uint32_t)(bp * kTokens);
                    // 32 tokens take 8 columns per part: the parts of each 32 lie side by side
    #pragma unroll
                    for (int part = 0; part < 2; part++)
    #pragma unroll
                        for (int k = 0; k < kTokens / 32; k++)
                            tc_mma_f8_ts(tmem_o + (uint32_t)(bo * D), p + (uint32_t)(16 * k + 8 * part),
                                         va + (uint64_t)(k * (32 * D) >> 4), id_o, (part > 0 || k > 0) ? 1u : 0u, elected);
                    tc_commit_elected(B.v_empty(vs), elected);
                    tc_commit_elected(B.o_full(bo), elected);
                    if (++vs == a.nv) vs = 0;
                    if (++bp == kSBufs) bp = 0;
                    if (++bo == kOBufs) bo = 0;
                    np++;
                    if (lane < 3) eye.next();
                }
                if (scores) {
                    const uint64_t ka = kd + (uint64_t)((uint32_t)ks * kTile >> 4);
                    const uint64_t qa = qd + (uint64_t)((uint32_t)qb * (2u * kRows * D) >> 4);
    #pragma unroll
                    for (int part = 0; part < 2; part++)
    #pragma unroll
                        for (int k = 0; k < D / 32; k++)
                            tc_mma_f8(tmem + (uint32_t)(bs * kTokens),
                                      qa + (uint64_t)(part * (kRows * D) >> 4) + (uint64_t)(2 * k), ka + (uint64_t)(2 * k),
                                      id_s, (part > 0 || k > 0) ? 1u : 0u, elected);
                    tc_commit_elected(B.k_empty(ks), elected);
                    tc_commit_elected(B.s_full(bs), elected);
                    if (++ks == a.nk) ks = 0;
                    if (++bs == kSBufs) bs = 0;
                    ns++;
                    if (lane == 3) eye.next();
                }
            }
            if (elect_one()) tc_commit(B.mma_done());
            __syncwarp();
            if (lane == 0) drain(B.mma_done(), 0u, abort_flag);
            __syncwarp();
        } else {
            segment_role<SHARED>(a, smem, F, B, *start, abort_flag);
        }
    } else if (warp < kJoinWarp) {
        regs_dec<kRegsSoft>();
        // -------------------------------------------------------- softmax
        const int sw = warp - kFirstSoft, wg = sw >> 2, ew = sw & 3;
        const int row = 32 * ew + lane;  // row of the tile (TMEM lane); also the token it cleans
        const uint32_t lanes = (uint32_t)(32 * ew) << 16;
        float2 *ml = reinterpret_cast<float2 *>(smem + F.ml);
        uint32_t *nan = reinterpret_cast<uint32_t *>(smem + F.nan);
        const int page_shift = 31 - __clz(a.k.kv.page);
        // the tokens of a tile that this warp's copy of the rows takes
        constexpr int kTake = kTokens / COPIES, kWide = kTake < 64 ? kTake : 64;
        const int h0 = ew * COPIES / 4 * kTake;
        int done = 0;  // tiles of earlier segments

#pragma unroll 1
        for (int seg = COPIES == 1 ? 0 : -1;; seg++) {  // (-1: only the first segment's queries)
            const int buf = seg & 1;
            // (no barrier stands between these warps: after an abort each leaves by itself)
            if (seg >= 0 && !warp_wait(B.q_full(buf), (uint32_t)(seg >> 1) & 1u, 0xc31u, abort_flag)) break;
            const SegOf<SHARED> *sg = reinterpret_cast<const SegOf<SHARED> *>(smem + L.seg) + (seg & (kSegs - 1));
            const RowInfo ri = reinterpret_cast<const RowInfo *>(smem + L.rows)[buf * kRows + row];
            const int count = seg < 0 ? 0 : sg->count, tile0 = sg->tile0, see_all = sg->see_all, see_max = sg->see_max;
            if (seg >= 0 && count == 0) break;
            bool asked = COPIES == 1;  // the next segment's queries are loaded

            // scores of tile t of the segment -> weights; its reference and sum
#pragma unroll 1
            for (int t = (wg + kGroups - done % kGroups) % kGroups;; t += kGroups) {
                // (with several copies these warps have the time, the joining ones do not)
                if (!asked)
                    asked = segment_queries<D, COPIES, SHARED>(a, smem, L, B, seg + 1, sw, 4 * kGroups, t >= count, abort_flag);
                if (t >= count) break;
                const int u = done + t, sb = u % kSBufs, vb = u % a.nv;
                const float4 *chunk = reinterpret_cast<const float4 *>(smem + F.chunk) + vb * kMaxSlots;
                soft_wait(B.c_full(vb), (uint32_t)(u / a.nv) & 1u, 0xc11u, abort_flag);
                const bool special = (tile0 + t + 1) * kTokens > see_all;
                const int lim = min(max(ri.pos + 1 - (tile0 + t) * kTokens, 0), kTokens);  // tokens the row sees
                uint32_t word = 0;
                if (special) {
                    const int tk = (tile0 + t) * kTokens + row;
                    soft_wait(B.v_full(vb), (uint32_t)(u / a.nv) & 1u, 0xc10u + vb, abort_flag);
                    const bool bad = clean_values<D>(smem + L.v + (uint32_t)vb * kTile, row, tk, see_all, see_max);
                    word = __ballot_sync(0xffffffffu, bad);
                    fence_proxy_async_smem();
                }
                soft_wait(B.s_full(sb), (uint32_t)(u / kSBufs) & 1u, 0xc00u + sb, abort_flag);
                // (from here on: these scores are there, so the outputs of tile u - kSBufs have been
                // issued, so those of tile u - kSBufs - kOBufs have been joined: kRing places do)
                if (lane == 0) nan[(u % kRing) * 4 + ew] = word;
                tc_fence_after();
                const uint32_t ts = tmem + (uint32_t)(sb * kTokens) + lanes;
                // loops over 32 tokens are not unrolled: the body must stay in the instruction cache
                float mx = -INFINITY, mv = -INFINITY;  // largest score; and with its value scale
#pragma unroll 1
                for (int h = h0; h < h0 + kTake; h += kWide) {
                    float x[kWide];
                    tmem_ld32(ts + h, x);
                    if constexpr (kWide == 64) tmem_ld32(ts + h + 32, x + 32);
                    tmem_ld_wait(x);
                    if (special) {
#pragma unroll
                        for (int i = 0; i < kWide; i++) x[i] = h + i < lim ? x[i] : -INFINITY;
                    }
#pragma unroll
                    for (int q = 0; q < kWide / 16; q++) {
                        float m4[4];
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            m4[i] = fmaxf(fmaxf(x[16 * q + i], x[16 * q + 4 + i]),
                                          fmaxf(x[16 * q + 8 + i], x[16 * q + 12 + i]));
                        const float2 c = *reinterpret_cast<const float2 *>(chunk + ((h + 16 * q) >> page_shift));
                        const float s = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c.x;
                        mx = fmaxf(mx, s);
                        mv = fmaxf(mv, fmaf(s, ri.qs, c.y));
                    }
                }
                const float mt = mv - kTop, base = mt == -INFINITY ? 0.f : mt;
                // a value scale's logarithm counts as `low` at least: weights on it are below 2^(kTop - 30)
                const float low = mt == -INFINITY ? 0.f : fmaf(-mx, ri.qs, mv) - 30.f, inv_low = ex2(-low);
                float l = 0.f;
#pragma unroll 1
                for (int h = h0; h < h0 + kTake; h += 32) {
                    float x[32];
                    tmem_ld32(ts + h, x);
                    uint64_t A2[2], C2[2];
                    float r[2];
#pragma unroll
                    for (int q = 0; q < 2; q++) {
                        const float4 c = chunk[(h + 16 * q) >> page_shift];
                        const float A = c.x * ri.qs, C = max_nan(c.z, low) - base;
                        A2[q] = pack2(A, A);
                        C2[q] = pack2(C, C);
                        r[q] = fminf(c.w, inv_low);
                    }
                    tmem_ld_wait(x);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        unpack2(fma2(pack2(x[i], x[i + 1]), A2[i >> 4], C2[i >> 4]), x[i], x[i + 1]);
                        x[i] = ex2(x[i]);
                        x[i + 1] = ex2(x[i + 1]);
                    }
                    if (special) {
#pragma unroll
                        for (int i = 0; i < 32; i++) x[i] = h + i < lim ? x[i] : 0.f;
                    }
                    uint32_t w[16];  // the 32 tokens' first parts, then their second parts
#pragma unroll
                    for (int q = 0; q < 2; q++) {
                        uint64_t s0 = 0, s1 = 0;
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const int i = 16 * q + 4 * j;
                            const uint64_t e0 = pack2(x[i], x[i + 1]), e1 = pack2(x[i + 2], x[i + 3]);
                            s0 = add2(s0, e0);
                            s1 = add2(s1, e1);
                            float hi[4], lo[4];
                            split2(e0, hi[0], hi[1], lo[0], lo[1]);
                            split2(e1, hi[2], hi[3], lo[2], lo[3]);
                            w[4 * q + j] = e4m3x4_rn(hi[0], hi[1], hi[2], hi[3]);
                            w[8 + 4 * q + j] = e4m3x4_rn(lo[0], lo[1], lo[2], lo[3]);
                        }
                        float a0, a1;
                        unpack2(add2(s0, s1), a0, a1);
                        l = fmaf(a0 + a1, r[q], l);
                    }
                    tmem_st16(ts + (h >> 1), w);  // over scores that have been read
                }
                if constexpr (COPIES > 1) {  // the other copies' tokens have no weight in this one
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; i++) w[i] = 0u;
#pragma unroll
                    for (int i = 1; i < COPIES; i++)
#pragma unroll
                        for (int h = 0; h < kTake; h += 32) tmem_st16(ts + (((h0 + i * kTake + h) & (kTokens - 1)) >> 1), w);
                }
                tmem_st_wait();
                ml[(u % kRing) * kRows + row] = make_float2(mt, l);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(B.p_ready(sb));
            }

            if (seg < 0) continue;
            done += count;
            if (lane == 0) {
                mbar_arrive(B.q_empty(buf));
                mbar_arrive(B.seg_empty(seg % kSegs));
            }
        }
    } else {
        regs_inc<kRegsJoin>();
        // ------------------------------------------------- joining of outputs
        const int ew = warp & 3, row = 32 * ew + lane;
        const uint32_t lanes = (uint32_t)(32 * ew) << 16;
        const float2 *ml = reinterpret_cast<const float2 *>(smem + F.ml) + row;
        const uint32_t *nan = reinterpret_cast<const uint32_t *>(smem + F.nan);
        const size_t slot_floats = (size_t)a.rpt * D + 2 * a.rpt;
        float o[D];
        int u = 0, shared = 0;  // tiles joined; units shared with other CTAs
        // segment s's queries are loaded at the start of segment s - 1, whose first output is still far
        if constexpr (COPIES == 1) segment_queries<D, COPIES, SHARED>(a, smem, L, B, 0, ew, 4, true, abort_flag);

#pragma unroll 1
        for (int seg = 0;; seg++) {
            const int buf = seg & 1;
            if constexpr (COPIES == 1) {
                if (!warp_wait(B.q_full(buf), (uint32_t)(seg >> 1) & 1u, 0xc32u, abort_flag)) break;
            } else {
                // (one thread decides for all whether to go on, as barriers of the warpgroup follow)
                if (row == 0) *go = lane_wait(B.q_full(buf), (uint32_t)(seg >> 1) & 1u, 0xc32u, abort_flag) ? 1 : 0;
                named_barrier(kBarJoin, 128);
                if (*(volatile int *)go == 0) break;
                soft_wait(B.q_full(buf), (uint32_t)(seg >> 1) & 1u, 0xc34u, abort_flag);
            }
            const SegOf<SHARED> *sg = reinterpret_cast<const SegOf<SHARED> *>(smem + L.seg) + seg % kSegs;
            const RowInfo ri = reinterpret_cast<const RowInfo *>(smem + L.rows)[buf * kRows + row];
            const int count = sg->count, tile0 = sg->tile0;
            if (count == 0) break;
            if constexpr (COPIES == 1) segment_queries<D, COPIES, SHARED>(a, smem, L, B, seg + 1, ew, 4, true, abort_flag);
            float m_run = -INFINITY, l_run = 0.f;
#pragma unroll
            for (int i = 0; i < D; i++) o[i] = 0.f;
#pragma unroll 1
            for (int t = 0; t < count; t++, u++) {
                const int ob = u % kOBufs;
                soft_wait(B.o_full(ob), (uint32_t)(u / kOBufs) & 1u, 0xc20u, abort_flag);
                tc_fence_after();
                const float2 v = ml[(u % kRing) * kRows];
                const uint4 nm = *reinterpret_cast<const uint4 *>(nan + (u % kRing) * 4);
                const float m = fmaxf(m_run, v.x);
                const float f_old = m_run == -INFINITY ? 0.f : ex2_low(m_run - m),
                            f_new = v.x == -INFINITY ? 0.f : ex2_low(v.x - m);
                m_run = m;
                l_run = fmaf(l_run, f_old, v.y * f_new);
                const uint64_t g2 = pack2(f_new, f_new);
                if (__any_sync(0xffffffffu, f_old != 1.f)) {  // some row's maximum has moved
                    const uint64_t k2 = pack2(f_old, f_old);
#pragma unroll
                    for (int i = 0; i < D; i += 2) unpack2(mul2(pack2(o[i], o[i + 1]), k2), o[i], o[i + 1]);
                }
#pragma unroll
                for (int h = 0; h < D; h += 32) {
                    float y[32];
                    tmem_ld32(tmem_o + (uint32_t)(ob * D + h) + lanes, y);
                    tmem_ld_wait(y);
                    if (h + 32 == D) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(B.o_empty(ob));
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 2)
                        unpack2(fma2(pack2(y[i], y[i + 1]), g2, pack2(o[h + i], o[h + i + 1])), o[h + i], o[h + i + 1]);
                }
                // NaN values that only some rows see, back into those rows' outputs
                if ((nm.x | nm.y | nm.z | nm.w) != 0u) {
#pragma unroll 1
                    for (int k = 0; k < kTokens; k++) {
                        const uint32_t word = k < 32 ? nm.x : k < 64 ? nm.y : k < 96 ? nm.z : nm.w;
                        const int tn = (tile0 + t) * kTokens + k;
                        if (((word >> (k & 31)) & 1u) == 0u || tn > ri.pos) continue;
                        const uint8_t *code = value_codes(a, *sg, tn);
                        if (code == nullptr) continue;
#pragma unroll
                        for (int i = 0; i < D; i++)
                            if ((code[i] & 0x7fu) == 0x7fu) o[i] = kNan;
                    }
                }
            }

            if constexpr (COPIES > 1) {
                // the copies' results: all to the same reference, then added up in the first one's
                // warps, 32 values of the head at a time
                constexpr int kSpan = kRows / COPIES, kFirst = 4 / COPIES;
                float2 *mlc = reinterpret_cast<float2 *>(smem + F.mlc);
                float4 *merge = reinterpret_cast<float4 *>(smem + F.merge) + lane * 9;
                mlc[row] = make_float2(m_run, l_run);
                named_barrier(kBarJoin, 128);
                float2 v[COPIES];
                float m = -INFINITY, l = 0.f;
#pragma unroll
                for (int i = 0; i < COPIES; i++) {
                    v[i] = mlc[(row & (kSpan - 1)) + i * kSpan];
                    m = fmaxf(m, v[i].x);
                }
#pragma unroll
                for (int i = 0; i < COPIES; i++)
                    l += v[i].y == 0.f ? 0.f : v[i].y * ex2_low(v[i].x - m);  // (sum 0: it saw nothing; NaN stays)
                const float f = l_run == 0.f ? 0.f : ex2_low(m_run - m);
                m_run = m;
                l_run = l;
                const uint64_t f2 = pack2(f, f);
#pragma unroll
                for (int i = 0; i < D; i += 2) unpack2(mul2(pack2(o[i], o[i + 1]), f2), o[i], o[i + 1]);
#pragma unroll
                for (int h = 0; h < D; h += 32) {
                    if (ew >= kFirst) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            merge[(ew - kFirst) * (32 * 9) + i / 4] =
                                make_float4(o[h + i], o[h + i + 1], o[h + i + 2], o[h + i + 3]);
                    }
                    named_barrier(kBarJoin, 128);
                    if (ew < kFirst) {
#pragma unroll 1
                        for (int k = ew; k < 4 - kFirst; k += kFirst) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                const float4 y = merge[k * (32 * 9) + i / 4];
                                unpack2(add2(pack2(o[h + i], o[h + i + 1]), pack2(y.x, y.y)), o[h + i], o[h + i + 1]);
                                unpack2(add2(pack2(o[h + i + 2], o[h + i + 3]), pack2(y.z, y.w)), o[h + i + 2], o[h + i + 3]);
                            }
                        }
                    }
                    if (h + 32 < D) named_barrier(kBarJoin, 128);
                }
            }
            float *part = count < sg->nt ? a.part + (size_t)(2 * (int)blockIdx.x + (tile0 == 0 ? 1 : 0)) * slot_floats
                                        : nullptr;
            if (ri.row >= 0 && ew * COPIES < 4 && !*(volatile int *)abort_flag) {
                if (part != nullptr) {
                    float *d = part + (size_t)row * D;
#pragma unroll
                    for (int i = 0; i < D; i += 4)
                        *reinterpret_cast<float4 *>(d + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    *reinterpret_cast<float2 *>(part + (size_t)a.rpt * D + 2 * row) = make_float2(m_run, l_run);
                } else if (SHARED && a.what == kPrefixes) {
                    const size_t at = (size_t)ri.row * a.k.heads_q + ri.head;
                    float *d = a.half + at * D;
#pragma unroll
                    for (int i = 0; i < D; i += 4)
                        *reinterpret_cast<float4 *>(d + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    a.half_ml[at] = make_float2(m_run, l_run);
                } else {
                    float inv = l_run == 0.f ? 0.f : 1.f / l_run;  // (sum 0: it saw nothing; NaN stays)
                    float lse = 0.f;
                    if constexpr (SHARED) {
                        const size_t at = (size_t)ri.row * a.k.heads_q + ri.head;
                        const Halves h(a, at, m_run, l_run);
                        lse = h.lse;
                        inv = h.own;
                        if (a.what == kOwn) {
                            const float4 *p = reinterpret_cast<const float4 *>(a.half + at * D);
#pragma unroll
                            for (int i = 0; i < D; i += 4) {
                                const float4 x = __ldg(p + i / 4);
                                o[i] = fmaf(o[i], inv, x.x * h.prefix);
                                o[i + 1] = fmaf(o[i + 1], inv, x.y * h.prefix);
                                o[i + 2] = fmaf(o[i + 2], inv, x.z * h.prefix);
                                o[i + 3] = fmaf(o[i + 3], inv, x.w * h.prefix);
                            }
                            inv = 1.f;
                        }
                    }
                    uint16_t *d = a.k.out + (size_t)ri.row * a.k.ldo + (size_t)ri.head * D;
#pragma unroll
                    for (int i = 0; i < D; i += 8) {
                        uint32_t b[4];
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const __nv_bfloat162 z = __floats2bfloat162_rn(o[i + 2 * j] * inv, o[i + 2 * j + 1] * inv);
                            b[j] = *reinterpret_cast<const uint32_t *>(&z);
                        }
                        *reinterpret_cast<uint4 *>(d + i) = make_uint4(b[0], b[1], b[2], b[3]);
                    }
                    if (SHARED && a.k.lse != nullptr)
                        a.k.lse[(size_t)ri.row * a.k.heads_q + ri.head] = lse;
                    else if (a.k.lse != nullptr)
                        a.k.lse[(size_t)ri.row * a.k.heads_q + ri.head] =
                            l_run == 0.f ? -INFINITY : kLn2 * (m_run + log2f(l_run));
                }
            }
            if (part != nullptr) {
                if (row == 0) {
                    reinterpret_cast<SegOf<SHARED> *>(smem + L.split)[shared] = *sg;
                    *n_shared = shared + 1;
                }
                shared++;
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(B.q_empty(buf));
                mbar_arrive(B.seg_empty(seg % kSegs));
            }
        }
    }
    if (warp >= kFirstSoft) {
        named_barrier(kBarAll, kSoft);  // the list of shared units is complete
        join_role<D, kSoft, SHARED>(a, line, (int)blockIdx.x, reinterpret_cast<const SegOf<SHARED> *>(smem + L.split), *n_shared,
                            tid - 32 * kFirstSoft, kBarAll, abort_flag);
    }
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && *abort_flag != 0) set_status(st, MOE_ERR_TIMEOUT, (unsigned)*abort_flag);
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D, int COPIES, bool SHARED>
cudaError_t launch(const CUtensorMap &tm, AttnArgs a, int sms, int smem_max, cudaStream_t st) {
    static PerDevice smem_set(0);
    // (adding up the copies makes a unit's fixed cost larger; 24 ragged sequences of up to 8192, 4 rows:
    // 91 us with 3 tiles for it, 87 with 4, 80 with 6; one copy: 80, 81 and 84 for 48 x 9 rows, heads of 64)
    a.over = COPIES == 1 ? 3 : COPIES == 2 ? 4 : 6;
    a.nk = a.nv = 2;
    while (true) {  // as many stages as fit, values first
        AttnArgs b = a;
        if (b.nv < kMaxStages && b.nv < b.nk + 1)
            b.nv++;
        else if (b.nk < kMaxStages)
            b.nk++;
        else
            break;
        if (RowsSmem(D, b.nk, b.nv, COPIES).total + 1024u > (uint32_t)smem_max) break;
        a = b;
    }
    const size_t smem = RowsSmem(D, a.nk, a.nv, COPIES).total + 1024;
    if (smem > (size_t)smem_max) return cudaErrorNotSupported;
    cudaError_t e = ensure_dynamic_smem(kv_attention_rows_kernel<D, COPIES, SHARED>, smem, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;  // the join waits for all CTAs
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_attention_rows_kernel<D, COPIES, SHARED>, tm, a);
}

template <bool SHARED>
cudaError_t launch_rows(const CUtensorMap &tm, AttnArgs a, int sms, int smem_max, cudaStream_t st) {
    // Copies pay by the tile and cost by the unit, so not for heads of 128 where the table has room for
    // one tile of tokens only: 256 sequences of 128 tokens, 3 rows of 7 heads 96 us with copies, 90
    // without; 5 rows 114 and 99; of 256 tokens 105 and 113, 121 and 132.  (Heads of 64, half the
    // values to add up: 43 with copies at 128 tokens, 45 without.)
    const bool one_tile = a.k.kv.dim == 128 && (int64_t)a.k.table_width * a.k.kv.page <= kTokens;
    const int copies = a.rpt > 64 || one_tile ? 1 : a.rpt <= 32 ? 4 : 2;
    if (a.k.kv.dim == 128) {
        if (copies == 4) return launch<128, 4, SHARED>(tm, a, sms, smem_max, st);
        return copies == 2 ? launch<128, 2, SHARED>(tm, a, sms, smem_max, st) : launch<128, 1, SHARED>(tm, a, sms, smem_max, st);
    }
    if (copies == 4) return launch<64, 4, SHARED>(tm, a, sms, smem_max, st);
    return copies == 2 ? launch<64, 2, SHARED>(tm, a, sms, smem_max, st) : launch<64, 1, SHARED>(tm, a, sms, smem_max, st);
}

}  // namespace
}  // namespace moe
