// Attention of a few rows per sequence over the paged 8-bit key/value cache, on the
// tensor cores (tcgen05 kind::f8f6f4).
//
//   s[t][r] = ks_t * (k_t . q_r),  m_r = max_t s,  o_r = sum_t 2^(s - m) vs_t v_t / sum_t 2^(s - m)
//
// (log2 units: scale * log2(e) is folded into ks).  Few rows, many tokens: the cache is
// read once and everything else must hide behind that read, so
//
//   - Tokens, not rows, lie along M: S^T = K Q^T (M = 128 tokens, N = the rows of all
//     query heads of one key/value head) and O^T = V^T P^T (M = head_dim, N = rows,
//     K = 128 tokens).  However few the rows, every MMA is full along M, and K and V are
//     the A operands exactly as the tensor copies left them: codes go from HBM to shared
//     memory to the tensor cores with no conversion.  V^T is V's tile read M-major.
//   - What multiplies the codes must be E4M3 too.  A bf16 query is exactly the sum of two
//     E4M3 parts (4 + 4 significant bits) after a power of two per row; a weight is
//     written as two parts as well (8 bits, as bf16 has).  Each product runs twice into
//     the same accumulator; the tensor pipe has room (both products of a 128-token tile
//     take about 500 clocks of the 1400 that its 32 KB take from HBM).
//   - Pages' scales: ks_t multiplies the score of lane t; vs_t, relative to the tile's
//     largest, multiplies the weight before it is split.  Weights are taken relative to
//     the tile's own maximum and each tile's O^T is a fresh accumulator, joined with the
//     running one in registers: what E4M3's range cannot hold is then below 2^-17 of the
//     tile's largest term, however far another token stands above the tile.
//   - Work: the (sequence, row tile, head, 128-token tile) units of the whole call in one
//     line, cut into equal shares, one per SM.  A share may begin and end inside a
//     sequence; such partial results go to the workspace and, after a grid barrier
//     (cooperative launch), the CTAs that worked on the sequence join it, each some rows.
//     Shares are cut by the lengths on the device, so a captured graph serves any lengths.
//
// Roles: warp 0 copies (tensor copies of each page's K and V, the pages' scales by
// cp.async), warp 1 issues MMAs, warps 4-7 and 8-11 are two softmax warpgroups, each with
// half of the rows: TMEM lane = token for the scores, = value for the outputs.
#include <algorithm>

#include "kv_internal.cuh"
#include "sm100_tensor.cuh"

namespace moe {
namespace {

constexpr int kTokens = 128;    // tokens per tile
constexpr int kThreads = 384;
constexpr int kSoftThreads = 256;
constexpr int kMaxStages = 6;
constexpr int kMaxLen = 1 << 30;         // tokens of a sequence
constexpr int kMaxTileRows = 1 << 24;    // max_rows * query heads per key/value head
constexpr int kMaxSlots = kTokens / 16;  // pages per tile
constexpr uint32_t kSwizzle64B = 4;
constexpr int kStKvArrive = 40, kStKvExit = 5;  // StatusWord::pad

struct AttnArgs {
    KvAttentionArgs k;
    int group;      // query heads per key/value head
    int rpt;        // rows per tile (a multiple of 16, 2 * RW)
    int nrt;        // row tiles of max_rows rows
    int ns;         // pipeline stages
    float scale2;   // scale * log2(e)
    float *part;    // partial results: 2 slots per CTA of [rpt][dim] + [rpt][2]
};

// Shared memory, in bytes from a 1024-byte aligned base.
struct Smem {
    uint32_t kv, q, p, scales, smax, ref, ab, rows, lsum, bars, misc, total;
    __host__ __device__ Smem(int dim, int rpt, int ns) {
        const uint32_t rw = rpt / 2;
        uint32_t o = 0;
        kv = o;     o += (uint32_t)ns * 2u * kTokens * dim;   // [ns][K, V][128][dim]
        q = o;      o += 2u * rpt * dim;                      // [2 parts][rpt][dim]
        p = o;      o += 4u * rpt * kTokens;                  // [2 buffers][2 parts][rpt / 16][128][16]
        scales = o; o += (uint32_t)kMaxStages * 2u * kMaxSlots * 4u;
        smax = o;   o += 2u * 2u * 4u * rw * 4u;              // [2 buffers][wg][warp][rw]
        ref = o;    o += 8u * rw * 8u;                        // [warp][rw] (q scale, reference)
        ab = o;     o += 8u * 2u * rw * 8u;                   // [warp][2 buffers][rw] (old, new factors)
        rows = o;   o += 2u * (uint32_t)rpt * 12u;            // [2][rpt] (row, head, q scale)
        lsum = o;   o += 2u * 4u * rw * 4u;                   // [wg][warp][rw]
        o = (o + 15u) & ~15u;
        bars = o;   o += (2u * kMaxStages + 8u) * 8u;
        misc = o;   o += 256u;
        total = o;
    }
};

// One (sequence, row tile): its rows, tokens and tiles.
struct Item {
    int b, rt, row0, n, len, nt;
    bool ok;
};

__device__ __forceinline__ Item load_item(const AttnArgs &a, int it) {
    Item x;
    x.b = it / a.nrt;
    x.rt = it - x.b * a.nrt;
    int hi;
    x.ok = seq_rows(a.k.cu_rows, x.b, a.k.rows, x.row0, hi);
    x.n = hi - x.row0;
    if (x.n > a.k.max_rows) {
        x.n = a.k.max_rows;
        x.ok = false;
    }
    const int64_t room = min((int64_t)a.k.table_width * a.k.kv.page, (int64_t)kMaxLen);
    const int len = max(a.k.kv_len[x.b], 0);
    if ((int64_t)len > room) x.ok = false;
    x.len = (int)min((int64_t)len, room);
    x.nt = 0;
    if (x.rt * a.rpt < x.n * a.group) {
        const int last = min(x.n - 1, ((x.rt + 1) * a.rpt - 1) / a.group);  // last row of the tile
        const int see = min(x.len, max(0, x.len - x.n + last + 1));
        x.nt = max(1, (see + kTokens - 1) / kTokens);
    }
    return x;
}

// A CTA's share: the line of (item, head, tile) units from w to hi, walked in segments of
// one (item, head) each.  All roles walk it alike.
struct Walk {
    const AttnArgs &a;
    int64_t w, hi, first;  // next unit; end; first unit of the item
    int it;
    Item x;
    int head, tile0, count;  // the segment
    int see_all, see_max;    // tokens every row of the tile sees, and any row

    __device__ Walk(const AttnArgs &args, int64_t lo, int64_t hi_, int64_t first_, int it_)
        : a(args), w(lo), hi(hi_), first(first_), it(it_) {
        if (valid()) {
            x = load_item(a, it);
            load();
        }
    }
    __device__ bool valid() const { return w < hi; }
    __device__ void load() {
        while (w - first >= x.nt * (int64_t)a.k.kv.heads) {
            first += (int64_t)x.nt * a.k.kv.heads;
            x = load_item(a, ++it);
        }
        const int local = (int)(w - first);
        head = local / x.nt;
        tile0 = local - head * x.nt;
        count = (int)min((int64_t)(x.nt - tile0), hi - w);
        const int q0 = x.rt * a.rpt / a.group, q1 = min(x.n - 1, ((x.rt + 1) * a.rpt - 1) / a.group);
        see_all = min(x.len, max(0, x.len - x.n + q0 + 1));
        see_max = min(x.len, max(0, x.len - x.n + q1 + 1));
    }
    __device__ void next() {
        w += count;
        if (valid()) load();
    }
    __device__ int64_t unit0() const { return first + (int64_t)head * x.nt; }  // the unit's first tile
    __device__ bool split() const { return count < x.nt; }
};

// The CTA whose share of `total` units over `ctas` CTAs holds unit w.
__device__ __forceinline__ int cta_of(int64_t w, int64_t total, int ctas) {
    return (int)(((w + 1) * ctas - 1) / total);
}

// ------------------------------------------------------------ PTX

__device__ __forceinline__ uint32_t idesc_f8(int m, int n, bool transposed) {
    uint32_t d = 1u << 4;                     // fp32 accumulator; A and B E4M3 (0)
    if (transposed) d |= (1u << 15) | (1u << 16);  // both operands M / N-major
    d |= (uint32_t)(n >> 3) << 17;
    d |= (uint32_t)(m >> 4) << 24;
    return d;
}

__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 8 accumulator columns of this warp's 32 lanes, not waited for.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float *v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr)
                 : "memory");
}
// Wait for them; the registers pass through, so that no use moves before the wait.
template <int N>
__device__ __forceinline__ void tmem_ld_wait(float (&v)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; i++) asm volatile("" : "+f"(v[i]));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 4 bytes global -> shared, asynchronously; zero without reading if !ok.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
// One arrival on `bar` once this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Reduce N rows (v[i] of every lane) over the warp's 32 lanes by halving: lane l ends with
// the result of row l >> log2(32 / N), after N - 1 exchanges plus log2(32 / N).
template <int N, typename Op>
__device__ __forceinline__ float reduce_rows(float (&v)[N], int lane, Op op) {
#pragma unroll
    for (int h = N / 2, mask = 16; h >= 1; h >>= 1, mask >>= 1) {
        const bool up = (lane & mask) != 0;
#pragma unroll
        for (int i = 0; i < h; i++) {
            const float send = up ? v[i] : v[i + h], keep = up ? v[i + h] : v[i];
            v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, mask));
        }
    }
    float r = v[0];
#pragma unroll
    for (int mask = 16 / N; mask >= 1; mask >>= 1) r = op(r, __shfl_xor_sync(0xffffffffu, r, mask));
    return r;
}

// RW rows in pieces of 32, 16 and 8 for reduce_rows.
template <int RW>
struct Pieces {
    static constexpr int n = RW / 32 + ((RW & 16) ? 1 : 0) + ((RW & 8) ? 1 : 0);
    __host__ __device__ static constexpr int size(int i) { return i < RW / 32 ? 32 : (i == RW / 32 && (RW & 16)) ? 16 : 8; }
    __host__ __device__ static constexpr int off(int i) {
        int o = 0;
        for (int j = 0; j < i; j++) o += size(j);
        return o;
    }
};

struct MaxOp {
    __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct AddOp {
    __device__ float operator()(float a, float b) const { return a + b; }
};

template <int I>
struct Index {
    static constexpr int value = I;
};

// f(piece index as a constant) for each piece.
template <int RW, int I = 0, typename F>
__device__ __forceinline__ void each_piece(F &&f) {
    if constexpr (I < Pieces<RW>::n) {
        f(Index<I>{});
        each_piece<RW, I + 1>(f);
    }
}

// The two E4M3 parts of a value: the nearest of 4 significant bits, and what is left.
__device__ __forceinline__ float part_hi(float x) {
    return __uint_as_float((__float_as_uint(x) + 0x80000u) & 0xfff00000u);
}

template <int D, int RW>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_kernel(const __grid_constant__ CUtensorMap tm,
                                                                    const AttnArgs a) {
    constexpr int kRpt = 2 * RW;
    constexpr uint32_t kTile = kTokens * D;           // bytes of a K or V tile
    constexpr uint32_t kSwz = D == 128 ? kSwizzle128B : kSwizzle64B;
    constexpr uint32_t kGroup8 = 8 * D;               // bytes of 8 rows
    constexpr uint32_t kTmemCols = 4 * kRpt <= 64 ? 64 : 4 * kRpt <= 128 ? 128 : 4 * kRpt <= 256 ? 256 : 512;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = (unsigned char *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const int ns = a.ns;
    const Smem L(D, kRpt, ns);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L.bars);
    uint64_t *empty = full + kMaxStages;
    uint64_t *s_full = empty + kMaxStages;   // [2] scores in TMEM
    uint64_t *p_ready = s_full + 2;          // [2] weights in shared memory, scores read
    uint64_t *o_full = p_ready + 2;          // [2] outputs in TMEM
    uint64_t *q_ready = o_full + 2;
    uint64_t *mma_done = q_ready + 1;
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + L.misc);
    uint32_t *tmem_slot = misc;
    int *abort_flag = reinterpret_cast<int *>(misc + 1);
    uint32_t *nan_mask = misc + 4;                                    // [4 buffers][4 warps]
    int64_t *plan = reinterpret_cast<int64_t *>(misc + 20);           // first, item; then the scan's sums
    int64_t *sums = plan + 2;
    StatusWord *st = a.k.st;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // ------------------------------------------------------------ the plan
    const int items = a.k.seqs * a.nrt;
    const int per = (items + kThreads - 1) / kThreads;
    const int i0 = min(tid * per, items), i1 = min(i0 + per, items);
    int64_t mine = 0;
    bool good = true;
    for (int i = i0; i < i1; i++) {
        const Item x = load_item(a, i);
        good &= x.ok;
        mine += (int64_t)x.nt * a.k.kv.heads;
    }
    if (!good && blockIdx.x == 0) set_status(st, MOE_ERR_BAD_PAGE, 1);
    int64_t pre = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, pre, d);
        if (lane >= d) pre += o;
    }
    if (lane == 31) sums[warp] = pre;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; w++) {
        if (w < warp) pre += sums[w];
        total += sums[w];
    }
    pre -= mine;
    const int ctas = (int)min((int64_t)gridDim.x, total), cta = blockIdx.x;
    if (cta >= ctas) return;  // the whole CTA: nothing set up yet
    const int64_t lo = total * cta / ctas, hi = total * (cta + 1) / ctas;
    if (lo >= pre && lo < pre + mine) {
        int64_t at = pre;
        for (int i = i0; i < i1; i++) {
            const int64_t u = (int64_t)load_item(a, i).nt * a.k.kv.heads;
            if (lo < at + u) {
                plan[0] = at;
                plan[1] = i;
                break;
            }
            at += u;
        }
    }
    if (tid == 0) {
        for (int s = 0; s < ns; s++) {
            mbar_init(&full[s], 33);  // the expect-tx arrival, and every copying lane's scales
            mbar_init(&empty[s], 1);  // MMA commit
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(&s_full[b], 1);
            mbar_init(&p_ready[b], 8);  // the softmax warps
            mbar_init(&o_full[b], 1);
        }
        mbar_init(q_ready, 8);
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tmem_o = tmem + 2 * kRpt;
    Walk W(a, lo, hi, plan[0], (int)plan[1]);

    int it_issued = 0;
    if (warp == 0) {
        // ---------------------------------------------------------- copies
        const KvView &kv = a.k.kv;
        const int P = kv.page, slots = kTokens / P;
        int g = 0, s = 0;
        uint32_t ph = 0;
        bool run = true;
        for (; run && W.valid(); W.next()) {
            const int32_t *row = a.k.page_table + (size_t)W.x.b * a.k.table_width;
            const int pages = (W.see_max + P - 1) / P;
            const int c0 = W.tile0 * slots, c1 = min(pages, (W.tile0 + W.count) * slots);
            // page numbers, 32 columns at a time: lane l holds column base + l, and the next 32
            int base = c0;
            int id = base + lane < c1 ? row[base + lane] : -1;
            int id2 = base + 32 + lane < c1 ? row[base + 32 + lane] : -1;
            for (int t = 0; t < W.count; t++, g++) {
                int okl = 1;
                if (lane == 0) okl = mbar_wait_or_abort(&empty[s], ph ^ 1u, st, 0xa00u + s, abort_flag);
                if (!__shfl_sync(0xffffffffu, okl, 0)) {
                    if (lane == 0) *abort_flag = 1;
                    run = false;
                    break;
                }
                const int col = (W.tile0 + t) * slots;
                if (col >= base + 32) {
                    base += 32;
                    id = id2;
                    id2 = base + 32 + lane < c1 ? row[base + 32 + lane] : -1;
                }
                const int used = max(0, min(slots, c1 - col));
                const int page = __shfl_sync(0xffffffffu, id, (col - base + lane) & 31);
                if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)used * 2u * (uint32_t)(P * D));
                __syncwarp();
                if (lane < kMaxSlots) {
                    const bool have = lane < used;
                    const bool ok = have && page >= 0 && page < kv.n_pages;
                    if (have && !ok) set_status(st, MOE_ERR_BAD_PAGE, 3);
                    uint8_t *dst = smem + L.kv + (uint32_t)s * 2u * kTile + (uint32_t)lane * (uint32_t)(P * D);
                    if (have) {
                        // a page outside the cache lies outside the tensor: zeros arrive
                        const int pg = ok ? page : kv.n_pages;
                        tma_load_3d(dst, &tm, 0, W.head * P, pg, &full[s]);
                        tma_load_3d(dst + kTile, &tm, 0, (kv.heads + W.head) * P, pg, &full[s]);
                    }
                    const uint32_t sc = smem_u32(smem + L.scales) + (uint32_t)(s * 2 * kMaxSlots + lane) * 4u;
                    const float *src = kv.scale(ok ? page : 0, a.k.layer, 0, W.head);
                    cp_async4(sc, src, ok);
                    cp_async4(sc + kMaxSlots * 4u, src + kv.heads, ok);
                }
                cp_async_arrive(&full[s]);
                it_issued = g + 1;
                if (++s == ns) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issue
        const uint32_t id_s = idesc_f8(128, kRpt, false), id_o = idesc_f8(D, kRpt, true);
        const uint64_t kd = smem_desc(smem_u32(smem + L.kv), 16, kGroup8, kSwz);
        const uint64_t vd = smem_desc(smem_u32(smem + L.kv) + kTile, kGroup8, kGroup8, kSwz);
        const uint64_t qd = smem_desc(smem_u32(smem + L.q), 16, kGroup8, kSwz);
        // weights: N-major without swizzle, 16 rows x 8 tokens (128 bytes) per core matrix,
        // 8-token groups 128 bytes and 16-row chunks 2 KB apart
        const uint64_t pd = smem_desc(smem_u32(smem + L.p), 128, kTokens * 16, kSwizzleNone);
        int g = 0, s = 0, seg = 0;
        uint32_t ph = 0;
        bool run = true, pending = false;
        int pv_s = 0;
        auto wait = [&](uint64_t *bar, uint32_t parity, unsigned where) {
            int okl = 1;
            if (lane == 0) okl = mbar_wait_or_abort(bar, parity, st, where, abort_flag);
            okl = __shfl_sync(0xffffffffu, okl, 0);
            if (!okl && lane == 0) *abort_flag = 1;
            return okl != 0;
        };
        // O^T of tile g - 1, whose stage is pv_s
        auto issue_pv = [&]() {
            const int u = g - 1, buf = u & 1;
            pending = false;
            if (!wait(&p_ready[buf], (uint32_t)(u >> 1) & 1u, 0xb10u + buf)) return false;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t va = vd + (uint64_t)((uint32_t)pv_s * (2u * kTile) >> 4);
                const uint64_t pb = pd + (uint64_t)((uint32_t)buf * (2u * kRpt * kTokens) >> 4);
#pragma unroll
                for (int part = 0; part < 2; part++)
#pragma unroll
                    for (int ks = 0; ks < kTokens / 32; ks++)
                        tc_mma_f8(tmem_o + (uint32_t)(buf * kRpt), va + (uint64_t)(ks * (32 * D) >> 4),
                                  pb + (uint64_t)(part * (kRpt * kTokens) >> 4) + (uint64_t)(ks * 32), id_o,
                                  (part > 0 || ks > 0) ? 1u : 0u);
                tc_commit(&empty[pv_s]);
                tc_commit(&o_full[buf]);
            }
            __syncwarp();
            return true;
        };
        for (; run && W.valid(); W.next(), seg++) {
            if (pending && !(run = issue_pv())) break;
            if (!(run = wait(q_ready, (uint32_t)seg & 1u, 0xb20u))) break;
            for (int t = 0; t < W.count; t++) {
                if (!(run = wait(&full[s], ph, 0xb00u + s))) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t ka = kd + (uint64_t)((uint32_t)s * (2u * kTile) >> 4);
#pragma unroll
                    for (int part = 0; part < 2; part++)
#pragma unroll
                        for (int ks = 0; ks < D / 32; ks++)
                            tc_mma_f8(tmem + (uint32_t)((g & 1) * kRpt), ka + (uint64_t)(2 * ks),
                                      qd + (uint64_t)(part * (kRpt * D) >> 4) + (uint64_t)(2 * ks), id_s,
                                      (part > 0 || ks > 0) ? 1u : 0u);
                    tc_commit(&s_full[g & 1]);
                }
                __syncwarp();
                if (pending && !(run = issue_pv())) break;
                pending = true;
                pv_s = s;
                g++;
                if (++s == ns) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (run && pending) issue_pv();
        // every MMA has finished before TMEM is released
        if (elect_one()) tc_commit(mma_done);
        __syncwarp();
        if (lane == 0) mbar_wait(mma_done, 0u, st, 0xb30u);
        __syncwarp();
    } else if (warp >= 4) {
        // -------------------------------------------------------- softmax
        const int ew = warp & 3, wg = (warp - 4) >> 2, sw = warp - 4;
        const int tok = 32 * ew + lane;                 // token of the tile (TMEM lane)
        const uint32_t lanes = (uint32_t)(32 * ew) << 16;
        const int bar_id = 1 + wg;
        float *smax = reinterpret_cast<float *>(smem + L.smax) + wg * 4 * RW;  // + buf * 8 * RW + warp * RW
        float2 *ref = reinterpret_cast<float2 *>(smem + L.ref) + sw * RW;
        float2 *ab = reinterpret_cast<float2 *>(smem + L.ab) + sw * 2 * RW;
        float *lsum = reinterpret_cast<float *>(smem + L.lsum) + wg * 4 * RW;
        int *rows = reinterpret_cast<int *>(smem + L.rows) + wg * RW;  // + par * 3 * kRpt; [row | head | q scale]
        const float *scales = reinterpret_cast<const float *>(smem + L.scales);
        const KvView &kv = a.k.kv;
        const int page_shift = 31 - __clz(kv.page);
        constexpr int NP = Pieces<RW>::n;
        float o[RW] = {};
        float m_run[NP] = {}, l_run[NP] = {}, qs[NP] = {};
        int g = 0, s = 0, par = 0;
        uint32_t ph = 0;

        // The tile's queries as two E4M3 parts (this warpgroup's rows), with a power of two
        // per row that puts its largest value into [128, 256).
        auto load_q = [&](const Walk &w, int par_) {
            int *rr = rows + par_ * 3 * kRpt;
            for (int i = ew; i < RW; i += 4) {
                const int r = wg * RW + i, R = w.x.rt * kRpt + r;
                const bool live = R < w.x.n * a.group;
                const int qi = R / a.group, row = w.x.row0 + qi, hq = w.head * a.group + R - qi * a.group;
                constexpr int V = D / 32;
                float x[V];
                uint32_t amax = 0;
#pragma unroll
                for (int j = 0; j < V; j += 2) {
                    uint32_t u = 0;
                    if (live)
                        u = *reinterpret_cast<const uint32_t *>(a.k.q + (size_t)row * a.k.ldq + (size_t)hq * D +
                                                                lane * V + j);
                    x[j] = __uint_as_float(u << 16);
                    x[j + 1] = __uint_as_float(u & 0xffff0000u);
                    const uint32_t m0 = (u & 0x7fffu), m1 = (u >> 16) & 0x7fffu;
                    amax = max(amax, max(m0 < 0x7f80u ? m0 : 0u, m1 < 0x7f80u ? m1 : 0u));
                }
                amax = __reduce_max_sync(0xffffffffu, amax);
                const int up = amax == 0 ? 0 : min(126, 7 - ((int)(amax >> 7) - 127));
                const float f = __uint_as_float((uint32_t)(127 + up) << 23);
                float h[V], l[V];
#pragma unroll
                for (int j = 0; j < V; j++) {
                    h[j] = part_hi(x[j] * f);
                    l[j] = x[j] * f - h[j];
                }
                // 16-byte chunks of a row are permuted by the swizzle of the K tile
                const uint32_t byte = (uint32_t)(lane * V), chunk = byte >> 4;
                const uint32_t swz = D == 128 ? (uint32_t)(r & 7) : (uint32_t)((r >> 1) & 3);
                uint8_t *dst = smem + L.q + (uint32_t)r * D + ((chunk ^ swz) << 4) + (byte & 15u);
                if constexpr (D == 128) {
                    *reinterpret_cast<uint32_t *>(dst) = e4m3x4_rn(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint32_t *>(dst + kRpt * D) = e4m3x4_rn(l[0], l[1], l[2], l[3]);
                } else {
                    *reinterpret_cast<uint16_t *>(dst) = (uint16_t)e4m3x2_rn(h[0], h[1]);
                    *reinterpret_cast<uint16_t *>(dst + kRpt * D) = (uint16_t)e4m3x2_rn(l[0], l[1]);
                }
                if (lane == 0) {
                    rr[i] = live ? row : -1;
                    rr[kRpt + i] = hq;
                    rr[2 * kRpt + i] = (127 - up) << 23;
                }
            }
            fence_proxy_async_smem();
            named_barrier(bar_id, 128);  // the rows' data is read by the whole warpgroup
            if (lane == 0) mbar_arrive(q_ready);
        };

        // Waits that cannot deadlock the warpgroup's barriers: after an abort nothing waits.
        auto wait = [&](uint64_t *bar, uint32_t parity, unsigned where) {
            if (!*(volatile int *)abort_flag && !mbar_wait_or_abort(bar, parity, st, where, abort_flag)) *abort_flag = 1;
            __syncwarp();
        };

        // Scores of tile u -> weights in shared memory; running maxima and sums.
        auto softmax = [&](const Walk &w, int tile) {
            const int buf = g & 1;
            const int t = tile * kTokens + tok;
            wait(&s_full[buf], (uint32_t)(g >> 1) & 1u, 0xc00u + buf);
            wait(&full[s], ph, 0xc10u + s);  // (complete: the scores were computed from it)
            tc_fence_after();
            float x[RW];
#pragma unroll
            for (int i = 0; i < RW; i += 8) tmem_ld8(tmem + (uint32_t)(buf * kRpt + wg * RW + i) + lanes, x + i);
            tmem_ld_wait(x);
            const bool special = (tile + 1) * kTokens > w.see_all;
            const float *sc = scales + s * 2 * kMaxSlots;
            const float ks = sc[tok >> page_shift] * a.scale2;
            // V scales relative to the tile's largest (finite) one
            const int slots = kTokens >> page_shift;
            float vmax = 0.f;
            for (int j = 0; j < slots; j++) {
                const float v = sc[kMaxSlots + j];
                vmax = v < INFINITY ? fmaxf(vmax, v) : vmax;
            }
            const float vs = sc[kMaxSlots + (tok >> page_shift)];
            const float vone = vmax > 0.f ? vmax : 1.f;
            float c = 256.f * (vs / vone);
            if (!(vs < INFINITY)) c = __uint_as_float(0x7fc00000u);
            if (t >= w.see_max) c = 0.f;
#pragma unroll
            for (int i = 0; i < RW; i++) x[i] *= ks;
            if (special) {
                // row r sees token t if r >= rmin
                const int rmin = t >= w.see_max ? RW : a.group * max(0, t - (w.x.len - w.x.n)) - w.x.rt * kRpt - wg * RW;
#pragma unroll
                for (int i = 0; i < RW; i++) x[i] = i >= rmin ? x[i] : -INFINITY;
                if (wg == 0) {
                    // V rows that no row sees hold anything: zero.  NaN in rows that only some
                    // rows see must not reach the others: zero here, put back in the output.
                    uint8_t *v = smem + L.kv + (uint32_t)s * 2u * kTile + kTile + (uint32_t)tok * D;
                    bool bad = false;
                    if (t >= w.see_all) {
#pragma unroll
                        for (int j = 0; j < D / 16; j++) {
                            uint4 *q = reinterpret_cast<uint4 *>(v) + j;
                            uint4 z = make_uint4(0u, 0u, 0u, 0u);
                            if (t < w.see_max) {
                                z = *q;
                                uint32_t *zw = &z.x;
#pragma unroll
                                for (int k = 0; k < 4; k++) {
                                    const uint32_t n = __vcmpeq4(zw[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                    bad |= n != 0;
                                    zw[k] &= ~n;
                                }
                            }
                            *q = z;
                        }
                    }
                    const uint32_t mask = __ballot_sync(0xffffffffu, bad);
                    if (lane == 0) nan_mask[(g & 3) * 4 + ew] = mask;
                }
            } else if (wg == 0 && lane == 0) {
                nan_mask[(g & 3) * 4 + ew] = 0u;
            }
            // the tile's maximum of each row: over the warp's tokens, then over the four warps
            float *mx = smax + buf * 8 * RW;
            each_piece<RW>([&](auto I) {
                constexpr int pc = decltype(I)::value, N = Pieces<RW>::size(pc), off = Pieces<RW>::off(pc);
                float v[N];
#pragma unroll
                for (int i = 0; i < N; i++) v[i] = x[off + i];
                const float r = reduce_rows<N>(v, lane, MaxOp());
                mx[ew * RW + off + (lane * N >> 5)] = r;
            });
            named_barrier(bar_id, 128);
            float old[NP], now[NP];
            each_piece<RW>([&](auto I) {
                constexpr int pc = decltype(I)::value, N = Pieces<RW>::size(pc), off = Pieces<RW>::off(pc);
                const int r = off + (lane * N >> 5);
                const float mt = fmaxf(fmaxf(mx[r], mx[RW + r]), fmaxf(mx[2 * RW + r], mx[3 * RW + r])) * qs[pc];
                const float m = fmaxf(m_run[pc], mt);
                old[pc] = m_run[pc] == -INFINITY ? 0.f : ex2(m_run[pc] - m);
                now[pc] = mt == -INFINITY ? 0.f : ex2(mt - m);
                m_run[pc] = m;
                ref[r] = make_float2(qs[pc], mt == -INFINITY ? 0.f : mt);
                ab[buf * RW + r] = make_float2(old[pc], now[pc] * (vone * (1.f / 256.f)));
            });
            __syncwarp();
            uint8_t *pw = smem + L.p + (uint32_t)buf * (2u * kRpt * kTokens) + (uint32_t)tok * 16u;
            each_piece<RW>([&](auto I) {
                constexpr int pc = decltype(I)::value, N = Pieces<RW>::size(pc), off = Pieces<RW>::off(pc);
                float p[N];
#pragma unroll
                for (int i = 0; i < N; i += 8) {
                    float h[8], l[8];
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const float2 rq = ref[off + i + j];
                        const float y = fmaf(x[off + i + j], rq.x, -rq.y);
                        const float e = ex2(y);
                        p[i + j] = e;
                        float wv = e * c;
                        if (special) wv = x[off + i + j] == -INFINITY ? 0.f : wv;
                        h[j] = part_hi(wv);
                        l[j] = wv - h[j];
                    }
                    const int r = wg * RW + off + i;  // 8 rows: half a 16-row chunk
                    uint8_t *d = pw + (uint32_t)(r >> 4) * (kTokens * 16u) + (uint32_t)(r & 8);
                    *reinterpret_cast<uint2 *>(d) =
                        make_uint2(e4m3x4_rn(h[0], h[1], h[2], h[3]), e4m3x4_rn(h[4], h[5], h[6], h[7]));
                    *reinterpret_cast<uint2 *>(d + kRpt * kTokens) =
                        make_uint2(e4m3x4_rn(l[0], l[1], l[2], l[3]), e4m3x4_rn(l[4], l[5], l[6], l[7]));
                }
                const float sum = reduce_rows<N>(p, lane, AddOp());
                l_run[pc] = l_run[pc] * old[pc] + sum * now[pc];
            });
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready[buf]);
            g++;
            if (++s == ns) {
                s = 0;
                ph ^= 1u;
            }
        };

        // Add O^T of tile u to the running output.
        auto join_tile = [&](const Walk &w, int u, int tile) {
            const int buf = u & 1;
            wait(&o_full[buf], (uint32_t)(u >> 1) & 1u, 0xc20u + buf);
            tc_fence_after();
            float y[RW];
#pragma unroll
            for (int i = 0; i < RW; i += 8) tmem_ld8(tmem_o + (uint32_t)(buf * kRpt + wg * RW + i) + lanes, y + i);
            tmem_ld_wait(y);
            const float2 *f = ab + buf * RW;
#pragma unroll
            for (int i = 0; i < RW; i++) {
                const float2 k = f[i];
                o[i] = fmaf(y[i], k.y, o[i] * k.x);
            }
            // NaN values that only some rows see (see softmax)
            const uint4 nm = *reinterpret_cast<const uint4 *>(nan_mask + (u & 3) * 4);
            if ((nm.x | nm.y | nm.z | nm.w) != 0u) {
                const int d = D == 128 ? tok : 16 * ew + lane;
                for (int k = 0; k < kTokens; k++) {
                    const uint32_t word = k < 32 ? nm.x : k < 64 ? nm.y : k < 96 ? nm.z : nm.w;
                    if (!((word >> (k & 31)) & 1u) || (D == 64 && lane >= 16)) continue;
                    const int t = tile * kTokens + k;
                    const int page = a.k.page_table[(size_t)w.x.b * a.k.table_width + (t >> page_shift)];
                    if (page < 0 || page >= kv.n_pages) continue;
                    const uint8_t code = kv.codes(page, a.k.layer, 1, w.head)[(t & (kv.page - 1)) * D + d];
                    if ((code & 0x7fu) != 0x7fu) continue;
                    const int rmin = a.group * max(0, t - (w.x.len - w.x.n)) - w.x.rt * kRpt - wg * RW;
#pragma unroll
                    for (int i = 0; i < RW; i++)
                        if (i >= rmin) o[i] = __uint_as_float(0x7fc00000u);
                }
            }
        };

        const int dcol = D == 128 ? tok : 16 * ew + lane;       // value of the head this lane holds
        const bool dlive = D == 128 || lane < 16;
        const size_t slot_floats = (size_t)kRpt * D + 2 * kRpt;
        if (W.valid()) load_q(W, 0);
        while (W.valid()) {
            const Walk cur = W;
            int *rr = rows + par * 3 * kRpt;
            each_piece<RW>([&](auto I) {
                constexpr int pc = decltype(I)::value, N = Pieces<RW>::size(pc), off = Pieces<RW>::off(pc);
                qs[pc] = __int_as_float(rr[2 * kRpt + off + (lane * N >> 5)]);
                m_run[pc] = -INFINITY;
                l_run[pc] = 0.f;
            });
#pragma unroll
            for (int i = 0; i < RW; i++) o[i] = 0.f;
            for (int t = 0; t < cur.count; t++) {
                softmax(cur, cur.tile0 + t);
                if (t > 0) join_tile(cur, g - 2, cur.tile0 + t - 1);
            }
            // the next segment's queries (every score of this one has been computed)
            W.next();
            if (W.valid()) load_q(W, par ^ 1);
            join_tile(cur, g - 1, cur.tile0 + cur.count - 1);
            // sums over the four warps
            each_piece<RW>([&](auto I) {
                constexpr int pc = decltype(I)::value, N = Pieces<RW>::size(pc), off = Pieces<RW>::off(pc);
                lsum[ew * RW + off + (lane * N >> 5)] = l_run[pc];
            });
            named_barrier(bar_id, 128);
            float *part = cur.split() ? a.part + (size_t)(2 * cta + (cur.tile0 == 0 ? 1 : 0)) * slot_floats : nullptr;
            each_piece<RW>([&](auto I) {
                constexpr int pc = decltype(I)::value, N = Pieces<RW>::size(pc), off = Pieces<RW>::off(pc);
                const int r = off + (lane * N >> 5);
                const float l = lsum[r] + lsum[RW + r] + lsum[2 * RW + r] + lsum[3 * RW + r];
                ref[r] = make_float2(m_run[pc] == -INFINITY ? 0.f : 1.f / l, 0.f);
                if (ew == 0 && (lane * N & 31) == 0) {  // one lane per row
                    if (part != nullptr) {
                        float *ml = part + (size_t)kRpt * D + 2 * (wg * RW + r);
                        ml[0] = m_run[pc];
                        ml[1] = l;
                    } else if (a.k.lse != nullptr && rr[r] >= 0) {
                        a.k.lse[(size_t)rr[r] * a.k.heads_q + rr[kRpt + r]] =
                            m_run[pc] == -INFINITY ? -INFINITY : 0.6931471805599453f * (m_run[pc] + log2f(l));
                    }
                }
            });
            __syncwarp();
            if (dlive && !*(volatile int *)abort_flag) {
#pragma unroll
                for (int i = 0; i < RW; i++) {
                    if (rr[i] < 0) continue;
                    if (part != nullptr)
                        part[(size_t)(wg * RW + i) * D + dcol] = o[i];
                    else
                        a.k.out[(size_t)rr[i] * a.k.ldo + (size_t)rr[kRpt + i] * D + dcol] =
                            __bfloat16_as_ushort(__float2bfloat16(o[i] * ref[i].x));
                }
            }
            named_barrier(bar_id, 128);  // lsum and this parity's rows are free
            par ^= 1;
        }

        // ----------------------------------------- units shared with other CTAs
        unsigned int *arrive = &st->pad[kStKvArrive], *leave = &st->pad[kStKvExit];
        __threadfence();
        named_barrier(3, kSoftThreads);
        if (tid == 128) red_release_gpu_add(arrive, 1u);
        bool waited = false;
        for (Walk J(a, lo, hi, plan[0], (int)plan[1]); J.valid(); J.next()) {
            if (!J.split()) continue;
            if (!waited) {
                waited = true;
                if (tid == 128 && *(volatile int *)abort_flag == 0) {
                    const uint64_t t0 = global_timer_ns(), lim = g_wait_limit_ns;
                    while (ld_acquire_gpu(arrive) < (unsigned)ctas) {
                        if (global_timer_ns() - t0 > lim) {
                            set_status(st, MOE_ERR_TIMEOUT, 0xd00u);
                            *abort_flag = 1;
                            break;
                        }
                    }
                }
                named_barrier(3, kSoftThreads);
            }
            if (*(volatile int *)abort_flag) continue;
            const int64_t u0 = J.unit0();
            const int c0 = cta_of(u0, total, ctas), c1 = cta_of(u0 + J.x.nt - 1, total, ctas), parts = c1 - c0 + 1;
            const int nrows = min(kRpt, J.x.n * a.group - J.x.rt * kRpt);
            // rows cta - c0, + parts, ...: a warp per row, lanes over the head's values
            for (int r = (cta - c0) + parts * sw; r < nrows; r += parts * (kSoftThreads / 32)) {
                constexpr int V = D / 32;
                float m = -INFINITY;
                for (int p = lane; p < parts; p += 32) {
                    const float *slot = a.part + (size_t)(2 * (c0 + p) + (p == 0 ? 1 : 0)) * slot_floats;
                    m = fmaxf(m, __ldcg(slot + (size_t)kRpt * D + 2 * r));
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                float l = 0.f, acc[V];
#pragma unroll
                for (int j = 0; j < V; j++) acc[j] = 0.f;
#pragma unroll 4
                for (int p = 0; p < parts; p++) {
                    const float *slot = a.part + (size_t)(2 * (c0 + p) + (p == 0 ? 1 : 0)) * slot_floats;
                    const float2 ml = __ldcg(reinterpret_cast<const float2 *>(slot + (size_t)kRpt * D + 2 * r));
                    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - m);
                    l += ml.y * f;
                    const float *v = slot + (size_t)r * D + lane * V;
                    if constexpr (V == 4) {
                        const float4 x = __ldcg(reinterpret_cast<const float4 *>(v));
                        acc[0] = fmaf(x.x, f, acc[0]);
                        acc[1] = fmaf(x.y, f, acc[1]);
                        acc[2] = fmaf(x.z, f, acc[2]);
                        acc[3] = fmaf(x.w, f, acc[3]);
                    } else {
                        const float2 x = __ldcg(reinterpret_cast<const float2 *>(v));
                        acc[0] = fmaf(x.x, f, acc[0]);
                        acc[1] = fmaf(x.y, f, acc[1]);
                    }
                }
                const int R = J.x.rt * kRpt + r, qi = R / a.group, row = J.x.row0 + qi;
                const int hq = J.head * a.group + R - qi * a.group;
                const float inv = m == -INFINITY ? 0.f : 1.f / l;
                uint16_t *out = a.k.out + (size_t)row * a.k.ldo + (size_t)hq * D + lane * V;
#pragma unroll
                for (int j = 0; j < V; j++) out[j] = __bfloat16_as_ushort(__float2bfloat16(acc[j] * inv));
                if (a.k.lse != nullptr && lane == 0)
                    a.k.lse[(size_t)row * a.k.heads_q + hq] =
                        m == -INFINITY ? -INFINITY : 0.6931471805599453f * (m + log2f(l));
            }
        }
        named_barrier(3, kSoftThreads);
        if (tid == 128 && atomicAdd(leave, 1u) == (unsigned)ctas - 1u) {
            // every CTA has arrived and has stopped polling
            *(volatile unsigned int *)arrive = 0u;
            *(volatile unsigned int *)leave = 0u;
        }
    }
    // nothing may still be in flight when TMEM is released and the CTA exits
    if (warp == 0 && lane == 0) {
        for (int it = max(0, it_issued - ns); it < it_issued; it++)
            mbar_wait(&full[it % ns], (uint32_t)(it / ns) & 1u, st, 0xa40u);
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

PerDevice g_sms(0), g_smem_max(0);

// Rows per tile: all rows of a head group if they fit 128, else even tiles of at most 128.
int rows_per_tile(int max_rows, int group) {
    const int rows = std::max(1, max_rows * group);  // at most kMaxTileRows
    const int tiles = (rows + 127) / 128;
    return ((rows + tiles - 1) / tiles + 15) / 16 * 16;
}

template <int D, int RW>
cudaError_t launch(const CUtensorMap &tm, AttnArgs a, int sms, int smem_max, cudaStream_t st) {
    static PerDevice smem_set(0);
    int ns = kMaxStages;
    while (ns > 2 && Smem(D, 2 * RW, ns).total + 1024u > (uint32_t)smem_max) ns--;
    a.ns = ns;
    const size_t smem = Smem(D, 2 * RW, ns).total + 1024;
    if (smem > (size_t)smem_max) return cudaErrorNotSupported;
    cudaError_t e = ensure_dynamic_smem(kv_attention_kernel<D, RW>, smem, smem_set);
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
    return cudaLaunchKernelEx(&cfg, kv_attention_kernel<D, RW>, tm, a);
}

template <int D>
cudaError_t launch_dim(const CUtensorMap &tm, const AttnArgs &a, int sms, int smem_max, cudaStream_t st) {
    switch (a.rpt) {
        case 16: return launch<D, 8>(tm, a, sms, smem_max, st);
        case 32: return launch<D, 16>(tm, a, sms, smem_max, st);
        case 48: return launch<D, 24>(tm, a, sms, smem_max, st);
        case 64: return launch<D, 32>(tm, a, sms, smem_max, st);
        case 80: return launch<D, 40>(tm, a, sms, smem_max, st);
        case 96: return launch<D, 48>(tm, a, sms, smem_max, st);
        case 112: return launch<D, 56>(tm, a, sms, smem_max, st);
        case 128: return launch<D, 64>(tm, a, sms, smem_max, st);
    }
    return cudaErrorNotSupported;
}

}  // namespace

cudaError_t set_wait_limit_kv_attention(uint64_t ns) { return set_wait_limit_here(ns); }

cudaError_t kv_attention_workspace_bytes(const KvView &kv, int max_rows, int heads_q, size_t *bytes) {
    int sms = 0;
    const cudaError_t e = device_attr(cudaDevAttrMultiProcessorCount, g_sms, &sms);
    if (e != cudaSuccess) return e;
    if ((int64_t)max_rows * (heads_q / kv.heads) > kMaxTileRows) return cudaErrorNotSupported;
    const size_t rpt = (size_t)rows_per_tile(max_rows, heads_q / kv.heads);
    *bytes = sizeof(StatusWord) + (size_t)2 * sms * (rpt * kv.dim + 2 * rpt) * sizeof(float);
    return cudaSuccess;
}

cudaError_t launch_kv_attention(const KvAttentionArgs &k, void *ws, cudaStream_t st) {
    cudaError_t e = get_encoder();
    if (e != cudaSuccess) return e;
    int sms = 0, smem_max = 0;
    if ((e = device_attr(cudaDevAttrMultiProcessorCount, g_sms, &sms)) != cudaSuccess) return e;
    if ((e = device_attr(cudaDevAttrMaxSharedMemoryPerBlockOptin, g_smem_max, &smem_max)) != cudaSuccess) return e;
    AttnArgs a;
    a.k = k;
    a.group = k.heads_q / k.kv.heads;
    a.rpt = rows_per_tile(k.max_rows, a.group);
    a.nrt = std::max(1, (k.max_rows * a.group + a.rpt - 1) / a.rpt);
    if ((int64_t)a.nrt * k.seqs > (1 << 30)) return cudaErrorNotSupported;
    a.scale2 = k.scale * 1.4426950408889634f;
    a.part = reinterpret_cast<float *>((char *)ws + sizeof(StatusWord));
    // the layer as a tensor of bytes [page][side, head, slot][value]
    const KvView &v = k.kv;
    CUtensorMap tm;
    cuuint64_t dims[3] = {(cuuint64_t)v.dim, (cuuint64_t)2 * v.heads * v.page, (cuuint64_t)v.n_pages};
    cuuint64_t strides[2] = {(cuuint64_t)v.dim, v.page_rec};
    cuuint32_t box[3] = {(cuuint32_t)v.dim, (cuuint32_t)v.page, 1};
    cuuint32_t es[3] = {1, 1, 1};
    const CUresult r = g_encode(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, v.base + (uint64_t)k.layer * v.layer_rec, dims,
                                strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                v.dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
    TraceScope trace_scope("kv_attention", st);
    return v.dim == 128 ? launch_dim<128>(tm, a, sms, smem_max, st) : launch_dim<64>(tm, a, sms, smem_max, st);
}

}  // namespace moe
