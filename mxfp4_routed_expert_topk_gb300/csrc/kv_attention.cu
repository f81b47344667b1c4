// Cache attention, the form for few rows (up to 16 per row tile: all query heads of a
// key/value head of one token, or of two or three drafted ones), and the choice between the forms.
//
// Tokens, not rows, lie along M: S^T = K Q^T (M = 128 tokens, N = rows) and O^T = V^T P^T
// (M = head_dim, N = rows, K = 128 tokens).  However few the rows, every MMA is full along M,
// and K and V are its A operand (V^T is V's tile read M-major).  The TMEM lane of a score is
// its token, so a thread has one token's scores and writes the rows' weights as one vector of
// its token (P^T is N-major); the maximum and sum of a row run across lanes.
//
// What bounds it is HBM for long sequences: one token for each of 64 sequences of up to 16384
// (8 heads of 128, 7 query heads each) takes 189 us at 1119 MB, 5.9 TB/s (87 % of a copy's rate).
// A tile takes about 2800 clocks from its scores to its output (TMEM read, two cross-lane
// reductions, a warpgroup barrier, the exponentials, the fences and the two MMA groups), twice
// what its 32 KB take from HBM.  So a CTA has three workers, each a softmax warpgroup with a
// warp that feeds it, and each worker has a share of its own: nothing is exchanged between
// them, and one's end of a unit overlaps with the others' tiles.  (Three warpgroups on one
// share, joined at each unit's end: 256 sequences of 128 tokens 84 us, so 44, both from cold
// caches.  Four such: 66 us in place of 62 for 96 sequences of 512.)  Short calls are bound by
// the start (6 us: launch, shares, the first loads) and by code that runs once: fetching it from
// cold caches takes 300 clocks per 8 instructions.
#include <algorithm>

#include "kv_attention.cuh"

namespace moe {
namespace {

// Rows of a row tile.  This form with 32 took 165 us for 4 rows in each of 24 sequences of 8192,
// where the rows form took 117.  With 7, 14 and 16 rows of heads of 128 this one takes 102, 106 and
// 107 us there, the rows form 107, 109 and 109; with 8 and 16 rows of heads of 64 53 and 54, so 54
// and 56.  96 sequences of 512: 14 rows of 128 56 and 67; only 16 rows of 64 37 and 35.
constexpr int kRows = 16;
// Workers of a CTA, a softmax warpgroup each.
constexpr int kWorkers = 3;
constexpr int kThreads = 32 * kFirstSoft + 128 * kWorkers;
constexpr int kStages = 2;    // tiles per worker: one under work, one on its way
constexpr uint32_t kTmemCols = 256;

struct FewSmem {
    uint32_t kv, q, p, scales, seg, split, rows, smax, ref, ab, lsum, nan, bars, misc, total;
    __host__ __device__ FewSmem(int dim) {
        uint32_t o = 0;
        kv = o;     o += (uint32_t)kWorkers * kStages * 2u * kTokens * dim;         // [worker][stage][keys, values]
        q = o;      o += (uint32_t)kWorkers * 2u * kRows * dim;                     // [worker][part][row]
        p = o;      o += (uint32_t)kWorkers * 2u * kRows * kTokens;                 // [worker][part][128][16]: weights
        scales = o; o += (uint32_t)kWorkers * kStages * 2u * kMaxSlots * 4u;        // [worker][stage][keys', values']
        rows = o;   o += (uint32_t)kWorkers * 2u * kRows * (uint32_t)sizeof(RowInfo);  // [worker][buffer]
        smax = o;   o += (uint32_t)kWorkers * 2u * 4u * kRows * 4u;                 // [worker][2][warp][row]
        ref = o;    o += (uint32_t)kWorkers * 4u * 2u * kRows * 4u;                 // [warp][query scales, references][row]
        ab = o;     o += (uint32_t)kWorkers * 4u * kRows * 8u;                      // [warp][row] (factors of the outputs)
        lsum = o;   o += (uint32_t)kWorkers * 4u * kRows * 4u;                      // [warp][row]
        nan = o;    o += (uint32_t)kWorkers * 2u * 4u * 4u;                         // [worker][2][warp] tokens with NaN values
        seg = o;    o += (uint32_t)kWorkers * 2u * (uint32_t)sizeof(Seg);           // [worker][buffer]
        split = o;  o += (uint32_t)kWorkers * 2u * (uint32_t)sizeof(Seg);           // units shared with other workers
        bars = o;   o += ((uint32_t)kWorkers * 16u + 1u) * 8u;
        o = (o + 15u) & ~15u;
        misc = o;   o += 512u;
        total = o;
    }
};

// A worker's barriers.
struct FewBars {
    uint64_t *b;
    __device__ uint64_t *k_full(int s) const { return b + s; }
    __device__ uint64_t *v_full(int s) const { return b + 2 + s; }
    __device__ uint64_t *empty(int s) const { return b + 4 + s; }      // the stage's keys and values are read
    // A segment's description and queries, by its parity: the next segment's may come before the
    // softmax has looked at this one's (a segment of one tile needs nothing of it until then).
    __device__ uint64_t *q_full(int s) const { return b + 6 + s; }
    __device__ uint64_t *seg_empty(int s) const { return b + 8 + s; }  // its description is read
    __device__ uint64_t *q_free() const { return b + 10; }             // its last scores are there
    __device__ uint64_t *s_full() const { return b + 11; }             // scores in TMEM
    __device__ uint64_t *p_ready() const { return b + 12; }            // weights written, scores read
    __device__ uint64_t *o_full() const { return b + 13; }             // outputs in TMEM
};

// Feeds one worker (a warp): walks its share, copies tiles, loads queries, whichever is possible.
template <int D, int P>
__device__ __forceinline__ void feed(const AttnArgs &a, const CUtensorMap *tm, unsigned char *smem, const FewSmem &F,
                                     int w, const FewBars &B, const Start &start, int *abort_flag) {
    constexpr uint32_t kTile = kTokens * D;
    const int lane = threadIdx.x & 31;
    const uint32_t elected = elect_one();
    unsigned char *kv = smem + F.kv + (uint32_t)w * (kStages * 2u * kTile);
    float *scales = reinterpret_cast<float *>(smem + F.scales) + w * kStages * 2 * kMaxSlots;
    Seg *ring = reinterpret_cast<Seg *>(smem + F.seg) + 2 * w;
    Walk W(a, start);
    Pages<P> pg;
    Watch eye = lane == 0 ? Watch{B.empty(0), kStages, 0, 1u}
                : lane == 1 ? Watch{B.q_free(), 1, 0, 1u}
                            : Watch{B.seg_empty(0), 2, 0, 1u};
    int issued = 0;
    uint64_t idle = 0;
    bool run = true;
#pragma unroll 1
    for (int seg = 0; run; seg++) {
        const Seg g = W.next();
        if (g.count > 0) {
            prefetch_queries(a, g);
            pg.start(a, g);
        }
        bool told = false;  // description and queries are out
        int t = 0;
#pragma unroll 1
        while (t < g.count || !told) {
            const uint32_t m = __ballot_sync(0xffffffffu, lane < 3 && eye.ready());
            if (t < g.count && (m & 1u) != 0u) {
                const int st = issued & (kStages - 1);
                unsigned char *dst = kv + (uint32_t)st * (2u * kTile);
                pg.template copy<D>(tm, dst, g.head * P, B.k_full(st), elected);
                pg.template copy<D>(tm, dst + kTile, (a.k.kv.heads + g.head) * P, B.v_full(st), elected);
                pg.copy_scales(a, g.head, scales + st * 2 * kMaxSlots, B.v_full(st));
                pg.next_tile();
                issued++;
                t++;
                if (lane == 0) eye.next();
            } else if (!told && (m & 6u) == 6u) {
                __syncwarp();  // (lanes 1 and 2 have seen the places free; a vote orders no memory)
                if (lane == 0) ring[seg & 1] = g;
                if (g.count > 0)
                    load_queries<D, kRows>(a, reinterpret_cast<RowInfo *>(smem + F.rows) + (2 * w + (seg & 1)) * kRows,
                                              smem + F.q + (uint32_t)w * (2u * kRows * D), g, 0, 1);
                __syncwarp();
                if (lane == 0) mbar_arrive(B.q_full(seg & 1));
                told = true;
                if (lane == 1 || lane == 2) eye.next();
            } else {
                if (!(run = !__any_sync(0xffffffffu, expired(idle, 0xa00u + w, abort_flag)))) break;
                continue;
            }
            idle = 0;
        }
        if (g.count == 0) break;
    }
    // nothing may be in flight when the CTA exits
    if (lane == 0) {
        for (int i = max(0, issued - kStages); i < issued; i++) {
            const uint32_t parity = (uint32_t)(i / kStages) & 1u;
            drain(B.k_full(i & (kStages - 1)), parity, abort_flag);
            drain(B.v_full(i & (kStages - 1)), parity, abort_flag);
        }
    }
    __syncwarp();
}

// Sum N rows (v[i] of every lane) over the warp's 32 lanes by halving: lane l ends with the sum
// of row l * N / 32, after N - 1 exchanges plus log2(32 / N).
template <int N>
__device__ __forceinline__ float reduce_rows(float (&v)[N], int lane) {
#pragma unroll
    for (int h = N / 2, mask = 16; h >= 1; h >>= 1, mask >>= 1) {
        const bool up = (lane & mask) != 0;
#pragma unroll
        for (int i = 0; i < h; i++) {
            const float send = up ? v[i] : v[i + h], keep = up ? v[i + h] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, mask);
        }
    }
    float r = v[0];
#pragma unroll
    for (int mask = 16 / N; mask >= 1; mask >>= 1) r += __shfl_xor_sync(0xffffffffu, r, mask);
    return r;
}

// Maximum over the warp's lanes, in all of them (NaN is passed over); half a shuffle's time.
__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_few_kernel(const __grid_constant__ CUtensorMap tm,
                                                                        const AttnArgs a) {
    constexpr int R = kRows;
    constexpr uint32_t kTile = kTokens * D;  // bytes of a K or V tile
    constexpr uint32_t kSwz = D == 128 ? kSwizzle128B : kSwizzle64B;
    constexpr uint32_t kGroup8 = 8 * D;      // bytes of 8 rows
    constexpr uint32_t kPBytes = R * kTokens;  // one part of one tile's weights
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = (unsigned char *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const FewSmem F(D);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + F.bars), *mma_done = bars + 16 * kWorkers;
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + F.misc);
    uint32_t *tmem_slot = misc;
    int *abort_flag = reinterpret_cast<int *>(misc + 1);
    int *go = reinterpret_cast<int *>(misc + 2);  // [worker]
    int64_t *sums = reinterpret_cast<int64_t *>(misc + 8);
    Start *start = reinterpret_cast<Start *>(misc + 56);  // [worker]
    static_assert(kThreads / 32 * 12 <= 48 * 4 && kWorkers * sizeof(Start) <= 72 * 4, "misc");
    StatusWord *st = a.k.st;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const Line line = cut_line<kThreads, kWorkers>(a, sums, start);
    if ((int)blockIdx.x >= line.workers) return;  // the whole CTA: nothing set up yet
    if (tid == 0) {
        for (int w = 0; w < kWorkers; w++) {
            const FewBars B{bars + 16 * w};
            for (int s = 0; s < kStages; s++) {
                mbar_init(B.k_full(s), 1);
                mbar_init(B.v_full(s), 1 + kTokens / a.k.kv.page);  // the expect-tx arrival, and each page's scales
                mbar_init(B.empty(s), 1);
            }
            mbar_init(B.q_full(0), 1);
            mbar_init(B.q_full(1), 1);
            mbar_init(B.q_free(), 1);
            mbar_init(B.seg_empty(0), 4);
            mbar_init(B.seg_empty(1), 4);
            mbar_init(B.s_full(), 1);
            mbar_init(B.p_ready(), 4);
            mbar_init(B.o_full(), 1);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tmem_o = tmem + 2 * kWorkers * R;

    if (warp < kFirstSoft && warp != 1) {
        const int w = warp == 0 ? 0 : warp - 1;
        const FewBars B{bars + 16 * w};
        switch (a.k.kv.page) {
            case 16: feed<D, 16>(a, &tm, smem, F, w, B, start[w], abort_flag); break;
            case 32: feed<D, 32>(a, &tm, smem, F, w, B, start[w], abort_flag); break;
            case 64: feed<D, 64>(a, &tm, smem, F, w, B, start[w], abort_flag); break;
            case 128: feed<D, 128>(a, &tm, smem, F, w, B, start[w], abort_flag); break;
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issue
        const uint32_t id_s = idesc_f8(128, 2 * R, false, false), id_o = idesc_f8(D, 2 * R, true, true);
        const uint64_t kd = smem_desc(smem_u32(smem + F.kv), 16, kGroup8, kSwz);
        const uint64_t vd = smem_desc(smem_u32(smem + F.kv) + kTile, kGroup8, kGroup8, kSwz);
        const uint64_t qd = smem_desc(smem_u32(smem + F.q), 16, kGroup8, kSwz);
        // weights: N-major without swizzle, 16 rows x 8 tokens (128 bytes) per core matrix,
        // 8-token groups 128 bytes and 16-row chunks 2 KB apart
        const uint64_t pd = smem_desc(smem_u32(smem + F.p), 128, kTokens * 16, kSwizzleNone);
        int ns[kWorkers], np[kWorkers], end[kWorkers], segs[kWorkers];  // scores / outputs issued; tiles and segments known
        uint32_t open = (1u << kWorkers) - 1u;                          // workers whose shares have not ended
#pragma unroll
        for (int w = 0; w < kWorkers; w++) ns[w] = np[w] = end[w] = segs[w] = 0;
        const uint32_t elected = elect_one();
        // Whichever is ready, of each worker: the outputs of tile np, then the scores of tile ns
        // (once the weights of the one before have been read, and with the segment's queries).
        // Lanes 4 w + 0 .. 3 look at one barrier each; a vote makes the outcome uniform, which keeps
        // the descriptors in uniform registers.  Each worker is looked at in its turn: with one vote
        // for all of them the first was 6 % ahead of the last at the end (64 x 1: 204 us, so 195).
        const FewBars mine{bars + 16 * min(lane >> 2, kWorkers - 1)};
        Watch eye = (lane & 3) == 0   ? Watch{mine.p_ready(), 1, 0, 0u}
                    : (lane & 3) == 1 ? Watch{mine.v_full(0), kStages, 0, 0u}
                    : (lane & 3) == 2 ? Watch{mine.k_full(0), kStages, 0, 0u}
                                      : Watch{mine.q_full(0), 2, 0, 0u};
        uint64_t idle = 0;  // since when nothing has been ready
#pragma unroll 1
        while (open != 0u) {
            bool any = false;
#pragma unroll
            for (int w = 0; w < kWorkers; w++) {
                const uint32_t m = __ballot_sync(0xffffffffu, (lane >> 2) == w && eye.ready()) >> (4 * w);
                const FewBars B{bars + 16 * w};
                const bool out = np[w] < ns[w] && (m & 3u) == 3u;
                __syncwarp();  // what one lane has seen holds for all (a vote orders no memory)
                if (out) {
                    tc_fence_after();
                    const int s = np[w] & (kStages - 1);
                    const uint64_t va = vd + (uint64_t)((uint32_t)(w * kStages + s) * (2u * kTile) >> 4);
                    const uint64_t pb = pd + (uint64_t)((uint32_t)w * (2u * kPBytes) >> 4);
#pragma unroll
                    for (int k = 0; k < kTokens / 32; k++)
                        tc_mma_f8(tmem_o + (uint32_t)(w * 2 * R), va + (uint64_t)(k * (32 * D) >> 4),
                                  pb + (uint64_t)(k * 32), id_o, k > 0 ? 1u : 0u, elected);
                    tc_commit_elected(B.empty(s), elected);
                    tc_commit_elected(B.o_full(), elected);
                    np[w]++;
                    if ((lane >> 2) == w && (lane & 3) < 2) eye.next();
                    any = true;
                }
                if (ns[w] == end[w] && (open >> w & 1u) != 0u && np[w] == ns[w] && (m & 8u) != 0u) {
                    // the next segment's queries are there
                    const volatile Seg *sg = reinterpret_cast<const volatile Seg *>(smem + F.seg) + 2 * w + (segs[w] & 1);
                    const int count = __shfl_sync(0xffffffffu, sg->count, 0);
                    end[w] += count;
                    segs[w]++;
                    if (__any_sync(0xffffffffu, count == 0)) open &= ~(1u << w);
                    if ((lane >> 2) == w && (lane & 3) == 3) eye.next();
                    any = true;
                }
                if (ns[w] < end[w] && ns[w] == np[w] && (m & 4u) != 0u) {
                    tc_fence_after();
                    const int s = ns[w] & (kStages - 1);
                    const uint64_t ka = kd + (uint64_t)((uint32_t)(w * kStages + s) * (2u * kTile) >> 4);
                    const uint64_t qa = qd + (uint64_t)((uint32_t)w * (2u * R * D) >> 4);
#pragma unroll
                    for (int k = 0; k < D / 32; k++)
                        tc_mma_f8(tmem + (uint32_t)(w * 2 * R), ka + (uint64_t)(2 * k), qa + (uint64_t)(2 * k), id_s,
                                  k > 0 ? 1u : 0u, elected);
                    tc_commit_elected(B.s_full(), elected);
                    if (++ns[w] == end[w]) tc_commit_elected(B.q_free(), elected);
                    if ((lane >> 2) == w && (lane & 3) == 2) eye.next();
                    any = true;
                }
            }
            if (any) {
                idle = 0;
            } else if (__any_sync(0xffffffffu, expired(idle, 0xb00u, abort_flag))) {
                break;
            }
        }
        // every MMA has finished before TMEM is released
        if (elect_one()) tc_commit(mma_done);
        __syncwarp();
        if (lane == 0) drain(mma_done, 0u, abort_flag);
        __syncwarp();
    } else {
        // -------------------------------------------------------- softmax
        const int sw = warp - kFirstSoft, wg = sw >> 2, ew = sw & 3, wtid = tid & 127;
        const int worker = (int)(blockIdx.x + wg * gridDim.x), bar = 1 + wg;
        const FewBars B{bars + 16 * wg};
        const int tok = wtid;                           // token of the tile (TMEM lane)
        const uint32_t lanes = (uint32_t)(32 * ew) << 16;
        const int row = lane >> 1;                      // the row whose maximum and sum this lane holds
        float *smax = reinterpret_cast<float *>(smem + F.smax) + wg * 8 * R;
        float *qscale = reinterpret_cast<float *>(smem + F.ref) + sw * 2 * R, *ref = qscale + R;
        float2 *ab = reinterpret_cast<float2 *>(smem + F.ab) + sw * R;
        float *lsum = reinterpret_cast<float *>(smem + F.lsum) + wg * 4 * R;
        uint32_t *nan = reinterpret_cast<uint32_t *>(smem + F.nan) + wg * 8;
        Seg *split = reinterpret_cast<Seg *>(smem + F.split) + 2 * wg;
        const int page_shift = 31 - __clz(a.k.kv.page);
        const int dcol = D == 128 ? tok : 16 * ew + lane;  // value of the head this lane holds
        const bool dlive = D == 128 || lane < 16;          // (64-wide heads fill 16 lanes of each warp)
        const size_t slot_floats = (size_t)R * D + 2 * R;
        float o[R];
        int mine = 0;    // tiles of earlier segments
        int shared = 0;  // units shared with other workers

#pragma unroll 1
        for (int seg = 0;; seg++) {
            // (one thread decides for all whether to go on: after an abort the description may be missing)
            if (wtid == 0) go[wg] = lane_wait(B.q_full(seg & 1), (uint32_t)(seg >> 1) & 1u, 0xc30u, abort_flag) ? 1 : 0;
            named_barrier(bar, 128);
            if (*(volatile int *)(go + wg) == 0) break;
            soft_wait(B.q_full(seg & 1), (uint32_t)(seg >> 1) & 1u, 0xc31u, abort_flag);
            const Seg *sg = reinterpret_cast<const Seg *>(smem + F.seg) + 2 * wg + (seg & 1);
            const RowInfo *rows = reinterpret_cast<const RowInfo *>(smem + F.rows) + (2 * wg + (seg & 1)) * R;
            const int count = sg->count, tile0 = sg->tile0, see_all = sg->see_all, see_max = sg->see_max;
            if (count == 0) break;
            qscale[row] = rows[row].qs;
            __syncwarp();
            float m_run = -INFINITY, l_run = 0.f;
#pragma unroll
            for (int i = 0; i < R; i++) o[i] = 0.f;

#pragma unroll 1
            for (int t = 0;; t++) {
                if (t > 0) {  // add O^T of the tile before to the running output
                    soft_wait(B.o_full(), (uint32_t)(mine - 1) & 1u, 0xc20u, abort_flag);
                    tc_fence_after();
                    // (the first parts' product, then the second parts')
                    float y[2 * R];
#pragma unroll
                    for (int j = 0; j < 2 * R; j += 8) tmem_ld8(tmem_o + (uint32_t)(wg * 2 * R + j) + lanes, y + j);
                    tmem_ld_wait(y);
#pragma unroll
                    for (int j = 0; j < R; j++) {
                        const float2 k = ab[j];
                        o[j] = fmaf(y[j] + y[R + j], k.y, o[j] * k.x);
                    }
                    // NaN values that only some rows see, back into those rows' outputs
                    const uint32_t *words = nan + ((mine - 1) & 1) * 4;
                    const uint4 nm = *reinterpret_cast<const uint4 *>(words);
                    if ((nm.x | nm.y | nm.z | nm.w) != 0u) {
#pragma unroll 1
                        for (int w = 0; w < 4; w++) {
                            for (uint32_t word = words[w]; word != 0u; word &= word - 1u) {
                                const int tn = (tile0 + t - 1) * kTokens + 32 * w + __ffs((int)word) - 1;
                                const uint8_t *code = value_codes(a, sg->b, sg->head, tn);
                                if (!dlive || code == nullptr || (code[dcol] & 0x7fu) != 0x7fu) continue;
#pragma unroll
                                for (int i = 0; i < R; i++)
                                    if (tn <= rows[i].pos) o[i] = kNan;
                            }
                        }
                    }
                }
                if (t >= count) break;
                const int stage = mine & (kStages - 1);
                const int tk = (tile0 + t) * kTokens + tok;
                soft_wait(B.s_full(), (uint32_t)mine & 1u, 0xc00u, abort_flag);
                tc_fence_after();
                // scores with the queries' first parts, then with their second parts
                float x[R], x2[R];
#pragma unroll
                for (int i = 0; i < R; i += 8) {
                    tmem_ld8(tmem + (uint32_t)(wg * 2 * R + i) + lanes, x + i);
                    tmem_ld8(tmem + (uint32_t)(wg * 2 * R + R + i) + lanes, x2 + i);
                }
                soft_wait(B.v_full(stage), (uint32_t)(mine / kStages) & 1u, 0xc10u, abort_flag);
                const float *sc = reinterpret_cast<const float *>(smem + F.scales) + (wg * kStages + stage) * 2 * kMaxSlots;
                const float ks = sc[tok >> page_shift] * a.scale2;
                const float sv = sc[kMaxSlots + (tok >> page_shift)];
                const float vs = fabsf(sv) < INFINITY ? sv : kNan;
                const float lv = fmaxf(lg2(fabsf(vs)), kLowScale);  // (NaN: the output is NaN at any reference)
                const bool special = (tile0 + t + 1) * kTokens > see_all;
                tmem_ld_wait(x);
                tmem_ld_wait(x2);
#pragma unroll
                for (int i = 0; i < R; i++) x[i] = (x[i] + x2[i]) * ks;
                uint32_t word = 0;
                if (special) {
#pragma unroll
                    for (int i = 0; i < R; i++) x[i] = tk <= rows[i].pos ? x[i] : -INFINITY;
                    unsigned char *v = smem + F.kv + (uint32_t)(wg * kStages + stage) * (2u * kTile) + kTile;
                    const bool bad = clean_values<D>(v, tok, tk, see_all, see_max);
                    word = __ballot_sync(0xffffffffu, bad);
                }
                if (lane == 0) nan[(mine & 1) * 4 + ew] = word;
                // the tile's maximum of each row: over the warp's tokens, then over the four warps
                float *mx = smax + (mine & 1) * 4 * R;
#pragma unroll
                for (int i = 0; i < R; i += 4) {
                    const float4 k = *reinterpret_cast<const float4 *>(qscale + i);
                    const float4 v = make_float4(warp_max(fmaf(x[i], k.x, lv)), warp_max(fmaf(x[i + 1], k.y, lv)),
                                                 warp_max(fmaf(x[i + 2], k.z, lv)), warp_max(fmaf(x[i + 3], k.w, lv)));
                    if (lane == 0) *reinterpret_cast<float4 *>(mx + ew * R + i) = v;
                }
                named_barrier(bar, 128);
                const float mt = fmaxf(fmaxf(mx[row], mx[R + row]), fmaxf(mx[2 * R + row], mx[3 * R + row])) - kTop;
                const float m = fmaxf(m_run, mt);
                const float f_old = m_run == -INFINITY ? 0.f : ex2_low(m_run - m),
                            f_new = mt == -INFINITY ? 0.f : ex2_low(mt - m);
                m_run = m;
                ref[row] = mt == -INFINITY ? 0.f : mt;
                ab[row] = make_float2(f_old, f_new);
                __syncwarp();
                uint8_t *pw = smem + F.p + (uint32_t)wg * (2u * kPBytes) + (uint32_t)tok * 16u;
                float p[R];
                uint32_t h4[4], l4[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    float h[4], l[4];
                    const float4 q4 = *reinterpret_cast<const float4 *>(qscale + 4 * j);
                    const float4 r4 = *reinterpret_cast<const float4 *>(ref + 4 * j);
                    const float qk[4] = {q4.x, q4.y, q4.z, q4.w}, rk[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const int r = 4 * j + k;
                        p[r] = ex2(fmaf(x[r], qk[k], -rk[k]));
                        float w = p[r] * vs;
                        if (special) w = x[r] == -INFINITY ? 0.f : w;
                        h[k] = part_hi(w);
                        l[k] = w - h[k];
                    }
                    h4[j] = e4m3x4_rn(h[0], h[1], h[2], h[3]);
                    l4[j] = e4m3x4_rn(l[0], l[1], l[2], l[3]);
                }
                *reinterpret_cast<uint4 *>(pw) = make_uint4(h4[0], h4[1], h4[2], h4[3]);
                *reinterpret_cast<uint4 *>(pw + kPBytes) = make_uint4(l4[0], l4[1], l4[2], l4[3]);
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(B.p_ready());
                l_run = l_run * f_old + reduce_rows<R>(p, lane) * f_new;
                mine++;
            }
            // the four warps' sums, then the rows' results (every warp has every row's reference)
            lsum[ew * R + row] = l_run;
            named_barrier(bar, 128);
            const float l = (lsum[row] + lsum[R + row]) + (lsum[2 * R + row] + lsum[3 * R + row]);
            const bool part_of = count < sg->nt;
            float *part = part_of ? a.part + (size_t)(2 * worker + (tile0 == 0 ? 1 : 0)) * slot_floats : nullptr;
            // (a row that saw nothing is told by its sum; NaN stays)
            ab[row].y = part_of ? 1.f : l == 0.f ? 0.f : 1.f / l;
            const bool live = *(volatile int *)abort_flag == 0;
            if (ew == 0 && (lane & 1) == 0 && rows[row].row >= 0 && live) {  // one lane per row
                if (part_of)
                    *reinterpret_cast<float2 *>(part + (size_t)R * D + 2 * row) = make_float2(m_run, l);
                else if (a.k.lse != nullptr)
                    a.k.lse[(size_t)rows[row].row * a.k.heads_q + rows[row].head] =
                        l == 0.f ? -INFINITY : kLn2 * (m_run + log2f(l));
            }
            __syncwarp();
            if (dlive && live) {
#pragma unroll
                for (int i = 0; i < R; i++) {
                    const RowInfo ri = rows[i];
                    if (ri.row < 0) continue;
                    const float y = o[i] * ab[i].y;
                    if (part_of)
                        part[(size_t)i * D + dcol] = y;
                    else
                        a.k.out[(size_t)ri.row * a.k.ldo + (size_t)ri.head * D + dcol] =
                            __bfloat16_as_ushort(__float2bfloat16(y));
                }
            }
            if (part_of) {
                if (wtid == 0) split[shared] = *sg;
                shared++;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(B.seg_empty(seg & 1));
        }
        named_barrier(bar, 128);  // the list of shared units is complete
        if (worker < line.workers) join_role<D, 128>(a, line, worker, split, shared, wtid, bar, abort_flag);
    }
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && *abort_flag != 0) set_status(st, MOE_ERR_TIMEOUT, (unsigned)*abort_flag);
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

PerDevice g_sms(0), g_smem_max(0);

// Rows per row tile: all rows of a head group if they fit 128, else even tiles of at most 128.
int rows_per_tile(int max_rows, int group) {
    const int rows = std::max(1, max_rows * group);  // at most 2^24
    const int tiles = (rows + 127) / 128;
    return ((rows + tiles - 1) / tiles + 15) / 16 * 16;
}

template <int D>
cudaError_t launch_few(const CUtensorMap &tm, AttnArgs a, int sms, int smem_max, cudaStream_t st) {
    static PerDevice smem_set(0);
    a.over = 2;  // (1 to 4 measure alike)
    const size_t smem = FewSmem(D).total + 1024;
    if (smem > (size_t)smem_max) return cudaErrorNotSupported;
    cudaError_t e = ensure_dynamic_smem(kv_attention_few_kernel<D>, smem, smem_set);
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
    return cudaLaunchKernelEx(&cfg, kv_attention_few_kernel<D>, tm, a);
}

}  // namespace

cudaError_t set_wait_limit_kv_attention(uint64_t ns) {
    const cudaError_t e = set_wait_limit_here(ns);
    return e != cudaSuccess ? e : set_wait_limit_kv_attention_rows(ns);
}

cudaError_t kv_attention_workspace_bytes(const KvView &kv, int max_rows, int heads_q, size_t *bytes) {
    int sms = 0;
    const cudaError_t e = device_attr(cudaDevAttrMultiProcessorCount, g_sms, &sms);
    if (e != cudaSuccess) return e;
    // two slots per worker, the larger need of the two forms; a size serves fewer rows too, whose
    // tiles may be larger (17 x 8 rows are two tiles of 80, 16 x 8 are one of 128)
    const int group = heads_q / kv.heads;
    const size_t rows = std::max(max_rows * group > 128 ? 128 : rows_per_tile(max_rows, group), kWorkers * kRows);
    *bytes = sizeof(StatusWord) + (size_t)2 * sms * rows * (kv.dim + 2) * sizeof(float);
    return cudaSuccess;
}

cudaError_t launch_kv_attention(const KvAttentionArgs &k, void *ws, cudaStream_t st) {
    cudaError_t e = get_encoder();
    if (e != cudaSuccess) return e;
    int sms = 0, smem_max = 0;
    if ((e = device_attr(cudaDevAttrMultiProcessorCount, g_sms, &sms)) != cudaSuccess) return e;
    if ((e = device_attr(cudaDevAttrMaxSharedMemoryPerBlockOptin, g_smem_max, &smem_max)) != cudaSuccess) return e;
    AttnArgs a = {};
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
    if (a.rpt > kRows) return launch_attention_rows(tm, a, sms, smem_max, st);
    return v.dim == 128 ? launch_few<128>(tm, a, sms, smem_max, st) : launch_few<64>(tm, a, sms, smem_max, st);
}

}  // namespace moe
