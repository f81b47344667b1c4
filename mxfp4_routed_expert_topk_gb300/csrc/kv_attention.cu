// Cache attention, the form for few rows (up to 32 per row tile: all query heads of a
// key/value head of one token, or of a few drafted ones), and the choice between the forms.
//
// Tokens, not rows, lie along M: S^T = K Q^T (M = 128 tokens, N = rows) and O^T = V^T P^T
// (M = head_dim, N = rows, K = 128 tokens).  However few the rows, every MMA is full along M,
// and K and V are its A operand (V^T is V's tile read M-major).  The TMEM lane of a score is
// its token, so a thread has one token's scores and writes the rows' weights as one vector of
// its token (P^T is N-major); the maximum and sum of a row run across lanes, by halving
// exchanges that leave each lane one row.
//
// What bounds it is the time one tile takes from its scores to its output (about 2800 clocks:
// TMEM read, two cross-lane reductions, a warpgroup barrier, the exponentials, the fences and
// the two MMA groups), twice what the tile's 32 KB take from HBM.  So three warpgroups take
// tiles in turn, each with its own running maximum, sum and output, joined in shared memory at
// the segment's end; keys and values have rings of their own, as a key stage is free as soon
// as the scores are there, while a value stage waits for the weights.
#include <algorithm>

#include "kv_attention.cuh"

namespace moe {
namespace {

constexpr int kBarAll = 7;  // named barrier of all softmax threads (warpgroup w: 1 + w)
// Softmax warpgroups.  Four (for 16 rows; 32 take more registers than that leaves) were slower:
// 96 sequences of 512 tokens 66 us in place of 62, one of 300 tokens 23 in place of 21 (cold).
constexpr int kGroups = 3;

struct FewSmem {
    CommonSmem c;
    uint32_t p, smax, ref, ab, lsum, mrow, nan, total;
    __host__ __device__ FewSmem(int dim, int r, int nk, int nv) : c(dim, r, nk, nv) {
        uint32_t o = (c.total + 127u) & ~127u;
        p = o;     o += (uint32_t)kGroups * 2u * r * kTokens;       // [group][part][r / 16][128][16]
        smax = o;  o += (uint32_t)kGroups * 2u * 4u * r * 4u;       // [group][2][warp][r]
        ref = o;   o += (uint32_t)kGroups * 4u * r * 8u;            // [warp][r] (query scale, reference)
        ab = o;    o += (uint32_t)kGroups * 4u * r * 8u;            // [warp][r] (factor of the old output, of the new)
        lsum = o;  o += (uint32_t)kGroups * 4u * r * 4u;            // [warp][r]
        mrow = o;  o += (uint32_t)kGroups * r * 4u;                 // [group][r]
        nan = o;   o += (uint32_t)kGroups * 4u * 4u;                // [group][warp] tokens whose values hold partial NaN
        total = o;
    }
};

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

template <int D, int R>
__global__ void __launch_bounds__(32 * kFirstSoft + 128 * kGroups, 1)
    kv_attention_few_kernel(const __grid_constant__ CUtensorMap tm, const AttnArgs a) {
    constexpr int kSoft = 128 * kGroups, kThreads = 32 * kFirstSoft + kSoft;
    constexpr uint32_t kTile = kTokens * D;  // bytes of a K or V tile
    constexpr uint32_t kSwz = D == 128 ? kSwizzle128B : kSwizzle64B;
    constexpr uint32_t kGroup8 = 8 * D;      // bytes of 8 rows
    constexpr uint32_t kTmemCols = 4 * kGroups * R <= 256 ? 256 : 512;
    constexpr uint32_t kPBytes = R * kTokens;  // one part of one tile's weights
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = (unsigned char *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const FewSmem F(D, R, a.nk, a.nv);
    const CommonSmem &L = F.c;
    const Bars B{reinterpret_cast<uint64_t *>(smem + L.bars)};
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + L.misc);
    uint32_t *tmem_slot = misc;
    int *abort_flag = reinterpret_cast<int *>(misc + 1);
    int *go = reinterpret_cast<int *>(misc + 2);
    int64_t *plan = reinterpret_cast<int64_t *>(misc + 8);
    StatusWord *st = a.k.st;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const Share S = cut_shares<kThreads>(a, plan);
    if ((int)blockIdx.x >= S.ctas) return;  // the whole CTA: nothing set up yet
    if (tid == 0) {
        for (int s = 0; s < a.nk; s++) {
            mbar_init(B.k_full(s), 1);
            mbar_init(B.k_empty(s), 1);
        }
        for (int s = 0; s < a.nv; s++) {
            mbar_init(B.v_full(s), 1 + kTokens / a.k.kv.page);  // the expect-tx arrival, and each page's scales
            mbar_init(B.v_empty(s), 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(B.q_full(b), 1);
            mbar_init(B.q_empty(b), 4 * kGroups);
        }
        for (int w = 0; w < kGroups; w++) {
            mbar_init(B.s_full(w), 1);
            mbar_init(B.p_ready(w), 4);
            mbar_init(B.o_full(w), 1);
        }
        for (int b = 0; b < kSegs; b++) {
            mbar_init(B.seg_full(b), 1);
            mbar_init(B.seg_empty(b), 2 + kSoft / 32);  // the copying warps, and the softmax
        }
        mbar_init(B.mma_done(), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tmem_o = tmem + 2 * kGroups * R;

    if (warp == 0) {
        copy_role<D, 0>(a, &tm, smem, L, B, abort_flag);
    } else if (warp == 2) {
        copy_role<D, 1>(a, &tm, smem, L, B, abort_flag);
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issue
        const uint32_t id_s = idesc_f8(128, 2 * R, false, false), id_o = idesc_f8(D, 2 * R, true, true);
        const uint64_t kd = smem_desc(smem_u32(smem + L.k), 16, kGroup8, kSwz);
        const uint64_t vd = smem_desc(smem_u32(smem + L.v), kGroup8, kGroup8, kSwz);
        const uint64_t qd = smem_desc(smem_u32(smem + L.q), 16, kGroup8, kSwz);
        // weights: N-major without swizzle, 16 rows x 8 tokens (128 bytes) per core matrix,
        // 8-token groups 128 bytes and 16-row chunks 2 KB apart
        const uint64_t pd = smem_desc(smem_u32(smem + F.p), 128, kTokens * 16, kSwizzleNone);
        int ks = 0, vs = 0;  // stages
        int ns = 0, np = 0, ws = 0, wp = 0;  // scores / outputs issued, and their warpgroups
        int seg = 0, seg_end = 0, qb = 0;
        bool last = false;                   // seg_end is the share's end
        const uint32_t elected = elect_one();
        // Whichever is ready: the outputs of tile np, the scores of tile ns (a warpgroup's next
        // scores once its last weights have been read, and only with the segment's queries).
        // Lanes 0 to 3 look at one barrier each; a vote makes the outcome uniform, which keeps
        // the descriptors in uniform registers.
        Watch eye = lane == 0   ? Watch{B.p_ready(0), kGroups, 0, 0u}
                    : lane == 1 ? Watch{B.v_full(0), a.nv, 0, 0u}
                    : lane == 2 ? Watch{B.k_full(0), a.nk, 0, 0u}
                                : Watch{B.q_full(0), 2, 0, 0u};
        uint64_t idle = 0;  // since when nothing has been ready
        while (!(last && np == seg_end)) {
            const uint32_t m = __ballot_sync(0xffffffffu, lane < 4 && eye.ready());
            const bool out = np < ns && (m & 3u) == 3u;
            if (ns == seg_end && !last && (m & 8u) != 0u) {  // the next segment's queries are there
                const volatile Seg *sg = reinterpret_cast<const volatile Seg *>(smem + L.seg) + seg % kSegs;
                const int count = __shfl_sync(0xffffffffu, sg->count, 0);
                qb = seg & 1;
                seg_end += count;
                last = __any_sync(0xffffffffu, count == 0);
                seg++;
                if (lane == 3) eye.next();
            }
            const bool scores = ns < seg_end && ns < np + kGroups && (m & 4u) != 0u;
            if (!out && !scores) {
                if (__any_sync(0xffffffffu, expired(idle, 0xb00u, abort_flag))) break;
                continue;
            }
            idle = 0;
            tc_fence_after();
            if (out) {
                const uint64_t va = vd + (uint64_t)((uint32_t)vs * kTile >> 4);
                const uint64_t pb = pd + (uint64_t)((uint32_t)wp * (2u * kPBytes) >> 4);
#pragma unroll
                for (int k = 0; k < kTokens / 32; k++)
                    tc_mma_f8(tmem_o + (uint32_t)(wp * 2 * R), va + (uint64_t)(k * (32 * D) >> 4), pb + (uint64_t)(k * 32),
                              id_o, k > 0 ? 1u : 0u, elected);
                tc_commit_elected(B.v_empty(vs), elected);
                tc_commit_elected(B.o_full(wp), elected);
                if (++vs == a.nv) vs = 0;
                if (++wp == kGroups) wp = 0;
                np++;
                if (lane < 2) eye.next();
            }
            if (scores) {
                const uint64_t ka = kd + (uint64_t)((uint32_t)ks * kTile >> 4);
                const uint64_t qa = qd + (uint64_t)((uint32_t)qb * (2u * R * D) >> 4);
#pragma unroll
                for (int k = 0; k < D / 32; k++)
                    tc_mma_f8(tmem + (uint32_t)(ws * 2 * R), ka + (uint64_t)(2 * k), qa + (uint64_t)(2 * k), id_s,
                              k > 0 ? 1u : 0u, elected);
                tc_commit_elected(B.k_empty(ks), elected);
                tc_commit_elected(B.s_full(ws), elected);
                if (++ks == a.nk) ks = 0;
                if (++ws == kGroups) ws = 0;
                ns++;
                if (lane == 2) eye.next();
            }
        }
        // every MMA has finished before TMEM is released
        if (elect_one()) tc_commit(B.mma_done());
        __syncwarp();
        if (lane == 0) drain(B.mma_done(), 0u, abort_flag);
        __syncwarp();
    } else if (warp < kFirstSoft) {
        segment_query_role<D, R>(a, smem, L, B, S, plan, abort_flag);
    } else {
        // -------------------------------------------------------- softmax
        const int sw = warp - kFirstSoft, wg = sw >> 2, ew = sw & 3, stid = tid - 32 * kFirstSoft;
        const int tok = 32 * ew + lane;                 // token of the tile (TMEM lane)
        const uint32_t lanes = (uint32_t)(32 * ew) << 16;
        const int row = lane * R >> 5;                  // the row whose maximum and sum this lane holds
        float *smax = reinterpret_cast<float *>(smem + F.smax) + wg * 8 * R;
        float2 *ref = reinterpret_cast<float2 *>(smem + F.ref) + sw * R;
        float2 *ab = reinterpret_cast<float2 *>(smem + F.ab) + sw * R;
        float *lsum = reinterpret_cast<float *>(smem + F.lsum), *mrow = reinterpret_cast<float *>(smem + F.mrow);
        uint32_t *nan = reinterpret_cast<uint32_t *>(smem + F.nan) + wg * 4;
        float *merge = reinterpret_cast<float *>(smem + F.p);  // [R][D]: the weights are done with by then
        const float *scales = reinterpret_cast<const float *>(smem + L.scales);
        const int page_shift = 31 - __clz(a.k.kv.page);
        const int dcol = D == 128 ? tok : 16 * ew + lane;  // value of the head this lane holds
        const bool dlive = D == 128 || lane < 16;          // (64-wide heads fill 16 lanes of each warp)
        const size_t slot_floats = (size_t)R * D + 2 * R;
        float o[R];
        int done = 0, mine = 0;  // tiles of earlier segments; tiles this warpgroup has taken
        int shared = 0;          // units shared with other CTAs
        // the first segment's data is there (one thread decides for all: see below)
        if (stid == 0) *go = lane_wait(B.q_full(0), 0u, 0xc30u, abort_flag) ? 1 : 0;
        named_barrier(kBarAll, kSoft);

#pragma unroll 1
        for (int seg = 0;; seg++) {
            // after an abort the segment's description may be missing: all leave together
            if (*(volatile int *)go == 0) break;
            const int buf = seg & 1;
            soft_wait(B.q_full(buf), (uint32_t)(seg >> 1) & 1u, 0xc31u, abort_flag);
            const Seg *sg = reinterpret_cast<const Seg *>(smem + L.seg) + seg % kSegs;
            const RowInfo *rows = reinterpret_cast<const RowInfo *>(smem + L.rows) + buf * R;
            const int count = sg->count, tile0 = sg->tile0, see_all = sg->see_all, see_max = sg->see_max;
            if (count == 0) break;
            const float qs = rows[row].qs;
            float m_run = -INFINITY, l_run = 0.f;
#pragma unroll
            for (int i = 0; i < R; i++) o[i] = 0.f;
            bool pending = false;
            int joined = 0;             // tile whose output is outstanding

            // Add O^T of the outstanding tile to the running output.
            auto join_tile = [&]() {
                soft_wait(B.o_full(wg), (uint32_t)(mine - 1) & 1u, 0xc20u + wg, abort_flag);
                tc_fence_after();
                // (16 rows at a time: the first parts' product, then the second parts')
#pragma unroll
                for (int i = 0; i < R; i += 16) {
                    float y[32];
#pragma unroll
                    for (int j = 0; j < 16; j += 8) {
                        tmem_ld8(tmem_o + (uint32_t)(wg * 2 * R + i + j) + lanes, y + j);
                        tmem_ld8(tmem_o + (uint32_t)(wg * 2 * R + R + i + j) + lanes, y + 16 + j);
                    }
                    tmem_ld_wait(y);
#pragma unroll
                    for (int j = 0; j < 16; j++) {
                        const float2 k = ab[i + j];
                        o[i + j] = fmaf(y[j] + y[16 + j], k.y, o[i + j] * k.x);
                    }
                }
                // NaN values that only some rows see, back into those rows' outputs
                const uint4 nm = *reinterpret_cast<const uint4 *>(nan);
                if ((nm.x | nm.y | nm.z | nm.w) != 0u) {
#pragma unroll 1
                    for (int w = 0; w < 4; w++) {
                        for (uint32_t word = nan[w]; word != 0u; word &= word - 1u) {
                            const int tn = joined * kTokens + 32 * w + __ffs((int)word) - 1;
                            const uint8_t *code = value_codes(a, sg->b, sg->head, tn);
                            if (!dlive || code == nullptr || (code[dcol] & 0x7fu) != 0x7fu) continue;
#pragma unroll
                            for (int i = 0; i < R; i++)
                                if (tn <= rows[i].pos) o[i] = kNan;
                        }
                    }
                }
                pending = false;
            };

            for (int t = (wg - done % kGroups + kGroups) % kGroups;; t += kGroups) {
                if (pending) join_tile();
                if (t >= count) break;
                const int u = done + t;              // tile of the share
                const int vs_ = u % a.nv;
                const int tk = (tile0 + t) * kTokens + tok;
                soft_wait(B.s_full(wg), (uint32_t)mine & 1u, 0xc00u + wg, abort_flag);
                tc_fence_after();
                // scores with the queries' first parts, then with their second parts
                float x[R], x2[R];
#pragma unroll
                for (int i = 0; i < R; i += 8) {
                    tmem_ld8(tmem + (uint32_t)(wg * 2 * R + i) + lanes, x + i);
                    tmem_ld8(tmem + (uint32_t)(wg * 2 * R + R + i) + lanes, x2 + i);
                }
                soft_wait(B.v_full(vs_), (uint32_t)(u / a.nv) & 1u, 0xc10u + vs_, abort_flag);
                const float *sc = scales + vs_ * 2 * kMaxSlots;
                const float ks = sc[tok >> page_shift] * a.scale2;
                // value scales relative to the tile's largest (finite) one
                float vone = 0.f;
                for (int j = 0; j < (kTokens >> page_shift); j++) {
                    const float v = sc[kMaxSlots + j];
                    vone = v < INFINITY ? fmaxf(vone, v) : vone;
                }
                vone = vone > 0.f ? vone : 1.f;
                const float vs = sc[kMaxSlots + (tok >> page_shift)];
                float c = vs < INFINITY ? 256.f * __fdividef(vs, vone) : kNan;
                if (tk >= see_max) c = 0.f;
                const bool special = (tile0 + t + 1) * kTokens > see_all;
                tmem_ld_wait(x);
                tmem_ld_wait(x2);
#pragma unroll
                for (int i = 0; i < R; i++) x[i] = (x[i] + x2[i]) * ks;
                uint32_t word = 0;
                if (special) {
#pragma unroll
                    for (int i = 0; i < R; i++) x[i] = tk <= rows[i].pos ? x[i] : -INFINITY;
                    const bool bad = clean_values<D>(smem + L.v + (uint32_t)vs_ * kTile, tok, tk, see_all, see_max);
                    word = __ballot_sync(0xffffffffu, bad);
                }
                if (lane == 0) nan[ew] = word;
                // the tile's maximum of each row: over the warp's tokens, then over the four warps
                float *mx = smax + (mine & 1) * 4 * R;
#pragma unroll
                for (int i = 0; i < R; i += 4) {
                    const float4 v = make_float4(warp_max(x[i]), warp_max(x[i + 1]), warp_max(x[i + 2]), warp_max(x[i + 3]));
                    if (lane == 0) *reinterpret_cast<float4 *>(mx + ew * R + i) = v;
                }
                named_barrier(1 + wg, 128);
                const float mt = fmaxf(fmaxf(mx[row], mx[R + row]), fmaxf(mx[2 * R + row], mx[3 * R + row])) * qs;
                const float m = fmaxf(m_run, mt);
                const float f_old = m_run == -INFINITY ? 0.f : ex2(m_run - m), f_new = mt == -INFINITY ? 0.f : ex2(mt - m);
                m_run = m;
                ref[row] = make_float2(qs, mt == -INFINITY ? 0.f : mt);
                ab[row] = make_float2(f_old, f_new * (vone * (1.f / 256.f)));
                __syncwarp();
                uint8_t *pw = smem + F.p + (uint32_t)wg * (2u * kPBytes) + (uint32_t)tok * 16u;
                float p[R];
#pragma unroll
                for (int i = 0; i < R; i += 16) {
                    uint32_t h4[4], l4[4];
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        float h[4], l[4];
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const int r = i + 4 * j + k;
                            const float2 rq = ref[r];
                            p[r] = ex2(fmaf(x[r], rq.x, -rq.y));
                            float w = p[r] * c;
                            if (special) w = x[r] == -INFINITY ? 0.f : w;
                            h[k] = part_hi(w);
                            l[k] = w - h[k];
                        }
                        h4[j] = e4m3x4_rn(h[0], h[1], h[2], h[3]);
                        l4[j] = e4m3x4_rn(l[0], l[1], l[2], l[3]);
                    }
                    uint8_t *d = pw + (uint32_t)(i >> 4) * (kTokens * 16u);
                    *reinterpret_cast<uint4 *>(d) = make_uint4(h4[0], h4[1], h4[2], h4[3]);
                    *reinterpret_cast<uint4 *>(d + kPBytes) = make_uint4(l4[0], l4[1], l4[2], l4[3]);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(B.p_ready(wg));
                l_run = l_run * f_old + reduce_rows<R>(p, lane) * f_new;
                mine++;
                pending = true;
                joined = tile0 + t;
            }
            // the warpgroups' running values, joined: all to the same reference, then handed on from
            // the last group to the first
            lsum[sw * R + row] = l_run;
            if (ew == 0) mrow[wg * R + row] = m_run;
            named_barrier(kBarAll, kSoft);
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < kGroups; w++) m = fmaxf(m, mrow[w * R + row]);
#pragma unroll
            for (int w = 0; w < kGroups; w++) {
                const float mw = mrow[w * R + row], *lw = lsum + 4 * w * R + row;
                const float lsum4 = (lw[0] + lw[R]) + (lw[2 * R] + lw[3 * R]);
                const float f = lsum4 == 0.f ? 0.f : ex2(mw - m);  // (sum 0: it saw nothing; NaN stays)
                l += lsum4 == 0.f ? 0.f : f * lsum4;
                if (w == wg) ab[row].x = f;
            }
            float *part = count < sg->nt ? a.part + (size_t)(2 * (int)blockIdx.x + (tile0 == 0 ? 1 : 0)) * slot_floats
                                         : nullptr;
            if (part == nullptr && wg == 0) ab[row].y = l == 0.f ? 0.f : 1.f / l;
            if (sw == 0 && (lane * R & 31) < R && rows[row].row >= 0 && *(volatile int *)abort_flag == 0) {  // one lane per row
                if (part != nullptr)
                    *reinterpret_cast<float2 *>(part + (size_t)R * D + 2 * row) = make_float2(m, l);
                else if (a.k.lse != nullptr)
                    a.k.lse[(size_t)rows[row].row * a.k.heads_q + rows[row].head] =
                        l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < R; i++) o[i] *= ab[i].x;
#pragma unroll 1
            for (int w = kGroups - 1; w > 0; w--) {
                if (wg == w && dlive) {
#pragma unroll
                    for (int i = 0; i < R; i++) merge[i * D + dcol] = o[i];
                }
                if (wg == w || wg == w - 1) named_barrier(8 + w, 256);
                if (wg == w - 1 && dlive) {
#pragma unroll
                    for (int i = 0; i < R; i++) o[i] += merge[i * D + dcol];
                }
            }
            if (wg == 0 && dlive) {
#pragma unroll
                for (int i = 0; i < R; i++) merge[i * D + dcol] = o[i];  // (this thread's own places)
#pragma unroll 1
                for (int i = 0; i < R; i++) {
                    const RowInfo ri = rows[i];
                    if (ri.row < 0 || *(volatile int *)abort_flag != 0) continue;
                    const float y = merge[i * D + dcol];
                    if (part != nullptr)
                        part[(size_t)i * D + dcol] = y;
                    else
                        a.k.out[(size_t)ri.row * a.k.ldo + (size_t)ri.head * D + dcol] =
                            __bfloat16_as_ushort(__float2bfloat16(y * ab[i].y));
                }
            }
            if (part != nullptr) {
                if (stid == 0) reinterpret_cast<Seg *>(smem + L.split)[shared] = *sg;
                shared++;
            }
            done += count;
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(B.q_empty(buf));
                mbar_arrive(B.seg_empty(seg % kSegs));
            }
            if (stid == 0)
                *go = lane_wait(B.q_full(buf ^ 1), (uint32_t)((seg + 1) >> 1) & 1u, 0xc32u, abort_flag) ? 1 : 0;
            named_barrier(kBarAll, kSoft);  // the merged values are read
        }
        join_role<D, kSoft>(a, S, reinterpret_cast<const Seg *>(smem + L.split), shared, kBarAll, abort_flag);
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

template <int D, int R>
cudaError_t launch_few(const CUtensorMap &tm, AttnArgs a, int sms, int smem_max, cudaStream_t st) {
    static PerDevice smem_set(0);
    a.over = 8;
    // as many stages as fit, values ahead of keys (a value stage is held for the whole softmax)
    a.nk = 2;
    a.nv = 3;
    while (true) {
        AttnArgs b = a;
        if (b.nv < kMaxStages && b.nv < b.nk + kGroups)
            b.nv++;
        else if (b.nk < kMaxStages)
            b.nk++;
        else
            break;
        if (FewSmem(D, R, b.nk, b.nv).total + 1024u > (uint32_t)smem_max) break;
        a = b;
    }
    const size_t smem = FewSmem(D, R, a.nk, a.nv).total + 1024;
    if (smem > (size_t)smem_max) return cudaErrorNotSupported;
    cudaError_t e = ensure_dynamic_smem(kv_attention_few_kernel<D, R>, smem, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)sms);
    cfg.blockDim = dim3(32 * kFirstSoft + 128 * kGroups);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;  // the join waits for all CTAs
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_attention_few_kernel<D, R>, tm, a);
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
    if (a.rpt > 32) return launch_attention_rows(tm, a, sms, smem_max, st);
    if (v.dim == 128)
        return a.rpt == 16 ? launch_few<128, 16>(tm, a, sms, smem_max, st) : launch_few<128, 32>(tm, a, sms, smem_max, st);
    return a.rpt == 16 ? launch_few<64, 16>(tm, a, sms, smem_max, st) : launch_few<64, 32>(tm, a, sms, smem_max, st);
}

}  // namespace moe
