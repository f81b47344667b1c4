// What the two forms of the cache attention share: the division of work, copies, query loading,
// and the joining of results that several workers hold parts of.
//
//   s[t][r] = ks_t * (k_t . q_r),  m_r = max_t s,  o_r = sum_t 2^(s - m) vs_t v_t / sum_t 2^(s - m)
//
// (log2 units: scale * log2(e) is folded into the scores).  Few rows, many tokens: the cache
// is read once, and everything else must hide behind that read.
//
//   - Codes go from HBM to shared memory to the tensor cores (kind::f8f6f4) as they lie in
//     the cache, with no conversion.  What multiplies them must be E4M3 too: a bf16 query is
//     the sum of two E4M3 parts (4 + 4 significant bits) after a power of two per row, exactly
//     from 2^-9 of the row's largest value on and to 2^-17 of that below, and a weight is written
//     as two parts as well (8 bits, as bf16 has).  Each product runs twice into the same
//     accumulator; the tensor pipe has room for it.
//   - A weight carries its page's value scale into the tensor cores: w = 2^(s - ref) vs.  ref is a
//     row's own, over the tokens that it sees of the 128-token tile: max(s + log2 vs) - 8, so that
//     its largest w is 256, and what E4M3's range cannot hold is below 2^-17 of that, whatever
//     scales other tokens of the tile have.  (One reference for the scales of the whole tile lost
//     the weights on pages with scales far below the tile's largest.)  The sums of 2^(s - ref)
//     go by the same reference; so that they stay in range, a scale below 2^-90 counts as 2^-90 in
//     it.  Each tile's output is a fresh accumulator joined with the running one in registers.
//   - Work: the (sequence, row tile, head, 128-token tile) units of the call in one line, cut
//     into equal shares, one per worker (one or three of an SM).  A share may begin and end
//     inside a sequence: such partial results go to the workspace and, after a grid barrier
//     (cooperative launch), the workers that share the sequence join it, each some rows.  Shares
//     are cut by the lengths on the device, so a captured graph serves any lengths.
//
// Roles of a CTA: warp 1 issues MMAs; the other three of the first four warps walk the share,
// copy tiles and load queries (one for each worker in the few-rows form; keys, values and the
// walk in the rows form); the rest are softmax warpgroups.
#pragma once

#include <type_traits>

#include "kv_internal.cuh"
#include "sm100_tensor.cuh"

namespace moe {
namespace {

constexpr int kTokens = 128;             // tokens per tile
constexpr int kMaxSlots = kTokens / 16;  // pages per tile
constexpr uint32_t kSwizzle64B = 4;
constexpr int kStKvArrive = 40, kStKvExit = 5;  // StatusWord::pad
constexpr int kFirstSoft = 4;            // first softmax warp
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNan = __builtin_nanf("");
constexpr float kLowScale = -90.f;       // log2 of the smallest value scale in a reference
constexpr float kTop = 8.f;              // log2 of a tile's largest weight

}  // namespace

// The groups' prefixes, every row of a group seeing all of its; what each sequence has of its own; or
// each sequence's prefix and own tokens together, nothing shared.
enum SharedPart { kPrefixes, kOwn, kWhole };

struct AttnArgs {
    KvAttentionArgs k;
    int group;      // query heads per key/value head
    int rpt;        // rows per row tile
    int nrt;        // row tiles of max_rows rows
    int nk, nv;     // stages of the key and value rings (rows form)
    int over;       // what starting a unit costs, in tiles
    float scale2;   // scale * log2(e)
    float *part;    // partial results: 2 slots per worker of [rpt][dim] + [rpt][2]
    // With shared prefixes: what a launch is about.
    const int32_t *cu_groups, *prefix_len;
    int groups, group_rows;  // groups, and the most rows of one
    SharedPart what;
    // sums over the prefixes in fp32 [rows][heads_q][dim], and the references and sums of weights that they go
    // by [rows][heads_q]: written over prefixes, and added to what is found over own tokens
    float *half;
    float2 *half_ml;
};

namespace {

// A segment: consecutive tiles of one (sequence, row tile, head) in a CTA's share.
struct Seg {
    int b, rt, n, len, row0, head, tile0;
    int q0, q1, h0;        // rows of the tile: the first, the last, and the first's head of the group
    int count;             // tiles; 0: the share ends here
    int see_all, see_max;  // tokens that every row of the tile sees, and that any row sees
    int nt;                // the unit's tiles: more than `count` if other CTAs have some of them
    int64_t u0;            // position of its first tile on the line
};
// With shared prefixes: the columns of the prefix, and the sequence whose row of the table names them.
struct SharedSeg : Seg {
    int col0, lead;
};
template <bool SHARED>
using SegOf = std::conditional_t<SHARED, SharedSeg, Seg>;

// One row of a row tile.
struct RowInfo {
    int row, head;  // row of q (-1: none), query head
    float qs;       // power of two: query = qs * (sum of its parts)
    int pos;        // the token it stands at (-1: sees nothing)
};

// One (sequence, row tile): its rows, tokens and tiles.
struct Item {
    int b, rt, row0, n, len, nt;
    bool ok;
};
struct SharedItem : Item {
    int col0, lead;
};
template <bool SHARED>
using ItemOf = std::conditional_t<SHARED, SharedItem, Item>;

// Tokens of a group's prefix that lie in whole pages.
__device__ __forceinline__ int whole_pages(const AttnArgs &a, int g) {
    return max(a.prefix_len[g], 0) & -a.k.kv.page;
}

// The sequence whose row of the table names a prefix's pages: the first of g0 .. g1 - 1 that has rows
// (one that has ended may have given its pages back).
__device__ __forceinline__ int lead_of(const AttnArgs &a, int g0, int g1) {
    const int row = a.k.cu_rows[g0];
    if (a.k.cu_rows[g0 + 1] > row) return g0;
    while (g1 - g0 > 1) {  // the last that begins at or before the first row
        const int mid = (g0 + g1) >> 1;
        if (a.k.cu_rows[mid] <= row)
            g0 = mid;
        else
            g1 = mid;
    }
    return g0;
}

// What load_item finds, where a group's prefix or a sequence's own tokens are the item.
__device__ __forceinline__ void load_shared(const AttnArgs &a, SharedItem &x) {
    const int64_t room = min((int64_t)a.k.table_width * a.k.kv.page, (int64_t)kMaxLen);
    int hi, len;
    if (a.what == kPrefixes) {
        const int g = x.b, g0 = a.cu_groups[g], g1 = a.cu_groups[g + 1];
        // the groups take all sequences, in order
        x.ok = g0 >= 0 && g0 <= g1 && g1 <= a.k.seqs && (g > 0 || g0 == 0) && (g + 1 < a.groups || g1 == a.k.seqs);
        x.b = x.ok && g0 < g1 ? lead_of(a, g0, g1) : 0;
        x.row0 = hi = 0;
        if (x.ok) {
            x.row0 = a.k.cu_rows[g0];
            hi = a.k.cu_rows[g1];
            if (x.row0 < 0 || x.row0 > hi || hi > a.k.rows) {
                x.row0 = hi = 0;
                x.ok = false;
            }
        }
        x.n = hi - x.row0;
        x.col0 = 0;
        x.lead = x.b;
        len = whole_pages(a, g);
    } else {
        x.ok = seq_rows(a.k.cu_rows, x.b, a.k.rows, x.row0, hi);
        x.n = hi - x.row0;
        int g = 0, end = a.groups;  // the last group that begins at or before the sequence
        while (end - g > 1) {
            const int mid = (g + end) >> 1;
            if (a.cu_groups[mid] <= x.b)
                g = mid;
            else
                end = mid;
        }
        // (over all, the groups are not looked at one by one)
        const int g0 = a.cu_groups[g], g1 = a.cu_groups[g + 1];
        if (a.what == kWhole && (!(g0 >= 0 && g0 <= x.b && x.b < g1 && g1 <= a.k.seqs) ||
                                 a.k.cu_rows[g1] - a.k.cu_rows[g0] > a.group_rows))
            x.ok = false;
        const int prefix = whole_pages(a, g), before = (int)min((int64_t)prefix, room);
        if (prefix > before) x.ok = false;
        x.col0 = before / a.k.kv.page;
        x.lead = a.what == kWhole && x.ok && x.n > 0 && before > 0 ? lead_of(a, g0, g1) : 0;
        const int all = max(a.k.kv_len[x.b], 0);
        if ((int64_t)all > room) x.ok = false;
        len = (int)min((int64_t)all, room) - before;
        if (x.n > 0 && before > 0 && len < x.n) x.ok = false;  // new rows stand in the prefix
        len = max(len, 0) + (a.what == kWhole ? before : 0);
    }
    if (x.n > a.k.max_rows) {
        x.n = a.k.max_rows;
        x.ok = false;
    }
    if (x.n > 0 && (int64_t)len > room) x.ok = false;
    x.len = (int)min((int64_t)len, room);
    x.nt = 0;
    if (x.rt * a.rpt < x.n * a.group) {
        const int last = a.nrt == 1 ? x.n - 1 : min(x.n - 1, ((x.rt + 1) * a.rpt - 1) / a.group);
        const int see = a.what == kPrefixes ? x.len : min(x.len, max(0, x.len - x.n + last + 1));
        x.nt = max(1, (see + kTokens - 1) / kTokens);
    }
}

template <bool SHARED>
__device__ __forceinline__ ItemOf<SHARED> load_item(const AttnArgs &a, int it) {
    ItemOf<SHARED> x;
    x.b = a.nrt == 1 ? it : it / a.nrt;
    x.rt = it - x.b * a.nrt;
    if constexpr (SHARED) {
        load_shared(a, x);
        return x;
    }
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
        const int last = a.nrt == 1 ? x.n - 1 : min(x.n - 1, ((x.rt + 1) * a.rpt - 1) / a.group);  // row of the tile
        const int see = min(x.len, max(0, x.len - x.n + last + 1));
        x.nt = max(1, (see + kTokens - 1) / kTokens);
    }
    return x;
}

// The line of units: a unit is one (item, head), `over` positions that stand for its fixed
// cost, then its tiles.  It is cut into equal shares, one per worker; a CTA has NW workers
// (numbers blockIdx.x, + gridDim.x, ...), which walk their shares independently.
struct Line {
    int64_t total, share;  // positions; of a worker, the first `more` of them one more
    int workers, more;     // workers with a share: the first ones
    // (divisions of 32 bits wherever the numbers allow: all of this is code that runs once, and
    // fetching it is what it costs)
    static __device__ __forceinline__ int64_t ratio(int64_t x, int64_t y) {
        return ((x | y) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
    }
    // Shares no shorter than pays: k workers on a unit of L positions take its tiles in L / k steps
    // but leave k parts to be joined one after the other, kJoin of which take a tile's time; L / k +
    // k / kJoin is least at shares of sqrt(L / kJoin).  The longest unit sets the limit, as it is the
    // one that is waited for.  (One sequence of 100000 tokens, one head, 4 query heads: 50 us, alone
    // or beside 63 short ones; with every worker on it 133.  With a limit by the number of units,
    // 118 beside the short ones.  kJoin = 2: 55, 10: 49.)
    __device__ __forceinline__ void set(int64_t total_, int longest, int max_workers) {
        constexpr float kJoin = 5.f;
        total = total_;
        const float pay = ceilf((float)total * __fsqrt_rn(kJoin / (float)longest));
        workers = (int)min((int64_t)fminf(pay, (float)max_workers), total);
        share = workers > 0 ? ratio(total, workers) : 0;
        more = (int)(total - share * workers);
    }
    // Where worker w's share begins (past the last worker: the end).
    __device__ __forceinline__ int64_t cut(int w) const { return w < workers ? w * share + min(w, more) : total; }
    // The worker that has position x.
    __device__ __forceinline__ int worker_of(int64_t x) const {
        const int64_t longer = (share + 1) * more;
        const bool in = x < longer;
        return (in ? 0 : more) + (int)ratio(in ? x : x - longer, in ? share + 1 : share);
    }
};

__device__ __forceinline__ int unit_length(const AttnArgs &a, const Item &x) { return x.nt == 0 ? 0 : x.nt + a.over; }

// A worker's share, and the item it starts in: its first position, number and description.
template <bool SHARED>
struct Start {
    int64_t lo, hi, first;
    int item;
    ItemOf<SHARED> x;
};

// Cut the line (all NT threads; `sums`: NT / 32 x 12 bytes of shared memory); the CTA's workers'
// starts are in start[] after the caller's next barrier.
template <int NT, int NW, bool SHARED>
__device__ __forceinline__ Line cut_line(const AttnArgs &a, int64_t *sums, Start<SHARED> *start) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int items = (SHARED && a.what == kPrefixes ? a.groups : a.k.seqs) * a.nrt;
    const int per = (items + NT - 1) / NT;
    const int i0 = min(tid * per, items), i1 = min(i0 + per, items);
    if (SHARED && a.what == kWhole && blockIdx.x == 0) {  // (else the groups themselves are the items)
        for (int g = tid; g < a.groups; g += NT) {
            const int g0 = a.cu_groups[g], g1 = a.cu_groups[g + 1];
            if (g0 > g1 || (g == 0 && g0 != 0) || (g + 1 == a.groups && g1 != a.k.seqs)) set_status(a.k.st, MOE_ERR_BAD_PAGE, 1);
        }
    }
    // two rounds over the thread's items: their sum, then those that hold the workers' starts
    Line l;
    int64_t mine = 0, pre = 0, lo[NW];
    int longest = 0, *tops = reinterpret_cast<int *>(sums + NT / 32);  // length of the longest unit
#pragma unroll 1
    for (int round = 0; round < 2; round++) {
        int64_t at = pre;
        bool good = true;
#pragma unroll 1
        for (int i = i0; i < i1; i++) {
            const ItemOf<SHARED> x = load_item<SHARED>(a, i);
            good &= x.ok;
            const int len = unit_length(a, x);
            longest = max(longest, len);
            const int64_t u = (int64_t)len * a.k.kv.heads;
            if (round == 1) {
#pragma unroll
                for (int w = 0; w < NW; w++) {
                    if (lo[w] >= at && lo[w] < at + u) {
                        start[w].first = at;
                        start[w].item = i;
                        start[w].x = x;
                    }
                }
            }
            at += u;
        }
        if (round == 1) break;
        mine = at;
        if (!good && blockIdx.x == 0) set_status(a.k.st, MOE_ERR_BAD_PAGE, 1);
        pre = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, pre, d);
            if (lane >= d) pre += o;
        }
        longest = __reduce_max_sync(0xffffffffu, longest);
        if (lane == 31) {
            sums[warp] = pre;
            tops[warp] = longest;
        }
        __syncthreads();
        int64_t total = 0;
#pragma unroll 1
        for (int w = 0; w < NT / 32; w++) {
            if (w < warp) pre += sums[w];
            total += sums[w];
            longest = max(longest, tops[w]);
        }
        pre -= mine;
        l.set(total, longest, (int)gridDim.x * NW);
        bool holds = false;
#pragma unroll
        for (int w = 0; w < NW; w++) {
            const int worker = (int)(blockIdx.x + w * gridDim.x);
            lo[w] = l.cut(worker);  // (without a share: past every item)
            if (tid == 0) {
                start[w].lo = lo[w];
                start[w].hi = l.cut(worker + 1);
            }
            holds |= lo[w] >= pre && lo[w] < pre + mine;
        }
        if (!holds) break;
    }
    return l;
}

// ------------------------------------------------------------ PTX

// Instruction descriptor of kind::f8f6f4, E4M3 x E4M3 -> fp32; tm, tn: operand M / N-major.
__device__ __forceinline__ uint32_t idesc_f8(int m, int n, bool tm, bool tn) {
    uint32_t d = 1u << 4;
    if (tm) d |= 1u << 15;
    if (tn) d |= 1u << 16;
    d |= (uint32_t)(n >> 3) << 17;
    d |= (uint32_t)(m >> 4) << 24;
    return d;
}

// An MMA issued by the one lane with `elected` set, in converged code: the predicate stands on
// the instruction itself, so its operands stay in uniform registers.  (Inside an `if` of one
// lane each MMA took 107 clocks to issue whatever its size; this form issues M = 128, K = 32 at
// 39 clocks for N = 16 and 64 for N = 128, the rate of the tensor pipe.)
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate, uint32_t elected) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(elected)
        : "memory");
}

// A in TMEM: row = lane, four 8-bit values along K per 32-bit column.
__device__ __forceinline__ void tc_mma_f8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate, uint32_t elected) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(elected)
        : "memory");
}

__device__ __forceinline__ void tc_commit_elected(uint64_t *bar, uint32_t elected) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(elected)
        : "memory");
}

// Accumulator columns of this warp's 32 lanes, not waited for.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float *v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
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
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// log2 and division to a few units of the last place.
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^x to 2 units of the last place, 0 below 2^-126.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The same to twice that with results down to 2^-149: references differ by value scales, too, and a
// sum far below another reference may be the larger one.  (The instruction's own form for such
// results took 2 us more for 4 x 17 rows.)
__device__ __forceinline__ float ex2_low(float x) {
    const float y = ex2(0.5f * x);
    return y * y;
}

// 4 bytes global -> shared, asynchronously; zero without reading if !ok.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
// One arrival on `bar` once this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The first of a value's two E4M3 parts: its nearest of 4 significant bits.  (NaN gives some
// number; the second part, value - first, is then NaN.)
__device__ __forceinline__ float part_hi(float x) {
    return __uint_as_float((__float_as_uint(x) + 0x80000u) & 0xfff00000u);
}

// The same for queries: none below E4M3's normal range, where the first part would be rounded
// when it is encoded and the second, left from the unrounded one, again.  So the two are off
// by half of E4M3's smallest step, 2^-10, at most.
__device__ __forceinline__ float query_hi(float x) { return fabsf(x) < 0.015625f ? 0.f : part_hi(x); }

// A ring of stages: slot and phase parity of the next use.
struct Ring {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(int n) {
        if (++s == n) {
            s = 0;
            ph ^= 1u;
        }
    }
};

// Whether the phase of parity `parity` is complete, without waiting (try_wait may suspend the
// thread for a while).
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Waits.  A wait that outlasts the limit writes `where` (not 0) to *abort_flag and gives up, as
// does every other wait of the CTA once the flag is set; the CTA reports it at its end.  All
// roles share one instruction cache and the kernel feels it when their loops do not fit, so
// these are kept short.
__device__ __forceinline__ bool expired(uint64_t &t0, unsigned where, int *abort_flag) {
    if (*(const volatile int *)abort_flag != 0) return true;
    const uint64_t now = global_timer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 <= g_wait_limit_ns) return false;
    *(volatile int *)abort_flag = (int)where;
    return true;
}

// A wait of a whole converged warp.  False after an abort or timeout.  The votes make the
// outcome uniform, so that what follows (descriptors, copies, MMAs) stays in uniform registers.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, unsigned where, int *abort_flag) {
    uint64_t t0 = 0;
    while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
        if (__any_sync(0xffffffffu, expired(t0, where, abort_flag))) return false;
    return true;
}

// A wait in the softmax warps, whose warpgroup barriers must match: after an abort nothing
// waits, and the code runs on to its end.
__device__ __forceinline__ void soft_wait(uint64_t *bar, uint32_t parity, unsigned where, int *abort_flag) {
    uint64_t t0 = 0;
    for (int n = 1; !mbar_try_wait(bar, parity); n++)  // (the timer costs issue slots: not each time)
        if ((n & 15) == 0 && expired(t0, where, abort_flag)) break;
    __syncwarp();
}

// One thread's wait; false after an abort or timeout.
__device__ __forceinline__ bool lane_wait(uint64_t *bar, uint32_t parity, unsigned where, int *abort_flag) {
    uint64_t t0 = 0;
    while (!mbar_try_wait(bar, parity))
        if (expired(t0, where, abort_flag)) return false;
    return true;
}

// Wait for copies or MMAs in flight, before the CTA exits, even after an abort: within the
// limit, but never less than 0.1 s, as what is in flight writes to this CTA's memory.
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity, int *abort_flag) {
    const uint64_t t0 = global_timer_ns(), lim = max(g_wait_limit_ns, (uint64_t)100000000);
    while (!mbar_try_wait(bar, parity)) {
        if (global_timer_ns() - t0 > lim) {
            *(volatile int *)abort_flag = 0xfff;
            break;
        }
    }
}

// What one lane of the MMA warp watches: a ring of barriers.
struct Watch {
    uint64_t *base;
    int n, i;
    uint32_t parity;
    __device__ __forceinline__ bool ready() const { return mbar_test(base + i, parity); }
    __device__ __forceinline__ void next() {
        if (++i == n) {
            i = 0;
            parity ^= 1u;
        }
    }
};

// ------------------------------------------- copies (warp 0: keys, warp 2: values, scales)
// As with the MMAs, the predicate stands on the copy itself and the warp stays converged.
__device__ __forceinline__ void tma_load_3d_elected(void *dst, const CUtensorMap *map, int c0, int c1, int c2,
                                                    uint64_t *bar, uint32_t elected) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];\n\t}" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar)), "r"(elected)
        : "memory");
}

// The page numbers of a segment, 32 columns of the table at a time: lane l holds column
// base + l, and the next 32.  One past the last page stands for a page outside the cache (it
// lies outside the tensor: zeros arrive) and for columns past the sequence's end.
template <int P, bool SHARED>
struct Pages {
    static constexpr int kSlots = kTokens / P;
    const int32_t *row;
    StatusWord *st;
    int n_pages, c1, at, left, id, id2, ahead;  // column of the tile in the 32; columns from the tile on
    const int32_t *lead;  // (SHARED) the row that names the first `split` columns
    int split;

    __device__ __forceinline__ int number(int col) const {
        if (col >= c1) return n_pages;
        const int page = SHARED && col < split ? lead[col] : row[col];
        if (page >= 0 && page < n_pages) return page;
        set_status(st, MOE_ERR_BAD_PAGE, 3);
        return n_pages;
    }
    __device__ __forceinline__ void start(const AttnArgs &a, const SegOf<SHARED> &g) {
        const int lane = threadIdx.x & 31, c0 = g.tile0 * kSlots;
        row = a.k.page_table + (size_t)g.b * a.k.table_width;
        if constexpr (SHARED) {
            if (a.what == kOwn) row += g.col0;
            lead = a.k.page_table + (size_t)g.lead * a.k.table_width;
            split = a.what == kWhole ? g.col0 : 0;
        }
        st = a.k.st;
        n_pages = a.k.kv.n_pages;
        c1 = min((g.see_max + P - 1) / P, (g.tile0 + g.count) * kSlots);
        at = 0;
        left = c1 - c0;
        id = number(c0 + lane);
        id2 = number(c0 + 32 + lane);
        ahead = c0 + 64;
    }
    __device__ __forceinline__ void next_tile() {
        at += kSlots;
        left -= kSlots;
        if (at == 32) {
            at = 0;
            id = id2;
            id2 = number(ahead + (int)(threadIdx.x & 31));
            ahead += 32;
        }
    }
    // One side (rows from y on of each page) of the tile's pages -> dst.
    template <int D>
    __device__ __forceinline__ void copy(const CUtensorMap *tm, unsigned char *dst, int y, uint64_t *full,
                                         uint32_t elected) const {
        if (left >= kSlots) {
            if (elected) mbar_arrive_expect_tx(full, kTokens * D);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kSlots; j++)
                tma_load_3d_elected(dst + j * (P * D), tm, 0, y, __shfl_sync(0xffffffffu, id, at + j), full, elected);
        } else {  // the sequence ends in this tile
            if (elected) mbar_arrive_expect_tx(full, (uint32_t)max(left, 0) * (uint32_t)(P * D));
            __syncwarp();
#pragma unroll 1
            for (int j = 0; j < left; j++)
                tma_load_3d_elected(dst + j * (P * D), tm, 0, y, __shfl_sync(0xffffffffu, id, at + j), full, elected);
        }
    }
    // The tile's scales of both sides -> [keys', values'][kMaxSlots] (kSlots arrivals on `full`).
    __device__ __forceinline__ void copy_scales(const AttnArgs &a, int head, float *dst, uint64_t *full) const {
        const int lane = threadIdx.x & 31, page = __shfl_sync(0xffffffffu, id, (at + lane) & 31);
        if (lane < kSlots) {
            const KvView &kv = a.k.kv;
            const bool ok = lane < left && page < n_pages;
            const uint32_t sc = smem_u32(dst + lane);
            const uint8_t *src = reinterpret_cast<const uint8_t *>(kv.scale(0, a.k.layer, 0, head)) +
                                 (uint64_t)(ok ? page : 0) * kv.page_rec;
            cp_async4(sc, src, ok);
            cp_async4(sc + kMaxSlots * 4u, src + 4 * kv.heads, ok);
            cp_async_arrive(full);
        }
    }
};

// ------------------------------------------------------------------ queries
// Warp w's part (of nw) of the rows of a segment's row tile: their data, and their queries as
// two E4M3 parts, after a power of two that puts a row's largest value into [128, 256).  A
// lane takes 8 values, so a pass covers 2 rows of 128 or 4 of 64; the next pass's loads are in
// flight while one is converted.  One pass per turn: this code runs once per segment, and
// fetching an unrolled loop costs more than the latency that it hides (four passes in flight:
// one sequence of 300 tokens 31 us in place of 27; all four words of a lane at once in the rows
// form: 4 x 17 rows 325 us in place of 321).  kCopies: how often the rows stand in the tile.
template <int D, int R, bool SHARED, int kCopies = 1>
__device__ __forceinline__ void load_queries(const AttnArgs &a, RowInfo *rows, unsigned char *q0, const Seg &g, int w,
                                             int nw) {
    constexpr int kLanes = D / 8, kPass = 32 / kLanes;
    const int lane = threadIdx.x & 31, sub = lane / kLanes, col = lane % kLanes;
    constexpr int kSpan = R / kCopies;                          // places of a copy
    const int live = min(a.rpt, g.n * a.group - g.rt * a.rpt);  // rows of the tile
    // rows past the tile see nothing (their queries are what was there: nobody reads their results)
    for (int r = live + 32 * w + lane; r < kSpan; r += 32 * nw) {
        RowInfo none = {-1, 0, 1.f, -1};
#pragma unroll
        for (int i = 0; i < kCopies; i++) rows[r + i * kSpan] = none;
    }
    const int per = (live + nw * kPass - 1) / (nw * kPass) * kPass;  // (whole passes: any two warps write apart)
    const int r0 = min(w * per, live), r1 = min(r0 + per, live);
    // this lane's row of the next pass, as (row, head of the group); a pass moves it on
    int qi = g.q0, hd = g.h0 + r0 + sub;
    if (r0 > 0) {
        qi += hd / a.group;
        hd %= a.group;
    }
    uint4 u;
    auto load = [&](int r) {
        while (hd >= a.group) {
            hd -= a.group;
            qi++;
        }
        u = make_uint4(0u, 0u, 0u, 0u);
        if (r + sub < r1)
            u = *reinterpret_cast<const uint4 *>(a.k.q + (size_t)(g.row0 + qi) * a.k.ldq +
                                                 (size_t)(g.head * a.group + hd) * D + col * 8);
    };
    load(r0);
#pragma unroll 1
    for (int r = r0; r < r1; r += kPass) {
        uint32_t v[4] = {u.x, u.y, u.z, u.w};
        RowInfo ri;
        ri.row = g.row0 + qi;
        ri.head = g.head * a.group + hd;
        ri.pos = SHARED && a.what == kPrefixes ? g.len - 1 : g.len - g.n + qi;
        hd += kPass;
        load(r + kPass);
        // largest magnitude over finite values, two columns of them
        constexpr uint32_t kMag = 0x7fff7fffu;
        uint32_t top = __vmaxu2(__vmaxu2(v[0] & kMag, v[1] & kMag), __vmaxu2(v[2] & kMag, v[3] & kMag));
        if (__any_sync(0xffffffffu, max(top & 0xffffu, top >> 16) >= 0x7f80u)) {
            top = 0;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint32_t m = v[j] & kMag;
                top = __vmaxu2(top, m & ~__vcmpgeu2(m, 0x7f807f80u));
            }
        }
        top = max(top & 0xffffu, top >> 16);
#pragma unroll 1
        for (int d = kLanes / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        const int up = top == 0 ? 0 : min(126, 7 - ((int)(top >> 7) - 127));
        const float f = __uint_as_float((uint32_t)(127 + up) << 23);
        ri.qs = __uint_as_float((uint32_t)(127 - up) << 23);
        // 16-byte chunks of a row are permuted as the tensor copies permute the keys'
        const int rr = r + sub;
        const uint32_t swz = D == 128 ? (uint32_t)(rr & 7) : (uint32_t)((rr >> 1) & 3);
        unsigned char *dst = q0 + (uint32_t)rr * D + (((uint32_t)(col >> 1) ^ swz) << 4) + (uint32_t)(col & 1) * 8u;
        uint64_t hi = 0, lo = 0;  // codes of the 8 values
#pragma unroll 1
        for (int j = 0; j < 4; j++) {
            const float y0 = __uint_as_float(v[0] << 16) * f, y1 = __uint_as_float(v[0] & 0xffff0000u) * f;
            const float h0 = query_hi(y0), h1 = query_hi(y1);
            hi = hi >> 16 | (uint64_t)e4m3x2_rn(h0, h1) << 48;
            lo = lo >> 16 | (uint64_t)e4m3x2_rn(y0 - h0, y1 - h1) << 48;
            v[0] = v[1];
            v[1] = v[2];
            v[2] = v[3];
        }
        if (rr < r1) {
#pragma unroll
            for (int i = 0; i < kCopies; i++) {  // (a copy lies whole swizzle periods further on)
                *reinterpret_cast<uint64_t *>(dst + i * (kSpan * D)) = hi;
                *reinterpret_cast<uint64_t *>(dst + (R + i * kSpan) * D) = lo;
                if (col == 0) rows[rr + i * kSpan] = ri;
            }
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// ------------------------------------------------------------------- segments
// Walks a worker's share.
template <bool SHARED>
struct Walk {
    const AttnArgs &a;
    int64_t w, hi, first;  // next position, end of the share; first position of the item
    int it;
    ItemOf<SHARED> x;

    __device__ __forceinline__ Walk(const AttnArgs &a_, const Start<SHARED> &st)
        : a(a_), w(st.lo), hi(st.hi), first(st.first), it(st.item), x(st.x) {}

    // The next segment; count 0 at the end of the share.
    __device__ __forceinline__ SegOf<SHARED> next() {
        SegOf<SHARED> g;
        g.count = 0;
#pragma unroll 1
        while (w < hi) {  // the next positions with tiles
            const int len = unit_length(a, x);
            const int64_t units = (int64_t)len * a.k.kv.heads, local = w - first;
            if (local >= units) {
                first += units;
                x = load_item<SHARED>(a, ++it);
                continue;
            }
            // (a division of 32 bits wherever the numbers allow)
            g.head = (local >> 31) == 0 ? (int)((uint32_t)local / (uint32_t)len) : (int)(local / len);
            const int pos = (int)(local - (int64_t)g.head * len);
            const int end = (int)min((int64_t)len, pos + (hi - w));
            w += end - pos;
            g.tile0 = max(0, pos - a.over);
            g.count = max(0, end - a.over) - g.tile0;
            if (g.count > 0) break;
        }
        g.count = max(g.count, 0);
        if (g.count != 0) {
            g.b = x.b;
            g.rt = x.rt;
            g.n = x.n;
            g.len = x.len;
            g.row0 = x.row0;
            // the tile's first and last row, and the first's head of the group
            int q0 = 0, q1 = x.n - 1;
            if (a.nrt > 1) {
                q0 = x.rt * a.rpt / a.group;
                q1 = min(q1, ((x.rt + 1) * a.rpt - 1) / a.group);
            }
            g.q0 = q0;
            g.q1 = q1;
            g.h0 = x.rt * a.rpt - q0 * a.group;
            g.see_all = min(x.len, max(0, x.len - x.n + q0 + 1));
            g.see_max = min(x.len, max(0, x.len - x.n + q1 + 1));
            if constexpr (SHARED) {
                if (a.what == kPrefixes) g.see_all = g.see_max = x.len;
                g.col0 = x.col0;
                g.lead = x.lead;
            }
            g.nt = x.nt;
            g.u0 = first + (int64_t)g.head * unit_length(a, x) + a.over;
        }
        return g;
    }
};

// Asks for a segment's queries ahead of their use (into L2): rows' heads of the group lie side
// by side.
__device__ __forceinline__ void prefetch_queries(const AttnArgs &a, const Seg &g) {
    const int bytes = a.group * a.k.kv.dim * 2;
    const char *at = reinterpret_cast<const char *>(a.k.q + (size_t)(g.row0 + g.q0) * a.k.ldq) + (size_t)g.head * bytes;
#pragma unroll 1
    for (int r = g.q0; r <= g.q1; r++, at += a.k.ldq * 2)
#pragma unroll 1
        for (int i = (threadIdx.x & 31) * 128; i < bytes; i += 32 * 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(at + i));
}

// Value rows of the tile's tokens in shared memory, for one tile that not every row sees
// whole (thread = token `tok` of the tile, which is token t of the sequence): rows that no
// row sees hold anything and become zero; NaN in rows that only some rows see must not reach
// the others, so it becomes zero here and is put back in the outputs (the returned truth).
template <int D>
__device__ __forceinline__ bool clean_values(unsigned char *tile, int tok, int t, int see_all, int see_max) {
    bool bad = false;
    if (t < see_all) return false;
#pragma unroll 1
    for (int j = 0; j < D / 16; j++) {
        uint4 *q = reinterpret_cast<uint4 *>(tile + (uint32_t)tok * D) + j;
        uint4 z = make_uint4(0u, 0u, 0u, 0u);
        if (t < see_max) {
            z = *q;
            uint32_t w[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const uint32_t n = __vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                bad |= n != 0;
                w[k] &= ~n;
            }
            z = make_uint4(w[0], w[1], w[2], w[3]);
        }
        *q = z;
    }
    return bad;
}

// Code of value d of token t as it lies in the cache (0 if its page is outside).
template <typename SEG>
__device__ __forceinline__ const uint8_t *value_codes(const AttnArgs &a, const SEG &g, int t) {
    const int P = a.k.kv.page;
    const int32_t *row = a.k.page_table + (size_t)g.b * a.k.table_width;
    if constexpr (std::is_same_v<SEG, SharedSeg>) {
        if (a.what == kOwn) row += g.col0;
        if (a.what == kWhole && t / P < g.col0) row = a.k.page_table + (size_t)g.lead * a.k.table_width;
    }
    const int page = row[t / P];
    if (page < 0 || page >= a.k.kv.n_pages) return nullptr;
    return a.k.kv.codes(page, a.k.layer, 1, g.head) + (size_t)(t % P) * a.k.kv.dim;
}

// A row's sums over its own tokens (by reference `ref`; l: of its weights) with those over the prefix of its
// group.  References hold value scales, as everywhere: a part whose weights are far below the other's may
// still have the larger products.
struct Halves {
    float own, prefix, lse;  // factors of the two; the logarithm of the whole sum
    __device__ __forceinline__ Halves(const AttnArgs &a, size_t at, float ref, float l) {
        const float2 p = a.what == kOwn ? __ldg(a.half_ml + at) : make_float2(-INFINITY, 0.f);
        const float m = fmaxf(ref, p.x);
        // (as roots: a sum may be large where its reference is more than 126 below; sum 0: it saw nothing; NaN stays)
        own = l == 0.f ? 0.f : ex2(0.5f * (ref - m));
        prefix = p.y == 0.f ? 0.f : ex2(0.5f * (p.x - m));
        const float all = fmaf(own * l, own, prefix * p.y * prefix), inv = all == 0.f ? 0.f : 1.f / all;
        lse = all == 0.f ? -INFINITY : kLn2 * (m + log2f(all));
        own *= own * inv;
        prefix *= prefix * inv;
    }
    __device__ __forceinline__ float add(float o, float p) const { return fmaf(o, own, p * prefix); }
};

// ---------------------------------------- units shared with other workers
// All NT threads of a worker (tid: 0 .. NT-1), after its last segment: partial results are
// published, and once every worker has done so this one joins its rows of the (at most two)
// units it shares, `shared` of which stand in `list`.
template <int D, int NT, bool SHARED>
__device__ __forceinline__ void join_role(const AttnArgs &a, const Line &line, int worker, const SegOf<SHARED> *list, int shared,
                                          int tid, int bar_id, int *abort_flag) {
    StatusWord *st = a.k.st;
    const int lane = tid & 31, sw = tid >> 5;
    const size_t slot_floats = (size_t)a.rpt * D + 2 * a.rpt;
    unsigned int *arrive = &st->pad[kStKvArrive], *leave = &st->pad[kStKvExit];
    __threadfence();
    named_barrier(bar_id, NT);
    if (tid == 0) red_release_gpu_add(arrive, 1u);
    // the (at most two) units: the workers that share each, and this one's rows of it
    int c0[2], parts[2], mine[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        c0[i] = parts[i] = mine[i] = 0;
        if (i < shared) {
            const Seg &g = list[i];
            c0[i] = line.worker_of(g.u0);
            parts[i] = line.worker_of(g.u0 + g.nt - 1) - c0[i] + 1;
            const int nrows = min(a.rpt, g.n * a.group - g.rt * a.rpt);
            mine[i] = max(0, (nrows - (worker - c0[i]) + parts[i] - 1) / parts[i]);  // rows worker - c0, + parts, ...
        }
    }
    if (shared > 0) {
        if (tid == 0 && *(volatile int *)abort_flag == 0) {
            const uint64_t t0 = global_timer_ns(), lim = g_wait_limit_ns;
            while (ld_acquire_gpu(arrive) < (unsigned)line.workers) {
                if (global_timer_ns() - t0 > lim) {
                    *(volatile int *)abort_flag = 0xd00;
                    break;
                }
            }
        }
        named_barrier(bar_id, NT);
        // a warp per row, lanes over the head's values
#pragma unroll 1
        for (int j = sw; j < mine[0] + mine[1]; j += NT / 32) {
            if (*(volatile int *)abort_flag) break;
            const bool second = j >= mine[0];
            const Seg &g = list[second ? 1 : 0];
            const int c0_ = second ? c0[1] : c0[0], parts_ = second ? parts[1] : parts[0];
            const int r = worker - c0_ + parts_ * (second ? j - mine[0] : j);
            constexpr int V = D / 32, U = 4;  // values per lane; parts whose loads are in flight together
            auto slot_of = [&](int p) { return a.part + (size_t)(2 * (c0_ + p) + (p == 0 ? 1 : 0)) * slot_floats; };
            auto load = [&](int p, float (&x)[V]) {
                const float *v = slot_of(p) + (size_t)r * D + lane * V;
                if constexpr (V == 4) {
                    const float4 t = __ldcg(reinterpret_cast<const float4 *>(v));
                    x[0] = t.x;
                    x[1] = t.y;
                    x[2] = t.z;
                    x[3] = t.w;
                } else {
                    const float2 t = __ldcg(reinterpret_cast<const float2 *>(v));
                    x[0] = t.x;
                    x[1] = t.y;
                }
            };
            float x[U][V], acc[V], l = 0.f, m = -INFINITY;
#pragma unroll
            for (int j = 0; j < V; j++) acc[j] = 0.f;
#pragma unroll
            for (int i = 0; i < U; i++)
                if (i < parts_) load(i, x[i]);
            // references and sums, a lane per part (the first 32, and what more there is one by one)
            float2 ml = make_float2(-INFINITY, 0.f);
            if (lane < parts_) ml = __ldcg(reinterpret_cast<const float2 *>(slot_of(lane) + (size_t)a.rpt * D + 2 * r));
            m = ml.x;
            for (int p = lane + 32; p < parts_; p += 32) m = fmaxf(m, __ldcg(slot_of(p) + (size_t)a.rpt * D + 2 * r));
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            const float mine = ml.y == 0.f ? 0.f : ex2_low(ml.x - m);  // (sum 0: it saw nothing; NaN stays)
#pragma unroll 1
            for (int p = 0; p < parts_; p += U) {
#pragma unroll
                for (int i = 0; i < U; i++) {
                    if (p + i >= parts_) continue;
                    float f, s;
                    if (p + i < 32) {
                        f = __shfl_sync(0xffffffffu, mine, p + i);
                        s = __shfl_sync(0xffffffffu, ml.y, p + i);
                    } else {
                        const float2 t = __ldcg(reinterpret_cast<const float2 *>(slot_of(p + i) + (size_t)a.rpt * D + 2 * r));
                        f = t.y == 0.f ? 0.f : ex2_low(t.x - m);
                        s = t.y;
                    }
                    l = fmaf(s, f, l);
#pragma unroll
                    for (int j = 0; j < V; j++) acc[j] = fmaf(x[i][j], f, acc[j]);
                }
#pragma unroll
                for (int i = 0; i < U; i++)
                    if (p + U + i < parts_) load(p + U + i, x[i]);
            }
            const int R = g.rt * a.rpt + r, qi = R / a.group, row = g.row0 + qi;
            const int hq = g.head * a.group + R - qi * a.group;
            uint16_t *out = a.k.out + (size_t)row * a.k.ldo + (size_t)hq * D + lane * V;
            if constexpr (SHARED) {
                const size_t at = (size_t)row * a.k.heads_q + hq;
                float *half = a.half + at * D + lane * V;
                if (a.what == kPrefixes) {
#pragma unroll
                    for (int j = 0; j < V; j++) half[j] = acc[j];
                    if (lane == 0) a.half_ml[at] = make_float2(m, l);
                    continue;
                }
                const Halves h(a, at, m, l);
#pragma unroll
                for (int j = 0; j < V; j++)
                    out[j] = __bfloat16_as_ushort(__float2bfloat16(h.add(acc[j], a.what == kOwn ? __ldg(half + j) : 0.f)));
                if (a.k.lse != nullptr && lane == 0) a.k.lse[at] = h.lse;
            } else {
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                for (int j = 0; j < V; j++) out[j] = __bfloat16_as_ushort(__float2bfloat16(acc[j] * inv));
                if (a.k.lse != nullptr && lane == 0)
                    a.k.lse[(size_t)row * a.k.heads_q + hq] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
            }
        }
    }
    named_barrier(bar_id, NT);
    if (tid == 0 && atomicAdd(leave, 1u) == (unsigned)line.workers - 1u) {
        // every worker has arrived and has stopped polling
        *(volatile unsigned int *)arrive = 0u;
        *(volatile unsigned int *)leave = 0u;
    }
}

}  // namespace

// The two forms, by the number of rows of a row tile: tokens along the tensor cores' M for
// up to 16 rows (kv_attention_few.cuh), rows along M for up to 128 (kv_attention_rows.cuh).
cudaError_t launch_attention_rows(const CUtensorMap &tm, AttnArgs a, int sms, int smem_max, cudaStream_t st);
cudaError_t set_wait_limit_kv_attention_rows(uint64_t ns);
cudaError_t set_wait_limit_kv_attention_shared(uint64_t ns);

}  // namespace moe
