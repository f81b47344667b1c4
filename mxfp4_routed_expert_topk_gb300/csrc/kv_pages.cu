// Pages of a paged cache, found and given back on the GPU from the sequences' lengths.
//
// A page is free while its count of holders is 0, so there is no list to keep in order: the pages
// that a call takes are the lowest-numbered free ones, whatever happened before, and giving pages
// back is a subtraction per page, which comes to the same in any order.
//
// Reserving is one cluster of CTAs.  Every CTA sums the sequences' needs by itself (a scan over the
// block) and counts the free pages of its part of the pool; the counts are exchanged through
// distributed shared memory, so that every warp knows the numbers of its free pages among all.  The
// lowest ones lie in few CTAs' parts: those hand them to all CTAs' shared memory, and every thread
// then looks up one or two places in the line of (sequence, column) for its pages.  Nothing is written
// before the call is known to succeed, so a call that cannot be served changes nothing.
//
// What bounds it is the chain: 64 sequences of which none needs a page take 6 us (3 of them loads one
// after the other and sums).  512 sequences that take 7200 pages of 400000 and map 115000 rows take 31 us
// (by stamps: needs 4, counting 6, exchange 2, handing out 8, rows 10; the rest is start and end); where
// the warps that find the pages also looked up their places it was 57.  Called from Python either takes 35
// to 45.
#include <algorithm>

#include "kv_internal.cuh"
#include "sm100_tensor.cuh"

namespace moe {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kSteps = 16;   // pieces of a warp's pages
constexpr int kHand = 4096;  // pages that a CTA is handed at a time

struct Sums {
    int64_t pages, rows;
};

__device__ __forceinline__ void store_cluster_i32(int *mine, uint32_t rank, int v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(mine, rank)), "r"(v) : "memory");
}

// Pages and rows that sequence b asks for; false if it cannot have them.
__device__ __forceinline__ bool asks(const KvReserveArgs &a, int b, int start, Sums &s) {
    const int n = a.new_rows[b];
    s.pages = s.rows = 0;
    if (n == 0) return true;  // an idle sequence may stand anywhere
    if (n < 0 || start < 0) return false;
    const int64_t end = (int64_t)start + n;
    if (end > min((int64_t)a.table_width * a.page, (int64_t)kMaxLen)) return false;
    const int c0 = (start + a.page - 1) / a.page;
    s.pages = (end + a.page - 1) / a.page - c0;
    s.rows = n;
    if (start % a.page != 0) {  // rows join older ones in a page: nobody else may hold it
        const int p = a.page_table[(size_t)b * a.table_width + start / a.page];
        return p >= 0 && p < a.n_pages && a.refs[p] == 1;
    }
    return true;
}

// The last i of 0 .. n - 1 with at[i] <= x (at ascends, at[0] <= x).
__device__ __forceinline__ int place_of(const int *at, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads, 1) kv_reserve_kernel(const KvReserveArgs a) {
    extern __shared__ int s_dyn[];
    int *s_page = s_dyn, *s_row = s_page + a.seqs + 1, *s_start = s_row + a.seqs + 1;  // pages, rows before a sequence
    __shared__ Sums s_warp[kWarps];
    __shared__ int s_free[kSteps * kWarps], s_sum[kWarps], s_cta[kCluster], s_hand[kHand];
    const int shift = 31 - __clz(a.page);
    const int rank = (int)cluster_ctarank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    cluster_arrive();  // waited for before the first remote store: by then every CTA has started

    // the needs, and what stands before each sequence
    const int per = (a.seqs + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, a.seqs), b1 = min(b0 + per, a.seqs);
    Sums mine = {0, 0};
    bool ok = true;
    for (int b = b0; b < b1; b++) {
        const int start = a.start[b];
        Sums s;
        ok &= asks(a, b, start, s);
        s_start[b] = start;
        s_page[b] = (int)mine.pages;  // (from the thread's first; a call with more than 2^31 fails)
        s_row[b] = (int)mine.rows;
        mine.pages += s.pages;
        mine.rows += s.rows;
    }
    Sums upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t p = __shfl_up_sync(0xffffffffu, upto.pages, d), r = __shfl_up_sync(0xffffffffu, upto.rows, d);
        if (lane >= d) {
            upto.pages += p;
            upto.rows += r;
        }
    }
    if (lane == 31) s_warp[warp] = upto;
    unsigned code = __syncthreads_and(ok) ? MOE_OK : MOE_ERR_BAD_PAGE;
    Sums total = {0, 0}, before = {upto.pages - mine.pages, upto.rows - mine.rows};
    for (int w = 0; w < kWarps; w++) {
        if (w < warp) {
            before.pages += s_warp[w].pages;
            before.rows += s_warp[w].rows;
        }
        total.pages += s_warp[w].pages;
        total.rows += s_warp[w].rows;
    }
    for (int b = b0; b < b1; b++) {
        s_page[b] += (int)before.pages;
        s_row[b] += (int)before.rows;
    }
    if (tid == 0) {
        s_page[a.seqs] = (int)total.pages;
        s_row[a.seqs] = (int)total.rows;
    }
    if (total.rows > a.rows) code = MOE_ERR_BAD_PAGE;
    if (code == MOE_OK && total.pages > a.n_pages) code = MOE_ERR_NO_PAGE;
    const int need = (int)total.pages;
    const bool search = code == MOE_OK && need > 0;  // (the same in every CTA)

    // The CTA's pages: kSteps times kWarps pieces in a row, a warp's pages 4 to a lane.
    const int piece = ((a.n_pages + kCluster * kSteps * kWarps - 1) / (kCluster * kSteps * kWarps) + 127) / 128 * 128;
    const bool vec = ((uintptr_t)a.refs & 15u) == 0;
    auto begin = [&](int step) {  // of this warp's piece
        return (int)min((int64_t)((rank * kSteps + step) * kWarps + warp) * piece, (int64_t)a.n_pages);
    };
    auto free_of = [&](int p, int end) -> uint32_t {  // of pages p .. p + 3, a bit each
        uint32_t m = 0;
        if (vec && p + 4 <= end) {
            const int4 r = __ldcg(reinterpret_cast<const int4 *>(a.refs + p));
            m = (r.x == 0 ? 1u : 0u) | (r.y == 0 ? 2u : 0u) | (r.z == 0 ? 4u : 0u) | (r.w == 0 ? 8u : 0u);
        } else {
            for (int k = 0; k < 4; k++)
                if (p + k < end && __ldcg(a.refs + p + k) == 0) m |= 1u << k;
        }
        return m;
    };
    if (search) {
        constexpr int kSide = 8;  // pieces whose loads are in flight together
        for (int s0 = 0; s0 < kSteps; s0 += kSide) {
            int found[kSide];
#pragma unroll
            for (int j = 0; j < kSide; j++) found[j] = 0;
            for (int i = 4 * lane; i - 4 * lane < piece; i += 128) {
#pragma unroll
                for (int j = 0; j < kSide; j++) {
                    const int p = begin(s0 + j) + i, end = min(begin(s0 + j) + piece, a.n_pages);
                    found[j] += p < end ? __popc(free_of(p, end)) : 0;
                }
            }
#pragma unroll
            for (int j = 0; j < kSide; j++) {
                const int sum = __reduce_add_sync(0xffffffffu, found[j]);
                if (lane == 0) s_free[(s0 + j) * kWarps + warp] = sum;
            }
        }
    }
    __syncthreads();
    int cta = 0;
    if (search) {  // running sums of the pieces' free pages
        static_assert(kSteps * kWarps <= kThreads, "a thread per piece");
        const int mine = tid < kSteps * kWarps ? s_free[tid] : 0;
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += o;
        }
        if (lane == 31) s_sum[warp] = upto;
        __syncthreads();
        upto -= mine;
        for (int w = 0; w < kSteps; w++) {
            if (w < warp) upto += s_sum[w];
            cta += s_sum[w];
        }
        if (tid < kSteps * kWarps) s_free[tid] = upto;
    }
    cluster_wait();
    if (tid < kCluster) store_cluster_i32(s_cta + rank, (uint32_t)tid, cta);
    cluster_sync();  // the counts are there; every check has been made
    int all = 0, first = 0;  // free pages; those of the CTAs before this one
    for (int k = 0; k < kCluster; k++) {
        if (k < rank) first += s_cta[k];
        all += s_cta[k];
    }
    if (search && all < need) code = MOE_ERR_NO_PAGE;
    if (code != MOE_OK && rank == 0 && tid == 0) set_status(a.st, code, (unsigned)min(total.pages, (int64_t)0x7fffffff));

    for (int b = rank * kThreads + tid; b <= a.seqs; b += kCluster * kThreads) {
        a.cu_rows[b] = code == MOE_OK ? s_row[b] : 0;
        if (b < a.seqs) a.kv_len[b] = s_start[b] + (code == MOE_OK ? s_row[b + 1] - s_row[b] : 0);
    }
    if (code != MOE_OK) return;
    if (search) {
        for (int from = 0; from < need; from += kCluster * kHand) {
            const int to = min(from + kCluster * kHand, need);
            if (from > 0) cluster_sync();  // (those of the round before are taken)
            for (int step = 0; step < kSteps; step++) {
                // this piece's first free page among all (those before `from` are taken, and not free now)
                int at = max(first + s_free[step * kWarps + warp], from);
                if (at >= to) break;
                const int end = min(begin(step) + piece, a.n_pages);
                for (int p = begin(step) + 4 * lane; p - 4 * lane < end && at < to; p += 128) {
                    const uint32_t m = p < end ? free_of(p, end) : 0u;
                    int upto = __popc(m);
                    const int own = upto;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const int o = __shfl_up_sync(0xffffffffu, upto, d);
                        if (lane >= d) upto += o;
                    }
                    int k = at + upto - own;
                    at += __shfl_sync(0xffffffffu, upto, 31);
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        if ((m >> i & 1u) == 0u) continue;
                        const int h = k - from;
                        if (k < to) store_cluster_i32(s_hand + h % kHand, (uint32_t)(h / kHand), p + i);
                        k++;
                    }
                }
            }
            cluster_sync();
            for (int i = tid; i < kHand; i += kThreads) {
                const int k = from + rank * kHand + i;
                if (k >= to) break;
                const int b = place_of(s_page, a.seqs, k), page = s_hand[i];
                const int col = ((s_start[b] + a.page - 1) >> shift) + k - s_page[b];
                a.refs[page] = 1;
                a.page_table[(size_t)b * a.table_width + col] = page;
            }
        }
        cluster_sync();  // the table is complete
    }
    if (a.row_seq == nullptr && a.row_pos == nullptr && a.row_slot == nullptr) return;
    // four rows of a thread at a time: their searches and loads go side by side
    constexpr int kSide = 4, kStep = kCluster * kThreads;
    for (int r0 = rank * kThreads + tid; r0 < (int)total.rows; r0 += kSide * kStep) {
        int lo[kSide], hi[kSide];
#pragma unroll
        for (int j = 0; j < kSide; j++) lo[j] = 0, hi[j] = a.seqs;
        for (int n = a.seqs; n > 1; n = (n + 1) >> 1) {
#pragma unroll
            for (int j = 0; j < kSide; j++) {
                const int mid = (lo[j] + hi[j]) >> 1;
                if (hi[j] - lo[j] <= 1) continue;
                if (s_row[mid] <= r0 + j * kStep)
                    lo[j] = mid;
                else
                    hi[j] = mid;
            }
        }
        int pos[kSide], page[kSide];
#pragma unroll
        for (int j = 0; j < kSide; j++) {
            const int r = r0 + j * kStep;
            pos[j] = s_start[lo[j]] + r - s_row[lo[j]];
            page[j] = 0;
            if (r < (int)total.rows && a.row_slot != nullptr)
                page[j] = __ldcg(a.page_table + (size_t)lo[j] * a.table_width + (pos[j] >> shift));
        }
#pragma unroll
        for (int j = 0; j < kSide; j++) {
            const int r = r0 + j * kStep;
            if (r >= (int)total.rows) break;
            if (a.row_seq != nullptr) a.row_seq[r] = lo[j];
            if (a.row_pos != nullptr) a.row_pos[r] = pos[j];
            if (a.row_slot != nullptr) a.row_slot[r] = ((int64_t)page[j] << shift) + (pos[j] & (a.page - 1));
        }
    }
}

// A block per sequence: its dropped columns.
__global__ void __launch_bounds__(128) kv_release_kernel(const KvReleaseArgs a) {
    const int b = blockIdx.x, keep = a.keep[b], len = a.kv_len[b];
    if (keep >= 0 && len <= keep) return;
    if (keep < 0 || (int64_t)len > (int64_t)a.table_width * a.page) {
        if (threadIdx.x == 0) set_status(a.st, MOE_ERR_BAD_PAGE, 1);
        return;
    }
    const int c0 = (int)(((int64_t)keep + a.page - 1) / a.page), c1 = (int)(((int64_t)len + a.page - 1) / a.page);
    for (int c = c0 + (int)threadIdx.x; c < c1; c += (int)blockDim.x) {
        int32_t *entry = a.page_table + (size_t)b * a.table_width + c;
        const int p = *entry;
        *entry = -1;
        bool ok = p >= 0 && p < a.n_pages;
        if (ok && atomicSub(a.refs + p, 1) <= 0) {  // nobody held it
            atomicAdd(a.refs + p, 1);
            ok = false;
        }
        if (!ok) set_status(a.st, MOE_ERR_BAD_PAGE, 2);
    }
}

}  // namespace

cudaError_t launch_kv_reserve(const KvReserveArgs &a, cudaStream_t st) {
    static PerDevice smem_set(0);
    const size_t smem = (size_t)3 * (a.seqs + 1) * sizeof(int);
    const cudaError_t e = ensure_dynamic_smem(kv_reserve_kernel, smem, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    TraceScope trace_scope("kv_reserve", st);
    return cudaLaunchKernelEx(&cfg, kv_reserve_kernel, a);
}

cudaError_t launch_kv_release(const KvReleaseArgs &a, cudaStream_t st) {
    TraceScope trace_scope("kv_release", st);
    kv_release_kernel<<<dim3((unsigned)a.seqs), dim3(128), 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
