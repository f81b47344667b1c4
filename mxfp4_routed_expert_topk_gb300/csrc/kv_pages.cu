// Pages of a paged cache, found and given back on the GPU from the sequences' lengths.
//
// A page is free while its count of holders is 0, so there is no list to keep in order: the pages
// that a call takes are the lowest-numbered free ones, whatever happened before, and giving pages
// back is a subtraction per page, which comes to the same in any order.
//
// Reserving is one cluster of CTAs.  Every CTA sums the sequences' needs by itself (a scan over the
// block) and counts the free pages of its part of the pool; the counts are exchanged through
// distributed shared memory, and the CTA that finds free page number k writes it into the place
// that is k-th in the line of (sequence, column).  Nothing is written before the call is known to
// succeed, so a call that cannot be served changes nothing.
#include <algorithm>

#include "kv_internal.cuh"
#include "sm100_tensor.cuh"

namespace moe {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;

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
    __shared__ int s_free[kWarps], s_cta[kCluster];
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

    // this warp's pages: consecutive ones, 4 to a lane
    const int part = ((a.n_pages + kCluster - 1) / kCluster + 127) / 128 * 128;
    const int lo = min((int64_t)rank * part, (int64_t)a.n_pages), hi = min((int64_t)lo + part, (int64_t)a.n_pages);
    const int chunk = (part / 128 + kWarps - 1) / kWarps * 128;
    const int w0 = min(lo + warp * chunk, hi), w1 = min(w0 + chunk, hi);
    const bool vec = ((uintptr_t)a.refs & 15u) == 0;
    auto free_of = [&](int p) -> uint32_t {  // of pages p .. p + 3, a bit each
        uint32_t m = 0;
        if (vec && p + 4 <= w1) {
            const int4 r = __ldcg(reinterpret_cast<const int4 *>(a.refs + p));
            m = (r.x == 0 ? 1u : 0u) | (r.y == 0 ? 2u : 0u) | (r.z == 0 ? 4u : 0u) | (r.w == 0 ? 8u : 0u);
        } else {
            for (int k = 0; k < 4; k++)
                if (p + k < w1 && __ldcg(a.refs + p + k) == 0) m |= 1u << k;
        }
        return m;
    };
    int found = 0;
    if (search)
#pragma unroll 4
        for (int p = w0 + 4 * lane; p < w1; p += 128) found += __popc(free_of(p));
    found = __reduce_add_sync(0xffffffffu, found);
    if (lane == 0) s_free[warp] = found;
    __syncthreads();
    int cta = 0, at = 0;
    for (int w = 0; w < kWarps; w++) {
        if (w < warp) at += s_free[w];
        cta += s_free[w];
    }
    cluster_wait();
    if (tid < kCluster) store_cluster_i32(s_cta + rank, (uint32_t)tid, cta);
    cluster_sync();  // the counts are there; every check has been made
    int all = 0;
    for (int k = 0; k < kCluster; k++) {
        if (k < rank) at += s_cta[k];
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
        for (int p0 = w0; p0 < w1 && at < need; p0 += 128) {
            const int p = p0 + 4 * lane;
            const uint32_t m = p < w1 ? free_of(p) : 0u;
            int upto = __popc(m);
            const int own = upto;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += o;
            }
            int k = at + upto - own;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if ((m >> i & 1u) == 0u) continue;
                if (k < need) {
                    const int b = place_of(s_page, a.seqs, k);
                    const int col = (s_start[b] + a.page - 1) / a.page + k - s_page[b];
                    a.refs[p + i] = 1;
                    a.page_table[(size_t)b * a.table_width + col] = p + i;
                }
                k++;
            }
            at += __shfl_sync(0xffffffffu, upto, 31);
        }
        cluster_sync();  // the table is complete
    }
    if (a.row_seq == nullptr && a.row_pos == nullptr && a.row_slot == nullptr) return;
    for (int r = rank * kThreads + tid; r < (int)total.rows; r += kCluster * kThreads) {
        const int b = place_of(s_row, a.seqs, r), pos = s_start[b] + r - s_row[b];
        if (a.row_seq != nullptr) a.row_seq[r] = b;
        if (a.row_pos != nullptr) a.row_pos[r] = pos;
        if (a.row_slot != nullptr)
            a.row_slot[r] = (int64_t)__ldcg(a.page_table + (size_t)b * a.table_width + pos / a.page) * a.page + pos % a.page;
    }
}

// A block per sequence: its dropped columns.
__global__ void __launch_bounds__(128) kv_release_kernel(const KvReleaseArgs a) {
    const int b = blockIdx.x, keep = a.keep[b], len = a.kv_len[b];
    if (len <= keep) return;
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
