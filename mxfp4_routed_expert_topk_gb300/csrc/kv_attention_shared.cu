// Cache attention of sequences that share prefixes: a prompt that several continuations are sampled
// from, or a document that many requests ask about.
//
// Every row of a group sees all of its prefix, so a row's result is
//
//   o = (2^(m1 - m) o1 + 2^(m2 - m) o2) / (2^(m1 - m) l1 + 2^(m2 - m) l2),  m = max(m1, m2)
//
// with o1, o2 its sums of weighted values over the prefix and over the sequence's own tokens, l1, l2 those of
// the weights, and m1, m2 the references that they go by.  The first is one problem per group, with all of
// the group's rows in row tiles that read the prefix once for up to 128 of them, and its results go to the
// workspace in fp32; the second is one per sequence and adds the first when it writes its own.  Both are the
// cache attention's kernels with other lengths and tables.
//
// Small batches run once, each sequence over its prefix and its own tokens: two runs take 38 us or more,
// however little there is to do.
#include <algorithm>

#include "kv_attention_few.cuh"
#include "kv_attention_rows.cuh"

namespace moe {
namespace {

// Tiles per SM (as many as the tables have room for: the lengths are known on the device alone, so short
// sequences with wide tables run twice) up to which a batch is small.  Once / twice, one row of
// 56 heads of 128, tables as wide as the sequences are long: 16 sequences of 2000 + 200 tokens (14 tiles per SM)
// 33 / 49 us, 64 of 1000 + 100 (30) 51 / 57, 2 of 30000 (25) 47 / 58, 8 of 16000 (53) 61 / 53, 64 of 4000 +
// 300 (115) 112 / 78; five rows, 32 of 2000 + 300 (30) 72 / 79.
constexpr int kSmall = 32;

cudaError_t run(const AttnSetup &s, cudaStream_t st) {
    if (s.a.rpt > kFewRows) return launch_rows<true>(s.tm, s.a, s.sms, s.smem_max, st);
    return launch_few_of<true>(s.tm, s.a, s.sms, s.smem_max, st);
}

}  // namespace

cudaError_t set_wait_limit_kv_attention_shared(uint64_t ns) { return set_wait_limit_here(ns); }

cudaError_t kv_attention_shared_workspace_bytes(const KvView &kv, int rows, int max_rows, int max_group_rows, int heads_q,
                                                size_t *bytes) {
    size_t own = 0, prefix = 0;
    cudaError_t e = part_bytes(kv, max_rows, heads_q, &own);
    if (e == cudaSuccess) e = part_bytes(kv, max_group_rows, heads_q, &prefix);
    *bytes = sizeof(StatusWord) + std::max(own, prefix) + (size_t)rows * heads_q * (kv.dim + 2) * sizeof(float);
    return e;
}

cudaError_t launch_kv_attention_shared(const KvAttentionArgs &k, const int32_t *cu_groups, const int32_t *prefix_len,
                                       int groups, int max_group_rows, void *ws, cudaStream_t st) {
    AttnSetup s;
    cudaError_t e = set_up(k, ws, s);
    if (e != cudaSuccess) return e;
    size_t own = 0, prefix = 0;
    if ((e = part_bytes(k.kv, k.max_rows, k.heads_q, &own)) != cudaSuccess) return e;
    if ((e = part_bytes(k.kv, max_group_rows, k.heads_q, &prefix)) != cudaSuccess) return e;
    s.a.half = reinterpret_cast<float *>((char *)ws + sizeof(StatusWord) + std::max(own, prefix));
    s.a.half_ml = reinterpret_cast<float2 *>(s.a.half + (size_t)k.rows * k.heads_q * k.kv.dim);
    s.a.cu_groups = cu_groups;
    s.a.prefix_len = prefix_len;
    s.a.groups = groups;
    s.a.group_rows = max_group_rows;
    TraceScope trace_scope("kv_attention_shared", st);
    // (lengths are known on the device alone: by the most tiles that the tables have room for)
    const double tiles = (double)(((int64_t)k.table_width * k.kv.page + kTokens - 1) / kTokens) * k.seqs * s.a.nrt * k.kv.heads;
    if (tiles <= (double)kSmall * s.sms) {
        s.a.what = kWhole;
        return run(s, st);
    }
    AttnSetup t = s;
    t.a.what = kPrefixes;
    t.a.k.max_rows = max_group_rows;
    if ((e = set_tiles(t.a, groups)) != cudaSuccess || (e = run(t, st)) != cudaSuccess) return e;
    s.a.what = kOwn;
    return run(s, st);
}

}  // namespace moe
