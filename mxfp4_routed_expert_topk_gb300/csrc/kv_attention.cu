// Cache attention: the choice between its two forms, and what is set up for both.
#include <algorithm>

#include "kv_attention_few.cuh"

namespace moe {
cudaError_t set_wait_limit_kv_attention(uint64_t ns) {
    const cudaError_t e = set_wait_limit_here(ns);
    if (e != cudaSuccess) return e;
    const cudaError_t r = set_wait_limit_kv_attention_rows(ns);
    return r != cudaSuccess ? r : set_wait_limit_kv_attention_shared(ns);
}

cudaError_t kv_attention_workspace_bytes(const KvView &kv, int max_rows, int heads_q, size_t *bytes) {
    size_t part = 0;
    const cudaError_t e = part_bytes(kv, max_rows, heads_q, &part);
    *bytes = sizeof(StatusWord) + part;
    return e;
}

cudaError_t launch_kv_attention(const KvAttentionArgs &k, void *ws, cudaStream_t st) {
    AttnSetup s;
    const cudaError_t e = set_up(k, ws, s);
    if (e != cudaSuccess) return e;
    TraceScope trace_scope("kv_attention", st);
    if (s.a.rpt > kFewRows) return launch_attention_rows(s.tm, s.a, s.sms, s.smem_max, st);
    return launch_few_of<false>(s.tm, s.a, s.sms, s.smem_max, st);
}

}  // namespace moe
