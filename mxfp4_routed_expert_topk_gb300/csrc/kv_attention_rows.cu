// Cache attention, the form for row tiles of more than 16 rows.
#include "kv_attention_rows.cuh"

namespace moe {

cudaError_t set_wait_limit_kv_attention_rows(uint64_t ns) { return set_wait_limit_here(ns); }

cudaError_t launch_attention_rows(const CUtensorMap &tm, AttnArgs a, int sms, int smem_max, cudaStream_t st) {
    return launch_rows<false>(tm, a, sms, smem_max, st);
}

}  // namespace moe
