// kv_attention_f16_fp8.hip -- paged decode attention, fp16 io, E4M3 cache.
#include "kv_attention_kernel.hpp"

namespace rs {

hipError_t launch_kv_attention_f16_fp8(const KvAttention& a, const KvPlan& p, int D, hipStream_t s)
{
    return kv_attention_pick<KV_F16, true>(a, p, D, s);
}

}  // namespace rs
