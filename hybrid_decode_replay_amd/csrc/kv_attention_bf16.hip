// kv_attention_bf16.hip -- paged decode attention, bf16 io and cache.
#include "kv_attention_kernel.hpp"

namespace rs {

hipError_t launch_kv_attention_bf16(const KvAttention& a, const KvPlan& p, int D, hipStream_t s)
{
    return kv_attention_pick<KV_BF16, false>(a, p, D, s);
}

}  // namespace rs
