// kv_io.hpp -- element types of the paged key/value cache kernels.
#pragma once
#include "common.hpp"
#include "kv.hpp"
#include "rc.hpp"

namespace rs {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two fp32 values as a pair of io elements (round to nearest even), and back.
template <int IO>
__device__ __forceinline__ uint32_t kv_pack(float a, float b)
{
    if constexpr (IO == KV_BF16) return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
    else return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
}
template <int IO>
__device__ __forceinline__ void kv_unpack(uint32_t w, float& a, float& b)
{
    if constexpr (IO == KV_BF16) {
        a = __builtin_bit_cast(float, w << 16);
        b = __builtin_bit_cast(float, w & 0xffff0000u);
    } else {
        const f16x2 h = __builtin_bit_cast(f16x2, w);
        a = (float)h.x;
        b = (float)h.y;
    }
}
// Eight consecutive io elements.
template <int IO>
__device__ __forceinline__ void kv_unpack8(u32x4 w, float (&x)[8])
{
    kv_unpack<IO>(w.x, x[0], x[1]);
    kv_unpack<IO>(w.y, x[2], x[3]);
    kv_unpack<IO>(w.z, x[4], x[5]);
    kv_unpack<IO>(w.w, x[6], x[7]);
}
template <int IO>
__device__ __forceinline__ u32x4 kv_pack8(const float (&x)[8])
{
    return u32x4{kv_pack<IO>(x[0], x[1]), kv_pack<IO>(x[2], x[3]), kv_pack<IO>(x[4], x[5]), kv_pack<IO>(x[6], x[7])};
}

}  // namespace rs
