// kv_append.hip -- a step's rows on their way into the paged cache: q and k rotated, q written
// out, k and v written to their slots.
//
// A row is (Hq + 2 Hkv) heads of D channels.  Its work items are pairs of 16-byte chunks: in the
// halves style a chunk of eight channels and the chunk rot_dim / 2 further, so that both ends of
// eight rotated pairs are in one lane; elsewhere two neighbouring chunks.  The row's cosines and
// sines are formed once, in LDS, and serve all of its heads: the angle is pos * freq in fp64 as a
// fraction of a turn (exact to 2^-52 of the number of turns, so a position of 10^6 still has its
// angle to 10^-9), the fraction goes to sincospi in fp32.
//
// Bound by HBM: q, k and v are read once and written once.
#include <type_traits>

#include "kv_io.hpp"

namespace rs {

// One 16-byte chunk in registers to the cache, as io elements or as E4M3 codes of x / scale.
template <int IO, bool FP8>
__device__ __forceinline__ void store_cached(void* cache, size_t at, const float (&x)[8], float scale)
{
    if constexpr (FP8) {
        // a true division: the code is that of the correctly rounded quotient
        const u32x2 w = {pack_e4m3(f32x4{x[0] / scale, x[1] / scale, x[2] / scale, x[3] / scale}),
                         pack_e4m3(f32x4{x[4] / scale, x[5] / scale, x[6] / scale, x[7] / scale})};
        *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(cache) + at) = w;
    } else {
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(cache) + at) = kv_pack8<IO>(x);
    }
}

// R rows per workgroup.
template <int IO, bool FP8, int STYLE, int R>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppend a, int log_items)
{
    __shared__ float2 turn[R][128];      // cos, sin of each rotated pair
    __shared__ int64_t slot[R];
    const int tid = threadIdx.x, row0 = blockIdx.x * R;
    const int pairs = a.rot >> 1;
    if (tid < R) {
        int64_t s = row0 + tid < a.rows ? a.slots[row0 + tid] : -1;
        if (s >= a.nslots) {
            if (a.err) atomicOr(a.err, KVERR_BAD_SLOT);
            s = -1;
        }
        slot[tid] = s;
    }
    for (int i = tid; i < R * pairs; i += 256) {
        const int r = i / pairs, p = i - r * pairs;
        if (row0 + r < a.rows) {
            const int ax = a.axis ? a.axis[p] : 0;
            float2 cs = {1.f, 0.f};
            if (ax < a.naxes) {
                const double turns = (double)a.pos[(size_t)ax * a.rows + row0 + r] *
                                     ((double)a.freq[p] * 0.15915494309189533577);      // 1 / (2 pi)
                const float f = (float)(turns - __builtin_rint(turns));
                sincospif(2.f * f, &cs.y, &cs.x);
            }
            turn[r][p] = cs;
        }
    }
    __syncthreads();
    const int heads = (a.q ? a.Hq : 0) + 2 * a.Hkv;
    const int per_row = heads << log_items;                  // D / 16 items per head
    const int rot_items = a.rot >> 4;                        // items of a head with rotated channels
    const int h0 = a.q ? 0 : a.Hq;
#pragma unroll 1
    for (int i = tid; i < R * per_row; i += 256) {
        const int r = R == 1 ? 0 : i / per_row;
        const int64_t sl = slot[r];
        if (sl < 0) continue;
        const int j = i - r * per_row;
        const int h = h0 + (j >> log_items), it = j & ((1 << log_items) - 1);
        const size_t row = (size_t)(row0 + r);
        const uint16_t* src;
        int hk = 0;
        if (h < a.Hq) src = static_cast<const uint16_t*>(a.q) + row * a.q_stride + (size_t)h * a.D;
        else if (h < a.Hq + a.Hkv) src = static_cast<const uint16_t*>(a.k) + row * a.k_stride + (size_t)(hk = h - a.Hq) * a.D;
        else src = static_cast<const uint16_t*>(a.v) + row * a.v_stride + (size_t)(hk = h - a.Hq - a.Hkv) * a.D;
        const bool turned = it < rot_items && h < a.Hq + a.Hkv;
        // the item's two chunks (first channel of each)
        const bool apart = STYLE == KV_ROT_HALVES && it < rot_items;
        const int c0 = apart ? 8 * it : 16 * it, c1 = apart ? c0 + pairs : c0 + 8;
        float x[8], y[8];
        kv_unpack8<IO>(__builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src + c0)), x);
        kv_unpack8<IO>(__builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src + c1)), y);
        if (turned) {
            if constexpr (STYLE == KV_ROT_HALVES) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 cs = turn[r][c0 + e];
                    const float u = x[e], w = y[e];
                    x[e] = u * cs.x - w * cs.y;
                    y[e] = w * cs.x + u * cs.y;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 c = turn[r][(c0 + e) >> 1], d = turn[r][(c1 + e) >> 1];
                    const float u = x[e], w = x[e + 1], s = y[e], t = y[e + 1];
                    x[e] = u * c.x - w * c.y;
                    x[e + 1] = w * c.x + u * c.y;
                    y[e] = s * d.x - t * d.y;
                    y[e + 1] = t * d.x + s * d.y;
                }
            }
        }
        if (h < a.Hq) {
            uint16_t* dst = static_cast<uint16_t*>(a.q_out) + (row * a.Hq + h) * a.D;
            *reinterpret_cast<u32x4*>(dst + c0) = kv_pack8<IO>(x);
            *reinterpret_cast<u32x4*>(dst + c1) = kv_pack8<IO>(y);
        } else {
            const bool is_k = h < a.Hq + a.Hkv;
            void* cache = is_k ? a.K : a.V;
            const size_t page = (size_t)(sl >> a.page_shift), off = (size_t)sl & ((1u << a.page_shift) - 1);
            const size_t at = (((page * a.Hkv + hk) << a.page_shift) + off) * a.D;
            const float scale = FP8 ? (is_k ? a.k_scale : a.v_scale)[hk] : 1.f;
            store_cached<IO, FP8>(cache, at + c0, x, scale);
            store_cached<IO, FP8>(cache, at + c1, y, scale);
        }
    }
}

template <int IO, bool FP8, int STYLE>
static void start(const KvAppend& a, hipStream_t s)
{
    const int log_items = a.D == 64 ? 2 : (a.D == 128 ? 3 : 4);
    if (a.rows <= 1024) {
        hipLaunchKernelGGL((kv_append_kernel<IO, FP8, STYLE, 1>), dim3(a.rows), dim3(256), 0, s, a, log_items);
    } else {
        hipLaunchKernelGGL((kv_append_kernel<IO, FP8, STYLE, 4>), dim3((a.rows + 3) / 4), dim3(256), 0, s, a, log_items);
    }
}

hipError_t launch_kv_append(const KvAppend& a, int io, bool fp8, int style, hipStream_t s)
{
    auto with = [&](auto iot, auto f8) {
        if (style == KV_ROT_HALVES) start<decltype(iot)::value, decltype(f8)::value, KV_ROT_HALVES>(a, s);
        else start<decltype(iot)::value, decltype(f8)::value, KV_ROT_ADJACENT>(a, s);
    };
    using std::integral_constant;
    if (io == KV_BF16) {
        if (fp8) with(integral_constant<int, KV_BF16>{}, integral_constant<bool, true>{});
        else with(integral_constant<int, KV_BF16>{}, integral_constant<bool, false>{});
    } else {
        if (fp8) with(integral_constant<int, KV_F16>{}, integral_constant<bool, true>{});
        else with(integral_constant<int, KV_F16>{}, integral_constant<bool, false>{});
    }
    return hipGetLastError();
}

}  // namespace rs
