// kv_append.hip -- a step's rows on their way into the paged cache: q and k rotated, q written
// out, k and v written to their slots.
//
// A row is (Hq + 2 Hkv) heads of D channels.  Its work items are pairs of 16-byte chunks: in the
// halves style a chunk of eight channels and the chunk rot_dim / 2 further, so that both ends of
// eight rotated pairs are in one lane; elsewhere two chunks half a run apart, so that neighbouring
// lanes write neighbouring chunks (32-byte pieces per lane cost streamed stores 40 %).  The row's
// cosines and sines are formed once, in LDS, and serve all of its heads: the angle is pos * freq in
// fp64 as a fraction of a turn (exact to 2^-52 of the number of turns, so a position of 10^6 still has
// its angle to 10^-9), the fraction goes to sincospi in fp32 (off by at most 2^-26 of a turn, 1e-7
// radians, of the order of sine's and cosine's own fp32 roundings).
//
// Bound by HBM: q, k and v are read once and written once.  16387 rows of 32 + 2 x 8 heads of 128
// channels, 403 MB: 73 us, 5.5 TB/s, against 5.9 TB/s of a copy; on an E4M3 cache, 369 MB, 69 us.  1024 rows
// of 16 + 2 x 2 heads of 256 on an E4M3 cache 6.2 us, one row 2.9 (launch and three dependent loads).  Rows
// of more items than one pass holds wait for their next pass's loads: 64 + 2 x 8 heads of 128, 671 MB, 120
// us (5.6 TB/s), of 256 channels 255 us (5.3), 1024 such rows 11.5 and 17.4 us.  Idle rows are read (the loads
// do not wait for the slots): with a quarter of 16387 idle 107 us for 120.
#include <type_traits>

#include "kv_io.hpp"

namespace rs {

// Stores of large calls bypass the caches: nothing reads those rows again soon.
template <bool STREAM, typename T>
__device__ __forceinline__ void kv_store(T* p, T v)
{
    if constexpr (STREAM) __builtin_nontemporal_store(v, p);
    else *p = v;
}

// One 16-byte chunk in registers to the cache, as io elements or as E4M3 codes of x / scale.
template <int IO, bool FP8, bool STREAM>
__device__ __forceinline__ void store_cached(void* cache, size_t at, const float (&x)[8], float scale)
{
    if constexpr (FP8) {
        // a true division: the code is that of the correctly rounded quotient
        const u32x2 w = {pack_e4m3(f32x4{x[0] / scale, x[1] / scale, x[2] / scale, x[3] / scale}),
                         pack_e4m3(f32x4{x[4] / scale, x[5] / scale, x[6] / scale, x[7] / scale})};
        kv_store<STREAM>(reinterpret_cast<u32x2*>(static_cast<uint8_t*>(cache) + at), w);
    } else {
        kv_store<STREAM>(reinterpret_cast<u32x4*>(static_cast<uint16_t*>(cache) + at), kv_pack8<IO>(x));
    }
}

// R rows per workgroup, U items of a thread in flight at a time.  The first items are requested before
// the angles are formed.
template <int IO, bool FP8, int STYLE, int R, int U>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppend a, int log_items)
{
    __shared__ float2 turn[R][128];      // cos, sin of each rotated pair
    __shared__ int64_t slot[R];
    const int tid = threadIdx.x, row0 = blockIdx.x * R;
    const int pairs = a.rot >> 1, rot_items = a.rot >> 4;    // items of a head with rotated channels
    const int h0 = a.q ? 0 : a.Hq, heads = a.Hq - h0 + 2 * a.Hkv;
    const int per_row = heads << log_items;                  // D / 16 items per head
    const int total = min(R, a.rows - row0) * per_row;
    u32x4 w[U][2];
    // row, head and item of index i, and its two chunks' first channels
    struct Item {
        int r, h, it, c0, c1;
    };
    auto item = [&](int i) {
        Item x;
        x.r = 0;
#pragma unroll
        for (int k = 1; k < R; ++k) x.r += i >= k * per_row ? 1 : 0;
        const int j = i - x.r * per_row;
        x.h = h0 + (j >> log_items);
        x.it = j & ((1 << log_items) - 1);
        // neighbouring items are neighbouring chunks: halves of the rotated channels and of the rest, or
        // of the whole head where pairs are neighbours
        const bool rest = STYLE == KV_ROT_HALVES && x.it >= rot_items;
        x.c0 = 8 * (rest ? x.it + rot_items : x.it);
        x.c1 = x.c0 + (STYLE == KV_ROT_HALVES ? (rest ? (a.D - a.rot) >> 1 : pairs) : a.D >> 1);
        return x;
    };
    auto request = [&](int base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = base + u * 256;
            if (i >= total) continue;
            const Item x = item(i);
            const size_t row = (size_t)(row0 + x.r);
            const uint16_t* src;
            if (x.h < a.Hq) src = static_cast<const uint16_t*>(a.q) + row * a.q_stride + (size_t)x.h * a.D;
            else if (x.h < a.Hq + a.Hkv) src = static_cast<const uint16_t*>(a.k) + row * a.k_stride + (size_t)(x.h - a.Hq) * a.D;
            else src = static_cast<const uint16_t*>(a.v) + row * a.v_stride + (size_t)(x.h - a.Hq - a.Hkv) * a.D;
            w[u][0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src + x.c0));
            w[u][1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src + x.c1));
        }
    };
    if (tid < R) {
        int64_t s = row0 + tid < a.rows ? a.slots[row0 + tid] : -1;
        if (s >= a.nslots) {
            if (a.err) atomicOr(a.err, KVERR_BAD_SLOT);
            s = -1;
        }
        slot[tid] = s;
    }
    request(tid);
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
#pragma unroll 1
    for (int base = tid; base < total; base += 256 * U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (base + u * 256 >= total) continue;
            const Item t = item(base + u * 256);
            const int64_t sl = slot[t.r];
            if (sl < 0) continue;
            const bool is_q = t.h < a.Hq, is_k = !is_q && t.h < a.Hq + a.Hkv;
            float x[8], y[8];
            kv_unpack8<IO>(w[u][0], x);
            kv_unpack8<IO>(w[u][1], y);
            if (is_q || is_k) {
                if (STYLE == KV_ROT_HALVES && t.it < rot_items) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 cs = turn[t.r][t.c0 + e];
                        const float p = x[e], q = y[e];
                        x[e] = p * cs.x - q * cs.y;
                        y[e] = q * cs.x + p * cs.y;
                    }
                }
                if constexpr (STYLE == KV_ROT_ADJACENT) {
                    auto turn_chunk = [&](float (&z)[8], int c) {
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const float2 cs = turn[t.r][(c + e) >> 1];
                            const float p = z[e], q = z[e + 1];
                            z[e] = p * cs.x - q * cs.y;
                            z[e + 1] = q * cs.x + p * cs.y;
                        }
                    };
                    if (t.c0 < a.rot) turn_chunk(x, t.c0);
                    if (t.c1 < a.rot) turn_chunk(y, t.c1);
                }
            }
            constexpr bool STREAM = R > 1;
            if (is_q) {
                uint16_t* dst = static_cast<uint16_t*>(a.q_out) + ((size_t)(row0 + t.r) * a.Hq + t.h) * a.D;
                kv_store<STREAM>(reinterpret_cast<u32x4*>(dst + t.c0), kv_pack8<IO>(x));
                kv_store<STREAM>(reinterpret_cast<u32x4*>(dst + t.c1), kv_pack8<IO>(y));
            } else {
                const int hk = t.h - a.Hq - (is_k ? 0 : a.Hkv);
                void* cache = is_k ? a.K : a.V;
                const size_t page = (size_t)(sl >> a.page_shift), off = (size_t)sl & ((1u << a.page_shift) - 1);
                const size_t at = (((page * a.Hkv + hk) << a.page_shift) + off) * a.D;
                const float scale = FP8 ? (is_k ? a.k_scale : a.v_scale)[hk] : 1.f;
                store_cached<IO, FP8, STREAM>(cache, at + t.c0, x, scale);
                store_cached<IO, FP8, STREAM>(cache, at + t.c1, y, scale);
            }
        }
        if (base + 256 * U < total) request(base + 256 * U);
    }
}

template <int IO, bool FP8, int STYLE>
static void start(const KvAppend& a, hipStream_t s)
{
    const int log_items = a.D == 64 ? 2 : (a.D == 128 ? 3 : 4);
    // Up to some rows a CU the latency of one counts, and what they write is read by the attention that
    // follows; past that two rows share a workgroup (2048 rows 11.4 us with four, 9.4 with two), and
    // streamed stores pay (16387 rows 80 -> 73 us).
    if (a.rows <= 1024) {
        hipLaunchKernelGGL((kv_append_kernel<IO, FP8, STYLE, 1, 2>), dim3(a.rows), dim3(256), 0, s, a, log_items);
    } else {
        hipLaunchKernelGGL((kv_append_kernel<IO, FP8, STYLE, 2, 3>), dim3((a.rows + 1) / 2), dim3(256), 0, s, a, log_items);
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
