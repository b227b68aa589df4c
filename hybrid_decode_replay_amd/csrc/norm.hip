// norm.hip -- root-mean-square norm with the residual's addition (replay_norm).
//
//   s = x + res,  y = s / sqrt(mean s^2 + eps) * w,  y as 16-bit values or E4M3 codes with a scale per 128 channels.
//
// One pass: a run of n channels is held in the registers of the lanes that share it (eight consecutive channels a lane
// and step), so x and res are read once and sum, y and the scales written once.  HBM bound: 6 bytes read and written a
// value (no residual: 2) and 1 or 2 of y, against some 20 instructions.  16387 rows of 4096 bf16 channels with a residual to
// E4M3 (472 MB) 73 us, 6.4 TB/s; 262144 heads of 128 (134 MB) 22.6 us, 5.9 TB/s; one row 3.1 us, 256 rows 4.6 us (a run of 4096
// channels needs 256 lanes for that: a wave would hold 64 values a lane and wait for them eight loads at a time).
#include "kv_io.hpp"
#include "mixer.hpp"

namespace rs {

// Largest of the 16 lanes of a row of lanes, for every one of them.
__device__ __forceinline__ float max16(float v)
{
    v = fmaxf(v, dpp_mov<DPP_QUAD_XOR1>(v));
    v = fmaxf(v, dpp_mov<DPP_QUAD_XOR2>(v));
    v = fmaxf(v, dpp_mov<DPP_ROW_HALF_MIRROR>(v));
    return fmaxf(v, dpp_mov<DPP_ROW_MIRROR>(v));
}

// An infinity as the largest finite number (NaN stays): the scale stays finite and the codes saturate.
__device__ __forceinline__ float finite(float v)
{
    return __builtin_fabsf(v) == __builtin_inff() ? __builtin_copysignf(3.40282346638528859812e38f, v) : v;
}

// LPR lanes share a run: 16, 32 or 64 of a wave (several runs a wave), or a workgroup of 256.  NC steps of 8 channels a
// lane.  Chunk i of a lane is lane + i * LPR, so 16 neighbouring lanes hold 128 consecutive channels: one E4M3 group.
template <int IO, bool FP8, int LPR, int NC>
__global__ void __launch_bounds__(256) norm_kernel(NormArgs a)
{
    constexpr int RUNS = 256 / LPR;                   // runs of a workgroup
    const int lane = threadIdx.x % LPR;
    const uint32_t run = blockIdx.x * RUNS + threadIdx.x / LPR;
    const bool live = run < a.runs;
    const uint32_t at = live ? run : a.runs - 1;
    const uint32_t row = a.heads == 1 ? at : a.mg_heads ? div_magic(at, a.mg_heads) : at / a.heads, head = at - row * a.heads;
    const int chunks = a.n >> 3;
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + (int64_t)row * a.x_stride + (int64_t)head * a.n;
    const uint16_t* res = a.res ? static_cast<const uint16_t*>(a.res) + (int64_t)row * a.res_stride + (int64_t)head * a.n : nullptr;
    const size_t out = (size_t)at * a.n;              // (outputs are contiguous: run after run)

    u32x4 wx[NC], wr[NC], ww[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = lane + i * LPR;
        wx[i] = wr[i] = ww[i] = u32x4{0, 0, 0, 0};
        if (c < chunks) {
            wx[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(x) + c);
            if (res) wr[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(res) + c);
            if (a.weight) ww[i] = reinterpret_cast<const u32x4*>(a.weight)[c];
        }
    }
    float s[NC][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        kv_unpack8<IO>(wx[i], s[i]);
        if (res) {
            float r[8];
            kv_unpack8<IO>(wr[i], r);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[i][j] += r[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(s[i][j], s[i][j], ss);
        const int c = lane + i * LPR;
        if (a.sum && live && c < chunks)
            __builtin_nontemporal_store(kv_pack8<IO>(s[i]), reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.sum) + out) + c);
    }
    auto run_sum = [](float v) {
        if constexpr (LPR <= 64) {
            return group_sum<LPR>(v);
        } else {
            __shared__ float part[4];
            v = group_sum<64>(v);
            if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
            __syncthreads();
            return (part[0] + part[1]) + (part[2] + part[3]);
        }
    };
    float mean = __builtin_fmaf(run_sum(ss), a.inv_n, a.eps);
    // A run whose squares left the fp32 range (their sum is an infinity, or so small that squares lost bits and eps does not
    // cover it) once more, times a power of two.  (Runs beside it in a wave take part with 1, so that no lane is apart.)
    constexpr uint32_t LOW = 27u << 23, END = 0x7f800000u;         // 2^-100, infinity
    const bool out_of_range = __builtin_bit_cast(uint32_t, mean) - LOW >= END - LOW;
    if (__builtin_expect(__ballot(out_of_range) != 0, 0)) {
        const float p = !out_of_range ? 1.f : mean < 1.f ? 0x1p100f : 0x1p-80f;
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[i][j] *= p;
                ss = __builtin_fmaf(s[i][j], s[i][j], ss);
            }
        if constexpr (LPR > 64) __syncthreads();
        mean = __builtin_fmaf(run_sum(ss), a.inv_n, a.eps * p * p);
    }
    // (the square root and the division are rounded to fp32 each: E4M3 scales are fp32 outputs)
    const float inv = 1.f / __builtin_sqrtf(mean);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = lane + i * LPR;
        float w[8];
        if (a.weight) {
            kv_unpack8<IO>(ww[i], w);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[i][j] *= inv * w[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) s[i][j] *= inv;
        }
        if constexpr (!FP8) {
            if (live && c < chunks)
                __builtin_nontemporal_store(kv_pack8<IO>(s[i]), reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.y) + out) + c);
        } else {
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[i][j] = finite(s[i][j]);
                top = fmaxf(top, __builtin_fabsf(s[i][j]));
            }
            top = max16(top);                          // (n is a multiple of 128: whole groups of lanes are past the end)
            const float scale = fmaxf(top / 448.f, 1.17549435e-38f), r = 1.f / scale;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // y / scale to the last place: the product's rest once more
                const float q = s[i][j] * r;
                s[i][j] = __builtin_fmaf(__builtin_fmaf(-q, scale, s[i][j]), r, q);
            }
            if (live && c < chunks) {
                const u32x2 codes = {pack_e4m3(f32x4{s[i][0], s[i][1], s[i][2], s[i][3]}),
                                     pack_e4m3(f32x4{s[i][4], s[i][5], s[i][6], s[i][7]})};
                reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.y) + out)[c] = codes;
                if ((lane & 15) == 0) a.y_scale[(out >> 7) + (c >> 4)] = scale;
            }
        }
    }
}

namespace {

template <int IO, bool FP8, int LPR, int NC>
hipError_t run(const NormArgs& a, hipStream_t s)
{
    constexpr uint32_t RUNS = 256 / LPR;
    norm_kernel<IO, FP8, LPR, NC><<<(a.runs + RUNS - 1) / RUNS, 256, 0, s>>>(a);
    return hipGetLastError();
}

template <int IO, bool FP8>
hipError_t pick(const NormArgs& a, hipStream_t s)
{
    if (a.n <= 128) return run<IO, FP8, 16, 1>(a, s);
    if (a.n <= 256) return run<IO, FP8, 32, 1>(a, s);
    if (a.n <= 512) return run<IO, FP8, 64, 1>(a, s);
    if (a.n <= 1024) return run<IO, FP8, 64, 2>(a, s);
    if (a.n <= 2048) return run<IO, FP8, 256, 1>(a, s);
    if (a.n <= 4096) return run<IO, FP8, 256, 2>(a, s);
    if (a.n <= 8192) return run<IO, FP8, 256, 4>(a, s);
    return run<IO, FP8, 256, 8>(a, s);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, int io, bool fp8, hipStream_t s)
{
    if (io == MIX_BF16) return fp8 ? pick<KV_BF16, true>(a, s) : pick<KV_BF16, false>(a, s);
    return fp8 ? pick<KV_F16, true>(a, s) : pick<KV_F16, false>(a, s);
}

}  // namespace rs
