// gdn_prefill.hip -- the gated delta rule over packed prompts, token by token (replay_gdn_prefill).
//
//   e = v - alpha S k,  S = alpha S + beta e k^T,  o = scale S q
//
// Rows of S (channels of d_v) do not depend on one another: 16 lanes hold a row's d_k values in registers, a wave 4 RPL
// rows.  The inputs of the next token are on their way while one is computed.  Bound by that chain of a token: 0.6 us each (bf16,
// 32 heads of 128 x 128: 32768 tokens of one sequence 20.3 ms, where chunks on the matrix cores take 1.2), so it is the way of
// what the chunks do not take: fp32 inputs, whose products would need three times the terms, and d_k below 64.
#include "common.hpp"
#include "mixer.hpp"

namespace rs {

// EL consecutive io values at p (aligned to their size).
template <int IO, int EL>
__device__ __forceinline__ void ld_row(const void* p, float (&x)[EL])
{
    if constexpr (IO == IO_F32) {
        lds_row_load<EL>(static_cast<const float*>(p), x);
    } else {
        struct __attribute__((aligned(EL >= 8 ? 16 : 2 * EL))) { uint16_t v[EL]; } t;
        __builtin_memcpy(&t, __builtin_assume_aligned(p, EL >= 8 ? 16 : 2 * EL), sizeof t);
#pragma unroll
        for (int i = 0; i < EL; ++i) x[i] = bf16_bits_to_f32(t.v[i]);
    }
}

template <int IO, int EL, int RPL>
__global__ void __launch_bounds__(256) gdn_tokens_kernel(PrefillArgs a, int slices)
{
    const int lane = threadIdx.x & 15, slice = blockIdx.x % slices, bh = blockIdx.x / slices, b = bh / a.H, h = bh - b * a.H;
    const int row = (slice * 16 + (threadIdx.x >> 4)) * RPL;       // the first of this lane's rows
    if (row >= a.C) return;                                        // (d_v is a multiple of 16, RPL of 1, 2 or 4)
    constexpr int R = 16 * EL;
    const int g = h / a.hpg;
    int first = min(max(a.starts[b], 0), a.rows), last = min(max(a.starts[b + 1], 0), a.rows);
    const size_t at = ((size_t)bh * a.C + row) * R + lane * EL;
    float S[RPL][EL];
#pragma unroll
    for (int i = 0; i < RPL; ++i) {
        if (a.S_in) {
            lds_row_load<EL>(a.S_in + at + (size_t)i * R, S[i]);
        } else {
#pragma unroll
            for (int j = 0; j < EL; ++j) S[i][j] = 0.f;
        }
    }
    constexpr int SZ = IO == IO_F32 ? 4 : 2;
    const char* qp = static_cast<const char*>(a.q) + ((int64_t)first * a.q_stride + g * R + lane * EL) * SZ;
    const char* kp = static_cast<const char*>(a.k) + ((int64_t)first * a.k_stride + g * R + lane * EL) * SZ;
    const char* vp = static_cast<const char*>(a.v) + ((int64_t)first * a.v_stride + h * a.C + row) * SZ;
    float q[EL], k[EL], v[RPL], alpha = 0.f, beta = 0.f;
    auto fetch = [&](int t) {
        ld_row<IO>(qp, q);
        ld_row<IO>(kp, k);
        ld_row<IO>(vp, v);
        alpha = a.alpha[(size_t)t * a.H + h];
        beta = a.beta[(size_t)t * a.H + h];
        qp += a.q_stride * SZ;
        kp += a.k_stride * SZ;
        vp += a.v_stride * SZ;
    };
    if (first < last) fetch(first);
    for (int t = first; t < last; ++t) {
        float cq[EL], ck[EL], cv[RPL];
#pragma unroll
        for (int j = 0; j < EL; ++j) {
            cq[j] = q[j];
            ck[j] = k[j];
        }
#pragma unroll
        for (int i = 0; i < RPL; ++i) cv[i] = v[i];
        const float ca = alpha, cb = beta;
        if (t + 1 < last) fetch(t + 1);
        float y[RPL];
#pragma unroll
        for (int i = 0; i < RPL; ++i) {
            float d = 0.f;
#pragma unroll
            for (int j = 0; j < EL; ++j) {
                S[i][j] *= ca;
                d = __builtin_fmaf(S[i][j], ck[j], d);
            }
            const float u = cb * (cv[i] - group_sum<16>(d));
            float o = 0.f;
#pragma unroll
            for (int j = 0; j < EL; ++j) {
                S[i][j] = __builtin_fmaf(u, ck[j], S[i][j]);
                o = __builtin_fmaf(S[i][j], cq[j], o);
            }
            y[i] = a.scale * group_sum<16>(o);
        }
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < RPL; ++i) st_io<IO>(a.o, ((size_t)t * a.H + h) * a.C + row + i, y[i]);
        }
    }
    if (a.S_out) {
#pragma unroll
        for (int i = 0; i < RPL; ++i) lds_row_store<EL>(a.S_out + at + (size_t)i * R, S[i]);
    }
}

namespace {

template <int IO, int EL>
hipError_t run(const PrefillArgs& a, hipStream_t s)
{
    const uint32_t heads = (uint32_t)a.B * a.H;
    // one row a lane where that fills the chip no more than once, else four: the loads of q and k serve more rows
    if (heads * (a.C / 16) <= 256 || EL == 16) {
        const int slices = a.C / 16;
        gdn_tokens_kernel<IO, EL, 1><<<heads * slices, 256, 0, s>>>(a, slices);
    } else {
        const int slices = (a.C + 63) / 64;
        gdn_tokens_kernel<IO, EL, 4><<<heads * slices, 256, 0, s>>>(a, slices);
    }
    return hipGetLastError();
}

template <int IO>
hipError_t pick(const PrefillArgs& a, hipStream_t s)
{
    switch (a.R) {
    case 16: return run<IO, 1>(a, s);
    case 32: return run<IO, 2>(a, s);
    case 64: return run<IO, 4>(a, s);
    case 128: return run<IO, 8>(a, s);
    default: return run<IO, 16>(a, s);
    }
}

}  // namespace

hipError_t launch_gdn_prefill_tokens(const PrefillArgs& a, bool f32, hipStream_t s)
{
    return f32 ? pick<IO_F32>(a, s) : pick<IO_BF16>(a, s);
}

}  // namespace rs
