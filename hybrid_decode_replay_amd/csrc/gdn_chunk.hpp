// gdn_chunk.hpp -- what the chunked and the short prompt kernels of the gated delta rule share: the order of rows in a tile,
// sequences' spans, fp32 operands as bf16 terms.
#pragma once
#include "common.hpp"
#include "mixer.hpp"

namespace rs {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int CHUNK = GDN_CHUNK;
static_assert(CHUNK == 64, "tiles and fragments are laid out for 64 tokens");
constexpr int FRAGS = 6;                       // (row tile, 32 tokens) pairs of a lower triangle: 0, 1, 2 x 2, 3 x 2
constexpr int PIECE_P = 3 * FRAGS, PIECE_G = 5 * FRAGS;      // 1 KiB pieces: T (three terms), P (fp32), the g's
static_assert((PIECE_G + 1) * 1024 == GDN_CHUNK_BYTES, "layout of a chunk in the workspace");

// Token of row r of tile t (and d_k channel, of the state's tiles).
__device__ __forceinline__ constexpr int tile_row(int t, int r) { return 32 * (t >> 1) + 8 * (r >> 2) + 4 * (t & 1) + (r & 3); }

// Where a row of k or q stands in LDS: its 16-byte chunks are exchanged by its place in its tile, so that the 16 rows of an
// operand, and the four rows of each of a wave's reads across, are spread over the banks.
__device__ __forceinline__ constexpr int spread(int row) { return (row & 3) | ((row >> 1) & 12); }

// Rows of sequence b.
struct Span {
    int first, count;
};
__device__ __forceinline__ Span span_of(const PrefillArgs& a, int b)
{
    const int lo = min(max(a.starts[b], 0), a.rows), hi = min(max(a.starts[b + 1], 0), a.rows);
    return Span{lo, max(hi - lo, 0)};
}

// The k-th of the chunked kernels' sequences, and how many of them are before it; of up to 64 the k-th by length, the longest
// first: a launch's last workgroups are then its shortest.  b -1: there is none.  Sequence b's chunks stand in the workspace
// from first / 64 + ahead on: ranges of rows that do not overlap have chunks of their own there, and as ahead is below
// `most` none is past its end.
struct Turn {
    int b, ahead;
};
__device__ __forceinline__ Turn turn_of(const PrefillArgs& a, int k)
{
    if (a.skip < 0 && (a.B == 1 || a.B > 64)) return Turn{k, k};
    const int lane = lane_id();
    if (a.B > 64) {
        int n = 0;
        for (int b0 = 0; b0 < a.B; b0 += 64) {
            const int i = b0 + lane;
            const uint64_t mask = __ballot(i < a.B && span_of(a, min(i, a.B - 1)).count > a.skip);
            const int here = __popcll(mask);
            if (k < n + here) {
                const bool it = (mask >> lane & 1) && __popcll(mask & ((1ull << lane) - 1)) == k - n;
                return Turn{b0 + (int)__builtin_ctzll(__ballot(it)), k};
            }
            n += here;
        }
        return Turn{-1, 0};
    }
    const int mine = lane < a.B ? span_of(a, lane).count : -1;
    int rank = 0;
    for (int i = 0; i < a.B; ++i) {
        const int c = __builtin_amdgcn_readlane(mine, i);
        rank += c > mine || (c == mine && i < lane);
    }
    const int b = __builtin_ctzll(__ballot(lane < a.B && rank == k));
    const uint64_t taken = __ballot(lane < a.B && mine > a.skip);
    if (!(taken >> b & 1)) return Turn{-1, 0};
    return Turn{b, (int)__popcll(taken & ((1ull << b) - 1))};
}

// x as bf16 terms cut off eight bits at a time (hi + mid + lo is x), four values to two words of each term.
struct Cut {
    u32x2 t[3];
};
__device__ __forceinline__ Cut cut(f32x4 x)
{
    Cut c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float x0 = x[2 * i], x1 = x[2 * i + 1];
#pragma unroll
        for (int e = 0; e < 3; ++e) {
            const uint32_t a = __builtin_bit_cast(uint32_t, x0), b = __builtin_bit_cast(uint32_t, x1);
            c.t[e][i] = __builtin_amdgcn_perm(b, a, 0x07060302u);          // the upper halves of a and b
            x0 -= __builtin_bit_cast(float, a & 0xffff0000u);
            x1 -= __builtin_bit_cast(float, b & 0xffff0000u);
        }
    }
    return c;
}
__device__ __forceinline__ bf16x8 join(u32x2 lo, u32x2 hi) { return __builtin_bit_cast(bf16x8, u32x4{lo.x, lo.y, hi.x, hi.y}); }
struct Terms3 {
    bf16x8 t[3];
};
__device__ __forceinline__ Terms3 cut3(f32x4 lo, f32x4 hi)
{
    const Cut a = cut(lo), b = cut(hi);
    return Terms3{{join(a.t[0], b.t[0]), join(a.t[1], b.t[1]), join(a.t[2], b.t[2])}};
}
__device__ __forceinline__ Terms3 cut3(const float (&x)[8])
{
    return cut3(f32x4{x[0], x[1], x[2], x[3]}, f32x4{x[4], x[5], x[6], x[7]});
}

// A product of two operands in terms, down to 2^-24: a sum for each size of term, the smallest joined first.
__device__ __forceinline__ void product24(const bf16x8 (&x)[3], const bf16x8 (&y)[3], f32x4 (&sum)[3])
{
#pragma unroll
    for (int e = 0; e < 3; ++e) sum[e] = mfma16x16x32bf16(x[0], y[e], sum[e]);
    sum[0] = mfma16x16x32bf16(x[2], y[0], sum[0]);
#pragma unroll
    for (int e = 0; e < 2; ++e) sum[2 - e] = mfma16x16x32bf16(x[1], y[e], sum[2 - e]);
}
__device__ __forceinline__ f32x4 product24(const Terms3& x, const Terms3& y)
{
    f32x4 sum[3] = {};
    product24(x.t, y.t, sum);
    return sum[0] + (sum[1] + sum[2]);
}

// Four rows of 16 values each, read across: lane (r, q) gets column r of the four rows that its group of 16 lanes points at,
// lane j of a group at values 4 (j % 4) .. of row j / 4.
__device__ __forceinline__ u32x2 read_across(const uint8_t* p)
{
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)p));
}

// A kernel's first argument, read once more: what is worked out of it is not kept in scalar registers from the start on.
__device__ __forceinline__ const PrefillArgs& args_again()
{
    auto from = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(from));
    return *(const PrefillArgs*)from;
}

// Sums over lanes 0 .. lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ double lanes_before(double x)
{
    const u32x2 w = __builtin_bit_cast(u32x2, x);
    const u32x2 y = {(uint32_t)__builtin_amdgcn_update_dpp(0, (int)w.x, CTRL, ROWS, 0xf, false),
                     (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w.y, CTRL, ROWS, 0xf, false)};
    return __builtin_bit_cast(double, y);
}
__device__ __forceinline__ double prefix_sum(double x)
{
    x += lanes_before<0x111, 0xf>(x);              // within rows of 16: 1, 2, 4, 8 lanes on
    x += lanes_before<0x112, 0xf>(x);
    x += lanes_before<0x114, 0xf>(x);
    x += lanes_before<0x118, 0xf>(x);
    x += lanes_before<0x142, 0xa>(x);              // a row's last lane to the next row (of 1 and 3),
    return x + lanes_before<0x143, 0xc>(x);        // lane 31 to the rows behind it
}

// The g's of a chunk (products of alpha over its tokens up to each) as powers of two, 2^(whole + part): sums of log2 alpha in
// 64 bits, whose whole part is kept apart, so that the ratio of two g's is as near for far tokens as for near ones.  The
// logarithm is alpha's exponent and the fp32 logarithm of a mantissa in [1/sqrt 2, sqrt 2): off by some 2^-25 a token whatever
// alpha is, as a product of the alphas in fp32 would be.  alpha 0 counts as 2^-200 (no fp32 number is left after it); tokens
// that are not live keep the state.
struct Power {
    int whole;
    float part;
};
__device__ __forceinline__ Power decay_of(float alpha, bool live)
{
    float m = __builtin_amdgcn_frexp_mantf(alpha);
    int e = __builtin_amdgcn_frexp_expf(alpha);
    if (m < 0.70710678f) {
        m += m;
        --e;
    }
    const double l = (double)log2f(m) + (double)e;
    const double x = prefix_sum(!live ? 0.0 : l < -200.0 ? -200.0 : l);
    const double w = floor(fmax(fmin(x, 16384.0), -16384.0));      // (of an infinity or NaN: the part is one)
    return Power{(int)w, (float)(x - w)};
}
// 2^(whole + part), parts being differences of two: within 1 of 0.
__device__ __forceinline__ float power(int whole, float part) { return __builtin_ldexpf(__builtin_amdgcn_exp2f(part), whole); }

// 0, or 1 where x is an infinity or NaN.
__device__ __forceinline__ int not_finite(float x) { return (__builtin_bit_cast(uint32_t, x) & 0x7f800000u) == 0x7f800000u; }

// A strip of 16 d_v columns from column col0 on, token by token, by one wave.  The products of a chunk multiply what a token
// must not see by zero, which an infinity or NaN (of the inputs, or of values that overflow) passes: one that gets into u
// stays in the state, so where a sequence's last state is not finite its strip is gone over once more in this way.  So it
// is where an o was not finite: scale q k^T can overflow where u, or what a token has forgotten, would have made it small.
// One wave a strip, a token's loads waited for: 1.15 us a token (32768 tokens 38 ms, 4000 4.9), whatever else the call holds.
// (With the arguments kept for it in the chunks' scalar registers, one prompt of 32768 tokens took 1205 us where it took 1095.)
template <int R>
__device__ __forceinline__ void strip_by_tokens(const Span& s, int b, int h, int col0)
{
    const PrefillArgs& a = args_again();
    constexpr int M = R / 32;
    const int lane = lane_id(), r = lane & 15, q = lane >> 4, g = h / a.hpg;
    const size_t at = (((size_t)b * a.H + h) * a.C + col0 + r) * R + 8 * q;
    float S[M][8];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int e = 0; e < 8; ++e) S[m][e] = a.S_in ? a.S_in[at + 32 * m + e] : 0.f;
    auto sum4 = [](float x) {
        x += __shfl_xor(x, 16, 64);
        return x + __shfl_xor(x, 32, 64);
    };
    for (int i = 0; i < s.count; ++i) {
        const int64_t row = s.first + i;
        const uint16_t* kp = static_cast<const uint16_t*>(a.k) + row * a.k_stride + g * R + 8 * q;
        const uint16_t* qp = static_cast<const uint16_t*>(a.q) + row * a.q_stride + g * R + 8 * q;
        const float v = bf16_bits_to_f32(static_cast<const uint16_t*>(a.v)[row * a.v_stride + h * a.C + col0 + r]);
        const float alpha = a.alpha[row * a.H + h], beta = a.beta[row * a.H + h];
        float d = 0.f, o = 0.f;
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                S[m][e] *= alpha;
                d = __builtin_fmaf(S[m][e], bf16_bits_to_f32(kp[32 * m + e]), d);
            }
        const float u = beta * (v - sum4(d));
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                S[m][e] = __builtin_fmaf(u, bf16_bits_to_f32(kp[32 * m + e]), S[m][e]);
                o = __builtin_fmaf(S[m][e], bf16_bits_to_f32(qp[32 * m + e]), o);
            }
        o = a.scale * sum4(o);
        if (q == 0) static_cast<uint16_t*>(a.o)[(row * a.H + h) * a.C + col0 + r] = f32_to_bf16_bits(o);
    }
    if (!a.S_out) return;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int e = 0; e < 8; ++e) a.S_out[at + 32 * m + e] = S[m][e];
}

__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n s_barrier" ::: "memory"); }

}  // namespace rs
