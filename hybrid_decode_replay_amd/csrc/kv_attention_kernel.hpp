// kv_attention_kernel.hpp -- decode attention over a paged key/value cache (included by one
// translation unit per io type).
//
// Mathematics.  For the rows r (drafts x query heads) that share a key/value head, one pass over
// the tokens keeps a reference exponent m_r, a sum l_r and an output O_r (base-2 exponentials):
//   s = scale log2(e) q_r.K_j,  p = 2^(s - m_r),  l_r += p,  O_r += p V_j
// and whenever a score passes m_r by more than SLACK, m_r moves to the new maximum and l_r, O_r
// shrink by 2^(old - new).  Partial (m, l, O) of different waves, workgroups and splits join by
// the same rule; o = O / l, lse = ln 2 (m + log2 l).
//
// Bound by HBM: a token's 2 D values serve all rows of its head and are used once, 8 to 64 flop a
// byte.  So the design keeps loads in flight and the rest out of their way:
//
//  * Scores as S^T = K Q^T and outputs as O^T = V^T P^T on 16x16x32 products.  The result layout of
//    the first (lane: query row l%16, tokens 4(l/16)..+3 of a 16-token block) is the operand layout
//    of the second for the same query rows if its k index runs over (block, token in the lane's
//    four) -- so the weights go from one product to the other in registers, with no exchange
//    between lanes and no LDS.
//  * V^T's operand wants eight tokens of one channel in a lane; memory has eight channels of one
//    token.  A lane loads 16 bytes (eight channels) of each of its eight tokens and regroups the
//    8x8 block with byte permutes: sub-product j takes channel j of every lane's eight, so the
//    16 lanes of a row load whole rows of V.
//  * Each wave takes 32 tokens at a time, its K and V in single-buffered registers: the next
//    tokens' K is requested as soon as the scores are formed and their V as soon as the outputs
//    are, so 8 to 16 KiB a wave are always on the way and 8 to 16 waves a CU cover the latency.
//  * Tokens of one page are contiguous; page numbers are wave-uniform and come by scalar loads one
//    iteration ahead.
//  * Work is cut evenly, whatever the lengths: the (sequence, head, 128-token tile) units form one
//    line and workgroup w takes [w N / W, (w + 1) N / W).  Ranges that cover a head alone write its
//    output; the others leave partial rows that kv_combine_kernel joins.  The line depends on the
//    lengths alone, so results repeat.
//  * Weights are carried as two io-type terms (hi + lo, relative 2^-17 for bf16, 2^-22 for fp16):
//    the products have room to spare, and the output's error stays that of its own rounding.
#pragma once
#include <type_traits>

#include "kv_io.hpp"

namespace rs {

constexpr int KV_TILE = 128;                 // tokens of a work unit
constexpr int KV_SUB = 32;                   // tokens a wave takes at once
constexpr float KV_SLACK = 5.f;              // powers of two a weight may pass its reference by
constexpr int KV_OROW = 132;                 // floats per row of the join buffer (128 + padding)
constexpr int KV_MAX_WG = 1024;              // workgroups of a call

// x, but not to the compiler: what is computed from it stays where it is written, instead of
// being carried in registers through the token loop.
__device__ __forceinline__ int kv_opaque(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}

template <int IO>
struct KvOp {                                // matrix operand: eight io elements
    using T = typename std::conditional<IO == KV_BF16, bf16x8, f16x8>::type;
};
template <int IO>
__device__ __forceinline__ f32x4 kv_mfma(u32x4 a, u32x4 b, f32x4 c)
{
    using T = typename KvOp<IO>::T;
    if constexpr (IO == KV_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b), c, 0, 0, 0);
}

// Bytes 2 HI, 2 HI + 1 of a word of E4M3 codes as two io elements (exact: every E4M3 value is one).
template <int IO, bool HI>
__device__ __forceinline__ uint32_t kv_from_e4m3(uint32_t w)
{
    if constexpr (IO == KV_BF16)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, HI));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, HI));
}

// p0, p1 as hi + lo pairs of io elements.
template <int IO>
__device__ __forceinline__ void kv_split(float p0, float p1, uint32_t& hi, uint32_t& lo)
{
    hi = kv_pack<IO>(p0, p1);
    float h0, h1;
    kv_unpack<IO>(hi, h0, h1);
    lo = kv_pack<IO>(p0 - h0, p1 - h1);
}

// Nonzero if a word of cached values holds an infinity or NaN.
template <int IO, bool FP8>
__device__ __forceinline__ uint32_t kv_odd(uint32_t w)
{
    if constexpr (FP8) return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;       // E4M3 has NaN alone
    else {
        const uint32_t ex = IO == KV_BF16 ? 0x7f80u : 0x7c00u;
        return (uint32_t)((w & ex) == ex) | (uint32_t)((w >> 16 & ex) == ex);
    }
}

// A load of the cache's stream: past the caches unless the waves of a workgroup share it.
template <bool STREAM, typename T>
__device__ __forceinline__ T kv_load(const uint8_t* p)
{
    if constexpr (STREAM) return __builtin_nontemporal_load(reinterpret_cast<const T*>(p));
    else return *reinterpret_cast<const T*>(p);
}

// First and last visible position of a sequence's rows and its tiles.
struct KvRange {
    int end, base, tiles;
};
__device__ __forceinline__ KvRange kv_range(const KvAttention& a, int end, bool active)
{
    KvRange r;
    r.end = min(max(end, 0), a.max_pages << a.page_shift);
    const int lo = a.window > 0 ? max(0, r.end - a.T - a.window + 1) : 0;
    r.base = lo & ~(KV_SUB - 1);
    r.tiles = active ? max(1, (r.end - r.base + KV_TILE - 1) / KV_TILE) : 0;    // an empty row has an output too
    return r;
}

// The even cut of N units over W workgroups: the first N % W take one more than the others.
struct KvCut {
    int each, more;                          // N / W, N % W
    __device__ __forceinline__ int first(int w) const { return w * each + min(w, more); }
    __device__ __forceinline__ int owner(int u) const
    {
        const int head = more * (each + 1);
        return u < head ? u / (each + 1) : more + (u - head) / each;
    }
};

// Result of a row: outputs of eight consecutive channels.
template <int IO>
__device__ __forceinline__ void kv_store_o(const KvAttention& a, int b, int hkv, int row, int d, int D,
                                           const float (&x)[8])
{
    const int t = row / a.group, h = hkv * a.group + row - t * a.group;
    uint16_t* o = static_cast<uint16_t*>(a.o) + (((size_t)t * a.B + b) * a.Hq + h) * D + d;
    *reinterpret_cast<u32x4*>(o) = kv_pack8<IO>(x);
}
__device__ __forceinline__ void kv_store_lse(const KvAttention& a, int b, int hkv, int row, float m, float l)
{
    if (!a.lse) return;
    const int t = row / a.group, h = hkv * a.group + row - t * a.group;
    a.lse[((size_t)t * a.B + b) * a.Hq + h] = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
}

// D channels, RB blocks of 16 rows per wave, RW groups of waves with rows of their own (the 4 / RW
// waves of a group share its tokens).  Shared memory: prefix sums [B + 1] (dynamic).
template <int IO, bool FP8, int D, int RB, int RW, int OCC>
__global__ __launch_bounds__(256, OCC) void kv_attention_kernel(KvAttention a)
{
    constexpr int NTW = 4 / RW;              // waves that split a row group's tokens
    constexpr int KS = D / 32;               // products along a head
    constexpr int JN = D / 16;               // 16-channel groups of the output
    constexpr int EB = FP8 ? 1 : 2;          // bytes of a cached value
    constexpr int VE = JN < 16 / EB ? JN : 16 / EB;   // channels a lane loads of a token at once
    constexpr int VL = JN / VE;              // such loads per token
    constexpr int VW = VE * EB / 4;          // words of such a load
    constexpr int KL = D * EB / 64;          // 16-byte loads of K per token and lane
    constexpr int JP = JN < 8 ? JN : 8;      // 16-channel groups joined at once
    constexpr float OFF = IO == KV_F16 ? 10.f : 0.f;  // fp16 weights stay clear of its subnormals

    extern __shared__ int s_pre[];
    // the waves' queries in operand order while tokens pass, their outputs when they are joined
    __shared__ union {
        u32x4 q[4][RB * KS][64];
        float o[4][16][KV_OROW];
    } sh;
    auto& s_o = sh.o;
    __shared__ float s_m[4][16], s_l[4][16];
    __shared__ int s_wave[4];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = uni(tid >> 6), rg = wv % RW, tw = wv / RW;
    const int n = lane & 15, g = lane >> 4;
    const int hc = a.Hkv * a.nchunk;

    // ---- the line of units: prefix sums of tiles over the batch
    {
        int carry = 0;
        for (int b0 = 0; b0 < a.B; b0 += 256) {
            const int b = b0 + tid;
            int v = 0;
            if (b < a.B) {
                const int e = a.end[b];
                v = kv_range(a, e, !a.active || a.active[b]).tiles * hc;
                if (blockIdx.x == 0 && a.err && (e < 0 || e > (a.max_pages << a.page_shift))) atomicOr(a.err, KVERR_BAD_SLOT);
            }
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int u = __shfl_up(v, o, 64);
                if (lane >= o) v += u;
            }
            if (lane == 63) s_wave[wv] = v;
            __syncthreads();
            int before = carry;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i < wv) before += s_wave[i];
                carry += s_wave[i];
            }
            if (b < a.B) s_pre[b + 1] = before + v;
            if (b == 0) s_pre[0] = 0;
            __syncthreads();
        }
    }
    // at most a unit each, so that no workgroup inside a split range is without one
    const int N = uni(s_pre[a.B]), W = min((int)gridDim.x, N);
    const bool by_range = a.B * hc <= (int)gridDim.x;
    if (!by_range && tid == 0) a.meta[2 * blockIdx.x] = -1;
    if ((int)blockIdx.x >= W) return;
    const KvCut cut{N / W, N % W};
    int u = cut.first(blockIdx.x);
    const int u1 = u + cut.each + ((int)blockIdx.x < cut.more ? 1 : 0);
    for (int i = tid; i < a.B; i += 256)
        if (s_pre[i] <= u && u < s_pre[i + 1]) s_wave[0] = i;
    __syncthreads();
    int b = uni(s_wave[0]);                  // the sequence of unit u

#pragma unroll 1
    while (u < u1) {
        while (uni(s_pre[b + 1]) <= u) ++b;
        const KvRange rng = kv_range(a, uload(a.end + b), true);
        const int pre = uni(s_pre[b]), seg = (u - pre) / rng.tiles;
        const int ta = u - pre - seg * rng.tiles, tb = min(rng.tiles, ta + u1 - u);
        const int hkv = seg / a.nchunk, chunk = seg - hkv * a.nchunk;
        const int end = rng.end;
        const int tend = min(rng.base + tb * KV_TILE, end);
        const int32_t* table = a.table + (size_t)b * a.max_pages;

        const float sc = FP8 ? a.scale_log2 * uload(a.k_scale + hkv) : a.scale_log2;
        const float sc_abs = __builtin_fabsf(sc);
        int lim_hi[RB], lim_lo[RB];          // visible positions of the row

        float m[RB], l[RB];
        f32x4 O[RB][JN];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            m[rb] = -INFINITY;
            l[rb] = 0.f;
#pragma unroll
            for (int j = 0; j < JN; ++j) O[rb][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }

        // ---- tokens
        const int step = NTW * KV_SUB;
        const int t_first = rng.base + ta * KV_TILE + tw * KV_SUB;
        const int all_hi = end - a.T + 1;                                       // every row sees [all_lo, all_hi)
        const int all_lo = a.window > 0 ? max(0, end - a.window) : 0;
        const size_t head_bytes = ((size_t)D << a.page_shift) * EB;             // one head's part of a page
        const uint8_t* Kc = static_cast<const uint8_t*>(a.K) + hkv * head_bytes;
        const uint8_t* Vc = static_cast<const uint8_t*>(a.V) + hkv * head_bytes;
        const size_t page_bytes = head_bytes * a.Hkv;
        const uint32_t koff = n * D * EB + g * 16;                                  // token n, 16 bytes g
        const uint32_t voff = g * 4 * D * EB + n * VE * EB;                         // tokens 4 g.., channels VE n..

        u32x4 kf[2][KL];
        uint32_t vf[2][4][VL][VW];
        // Page and byte offset in the cache of the 16 tokens at t.  The page number is held inside the
        // cache whatever the table says; positions whose entry is wrong are masked below.
        auto page_of = [&](int t) { return (uint32_t)uload(table + (min(t, end - 1) >> a.page_shift)); };
        auto locate = [&](uint32_t entry, int t) {
            const int at = min(t, end - 1);
            const uint32_t page = min(entry, (uint32_t)a.npages - 1);
            return wave_uniform(page * page_bytes + (size_t)((at & ~15) & ((1 << a.page_shift) - 1)) * (D * EB));
        };
        auto load_k = [&](size_t b0, size_t b1) {
#pragma unroll
            for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                for (int i = 0; i < KL; ++i)
                    kf[blk][i] = kv_load<RW == 1, u32x4>(Kc + (blk ? b1 : b0) + i * 64 + koff);
        };
        auto load_v = [&](size_t b0, size_t b1) {
#pragma unroll
            for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int v = 0; v < VL; ++v) {
                        const uint8_t* p = Vc + (blk ? b1 : b0) + (r * D * EB + v * 16 * VE * EB) + voff;
                        if constexpr (VW == 4) {
                            const u32x4 w = kv_load<RW == 1, u32x4>(p);
                            vf[blk][r][v][0] = w.x;
                            vf[blk][r][v][1] = w.y;
                            vf[blk][r][v][2] = w.z;
                            vf[blk][r][v][3] = w.w;
                        } else if constexpr (VW == 2) {
                            const u32x2 w = kv_load<RW == 1, u32x2>(p);
                            vf[blk][r][v][0] = w.x;
                            vf[blk][r][v][1] = w.y;
                        } else {
                            vf[blk][r][v][0] = kv_load<RW == 1, uint32_t>(p);
                        }
                    }
        };
        // scores of the 32 tokens in kf (raw products)
        auto scores = [&](f32x4 (&s)[RB][2]) {
            asm volatile("" ::: "memory");       // queries stay in LDS from block to block
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) s[rb][0] = s[rb][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                u32x4 qf[RB];
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) qf[rb] = sh.q[wv][rb * KS + i][lane];
#pragma unroll
                for (int blk = 0; blk < 2; ++blk) {
                    u32x4 A;
                    if constexpr (FP8) {
                        const u32x4 w = kf[blk][i >> 1];
                        const uint32_t w0 = (i & 1) ? w.z : w.x, w1 = (i & 1) ? w.w : w.y;
                        A = u32x4{kv_from_e4m3<IO, false>(w0), kv_from_e4m3<IO, true>(w0),
                                  kv_from_e4m3<IO, false>(w1), kv_from_e4m3<IO, true>(w1)};
                    } else {
                        A = kf[blk][i];
                    }
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb) s[rb][blk] = kv_mfma<IO>(A, qf[rb], s[rb][blk]);
                }
            }
        };
        // Scores to weights (hi + lo), with the running reference, sum and outputs kept in step.
        // see: which of the lane's eight tokens row block rb's row sees.
        auto weights = [&](f32x4 (&s)[RB][2], const uint32_t (&see)[RB], auto masked, u32x4 (&ph)[RB], u32x4 (&pl)[RB]) {
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                float top = -INFINITY;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    top = fmaxf(top, !decltype(masked)::value || (see[rb] >> e & 1) ? s[rb][e >> 2][e & 3] : -INFINITY);
                top *= sc_abs;
                if (__builtin_amdgcn_ballot_w64(top > m[rb] + (OFF + KV_SLACK)) != 0) {
                    // the row's maximum over the 32 tokens; its four lanes agree on the reference
                    const float mx = max_over_row_groups(top);
                    const float mn = mx > m[rb] + (OFF + KV_SLACK) ? mx - OFF : m[rb];
                    const float f = mn == m[rb] ? 1.f : __builtin_amdgcn_exp2f(m[rb] - mn);
                    m[rb] = mn;
                    l[rb] *= f;
#pragma unroll
                    for (int j = 0; j < JN; ++j) O[rb][j] *= f;
                }
                const float ref = m[rb] == -INFINITY ? 0.f : m[rb];
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float p[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int e = 2 * i + k;
                        // one rounding between the score and its exponent
                        p[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[rb][e >> 2][e & 3], sc_abs, -ref));
                        if constexpr (decltype(masked)::value) p[k] = (see[rb] >> e & 1) ? p[k] : 0.f;
                        l[rb] += p[k];
                    }
                    kv_split<IO>(p[0], p[1], hi[i], lo[i]);
                }
                ph[rb] = u32x4{hi[0], hi[1], hi[2], hi[3]};
                pl[rb] = u32x4{lo[0], lo[1], lo[2], lo[3]};
            }
        };
        // O += V^T P^T for the wave's 32 tokens, of all rows or of those in mine
        auto outputs = [&](const u32x4 (&ph)[RB], const u32x4 (&pl)[RB], auto some, const bool (&mine)[RB]) {
            auto add = [&](u32x4 A, int j) {
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) {
                    const f32x4 x = kv_mfma<IO>(A, pl[rb], kv_mfma<IO>(A, ph[rb], O[rb][j]));
                    if constexpr (decltype(some)::value) O[rb][j] = mine[rb] ? x : O[rb][j];
                    else O[rb][j] = x;
                }
                if constexpr (decltype(some)::value) __builtin_amdgcn_sched_barrier(0);
            };
#pragma unroll
            for (int v = 0; v < VL; ++v) {
                if constexpr (FP8) {
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        // four channels of eight tokens: bytes of two tokens side by side, then widened
                        uint32_t e[4][4];
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const uint32_t x = vf[t >> 1][(t & 1) * 2][v][w], y = vf[t >> 1][(t & 1) * 2 + 1][v][w];
                            const uint32_t c01 = __builtin_amdgcn_perm(y, x, 0x05010400u);
                            const uint32_t c23 = __builtin_amdgcn_perm(y, x, 0x07030602u);
                            e[0][t] = kv_from_e4m3<IO, false>(c01);
                            e[1][t] = kv_from_e4m3<IO, true>(c01);
                            e[2][t] = kv_from_e4m3<IO, false>(c23);
                            e[3][t] = kv_from_e4m3<IO, true>(c23);
                        }
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            add(u32x4{e[c][0], e[c][1], e[c][2], e[c][3]}, v * VE + w * 4 + c);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < VE; ++c) {
                        const uint32_t sel = (c & 1) ? 0x07060302u : 0x05040100u;
                        const int w = c >> 1;
                        const u32x4 A = {__builtin_amdgcn_perm(vf[0][1][v][w], vf[0][0][v][w], sel),
                                         __builtin_amdgcn_perm(vf[0][3][v][w], vf[0][2][v][w], sel),
                                         __builtin_amdgcn_perm(vf[1][1][v][w], vf[1][0][v][w], sel),
                                         __builtin_amdgcn_perm(vf[1][3][v][w], vf[1][2][v][w], sel)};
                        add(A, v * VE + c);
                    }
                }
            }
        };

        // ---- the first block's keys and values are requested before anything is waited for
        const int nb = t_first < tend ? (tend - t_first + step - 1) / step : 0;     // the wave's blocks
        int t0 = t_first;
        uint32_t p0 = 0, p1 = 0, c0 = 0, c1 = 0;     // table entries of the next and of the current block
        size_t b0 = 0, b1 = 0;
        if (nb > 0) {
            c0 = page_of(t0);
            c1 = page_of(t0 + 16);
            b0 = locate(c0, t0);
            b1 = locate(c1, t0 + 16);
            load_k(b0, b1);
            load_v(b0, b1);
            p0 = page_of(t0 + step);
            p1 = page_of(t0 + step + 16);
        }

        // ---- queries: row n of each of the wave's blocks, eight channels of each product.  Each wave
        // keeps its own copy in LDS; the barrier keeps it behind the previous range's join.
        __syncthreads();
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            const int nn = kv_opaque(lane & 15), row = chunk * a.rpc + (rg * RB + rb) * 16 + nn;
            const int t = row / a.group, h = hkv * a.group + row - t * a.group;
            const bool real = row < a.rows && (rg * RB + rb) * 16 + nn < a.rpc;
            lim_hi[rb] = real ? end - a.T + t + 1 : end;
            lim_lo[rb] = real && a.window > 0 ? max(0, lim_hi[rb] - a.window) : 0;
            const uint16_t* q = static_cast<const uint16_t*>(a.q) + ((size_t)t * a.B + b) * a.q_stride + (size_t)h * D;
            const uint32_t flip = sc < 0.f ? 0x80008000u : 0u;      // scores are scaled by |sc|
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                // the channels of K's loads: eight at a time, or halves of sixteen codes
                const int d = FP8 ? (i >> 1) * 64 + g * 16 + (i & 1) * 8 : i * 32 + g * 8;
                u32x4 w = real ? *reinterpret_cast<const u32x4*>(q + d) : u32x4{0, 0, 0, 0};
                w ^= u32x4{flip, flip, flip, flip};
                sh.q[wv][rb * KS + i][lane] = w;
            }
        }
        // a table entry outside the cache sends the whole range through the masked path
        bool wrong = false;
        for (int i = ((rng.base + ta * KV_TILE) >> a.page_shift) + lane;
             i < (tend + (1 << a.page_shift) - 1) >> a.page_shift; i += 64)
            wrong |= (uint32_t)table[i] >= (uint32_t)a.npages;
        wrong = __builtin_amdgcn_ballot_w64(wrong) != 0;
        if (wrong && lane == 0 && a.err) atomicOr(a.err, KVERR_BAD_SLOT);

        // ---- tokens.  Every block but the last requests the next one unconditionally: the waits for K
        // and V then count exactly the requests behind them.
        auto block = [&](auto more) {
            f32x4 s[RB][2];
            scores(s);
            const int cur = t0;
            const size_t cb0 = b0, cb1 = b1;
            const bool ok0 = c0 < (uint32_t)a.npages, ok1 = c1 < (uint32_t)a.npages;
            if constexpr (decltype(more)::value) {
                t0 += step;
                c0 = p0;
                c1 = p1;
                b0 = locate(c0, t0);
                b1 = locate(c1, t0 + 16);
                load_k(b0, b1);
                p0 = page_of(t0 + step);
                p1 = page_of(t0 + step + 16);
                __builtin_amdgcn_sched_barrier(0);
            }
            u32x4 ph[RB], pl[RB];
            uint32_t see[RB] = {};
            bool mine[RB] = {};
            if (!wrong && cur >= all_lo && cur + KV_SUB <= all_hi) {        // every row sees every token
                weights(s, see, std::false_type{}, ph, pl);
                outputs(ph, pl, std::false_type{}, mine);
            } else {
                const int mt = cur + 4 * kv_opaque(g);                      // the lane's first token
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int t = mt + (e >> 2) * 16 + (e & 3);
                        if (t < lim_hi[rb] && t >= lim_lo[rb] && (e < 4 ? ok0 : ok1)) see[rb] |= 1u << e;
                    }
                }
                weights(s, see, std::true_type{}, ph, pl);
                // Values that no row sees count as zero, so that 0 * NaN does not arise.  A value that only
                // some drafts see and that is no number would still reach the others: then, and only then,
                // the drafts are taken one by one.
                auto clear = [&](int lo, int hi) {
                    uint32_t odd = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int t = mt + (e >> 2) * 16 + (e & 3);
                        const bool sees = t < hi && t >= lo && (e < 4 ? ok0 : ok1);
                        const bool some = t < all_lo || t >= all_hi;
#pragma unroll
                        for (int v = 0; v < VL; ++v)
#pragma unroll
                            for (int w = 0; w < VW; ++w) {
                                const uint32_t x = sees ? vf[e >> 2][e & 3][v][w] : 0u;
                                vf[e >> 2][e & 3][v][w] = x;
                                if (some) odd |= kv_odd<IO, FP8>(x);
                            }
                    }
                    return __builtin_amdgcn_ballot_w64(odd != 0) != 0;
                };
                const bool odd = clear(a.window > 0 ? max(0, end - a.T + 1 - a.window) : 0, end);
                if (a.T == 1 || !odd) {
                    outputs(ph, pl, std::false_type{}, mine);
                } else {
#pragma unroll 1
                    for (int d = 0; d < a.T; ++d) {
                        const int hi = end - a.T + d + 1;
                        load_v(cb0, cb1);
                        clear(a.window > 0 ? max(0, hi - a.window) : 0, hi);
#pragma unroll
                        for (int rb = 0; rb < RB; ++rb) mine[rb] = lim_hi[rb] == hi;
                        outputs(ph, pl, std::true_type{}, mine);
                    }
                }
            }
            if constexpr (decltype(more)::value) {
                load_v(b0, b1);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if (nb > 0) {
#pragma unroll 1
            for (int left = nb - 1; left > 0; --left) block(std::true_type{});
            block(std::false_type{});
        }

        // ---- join the waves of each row group; whole ranges write the output
        const bool whole = ta == 0 && tb == rng.tiles;
        const int slot = 2 * blockIdx.x + (ta == 0 ? 1 : 0);
        const float vs = FP8 ? uload(a.v_scale + hkv) : 1.f;
        const int jt = kv_opaque(tid), jn = jt & 15, jg = (jt >> 4) & 3;
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            const float lw = sum_over_row_groups(l[rb]);
#pragma unroll
            for (int jp = 0; jp < JN; jp += JP) {
                __syncthreads();                                 // queries or the previous part are done with
                if (jp == 0 && jg == 0) {
                    s_m[wv][jn] = m[rb];
                    s_l[wv][jn] = lw;
                }
                // lane: row n, channels VE (4 g + r).. of each load's 16 VE
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int j = 0; j < JP; j += 4) {
                        const int jj = jp + j, d = (jj / VE) * 16 * VE + (4 * jg + r) * VE + jj % VE;
                        // channel within the joined 16 JP: whole loads of 16 VE, or the halves of one
                        const int c = VE <= JP ? d - jp * 16 : (4 * jg + r) * JP + j;
                        st4(&s_o[wv][jn][c], f32x4{O[rb][jj][r], O[rb][jj + 1][r], O[rb][jj + 2][r], O[rb][jj + 3][r]});
                    }
                __syncthreads();
                constexpr int C8 = JP * 2;                       // eight-channel pieces of a row
                for (int i = jt; i < RW * 16 * C8; i += 256) {
                    const int rr = i / C8, c = (i - rr * C8) * 8, grp = rr >> 4, nn = rr & 15;
                    const int rl = (grp * RB + rb) * 16 + nn, row = chunk * a.rpc + rl;
                    if (rl >= a.rpc || row >= a.rows) continue;
                    const int d = VE <= JP ? jp * 16 + c : (c / JP) * VE + jp + c % JP;
                    float M = -INFINITY, L = 0.f, x[8] = {};
#pragma unroll
                    for (int k = 0; k < NTW; ++k) M = fmaxf(M, s_m[k * RW + grp][nn]);
#pragma unroll
                    for (int k = 0; k < NTW; ++k) {
                        const float mk = s_m[k * RW + grp][nn];
                        const float f = mk == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(mk - M);
                        L += f * s_l[k * RW + grp][nn];
                        const f32x4 y0 = ld4(&s_o[k * RW + grp][nn][c]), y1 = ld4(&s_o[k * RW + grp][nn][c + 4]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[e] += f * y0[e];
                            x[4 + e] += f * y1[e];
                        }
                    }
                    if (whole) {
                        const float inv = L == 0.f ? 0.f : vs / L;
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] *= inv;
                        kv_store_o<IO>(a, b, hkv, row, d, D, x);
                        if (d == 0) kv_store_lse(a, b, hkv, row, M, L);
                    } else {
                        const size_t at = (size_t)slot * a.rpc + rl;
                        st4(a.part_o + at * D + d, f32x4{x[0], x[1], x[2], x[3]});
                        st4(a.part_o + at * D + d + 4, f32x4{x[4], x[5], x[6], x[7]});
                        if (d == 0) {
                            a.part_ml[2 * at] = M;
                            a.part_ml[2 * at + 1] = L;
                        }
                    }
                }
            }
        }
        if (tid == 0 && ta == 0 && (by_range || !whole)) {
            const int range = b * hc + seg;
            int32_t* mt = a.meta + 2 * (by_range ? range : (int)blockIdx.x);
            mt[0] = by_range ? (whole ? -1 : (int)blockIdx.x) : range;
            mt[1] = cut.owner(pre + (seg + 1) * rng.tiles - 1);
        }
        u += tb - ta;
    }
}

// Joins the partial rows of one split range, a row at a time.  blockIdx.x is the range where there
// are no more of them than workgroups, else the workgroup that opened it.  The parts' references and sums first, each part's weight into LDS, then the outputs by 256
// threads = D / 4 lanes of four channels x 1024 / D groups of parts.
template <int IO, bool FP8, int D, bool BY_RANGE>
__global__ __launch_bounds__(256) void kv_combine_kernel(KvAttention a)
{
    constexpr int CL = D / 4, PG = 256 / CL;
    __shared__ float s_x[PG][D], s_w[KV_MAX_WG], s_m[4], s_l[4];
    const int hc = a.Hkv * a.nchunk, found = uload(a.meta + 2 * blockIdx.x);
    const int range = BY_RANGE ? blockIdx.x : found, w0 = BY_RANGE ? found : blockIdx.x;
    const int b = max(range, 0) / hc, seg = range - b * hc;
    if ((BY_RANGE && a.active && !uload(a.active + b)) || found < 0) return;
    const int w1 = uload(a.meta + 2 * blockIdx.x + 1);
    const int np = w1 - w0 + 1, tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int hkv = seg / a.nchunk, chunk = seg - hkv * a.nchunk;
    const int c = tid % CL, pg = tid / CL;
    const float vs = FP8 ? uload(a.v_scale + hkv) : 1.f;
    const int rows = min(a.rpc, a.rows - chunk * a.rpc);
    // the opening workgroup's part is its last (slot 1), the others' their first (slot 0)
    auto part = [&](int i, int rl) { return (size_t)(2 * (w0 + i) + (i == 0 ? 1 : 0)) * a.rpc + rl; };
    for (int rl = blockIdx.y; rl < rows; rl += gridDim.y) {
        float M = -INFINITY, L = 0.f;
        for (int i = tid; i < np; i += 256) M = fmaxf(M, a.part_ml[2 * part(i, rl)]);
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor(M, o, 64));
        if (lane == 0) s_m[wv] = M;
        __syncthreads();
        M = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
        for (int i = tid; i < np; i += 256) {
            const float m = a.part_ml[2 * part(i, rl)];
            const float f = m == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - M);
            s_w[i] = f;
            L += f * a.part_ml[2 * part(i, rl) + 1];
        }
        L = wave_sum64(L);
        if (lane == 0) s_l[wv] = L;
        __syncthreads();
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int i = pg; i < np; i += PG) x += ld4(a.part_o + part(i, rl) * D + 4 * c) * s_w[i];
        st4(&s_x[pg][4 * c], x);
        __syncthreads();
        if (tid < D / 8) {
            L = s_l[0] + s_l[1] + s_l[2] + s_l[3];
            float y[8] = {};
#pragma unroll
            for (int k = 0; k < PG; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] += s_x[k][8 * tid + e];
            const float inv = L == 0.f ? 0.f : vs / L;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= inv;
            const int row = chunk * a.rpc + rl;
            kv_store_o<IO>(a, b, hkv, row, 8 * tid, D, y);
            if (tid == 0) kv_store_lse(a, b, hkv, row, M, L);
        }
        __syncthreads();
    }
}

template <int IO, bool FP8, int D, int RB, int RW, int OCC>
static hipError_t kv_attention_start(const KvAttention& a, const KvPlan& p, hipStream_t s)
{
    hipLaunchKernelGGL((kv_attention_kernel<IO, FP8, D, RB, RW, OCC>), dim3(p.nwg), dim3(256), (a.B + 1) * sizeof(int), s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int ranges = a.B * a.Hkv * a.nchunk, most = ranges <= p.nwg ? ranges : p.nwg;
    const int y = p.rpc < 8192 / most ? p.rpc : 8192 / most;         // rows side by side, within some waves of the chip
    if (ranges <= p.nwg) hipLaunchKernelGGL((kv_combine_kernel<IO, FP8, D, true>), dim3(ranges, y), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((kv_combine_kernel<IO, FP8, D, false>), dim3(p.nwg, y), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int IO, bool FP8>
static hipError_t kv_attention_pick(const KvAttention& a, const KvPlan& p, int D, hipStream_t s)
{
    // (row blocks per wave, row groups) of kv_attention_plan, and the workgroups a CU is cut for
    const int k = D * 100 + p.RB * 10 + p.RW;
    constexpr bool F = FP8;
    switch (k) {
        case 6411: return kv_attention_start<IO, F, 64, 1, 1, kv_occ(64, F, 1)>(a, p, s);
        case 6421: return kv_attention_start<IO, F, 64, 2, 1, kv_occ(64, F, 2)>(a, p, s);
        case 6422: return kv_attention_start<IO, F, 64, 2, 2, kv_occ(64, F, 2)>(a, p, s);
        case 6424: return kv_attention_start<IO, F, 64, 2, 4, kv_occ(64, F, 2)>(a, p, s);
        case 12811: return kv_attention_start<IO, F, 128, 1, 1, kv_occ(128, F, 1)>(a, p, s);
        case 12821: return kv_attention_start<IO, F, 128, 2, 1, kv_occ(128, F, 2)>(a, p, s);
        case 12822: return kv_attention_start<IO, F, 128, 2, 2, kv_occ(128, F, 2)>(a, p, s);
        case 12824: return kv_attention_start<IO, F, 128, 2, 4, kv_occ(128, F, 2)>(a, p, s);
        case 25611: return kv_attention_start<IO, F, 256, 1, 1, kv_occ(256, F, 1)>(a, p, s);
        case 25612: return kv_attention_start<IO, F, 256, 1, 2, kv_occ(256, F, 1)>(a, p, s);
        case 25614: return kv_attention_start<IO, F, 256, 1, 4, kv_occ(256, F, 1)>(a, p, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace rs
