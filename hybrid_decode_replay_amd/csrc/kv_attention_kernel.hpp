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
// Bound by HBM: a token's 2 D values serve all rows of its head and are used once, 4 to 64 flop a byte
// for one token a sequence, against some 300 at which the matrix units would be the limit.  So the
// design keeps loads in flight and the rest out of their way:
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
//  * Each wave takes 32 tokens at a time, K and V in single-buffered registers: the next tokens' K is
//    requested as soon as the scores are formed and their V as soon as the outputs are, so 8 to 16 KiB
//    a wave are always on the way, and eight waves a CU (four where a wave needs more registers) cover
//    the latency.  Queries stay in LDS for the registers' sake.  Page numbers are wave-uniform and come
//    by scalar loads one block ahead.
//  * Work is cut evenly, whatever the lengths: the (sequence, head, 128-token tile) units form one line
//    and the workgroups take equal stretches of it.  Ranges that a stretch covers write their outputs;
//    the others leave partial rows that kv_combine_kernel joins.  The line depends on the lengths
//    alone, so results repeat.  Ranges known to be short (kv_attention_whole) and many ranges of like
//    lengths (kv_order) get a workgroup each instead.
//  * Weights are carried as two io-type terms (hi + lo, relative 2^-16 for bf16, 2^-22 for fp16): one
//    term alone would double the error of the output's own rounding.  A third bf16 term (24 bits) moves
//    one output in 600 by a step and leaves the error against 64 bits at the rounding's own 0.0017; it
//    costs 1 % for 4 rows of a head, 1 to 5 % for 32, 6 % for 64 and 18 % for 128 on 128 channels (151 ->
//    178 us).
//  * More than 32 rows of a head (drafts x queries) would make the waves of a workgroup read the cache
//    again for each other: there it goes through LDS (kv_attention_wide_kernel).
//
// Measured with both launches, 537 MB of cache (131k tokens of 8 heads, 128 channels, bf16), read alone
// in 76 us at the 7.09 TB/s of a plain read: 93 us for 4 rows a head, 94 for 32, 107 for 64, 155 for 128, 264
// for 256 (two chunks).  The same bytes on 64 channels 93 (64 rows 117), on 256 channels 96 (32 rows 109, 64
// rows 122, 128 rows in two chunks 204), as E4M3 97 (32 rows 110, 64 rows 157, 128 rows 260: twice the tokens,
// and past 32 rows the work on a token counts, not its bytes).
#pragma once
#include <type_traits>

#include "kv_io.hpp"

namespace rs {

constexpr int KV_TILE = 128;                 // tokens of a work unit
constexpr int KV_SUB = 32;                   // tokens a wave takes at once
constexpr float KV_SLACK = 5.f;              // powers of two a weight may pass its reference by

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

// A load of the cache's stream (used once: past the caches).
template <typename T>
__device__ __forceinline__ T kv_stream(const uint8_t* p)
{
    return __builtin_nontemporal_load(reinterpret_cast<const T*>(p));
}
// N consecutive words, from the stream or from LDS.
template <int N, bool STREAM>
__device__ __forceinline__ void kv_words(const uint8_t* p, uint32_t (&w)[N])
{
    using T = typename std::conditional<N == 4, u32x4, typename std::conditional<N == 2, u32x2, uint32_t>::type>::type;
    T x;
    if constexpr (STREAM) x = kv_stream<T>(p);
    else x = *reinterpret_cast<const T*>(p);
    if constexpr (N == 1) w[0] = x;
    else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = x[i];
    }
}

// An `end` that the table cannot hold: taken as the nearest that it can.
__device__ __forceinline__ bool kv_bad_end(const KvAttention& a, int end)
{
    return end < 0 || end > (a.max_pages << a.page_shift);
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

// Result of a row: outputs of four or eight consecutive channels.
template <int IO, int N>
__device__ __forceinline__ void kv_store_o(const KvAttention& a, int b, int hkv, int row, int d, int D,
                                           const float (&x)[N])
{
    const int t = row / a.group, h = hkv * a.group + row - t * a.group;
    uint16_t* o = static_cast<uint16_t*>(a.o) + (((size_t)t * a.B + b) * a.Hq + h) * D + d;
    if constexpr (N == 8) *reinterpret_cast<u32x4*>(o) = kv_pack8<IO>(x);
    else *reinterpret_cast<u32x2*>(o) = u32x2{kv_pack<IO>(x[0], x[1]), kv_pack<IO>(x[2], x[3])};
}
__device__ __forceinline__ void kv_store_lse(const KvAttention& a, int b, int hkv, int row, float m, float l)
{
    if (!a.lse) return;
    const int t = row / a.group, h = hkv * a.group + row - t * a.group;
    a.lse[((size_t)t * a.B + b) * a.Hq + h] = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
}

// Sizes that follow from the cached type and the width of a head.
template <bool FP8, int D>
struct KvGeom {
    static constexpr int EB = FP8 ? 1 : 2;               // bytes of a cached value
    static constexpr int ROWB = D * EB;                  // bytes of a token's head
    static constexpr int KS = D / 32;                    // products along a head
    static constexpr int JN = D / 16;                    // 16-channel groups of the output
    static constexpr int VE = JN < 16 / EB ? JN : 16 / EB;   // channels a lane takes of a token at once
    static constexpr int VL = JN / VE;                   // such pieces per token
    static constexpr int VW = VE * EB / 4;               // words of such a piece
    static constexpr int KL = ROWB / 64;                 // 16-byte pieces of K per token and lane
};

// The line of units as a workgroup sees it, and its place on it.
struct KvLine {
    int hc, u, u1, b;                        // ranges per sequence; first and last + 1 unit; sequence of the first
    bool by_range, whole;
    KvCut cut;
};

// Prefix sums of tiles over the batch into s_pre [B + 1], and this workgroup's units; false if it
// has none.  `tmp` holds an entry per wave.
template <int NT>
__device__ __forceinline__ bool kv_line(const KvAttention& a, int* s_pre, int* tmp, KvLine& ln)
{
    const int tid = threadIdx.x, lane = tid & 63, wv = uni(tid >> 6);
    ln.hc = a.Hkv * a.nchunk;
    ln.whole = false;
    int carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        const int b = b0 + tid;
        int v = 0;
        if (b < a.B) {
            const int e = a.end[b];
            const bool active = !a.active || a.active[b];
            v = kv_range(a, e, active).tiles * ln.hc;
            if (blockIdx.x == 0 && active && a.err && kv_bad_end(a, e)) atomicOr(a.err, KVERR_BAD_SLOT);
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int x = __shfl_up(v, o, 64);
            if (lane >= o) v += x;
        }
        if (lane == 63) tmp[wv] = v;
        __syncthreads();
        int before = carry;
#pragma unroll
        for (int i = 0; i < NT / 64; ++i) {
            if (i < wv) before += tmp[i];
            carry += tmp[i];
        }
        if (b < a.B) s_pre[b + 1] = before + v;
        if (b == 0) s_pre[0] = 0;
        __syncthreads();
    }
    // at most a unit each, so that no workgroup inside a split range is without one
    const int N = uni(s_pre[a.B]), W = min(a.nwg, N);
    ln.by_range = a.B * ln.hc <= a.nwg;
    if (!ln.by_range && tid == 0) a.meta[2 * blockIdx.x] = -1;
    if ((int)blockIdx.x >= W) return false;
    const int each = uni(N / W);
    ln.cut = KvCut{each, N - each * W};
    ln.u = ln.cut.first(blockIdx.x);
    ln.u1 = ln.u + ln.cut.each + ((int)blockIdx.x < ln.cut.more ? 1 : 0);
    for (int i = tid; i < a.B; i += NT)
        if (s_pre[i] <= ln.u && ln.u < s_pre[i + 1]) tmp[0] = i;
    __syncthreads();
    ln.b = uni(tmp[0]);
    return true;
}

// A workgroup's part of one range: tiles [ta, tb) of sequence b, key/value head hkv, row chunk.
struct KvPart {
    int b, seg, hkv, chunk, ta, tb, tiles, end, base, tend;
    int all_lo, all_hi;                      // positions that every row sees
    const int32_t* table;
    float sc;                                // signed scale of the raw products, in powers of two
    __device__ __forceinline__ bool whole() const { return ta == 0 && tb == tiles; }
    // (a scale of zero would let masked scores through: the smallest normal number stands for it)
    __device__ __forceinline__ float sc_abs() const
    {
        const float x = __builtin_fabsf(sc);
        return x < 0x1p-126f ? 0x1p-126f : x;
    }
    // every row sees every one of the n tokens at t
    __device__ __forceinline__ bool full(int t, int n) const { return t >= all_lo && t + n <= all_hi; }
};
// Tiles [ta, tb) of range seg (head and row chunk) of sequence b.  Everything goes to scalar
// registers: the loops over tokens then branch without masks.
template <bool FP8>
__device__ __forceinline__ KvPart kv_part(const KvAttention& a, int b, const KvRange& rng, int seg, int ta, int tb)
{
    KvPart p;
    p.b = uni(b);
    p.tiles = uni(rng.tiles);
    p.seg = uni(seg);
    p.ta = uni(ta);
    p.tb = uni(tb);
    p.hkv = uni(p.seg / a.nchunk);
    p.chunk = uni(p.seg - p.hkv * a.nchunk);
    p.end = uni(rng.end);
    p.base = uni(rng.base);
    p.tend = uni(min(p.base + p.tb * KV_TILE, p.end));
    p.all_hi = uni(p.end - a.T + 1);
    p.all_lo = uni(a.window > 0 ? max(0, p.end - a.window) : 0);
    p.table = a.table + (size_t)p.b * a.max_pages;
    p.sc = FP8 ? a.scale_log2 * uload(a.k_scale + p.hkv) : a.scale_log2;
    return p;
}
// Where there are more ranges than the chip holds workgroups: whether each takes a range of its own, the
// longest first so that the last ones are short, and which.  Even shares need no join then; but a range
// longer than an even share would outlast the others, so with one such the line is cut instead.  Every
// wave finds it for itself: the tiles of the batch in N registers (at least B / 64), the length of the
// range at place `at` by bisection, counting with ballots (lengths in 32 steps, equal ones as they stand).
// Lengths of 64 to 4000, 128 channels, 8 heads, tables of 32768 tokens, E4M3: 128 sequences 122 us on the
// line, 100 by length, 256 sequences 210 and 182; the same with all but one sequence eight times shorter
// (on the line): 43 us without this choice, 44 with it, and 67 and 69.
struct KvOrder {
    bool whole;
    int b;
};
template <int N>
__device__ __forceinline__ KvOrder kv_order(const KvAttention& a, int at)
{
    const int lane = threadIdx.x & 63;
    int tiles[N], most = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int b = i * 64 + lane;
        tiles[i] = -1;
        if (b < a.B) {
            tiles[i] = kv_range(a, a.end[b], !a.active || a.active[b]).tiles;
            most = max(most, tiles[i]);
            sum += tiles[i];
        }
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        most = max(most, __shfl_xor(most, o, 64));
        sum += __shfl_xor(sum, o, 64);
    }
    most = uni(most);
    KvOrder r;
    r.whole = a.whole || (long long)most * a.nwg <= (long long)uni(sum) * (a.Hkv * a.nchunk);
    r.b = 0;
    if (!r.whole) return r;
    const int shift = max(0, 27 - __builtin_clz(most | 1));      // most >> shift is below 32
#pragma unroll
    for (int i = 0; i < N; ++i) tiles[i] >>= shift;
    auto as_long = [&](int n) {
        int c = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) c += __builtin_popcountll(__builtin_amdgcn_ballot_w64(tiles[i] >= n));
        return c;
    };
    int n = 0, left = at;                             // left: places after the longer ones
#pragma unroll
    for (int bit = 16; bit > 0; bit >>= 1) {
        const int c = as_long(n + bit);
        if (c > at) n += bit;
        else left = at - c;                           // (the last such count is that of n + 1)
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint64_t same = __builtin_amdgcn_ballot_w64(tiles[i] == n);
        const int c = __builtin_popcountll(same);
        if (left >= 0 && left < c) {
            const bool it = tiles[i] == n && (int)__builtin_popcountll(same & ((1ull << lane) - 1)) == left;
            r.b = i * 64 + __builtin_ctzll(__builtin_amdgcn_ballot_w64(it));
        }
        left -= c;
    }
    r.b = uni(r.b);
    return r;
}
// This workgroup's place on the line, or its range (ln.whole: u is its head and chunk); false if it has
// neither.
__device__ __forceinline__ bool kv_begin(const KvAttention& a, int* s_pre, int* tmp, KvLine& ln)
{
    const int hc = a.Hkv * a.nchunk, at = uni(blockIdx.x / hc), seg = uni(blockIdx.x - at * hc);
    int b = at;
    bool whole = a.whole;
    if (a.by_length) {
        const KvOrder o = a.B <= 256 ? kv_order<4>(a, at) : kv_order<KV_BY_LENGTH / 64>(a, at);
        whole = o.whole;
        b = o.b;
        if (!whole && (int)blockIdx.x >= a.nwg) return false;
        if (whole && !a.whole && (int)blockIdx.x < a.nwg && threadIdx.x == 0) a.meta[2 * blockIdx.x] = -1;
    }
    if (!whole) return kv_line<256>(a, s_pre, tmp, ln);
    ln.whole = true;
    ln.b = b;
    ln.u = seg;
    ln.u1 = seg + 1;
    if (a.active && !uload(a.active + b)) return false;
    if (seg == 0 && threadIdx.x == 0 && a.err && kv_bad_end(a, uload(a.end + b))) atomicOr(a.err, KVERR_BAD_SLOT);
    return true;
}
// Its next part.
template <bool FP8>
__device__ __forceinline__ KvPart kv_next_part(const KvAttention& a, const int* s_pre, KvLine& ln)
{
    if (!ln.whole)
        while (uni(s_pre[ln.b + 1]) <= ln.u) ++ln.b;
    const int b = uni(ln.b), u = uni(ln.u), at = ln.whole ? 0 : uni(u - s_pre[b]);
    const KvRange rng = kv_range(a, uload(a.end + b), true);
    const int seg = ln.whole ? u : at / rng.tiles, ta = ln.whole ? 0 : at - seg * rng.tiles;
    return kv_part<FP8>(a, b, rng, seg, ta, ln.whole ? rng.tiles : min(rng.tiles, ta + ln.u1 - u));
}

// Whether a table entry that some row of the part sees lies outside the cache (the part's blocks then
// take the masked path).  Pages before the first visible position, which may share a block with it,
// are nobody's: a window's table may have dropped them.
__device__ __forceinline__ bool kv_wrong_pages(const KvAttention& a, const KvPart& p, int lane)
{
    bool wrong = false;
    const int lo = a.window > 0 ? max(0, p.end - a.T - a.window + 1) : 0;
    for (int i = (max(p.base + p.ta * KV_TILE, lo) >> a.page_shift) + lane;
         i < (p.tend + (1 << a.page_shift) - 1) >> a.page_shift; i += 64)
        wrong |= (uint32_t)p.table[i] >= (uint32_t)a.npages;
    wrong = __builtin_amdgcn_ballot_w64(wrong) != 0;
    if (wrong && lane == 0 && a.err) atomicOr(a.err, KVERR_BAD_SLOT);
    return wrong;
}

// Where the 16 tokens at t lie.  The page number is held inside the cache whatever the table says;
// positions whose entry is wrong are masked.
__device__ __forceinline__ uint32_t kv_page_of(const KvAttention& a, const KvPart& p, int t)
{
    return (uint32_t)uload(p.table + (min(t, p.end - 1) >> a.page_shift));
}
template <int ROWB>
__device__ __forceinline__ size_t kv_locate(const KvAttention& a, const KvPart& p, uint32_t entry, int t)
{
    const size_t head = (size_t)ROWB << a.page_shift;
    const uint32_t page = min(entry, (uint32_t)a.npages - 1), off = (uint32_t)(min(t, p.end - 1) & ~15) & ((1u << a.page_shift) - 1);
    return wave_uniform(((size_t)page * a.Hkv + p.hkv) * head + (size_t)off * ROWB);
}

// The rows of one wave: RB blocks of 16, their softmax state and outputs, and 32 tokens' values, of
// which VP pieces (of VL) are held at a time.
template <int IO, bool FP8, int D, int RB, int VP>
struct KvRows {
    using G = KvGeom<FP8, D>;
    static constexpr int KS = G::KS, JN = G::JN, VE = G::VE, VL = G::VL, VW = G::VW;
    static constexpr float OFF = IO == KV_F16 ? 10.f : 0.f;   // fp16 weights stay clear of its subnormals

    float m[RB], l[RB];
    f32x4 O[RB][JN];
    int lim_hi[RB], lim_lo[RB];              // visible positions of the lane's row
    uint32_t vf[2][4][VP][VW];               // values of tokens 16 blk + 4 (lane / 16) + r

    __device__ __forceinline__ void init()
    {
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            m[rb] = -INFINITY;
            l[rb] = 0.f;
#pragma unroll
            for (int j = 0; j < JN; ++j) O[rb][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    }

    // Row limits, and the rows' queries in operand order to LDS: row block first + rb of the chunk.
    __device__ __forceinline__ void queries(const KvAttention& a, const KvPart& p, int first, u32x4 (*dst)[64], int lane)
    {
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            const int n = kv_opaque(lane & 15), g = lane >> 4, rl = (first + rb) * 16 + n, row = p.chunk * a.rpc + rl;
            const int t = row / a.group, h = p.hkv * a.group + row - t * a.group;
            const bool real = row < a.rows && rl < a.rpc;
            lim_hi[rb] = real ? p.end - a.T + t + 1 : p.end;
            lim_lo[rb] = real && a.window > 0 ? max(0, lim_hi[rb] - a.window) : 0;
            const uint16_t* q = static_cast<const uint16_t*>(a.q) + ((size_t)t * a.B + p.b) * a.q_stride + (size_t)h * D;
            const uint32_t flip = p.sc < 0.f ? 0x80008000u : 0u;      // scores are scaled by |sc|
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                // the channels of K's pieces: eight at a time, or halves of sixteen codes
                const int d = FP8 ? (i >> 1) * 64 + g * 16 + (i & 1) * 8 : i * 32 + g * 8;
                u32x4 w = real ? *reinterpret_cast<const u32x4*>(q + d) : u32x4{0, 0, 0, 0};
                w ^= u32x4{flip, flip, flip, flip};
                dst[rb * KS + i][lane] = w;
            }
        }
    }

    // Raw scores of 32 tokens; kf(blk, piece) gives 16 bytes of K, q the queries in LDS.
    // FROM_LDS: K is there too; two products' operands are read while the two before them run, and no
    // more than that ahead (registers).
    template <bool FROM_LDS, typename KF>
    __device__ __forceinline__ void scores(f32x4 (&s)[RB][2], const u32x4 (*q)[64], int lane, KF kf) const
    {
        constexpr int P = FP8 ? 1 : 2;                       // pieces of K that two products take
        u32x4 kw[2][2][P], qw[2][2][RB];
        auto read = [&](int i) {
#pragma unroll
            for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                for (int x = 0; x < P; ++x) kw[i & 1][blk][x] = kf(blk, i * P + x);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) qw[i & 1][x][rb] = q[rb * KS + 2 * i + x][lane];
        };
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) s[rb][0] = s[rb][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        read(0);
#pragma unroll
        for (int i = 0; i < KS / 2; ++i) {
            if (i + 1 < KS / 2) read(i + 1);
            if constexpr (FROM_LDS) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int blk = 0; blk < 2; ++blk) {
                    u32x4 A;
                    if constexpr (FP8) {
                        const u32x4 w = kw[i & 1][blk][0];
                        const uint32_t w0 = x ? w.z : w.x, w1 = x ? w.w : w.y;
                        A = u32x4{kv_from_e4m3<IO, false>(w0), kv_from_e4m3<IO, true>(w0),
                                  kv_from_e4m3<IO, false>(w1), kv_from_e4m3<IO, true>(w1)};
                    } else {
                        A = kw[i & 1][blk][x];
                    }
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb) s[rb][blk] = kv_mfma<IO>(A, qw[i & 1][x][rb], s[rb][blk]);
                }
        }
    }

    // Scores to weights (hi + lo), with the running reference, sum and outputs kept in step; a masked
    // score is -inf.
    __device__ __forceinline__ void weights(const f32x4 (&s)[RB][2], float sc, u32x4 (&ph)[RB], u32x4 (&pl)[RB])
    {
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            float top = s[rb][0][0];
#pragma unroll
            for (int e = 1; e < 8; ++e) top = fmaxf(top, s[rb][e >> 2][e & 3]);
            top *= sc;
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
                float w[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int e = 2 * i + k;
                    // one rounding between the score and its exponent
                    w[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[rb][e >> 2][e & 3], sc, -ref));
                    l[rb] += w[k];
                }
                kv_split<IO>(w[0], w[1], hi[i], lo[i]);
            }
            ph[rb] = u32x4{hi[0], hi[1], hi[2], hi[3]};
            pl[rb] = u32x4{lo[0], lo[1], lo[2], lo[3]};
        }
    }

    // O += V^T P^T for the pieces v0.. of the 32 tokens in vf, of all rows or of those in mine.
    template <bool SOME>
    __device__ __forceinline__ void outputs(int v0, const u32x4 (&ph)[RB], const u32x4 (&pl)[RB], const bool (&mine)[RB])
    {
        auto add = [&](u32x4 A, int j) {
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                const f32x4 x = kv_mfma<IO>(A, pl[rb], kv_mfma<IO>(A, ph[rb], O[rb][j]));
                if constexpr (SOME) O[rb][j] = mine[rb] ? x : O[rb][j];
                else O[rb][j] = x;
            }
            if constexpr (SOME) __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int v = 0; v < VP; ++v) {
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
                    for (int c = 0; c < 4; ++c) add(u32x4{e[c][0], e[c][1], e[c][2], e[c][3]}, (v0 + v) * VE + w * 4 + c);
                }
            } else {
#pragma unroll
                for (int c = 0; c < VE; ++c) {
                    const uint32_t sel = (c & 1) ? 0x07060302u : 0x05040100u;
                    const int w = c >> 1;
                    add(u32x4{__builtin_amdgcn_perm(vf[0][1][v][w], vf[0][0][v][w], sel),
                              __builtin_amdgcn_perm(vf[0][3][v][w], vf[0][2][v][w], sel),
                              __builtin_amdgcn_perm(vf[1][1][v][w], vf[1][0][v][w], sel),
                              __builtin_amdgcn_perm(vf[1][3][v][w], vf[1][2][v][w], sel)}, (v0 + v) * VE + c);
                }
            }
        }
    }

    // Values outside [lo, hi) or of a wrong page become zero.  mt: the lane's first token.
    __device__ __forceinline__ void clear(int mt, int lo, int hi, bool ok0, bool ok1)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int t = mt + (e >> 2) * 16 + (e & 3);
            const bool sees = t < hi && t >= lo && (e < 4 ? ok0 : ok1);
#pragma unroll
            for (int v = 0; v < VP; ++v)
#pragma unroll
                for (int w = 0; w < VW; ++w) vf[e >> 2][e & 3][v][w] = sees ? vf[e >> 2][e & 3][v][w] : 0u;
        }
    }
    // Whether some position that not every row sees holds no number.
    __device__ __forceinline__ bool odd(const KvPart& p, int mt) const
    {
        uint32_t x = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int t = mt + (e >> 2) * 16 + (e & 3);
            uint32_t y = 0;
#pragma unroll
            for (int v = 0; v < VP; ++v)
#pragma unroll
                for (int w = 0; w < VW; ++w) y |= kv_odd<IO, FP8>(vf[e >> 2][e & 3][v][w]);
            x |= t < p.all_lo || t >= p.all_hi ? y : 0u;
        }
        return __builtin_amdgcn_ballot_w64(x != 0) != 0;
    }

    // 32 tokens that every row sees, whose raw scores are s: weights and outputs.  values(v0) fills vf
    // with pieces v0...
    template <typename VF>
    __device__ __forceinline__ void take(const KvPart& p, const f32x4 (&s)[RB][2], VF values)
    {
        u32x4 ph[RB], pl[RB];
        const bool mine[RB] = {};
        values(0);                           // (on their way while the weights are formed)
        weights(s, p.sc_abs(), ph, pl);
#pragma unroll
        for (int v = 0; v < VL; v += VP) {
            if (v > 0) values(v);
            outputs<false>(v, ph, pl, mine);
        }
    }

    // The 32 tokens at t0, whoever sees them.  ok0, ok1: the two blocks' pages are in the cache.
    // values(v0, again) fills vf; again: not for the first time.
    template <typename VF>
    __device__ __forceinline__ void take_masked(const KvAttention& a, const KvPart& p, f32x4 (&s)[RB][2], int t0, bool ok0,
                                                bool ok1, int lane, VF values)
    {
        const int mt = t0 + 4 * kv_opaque(lane >> 4);                            // the lane's first token
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int t = mt + (e >> 2) * 16 + (e & 3);
                const bool sees = t < lim_hi[rb] && t >= lim_lo[rb] && (e < 4 ? ok0 : ok1);
                s[rb][e >> 2][e & 3] = sees ? s[rb][e >> 2][e & 3] : -INFINITY;
            }
        u32x4 ph[RB], pl[RB];
        weights(s, p.sc_abs(), ph, pl);
        // Values that no row sees count as zero, so that 0 * NaN does not arise.  A value that only some
        // drafts see and that is no number would still reach the others: then, and only then, the drafts
        // are taken one by one.
        const int lo = a.window > 0 ? max(0, p.all_hi - a.window) : 0;           // of any row
        bool apart = false;
        if constexpr (VP < VL) {                         // the pieces are not held: looked through first
            if (a.T > 1) {
#pragma unroll
                for (int v = 0; v < VL; v += VP) {
                    values(v, false);
                    clear(mt, lo, p.end, ok0, ok1);
                    apart |= odd(p, mt);
                }
            }
        }
#pragma unroll 1
        for (int d = apart ? 0 : -1; d < (apart ? a.T : 0); ++d) {
            const int hi = d < 0 ? p.end : p.all_hi + d;
            bool mine[RB];
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) mine[rb] = d < 0 || lim_hi[rb] == hi;
#pragma unroll
            for (int v = 0; v < VL; v += VP) {
                values(v, d >= 0);
                clear(mt, d < 0 ? lo : (a.window > 0 ? max(0, hi - a.window) : 0), hi, ok0, ok1);
                if (VP == VL && d < 0 && a.T > 1 && odd(p, mt)) {
                    apart = true;
                    continue;
                }
                outputs<true>(v, ph, pl, mine);
            }
        }
    }

    // Joins the NTW waves (wave = tw * RW + rg) that split a row group's tokens, JP 16-channel groups
    // at a time through so [waves][16][16 JP + 4]; a whole range writes its output, a part its partial rows.
    template <int NT, int RW, int NTW, int JP>
    __device__ __forceinline__ void join(const KvAttention& a, const KvPart& p, float (*so)[16][16 * JP + 4],
                                         float (*s_m)[16], float (*s_l)[16])
    {
        const bool whole = p.whole();
        const int slot = 2 * blockIdx.x + (p.ta == 0 ? 1 : 0);
        const float vs = FP8 ? uload(a.v_scale + p.hkv) : 1.f;
        const int jt = kv_opaque(threadIdx.x), jn = jt & 15, jg = (jt >> 4) & 3, wv = uni(threadIdx.x >> 6);
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            const float lw = sum_over_row_groups(l[rb]);
#pragma unroll
            for (int jp = 0; jp < JN; jp += JP) {
                __syncthreads();                                 // the queries, blocks or part before are done with
                if (jp == 0 && jg == 0) {
                    s_m[wv][jn] = m[rb];
                    s_l[wv][jn] = lw;
                }
                // lane: row n, channels VE (4 g + r).. of each piece's 16 VE; a round takes whole pieces,
                // or JP channels of every lane's VE
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int j = 0; j < JP; j += 4) {
                        const int jj = jp + j, d = (jj / VE) * 16 * VE + (4 * jg + r) * VE + jj % VE;
                        const int c = VE <= JP ? d - jp * 16 : (4 * jg + r) * JP + j;
                        st4(&so[wv][jn][c], f32x4{O[rb][jj][r], O[rb][jj + 1][r], O[rb][jj + 2][r], O[rb][jj + 3][r]});
                    }
                __syncthreads();
                // four channels at a time where a lane's run is no longer, else eight
                constexpr int CW = VE > JP && JP < 8 ? 4 : 8, C8 = 16 * JP / CW;
                for (int i = jt; i < RW * 16 * C8; i += NT) {
                    const int rr = i / C8, c = (i - rr * C8) * CW, grp = rr >> 4, nn = rr & 15;
                    const int rl = (grp * RB + rb) * 16 + nn, row = p.chunk * a.rpc + rl;
                    if (rl >= a.rpc || row >= a.rows) continue;
                    const int d = VE <= JP ? jp * 16 + c : (c / JP) * VE + (jp / VE) * 16 * VE + jp % VE + c % JP;
                    float M = -INFINITY, L = 0.f, x[CW] = {};
#pragma unroll
                    for (int k = 0; k < NTW; ++k) M = fmaxf(M, s_m[k * RW + grp][nn]);
#pragma unroll
                    for (int k = 0; k < NTW; ++k) {
                        const float mk = s_m[k * RW + grp][nn];
                        const float f = mk == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(mk - M);
                        L += f * s_l[k * RW + grp][nn];
#pragma unroll
                        for (int e = 0; e < CW; e += 4) {
                            const f32x4 y = ld4(&so[k * RW + grp][nn][c + e]);
#pragma unroll
                            for (int z = 0; z < 4; ++z) x[e + z] += f * y[z];
                        }
                    }
                    if (whole) {
                        const float inv = L == 0.f ? 0.f : vs / L;
#pragma unroll
                        for (int e = 0; e < CW; ++e) x[e] *= inv;
                        kv_store_o<IO>(a, p.b, p.hkv, row, d, D, x);
                        if (d == 0) kv_store_lse(a, p.b, p.hkv, row, M, L);
                    } else {
                        const size_t at = (size_t)slot * a.rpc + rl;
#pragma unroll
                        for (int e = 0; e < CW; e += 4)
                            st4(a.part_o + at * D + d + e, f32x4{x[e], x[e + 1], x[e + 2], x[e + 3]});
                        if (d == 0) {
                            a.part_ml[2 * at] = M;
                            a.part_ml[2 * at + 1] = L;
                        }
                    }
                }
            }
        }
    }
};

// After a part: the note for kv_combine_kernel, and on to the next part.
__device__ __forceinline__ void kv_next(const KvAttention& a, const KvPart& p, const int* s_pre, KvLine& ln)
{
    const bool whole = p.whole();
    if (threadIdx.x == 0 && p.ta == 0 && (ln.by_range || !whole)) {
        const int range = p.b * ln.hc + p.seg;
        int32_t* mt = a.meta + 2 * (ln.by_range ? range : (int)blockIdx.x);
        mt[0] = ln.by_range ? (whole ? -1 : (int)blockIdx.x) : range;
        mt[1] = ln.cut.owner(s_pre[p.b] + (p.seg + 1) * p.tiles - 1);
    }
    ln.u += p.tb - p.ta;
}

// Up to 16 RB rows share a key/value head: four waves split its tokens, each with K and V straight
// in registers.  Shared memory: prefix sums [B + 1] (dynamic).
template <int IO, bool FP8, int D, int RB, int OCC>
__global__ __launch_bounds__(256, OCC) void kv_attention_kernel(KvAttention a)
{
    using G = KvGeom<FP8, D>;
    using R = KvRows<IO, FP8, D, RB, G::VL>;
    constexpr int JP = G::JN < 8 ? G::JN : 8, EB = G::EB, VE = G::VE, VL = G::VL, VW = G::VW, KL = G::KL;
    extern __shared__ int s_pre[];
    // the waves' queries while tokens pass, their outputs when they are joined
    __shared__ union alignas(16) {
        u32x4 q[4][RB * G::KS][64];
        float o[4][16][16 * JP + 4];
    } sh;
    __shared__ float s_m[4][16], s_l[4][16];
    __shared__ int s_wave[4];
    const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
    KvLine ln;
    if (!kv_begin(a, s_pre, s_wave, ln)) return;
#pragma unroll 1
    while (ln.u < ln.u1) {
        const KvPart p = kv_next_part<FP8>(a, s_pre, ln);
        R rows;
        rows.init();
        constexpr int step = 4 * KV_SUB;
        const int t_first = p.base + p.ta * KV_TILE + wv * KV_SUB;
        const uint8_t* Kc = static_cast<const uint8_t*>(a.K);
        const uint8_t* Vc = static_cast<const uint8_t*>(a.V);
        const uint32_t koff = n * G::ROWB + g * 16;                             // token n, 16 bytes g
        const uint32_t voff = g * 4 * G::ROWB + n * VE * EB;                    // tokens 4 g.., channels VE n..
        u32x4 kf[2][KL];
        auto load_k = [&](size_t b0, size_t b1) {
#pragma unroll
            for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                for (int i = 0; i < KL; ++i) kf[blk][i] = kv_stream<u32x4>(Kc + (blk ? b1 : b0) + i * 64 + koff);
        };
        auto load_v = [&](size_t b0, size_t b1) {
#pragma unroll
            for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int v = 0; v < VL; ++v)
                        kv_words<VW, true>(Vc + (blk ? b1 : b0) + (r * G::ROWB + v * 16 * VE * EB) + voff, rows.vf[blk][r][v]);
        };
        // the first block's keys and values are requested before anything is waited for
        const int nb = t_first < p.tend ? (p.tend - t_first + step - 1) / step : 0;     // the wave's blocks
        int t0 = t_first;
        uint32_t p0 = 0, p1 = 0, c0 = 0, c1 = 0;     // table entries of the next and of the current block
        size_t b0 = 0, b1 = 0;
        if (nb > 0) {
            c0 = kv_page_of(a, p, t0);
            c1 = kv_page_of(a, p, t0 + 16);
            b0 = kv_locate<G::ROWB>(a, p, c0, t0);
            b1 = kv_locate<G::ROWB>(a, p, c1, t0 + 16);
            load_k(b0, b1);
            load_v(b0, b1);
            p0 = kv_page_of(a, p, t0 + step);
            p1 = kv_page_of(a, p, t0 + step + 16);
        }
        __syncthreads();                             // the join before is done with sh
        rows.queries(a, p, 0, sh.q[wv], lane);       // each wave keeps its own copy
        const bool wrong = kv_wrong_pages(a, p, lane);

        // Every block but the last requests the next one unconditionally: the waits for K and V then
        // count exactly the requests behind them.  Blocks that every row sees have a loop of their own
        // (its registers stay clear of the masks').
        int left = nb - 1;
        auto next_k = [&] {
            t0 += step;
            c0 = p0;
            c1 = p1;
            b0 = kv_locate<G::ROWB>(a, p, c0, t0);
            b1 = kv_locate<G::ROWB>(a, p, c1, t0 + 16);
            load_k(b0, b1);
            p0 = kv_page_of(a, p, t0 + step);
            p1 = kv_page_of(a, p, t0 + step + 16);
            __builtin_amdgcn_sched_barrier(0);
        };
        auto next_v = [&] {
            load_v(b0, b1);
            --left;
            __builtin_amdgcn_sched_barrier(0);
        };
        auto scores = [&](f32x4 (&s)[RB][2]) {
            asm volatile("" ::: "memory");           // queries stay in LDS from block to block
            rows.template scores<false>(s, sh.q[wv], lane, [&](int blk, int i) { return kf[blk][i]; });
        };
        auto masked = [&](auto more) {
            f32x4 s[RB][2];
            scores(s);
            const int cur = t0;
            const size_t cb0 = b0, cb1 = b1;
            const bool ok0 = c0 < (uint32_t)a.npages, ok1 = c1 < (uint32_t)a.npages;
            if constexpr (decltype(more)::value) next_k();
            rows.take_masked(a, p, s, cur, ok0, ok1, lane, [&](int, bool again) {
                if (again) load_v(cb0, cb1);
            });
            if constexpr (decltype(more)::value) next_v();
        };
        while (left > 0) {
#pragma unroll 1
            while (left > 0 && (wrong || !p.full(t0, KV_SUB))) masked(std::true_type{});
#pragma unroll 1
            while (left > 0 && !wrong && p.full(t0, KV_SUB)) {
                f32x4 s[RB][2];
                scores(s);
                next_k();
                rows.take(p, s, [](int) {});
                next_v();
            }
        }
        if (left == 0) {
            bool taken = false;
            if constexpr (D * RB < 512) {            // (more registers of outputs are not held twice)
                if ((taken = !wrong && p.full(t0, KV_SUB))) {
                    f32x4 s[RB][2];
                    scores(s);
                    rows.take(p, s, [](int) {});
                }
            }
            if (!taken) masked(std::false_type{});
        }
        rows.template join<256, 1, 4, JP>(a, p, sh.o, s_m, s_l);
        if (ln.whole) break;
        kv_next(a, p, s_pre, ln);
    }
}

// More rows: four waves in RW row groups of 16 RB rows, the 4 / RW waves of a group splitting its
// tokens.  The cache passes through LDS in stages of ST tokens, so that it is read once for all
// rows: each wave requests its quarter of the next stage into registers, and writes it to LDS when
// the workgroup is through with the stage before.  Two such workgroups a CU, so that one computes
// while the other turns its stage: one of eight waves took 111 us where two of four take 104 (64 rows
// over 131k tokens of 128 channels).  K's 16-byte pieces are permuted within a token
// (fold) so that 16 tokens' equal pieces lie in different banks.
template <int IO, bool FP8, int D, int RB, int RW>
__global__ __launch_bounds__(256, 2) void kv_attention_wide_kernel(KvAttention a)
{
    using G = KvGeom<FP8, D>;
    using R = KvRows<IO, FP8, D, RB, 1>;
    constexpr int NTW = 4 / RW, EB = G::EB, VE = G::VE, VW = G::VW, ROWB = G::ROWB;
    constexpr int ST = ROWB <= 128 ? KV_TILE : 16384 / ROWB;     // tokens of a stage
    constexpr int CPB = 16 * ROWB / 1024;                        // 1 KiB chunks of 16 tokens
    constexpr int NC = ST / 16 * CPB;                            // chunks of K, and of V
    constexpr int CJ = NC / 4;                                   // of them a wave's
    constexpr int TPC = 1024 / ROWB;                             // tokens of a chunk
    constexpr int FT = ROWB >= 256 ? 1 : 256 / ROWB, FM = ROWB / 16 < 16 ? ROWB / 16 - 1 : 15;
    constexpr int JP = 4;
    constexpr int CV = CPB > 4 ? CPB / 4 : 1;                    // different parts of a block a wave takes
    static_assert(NC % 4 == 0 && CJ % CV == 0 && (CPB > 4 || 4 % CPB == 0), "every wave takes whole chunks");
    extern __shared__ int s_pre[];
    __shared__ union alignas(16) {
        uint8_t kv[2][ST * ROWB];                                // a stage of K and of V
        float o[4][16][16 * JP + 4];
    } sh;
    __shared__ u32x4 s_q[RW][RB * G::KS][64];
    __shared__ float s_m[4][16], s_l[4][16];
    __shared__ int s_wave[4];
    const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6), rg = wv % RW, tw = wv / RW, n = lane & 15, g = lane >> 4;
    KvLine ln;
    if (!kv_begin(a, s_pre, s_wave, ln)) return;
    // chunk j of a wave is chunk wv + 4 j of the stage: block, and the lane's bytes in the block
    auto block_of = [&](int j) { return (wv + 4 * j) / CPB; };
    uint32_t koff[CV], voff[CV];
#pragma unroll
    for (int c = 0; c < CV; ++c) {
        const int part = (wv + 4 * c) % CPB, tok = part * TPC + lane * 16 / ROWB, pos = lane * 16 % ROWB / 16;
        voff[c] = part * 1024 + lane * 16;
        koff[c] = tok * ROWB + (pos ^ ((tok / FT) & FM)) * 16;
    }
#pragma unroll 1
    while (ln.u < ln.u1) {
        const KvPart p = kv_next_part<FP8>(a, s_pre, ln);
        R rows;
        rows.init();
        const uint8_t* Kc = static_cast<const uint8_t*>(a.K);
        const uint8_t* Vc = static_cast<const uint8_t*>(a.V);
        const int first = uni(p.base + p.ta * KV_TILE), ns = uni(first < p.tend ? (p.tend - first + ST - 1) / ST : 0);
        u32x4 kr[CJ], vr[CJ];                                    // the wave's chunks of the next stage
        uint32_t entry[CJ];                                      // and the pages of those after it
        auto pages = [&](int st) {
#pragma unroll
            for (int j = 0; j < CJ; ++j) entry[j] = kv_page_of(a, p, st + 16 * block_of(j));
        };
        auto request = [&](int st) {
#pragma unroll
            for (int j = 0; j < CJ; ++j) {
                const size_t at = kv_locate<ROWB>(a, p, entry[j], st + 16 * block_of(j));
                kr[j] = kv_stream<u32x4>(Kc + at + koff[j % CV]);
                vr[j] = kv_stream<u32x4>(Vc + at + voff[j % CV]);
            }
            pages(st + ST);
        };
        if (ns > 0) {
            pages(first);
            request(first);
        }
        __syncthreads();                                         // the join before is done with LDS
        rows.queries(a, p, rg * RB, s_q[rg], lane);              // (two waves write the same)
        const bool wrong = kv_wrong_pages(a, p, lane);
        int st = first;
        const int st_end = first + ns * ST;
        auto turn = [&] {                                        // the requested stage to LDS, the next one requested
            __syncthreads();                                     // the stage before is used up
#pragma unroll
            for (int j = 0; j < CJ; ++j) {
                const int c = wv + 4 * j;
                *reinterpret_cast<u32x4*>(sh.kv[0] + c * 1024 + lane * 16) = kr[j];
                *reinterpret_cast<u32x4*>(sh.kv[1] + c * 1024 + lane * 16) = vr[j];
            }
            if (st + ST < st_end) request(st + ST);
            __syncthreads();
        };
        const int fold = (n / FT) & FM;
        auto scores = [&](f32x4 (&s)[RB][2], int sb) {
            const uint8_t* ks = sh.kv[0] + (sb * KV_SUB + n) * ROWB;
            rows.template scores<true>(s, s_q[rg], lane, [&](int blk, int i) {
                return *reinterpret_cast<const u32x4*>(ks + blk * 16 * ROWB + ((i * 4 + g) ^ fold) * 16);
            });
            __builtin_amdgcn_sched_barrier(0);                   // V is read when K is used up
        };
        auto values = [&](int sb, int v) {
            const uint8_t* vs = sh.kv[1] + (sb * KV_SUB + 4 * g) * ROWB + n * VE * EB;
#pragma unroll
            for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    kv_words<VW, false>(vs + (blk * 16 + r) * ROWB + v * 16 * VE * EB, rows.vf[blk][r][0]);
        };
        while (st < st_end) {
#pragma unroll 1
            while (st < st_end && (wrong || !p.full(st, ST))) {
                turn();
                const int nsb = uni(min(ST, p.tend - st + KV_SUB - 1) / KV_SUB);
#pragma unroll 1
                for (int sb = tw; sb < nsb; sb += NTW) {
                    const int t0 = st + sb * KV_SUB;
                    f32x4 s[RB][2];
                    scores(s, sb);
                    const bool ok0 = kv_page_of(a, p, t0) < (uint32_t)a.npages;
                    const bool ok1 = kv_page_of(a, p, t0 + 16) < (uint32_t)a.npages;
                    rows.take_masked(a, p, s, t0, ok0, ok1, lane, [&](int v, bool) { values(sb, v); });
                }
                st += ST;
            }
#pragma unroll 1
            while (st < st_end && !wrong && p.full(st, ST)) {    // every row sees every token
                turn();
#pragma unroll 1
                for (int sb = tw; sb < ST / KV_SUB; sb += NTW) {
                    f32x4 s[RB][2];
                    scores(s, sb);
                    rows.take(p, s, [&](int v) { values(sb, v); });
                }
                st += ST;
            }
        }
        rows.template join<256, RW, NTW, JP>(a, p, sh.o, s_m, s_l);
        if (ln.whole) break;
        kv_next(a, p, s_pre, ln);
    }
}

// Joins the partial rows of one split range, a row at a time.  blockIdx.x is the range where there
// are no more of them than workgroups, else the workgroup that opened it.  256
// threads = D / 4 lanes of four channels x 1024 / D groups of parts.  Bound by the latency of its two
// dependent loads (5 us for 512 ranges of two or three parts), with many rows by the partial rows
// themselves: 12 us for 64 ranges of 64 rows on 256 channels (38 MB).
template <int IO, bool FP8, int D, bool BY_RANGE>
__global__ __launch_bounds__(256) void kv_combine_kernel(KvAttention a)
{
    constexpr int CL = D / 4, PG = 256 / CL;
    __shared__ float s_x[PG][D], s_m[PG], s_l[PG];
    const int hc = a.Hkv * a.nchunk, found = uload(a.meta + 2 * blockIdx.x);
    const int range = BY_RANGE ? blockIdx.x : found, w0 = BY_RANGE ? found : blockIdx.x;
    const int b = max(range, 0) / hc, seg = range - b * hc;
    if ((BY_RANGE && a.active && !uload(a.active + b)) || found < 0) return;
    const int w1 = uload(a.meta + 2 * blockIdx.x + 1);
    const int np = w1 - w0 + 1, tid = threadIdx.x;
    const int hkv = seg / a.nchunk, chunk = seg - hkv * a.nchunk;
    const int c = tid % CL, pg = tid / CL;
    const float vs = FP8 ? uload(a.v_scale + hkv) : 1.f;
    const int rows = min(a.rpc, a.rows - chunk * a.rpc);
    // the opening workgroup's part is its last (slot 1), the others' their first (slot 0)
    auto part = [&](int i, int rl) { return (size_t)(2 * (w0 + i) + (i == 0 ? 1 : 0)) * a.rpc + rl; };
    for (int rl = blockIdx.y; rl < rows; rl += gridDim.y) {
        float M = -INFINITY, L = 0.f;
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
        // eight parts at a time, all of their loads on the way together
        for (int i0 = pg; i0 < np; i0 += 8 * PG) {
            float m[8], l[8];
            f32x4 y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const size_t at = part(min(i0 + k * PG, np - 1), rl);
                m[k] = a.part_ml[2 * at];
                l[k] = a.part_ml[2 * at + 1];
                y[k] = ld4(a.part_o + at * D + 4 * c);
            }
            float mx = M;
#pragma unroll
            for (int k = 0; k < 8; ++k) mx = fmaxf(mx, m[k]);
            const float f0 = M == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(M - mx);
            M = mx;
            L *= f0;
            x *= f0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (i0 + k * PG >= np) continue;
                const float f = m[k] == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m[k] - M);
                L += l[k] * f;
                x += y[k] * f;
            }
        }
        st4(&s_x[pg][4 * c], x);
        if (c == 0) {
            s_m[pg] = M;
            s_l[pg] = L;
        }
        __syncthreads();
        if (tid < D / 8) {
            float MM = -INFINITY, LL = 0.f, y[8] = {};
#pragma unroll
            for (int k = 0; k < PG; ++k) MM = fmaxf(MM, s_m[k]);
#pragma unroll
            for (int k = 0; k < PG; ++k) {
                const float f = s_m[k] == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(s_m[k] - MM);
                LL += s_l[k] * f;
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] += s_x[k][8 * tid + e] * f;
            }
            const float inv = LL == 0.f ? 0.f : vs / LL;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= inv;
            const int row = chunk * a.rpc + rl;
            kv_store_o<IO>(a, b, hkv, row, 8 * tid, D, y);
            if (tid == 0) kv_store_lse(a, b, hkv, row, MM, LL);
        }
        __syncthreads();
    }
}

template <int IO, bool FP8, int D>
static hipError_t kv_attention_width(const KvAttention& a, const KvPlan& p, hipStream_t s)
{
    const int ranges = a.B * a.Hkv * a.nchunk;
    const size_t lds = a.whole ? 0 : (a.B + 1) * sizeof(int);
    const dim3 grid(a.whole || a.by_length ? ranges : p.nwg);
    if (p.wide) {
        if constexpr (D == 256) {
            hipLaunchKernelGGL((kv_attention_wide_kernel<IO, FP8, D, 1, 4>), grid, dim3(256), lds, s, a);
        } else {
            if (p.RW == 2) hipLaunchKernelGGL((kv_attention_wide_kernel<IO, FP8, D, 2, 2>), grid, dim3(256), lds, s, a);
            else hipLaunchKernelGGL((kv_attention_wide_kernel<IO, FP8, D, 2, 4>), grid, dim3(256), lds, s, a);
        }
    } else if (p.RB == 2) {
        hipLaunchKernelGGL((kv_attention_kernel<IO, FP8, D, 2, kv_occ(D, FP8, 2)>), grid, dim3(256), lds, s, a);
    } else {
        hipLaunchKernelGGL((kv_attention_kernel<IO, FP8, D, 1, kv_occ(D, FP8, 1)>), grid, dim3(256), lds, s, a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.whole) return e;
    const int most = ranges <= p.nwg ? ranges : p.nwg;
    const int y = p.rpc < 8192 / most ? p.rpc : 8192 / most;         // rows side by side, within some waves of the chip
    if (ranges <= p.nwg) hipLaunchKernelGGL((kv_combine_kernel<IO, FP8, D, true>), dim3(ranges, y), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((kv_combine_kernel<IO, FP8, D, false>), dim3(p.nwg, y), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int IO, bool FP8>
static hipError_t kv_attention_pick(const KvAttention& a, const KvPlan& p, int D, hipStream_t s)
{
    switch (D) {
        case 64: return kv_attention_width<IO, FP8, 64>(a, p, s);
        case 128: return kv_attention_width<IO, FP8, 128>(a, p, s);
        case 256: return kv_attention_width<IO, FP8, 256>(a, p, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace rs
