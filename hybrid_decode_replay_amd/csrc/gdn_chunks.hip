// gdn_chunks.hip -- the gated delta rule over packed prompts in chunks of 64 tokens (replay_gdn_prefill, bf16).
//
// With g_i the product of alpha over the chunk's tokens up to i, and S the state before the chunk (d_v x d_k):
//
//   A_ij = beta_i g_i / g_j k_i.k_j  (j < i),   T = (I + A)^-1 diag(beta),   P_ij = scale g_i / g_j q_i.k_j  (j <= i)
//   U = T (V - diag(g) K S^T),   O = scale diag(g) Q S^T + P U,   S' = g_64 S + U^T diag(g_64 / g_j) K
//
// T, P and the g's do not depend on S: gdn_chunk_kernel forms them for all chunks and heads at once and leaves them in
// the workspace as the matrix operands that gdn_state_kernel reads, which goes through the chunks of a sequence.  S^T, X =
// V - diag(g) K S^T and U come out of the matrix products in the lanes (column l % 16, rows 4 (l / 16) ..) where the next
// product wants them as its right operand.  For that the rows of a 16-row tile t are not consecutive: row r of it is token
// (or d_k channel)
//   32 (t / 2) + 8 (r / 4) + 4 (t % 2) + r % 4,
// which makes the eight values that a lane holds of tiles 2 s and 2 s + 1 consecutive ones: 32 s + 8 (l / 16) ...
//
// k and q are bf16 numbers; the fp32 operands (S, X, U, T, P) are cut into three bf16 terms of eight bits each, which hold
// all 24, and their products taken down to 2^-24.  Sums are fp32.  (o too: where new values take a large old state's place,
// Q S^T and P U cancel, and terms of 16 bits would leave 2^-16 of the old state in a small o.)
#include "gdn_chunk.hpp"

#include <type_traits>

namespace rs {

// ---- what does not depend on the state ---------------------------------------------------------------------------
// A workgroup of four waves takes a chunk and a group of heads.  k and q go through LDS once; the ten 16 x 16 tiles of the
// lower triangle of K K^T, and K Q^T in tiles whose rows are ordered as above (a lane then holds the eight values of P that it
// stores), stay in registers for the group's heads.  Each head's triangle is inverted in blocks of 16: the four diagonal
// blocks by forward substitution in one wave (a lane a column; the others form and store P meanwhile), then the blocks below
// them column by column, a wave each, in fp32 matrix products.  Bound by its bytes where chunks are many (16 ragged prompts by
// 32 heads read and write 916 MB in 156 us, 5.9 TB/s).
template <int R>
__global__ void __launch_bounds__(256, R == 256 ? 1 : 4) gdn_chunk_kernel(PrefillArgs a, uint8_t* ws)
{
    constexpr int LD = 68;                     // row stride of the 64 x 64 matrices in LDS, in floats
    constexpr int M = R / 32, RB = R * 2, CPR = RB / 16, KL = CPR / 4;
    constexpr int MAT = CHUNK * LD * 4, ROWS = 2 * CHUNK * RB;
    __shared__ __attribute__((aligned(16))) uint8_t both[ROWS > 2 * MAT ? ROWS : 2 * MAT];    // k and q, then T and A
    __shared__ __attribute__((aligned(16))) int gw[CHUNK];
    __shared__ __attribute__((aligned(16))) float gp[CHUNK], bt[CHUNK];
    static_assert((R == 256 ? 2 : 4) * (sizeof both + sizeof gw + sizeof gp + sizeof bt) <= 160 * 1024, "workgroups of a CU");
    float *tm = reinterpret_cast<float*>(both), *am = reinterpret_cast<float*>(both + MAT);
    // 16-byte chunks of a row are exchanged by this, so that 16 rows in order, and in a tile's order, are spread over the banks
    auto key = [](int row) { return ((row & 3) | (row >> 1 & 4) | (((row << 1) ^ (row >> 1)) & 8)) & (CPR - 1); };
    const int tid = threadIdx.x, lane = tid & 63, w = uni(tid >> 6), r = lane & 15, q = lane >> 4;
    const int slot = blockIdx.x / a.G, grp = blockIdx.x - slot * a.G;
    int b = -1, at_slot = 0, ahead = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        const Span s = span_of(a, min(b0 + lane, a.B - 1));
        const uint64_t taken = __ballot(b0 + lane < a.B && s.count > a.skip);
        const int from = s.first / CHUNK + ahead + __popcll(taken & ((1ull << lane) - 1));
        const uint64_t mask = __ballot((taken >> lane & 1) && slot >= from && slot < from + (s.count + CHUNK - 1) / CHUNK);
        if (mask) {
            const int l = 63 - __clzll((long long)mask);
            b = b0 + l;
            at_slot = __builtin_amdgcn_readlane(from, l);
        }
        ahead += __popcll(taken);
    }
    b = uni(b);
    if (b < 0) return;
    const Span s = span_of(a, b);
    const int first = s.first + (slot - uni(at_slot)) * CHUNK, n = min(CHUNK, s.first + s.count - first);

    // (tokens behind the last keep the state, and their beta is 0)
    float al, be;
    auto ask_gates = [&](int h) {
        const size_t at = (size_t)(first + min(lane, n - 1)) * a.H + h;
        al = a.alpha[at];
        be = a.beta[at];
    };
    auto gates = [&]() {
        const bool live = lane < n;
        const Power g2 = decay_of(al, live);
        gw[lane] = g2.whole;
        gp[lane] = g2.part;
        bt[lane] = live ? be : 0.f;
    };
    // (rows behind the last token repeat it)
    {
        const uint16_t* kp = static_cast<const uint16_t*>(a.k) + (int64_t)first * a.k_stride + grp * R;
        const uint16_t* qp = static_cast<const uint16_t*>(a.q) + (int64_t)first * a.q_stride + grp * R;
        u32x4 kl[KL], ql[KL];
        if (w == 0) ask_gates(grp * a.hpg);
#pragma unroll
        for (int i = 0; i < KL; ++i) {
            const int p = tid + 256 * i, row = min(p / CPR, n - 1), c = p % CPR * 8;
            kl[i] = *reinterpret_cast<const u32x4*>(kp + (int64_t)row * a.k_stride + c);
            ql[i] = *reinterpret_cast<const u32x4*>(qp + (int64_t)row * a.q_stride + c);
        }
#pragma unroll
        for (int i = 0; i < KL; ++i) {
            const int p = tid + 256 * i, row = p / CPR, at = row * RB + ((p % CPR ^ key(row)) * 16);
            *reinterpret_cast<u32x4*>(both + at) = kl[i];
            *reinterpret_cast<u32x4*>(both + CHUNK * RB + at) = ql[i];
        }
    }
    __syncthreads();
    if (w == 0) gates();
    // tiles of K K^T: (0, 0), (1, 1), (1, 0), (3, 0) of wave 0; (2, 2), (2, 1); (3, 3), (3, 2); (2, 0), (3, 1) of the others,
    // which have two of the pairs (row tile, 32 tokens) of P each.  Of 32 tokens or fewer: the first two tile rows alone.
    const bool few = n <= 32;
    const int rows[4] = {w == 0 ? 0 : w == 2 ? 3 : 2, w == 0 ? 1 : w == 1 ? 2 : 3, 1, 3}, cols[4] = {w == 3 ? 0 : w == 0 ? 0 : w + 1, w == 0 ? 1 : w == 2 ? 2 : 1, 0, 0};
    auto has = [&](int i) { return (i < 2 || w == 0) && (!few || rows[i] < 2); };
    auto piece = [&](int e, int& t, int& sg) {
        const int f = 2 * (w - 1) + e;
        t = f < 2 ? f : 2 + ((f - 2) >> 1);
        sg = f < 2 ? 0 : f & 1;
        return f;
    };
    const bool has_p = w > 0 && (!few || w == 1);
    auto operand = [&](int base, int row, int m) {
        return *reinterpret_cast<const bf16x8*>(both + base + row * RB + (((4 * m + q) ^ key(row)) * 16));
    };
    f32x4 kk[4], kq[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        kk[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (!has(i)) continue;
#pragma unroll
        for (int m = 0; m < M; ++m)
            kk[i] = mfma16x16x32bf16(operand(0, 16 * rows[i] + r, m), operand(0, 16 * cols[i] + r, m), kk[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) kk[i][e] = 16 * cols[i] + r < 16 * rows[i] + 4 * q + e ? kk[i][e] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        kq[e][0] = kq[e][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (!has_p) continue;
        int t, sg;
        piece(e, t, sg);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const bf16x8 bq = operand(CHUNK * RB, tile_row(t, r), m);
#pragma unroll
            for (int x = 0; x < 2; ++x) kq[e][x] = mfma16x16x32bf16(operand(0, tile_row(2 * sg + x, r), m), bq, kq[e][x]);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int k = 0; k < 4; ++k) kq[e][x][k] = 32 * sg + 8 * q + 4 * x + k <= tile_row(t, r) ? a.scale * kq[e][x][k] : 0.f;
    }
    __syncthreads();
    for (int h = grp * a.hpg; h < (grp + 1) * a.hpg; ++h) {
        uint8_t* out = ws + ((size_t)slot * a.H + h) * GDN_CHUNK_BYTES;
        // (of places that are masked, whose products are 0, a finite number)
        auto since = [&](int wi, float pi, int wj, float pj) { return power(min(wi - wj, 126), pi - pj); };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!has(i)) continue;
            const int col = 16 * cols[i] + r, row = 16 * rows[i] + 4 * q;
            const i32x4 wi = *reinterpret_cast<const i32x4*>(gw + row);
            const f32x4 pi = ld4(gp + row), be4 = ld4(bt + row);
            const int wj = gw[col];
            const float pj = gp[col];
#pragma unroll
            for (int e = 0; e < 4; ++e) am[(row + e) * LD + col] = be4[e] * since(wi[e], pi[e], wj, pj) * kk[i][e];
        }
        __syncthreads();
        if (w == 0) {
            // block q of the diagonal, column r of its inverse
            float t[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float* row = am + (16 * q + i) * LD + 16 * q;
                float x = i == r ? 1.f : 0.f;
#pragma unroll
                for (int j = 0; j < i; ++j) x = __builtin_fmaf(-row[j], t[j], x);
                t[i] = x;
                if (i == 8 || i == 12) __builtin_amdgcn_sched_barrier(0);       // (all rows at once would take the registers of a fourth workgroup)
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) tm[(16 * q + i) * LD + 16 * q + r] = t[i];
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (!has_p) break;
                int t, sg;
                const int f = piece(e, t, sg), i = tile_row(t, r), j0 = 32 * sg + 8 * q;
                const int wi = gw[i];
                const float pi = gp[i];
                f32x4 p[2];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        p[x][k] = since(wi, pi, gw[j0 + 4 * x + k], gp[j0 + 4 * x + k]) * kq[e][x][k];
#pragma unroll
                for (int x = 0; x < 2; ++x) *reinterpret_cast<f32x4*>(out + (PIECE_P + 2 * f + x) * 1024 + lane * 16) = p[x];
            }
            if (w == 1) {
                float* g = reinterpret_cast<float*>(out + PIECE_G * 1024);
                const float whole = power(gw[lane], gp[lane]);
                g[lane] = whole;
                g[CHUNK + lane] = a.scale * whole;
                g[2 * CHUNK + lane] = power(gw[CHUNK - 1] - gw[lane], gp[CHUNK - 1] - gp[lane]);
            }
        }
        __syncthreads();
        if (w < 3) {
            // column w of blocks: T_bc = -T_bb sum over k of A_bk T_kc.  A lane's four rows of a result are the four
            // values of the contraction that it hands to the next product.
            f32x4 col[4];
            auto product = [&](const float* left, int rb, int cb, f32x4 right, f32x4 sum) {
                const f32x4 l = ld4(left + (16 * rb + r) * LD + 16 * cb + 4 * q);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum = mfma16x16x4(l[e], right[e], sum);
                return sum;
            };
#pragma unroll
            for (int e = 0; e < 4; ++e) col[0][e] = tm[(16 * w + 4 * q + e) * LD + 16 * w + r];
#pragma unroll
            for (int d = 1; d < 4; ++d) {
                const int rb = w + d;
                if (rb > (few ? 1 : 3)) break;
                const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
                f32x4 sum = product(am, rb, w, col[0], zero);         // (a sum each: products of one would wait for one another)
#pragma unroll
                for (int k = 1; k < d; ++k) sum += product(am, rb, w + k, col[k], zero);
                col[d] = -product(tm, rb, rb, sum, zero);
#pragma unroll
                for (int e = 0; e < 4; ++e) tm[(16 * rb + 4 * q + e) * LD + 16 * w + r] = col[d][e];
            }
        }
        __syncthreads();
        for (int f = w; f < (few ? 2 : FRAGS); f += 4) {
            const int t = f < 2 ? f : 2 + ((f - 2) >> 1), sg = f < 2 ? 0 : (f & 1);
            const int i = tile_row(t, r), j0 = 32 * sg + 8 * q;
            const bool lower = j0 >> 4 <= i >> 4;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = lower ? tm[i * LD + j0 + e] * bt[j0 + e] : 0.f;
            const Terms3 c = cut3(v);
#pragma unroll
            for (int x = 0; x < 3; ++x) *reinterpret_cast<bf16x8*>(out + (x * FRAGS + f) * 1024 + lane * 16) = c.t[x];
        }
        if (h + 1 == (grp + 1) * a.hpg) break;
        if (w == 0) ask_gates(h + 1);
        __syncthreads();
        if (w == 0) gates();
        __syncthreads();
    }
}

// ---- from chunk to chunk -----------------------------------------------------------------------------------------
// A workgroup of four waves takes 16 NS columns of d_v of one sequence and head.  Wave w works on row tile w of the chunk's
// tokens (X, U, O) and on a quarter of the state's d_k channels; what each needs of the others' S, X and U passes through
// LDS as the bf16 terms that the products take: three barriers a chunk.  T, P, the g's, k, q and v of the chunks ahead are
// asked for as soon as those of this one are used.  The unit that takes vector loads (some 25 cycles for each KiB) is as
// busy as the matrix cores, so nothing is loaded twice: T, P and q as operands straight to registers, the g's and k through
// LDS for all four waves (k also read across, as k^T), v eight bytes a lane and turned in LDS.  Bound by the chain of the three
// exchanges: 512 chunks of one sequence by 32 heads 980 us, 1.9 us a chunk, of which the products of a wave are a fifth.
// One strip a workgroup where that gives 512 or fewer, else two, which read T, P, q and k once for both (16 ragged prompts, with
// the launch before: 818 us with two strips, 978 with one).
// Returns whether there is such a head.
template <int R, int NS>
__device__ __forceinline__ bool state_of(const PrefillArgs& a, const uint8_t* ws, int slices, int i8)
{
    constexpr int M = R / 32, TW = R / 64, RB = R * 2;      // 32-channel steps, state tiles of a wave, bytes of a k row
    constexpr int CPR = RB / 16, KL = CPR / 4;              // 16-byte chunks of a row, of k that a lane brings to LDS
    __shared__ __attribute__((aligned(16))) uint8_t kbuf[CHUNK * RB];
    __shared__ u32x4 sbuf[NS][M][3][64], xbuf[NS][2][3][64], dbuf[NS][2][3][64], ubuf[NS][2][3][64];
    __shared__ __attribute__((aligned(16))) float gbuf[3][CHUNK];
    static_assert(2 * (sizeof kbuf + sizeof sbuf + sizeof xbuf + sizeof dbuf + sizeof ubuf + sizeof gbuf) <= 160 * 1024, "workgroups of a CU");
    const int tid = threadIdx.x, lane = tid & 63, w = uni(tid >> 6), r = lane & 15, q = lane >> 4;
    // Workgroups go to the 8 XCDs in turn.  The slices of a head read the same operands and go to one XCD; heads go to all,
    // so that no XCD gets the longest sequences (16 ragged prompts, two for each XCD: 874 us against 818).
    const int spread8 = a.most * a.H % 8 == 0;
    const int kh = spread8 ? i8 / (8 * slices) * 8 + i8 % 8 : i8 / slices, sl = spread8 ? i8 / 8 % slices : i8 % slices;
    const Turn which = turn_of(a, kh / a.H);
    const int b = uni(which.b), h = kh % a.H, bh = b * a.H + h, g = h / a.hpg;
    if (b < 0 || which.ahead >= a.most) return false;
    const Span s = span_of(a, b);
    const int nc = (s.count + CHUNK - 1) / CHUNK;
    // columns of strip n (one past the last takes the last one's, and is not stored)
    const int strips = a.C / 16, strip0 = sl * NS;
    int col[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) col[n] = min(strip0 + n, strips - 1) * 16;

    const int sg_of = w >> 1, half = w & 1;                 // this wave's row tile among the 32-token steps
    const int my_row = tile_row(w, r), my_rows = tile_row(w, 4 * q);        // its rows as operands, and as results
    const uint8_t* pack = ws + ((size_t)(s.first / CHUNK + uni(which.ahead)) * a.H + h) * GDN_CHUNK_BYTES;
    const int64_t pack_step = (int64_t)a.H * GDN_CHUNK_BYTES;

    // where this lane reads a chunk's rows, from the chunk's first (rows behind the last token repeat it: their columns of T
    // and P are 0).  Worked out once, and again for a last chunk that is not whole.
    const uint16_t *qp, *vp, *klp[KL];
    auto place = [&](int last) {
        qp = static_cast<const uint16_t*>(a.q) + (int64_t)(s.first + min(my_row, last)) * a.q_stride + g * R + 8 * q;
        vp = static_cast<const uint16_t*>(a.v) + (int64_t)(s.first + min(tile_row(w, lane >> 2), last)) * a.v_stride + h * a.C + (lane & 3) * 4;
    };
    auto place_k = [&](int last) {
#pragma unroll
        for (int i = 0; i < KL; ++i)
            klp[i] = static_cast<const uint16_t*>(a.k) + (int64_t)(s.first + min((tid + 256 * i) / CPR, last)) * a.k_stride + g * R +
                     (tid + 256 * i) % CPR * 8;
    };
    const int tail = s.count - (nc - 1) * CHUNK;            // tokens of the last chunk
    // where this wave turns v (before U is formed, in its place) and o (behind the third barrier, in X's)
    uint16_t *turn_v = reinterpret_cast<uint16_t*>(ubuf) + w * NS * 256, *turn_o = reinterpret_cast<uint16_t*>(xbuf) + w * NS * 256;
    bf16x8 qf[M], tf[2][3];
    f32x4 pf[2][2];
    u32x4 kl[KL];
    u32x2 v[NS];
    float gl = 0.f;
    auto ask_k = [&](int c) {
        if (c == nc - 1 && tail < CHUNK) place_k(tail - 1);
#pragma unroll
        for (int i = 0; i < KL; ++i) kl[i] = *reinterpret_cast<const u32x4*>(klp[i] + (int64_t)c * CHUNK * a.k_stride);
        gl = reinterpret_cast<const float*>(pack + c * pack_step + PIECE_G * 1024)[min(tid, 3 * CHUNK - 1)];
    };
    auto keep_k = [&]() {
#pragma unroll
        for (int i = 0; i < KL; ++i) {
            const int p = tid + 256 * i, row = p / CPR;
            *reinterpret_cast<u32x4*>(kbuf + row * RB + ((p % CPR ^ (spread(row) & (CPR - 1))) * 16)) = kl[i];
        }
        if (w < 3) gbuf[w][lane] = gl;
    };
    auto ask_rows = [&](int c) {
#pragma unroll
        for (int m = 0; m < M; ++m) qf[m] = *reinterpret_cast<const bf16x8*>(qp + (int64_t)c * CHUNK * a.q_stride + 32 * m);
    };
    auto ask_v = [&](int c) {
#pragma unroll
        for (int n = 0; n < NS; ++n) v[n] = *reinterpret_cast<const u32x2*>(vp + (int64_t)c * CHUNK * a.v_stride + col[n]);
    };
    auto ask_t = [&](int c) {
        const uint8_t* from = pack + c * pack_step + lane * 16;
#pragma unroll
        for (int sg = 0; sg < 2; ++sg) {
            if (sg > sg_of) break;
            const int f = w < 2 ? w : 2 * w - 2 + sg;
#pragma unroll
            for (int e = 0; e < 3; ++e) tf[sg][e] = *reinterpret_cast<const bf16x8*>(from + (e * FRAGS + f) * 1024);
        }
    };
    auto ask_p = [&](int c) {
        const uint8_t* from = pack + c * pack_step + lane * 16;
#pragma unroll
        for (int sg = 0; sg < 2; ++sg) {
            if (sg > sg_of) break;
            const int f = w < 2 ? w : 2 * w - 2 + sg;
#pragma unroll
            for (int e = 0; e < 2; ++e) pf[sg][e] = *reinterpret_cast<const f32x4*>(from + (PIECE_P + 2 * f + e) * 1024);
        }
    };
    // this wave's part of the state, for everyone
    f32x4 S[NS][TW];
    auto tell_state = [&]() {
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            if constexpr (TW == 1) {
                const Cut c = cut(S[n][0]);
#pragma unroll
                for (int e = 0; e < 3; ++e) reinterpret_cast<u32x2*>(&sbuf[n][w >> 1][e][lane])[w & 1] = c.t[e];
            } else {
#pragma unroll
                for (int t = 0; t < TW; t += 2) {
                    const Terms3 c = cut3(S[n][t], S[n][t + 1]);
#pragma unroll
                    for (int e = 0; e < 3; ++e) sbuf[n][(w * TW + t) >> 1][e][lane] = __builtin_bit_cast(u32x4, c.t[e]);
                }
            }
        }
    };
    if (nc > 0) {
        place(nc > 1 ? CHUNK - 1 : tail - 1);
        place_k(CHUNK - 1);
        ask_k(0);
        ask_rows(0);
        ask_v(0);
        ask_t(0);
        ask_p(0);
        keep_k();
        ask_k(min(1, nc - 1));
    }
    const size_t sat = (size_t)bh * a.C * R + 8 * q;
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < TW; ++i) {
            const int t = w * TW + i;
            S[n][i] = a.S_in ? ld4(a.S_in + sat + (size_t)(col[n] + r) * R + 32 * (t >> 1) + 4 * (t & 1)) : f32x4{0.f, 0.f, 0.f, 0.f};
        }
    if (nc > 0) tell_state();
    float none = 0.f;                                       // NaN once an o was an infinity or NaN
    // One chunk; BOTH: it has more than 32 tokens.  (Of fewer, waves 2 and 3 have none, and U has none behind them.)
    auto chunk = [&](auto BOTH, int c) {
        constexpr bool both = decltype(BOTH)::value;
        const bool busy = both || w < 2;
        // (the last chunk asks for itself again: loads that depend on a condition would be waited for where it ends)
        const int next = min(c + 1, nc - 1);
        if (next == nc - 1 && tail < CHUNK) place(tail - 1);
        lds_barrier();
        // k across: d_k channels of this wave's tiles as rows, tokens 32 sg + 8 q .. + 7, four rows of 16 values at a time
        bf16x8 kt[2][TW];
#pragma unroll
        for (int sg = 0; sg < (both ? 2 : 1); ++sg)
#pragma unroll
            for (int i = 0; i < TW; ++i) {
                const int t = w * TW + i, row = 32 * sg + 8 * q + (r >> 2), ch = 4 * (t >> 1) + (r & 3);
                auto across = [&](int row) {
                    return read_across(kbuf + row * RB + ((ch ^ (spread(row) & (CPR - 1))) * 16) + (t & 1) * 8);
                };
                kt[sg][i] = join(across(row), across(row + 4));
            }
        const float whole = gbuf[0][CHUNK - 1];
        f32x4 x[NS], o[NS];
        if (busy) {
            // K S^T and Q S^T (a sum for each term: the products of one sum would wait for one another)
            bf16x8 kf[M];
#pragma unroll
            for (int m = 0; m < M; ++m)
                kf[m] = *reinterpret_cast<const bf16x8*>(kbuf + my_row * RB + (((4 * m + q) ^ (r & (CPR - 1))) * 16));
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                f32x4 xe[3] = {}, oe[3] = {};
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int e = 0; e < 3; ++e) {
                        const bf16x8 sc = __builtin_bit_cast(bf16x8, sbuf[n][m][e][lane]);
                        xe[e] = mfma16x16x32bf16(kf[m], sc, xe[e]);
                        oe[e] = mfma16x16x32bf16(qf[m], sc, oe[e]);
                    }
                x[n] = xe[0] + (xe[1] + xe[2]);
                o[n] = oe[0] + (oe[1] + oe[2]);
            }
        }
        ask_rows(next);
        if (busy) {
            // X, and O as far as the state before the chunk goes
#pragma unroll
            for (int n = 0; n < NS; ++n) *reinterpret_cast<u32x2*>(turn_v + n * 256 + lane * 4) = v[n];
            wave_lds_sync();
            const f32x4 gi = ld4(&gbuf[0][my_rows]), go = ld4(&gbuf[1][my_rows]);
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                const u32x2 y = read_across(reinterpret_cast<const uint8_t*>(turn_v + n * 256 + (4 * q + (r >> 2)) * 16 + (r & 3) * 4));
                const float vf[4] = {__builtin_bit_cast(float, y.x << 16), __builtin_bit_cast(float, y.x & 0xffff0000u),
                                     __builtin_bit_cast(float, y.y << 16), __builtin_bit_cast(float, y.y & 0xffff0000u)};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[n][i] = __builtin_fmaf(-gi[i], x[n][i], vf[i]);
                    o[n][i] *= go[i];
                }
                const Cut t = cut(x[n]);
#pragma unroll
                for (int e = 0; e < 3; ++e) reinterpret_cast<u32x2*>(&xbuf[n][sg_of][e][lane])[half] = t.t[e];
            }
        }
        ask_v(next);
        lds_barrier();
        if (busy) {
            // U = T X
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                f32x4 ue[3] = {};
#pragma unroll
                for (int sg = 0; sg < (both ? 2 : 1); ++sg) {
                    if (sg > sg_of) break;
                    bf16x8 xc[3];
#pragma unroll
                    for (int e = 0; e < 3; ++e) xc[e] = __builtin_bit_cast(bf16x8, xbuf[n][sg][e][lane]);
                    product24(tf[sg], xc, ue);
                }
                const f32x4 u = ue[0] + (ue[1] + ue[2]);
                const Cut t = cut(u), d = cut(u * ld4(&gbuf[2][my_rows]));
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    reinterpret_cast<u32x2*>(&dbuf[n][sg_of][e][lane])[half] = d.t[e];
                    reinterpret_cast<u32x2*>(&ubuf[n][sg_of][e][lane])[half] = t.t[e];
                }
            }
        }
        ask_t(next);
        lds_barrier();
        // S' = g S + K^T (U g / g_j), this wave's channels
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < TW; ++i) S[n][i] *= whole;
#pragma unroll
        for (int sg = 0; sg < (both ? 2 : 1); ++sg)
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    const bf16x8 uc = __builtin_bit_cast(bf16x8, dbuf[n][sg][e][lane]);
#pragma unroll
                    for (int i = 0; i < TW; ++i) S[n][i] = mfma16x16x32bf16(kt[sg][i], uc, S[n][i]);
                }
        if (busy) {
            // O += P U (P's terms are cut here: fp32 are a third fewer bytes in the workspace and registers that wait)
            f32x4 oe[NS][3];
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                oe[n][0] = o[n];
                oe[n][1] = oe[n][2] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int sg = 0; sg < (both ? 2 : 1); ++sg) {
                if (sg > sg_of) break;
                const Terms3 p = cut3(pf[sg][0], pf[sg][1]);
#pragma unroll
                for (int n = 0; n < NS; ++n) {
                    bf16x8 uc[3];
#pragma unroll
                    for (int e = 0; e < 3; ++e) uc[e] = __builtin_bit_cast(bf16x8, ubuf[n][sg][e][lane]);
                    product24(p.t, uc, oe[n]);
                }
            }
#pragma unroll
            for (int n = 0; n < NS; ++n) o[n] = oe[n][0] + (oe[n][1] + oe[n][2]);
        }
        tell_state();
        keep_k();
        ask_p(next);
        ask_k(min(c + 2, nc - 1));
        if (busy) {
            // through LDS, so that a lane stores eight bytes of a token
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) none = __builtin_fmaf(o[n][i], 0.f, none);
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) turn_o[n * 256 + (4 * q + i) * 16 + r] = f32_to_bf16_bits(o[n][i]);
            wave_lds_sync();
            const int row = tile_row(w, lane >> 2), left = s.count - c * CHUNK;
            uint16_t* op = static_cast<uint16_t*>(a.o) + ((size_t)(s.first + c * CHUNK + row) * a.H + h) * a.C + (lane & 3) * 4;
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                const u32x2 y = *reinterpret_cast<const u32x2*>(turn_o + n * 256 + lane * 4);
                if (row < left && strip0 + n < strips) *reinterpret_cast<u32x2*>(op + col[n]) = y;
            }
        }
    };
    for (int c = 0; c + 1 < nc; ++c) chunk(std::true_type{}, c);
    if (nc > 0) {
        if (tail > 32) chunk(std::true_type{}, nc - 1);
        else chunk(std::false_type{}, nc - 1);
        int bad = !(none == 0.f);
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < TW; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) bad |= not_finite(S[n][i][e]);
        if (__syncthreads_or(bad)) {
            // (the rows of o that the chunks wrote before those that are written now)
            __threadfence();
            __syncthreads();
            if (w < NS && strip0 + w < strips) strip_by_tokens<R>(s, b, h, (strip0 + w) * 16);
            return true;
        }
    }
    if (a.S_out) {
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < TW; ++i) {
                const int t = w * TW + i;
                if (strip0 + n < strips) st4(a.S_out + sat + (size_t)(col[n] + r) * R + 32 * (t >> 1) + 4 * (t & 1), S[n][i]);
            }
    }
    return true;
}

// Of sequences among short ones there may be few: workgroups that only find there is none for them take some 40 us for 192
// pieces by 32 heads, so no more than 2048 start and go on to the next ones.
template <int R, int NS, bool AMONG>
__global__ void __launch_bounds__(256, R == 256 ? 1 : 2) gdn_state_kernel(PrefillArgs a, const uint8_t* ws, int slices)
{
    if constexpr (AMONG) {
        const int all = a.most * a.H * slices;
        for (int i = blockIdx.x; i < all; i += gridDim.x) {
            // (the grid is whole heads for each XCD, so later turns are of later sequences)
            if (!state_of<R, NS>(args_again(), ws, slices, i)) break;
            __syncthreads();
        }
    } else {
        state_of<R, NS>(a, ws, slices, blockIdx.x);
    }
}

namespace {

template <int R, int NS>
hipError_t run(const PrefillArgs& a, uint8_t* ws, hipStream_t s)
{
    const int slices = (a.C / 16 + NS - 1) / NS;
    const uint32_t all = (uint32_t)a.most * a.H * slices, some = (2048 + 8 * slices - 1) / (8 * slices) * (8 * slices);
    if (a.skip < 0) gdn_state_kernel<R, NS, false><<<all, 256, 0, s>>>(a, ws, slices);
    else gdn_state_kernel<R, NS, true><<<min(all, some), 256, 0, s>>>(a, ws, slices);
    return hipGetLastError();
}

template <int R>
hipError_t pick(const PrefillArgs& a, uint8_t* ws, hipStream_t s)
{
    const uint32_t slots = (uint32_t)(a.rows / CHUNK + a.most);
    gdn_chunk_kernel<R><<<slots * a.G, 256, 0, s>>>(a, ws);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const long long strips = (long long)a.most * a.H * (a.C / 16);
    return strips <= 512 || R == 256 ? run<R, 1>(a, ws, s) : run<R, R == 256 ? 1 : 2>(a, ws, s);
}

}  // namespace

hipError_t launch_gdn_prefill_chunks(const PrefillArgs& a, uint8_t* ws, hipStream_t s)
{
    return a.R == 64 ? pick<64>(a, ws, s) : a.R == 128 ? pick<128>(a, ws, s) : pick<256>(a, ws, s);
}

}  // namespace rs
