// gdn_short.hip -- the gated delta rule over prompts, or pieces of them, of at most 32 tokens (replay_gdn_prefill, bf16).
//
// The chunk's algebra of gdn_chunks.hip in one launch: a workgroup takes a head, forms T and P of its tokens in LDS, and each
// of its four waves then takes strips of 16 d_v columns of the state one after the other, from load to store, the next one on
// its way: no barrier, no workspace.  Bound by the states' bytes: 192 pieces of 1 to 33 tokens by 32 heads (890 MB) 199 us.
#include "gdn_chunk.hpp"

namespace rs {

template <int R>
__global__ void __launch_bounds__(256, R == 256 ? 1 : 2) gdn_short_kernel(PrefillArgs a)
{
    constexpr int LD = 36, N = GDN_SHORT;
    constexpr int M = R / 32, NT = R / 16, RB = R * 2, CPR = RB / 16, KL = CPR / 8;
    static_assert(N == 32, "two row tiles");
    __shared__ __attribute__((aligned(16))) uint8_t kbuf[N * RB], qbuf[N * RB];
    __shared__ __attribute__((aligned(16))) float am[N * LD], tm[N * LD], pm[N * LD];
    __shared__ __attribute__((aligned(16))) uint16_t turn[4][2][16 * 16];      // v, then o, of a wave's strip
    __shared__ int gw[N];
    __shared__ float gp[N], bt[N];
    const int tid = threadIdx.x, lane = tid & 63, w = uni(tid >> 6), r = lane & 15, q = lane >> 4;
    const int bh = blockIdx.x, b = bh / a.H, h = bh - b * a.H, g = h / a.hpg;
    const Span s = span_of(a, b);
    const int n = s.count, strips = a.C / 16;
    if (n > N) return;

    const size_t sat = ((size_t)bh * a.C + r) * R + 8 * q;
    const uint16_t* vp[2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
        vp[t] = static_cast<const uint16_t*>(a.v) + (int64_t)(s.first + min(tile_row(t, lane >> 2), n - 1)) * a.v_stride + h * a.C + (lane & 3) * 4;
    f32x4 S[NT], Sn[NT];
    u32x2 vn[2];
    auto ask = [&](int strip) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
            Sn[t] = a.S_in ? ld4(a.S_in + sat + (size_t)strip * 16 * R + 32 * (t >> 1) + 4 * (t & 1)) : f32x4{0.f, 0.f, 0.f, 0.f};
        if (n > 0) {
#pragma unroll
            for (int t = 0; t < 2; ++t) vn[t] = *reinterpret_cast<const u32x2*>(vp[t] + strip * 16);
        }
    };
    auto keep = [&](int strip) {
        if (!a.S_out) return;
#pragma unroll
        for (int t = 0; t < NT; ++t) st4(a.S_out + sat + (size_t)strip * 16 * R + 32 * (t >> 1) + 4 * (t & 1), S[t]);
    };
    if (n == 0) {
        for (int strip = w; strip < strips; strip += 4) {
            ask(strip);
#pragma unroll
            for (int t = 0; t < NT; ++t) S[t] = Sn[t];
            keep(strip);
        }
        return;
    }

    // rows behind the last token repeat it; their beta is 0
    float al = 1.f, be = 0.f;
    if (w == 3) {
        const size_t at = (size_t)(s.first + min(lane, n - 1)) * a.H + h;
        al = a.alpha[at];
        be = a.beta[at];
    }
    {
        const uint16_t* kp = static_cast<const uint16_t*>(a.k) + (int64_t)s.first * a.k_stride + g * R;
        const uint16_t* qp = static_cast<const uint16_t*>(a.q) + (int64_t)s.first * a.q_stride + g * R;
        u32x4 kl[KL], ql[KL];
#pragma unroll
        for (int i = 0; i < KL; ++i) {
            const int p = tid + 256 * i, row = min(p / CPR, n - 1), c = p % CPR * 8;
            kl[i] = *reinterpret_cast<const u32x4*>(kp + (int64_t)row * a.k_stride + c);
            ql[i] = *reinterpret_cast<const u32x4*>(qp + (int64_t)row * a.q_stride + c);
        }
        if (w < strips) ask(w);
#pragma unroll
        for (int i = 0; i < KL; ++i) {
            const int p = tid + 256 * i, row = p / CPR, at = row * RB + ((p % CPR ^ (spread(row) & (CPR - 1))) * 16);
            *reinterpret_cast<u32x4*>(kbuf + at) = kl[i];
            *reinterpret_cast<u32x4*>(qbuf + at) = ql[i];
        }
    }
    if (w == 3) {
        const bool live = lane < n;
        const Power g2 = decay_of(al, live);
        if (lane < N) {
            gw[lane] = g2.whole;
            gp[lane] = g2.part;
            bt[lane] = live ? be : 0.f;
        }
    }
    lds_barrier();
    auto since = [&](int i, int j) { return power(gw[i] - gw[j], gp[i] - gp[j]); };
    if (w < 3) {
        // tiles (0, 0), (1, 1) and (1, 0) of K K^T and Q K^T, rows and columns in order
        const int rt = w > 0 ? 1 : 0, ct = w == 1 ? 1 : 0;
        auto operand = [&](const uint8_t* from, int t, int m) {
            const int row = 16 * t + r;
            return *reinterpret_cast<const bf16x8*>(from + row * RB + (((4 * m + q) ^ (spread(row) & (CPR - 1))) * 16));
        };
        f32x4 kk = {0.f, 0.f, 0.f, 0.f}, qk = kk;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const bf16x8 bk = operand(kbuf, ct, m);
            kk = mfma16x16x32bf16(operand(kbuf, rt, m), bk, kk);
            qk = mfma16x16x32bf16(operand(qbuf, rt, m), bk, qk);
        }
        const int col = 16 * ct + r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = 16 * rt + 4 * q + e;
            const float d = since(row, col);
            am[row * LD + col] = col < row ? bt[row] * d * kk[e] : 0.f;
            pm[row * LD + col] = col <= row ? a.scale * d * qk[e] : 0.f;
        }
    }
    lds_barrier();
    if (w == 3) {
        // the two diagonal blocks (lanes 32.. repeat them), a lane a column, then T_10 = -T_11 A_10 T_00
        const int d = q & 1;
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float* row = am + (16 * d + i) * LD + 16 * d;
            float x = i == r ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) x = __builtin_fmaf(-row[j], t[j], x);
            t[i] = x;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) tm[(16 * d + i) * LD + 16 * d + r] = t[i];
        wave_lds_sync();
        const f32x4 l0 = ld4(am + (16 + r) * LD + 4 * q), l1 = ld4(tm + (16 + r) * LD + 16 + 4 * q);
        f32x4 x = {0.f, 0.f, 0.f, 0.f}, y = x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x = mfma16x16x4(l0[e], tm[(4 * q + e) * LD + r], x);
#pragma unroll
        for (int e = 0; e < 4; ++e) y = mfma16x16x4(l1[e], x[e], y);
#pragma unroll
        for (int e = 0; e < 4; ++e) tm[(16 + 4 * q + e) * LD + r] = -y[e];
    }
    // K S^T and Q S^T of a strip (a sum for each term: the products of one sum would wait for one another)
    f32x4 x[2], o[2];
    auto read_out = [&]() {
        f32x4 xe[2][3], oe[2][3];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 3; ++e) xe[t][e] = oe[t][e] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const Terms3 sc = cut3(S[2 * m], S[2 * m + 1]);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int at = tile_row(t, r) * RB + (((4 * m + q) ^ (r & (CPR - 1))) * 16);
                const bf16x8 kf = *reinterpret_cast<const bf16x8*>(kbuf + at), qf = *reinterpret_cast<const bf16x8*>(qbuf + at);
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    xe[t][e] = mfma16x16x32bf16(kf, sc.t[e], xe[t][e]);
                    oe[t][e] = mfma16x16x32bf16(qf, sc.t[e], oe[t][e]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            x[t] = xe[t][0] + (xe[t][1] + xe[t][2]);
            o[t] = oe[t][0] + (oe[t][1] + oe[t][2]);
        }
    };
    u32x2 v[2];
    auto take = [&](int strip) {
#pragma unroll
        for (int t = 0; t < NT; ++t) S[t] = Sn[t];
#pragma unroll
        for (int t = 0; t < 2; ++t) v[t] = vn[t];
        if (strip + 4 < strips) ask(strip + 4);
        read_out();
    };
    if (w < strips) take(w);
    lds_barrier();
    if (w >= strips) return;
    Terms3 tf[2];
    Terms3 pf[2];
    f32x4 gi[2], gd[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int i = tile_row(t, r), j0 = 8 * q;
        const bool lower = j0 >> 4 <= i >> 4;                     // (nothing is kept of the tile above the diagonal)
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        const f32x4 b0 = ld4(bt + j0), b1 = ld4(bt + j0 + 4);
        tf[t] = cut3(lower ? ld4(tm + i * LD + j0) * b0 : zero, lower ? ld4(tm + i * LD + j0 + 4) * b1 : zero);
        pf[t] = cut3(lower ? ld4(pm + i * LD + j0) : zero, lower ? ld4(pm + i * LD + j0 + 4) : zero);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = tile_row(t, 4 * q + e);
            gi[t][e] = power(gw[row], gp[row]);
            gd[t][e] = since(N - 1, row);
        }
    }
    const float whole = power(gw[N - 1], gp[N - 1]);
    uint32_t again = 0;
    for (int strip = w; strip < strips; strip += 4) {
        if (strip != w) take(strip);
#pragma unroll
        for (int t = 0; t < 2; ++t) *reinterpret_cast<u32x2*>(&turn[w][t][lane * 4]) = v[t];
        wave_lds_sync();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const u32x2 y = read_across(reinterpret_cast<const uint8_t*>(&turn[w][t][(4 * q + (r >> 2)) * 16 + (r & 3) * 4]));
            const float vf[4] = {__builtin_bit_cast(float, y.x << 16), __builtin_bit_cast(float, y.x & 0xffff0000u),
                                 __builtin_bit_cast(float, y.y << 16), __builtin_bit_cast(float, y.y & 0xffff0000u)};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[t][e] = __builtin_fmaf(-gi[t][e], x[t][e], vf[e]);
                o[t][e] *= a.scale * gi[t][e];
            }
        }
        // U = T X, O += P U, S' = g S + K^T (U g / g_j)
        const Terms3 xc = cut3(x[0], x[1]);
        f32x4 u[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) u[t] = product24(tf[t], xc);
        const Terms3 uc = cut3(u[0], u[1]), dc = cut3(u[0] * gd[0], u[1] * gd[1]);
#pragma unroll
        for (int t = 0; t < 2; ++t) o[t] += product24(pf[t], uc);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int row = 8 * q + (r >> 2), ch = 4 * (t >> 1) + (r & 3), c8 = (t & 1) * 8;
            const bf16x8 kt = join(read_across(kbuf + row * RB + ((ch ^ (spread(row) & (CPR - 1))) * 16) + c8),
                                   read_across(kbuf + (row + 4) * RB + ((ch ^ (spread(row + 4) & (CPR - 1))) * 16) + c8));
            S[t] *= whole;
#pragma unroll
            for (int e = 0; e < 3; ++e) S[t] = mfma16x16x32bf16(kt, dc.t[e], S[t]);
        }
        int bad = 0;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) bad |= not_finite(S[t][e]);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) bad |= not_finite(o[t][e]);
        if (__ballot(bad)) {
            again |= 1u << strip;
            continue;
        }
        keep(strip);
        // O through LDS, so that a lane stores eight bytes of a token
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) turn[w][t][(4 * q + e) * 16 + r] = f32_to_bf16_bits(o[t][e]);
        wave_lds_sync();
        uint16_t* op = static_cast<uint16_t*>(a.o) + ((size_t)s.first * a.H + h) * a.C + strip * 16 + (lane & 3) * 4;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int row = tile_row(t, lane >> 2);
            const u32x2 y = *reinterpret_cast<const u32x2*>(&turn[w][t][lane * 4]);
            if (row < n) *reinterpret_cast<u32x2*>(op + (size_t)row * a.H * a.C) = y;
        }
        wave_lds_sync();
    }
    for (; again; again &= again - 1) strip_by_tokens<R>(s, b, h, __builtin_ctz(again) * 16);
}

hipError_t launch_gdn_prefill_short(const PrefillArgs& a, hipStream_t s)
{
    const uint32_t heads = (uint32_t)a.B * a.H;
    if (a.R == 64) gdn_short_kernel<64><<<heads, 256, 0, s>>>(a);
    else if (a.R == 128) gdn_short_kernel<128><<<heads, 256, 0, s>>>(a);
    else gdn_short_kernel<256><<<heads, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace rs
