// The steps of an attention kernel of one new token per sequence, of one warp and
// one unit of its ring: SUB tokens' keys or values, in 16-bit values (16 tokens) or
// 8-bit codes (32 tokens, with their scales).
//
// Products are taken transposed, tokens (keys) or dimensions (values) as the 16 rows
// of an MMA and 8 query heads as its columns: S^T = K q^T, O^T = V^T P^T.
//
// Codes become fp16, exactly, between shared memory and the product (one conversion
// for two), and the scales enter the scores and the probabilities in fp32, one
// multiplication a token, not the codes.  Queries are brought to fp16 by a power of
// two per head, so that bf16 ones lose nothing.  (mma.sync takes E4M3 as well, and
// queries can be sums of such terms, but it costs as much as the conversions and two
// fp16 products: 1 x 131,072 tokens 36.8 us so, where it was 29.9.)
#pragma once
#include "attend.cuh"
#include "kv8.cuh"

namespace mw4 {

// Over codes it is probabilities times the values' scales that enter a product, as sums of
// two fp16 terms; and a token that takes nearly all the weight may have no value, or one of a
// scale far from the others'.  So these have a reference of their own, the largest so far, which is
// taken to 2^kTop and follows when one passes 2^(kTop + kRoom); it lies a whole power of two, of
// -kReach to kReach, from the probabilities' own, which may be passed by 2^kGrow.  The second terms
// are taken 2^kLower larger and added up apart: their smallest step is then 2^-36, so that one is off
// by at most 2^-49 of the largest (2^-37 of 2^12, as scales are rounded up to powers of two).
// Multiplying the codes by 2^-kLower instead, which fp16 holds as well, costs more (16 mixed
// sequences of up to 32,768: 41.1 us, so 39.2, 38.6 without any of it).
constexpr int kTop = 13, kRoom = 2, kLower = 12, kReach = 120, kGrow = 4;
// Past this, fp32 scores are too coarse to tell by their sum with a scale's power whether a product has
// outgrown its reference; differences are taken each time.
constexpr float kCoarse = 262144.f;
// log2 of a number that is not negative, rounded up (of 0 and what lies below 2^-126: -127, -126).
MW4_DEV float exponent_up(float f) { return __uint_as_float(0x4b000000u | (__float_as_uint(f) + 0x7fffffu) >> 23) - (8388608.f + 127.f); }

// 16 bytes of which `size`, 0 or 16, come from src and the others are zeros.
MW4_DEV void cp_async_16_sized(uint32_t dst, const void* src, uint32_t size, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" :: "r"(dst), "l"(src), "r"(size), "l"(policy) : "memory");
}
MW4_DEV void cp_async_4_or_zero(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}

// The larger of a magnitude's bits and those of two 16-bit floats.
MW4_DEV uint32_t largest(uint32_t top, uint32_t u) { return max(top, max(u & 0x7fffu, (u >> 16) & 0x7fffu)); }

// What brings a head's queries to fp16, given the bits of the largest: bf16 by the
// power of two that takes it to 2^14 .. 2^15, `back` its inverse; fp16 as they are.
template <typename T> struct QueryScale;
template <> struct QueryScale<__nv_bfloat16> {
    float by, back;
    MW4_DEV explicit QueryScale(uint32_t top) {
        const uint32_t e = max(15u, top >> 7);   // below 2^-112 by 2^126
        by = __uint_as_float((268u - e) << 23);
        back = __uint_as_float((e - 14u) << 23);
    }
    MW4_DEV uint32_t to_f16(uint32_t u) const {
        const float2 f = Elem<__nv_bfloat16>::unpack(u);
        return Elem<__half>::pack(f.x * by, f.y * by);
    }
};
template <> struct QueryScale<__half> {
    static constexpr float back = 1.f;
    MW4_DEV explicit QueryScale(uint32_t) {}
    MW4_DEV uint32_t to_f16(uint32_t u) const { return u; }
};

// T: type of queries and outputs; E8: 8-bit codes; NB: blocks of 8 query heads.
template <typename T, bool E8, int D, int NB>
struct Steps {
    static constexpr bool E = E8;
    using P = typename std::conditional<E8, __half, T>::type;   // of the products
    static constexpr int SUB = E8 ? 32 : 16, R = SUB / 16;      // tokens of a unit, and 16 at a time
    static constexpr int ROW = E8 ? D : 2 * D, CH = ROW / 16;   // bytes of a token's keys, 16-byte pieces
    static constexpr int SCALES = SUB * ROW + 128;              // where the tokens' scales lie in a unit of keys,
                                                                // behind room for the pitch of a warp's outputs
    static constexpr int UNIT = SCALES + (E8 ? SUB * 8 : 0);
    static constexpr int HEADS = 8 * NB, QROW = D * 2, QCH = D / 8, QBYTES = HEADS * QROW;   // queries in shared memory
    static constexpr int PER = 32 / CH, COPIES = SUB / PER;     // rows of a warp-wide copy
    static constexpr int TURN = 8 / PER;                        // copies until the swizzle repeats

    // Where piece p of row r lies in its row: 8 consecutive rows' pieces share no bank.
    static MW4_DEV uint32_t swizzled(int p, int r) { return (p ^ (CH == 4 ? (r >> 1) & 3 : r & 7)) << 4; }

    // A lane's places in 16 tokens of a unit, pieces 2 i and 2 i + 1 (keys' rows are read as
    // they are, values' transposed), and in the queries.
    uint32_t at[CH >= 8 ? 4 : 2], q_at[NB == 1 ? 2 : 4];
    int g, t4;
    MW4_DEV Steps(int lane) : g(lane >> 2), t4(lane & 3) {
        const int t = lane & 15;
#pragma unroll
        for (int i = 0; i < (CH >= 8 ? 4 : 2); ++i) at[i] = t * ROW + swizzled(i * 2 + (lane >> 4), t);
        // one block of heads: two times 16 dimensions in one load; else two blocks
#pragma unroll
        for (int i = 0; i < (NB == 1 ? 2 : 4); ++i) {
            const int h = NB == 1 ? lane & 7 : (lane & 7) + ((lane >> 4) << 3);
            const int p = NB == 1 ? i * 4 + (lane >> 3) : i * 2 + ((lane >> 3) & 1);
            q_at[i] = h * QROW + ((p ^ (h & 7)) << 4);
        }
    }

    // ---- the queries: a piece of 8 dimensions a thread, in shared memory as products take them ----
    static constexpr int QN = (HEADS * QCH + kAttThreads - 1) / kAttThreads;
    static MW4_DEV void load_q(uint4 (&qp)[QN], const uint16_t* q, int heads) {
#pragma unroll
        for (int i = 0; i < QN; ++i) {
            const int e = threadIdx.x + i * kAttThreads;
            qp[i] = e < heads * QCH ? *reinterpret_cast<const uint4*>(q + e * 8) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
    // Of codes a product takes 16 dimensions as they lie: a lane's four codes are columns
    // 2 t4, 2 t4 + 1, 2 t4 + 8 and 2 t4 + 9.  The queries follow: those columns are
    // dimensions 4 t4 .. 4 t4 + 3 of the 16.  qs: log2 score per product of each head,
    // but for the keys' scale.
    static MW4_DEV void store_q(const uint4 (&qp)[QN], uint8_t* smem, float* qs, float scale_log2) {
#pragma unroll
        for (int i = 0; i < QN; ++i) {
            const int e = threadIdx.x + i * kAttThreads, h = e / QCH, at = e % QCH;   // a head's pieces lie in one warp
            if (!E8) {
                if (e < HEADS * QCH) {
                    *reinterpret_cast<uint4*>(smem + h * QROW + ((at ^ (h & 7)) << 4)) = qp[i];
                    if (at == 0) qs[h] = scale_log2;
                }
                continue;
            }
            uint32_t top = largest(largest(largest(largest(0u, qp[i].x), qp[i].y), qp[i].z), qp[i].w);
#pragma unroll
            for (int x = QCH / 2; x; x >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
            if (e < HEADS * QCH) {
                const QueryScale<T> f(top);
                uint8_t* row = smem + h * QROW + (at & 1) * 8;
                const int pair = at & ~1;
                *reinterpret_cast<uint2*>(row + (((pair) ^ (h & 7)) << 4)) = make_uint2(f.to_f16(qp[i].x), f.to_f16(qp[i].z));
                *reinterpret_cast<uint2*>(row + (((pair + 1) ^ (h & 7)) << 4)) = make_uint2(f.to_f16(qp[i].y), f.to_f16(qp[i].w));
                if (at == 0) qs[h] = scale_log2 * f.back;
            }
        }
    }

    // ---- a warp's results of a row: outputs (over codes against 2^m / inv), references and sums ----
    float o[NB][D / 16][4], m[NB][2], l[NB][2], inv[NB][2];
    // P^T of 16 tokens, 0..7 and 8..15: 16 bits, and what they leave.  One term alone would be off by
    // 2^-8 (bf16) or 2^-11 (fp16) of what the output is made of, and that shows where values cancel,
    // whatever the output's own rounding.
    uint32_t hi[NB][R][2], lo[NB][R][2];
    MW4_DEV void start() {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                m[n][c] = -INFINITY;
                l[n][c] = 0.f;
                inv[n][c] = power2(kReach);
            }
        }
    }

    // The tokens' keys: scores, the running maxima and sums, and the probabilities for the
    // values' product.  gone(t): token t of the unit takes no part.
    template <typename Gone>
    MW4_DEV void keys(uint32_t unit, const float* scales, uint32_t q_u, const float* sh_qs, bool some_gone, Gone gone) {
        float s[NB][R][4], odd[R][4];   // one block of heads: two chains of products each
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                odd[r][e] = 0.f;
#pragma unroll
                for (int n = 0; n < NB; ++n) s[n][r][e] = 0.f;
            }
#pragma unroll
        for (int kp = 0; kp < D / 32; ++kp) {
            uint32_t q8[4], k4[R][2][4];   // 32 dimensions: two products' operands
            if (NB == 1) ldsm4(q8, q_u + q_at[kp & 1] + (kp >> 1) * 128);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (E8) {
                    uint32_t x[4];
                    ldsm4(x, unit + at[kp & (CH >= 8 ? 3 : 1)] + (kp >> 2) * 128 + r * 16 * ROW);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        k4[r][c][0] = f16x2_of_codes((uint16_t)x[2 * c]);
                        k4[r][c][1] = f16x2_of_codes((uint16_t)x[2 * c + 1]);
                        k4[r][c][2] = f16x2_of_codes((uint16_t)(x[2 * c] >> 16));
                        k4[r][c][3] = f16x2_of_codes((uint16_t)(x[2 * c + 1] >> 16));
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 2; ++c) ldsm4(k4[r][c], unit + at[(kp * 2 + c) & 3] + ((kp * 2 + c) >> 2) * 128 + r * 16 * ROW);
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int kk = kp * 2 + c;
                uint32_t q4[4], q2[2];
                if (NB == 1) {
                    q4[0] = q8[2 * c];
                    q4[1] = q8[2 * c + 1];
                } else {
                    ldsm4(q4, q_u + q_at[kk & (NB == 1 ? 1 : 3)] + (kk >> 2) * 128);
                    if (NB == 3) ldsm2(q2, q_u + 16 * QROW + q_at[kk & (NB == 1 ? 1 : 3)] + (kk >> 2) * 128);
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    Elem<P>::mma(NB == 1 && c == 1 ? odd[r] : s[0][r], k4[r][c], q4[0], q4[1]);
                    if (NB > 1) Elem<P>::mma(s[1 % NB][r], k4[r][c], q4[2], q4[3]);
                    if (NB == 3) Elem<P>::mma(s[NB - 1][r], k4[r][c], q2[0], q2[1]);
                }
            }
        }
        // s[n][r][2 x + c] becomes the score of token 16 r + 8 x + g with head 2 t4 + c
        float vs[R][2], qs[NB][2];     // (in registers all the while, heads' factors cost spills)
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const float2 two = *reinterpret_cast<const float2*>(sh_qs + n * 8 + 2 * t4);
            qs[n][0] = two.x;
            qs[n][1] = two.y;
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float ks = E8 ? scales[r * 16 + x * 8 + g] : 1.f;
                if (E8) vs[r][x] = scales[SUB + r * 16 + x * 8 + g];
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        s[n][r][2 * x + c] = (NB == 1 ? s[n][r][2 * x + c] + odd[r][2 * x + c] : s[n][r][2 * x + c]) * (E8 ? qs[n][c] * ks : qs[n][c]);
            }
        if (some_gone) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (gone(r * 16 + x * 8 + g)) {
                        if (E8) vs[r][x] = 0.f;
#pragma unroll
                        for (int n = 0; n < NB; ++n) s[n][r][2 * x] = s[n][r][2 * x + 1] = -INFINITY;
                    }
        }
        if constexpr (E8) weigh_codes(s, vs);
        else weigh(s);
    }

    // The probabilities of 16-bit values from scores.  The reference that exponents are taken
    // against follows the maximum only when that has grown by more than kLazy.
    MW4_DEV void weigh(const float (&s)[NB][R][4]) {
        bool grow = false;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) grow |= s[n][r][e] > m[n][e & 1] + (Elem<P>::kBelow + Elem<P>::kLazy);
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float to = warp_most(fmaxf(m[n][c], most(s[n], c) - Elem<P>::kBelow));
                    const float f = m[n][c] == -INFINITY ? 0.f : ex2(m[n][c] - to);
                    m[n][c] = to;
                    rescale(n, c, f, f);
                }
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const float r0 = m[n][0] == -INFINITY ? 0.f : m[n][0], r1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float p0 = ex2(s[n][r][2 * x] - r0), p1 = ex2(s[n][r][2 * x + 1] - r1);
                    l[n][0] += p0;
                    l[n][1] += p1;
                    const uint32_t h = Elem<P>::pack(p0, p1);
                    hi[n][r][x] = transpose8(h);
                    const float2 back = Elem<P>::unpack(h);
                    lo[n][r][x] = transpose8(Elem<P>::pack(p0 - back.x, p1 - back.y));
                }
        }
    }

    // Those over codes, from scores and the values' scales: against 2^m, and times a scale against
    // 2^m / inv.
    MW4_DEV void weigh_codes(const float (&s)[NB][R][4], const float (&vs)[R][2]) {
        float lv[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int x = 0; x < 2; ++x) lv[r][x] = exponent_up(vs[r][x]);
        bool grow = false;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float top_p = m[n][c] + kGrow, top_w = m[n][c] - exponent_up(inv[n][c]) + (kTop + kRoom);
                grow |= fabsf(m[n][c]) > kCoarse;
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        grow |= s[n][r][2 * x + c] > top_p;
                        grow |= s[n][r][2 * x + c] + lv[r][x] > top_w;
                    }
            }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    // by whole powers of two, so that the products' reference can stay where it is
                    const bool none = m[n][c] == -INFINITY;
                    const float high = warp_most(most(s[n], c)), to = none ? high : m[n][c] + fmaxf(0.f, ceilf(high - m[n][c]));
                    float top = -INFINITY;
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int x = 0; x < 2; ++x) top = fmaxf(top, s[n][r][2 * x + c] - to + lv[r][x]);
                    // (fminf and fmaxf let go of a NaN, as of infinite scores)
                    const float by = none ? -INFINITY : m[n][c] - to, before = -exponent_up(inv[n][c]);
                    const float least = fmaxf(ceilf(warp_most(top)) - kTop, (float)-kReach);
                    const float now = fminf(fmaxf(rintf(before + by), least), (float)kReach);
                    m[n][c] = to;
                    inv[n][c] = power2(-(int)now);
                    rescale(n, c, ex2(by), ex2(by + (before - now)));
                }
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const float r0 = fmaxf(m[n][0], -FLT_MAX), r1 = fmaxf(m[n][1], -FLT_MAX);   // (of -inf: every score is)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float p0 = ex2(s[n][r][2 * x] - r0), p1 = ex2(s[n][r][2 * x + 1] - r1);
                    l[n][0] += p0;
                    l[n][1] += p1;
                    // (the scale last: one that is large meets a small inv or a probability of 0)
                    const float w0 = p0 * inv[n][0] * vs[r][x], w1 = p1 * inv[n][1] * vs[r][x];
                    const uint32_t h = Elem<P>::pack(w0, w1);
                    hi[n][r][x] = transpose8(h);
                    const float2 back = Elem<P>::unpack(h);
                    lo[n][r][x] = transpose8(Elem<P>::pack((w0 - back.x) * (1 << kLower), (w1 - back.y) * (1 << kLower)));
                }
        }
    }
    // This lane's largest score with head c of a block's two; the largest of lanes with the same heads.
    static MW4_DEV float most(const float (&s)[R][4], int c) {
        const float v = fmaxf(s[0][c], s[0][c + 2]);
        return R > 1 ? fmaxf(v, fmaxf(s[R - 1][c], s[R - 1][c + 2])) : v;
    }
    static MW4_DEV float warp_most(float v) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, x));
        return v;
    }
    MW4_DEV void rescale(int n, int c, float sums, float outputs) {
        l[n][c] *= sums;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            o[n][j][c] *= outputs;
            o[n][j][c + 2] *= outputs;
        }
    }

    // The tokens' values.  A transposed piece of codes gives a lane dimensions 2 g and 2 g + 1 of
    // two tokens; exchanged to pairs of tokens they are rows g and g + 8, so row g of a product is
    // dimension 2 g of its 16 and row g + 8 dimension 2 g + 1.  Of 16-bit values they are g and g + 8.
    MW4_DEV void values(uint32_t unit) {
        if constexpr (E8) {
#pragma unroll
            for (int jp = 0; jp < D / 32; ++jp) {
                uint32_t v[R][4];
#pragma unroll
                for (int r = 0; r < R; ++r) ldsm4_t(v[r], unit + at[jp & (CH >= 8 ? 3 : 1)] + (jp >> 2) * 128 + r * 16 * ROW);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float low[NB][4];      // of the second terms
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const uint32_t x = __byte_perm(v[r][2 * c], 0, 0x3120), y = __byte_perm(v[r][2 * c + 1], 0, 0x3120);
                        const uint32_t f[4] = {f16x2_of_codes((uint16_t)x), f16x2_of_codes((uint16_t)(x >> 16)),
                                               f16x2_of_codes((uint16_t)y), f16x2_of_codes((uint16_t)(y >> 16))};
#pragma unroll
                        for (int n = 0; n < NB; ++n) {
                            if (r == 0) low[n][0] = low[n][1] = low[n][2] = low[n][3] = 0.f;
                            Elem<P>::mma(o[n][jp * 2 + c], f, hi[n][r][0], hi[n][r][1]);
                            Elem<P>::mma(low[n], f, lo[n][r][0], lo[n][r][1]);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[n][jp * 2 + c][e] = fmaf(low[n][e], 1.f / (1 << kLower), o[n][jp * 2 + c][e]);
                }
            }
        } else {
#pragma unroll
            for (int jp = 0; jp < D / 32; ++jp)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t v[4];
                    ldsm4_t(v, unit + at[(jp * 2 + c) & 3] + ((jp * 2 + c) >> 2) * 128);
                    const uint32_t f[4] = {v[0], v[2], v[1], v[3]};
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        Elem<P>::mma(o[n][jp * 2 + c], f, hi[n][0][0], hi[n][0][1]);
                        Elem<P>::mma(o[n][jp * 2 + c], f, lo[n][0][0], lo[n][0][1]);
                    }
                }
        }
    }

    // The outputs of block n of heads into [8][D + 4] floats, whose pitch meets no bank
    // twice, brought to m and then by factors of heads 2 t4 and 2 t4 + 1.
    MW4_DEV void put(float* buf, int n, float by0, float by1) const {
        buf += 2 * t4 * (D + 4) + (E8 ? 2 * g : g);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                const float by = c ? by1 : by0;
                if (E8) {   // (one after the other: their product may be too small for what o * both is not)
                    const float back = __uint_as_float((254u << 23) - __float_as_uint(inv[n][c]));
                    *reinterpret_cast<float2*>(buf + c * (D + 4) + j * 16) = make_float2(o[n][j][c] * by * back, o[n][j][c + 2] * by * back);
                } else {
                    buf[c * (D + 4) + j * 16] = o[n][j][c] * by;
                    buf[c * (D + 4) + j * 16 + 8] = o[n][j][c + 2] * by;
                }
            }
    }
};

// How a warp asks for the tokens of its units: which page each lies on, and the
// copies of their rows into the ring.
template <typename St, typename Cut>
struct Loader {
    static constexpr int SUB = St::SUB, ROW = St::ROW, CH = St::CH, PER = St::PER;
    const AttendArgs& a;
    const Scales& sc;
    const Cut& cut;
    int lane, piece, row0;
    uint32_t swizzle[St::TURN];    // of this lane's piece in the rows that it copies
    uint64_t policy;
    bool any = false, bad_pages = false;   // of the unit: there is a token; and of the warp: it has met a page outside the cache
    uint32_t there = 0;            // the unit's tokens
    uint64_t off = 0;              // of this lane's token's row, or of the 8 tokens' that it is one of, in pieces
    int64_t scale_off = 0;
    bool mine = false;             // this lane's token is there
    MW4_DEV Loader(const AttendArgs& a, const Scales& sc, const Cut& cut, int lane)
        : a(a), sc(sc), cut(cut), lane(lane), piece(lane % CH), row0(lane / CH), policy(read_once()) {
#pragma unroll
        for (int i = 0; i < St::TURN; ++i) swizzle[i] = row0 * ROW + St::swizzled(piece, i * PER + row0);
    }
    // The page of token t of p's row, -1 for none.  Where 8 tokens from a multiple of 8 on
    // share a page and are one run in memory, one that is not seen beside one that is has theirs.
    MW4_DEV int read_page(const Place& p, int t) const {
        int v = -1;
        if (a.runs ? cut.any8(p, t & ~7) : cut.seen(p, t)) {
            const uint32_t e = div_by((uint32_t)t, a.c.page);
            if (e < (uint32_t)a.c.pages_per_seq) v = a.c.table[p.b * a.c.table_stride + e];
        }
        return v;
    }
    // `page` of this lane's `token` has arrived; no token where !more.
    MW4_DEV void look_up(const Place& p, int token, int page, uint64_t head_off, int kvh, bool more) {
        const uint32_t in = (uint32_t)token - div_by((uint32_t)token, a.c.page) * a.c.page.d;
        const bool seen = more && cut.seen(p, token), good = (unsigned)page < (unsigned)a.c.num_pages;
        mine = seen && good;
        there = __ballot_sync(0xffffffffu, mine);
        if (SUB == 16) there &= 0xffffu;
        any = more && cut.any(p, token - (lane & (SUB - 1)));
        if (__any_sync(0xffffffffu, seen && !good)) {
            if (seen && !good) raise_status(&a.ctrl->status, MOE_W4_STATUS_BAD_INDEX);
            bad_pages = true;
        }
        // (of no page: page 0's rows, an address of the cache, though nothing is read there)
        off = head_off + (uint64_t)(uint32_t)(good ? page : 0) * a.page_pieces + (uint64_t)(a.runs ? in - (lane & 7) : in) * a.slot_pieces;
        if (St::E) scale_off = mine ? (int64_t)page * sc.page_stride + kvh * sc.head_stride + (in >> sc.shift) : 0;
    }
    // Copies the unit's rows; those that are not there become zeros, and nothing is read for them.
    MW4_DEV void load(uint32_t to, const uint4* pool, bool keys) const {
        if (!any) return;
        if (a.runs) {
            const uint4* from = pool + (uint64_t)row0 * a.slot_pieces + piece;
            const uint64_t step = (uint64_t)PER * a.slot_pieces;
            if (there == (SUB == 32 ? 0xffffffffu : 0xffffu)) {   // nearly always
#pragma unroll
                for (int x = 0; x < SUB / 8; ++x) {
                    const uint4* src = from + __shfl_sync(0xffffffffu, off, x * 8);
#pragma unroll
                    for (int i = 0; i < 8 / PER; ++i) cp_async_16_to(to + swizzle[i] + (x * 8 + i * PER) * ROW, src + i * step, policy);
                }
                load_scales(to, keys);
                return;
            }
            const uint32_t rows = there >> row0;
#pragma unroll
            for (int x = 0; x < SUB / 8; ++x) {
                const uint4* src = from + __shfl_sync(0xffffffffu, off, x * 8);
#pragma unroll
                for (int i = 0; i < 8 / PER; ++i)
                    cp_async_16_sized(to + swizzle[i] + (x * 8 + i * PER) * ROW, src + i * step, (rows >> (x * 8 + i * PER) & 1) << 4, policy);
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < St::COPIES; ++i) {
                const int r = i * PER + row0;
                const uint64_t o = __shfl_sync(0xffffffffu, off, r);
                cp_async_16_or_zero(to + r * ROW + St::swizzled(piece, r), pool + (there >> r & 1 ? o + piece : 0), there >> r & 1);
            }
        }
        load_scales(to, keys);
    }
    // Of the unit's tokens, with its keys, those of keys and of values.
    MW4_DEV void load_scales(uint32_t to, bool keys) const {
        if (St::E && keys) {
            cp_async_4_or_zero(to + St::SCALES + lane * 4, sc.k + scale_off, mine);
            cp_async_4_or_zero(to + St::SCALES + SUB * 4 + lane * 4, sc.v + scale_off, mine);
        }
    }
    // Whether token t takes no part: not seen, or on a page outside the cache (rare, so looked up again).
    MW4_DEV bool gone(const Place& p, int t) const {
        return !cut.seen(p, t) || (bad_pages && (unsigned)read_page(p, t) >= (unsigned)a.c.num_pages);
    }
};

}  // namespace mw4
