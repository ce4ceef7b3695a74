// Attention of one new token per sequence over a paged key-value cache.
//
// For query head h of sequence b over its n cached tokens:
//   s_t = scale q.k_t,  p_t = exp(s_t - lse),  lse = log sum_t exp(s_t),
//   out = sum_t p_t v_t.
// Each token's keys and values are read once for the `group` query heads that
// share them: 4 D bytes per token and kv head for 4 D group flops, so HBM
// bounds it, and only the tensor pipe keeps the products out of the way (fp32
// FMAs would already bound it at a group of 8).
//
// Work split.  A row is a (sequence, kv head, block of up to 16 query heads);
// its tokens are cut into tiles of 64.  The tiles of all rows, in order, form
// one list that the CTAs of a resident grid share out in equal contiguous
// parts, so mixed lengths balance without the host knowing them.  A row that
// crosses CTAs leaves partial results (running maximum, sum, unnormalised
// output) that attend_join_kernel adds up in CTA order.
//
// Each warp is a pipeline of its own: it owns 16 tokens of every tile, keeps
// them arriving through cp.async several tiles ahead (across row ends), and
// holds its own running maximum, sum and output; warps meet only at row ends.
#include "serving.cuh"

namespace mw4 {

constexpr int kAttWarps = 4;
constexpr int kAttThreads = kAttWarps * 32;
constexpr int kSub = 16;                        // tokens of a warp's part of a tile
constexpr int kTile = kSub * kAttWarps;
constexpr int kHeads = 16;                      // query heads of a row, at most
constexpr int kMaxCtas = 152 * 3;               // partial records the workspace has room for
constexpr float kLazyRescale = 8.f;             // log2 growth of the maximum before a rescale

// Pipeline depth and CTAs per SM for a head size: about 100 to 200 KB of shared
// memory of every SM holds tiles in flight.
template <int D> struct AttCfg;
template <> struct AttCfg<64> { static constexpr int stages = 4, ctas = 3; };
template <> struct AttCfg<128> { static constexpr int stages = 3, ctas = 2; };
template <> struct AttCfg<256> { static constexpr int stages = 3, ctas = 1; };

struct AttendArgs {
    KvView c;
    const uint16_t* q;
    uint16_t* out;
    float* lse;         // or NULL
    int64_t q_stride, out_stride;
    int n_q_heads, group, head_blocks, max_len;
    float scale_log2;   // scale * log2(e)
    float* part_o;      // [2 * CTAs][kHeads][D] unnormalised outputs
    float* part_ml;     // [2 * CTAs][kHeads][2] running maximum (log2) and sum
    float* scores;      // [n_seqs][n_q_heads][score_stride] log2 scores, or NULL
    float* lse2;        // [n_seqs][n_q_heads] log2 of the sums, with scores
    int64_t score_stride;
    const float* weight;
    float* weight_out;
    int64_t track_seq, track_head;
    unsigned int* status;
};

template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
    MW4_DEV static uint32_t pack(float a, float b) {
        __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&v);
    }
    MW4_DEV static float2 unpack(uint32_t u) { return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&u)); }
    MW4_DEV static void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
template <> struct Elem<__half> {
    MW4_DEV static uint32_t pack(float a, float b) {
        __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&v);
    }
    MW4_DEV static float2 unpack(uint32_t u) { return __half22float2(*reinterpret_cast<__half2*>(&u)); }
    MW4_DEV static void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

MW4_DEV void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
MW4_DEV void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// 16 bytes, or zeros where !there (the source is not read then).
MW4_DEV void cp_async_16_or_zero(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// The list of tiles and its shares.  total >= 1; part c of `parts` starts at
// tile floor(c total / parts); parts <= total, so no part is empty.
struct Shares {
    int64_t total;
    int parts;
    MW4_DEV int64_t start(int c) const { return c * total / parts; }
    MW4_DEV int owner(int64_t tile) const { return (int)(((tile + 1) * parts - 1) / total); }
};

MW4_DEV int tiles_of(int len) { return max(1, (len + kTile - 1) / kTile); }

MW4_DEV int checked_len(const AttendArgs& a, int b) {
    const int n = a.c.lens[b];
    return n < 0 ? 0 : min(n, a.max_len);
}

// Sum of tiles_of over the sequences [0, end); every thread of a warp gets it.
MW4_DEV int64_t warp_tiles(const AttendArgs& a, int end) {
    int64_t n = 0;
    for (int b = threadIdx.x & 31; b < end; b += 32) n += tiles_of(checked_len(a, b));
#pragma unroll
    for (int off = 16; off; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
    return n;
}

// The sequence that holds tile x of the list and the first tile of that
// sequence, found by a whole warp.
MW4_DEV void find_seq(const AttendArgs& a, int rows, int64_t x, int& b, int64_t& first) {
    const int lane = threadIdx.x & 31;
    int64_t base = 0;
    for (int b0 = 0;; b0 += 32) {
        const int mine = b0 + lane < a.c.n_seqs ? tiles_of(checked_len(a, b0 + lane)) : 0;
        int64_t incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, (base + incl) * rows > x);
        if (past || b0 + 32 >= a.c.n_seqs) {
            const int at = past ? __ffs(past) - 1 : 31;
            b = b0 + at;
            first = (base + __shfl_sync(0xffffffffu, incl - mine, at)) * rows;
            return;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
}

// A place in the list of tiles.
struct Place {
    int b, row, tile, tiles, len;
};
MW4_DEV void next_place(const AttendArgs& a, int rows, Place& p) {
    if (++p.tile < p.tiles) return;
    p.tile = 0;
    if (++p.row < rows) return;
    p.row = 0;
    if (++p.b >= a.c.n_seqs) return;   // past the end: not used
    p.len = checked_len(a, p.b);
    p.tiles = tiles_of(p.len);
}

// GT: query heads of a row, 8 or 16.  The A operand of an MMA has 16 rows.
// With 8 heads the probabilities' upper 8 rows hold what rounding to 16 bits
// took from the lower 8, so they enter the product with about 16 (bf16) or 22
// (fp16) bits at no extra cost; with 16 heads that takes a second product.
template <typename T, int D, int GT>
__global__ void __launch_bounds__(kAttThreads, AttCfg<D>::ctas) attend_kernel(const AttendArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ float sh_m[kAttWarps][kHeads], sh_l[kAttWarps][kHeads];
    constexpr int S = AttCfg<D>::stages;
    constexpr int ROW = D * 2;                       // bytes of a token's keys
    constexpr int HALF = kSub * ROW, STAGE = 2 * HALF;
    constexpr int CH = D / 8;                        // 16-byte pieces of a row
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    uint8_t* ring = smem + warp * S * STAGE;
    const uint32_t ring_u = smem_u32(ring);
    griddep_wait();

    const int rows = a.c.n_kv_heads * a.head_blocks;
    Shares sh;
    sh.total = warp_tiles(a, a.c.n_seqs) * rows;
    sh.parts = (int)min((int64_t)gridDim.x, sh.total);
    const int cta = blockIdx.x;
    if (cta >= sh.parts) return;
    const int64_t x0 = sh.start(cta);
    const int items = (int)(sh.start(cta + 1) - x0);
    Place ld;
    int64_t seq_first;
    find_seq(a, rows, x0, ld.b, seq_first);
    ld.len = checked_len(a, ld.b);
    ld.tiles = tiles_of(ld.len);
    ld.row = (int)((x0 - seq_first) / ld.tiles);
    ld.tile = (int)((x0 - seq_first) % ld.tiles);
    Place at = ld;
    if (cta == 0)
        for (int b = threadIdx.x; b < a.c.n_seqs; b += kAttThreads)
            if (a.c.lens[b] < 0 || a.c.lens[b] > a.max_len) raise_status(a.status, MOE_W4_STATUS_BAD_INDEX);

    // the row of the cache that lane & 15 looks up for the next tile to load
    int64_t off = -1;
    auto look_up = [&]() {
        const int t = ld.tile * kTile + warp * kSub + (lane & 15);
        off = -1;
        if (t < ld.len) {
            off = kv_offset(a.c, ld.b, t);
            if (off < 0) raise_status(a.status, MOE_W4_STATUS_BAD_INDEX);
            else off += (ld.row / a.head_blocks) * a.c.head_stride;
        }
    };
    auto load = [&](int stage) {
        const uint32_t base = ring_u + stage * STAGE;
        if (ld.tile * kTile + warp * kSub < ld.len) {
            constexpr int PER = 32 / CH > 0 ? 32 / CH : 1;   // rows of one warp-wide copy
            constexpr int STEPS = kSub / PER;
            const int piece = lane % CH;
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int r = i * PER + lane / CH;
                const int64_t o = __shfl_sync(0xffffffffu, off, r);
                const uint32_t dst = base + r * ROW + ((piece ^ (r & 7)) << 4);
                const int64_t e = (o < 0 ? 0 : o) + piece * 8;
                cp_async_16_or_zero(dst, a.c.k + e, o >= 0);
                cp_async_16_or_zero(dst + HALF, a.c.v + e, o >= 0);
            }
        }
        cp_async_commit();
    };

    int loaded = 0;
    look_up();
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
        if (loaded < items) {
            load(i);
            next_place(a, rows, ld);
            ++loaded;
            if (loaded < items) look_up();
        } else {
            cp_async_commit();
        }
    }

    uint32_t qf[D / 16][4];
    float o[D / 8][4], m[2], l[2];
    auto start_row = [&]() {
        const int kvh = at.row / a.head_blocks, hb = at.row % a.head_blocks;
        const int heads = min(kHeads, a.group - hb * kHeads);
        const uint16_t* q = a.q + at.b * a.q_stride + (int64_t)(kvh * a.group + hb * kHeads) * D;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int col = kk * 16 + 2 * t4;
            qf[kk][0] = g < heads ? *reinterpret_cast<const uint32_t*>(q + g * D + col) : 0u;
            qf[kk][2] = g < heads ? *reinterpret_cast<const uint32_t*>(q + g * D + col + 8) : 0u;
            if (GT == 16) {
                qf[kk][1] = g + 8 < heads ? *reinterpret_cast<const uint32_t*>(q + (g + 8) * D + col) : 0u;
                qf[kk][3] = g + 8 < heads ? *reinterpret_cast<const uint32_t*>(q + (g + 8) * D + col + 8) : 0u;
            } else {
                qf[kk][1] = qf[kk][3] = 0u;
            }
        }
#pragma unroll
        for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    };

    int seg_first = at.tile;   // first tile of the row that this CTA has
    start_row();
    for (int i = 0; i < items; ++i) {
        cp_async_wait<S - 2>();
        __syncwarp();
        if (loaded < items) {
            load((i + S - 1) % S);
            next_place(a, rows, ld);
            ++loaded;
            if (loaded < items) look_up();
        } else {
            cp_async_commit();
        }
        const int kvh = at.row / a.head_blocks, hb = at.row % a.head_blocks;
        const int heads = min(kHeads, a.group - hb * kHeads);
        const int head0 = kvh * a.group + hb * kHeads;
        const int t0 = at.tile * kTile + warp * kSub;
        const uint32_t kb = ring_u + (i % S) * STAGE, vb = kb + HALF;
        if (t0 < at.len) {
            // two accumulators for each half of the tokens: shorter chains
            float s[2][2][4] = {};
            {
                const int token = (lane >> 4) * 8 + (lane & 7), half = (lane >> 3) & 1;
                const uint32_t addr = kb + token * ROW;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t bfr[4];
                    ldsm4(bfr, addr + (((kk * 2 + half) ^ (token & 7)) << 4));
                    Elem<T>::mma(s[kk & 1][0], qf[kk], bfr[0], bfr[1]);
                    Elem<T>::mma(s[kk & 1][1], qf[kk], bfr[2], bfr[3]);
                }
            }
            float x[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = t0 + j * 8 + 2 * t4 + (e & 1);
                    x[j][e] = t < at.len ? (s[0][j][e] + s[1][j][e]) * a.scale_log2 : -INFINITY;
                }
            if (a.scores) {
#pragma unroll
                for (int r = 0; r < GT / 8; ++r)
                    if (g + r * 8 < heads) {
                        float* p = a.scores + ((int64_t)at.b * a.n_q_heads + head0 + g + r * 8) * a.score_stride + t0 + 2 * t4;
                        *reinterpret_cast<float2*>(p) = make_float2(x[0][2 * r], x[0][2 * r + 1]);
                        *reinterpret_cast<float2*>(p + 8) = make_float2(x[1][2 * r], x[1][2 * r + 1]);
                    }
            }
            // The maximum that the exponents are taken against follows the true one
            // only when it is exceeded by more than 2^8: fp32 sums hold the range, and
            // the output is rescaled a few times a row instead of at every tile.
            float top[2];
            bool grow = false;
#pragma unroll
            for (int r = 0; r < GT / 8; ++r) {
                float v = fmaxf(fmaxf(x[0][2 * r], x[0][2 * r + 1]), fmaxf(x[1][2 * r], x[1][2 * r + 1]));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                top[r] = v;
                grow |= v > m[r] + kLazyRescale || (m[r] == -INFINITY && v > -INFINITY);
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int r = 0; r < GT / 8; ++r) {
                    const float to = fmaxf(m[r], top[r]);
                    const float f = m[r] == -INFINITY ? 0.f : ex2(m[r] - to);
                    m[r] = to;
                    l[r] *= f;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][2 * r] *= f;
                        o[n][2 * r + 1] *= f;
                        if (GT == 8) { o[n][2] *= f; o[n][3] *= f; }
                    }
                }
            }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int r = 0; r < GT / 8; ++r) {
                const float ref = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float p0 = ex2(x[j][2 * r] - ref), p1 = ex2(x[j][2 * r + 1] - ref);
                    l[r] += p0 + p1;
                    const uint32_t h = Elem<T>::pack(p0, p1);
                    const float2 back = Elem<T>::unpack(h);
                    hi[j * 2 + r] = h;
                    lo[j * 2 + r] = Elem<T>::pack(p0 - back.x, p1 - back.y);
                }
            }
            if (GT == 8) { hi[1] = lo[0]; hi[3] = lo[2]; }
            {
                const int token = ((lane >> 3) & 1) * 8 + (lane & 7), half = lane >> 4;
                const uint32_t addr = vb + token * ROW;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    uint32_t bfr[4];
                    ldsm4_t(bfr, addr + (((j * 2 + half) ^ (token & 7)) << 4));
                    Elem<T>::mma(o[2 * j], hi, bfr[0], bfr[1]);
                    Elem<T>::mma(o[2 * j + 1], hi, bfr[2], bfr[3]);
                    if (GT == 16) {
                        Elem<T>::mma(o[2 * j], lo, bfr[0], bfr[1]);
                        Elem<T>::mma(o[2 * j + 1], lo, bfr[2], bfr[3]);
                    }
                }
            }
        }

        const bool row_ends = at.tile == at.tiles - 1;
        if (row_ends || i == items - 1) {
            // the warps' results meet: common maximum, then outputs added in warp order
            // through the stage that this tile has just left
#pragma unroll
            for (int r = 0; r < GT / 8; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
                if (t4 == 0) { sh_m[warp][g + 8 * r] = m[r]; sh_l[warp][g + 8 * r] = l[r]; }
            }
            __syncthreads();
            float* mine = reinterpret_cast<float*>(ring + (i % S) * STAGE);
#pragma unroll
            for (int r = 0; r < GT / 8; ++r) {
                float M = sh_m[0][g + 8 * r];
#pragma unroll
                for (int w = 1; w < kAttWarps; ++w) M = fmaxf(M, sh_m[w][g + 8 * r]);
                const float f = m[r] == -INFINITY ? 0.f : ex2(m[r] - M);
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    float v0 = o[n][2 * r], v1 = o[n][2 * r + 1];
                    if (GT == 8) { v0 += o[n][2]; v1 += o[n][3]; }
                    const int col = (n * 8 + 2 * t4) ^ ((g & 3) * 8);
                    *reinterpret_cast<float2*>(mine + (g + 8 * r) * D + col) = make_float2(v0 * f, v1 * f);
                }
            }
            __syncthreads();
            const bool whole = row_ends && seg_first == 0;
            const int slot = cta * 2 + (seg_first == 0 ? 1 : 0);
            for (int e = threadIdx.x; e < heads * (D / 2); e += kAttThreads) {
                const int h = e / (D / 2), col = (e % (D / 2)) * 2;
                float M = sh_m[0][h];
#pragma unroll
                for (int w = 1; w < kAttWarps; ++w) M = fmaxf(M, sh_m[w][h]);
                float L = 0.f, v0 = 0.f, v1 = 0.f;
#pragma unroll
                for (int w = 0; w < kAttWarps; ++w) {
                    const float mw = sh_m[w][h];
                    L += sh_l[w][h] * (mw == -INFINITY ? 0.f : ex2(mw - M));
                    const float2 v = *reinterpret_cast<const float2*>(
                        reinterpret_cast<const float*>(smem + (w * S + i % S) * STAGE) + h * D + (col ^ ((h & 3) * 8)));
                    v0 += v.x;
                    v1 += v.y;
                }
                if (whole) {
                    // no token, or none with a score above -inf: zeros
                    const float inv = M == -INFINITY && L == 0.f ? 0.f : 1.f / L;
                    *reinterpret_cast<uint32_t*>(a.out + at.b * a.out_stride + (int64_t)(head0 + h) * D + col) =
                        Elem<T>::pack(v0 * inv, v1 * inv);
                    if (col == 0) {
                        const float lse2 = M == -INFINITY && L == 0.f ? -INFINITY : M + log2f(L);
                        const int64_t at_h = (int64_t)at.b * a.n_q_heads + head0 + h;
                        if (a.lse) a.lse[at_h] = lse2 * kLn2;
                        if (a.scores) a.lse2[at_h] = lse2;
                    }
                } else {
                    *reinterpret_cast<float2*>(a.part_o + ((int64_t)slot * kHeads + h) * D + col) = make_float2(v0, v1);
                    if (col == 0)
                        *reinterpret_cast<float2*>(a.part_ml + ((int64_t)slot * kHeads + h) * 2) = make_float2(M, L);
                }
            }
            __syncthreads();
        }
        next_place(a, rows, at);
        if (row_ends && i + 1 < items) {
            seg_first = 0;
            start_row();
        }
    }
}

// Adds up the partial results of the rows that cross CTAs.  Block x stands for
// row x where there are fewer rows than parts, else for the border between
// parts x - 1 and x (each split row is done by the first border inside it);
// blocks of y share the row's heads.
constexpr int kJoinThreads = 256;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const AttendArgs a, int attend_ctas, int by_row) {
    constexpr int LANES = D / 4, WAYS = kJoinThreads / LANES;
    __shared__ float sh_f[kMaxCtas + 1];
    __shared__ float sh_red[8];
    __shared__ float4 sh_o[WAYS][LANES];
    griddep_wait();
    const int rows = a.c.n_kv_heads * a.head_blocks;
    Shares sh;
    sh.total = warp_tiles(a, a.c.n_seqs) * rows;
    sh.parts = (int)min((int64_t)attend_ctas, sh.total);
    int b, row, tiles;
    int64_t first;   // first tile of the row
    if (by_row) {
        b = blockIdx.x / rows;
        row = blockIdx.x % rows;
        tiles = tiles_of(checked_len(a, b));
        first = warp_tiles(a, b) * rows + (int64_t)row * tiles;
    } else {
        const int c = blockIdx.x;
        if (c < 1 || c >= sh.parts) return;
        const int64_t x = sh.start(c);
        find_seq(a, rows, x, b, first);
        tiles = tiles_of(checked_len(a, b));
        row = (int)((x - first) / tiles);
        first += (int64_t)row * tiles;
        if (first == x || sh.start(c - 1) > first) return;   // no row cut here, or not its first cut
    }
    const int c0 = sh.owner(first), c1 = sh.owner(first + tiles - 1), parts = c1 - c0 + 1;
    if (parts == 1) return;
    const int kvh = row / a.head_blocks, hb = row % a.head_blocks;
    const int heads = min(kHeads, a.group - hb * kHeads);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int h = blockIdx.y; h < heads; h += gridDim.y) {
        auto slot = [&](int i) { return (int64_t)((c0 + i) * 2 + (i == 0 ? 1 : 0)) * kHeads + h; };
        float M = -INFINITY;
        for (int i = tid; i < parts; i += kJoinThreads) M = fmaxf(M, a.part_ml[slot(i) * 2]);
#pragma unroll
        for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        if (lane == 0) sh_red[warp] = M;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kJoinThreads / 32; ++w) M = fmaxf(M, sh_red[w]);
        __syncthreads();
        float L = 0.f;
        for (int i = tid; i < parts; i += kJoinThreads) {
            const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + slot(i) * 2);
            const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
            sh_f[i] = f;
            L += ml.y * f;
        }
        L = warp_sum(L);
        if (lane == 0) sh_red[warp] = L;
        __syncthreads();
        L = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinThreads / 32; ++w) L += sh_red[w];
        const int col = tid % LANES, way = tid / LANES;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int i = way; i < parts; i += WAYS) {
            const float4 p = *reinterpret_cast<const float4*>(a.part_o + slot(i) * D + col * 4);
            const float f = sh_f[i];
            v.x += p.x * f; v.y += p.y * f; v.z += p.z * f; v.w += p.w * f;
        }
        sh_o[way][col] = v;
        __syncthreads();
        const int head = kvh * a.group + hb * kHeads + h;
        const bool none = M == -INFINITY && L == 0.f;
        if (way == 0) {
#pragma unroll
            for (int w = 1; w < WAYS; ++w) {
                const float4 p = sh_o[w][col];
                v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
            }
            const float inv = none ? 0.f : 1.f / L;
            uint2 u = make_uint2(Elem<T>::pack(v.x * inv, v.y * inv), Elem<T>::pack(v.z * inv, v.w * inv));
            *reinterpret_cast<uint2*>(a.out + b * a.out_stride + (int64_t)head * D + col * 4) = u;
        }
        if (tid == 0) {
            const float lse2 = none ? -INFINITY : M + log2f(L);
            const int64_t at_h = (int64_t)b * a.n_q_heads + head;
            if (a.lse) a.lse[at_h] = lse2 * kLn2;
            if (a.scores) a.lse2[at_h] = lse2;
        }
        __syncthreads();
    }
}

// weight_out[t] = weight[t] + sum over the kv head's query heads of p_t, from
// the scores that the attention left.
constexpr int kWeightThreads = 256;
__global__ void __launch_bounds__(kWeightThreads) attend_weight_kernel(const AttendArgs a) {
    griddep_wait();
    const int b = blockIdx.z, kvh = blockIdx.y;
    const int t = blockIdx.x * kWeightThreads + threadIdx.x;
    if (t >= checked_len(a, b)) return;
    float w = 0.f;
    const int64_t head0 = (int64_t)b * a.n_q_heads + kvh * a.group;
    for (int h = 0; h < a.group; ++h) {
        const float lse2 = a.lse2[head0 + h];
        const float s = a.scores[(head0 + h) * a.score_stride + t];
        w += lse2 == -INFINITY ? 0.f : ex2(s - lse2);
    }
    const int64_t e = b * a.track_seq + kvh * a.track_head + t;
    a.weight_out[e] = a.weight[e] + w;
}

struct AttendWs {
    size_t part_o, part_ml, lse2, scores, total;
    int64_t score_stride;
};
static AttendWs attend_ws(const moe_w4_kv_cache& c, int n_q_heads, int max_len, bool track) {
    AttendWs w{};
    size_t o = MOE_W4_CTRL_BYTES;
    auto take = [&](size_t bytes) { const size_t at = o; o += round_up(bytes, 256); return at; };
    w.part_o = take((size_t)2 * kMaxCtas * kHeads * c.head_dim * 4);
    w.part_ml = take((size_t)2 * kMaxCtas * kHeads * 2 * 4);
    w.score_stride = (int64_t)round_up((size_t)max_len, kSub);
    if (track) {
        w.lse2 = take((size_t)c.n_seqs * n_q_heads * 4);
        w.scores = take((size_t)c.n_seqs * n_q_heads * (size_t)w.score_stride * 4);
    }
    w.total = o;
    return w;
}

template <typename T, int D>
static cudaError_t launch_attend(const AttendArgs& a, cudaStream_t st) {
    int dev = 0;
    const int sms = sm_count(&dev);
    if (sms < 1) return cudaErrorInvalidDevice;
    constexpr int smem = AttCfg<D>::stages * kAttWarps * 2 * kSub * D * 2;
    const int64_t rows = (int64_t)a.c.n_seqs * a.c.n_kv_heads * a.head_blocks;
    // no more CTAs than tiles the longest lengths could make
    const int64_t most = rows * ((a.max_len + kTile - 1) / kTile > 0 ? (a.max_len + kTile - 1) / kTile : 1);
    int64_t ctas = (int64_t)sms * AttCfg<D>::ctas;
    if (ctas > kMaxCtas) ctas = kMaxCtas;
    if (ctas > most) ctas = most;
    static std::atomic<unsigned> ready[2];
    auto kern = a.group <= 8 ? attend_kernel<T, D, 8> : attend_kernel<T, D, 16>;
    cudaError_t e = allow_smem((const void*)kern, smem, ready[a.group <= 8 ? 0 : 1], dev);
    if (e == cudaSuccess) e = launch_pdl(true, kern, dim3((unsigned)ctas), dim3(kAttThreads), smem, st, a);
    // rows can only be cut where there are fewer rows than tiles
    if (e == cudaSuccess && ctas > 1 && most > rows) {
        const int by_row = rows <= ctas;
        const int heads = a.group < kHeads ? a.group : kHeads;
        e = launch_pdl(true, attend_join_kernel<T, D>, dim3((unsigned)(by_row ? rows : ctas), by_row ? heads : 1),
                       dim3(kJoinThreads), 0, st, a, (int)ctas, by_row);
    }
    if (e == cudaSuccess && a.scores && a.max_len > 0)
        e = launch_pdl(true, attend_weight_kernel,
                       dim3((a.max_len + kWeightThreads - 1) / kWeightThreads, a.c.n_kv_heads, a.c.n_seqs),
                       dim3(kWeightThreads), 0, st, a);
    return e;
}

template <typename T>
static cudaError_t launch_attend_dim(int dim, const AttendArgs& a, cudaStream_t st) {
    return dim == 64 ? launch_attend<T, 64>(a, st) : dim == 128 ? launch_attend<T, 128>(a, st) : launch_attend<T, 256>(a, st);
}

static int check_heads(const moe_w4_kv_cache& c, int n_q_heads, int max_len) {
    if (n_q_heads < 1 || n_q_heads % c.n_kv_heads || max_len < 0 ||
        (int64_t)max_len > (int64_t)c.pages_per_seq * c.page_size)
        return MOE_W4_ERR_INVALID;
    return n_q_heads / c.n_kv_heads > 128 ? MOE_W4_ERR_UNSUPPORTED : MOE_W4_OK;
}

}  // namespace mw4

using namespace mw4;

extern "C" {

size_t moe_w4_attend_workspace_size(const moe_w4_kv_cache* c, int n_q_heads, int max_len, int with_track) {
    if (check_cache(c, false) != MOE_W4_OK || check_heads(*c, n_q_heads, max_len) != MOE_W4_OK) return 0;
    return attend_ws(*c, n_q_heads, max_len, with_track != 0).total;
}

int moe_w4_attend_decode(const moe_w4_kv_cache* c, int n_q_heads, const void* q, int64_t q_stride, float scale,
                         int max_len, void* out, int64_t out_stride, float* lse, const moe_w4_kv_track* track,
                         float* weight_out, void* workspace, size_t ws_bytes, cudaStream_t stream) {
    int r = check_cache(c, true);
    if (r || (r = check_heads(*c, n_q_heads, max_len))) return r;
    if (c->n_seqs == 0) return MOE_W4_OK;
    if (!q || !out || !(track == nullptr) != !(weight_out == nullptr)) return MOE_W4_ERR_INVALID;
    const int64_t width = (int64_t)n_q_heads * c->head_dim;
    if ((c->n_seqs > 1 && (q_stride < 0 || out_stride < width))) return MOE_W4_ERR_INVALID;
    if (track && ((r = check_track(track, false)) || max_len > track->slots)) return r ? r : MOE_W4_ERR_INVALID;
    if (misaligned(q, 16) || misaligned(out, 16) || q_stride % 8 || out_stride % 8 || misaligned(lse, 4) ||
        misaligned(weight_out, 4))
        return MOE_W4_ERR_ALIGN;
    const AttendWs w = attend_ws(*c, n_q_heads, max_len, track != nullptr);
    if ((r = check_workspace(workspace, ws_bytes, w.total))) return r;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    AttendArgs a{};
    a.c = kv_view(*c);
    a.q = static_cast<const uint16_t*>(q);
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.n_q_heads = n_q_heads;
    a.group = n_q_heads / c->n_kv_heads;
    a.head_blocks = (a.group + kHeads - 1) / kHeads;
    a.max_len = max_len;
    a.scale_log2 = scale * kLog2e;
    a.part_o = reinterpret_cast<float*>(ws + w.part_o);
    a.part_ml = reinterpret_cast<float*>(ws + w.part_ml);
    a.status = reinterpret_cast<unsigned int*>(ws);
    if (track) {
        a.lse2 = reinterpret_cast<float*>(ws + w.lse2);
        a.scores = reinterpret_cast<float*>(ws + w.scores);
        a.score_stride = w.score_stride;
        a.weight = track->weight;
        a.weight_out = weight_out;
        a.track_seq = track->seq_stride;
        a.track_head = track->head_stride;
    }
    return launched(c->dtype == MOE_W4_TYPE_BF16 ? launch_attend_dim<__nv_bfloat16>(c->head_dim, a, stream)
                                                 : launch_attend_dim<__half>(c->head_dim, a, stream));
}

}  // extern "C"
