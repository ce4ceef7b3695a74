// Attention of one new token per sequence over a paged key-value cache.
//
// For query head h of sequence b over its n cached tokens:
//   s_t = scale q.k_t,  p_t = exp(s_t - lse),  lse = log sum_t exp(s_t),
//   out = sum_t p_t v_t.
// Each token's keys and values are read once for the `group` query heads that
// share them: 4 D bytes per token and kv head for 4 D group flops, so HBM
// bounds it, and only the tensor pipe keeps the products out of the way (fp32
// FMAs would already bound it at a group of 8).  mma.sync is enough here: a
// tcgen05 tile of 128 rows would be nearly empty at 1 to 24 query heads.
//
// Work split.  A row is a (sequence, kv head, block of up to 24 query heads);
// its tokens are cut into tiles of 64.  The tiles of all rows, in order, form
// one list that the CTAs of a resident grid share out in equal contiguous
// parts, so mixed lengths balance without the host knowing them.  A row that
// crosses CTAs leaves partial results (reference maximum, sum, unnormalised
// output); at the end each of its CTAs waits for all of them (a cooperative
// launch, bounded waits) and adds up its own share of the row's output in CTA
// order, so that the join is spread over the CTAs too.
//
// Each warp is a pipeline of its own: it owns 16 tokens of every tile, keeps
// their keys and values arriving through cp.async in a ring of its own (units
// of 16 rows, across row ends), and holds its own reference maximum, sum and
// output; warps meet only at row ends.
//
// Products are taken transposed, tokens (keys) or dimensions (values) as the 16
// rows of an MMA and 8 query heads as its columns: S^T = K q^T, O^T = V^T P^T.
// With queries as rows instead half of every product was empty at a group of 8,
// and issue, not HBM, was the limit.  Now a warp issues about 600 instructions
// per 16 tokens of 256 dimensions, the tensor pipe is 11% busy, and loads are
// what warps wait for.
//
// Measured (CUDA graph): 1 x 131,072 tokens, 2 kv heads of 256, group 8: 47.7 us for
// 268 MB, 83% of the copy rate; 32 x 8192, 8 heads of 128, group 4: 165 us for
// 1.07 GB, 96%; bf16 and fp16 alike.  Pages that are no multiple of 8 slots are copied
// row by row (16 x 8192, 8 heads of 128: 101 us with a token a page, 88 with 16).  A call's fixed cost is about 10 us: lengths and page
// numbers (3 us), the first units (1.5), a row's end (2), its join (3).
#include <climits>

#include "serving.cuh"

namespace mw4 {

constexpr int kAttWarps = 4;
constexpr int kAttThreads = kAttWarps * 32;
constexpr int kSub = 16;                        // tokens of a warp's part of a tile
constexpr int kTile = kSub * kAttWarps;
constexpr int most_heads(int dim) { return dim == 256 ? 16 : 24; }   // query heads of a row
constexpr int kMaxSms = 160;                    // SMs that the workspace has room for

// Ring units per warp and CTAs per SM for a head size: 130 to 175 KB of every SM
// hold units in flight.  One more unit makes the queue longer, not the copies
// faster (16 mixed sequences, heads of 128, 4 units: 80 us against 73 with 3).
// NB blocks of 8 query heads: fewer CTAs where their outputs take the registers.
template <int D, int NB> struct AttCfg;
template <int NB> struct AttCfg<64, NB> { static constexpr int slots = 5, ctas = 4; };
template <> struct AttCfg<64, 3> { static constexpr int slots = 6, ctas = 3; };
template <> struct AttCfg<128, 1> { static constexpr int slots = 3, ctas = 3; };
template <> struct AttCfg<128, 2> { static constexpr int slots = 3, ctas = 3; };
template <> struct AttCfg<128, 3> { static constexpr int slots = 5, ctas = 2; };
template <int NB> struct AttCfg<256, NB> { static constexpr int slots = 2, ctas = 2; };
constexpr int unit_bytes(int dim) { return kSub * dim * 2 + 128; }   // 128 more for the pitch of a warp's outputs
constexpr int q_bytes(int dim, int blocks) { return blocks > 1 ? blocks * 8 * dim * 2 : 0; }
constexpr int most_ctas(int dim) { return kMaxSms * (dim == 64 ? AttCfg<64, 1>::ctas : dim == 128 ? AttCfg<128, 1>::ctas : AttCfg<256, 1>::ctas); }

// Arrivals at a split row, by the first of its CTAs: how many partial results
// are there, and how many of the row's CTAs are done with them.  The last to
// leave clears both, so a finished call leaves zeros.
struct RowSync {
    unsigned int arrived, left;
};

struct AttendArgs {
    KvView c;
    const uint16_t* q;
    uint16_t* out;
    float* lse;         // or NULL
    int64_t q_stride, out_stride;
    const uint4* k;     // the pools and their strides in pieces of 16 bytes
    const uint4* v;
    uint32_t page_pieces, head_pieces, slot_pieces;
    int n_q_heads, group, head_blocks, block_heads, max_len;   // a kv head's query heads in blocks
    int runs;           // 16 tokens are 1 or 2 runs in memory (pages of a multiple of 16 or 8 slots), or 0: any
    float scale_log2;   // scale * log2(e)
    float* part_o;      // [2 * CTAs][8 NB][D] unnormalised outputs
    float* part_ml;     // [2 * CTAs][8 NB][2] reference (log2) and sum of 2^(score - reference)
    RowSync* sync;      // [CTAs]
    float* scores;      // [n_seqs][n_q_heads][score_stride] log2 scores, or NULL
    float* lse2;        // [n_seqs][n_q_heads] log2 of the sums, with scores
    int64_t score_stride;
    const float* weight;
    float* weight_out;
    int64_t track_seq, track_head;
    Ctrl* ctrl;
};

// Probabilities are taken against a reference that lies kBelow under the running
// maximum (log2), so that the largest is 2^kBelow, and that follows it when it has
// grown by more than kLazy.  bf16 has fp32's range.  fp16 ends at 2^16 and has no
// step below 2^-24: with 13 + 2 the largest product term is 2^15 and the step
// 2^-37 of a warp's largest probability.  (Against the maximum itself it was 2^-24:
// where a first token without a value takes nearly all the weight and the output is
// that of tokens 18 nats below it, it was off by up to 54%; now by its rounding.)
template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
    static constexpr float kBelow = 0.f, kLazy = 8.f;
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
    static constexpr float kBelow = 13.f, kLazy = 2.f;
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
MW4_DEV void ldsm2(uint32_t (&r)[2], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}
// An 8 x 8 block of 16-bit values, two a lane, transposed.
MW4_DEV uint32_t transpose8(uint32_t v) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}
MW4_DEV void cp_async_16_to(uint32_t dst, const void* src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "l"(policy) : "memory");
}
// Keys and values leave L2 before what is used again (1 x 131,072 tokens of 2 heads
// of 256: 45.8 us, with the usual policy 48.8).  Most are read once a call; where head
// blocks or sequences share them it does not hurt either (16 x 16384, 4 heads of 128,
// group 48 in two blocks: 184.9 and 186.9; 16 sequences of 8192 with 7168 in common:
// 57.3 and 57.8).
MW4_DEV uint64_t read_once() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
// 16 bytes, or zeros where !there (the source is not read then).
MW4_DEV void cp_async_16_or_zero(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
MW4_DEV unsigned int ld_acquire(const unsigned int* p) {
    unsigned int v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// The list and its shares: 1 <= total < 2^31 places in `parts` <= total parts of
// q places, the first r of them one longer.
struct Shares {
    uint32_t total, parts, q, r;
    MW4_DEV Shares(uint32_t places, uint32_t most) : total(places), parts(min(most, places)) {
        q = total / parts;
        r = total - q * parts;
    }
    MW4_DEV uint32_t start(uint32_t c) const { return c * q + min(c, r); }
    MW4_DEV int owner(uint32_t place) const {
        const uint32_t longer = r * (q + 1);
        return (int)(place < longer ? place / (q + 1) : r + (place - longer) / q);
    }
};

MW4_DEV int tiles_of(int len) { return max(1, (len + kTile - 1) / kTile); }
// Places of a row in the list: its tiles and kRowCost more, with no tokens, for
// what the end of a row costs, about the time of a tile.  Without them the CTAs
// that got the short sequences of a mixed batch are the last by far (16 sequences
// of 1 to 32,768 tokens: 69.5 us against 64.0; with 2 the same 64.0).
constexpr int kRowCost = 1;
MW4_DEV uint32_t places_of(int len) { return tiles_of(len) + kRowCost; }

MW4_DEV int checked_len(const AttendArgs& a, int b) {
    const int n = a.c.lens[b];
    return n < 0 ? 0 : min(n, a.max_len);
}

// Sum of places_of over the sequences; every thread of a warp gets it.
MW4_DEV uint32_t warp_places(const int* lens, int n_seqs) {
    uint32_t n = 0;
    for (int b = threadIdx.x & 31; b < n_seqs; b += 32) n += places_of(lens[b]);
    return __reduce_add_sync(0xffffffffu, n);
}

// The sequence that holds place x of the list and the first place of that
// sequence, found by a whole warp.
MW4_DEV void find_seq(const int* lens, int n_seqs, uint32_t rows, uint32_t x, int& b, uint32_t& first) {
    const int lane = threadIdx.x & 31;
    uint32_t base = 0;
    for (int b0 = 0;; b0 += 32) {
        const uint32_t mine = b0 + lane < n_seqs ? places_of(lens[b0 + lane]) : 0;
        uint32_t incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, (base + incl) * rows > x);
        if (past) {   // always so for x below the total, at the last sequences if not before
            const int at = __ffs(past) - 1;
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
MW4_DEV void next_row(const int* lens, int n_seqs, int rows, Place& p) {
    p.tile = 0;
    if (++p.row < rows) return;
    p.row = 0;
    if (++p.b >= n_seqs) return;   // past the end: not used
    p.len = lens[p.b];
    p.tiles = tiles_of(p.len);
}

// lse from a head's reference (log2) and sum; none: no token, or none with a score
// above -inf.
MW4_DEV void write_lse(const AttendArgs& a, int b, int head, float M, float L, bool none) {
    const float lse2 = none ? -INFINITY : M + log2f(L);
    const int64_t at = (int64_t)b * a.n_q_heads + head;
    if (a.lse) a.lse[at] = lse2 * kLn2;
    if (a.scores) a.lse2[at] = lse2;
}

// A row that several CTAs have worked on, c0 first; none of them: parts = 0.
struct Shared {
    int c0, parts, b, row;
};

// Adds up this CTA's share of the outputs of the rows that it shares with others:
// one begun before its part of the list and one going on after it, both at once,
// as each step is a trip to L2 (64 sequences of up to 1000 tokens, 12 heads of 64,
// one after the other: 17.9 us).
template <typename T, int D, int HEADS>
MW4_DEV void join_rows(const AttendArgs& a, uint8_t* smem, int cta, const Shared& begun, const Shared& open) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int Q = D / 4;                                  // columns of four outputs of a head
    struct Share {                                            // of a row: its heads, this CTA's columns and their heads
        int heads, head0, lo, cols, h0, pairs;
    };
    auto share = [&](const Shared& r) {
        Share x{};
        if (r.parts == 0) return x;
        const int kvh = r.row / a.head_blocks, hb = r.row % a.head_blocks;
        x.heads = min(a.block_heads, a.group - hb * a.block_heads);
        x.head0 = kvh * a.group + hb * a.block_heads;
        const int total = x.heads * Q, per = (total + r.parts - 1) / r.parts;
        x.lo = (cta - r.c0) * per;
        x.cols = max(0, min(per, total - x.lo));
        x.h0 = x.lo / Q & ~1;
        x.pairs = (x.lo + x.cols - 1) / Q / 2 - x.h0 / 2 + 1;
        return x;
    };
    const Share xb = share(begun), xo = share(open);
    bool ok = true;
    if (lane == 0 && warp < 2) {
        const int c0 = warp ? open.c0 : begun.c0;
        const unsigned parts = warp ? open.parts : begun.parts;
        if (parts) {
            const uint64_t t0 = globaltimer();
            for (int it = 0; ld_acquire(&a.sync[c0].arrived) < parts; ++it)
                if ((it & 15) == 15 && globaltimer() - t0 > kWaitLimitNs) {
                    raise_status(&a.ctrl->status, MOE_W4_STATUS_WAIT_TIMEOUT);
                    ok = false;
                    break;
                }
            // the last to have seen them all clears the row's record
            if (ok && atomic_add_acq_rel_gpu(&a.sync[c0].left, 1) == parts - 1) {
                a.sync[c0].arrived = 0;
                a.sync[c0].left = 0;
            }
        }
    }
    if (!__syncthreads_and(ok)) return;                       // (the ring is free from here on)
    // everything the sums need in one trip, a warp for a part in turn: the heads'
    // maxima and sums (by pairs of heads), and the columns
    float4* room = reinterpret_cast<float4*>(smem);           // [parts][pairs]: m, sum, m, sum; [parts][cols]; the next row's
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const Shared r = which ? open : begun;
        const Share x = which ? xo : xb;
        if (x.cols == 0) continue;
        float4* ml = room;
        float4* part = ml + r.parts * x.pairs;
        room = part + r.parts * x.cols;
        // few columns: several parts to a warp
        const int wide = max(x.cols, x.pairs), lanes = wide > 16 ? 32 : wide > 8 ? 16 : wide > 4 ? 8 : 4;
        const int sub = lane / lanes, in = lane & (lanes - 1), subs = 32 / lanes;
#pragma unroll 1
        for (int i = warp * subs + sub; i < r.parts; i += kAttWarps * subs) {
            const int64_t sl = (int64_t)((r.c0 + i) * 2 + (i == 0 ? 1 : 0)) * HEADS;
            for (int e = in; e < x.pairs; e += lanes) cp_async_16(&ml[i * x.pairs + e], a.part_ml + (sl + x.h0 + e * 2) * 2);
            for (int e = in; e < x.cols; e += lanes) cp_async_16(&part[i * x.cols + e], a.part_o + sl * D + (x.lo + e) * 4);
        }
    }
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();
    room = reinterpret_cast<float4*>(smem);
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const Shared r = which ? open : begun;
        const Share x = which ? xo : xb;
        if (x.cols == 0) continue;
        const float4* ml = room;
        const float4* part = ml + r.parts * x.pairs;
        room += r.parts * (x.pairs + x.cols);
        // a group of lanes for a column, its lanes taking turns at the parts
        const int turns = x.cols > 64 ? 1 : x.cols > 32 ? 2 : x.cols > 16 ? 4 : x.cols > 8 ? 8 : x.cols > 4 ? 16 : 32;
        const int turn = tid & (turns - 1);
#pragma unroll 1
        for (int e = tid / turns; e - tid / turns < x.cols; e += kAttThreads / turns) {   // the same turns for every lane
            const int mine = min(e, x.cols - 1), h = (x.lo + mine) / Q;
            const float2* of = reinterpret_cast<const float2*>(ml) + h - x.h0;   // the head's, 2 pairs apart
            float M = -INFINITY, L = 0.f;
#pragma unroll 4
            for (int i = turn; i < r.parts; i += turns) M = fmaxf(M, of[i * 2 * x.pairs].x);
#pragma unroll 1
            for (int off = turns / 2; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int i = turn; i < r.parts; i += turns) {
                const float2 y = of[i * 2 * x.pairs];
                const float4 p = part[i * x.cols + mine];
                const float f = y.x == -INFINITY ? 0.f : ex2(y.x - M);
                L += y.y * f;
                v.x += p.x * f; v.y += p.y * f; v.z += p.z * f; v.w += p.w * f;
            }
#pragma unroll 1
            for (int off = turns / 2; off; off >>= 1) {
                L += __shfl_xor_sync(0xffffffffu, L, off);
                v.x += __shfl_xor_sync(0xffffffffu, v.x, off);
                v.y += __shfl_xor_sync(0xffffffffu, v.y, off);
                v.z += __shfl_xor_sync(0xffffffffu, v.z, off);
                v.w += __shfl_xor_sync(0xffffffffu, v.w, off);
            }
            if (e < x.cols && turn == 0) {
                const bool none = M == -INFINITY && L == 0.f;
                const float inv = none ? 0.f : 1.f / L;
                const int col = (x.lo + e - h * Q) * 4;
                *reinterpret_cast<uint2*>(a.out + r.b * a.out_stride + (int64_t)(x.head0 + h) * D + col) =
                    make_uint2(Elem<T>::pack(v.x * inv, v.y * inv), Elem<T>::pack(v.z * inv, v.w * inv));
                if (col == 0) write_lse(a, r.b, x.head0 + h, M, L, none);
            }
        }
    }
}

// NB: blocks of 8 query heads of a row, up to 3 (2 at 256 dimensions), so that a
// group of up to 24 reads its keys and values once.  The queries of one block stay
// in registers; those of more, whose outputs take their place, in shared memory
// (4 x 16384 tokens, 2 kv heads of 256, group 16: 43.3 us with them in registers
// that spill, 30.8 so; 16 x 16384, 4 heads of 128, group 24: 164.6 in two blocks of
// the list, 99.5 in one, 537 MB).
template <typename T, int D, int NB>
__global__ void __launch_bounds__(kAttThreads, AttCfg<D, NB>::ctas) attend_kernel(const AttendArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int HEADS = 8 * NB;
    __shared__ float sh_m[kAttWarps][HEADS], sh_l[kAttWarps][HEADS];
    constexpr int S = AttCfg<D, NB>::slots;
    constexpr int ROW = D * 2;                       // bytes of a token's keys
    constexpr int UNIT = unit_bytes(D);              // keys or values of 16 tokens
    constexpr int CH = D / 8;                        // 16-byte pieces of a row
    constexpr int PER = 32 / CH, STEPS = kSub / PER; // rows of a warp-wide copy
    constexpr int HALF = STEPS / 2;                  // copies of 8 rows
    constexpr int TURN = 8 / PER;                    // copies until the swizzle repeats
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    uint8_t* ring = smem + warp * S * UNIT;
    const uint32_t ring_u = smem_u32(ring), ring_end = ring_u + S * UNIT;
    griddep_wait();

    // The lengths, read once: whatever happens to them meanwhile, this CTA's view
    // of the list is one, and its accesses stay in range.
    const int rows = a.c.n_kv_heads * a.head_blocks, n_seqs = a.c.n_seqs;
    uint8_t* q_smem = smem + kAttWarps * S * UNIT;        // [HEADS][D], pieces of a head swizzled like a unit's
    int* lens = reinterpret_cast<int*>(q_smem + q_bytes(D, NB));
    const uint32_t cta = blockIdx.x;
    for (int b = threadIdx.x; b < n_seqs; b += kAttThreads) {
        const int n = a.c.lens[b];
        if (cta == 0 && (n < 0 || n > a.max_len)) raise_status(&a.ctrl->status, MOE_W4_STATUS_BAD_INDEX);
        lens[b] = n < 0 ? 0 : min(n, a.max_len);
    }
    __syncthreads();
    const Shares sh(warp_places(lens, n_seqs) * rows, gridDim.x);
    if (cta >= sh.parts) return;
    uint32_t place = sh.start(cta);                       // of `at` in the list
    const uint32_t end = sh.start(cta + 1);
    Place at;
    uint32_t seq_first;
    find_seq(lens, n_seqs, rows, place, at.b, seq_first);
    at.len = lens[at.b];
    at.tiles = tiles_of(at.len);
    at.row = (int)((place - seq_first) / places_of(at.len));
    at.tile = (int)(place - seq_first - at.row * places_of(at.len));
    if (at.tile >= at.tiles) {                            // past a row's tiles: on to the next
        place += places_of(at.len) - at.tile;
        if (place >= end) return;
        next_row(lens, n_seqs, rows, at);
    }

    // ---- loads: units in order, keys and values of one tile after the other ----
    // Offsets are in pieces of 16 bytes.  The block table is read one tile ahead of
    // the keys: behind a full queue of them that load takes microseconds.
    Place ld = at;                 // the tile loaded next
    bool more = true;              // to load
    int token = at.tile * kTile + warp * kSub + (lane & 15);   // of ld's tile, this lane's to look up
    int page = -1;                 // of token
    uint64_t head_off = 0;         // of ld's row
    uint64_t off = 0;              // of ld's tile: this lane's first piece of the run, its token's run, or its token's row
    bool run = false, any = false, there = false;
    bool bad_pages = false;        // the warp has met a page outside the cache
    auto read_page = [&](const Place& p, int t) {   // the page of token t of p's row
        int v = -1;
        if (t < p.len) {
            const uint32_t e = div_by((uint32_t)t, a.c.page);
            if (e < (uint32_t)a.c.pages_per_seq) v = a.c.table[p.b * a.c.table_stride + e];
        }
        return v;
    };
    const int piece = lane % CH, row0 = lane / CH;
    auto head_of = [&](const Place& p) { return (uint64_t)(p.row / a.head_blocks) * a.head_pieces; };
    auto look_up = [&]() {         // `page` has arrived: where ld's tile is
        const int t0 = token - (lane & 15);
        const uint32_t in = (uint32_t)token - div_by((uint32_t)token, a.c.page) * a.c.page.d;
        any = t0 < ld.len;
        there = (unsigned)page < (unsigned)a.c.num_pages;
        const bool bad = token < ld.len && !there;
        run = a.runs && t0 + kSub <= ld.len;
        if (__any_sync(0xffffffffu, bad)) {
            if (bad) raise_status(&a.ctrl->status, MOE_W4_STATUS_BAD_INDEX);
            run = false;
            bad_pages = true;
        }
        // of one run a lane starts row0 rows and a piece on; of two it knows its token's
        const uint32_t r = run ? a.runs == 1 ? in - (lane & 15) + row0 : in - (lane & 7) : in;
        off = head_off + (uint64_t)(uint32_t)page * a.page_pieces + (uint64_t)r * a.slot_pieces + (run && a.runs == 1 ? piece : 0);
    };
    uint32_t swizzle[TURN];        // of this lane's piece in the rows that it copies
#pragma unroll
    for (int i = 0; i < TURN; ++i) swizzle[i] = row0 * ROW + ((piece ^ ((i * PER + row0) & 7)) << 4);
    const uint64_t policy = read_once();
    const bool packed = a.slot_pieces == CH;   // a run's rows follow one another
    auto load = [&](uint32_t base, const uint4* pool) {
        if (run) {
            uint32_t to[TURN];
#pragma unroll
            for (int i = 0; i < TURN; ++i) to[i] = base + swizzle[i];
            const uint64_t step = (uint64_t)PER * a.slot_pieces;
            if (a.runs == 2) {
                const uint64_t other = __shfl_xor_sync(0xffffffffu, off, 8), more = (uint64_t)row0 * a.slot_pieces + piece;
                const uint4* p = pool + (lane & 8 ? other : off) + more;
                const uint4* p8 = pool + (lane & 8 ? off : other) + more;
#pragma unroll
                for (int i = 0; i < STEPS; ++i)
                    cp_async_16_to(to[i % TURN] + i * PER * ROW, (i < HALF ? p : p8) + i % HALF * step, policy);
            } else if (packed) {
                const uint4* p = pool + off;
#pragma unroll
                for (int i = 0; i < STEPS; ++i) cp_async_16_to(to[i % TURN] + i * PER * ROW, p + i * PER * CH, policy);
            } else {
                const uint4* p = pool + off;
#pragma unroll
                for (int i = 0; i < STEPS; ++i) cp_async_16_to(to[i % TURN] + i * PER * ROW, p + i * step, policy);
            }
        } else if (any) {
#pragma unroll 1
            for (int i = 0; i < STEPS; ++i) {
                const int r = i * PER + row0;
                const uint64_t o = __shfl_sync(0xffffffffu, off, r);
                const bool ok = __shfl_sync(0xffffffffu, there, r);
                cp_async_16_or_zero(base + r * ROW + ((piece ^ (r & 7)) << 4), pool + (ok ? o + piece : 0), ok);
            }
        }
        cp_async_commit();
    };
    int next_page = -1;            // read ahead, of the tile after ld
    Place ahead = at;
    int ahead_token = token;
    uint32_t ahead_place = place;
    bool more_ahead = true;
    auto read_ahead = [&]() {
        ++ahead_place;
        if (++ahead.tile == ahead.tiles) {
            ahead_place += kRowCost;
            next_row(lens, n_seqs, rows, ahead);
            ahead_token = warp * kSub + (lane & 15);
        } else {
            ahead_token += kTile;
        }
        more_ahead = ahead_place < end;
        if (more_ahead) next_page = read_page(ahead, ahead_token);
    };
    uint32_t fill = ring_u;
    bool values = false;           // the next unit is one of values
    auto load_unit = [&]() {
        if (more) {
            load(fill, values ? a.v : a.k);
            if (values && (more = more_ahead)) {
                if (ahead.row != ld.row || ahead.b != ld.b) head_off = head_of(ahead);
                ld = ahead;
                token = ahead_token;
                page = next_page;
                look_up();
                read_ahead();
            }
        } else {
            cp_async_commit();
        }
        values = !values;
        fill = fill + UNIT == ring_end ? ring_u : fill + UNIT;
    };
    page = read_page(ld, token);
    head_off = head_of(ld);
    read_ahead();

    // ---- the queries of a row, and its running results ----
    uint32_t qf[D / 16][2];
    float o[NB][D / 16][4], m[NB][2], l[NB][2];
    constexpr int QN = (HEADS * CH + kAttThreads - 1) / kAttThreads;   // pieces of a thread
    uint4 qp[QN];
    auto load_q = [&](const Place& p) {
        const int kvh = p.row / a.head_blocks, hb = p.row % a.head_blocks;
        const int heads = min(a.block_heads, a.group - hb * a.block_heads);
        const uint16_t* q = a.q + p.b * a.q_stride + (int64_t)(kvh * a.group + hb * a.block_heads) * D;
        if (NB == 1) {
            q += g * D + 2 * t4;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                qf[kk][0] = g < heads ? *reinterpret_cast<const uint32_t*>(q + kk * 16) : 0u;
                qf[kk][1] = g < heads ? *reinterpret_cast<const uint32_t*>(q + kk * 16 + 8) : 0u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < QN; ++i) {
                const int e = threadIdx.x + i * kAttThreads;
                qp[i] = e < heads * CH ? *reinterpret_cast<const uint4*>(q + e * 8) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
    };
    auto store_q = [&]() {
#pragma unroll
        for (int i = 0; i < QN; ++i) {
            const int e = threadIdx.x + i * kAttThreads, h = e / CH;
            if (e < HEADS * CH) *reinterpret_cast<uint4*>(q_smem + h * ROW + (((e % CH) ^ (h & 7)) << 4)) = qp[i];
        }
    };
    load_q(at);
    if (NB > 1) {
        store_q();
        __syncthreads();
    }
    look_up();
    // lanes' places in a unit of keys (rows tokens) and of values (rows tokens, transposed);
    // those of values are also the queries' (rows heads)
    uint32_t k_lane[4], v_lane[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int kt = lane & 15, vt = (lane & 7) + ((lane >> 4) << 3);
        k_lane[i] = kt * ROW + (((i * 2 + (lane >> 4)) ^ (kt & 7)) << 4);
        v_lane[i] = vt * ROW + (((i * 2 + ((lane >> 3) & 1)) ^ (vt & 7)) << 4);
    }

    // Rows shared with other CTAs: one begun before this CTA's part, one going on
    // after it.  Their first place in the list (-1: none) and tiles; sequence and row.
    int begun_first = -1, open_first = -1;
    int begun_tiles = 0, begun_b = 0, begun_row = 0, open_tiles = 0, open_b = 0, open_row = 0;
    const bool silent = cta == 0 && a.ctrl->pad[kCtrlInjectWord];   // the failure-detection test hook
    uint32_t take = ring_u;        // the next unit to use
    const uint32_t q_u = smem_u32(q_smem);

    // One turn a unit, the first S of them only to fill the ring: a single copy of
    // the loading code, as this kernel runs through much of its code just once.
    int first_place = (int)place - at.tile;   // of at's row in the list
    int first = at.tile;           // of the row, in this CTA
    int heads = 0, head0 = 0;
    bool fresh = true;             // a row begins
    uint32_t hi[NB][2], lo[NB][2]; // P^T of tokens 0..7 and 8..15: 16 bits, and what they leave
    auto start_row = [&]() {
        const int kvh = at.row / a.head_blocks, hb = at.row - kvh * a.head_blocks;
        heads = min(a.block_heads, a.group - hb * a.block_heads);
        head0 = kvh * a.group + hb * a.block_heads;
        first = at.tile;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int r = 0; r < 2; ++r) hi[n][r] = lo[n][r] = 0u;
        }
    };
    // The end of a row's tiles here: the warps' results meet, under a common maximum,
    // outputs added in warp order through the unit that has just been used.
    auto finish_row = [&](bool row_ends) {
        Place nx = at;
        next_row(lens, n_seqs, rows, nx);
        if (NB == 1 && place < end) load_q(nx);    // there by the time the next row begins
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], x);
                if (g == 0) {
                    sh_m[warp][n * 8 + 2 * t4 + c] = m[n][c];
                    sh_l[warp][n * 8 + 2 * t4 + c] = l[n][c];
                }
            }
        const bool whole = row_ends && first == 0;
        const int64_t slot = (int64_t)(cta * 2 + (first == 0 ? 1 : 0)) * HEADS;
        const uint32_t here = take - ring_u;
        float* buf = reinterpret_cast<float*>(ring + here) + 2 * t4 * (D + 4) + g;   // [8][D + 4]: no bank twice
#pragma unroll
        for (int n = 0; n < NB; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    buf[c * (D + 4) + j * 16] = o[n][j][c];
                    buf[c * (D + 4) + j * 16 + 8] = o[n][j][c + 2];
                }
            __syncthreads();
            const bool next_q = NB > 1 && n == NB - 1 && place < end;   // nobody uses the present ones any more
            if (next_q) load_q(nx);
            const int quads = min(8, heads - n * 8) * (D / 4);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const int e = threadIdx.x + i * kAttThreads;
                if (e >= quads) break;
                const int h8 = e / (D / 4), col = (e % (D / 4)) * 4, h = n * 8 + h8;
                float M = sh_m[0][h], L = 0.f;
#pragma unroll
                for (int w = 1; w < kAttWarps; ++w) M = fmaxf(M, sh_m[w][h]);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                const float* from = reinterpret_cast<const float*>(smem + here) + h8 * (D + 4) + col;
#pragma unroll
                for (int w = 0; w < kAttWarps; ++w, from += S * UNIT / 4) {
                    // a warp without a score above -inf: 0, or NaN where it has met one
                    const float f = sh_m[w][h] == -INFINITY ? (sh_l[w][h] == 0.f ? 0.f : NAN) : ex2(sh_m[w][h] - M);
                    const float4 p = *reinterpret_cast<const float4*>(from);
                    L += sh_l[w][h] * f;
                    v.x += p.x * f; v.y += p.y * f; v.z += p.z * f; v.w += p.w * f;
                }
                if (whole) {
                    const bool none = M == -INFINITY && L == 0.f;
                    const float inv = none ? 0.f : 1.f / L;
                    *reinterpret_cast<uint2*>(a.out + at.b * a.out_stride + (int64_t)(head0 + h) * D + col) =
                        make_uint2(Elem<T>::pack(v.x * inv, v.y * inv), Elem<T>::pack(v.z * inv, v.w * inv));
                    if (col == 0) write_lse(a, at.b, head0 + h, M, L, none);
                } else {
                    __stcg(reinterpret_cast<float4*>(a.part_o + (slot + h) * D + col), v);
                    if (col == 0) __stcg(reinterpret_cast<float2*>(a.part_ml + (slot + h) * 2), make_float2(M, L));
                }
            }
            if (next_q) store_q();
            __syncthreads();
        }
        if (!whole) {
            const int from = first_place;
            if (first == 0) {
                open_first = from;
                open_tiles = at.tiles; open_b = at.b; open_row = at.row;
            } else {
                begun_first = from;
                begun_tiles = at.tiles; begun_b = at.b; begun_row = at.row;
            }
            if (threadIdx.x == 0 && !silent) atomic_add_release_gpu(&a.sync[sh.owner(from)].arrived, 1);
        }
        at = nx;
        first_place = (int)place;
        fresh = true;
    };
    bool open = true;              // tiles are left
#pragma unroll 1
    for (int u = -S; open; ++u) {
        if (fresh && u >= 0) {
            start_row();
            fresh = false;
        }
        const int t0 = at.tile * kTile + warp * kSub;
        const bool mine = u >= 0 && t0 < at.len;
        cp_async_wait<S - 1>();
        __syncwarp();
        if (mine && !(u & 1)) {
            // S^T = K q^T: 16 tokens by 8 heads a block, two chains of accumulators
            float s[NB][2][4];
            {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][0][e] = s[n][1][e] = 0.f;
                uint32_t from[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) from[j] = take + k_lane[j];
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t k4[4];
                    ldsm4(k4, from[kk & 3] + (kk >> 2) * 128);
                    if (NB == 1) {
                        Elem<T>::mma(s[0][kk & 1], k4, qf[kk][0], qf[kk][1]);
                    } else {
                        uint32_t q4[4];
                        ldsm4(q4, q_u + v_lane[kk & 3] + (kk >> 2) * 128);
                        Elem<T>::mma(s[0][kk & 1], k4, q4[0], q4[1]);
                        Elem<T>::mma(s[1 % NB][kk & 1], k4, q4[2], q4[3]);
                        if (NB == 3) {
                            uint32_t q2[2];
                            ldsm2(q2, q_u + 16 * ROW + v_lane[kk & 3] + (kk >> 2) * 128);
                            Elem<T>::mma(s[NB - 1][kk & 1], k4, q2[0], q2[1]);
                        }
                    }
                }
            }
            {
                bool grow = false;
                // s[n][0][2r + c] becomes the score of token g + 8r with head 2 t4 + c
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][0][e] = (s[n][0][e] + s[n][1][e]) * a.scale_log2;
                if (t0 + kSub > at.len || bad_pages) {   // tokens past the length or without a page (zeros here)
                    bool none[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) none[r] = t0 + g + 8 * r >= at.len;
                    if (bad_pages)   // rare, so looked up again
#pragma unroll 1
                        for (int r = 0; r < 2; ++r) {
                            const bool off_page = (unsigned)read_page(at, t0 + g + 8 * r) >= (unsigned)a.c.num_pages;
                            none[0] |= r == 0 && off_page;
                            none[1] |= r == 1 && off_page;
                        }
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (none[e >> 1]) s[n][0][e] = -INFINITY;
                }
                if (a.scores) {
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int h = n * 8 + 2 * t4 + (e & 1), t = t0 + g + 8 * (e >> 1);
                            if (h < heads && t < at.len)
                                a.scores[((int64_t)at.b * a.n_q_heads + head0 + h) * a.score_stride + t] = s[n][0][e];
                        }
                }
                // The reference that the exponents are taken against follows the maximum
                // only when that has grown by more than kLazy: fp32 sums hold the range, and
                // the maximum is found and the output rescaled a few times a row.
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) grow |= s[n][0][e] > m[n][e & 1] + (Elem<T>::kBelow + Elem<T>::kLazy);
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float to = fmaxf(m[n][c], fmaxf(s[n][0][c], s[n][0][c + 2]) - Elem<T>::kBelow);
#pragma unroll
                            for (int x = 4; x < 32; x <<= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, x));
                            const float f = m[n][c] == -INFINITY ? 0.f : ex2(m[n][c] - to);
                            m[n][c] = to;
                            l[n][c] *= f;
#pragma unroll
                            for (int j = 0; j < D / 16; ++j) {
                                o[n][j][c] *= f;
                                o[n][j][c + 2] *= f;
                            }
                        }
                }
                // Probabilities enter the product as two 16-bit terms, about 16 (bf16) or 22
                // (fp16, or down to its smallest step) bits: one alone would cost as much
                // accuracy as the output's rounding.
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const float r0 = m[n][0] == -INFINITY ? 0.f : m[n][0], r1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float p0 = ex2(s[n][0][2 * r] - r0), p1 = ex2(s[n][0][2 * r + 1] - r1);
                        l[n][0] += p0;
                        l[n][1] += p1;
                        const uint32_t h = Elem<T>::pack(p0, p1);
                        const float2 back = Elem<T>::unpack(h);
                        hi[n][r] = transpose8(h);
                        lo[n][r] = transpose8(Elem<T>::pack(p0 - back.x, p1 - back.y));
                    }
                }
            }
        } else if (mine) {
            // O^T += V^T P^T: 16 dimensions by 8 heads a block
            uint32_t from[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) from[j] = take + v_lane[j];
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                uint32_t v4[4];
                ldsm4_t(v4, from[j & 3] + (j >> 2) * 128);
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    Elem<T>::mma(o[n][j], v4, hi[n][0], hi[n][1]);
                    Elem<T>::mma(o[n][j], v4, lo[n][0], lo[n][1]);
                }
            }
        }
        __syncwarp();
        const bool row_ends = at.tile == at.tiles - 1;
        if (u >= 0 && (u & 1)) {
            place += row_ends ? 1 + kRowCost : 1;
            open = place < end;
            if (row_ends || !open) finish_row(row_ends);
            else ++at.tile;
        }
        load_unit();
        if (u >= 0) take = take + UNIT == ring_end ? ring_u : take + UNIT;
    }
    cp_async_wait<0>();
    griddep_launch_dependents();

    // the rows shared with other CTAs
    Shared begun{0, 0, begun_b, begun_row}, going{(int)cta, 0, open_b, open_row};
    if (begun_first >= 0) {
        begun.c0 = sh.owner(begun_first);
        begun.parts = sh.owner(begun_first + begun_tiles - 1) - begun.c0 + 1;
    }
    if (open_first >= 0) going.parts = sh.owner(open_first + open_tiles - 1) - (int)cta + 1;
    if (begun.parts | going.parts) join_rows<T, D, HEADS>(a, smem, cta, begun, going);
}

// weight_out[t] = weight[t] + sum over the kv head's query heads of p_t, from
// the scores that the attention left.  Four tokens a thread; everything is asked
// for at once, before the length is known (the scores' rows are whole multiples
// of 16 tokens).
constexpr int kWeightThreads = 128, kWeightTokens = 4;
__global__ void __launch_bounds__(kWeightThreads) attend_weight_kernel(const AttendArgs a) {
    griddep_wait();
    const int b = blockIdx.z, kvh = blockIdx.y;
    const int t = (blockIdx.x * kWeightThreads + threadIdx.x) * kWeightTokens;
    if (t >= a.max_len) return;
    const int n = checked_len(a, b);
    const int64_t e = b * a.track_seq + kvh * a.track_head + t, head0 = (int64_t)b * a.n_q_heads + kvh * a.group;
    float before[kWeightTokens], w[kWeightTokens] = {};
#pragma unroll
    for (int k = 0; k < kWeightTokens; ++k) before[k] = t + k < n ? a.weight[e + k] : 0.f;
    const float* scores = a.scores + head0 * a.score_stride + t;
    for (int h0 = 0; h0 < a.group; h0 += 8) {
        float4 s[8];
        float lse2[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            const bool in = h0 + h < a.group;
            s[h] = in ? *reinterpret_cast<const float4*>(scores + (h0 + h) * a.score_stride) : make_float4(0.f, 0.f, 0.f, 0.f);
            lse2[h] = in ? a.lse2[head0 + h0 + h] : -INFINITY;
        }
#pragma unroll
        for (int h = 0; h < 8; ++h)
            if (lse2[h] != -INFINITY) {
                w[0] += ex2(s[h].x - lse2[h]);
                w[1] += ex2(s[h].y - lse2[h]);
                w[2] += ex2(s[h].z - lse2[h]);
                w[3] += ex2(s[h].w - lse2[h]);
            }
    }
#pragma unroll
    for (int k = 0; k < kWeightTokens; ++k)
        if (t + k < n) a.weight_out[e + k] = before[k] + w[k];
}

struct AttendWs {
    size_t sync, part_o, part_ml, lse2, scores, total;
    int64_t score_stride;
};
static AttendWs attend_ws(const moe_w4_kv_cache& c, int n_q_heads, int max_len, bool track) {
    AttendWs w{};
    // the arrival records come first, where no other operator writes: they have to
    // be zero between calls
    size_t o = MOE_W4_CTRL_BYTES + kSyncBytes;
    auto take = [&](size_t bytes) { const size_t at = o; o += round_up(bytes, 256); return at; };
    w.sync = MOE_W4_CTRL_BYTES;
    w.part_o = take((size_t)2 * most_ctas(c.head_dim) * most_heads(c.head_dim) * c.head_dim * 4);
    w.part_ml = take((size_t)2 * most_ctas(c.head_dim) * most_heads(c.head_dim) * 2 * 4);
    w.score_stride = (int64_t)round_up((size_t)max_len, kSub);
    if (track) {
        w.lse2 = take((size_t)c.n_seqs * n_q_heads * 4);
        w.scores = take((size_t)c.n_seqs * n_q_heads * (size_t)w.score_stride * 4);
    }
    w.total = o;
    return w;
}

template <typename T, int D, int NB>
static cudaError_t launch_attend(const AttendArgs& a, cudaStream_t st) {
    int dev = 0;
    const int sms = sm_count(&dev);
    if (sms < 1) return cudaErrorInvalidDevice;
    constexpr int ring = AttCfg<D, NB>::slots * kAttWarps * unit_bytes(D);
    // the join of a row holds parts * cols < 8 NB * D / 4 + parts columns, and parts *
    // pairs <= 4 NB + 2 parts maxima and sums; two rows share one CTA at most
    static_assert(ring >= 16 * (8 * NB + 3 * (kMaxSms * AttCfg<D, NB>::ctas + 1) + 4 * NB * D), "a join fits the ring");
    static_assert(AttCfg<D, NB>::ctas * kMaxSms <= most_ctas(D), "the workspace holds every CTA's parts");
    static_assert(most_ctas(D) * sizeof(RowSync) <= kRowSyncBytes, "a record for every CTA");
    const int64_t rows = (int64_t)a.c.n_seqs * a.c.n_kv_heads * a.head_blocks;
    // no more CTAs than places that the longest lengths could make
    const int64_t tiles = a.max_len > kTile ? (a.max_len + kTile - 1) / kTile : 1, most = rows * (tiles + kRowCost);
    // the lengths of very many sequences cost a CTA of an SM
    const int smem = ring + q_bytes(D, NB) + (int)round_up((size_t)a.c.n_seqs * 4, 16);
    const int per_sm = (228 << 10) / (smem + 2304) < AttCfg<D, NB>::ctas ? (228 << 10) / (smem + 2304) : AttCfg<D, NB>::ctas;
    int64_t ctas = (int64_t)sms * per_sm;
    if (ctas > kMaxSms * AttCfg<D, NB>::ctas) ctas = kMaxSms * AttCfg<D, NB>::ctas;
    if (ctas > most) ctas = most;
    static std::atomic<unsigned> ready;
    const auto kern = attend_kernel<T, D, NB>;
    cudaError_t e = allow_smem((const void*)kern, ring + q_bytes(D, NB) + MOE_W4_MAX_SEQS * 4, ready, dev);
    if (e != cudaSuccess) return e;
    // Rows can be cut only where there are more tiles than rows; CTAs that share a
    // row wait for one another, so all must be resident.
    const bool together = ctas > 1 && tiles > 1;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeCooperative;
    attr[1].val.cooperative = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kAttThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = together ? 2 : 1;
    do {   // a device shared with others may refuse a full grid: any smaller one will do
        cfg.gridDim = dim3((unsigned)ctas);
        e = cudaLaunchKernelEx(&cfg, kern, a);
    } while (e == cudaErrorCooperativeLaunchTooLarge && (cudaGetLastError(), ctas /= 2) > 0);
    if (e == cudaSuccess && a.scores && a.max_len > 0)
        e = launch_pdl(true, attend_weight_kernel,
                       dim3((a.max_len + kWeightThreads * kWeightTokens - 1) / (kWeightThreads * kWeightTokens),
                            a.c.n_kv_heads, a.c.n_seqs),
                       dim3(kWeightThreads), 0, st, a);
    return e;
}

template <typename T>
static cudaError_t launch_attend_dim(int dim, const AttendArgs& a, cudaStream_t st) {
    const int blocks = (a.block_heads + 7) / 8;
    if (dim == 256) return blocks == 1 ? launch_attend<T, 256, 1>(a, st) : launch_attend<T, 256, 2>(a, st);
    if (dim == 128)
        return blocks == 1 ? launch_attend<T, 128, 1>(a, st)
               : blocks == 2 ? launch_attend<T, 128, 2>(a, st) : launch_attend<T, 128, 3>(a, st);
    return blocks == 1 ? launch_attend<T, 64, 1>(a, st)
           : blocks == 2 ? launch_attend<T, 64, 2>(a, st) : launch_attend<T, 64, 3>(a, st);
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
    a.head_blocks = (a.group + most_heads(c->head_dim) - 1) / most_heads(c->head_dim);
    a.block_heads = (a.group + a.head_blocks - 1) / a.head_blocks;
    a.max_len = max_len;
    a.scale_log2 = scale * kLog2e;
    a.part_o = reinterpret_cast<float*>(ws + w.part_o);
    a.part_ml = reinterpret_cast<float*>(ws + w.part_ml);
    a.ctrl = reinterpret_cast<Ctrl*>(ws);
    a.sync = reinterpret_cast<RowSync*>(ws + w.sync);
    a.k = static_cast<const uint4*>(c->k);
    a.v = static_cast<const uint4*>(c->v);
    a.page_pieces = (uint32_t)(c->page_stride / 8);
    a.head_pieces = (uint32_t)(c->head_stride / 8);
    a.slot_pieces = (uint32_t)(c->slot_stride / 8);
    a.runs = c->page_size % 16 == 0 ? 1 : c->page_size % 8 == 0 ? 2 : 0;
    if (track) {
        a.lse2 = reinterpret_cast<float*>(ws + w.lse2);
        a.scores = reinterpret_cast<float*>(ws + w.scores);
        a.score_stride = w.score_stride;
        a.weight = track->weight;
        a.weight_out = weight_out;
        a.track_seq = track->seq_stride;
        a.track_head = track->head_stride;
    }
    const int64_t places = ((max_len > kTile ? ((int64_t)max_len + kTile - 1) / kTile : 1) + kRowCost) * c->n_seqs * c->n_kv_heads;
    if (places > INT_MAX / a.head_blocks) return MOE_W4_ERR_UNSUPPORTED;   // the list is indexed with 32 bits
    return launched(c->dtype == MOE_W4_TYPE_BF16 ? launch_attend_dim<__nv_bfloat16>(c->head_dim, a, stream)
                                                 : launch_attend_dim<__half>(c->head_dim, a, stream));
}

}  // extern "C"
