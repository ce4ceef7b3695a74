// Shared by the attention kernels of one new token per sequence: their arguments,
// the list of tiles and its shares, the join of rows that several CTAs have worked
// on, the workspace.
#pragma once
#include <climits>

#include "serving.cuh"

namespace mw4 {

constexpr int kAttWarps = 4;
constexpr int kAttThreads = kAttWarps * 32;
constexpr int most_heads(int dim) { return dim == 256 ? 16 : 24; }   // query heads of a row
constexpr int kMaxSms = 160;                    // SMs that the workspace has room for

constexpr int q_bytes(int dim, int blocks) { return blocks > 1 ? blocks * 8 * dim * 2 : 0; }
// CTAs of a grid at most: an SM has up to 4 (head_dim 64), 3 (128) or 2 (256).
constexpr int most_ctas(int dim) { return kMaxSms * (dim == 64 ? 4 : dim == 128 ? 3 : 2); }

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
    int runs;           // a warp's part of a tile is 1 or more equal runs of 8 tokens or more in memory, or 0: any
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
    int window, sink;   // 0: every token is seen; else those below sink and the last `window`
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
template <> struct Elem<__nv_bfloat16> : Pair16<__nv_bfloat16> {
    static constexpr float kBelow = 0.f, kLazy = 8.f;
    MW4_DEV static void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
template <> struct Elem<__half> : Pair16<__half> {
    static constexpr float kBelow = 13.f, kLazy = 2.f;
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

// n / d where the quotient is below 2^20 and d at most 2^30: an approximate one, off by one at most, put right.
MW4_DEV uint32_t div_small(uint32_t n, uint32_t d) {
    uint32_t q = (uint32_t)__fdividef((float)n, (float)d);
    const uint32_t r = n - q * d;
    if ((int)r < 0) --q;
    else if (r >= d) ++q;
    return q;
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
    MW4_DEV int owner(uint32_t place) const {   // (of several parts)
        const uint32_t longer = r * (q + 1);
        return (int)(place < longer ? div_small(place, q + 1) : r + div_small(place - longer, q));
    }
};

// Places of a row in the list: its tiles and kRowCost more, with no tokens, for
// what the end of a row costs, about the time of a tile.  Without them the CTAs
// that got the short sequences of a mixed batch are the last by far (16 sequences
// of 1 to 32,768 tokens: 69.5 us against 64.0; with 2 the same 64.0).
constexpr int kRowCost = 1;

// A place in the list of tiles.  With a window the tiles between the first tokens'
// and the window's are left out: tiles from `split` on lie `gap` tiles further.
struct Place {
    int b, row, tile, tiles, len;
    int first, low, split, gap;   // seen: tokens below `first` and from `low` on
};

// How the tokens of a sequence are cut into tiles of TILE, of which a warp has SUB.
// Tokens that are not seen take no part, as if they were not there; tiles lie at
// multiples of TILE all the same, so that a warp's tokens share pages as they do
// without a window.
template <int TILE, int SUB, bool WIN>
struct Cut {
    int window, sink;
    MW4_DEV explicit Cut(const AttendArgs& a) : window(a.window), sink(a.sink) {}
    MW4_DEV void set(Place& p) const {   // p.len is known
        const int all = (p.len + TILE - 1) / TILE;
        p.tiles = max(1, all);
        if (WIN) {
            p.low = max(0, window ? p.len - window : 0);
            p.first = min(sink, p.low);
            p.split = (p.first + TILE - 1) / TILE;
            p.gap = max(0, p.low / TILE - p.split);
            p.tiles = max(1, all - p.gap);
        }
    }
    MW4_DEV uint32_t places(int len) const {
        Place p;
        p.len = len;
        set(p);
        return p.tiles + kRowCost;
    }
    // the first token of a tile, and which tokens are seen: one, any or all of a warp's
    MW4_DEV int token(const Place& p, int tile) const { return (WIN && tile >= p.split ? tile + p.gap : tile) * TILE; }
    MW4_DEV bool seen(const Place& p, int t) const { return t < p.len && (!WIN || t < p.first || t >= p.low); }
    MW4_DEV bool any8(const Place& p, int t0) const { return t0 < p.len && (!WIN || t0 < p.first || t0 + 8 > p.low); }   // of 8 tokens
    MW4_DEV bool any(const Place& p, int t0) const { return t0 < p.len && (!WIN || t0 < p.first || t0 + SUB > p.low); }
    MW4_DEV bool all(const Place& p, int t0) const { return t0 + SUB <= p.len && (!WIN || t0 + SUB <= p.first || t0 >= p.low); }

    // Sum of the places over the sequences; every thread of a warp gets it.  A lane also
    // gets those of its sequence among the first 32, and of all up to it.
    MW4_DEV uint32_t warp_places(const int* lens, int n_seqs, uint32_t& mine, uint32_t& incl) const {
        const int lane = threadIdx.x & 31;
        mine = lane < n_seqs ? places(lens[lane]) : 0;
        incl = scan(mine, lane);
        uint32_t n = mine;
        if (n_seqs <= 32) return __shfl_sync(0xffffffffu, incl, 31);
        for (int b = lane + 32; b < n_seqs; b += 32) n += places(lens[b]);
        return __reduce_add_sync(0xffffffffu, n);
    }
    static MW4_DEV uint32_t scan(uint32_t mine, int lane) {
        uint32_t incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        return incl;
    }
    // The sequence that holds place x of the list and the first place of that
    // sequence, found by a whole warp; mine and incl as warp_places left them.
    MW4_DEV void find_seq(const int* lens, int n_seqs, uint32_t rows, uint32_t x, uint32_t mine, uint32_t incl, int& b,
                          uint32_t& first) const {
        const int lane = threadIdx.x & 31;
        uint32_t base = 0;
        for (int b0 = 0;; b0 += 32) {
            if (b0) {
                mine = b0 + lane < n_seqs ? places(lens[b0 + lane]) : 0;
                incl = scan(mine, lane);
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
    MW4_DEV void next_row(const int* lens, int n_seqs, int rows, Place& p) const {
        p.tile = 0;
        if (++p.row < rows) return;
        p.row = 0;
        if (++p.b >= n_seqs) return;   // past the end: not used
        p.len = lens[p.b];
        set(p);
    }
};

// Tiles of a row at most, for lengths up to max_len.
inline int64_t most_tiles(int64_t max_len, int tile, int window, int sink) {
    const int64_t all = max_len > tile ? (max_len + tile - 1) / tile : 1;
    if (!window) return all;
    const int64_t some = ((int64_t)sink + tile - 1) / tile + ((int64_t)window + tile - 1) / tile + 1;
    return some < all ? some : all;
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
    // The last to have seen them all clears the row's record.  (Each CTA's wait is over
    // before it counts itself here, and the next kernel comes after this one's end.)
    if (lane == 0 && warp < 2) {
        const int c0 = warp ? open.c0 : begun.c0;
        const unsigned parts = warp ? open.parts : begun.parts;
        if (parts && atomicAdd(&a.sync[c0].left, 1u) == parts - 1) {
            a.sync[c0].arrived = 0;
            a.sync[c0].left = 0;
        }
    }
}

struct AttendWs {
    size_t sync, part_o, part_ml, lse2, scores, total;
    int64_t score_stride;
};
inline AttendWs attend_ws(const moe_w4_kv_cache& c, int n_q_heads, int max_len, bool track) {
    AttendWs w{};
    // the arrival records come first, where no other operator writes: they have to
    // be zero between calls
    size_t o = MOE_W4_CTRL_BYTES + kSyncBytes;
    auto take = [&](size_t bytes) { const size_t at = o; o += round_up(bytes, 256); return at; };
    w.sync = MOE_W4_CTRL_BYTES;
    w.part_o = take((size_t)2 * most_ctas(c.head_dim) * most_heads(c.head_dim) * c.head_dim * 4);
    w.part_ml = take((size_t)2 * most_ctas(c.head_dim) * most_heads(c.head_dim) * 2 * 4);
    w.score_stride = (int64_t)round_up((size_t)max_len, 16);
    if (track) {
        w.lse2 = take((size_t)c.n_seqs * n_q_heads * 4);
        w.scores = take((size_t)c.n_seqs * n_q_heads * (size_t)w.score_stride * 4);
    }
    w.total = o;
    return w;
}

inline int check_heads(const moe_w4_kv_cache& c, int n_q_heads, int max_len) {
    if (n_q_heads < 1 || n_q_heads % c.n_kv_heads || max_len < 0 ||
        (int64_t)max_len > (int64_t)c.pages_per_seq * c.page_size)
        return MOE_W4_ERR_INVALID;
    return n_q_heads / c.n_kv_heads > 128 ? MOE_W4_ERR_UNSUPPORTED : MOE_W4_OK;
}


// What both kernels take; strides in pieces and runs are the kernel's own.
inline AttendArgs attend_args(const moe_w4_kv_cache& c, int n_q_heads, const void* q, int64_t q_stride, float scale,
                              int max_len, int window, int sink, void* out, int64_t out_stride, float* lse,
                              const AttendWs& w, uint8_t* ws) {
    AttendArgs a{};
    a.c = kv_view(c);
    a.q = static_cast<const uint16_t*>(q);
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.n_q_heads = n_q_heads;
    a.group = n_q_heads / c.n_kv_heads;
    a.head_blocks = (a.group + most_heads(c.head_dim) - 1) / most_heads(c.head_dim);
    a.block_heads = (a.group + a.head_blocks - 1) / a.head_blocks;
    a.max_len = max_len;
    a.window = window;
    a.sink = sink;
    a.scale_log2 = scale * kLog2e;
    a.part_o = reinterpret_cast<float*>(ws + w.part_o);
    a.part_ml = reinterpret_cast<float*>(ws + w.part_ml);
    a.ctrl = reinterpret_cast<Ctrl*>(ws);
    a.sync = reinterpret_cast<RowSync*>(ws + w.sync);
    a.k = static_cast<const uint4*>(c.k);
    a.v = static_cast<const uint4*>(c.v);
    return a;
}

}  // namespace mw4
