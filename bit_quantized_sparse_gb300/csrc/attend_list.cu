// Attention of one new token per sequence over a paged cache of 8-bit codes, or of
// 16-bit values with a window.
//
//   s_t = scale q.(ks_t K_t),  p_t = exp(s_t - lse),  lse = log sum_t exp(s_t),
//   out = sum_t p_t vs_t V_t,
// K and V E4M3 codes, ks and vs the scales of a token's block of its head (1 for
// 16-bit values), over the tokens that are seen: all, or with a window the first few
// and the last.
//
// Of codes half the bytes of the 16-bit cache are left, 2 D per token and kv head for
// 4 D group flops; HBM bounds it where rows are long.  The list of tiles, its shares
// and the join are those of the 16-bit kernel without a window (attend.cuh); of codes
// a warp has 32 tokens of a tile of 128, so that a unit of its ring is the same 32 D
// bytes.  Rows that are short take attend_short.cu.
//
// Measured (kernels alone): 1 x 131,072 tokens, 2 kv heads of 256, group 8, codes: 29.2
// us for 135 MB.  Its copies run at the copy rate for 19 us; 2 go before the first of
// them (lengths, the list, page numbers), 2 to a row's end, 2 until the last CTA is
// there, 3 to the join.  16 sequences of up to 32,768 tokens, 8 heads of 128, a scale
// for each token: 38.9 for 189 MB; 8 x 40,000 with a window of 4096 15.0 for 34 MB; 16
// bits, 32 of up to 8192 with a window of 1000, 8 heads of 128: 17.4 for 48 MB.  Groups of more
// than 8 and heads of 64 wait for their own instructions, not for copies: 8 x 16,384, 4 of 128,
// group 16: 43.9 for 135 MB; 4 x 116,918, 2 of 64, group 4: 37.6 for 120 MB.
#include <climits>

#include "attend_short.h"
#include "attend_steps.cuh"

namespace mw4 {

// Ring units per warp and CTAs per SM for a head size; NB blocks of 8 query heads.
// Over codes, two blocks of heads of 128 and three of 64: with 3 CTAs an SM registers would
// spill, 54 and 62 bytes (8 x 16,384 tokens, 4 kv heads of 128, group 16: 47.5 us, with 2 43.9,
// and with rings of 5 units 44.8; 16 x 8192, 4 of 64, group 24: 44.5, with 2 43.3).
template <bool E8, int D, int NB> struct ListCfg;
template <bool E8, int NB> struct ListCfg<E8, 64, NB> {
    static constexpr int slots = E8 && NB == 3 ? 8 : 5, ctas = NB == 1 ? 4 : E8 && NB == 3 ? 2 : 3;
};
template <bool E8, int NB> struct ListCfg<E8, 128, NB> { static constexpr int slots = 3, ctas = E8 && NB == 2 ? 2 : 3; };
template <bool E8> struct ListCfg<E8, 128, 3> { static constexpr int slots = 5, ctas = 2; };
template <bool E8, int NB> struct ListCfg<E8, 256, NB> { static constexpr int slots = 2, ctas = 2; };

// WIN: there is a window.
template <typename T, bool E8, int D, int NB, bool WIN>
__global__ void __launch_bounds__(kAttThreads, ListCfg<E8, D, NB>::ctas) attend_list_kernel(const AttendArgs a, const Scales s) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using St = Steps<T, E8, D, NB>;
    constexpr int HEADS = 8 * NB, SUB = St::SUB, TILE = SUB * kAttWarps, S = ListCfg<E8, D, NB>::slots;
    constexpr int UNIT = St::UNIT;
    __shared__ float sh_m[kAttWarps][HEADS], sh_l[kAttWarps][HEADS];
    __shared__ __align__(8) float sh_qs[HEADS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint8_t* ring = smem + warp * S * UNIT;
    const uint32_t ring_u = smem_u32(ring), ring_end = ring_u + S * UNIT;
    griddep_wait();

    // The lengths, read once: whatever happens to them meanwhile, this CTA's view
    // of the list is one, and its accesses stay in range.
    const int rows = a.c.n_kv_heads * a.head_blocks, n_seqs = a.c.n_seqs;
    uint8_t* q_smem = smem + kAttWarps * S * UNIT;        // the row's queries
    int* lens = reinterpret_cast<int*>(q_smem + St::QBYTES);
    const uint32_t cta = blockIdx.x;
    for (int b = threadIdx.x; b < n_seqs; b += kAttThreads) {
        const int n = a.c.lens[b];
        if (cta == 0 && (n < 0 || n > a.max_len)) raise_status(&a.ctrl->status, MOE_W4_STATUS_BAD_INDEX);
        lens[b] = n < 0 ? 0 : min(n, a.max_len);
    }
    __syncthreads();
    const Cut<TILE, SUB, WIN> cut(a);
    uint32_t places, places_incl;
    const Shares sh(cut.warp_places(lens, n_seqs, places, places_incl) * rows, gridDim.x);
    if (cta >= sh.parts) return;
    uint32_t place = sh.start(cta);                       // of `at` in the list
    const uint32_t end = sh.start(cta + 1);
    Place at;
    uint32_t seq_first;
    cut.find_seq(lens, n_seqs, rows, place, places, places_incl, at.b, seq_first);
    at.len = lens[at.b];
    cut.set(at);
    const uint32_t row_places = at.tiles + kRowCost;
    at.row = (int)div_small(place - seq_first, row_places);
    at.tile = (int)(place - seq_first - at.row * row_places);
    if (at.tile >= at.tiles) {                            // past a row's tiles: on to the next
        place += row_places - at.tile;
        if (place >= end) return;
        cut.next_row(lens, n_seqs, rows, at);
    }

    // ---- loads: units in order, keys and values of one tile after the other ----
    // Offsets are in pieces of 16 bytes.  The block table is read one tile ahead of
    // the keys: behind a full queue of them that load takes microseconds.
    Loader<St, decltype(cut)> loader(a, s, cut, lane);
    const int in_unit = lane & (SUB - 1);
    Place ld = at;                 // the tile loaded next
    bool more = true;              // to load
    int token = cut.token(at, at.tile) + warp * SUB + in_unit;   // of ld's tile, this lane's to look up
    int page = -1;                 // of token
    auto look_up = [&]() {
        const int kvh = ld.row / a.head_blocks;
        loader.look_up(ld, token, page, (uint64_t)kvh * a.head_pieces, kvh, true);
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
            cut.next_row(lens, n_seqs, rows, ahead);
            ahead_token = cut.token(ahead, 0) + warp * SUB + in_unit;
        } else {
            ahead_token = cut.token(ahead, ahead.tile) + warp * SUB + in_unit;
        }
        more_ahead = ahead_place < end;
        if (more_ahead) next_page = loader.read_page(ahead, ahead_token);
    };
    uint32_t fill = ring_u;
    bool values = false;           // the next unit is one of values
    auto load_unit = [&]() {
        if (more) {
            loader.load(fill, values ? a.v : a.k, !values);
            cp_async_commit();
            if (values && (more = more_ahead)) {
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
    page = loader.read_page(ld, token);
    read_ahead();

    // ---- the queries of a row, and its running results ----
    St st(lane);
    uint4 qp[St::QN];
    auto load_q = [&](const Place& p) {
        const int kvh = p.row / a.head_blocks, hb = p.row % a.head_blocks;
        const int heads = min(a.block_heads, a.group - hb * a.block_heads);
        St::load_q(qp, a.q + p.b * a.q_stride + (int64_t)(kvh * a.group + hb * a.block_heads) * D, heads);
    };
    load_q(at);
    St::store_q(qp, q_smem, sh_qs, a.scale_log2);
    __syncthreads();
    look_up();

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
    auto start_row = [&]() {
        const int kvh = at.row / a.head_blocks, hb = at.row - kvh * a.head_blocks;
        heads = min(a.block_heads, a.group - hb * a.block_heads);
        head0 = kvh * a.group + hb * a.block_heads;
        first = at.tile;
        st.start();
    };
    // The end of a row's tiles here: the warps' results meet, brought to a common
    // maximum, outputs added in warp order through the unit that has just been used.
    auto finish_row = [&](bool row_ends) {
        Place nx = at;
        cut.next_row(lens, n_seqs, rows, nx);
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) st.l[n][c] += __shfl_xor_sync(0xffffffffu, st.l[n][c], x);
                if (st.g == 0) sh_m[warp][n * 8 + 2 * st.t4 + c] = st.m[n][c];
            }
        __syncthreads();
        const bool whole = row_ends && first == 0;
        const int64_t slot = (int64_t)(cta * 2 + (first == 0 ? 1 : 0)) * HEADS;
        const uint32_t here = take - ring_u;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            float by[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int h = n * 8 + 2 * st.t4 + c;
                float M = sh_m[0][h];
#pragma unroll
                for (int w = 1; w < kAttWarps; ++w) M = fmaxf(M, sh_m[w][h]);
                // a warp without a score above -inf: 0, or NaN where it has met one
                const float f = st.m[n][c] == -INFINITY ? (st.l[n][c] == 0.f ? 0.f : NAN) : ex2(st.m[n][c] - M);
                by[c] = f;
                if (st.g == 0) sh_l[warp][h] = st.l[n][c] * f;
            }
            st.put(reinterpret_cast<float*>(ring + here), n, by[0], by[1]);
            __syncthreads();
            const bool next_q = n == NB - 1 && place < end;   // nobody uses the present ones any more
            if (next_q) load_q(nx);
            const int quads = min(8, heads - n * 8) * (D / 4);
#pragma unroll 1
            for (int e = threadIdx.x; e < quads; e += kAttThreads) {
                const int h8 = e / (D / 4), col = (e % (D / 4)) * 4, h = n * 8 + h8;
                const float* from = reinterpret_cast<const float*>(smem + here) + h8 * (D + 4) + col;
                float4 p[kAttWarps];
#pragma unroll
                for (int w = 0; w < kAttWarps; ++w) p[w] = *reinterpret_cast<const float4*>(from + w * (S * UNIT / 4));
                float4 v = p[0];
                float L = sh_l[0][h], M = sh_m[0][h];
#pragma unroll
                for (int w = 1; w < kAttWarps; ++w) {
                    v.x += p[w].x; v.y += p[w].y; v.z += p[w].z; v.w += p[w].w;
                    L += sh_l[w][h];
                    M = fmaxf(M, sh_m[w][h]);
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
            if (next_q) St::store_q(qp, q_smem, sh_qs, a.scale_log2);
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
        const int t0 = cut.token(at, at.tile) + warp * SUB;
        const bool mine = u >= 0 && cut.any(at, t0);
        cp_async_wait<S - 1>();
        __syncwarp();
        if (mine && !(u & 1))
            st.keys(take, reinterpret_cast<const float*>(ring + (take - ring_u) + St::SCALES), q_u, sh_qs,
                    !cut.all(at, t0) || loader.bad_pages, [&](int t) { return loader.gone(at, t0 + t); });
        else if (mine)
            st.values(take);
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

template <typename T, bool E8, int D, int NB, bool WIN>
static cudaError_t launch_list_win(const AttendArgs& a, const Scales& s, cudaStream_t st) {
    int dev = 0;
    const int sms = sm_count(&dev);
    if (sms < 1) return cudaErrorInvalidDevice;
    using St = Steps<T, E8, D, NB>;
    constexpr int ring = ListCfg<E8, D, NB>::slots * kAttWarps * St::UNIT, queries = St::QBYTES, TILE = St::SUB * kAttWarps;
    // the join of a row holds parts * cols < 8 NB * D / 4 + parts columns, and parts *
    // pairs <= 4 NB + 2 parts maxima and sums; two rows share one CTA at most
    static_assert(ring >= 16 * (8 * NB + 3 * (kMaxSms * ListCfg<E8, D, NB>::ctas + 1) + 4 * NB * D), "a join fits the ring");
    static_assert(ListCfg<E8, D, NB>::ctas * kMaxSms <= most_ctas(D), "the workspace holds every CTA's parts");
    static_assert(most_ctas(D) * sizeof(RowSync) <= kRowSyncBytes, "a record for every CTA");
    const int64_t rows = (int64_t)a.c.n_seqs * a.c.n_kv_heads * a.head_blocks;
    // no more CTAs than places that the longest lengths could make
    const int64_t tiles = most_tiles(a.max_len, TILE, a.window, a.sink), most = rows * (tiles + kRowCost);
    // the lengths of very many sequences cost a CTA of an SM
    const int smem = ring + queries + (int)round_up((size_t)a.c.n_seqs * 4, 16);
    const int per_sm = (228 << 10) / (smem + 2304) < ListCfg<E8, D, NB>::ctas ? (228 << 10) / (smem + 2304) : ListCfg<E8, D, NB>::ctas;
    int64_t ctas = (int64_t)sms * per_sm;
    if (ctas > kMaxSms * ListCfg<E8, D, NB>::ctas) ctas = kMaxSms * ListCfg<E8, D, NB>::ctas;
    if (ctas > most) ctas = most;
    static std::atomic<unsigned> ready;
    const auto kern = attend_list_kernel<T, E8, D, NB, WIN>;
    cudaError_t e = allow_smem((const void*)kern, ring + queries + MOE_W4_MAX_SEQS * 4, ready, dev);
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
        e = cudaLaunchKernelEx(&cfg, kern, a, s);
    } while (e == cudaErrorCooperativeLaunchTooLarge && (cudaGetLastError(), ctas /= 2) > 0);
    return e;
}

// (16-bit values without a window have a kernel of their own, which keeps a block's queries in registers and has
// no arithmetic of windows: 1 x 131,072, 16/2 heads of 256: 45.4 us, through this one 46.5; 16 x 30,000, 24/8 of
// 64: 152 and 172; 8 x 16,384, 96/4 of 128: 55.5 and 63.6)
template <typename T, bool E8, int D, int NB>
static cudaError_t launch_list(const AttendArgs& a, const Scales& s, cudaStream_t st) {
    if (!E8 || a.window) return launch_list_win<T, E8, D, NB, true>(a, s, st);
    return launch_list_win<T, E8, D, NB, !E8>(a, s, st);
}

template <typename T, bool E8>
static cudaError_t launch_list_dim(int dim, const AttendArgs& a, const Scales& s, cudaStream_t st) {
    const int blocks = (a.block_heads + 7) / 8;
    if (dim == 256) return blocks == 1 ? launch_list<T, E8, 256, 1>(a, s, st) : launch_list<T, E8, 256, 2>(a, s, st);
    if (dim == 128)
        return blocks == 1 ? launch_list<T, E8, 128, 1>(a, s, st)
               : blocks == 2 ? launch_list<T, E8, 128, 2>(a, s, st) : launch_list<T, E8, 128, 3>(a, s, st);
    return blocks == 1 ? launch_list<T, E8, 64, 1>(a, s, st)
           : blocks == 2 ? launch_list<T, E8, 64, 2>(a, s, st) : launch_list<T, E8, 64, 3>(a, s, st);
}

// A checked cache; codes come with their scales.
static int attend(const moe_w4_kv_cache& c, const Scales* scales, const moe_w4_attend_call& t, cudaStream_t stream) {
    int r = check_heads(c, t.n_q_heads, t.max_len);
    if (r) return r;
    if (t.window < 0 || t.sink < 0 || (!t.window && t.sink)) return MOE_W4_ERR_INVALID;
    if (c.n_seqs == 0) return MOE_W4_OK;
    if (!t.q || !t.out || (c.n_seqs > 1 && (t.q_stride < 0 || t.out_stride < (int64_t)t.n_q_heads * c.head_dim)))
        return MOE_W4_ERR_INVALID;
    if (misaligned(t.q, 16) || misaligned(t.out, 16) || t.q_stride % 8 || t.out_stride % 8 || misaligned(t.lse, 4))
        return MOE_W4_ERR_ALIGN;
    const AttendWs w = attend_ws(c, t.n_q_heads, t.max_len, false);
    if ((r = check_workspace(t.workspace, t.ws_bytes, w.total))) return r;
    AttendArgs a = attend_args(c, t.n_q_heads, t.q, t.q_stride, t.scale, t.max_len, t.window, t.sink, t.out, t.out_stride, t.lse, w,
                               static_cast<uint8_t*>(t.workspace));
    const bool e8 = scales != nullptr, bf16 = c.dtype == MOE_W4_TYPE_BF16;
    const int piece = e8 ? 16 : 8;      // elements
    a.page_pieces = (uint32_t)(c.page_stride / piece);
    a.head_pieces = (uint32_t)(c.head_stride / piece);
    a.slot_pieces = (uint32_t)(c.slot_stride / piece);
    a.runs = c.page_size % 8 == 0;
    const int64_t places = (most_tiles(t.max_len, (e8 ? 32 : 16) * kAttWarps, t.window, t.sink) + kRowCost) * c.n_seqs * c.n_kv_heads;
    if (places > INT_MAX / a.head_blocks) return MOE_W4_ERR_UNSUPPORTED;   // the list is indexed with 32 bits
    const Scales s = e8 ? *scales : Scales{};
    if (const int ctas = short_ctas(a, c.head_dim, e8)) return launched(launch_attend_short(c.dtype, c.head_dim, e8, a, s, ctas, stream));
    if (e8)
        return launched(bf16 ? launch_list_dim<__nv_bfloat16, true>(c.head_dim, a, s, stream)
                             : launch_list_dim<__half, true>(c.head_dim, a, s, stream));
    return launched(bf16 ? launch_list_dim<__nv_bfloat16, false>(c.head_dim, a, s, stream)
                         : launch_list_dim<__half, false>(c.head_dim, a, s, stream));
}

}  // namespace mw4

using namespace mw4;

extern "C" {

size_t moe_w4_kv8_attend_workspace_size(const moe_w4_kv8_cache* c, int n_q_heads, int max_len) {
    if (check_cache8(c, false) != MOE_W4_OK || check_heads(c->c, n_q_heads, max_len) != MOE_W4_OK) return 0;
    return attend_ws(c->c, n_q_heads, max_len, false).total;
}

int moe_w4_kv8_attend(const moe_w4_kv8_cache* c, const moe_w4_attend_call* t, cudaStream_t stream) {
    const int r = check_cache8(c, true);
    if (r) return r;
    if (!t) return MOE_W4_ERR_INVALID;
    const Scales s = scales_of(*c);
    return attend(c->c, &s, *t, stream);
}

int moe_w4_attend_window(const moe_w4_kv_cache* c, const moe_w4_attend_call* t, cudaStream_t stream) {
    const int r = check_cache(c, true);
    if (r) return r;
    return t ? attend(*c, nullptr, *t, stream) : MOE_W4_ERR_INVALID;
}

}  // extern "C"
