// Attention of one new token per sequence where rows are short: a cluster of CTAs for
// each row (sequence, kv head, block of query heads).
//
// The kernels that share out a list of tiles (attend.cu, attend_list.cu) balance any
// lengths, but each call costs them about 10 us: lengths and list before the first
// load, and a join through HBM and L2 with waits between CTAs.  Where every row has
// few tiles there is nothing to balance.  Here a CTA knows its row from its place in
// the grid, the cluster's CTAs take the row's tiles in turn, and their results meet
// through distributed shared memory: one cluster barrier, then each CTA adds up its
// share of the row's columns over all warps of the cluster.
//
// What bounds it is the chain of a call: length, page numbers, keys and values, one
// trip to memory after the other, then the products, the barrier and the join.
#include <climits>

#include "attend_steps.cuh"
#include "attend_short.h"

namespace mw4 {

constexpr int kShortCtas = 8;      // CTAs of a row at most: a portable cluster, whose warps are no more than a warp's lanes

// CTAs of an SM that registers leave room for, for a head size and blocks of 8 query
// heads; and ring units per warp: a CTA has a few tiles at most, and more units only
// add turns before the first product (1 x 300: 7.2 us with 2, 7.6 with 4).
constexpr int short_per_sm(int dim, int blocks) { return dim == 256 || (dim == 128 && blocks == 3) ? 2 : dim == 128 || blocks == 3 ? 3 : 4; }
template <int D, int NB> struct ShortCfg {
    static constexpr int slots = NB == 3 ? 3 : 2, ctas = short_per_sm(D, NB);
};

MW4_DEV uint32_t at_rank_u(uint32_t p, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(p), "r"(rank));
    return a;
}
MW4_DEV float4 ld_cluster4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}

template <typename T, bool E8, int D, int NB>
__global__ void __launch_bounds__(kAttThreads, ShortCfg<D, NB>::ctas) attend_short_kernel(const AttendArgs a, const Scales sc) {
    using St = Steps<T, E8, D, NB>;
    constexpr int S = ShortCfg<D, NB>::slots, SUB = St::SUB, TILE = SUB * kAttWarps, UNIT = St::UNIT, HEADS = St::HEADS;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ float2 sh_ml[kAttWarps][HEADS];       // reference maximum (log2) and sum of each warp
    __shared__ __align__(8) float sh_qs[HEADS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
    uint8_t* ring = smem + warp * S * UNIT;
    const uint32_t ring_u = smem_u32(ring), ring_end = ring_u + S * UNIT;
    uint8_t* q_smem = smem + kAttWarps * S * UNIT;
    griddep_wait();

    const int row = blockIdx.y, b = blockIdx.z;
    const int kvh = a.head_blocks == 1 ? row : row / a.head_blocks, hb = row - kvh * a.head_blocks;
    const int heads = min(a.block_heads, a.group - hb * a.block_heads), head0 = kvh * a.group + hb * a.block_heads;
    int n = __shfl_sync(0xffffffffu, a.c.lens[b], 0);   // one reading a warp
    uint4 qp[St::QN];
    St::load_q(qp, a.q + b * a.q_stride + (int64_t)head0 * D, heads);
    if ((n < 0 || n > a.max_len) && threadIdx.x == 0 && row == 0 && rank == 0) raise_status(&a.ctrl->status, MOE_W4_STATUS_BAD_INDEX);
    const Cut<TILE, SUB, true> cut(a);
    Place p;
    p.len = max(0, min(n, a.max_len));
    cut.set(p);

    // ---- loads: keys and values of one of the CTA's tiles after the other ----
    Loader<St, decltype(cut)> loader(a, sc, cut, lane);
    p.b = b;
    int ld = rank;                 // the tile loaded next
    auto token_of = [&](int tile) { return cut.token(p, tile) + warp * SUB + (lane & (SUB - 1)); };
    // page numbers of it and of the one after it
    int page = ld < p.tiles ? loader.read_page(p, token_of(ld)) : -1;
    int next_page = ld + ctas < p.tiles ? loader.read_page(p, token_of(ld + ctas)) : -1;
    const uint64_t head_off = (uint64_t)kvh * a.head_pieces;
    uint32_t fill = ring_u;
    bool values = false;           // the next unit is one of values
    auto load_unit = [&]() {
        if (!values) loader.look_up(p, token_of(ld), page, head_off, kvh, ld < p.tiles);
        loader.load(fill, values ? a.v : a.k, !values);
        cp_async_commit();
        fill = fill + UNIT == ring_end ? ring_u : fill + UNIT;
        if (values) {              // on to the next tile
            ld += ctas;
            page = next_page;
            next_page = ld + ctas < p.tiles ? loader.read_page(p, token_of(ld + ctas)) : -1;
        }
        values = !values;
    };

    St st(lane);
    const uint32_t q_u = smem_u32(q_smem);
    uint32_t take = ring_u;        // the next unit to use
    int tile = rank;
    bool fresh = true;
    // one turn a unit, the first S of them only to fill the ring: a single copy of the loading code
#pragma unroll 1
    for (int u = -S; tile < p.tiles || fresh; ++u) {
        if (u == 0) {
            fresh = false;
            St::store_q(qp, q_smem, sh_qs, a.scale_log2);
            __syncthreads();       // once in every warp, tiles or none
            st.start();
            if (tile >= p.tiles) break;
        }
        if (u >= 0) {
            cp_async_wait<S - 1>();
            __syncwarp();
            const int t0 = token_of(tile) - (lane & (SUB - 1));
            if (cut.any(p, t0)) {
                if (!(u & 1))
                    st.keys(take, reinterpret_cast<const float*>(ring + (take - ring_u) + St::SCALES), q_u, sh_qs,
                            !cut.all(p, t0) || loader.bad_pages, [&](int t) { return loader.gone(p, t0 + t); });
                else
                    st.values(take);
            }
            __syncwarp();
            if (u & 1) tile += ctas;
            take = take + UNIT == ring_end ? ring_u : take + UNIT;
        }
        load_unit();
    }
    cp_async_wait<0>();
    griddep_launch_dependents();

    // ---- the warps' results meet: each writes its own into its ring ----
    constexpr int OUT = S * UNIT / 4;                // floats of a ring
    float* outs = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) st.l[i][c] += __shfl_xor_sync(0xffffffffu, st.l[i][c], x);
            if (st.g == 0) sh_ml[warp][i * 8 + 2 * st.t4 + c] = make_float2(st.m[i][c], st.l[i][c]);
        }
        st.put(outs + i * 8 * (D + 4), i, 1.f, 1.f);
    }
    cluster_sync();
    // A warp in turn has up to 32 columns of four outputs of a head.  A lane works out
    // the factor of one of the cluster's warps, then adds up its column over all of them.
    constexpr int Q = D / 4, QW = Q < 32 ? Q : 32, GROUPS = 32 / QW;   // heads of 64: two groups of lanes share the warps out
    const int parts = ctas * kAttWarps, col = lane % QW, group = lane / QW;
    for (int w = rank * kAttWarps + warp; w < heads * (Q / QW); w += parts) {
        const int h = w / (Q / QW), at = (w % (Q / QW) * QW + col) * 4;
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < parts) {
            const int2 v = ld_cluster2(reinterpret_cast<const int*>(&sh_ml[lane % kAttWarps][h]), lane / kAttWarps);
            ml = make_float2(__int_as_float(v.x), __int_as_float(v.y));
        }
        float M = ml.x;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
        // a warp without a score above -inf: 0, or NaN where it has met one
        const float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : NAN) : ex2(ml.x - M);
        float L = ml.y * f;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
        const bool none = M == -INFINITY && L == 0.f;
        const float scaled = none ? 0.f : f / L;
        if (at == 0 && group == 0) write_lse(a, b, head0 + h, M, L, none);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        const uint32_t from = smem_u32(smem) + (h * (D + 4) + at) * 4;
#pragma unroll 1
        for (int i0 = 0; i0 < parts; i0 += kAttWarps) {   // a CTA's warps at a time
            float4 x[kAttWarps / GROUPS];
#pragma unroll
            for (int i = 0; i < kAttWarps / GROUPS; ++i) x[i] = ld_cluster4(at_rank_u(from + (i * GROUPS + group) * OUT * 4, i0 / kAttWarps));
#pragma unroll
            for (int i = 0; i < kAttWarps / GROUPS; ++i) {
                const float by = __shfl_sync(0xffffffffu, scaled, i0 + i * GROUPS + group);
                v.x += x[i].x * by; v.y += x[i].y * by; v.z += x[i].z * by; v.w += x[i].w * by;
            }
        }
        if (GROUPS > 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, QW & 31);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, QW & 31);
            v.z += __shfl_xor_sync(0xffffffffu, v.z, QW & 31);
            v.w += __shfl_xor_sync(0xffffffffu, v.w, QW & 31);
        }
        if (group == 0)
            *reinterpret_cast<uint2*>(a.out + b * a.out_stride + (int64_t)(head0 + h) * D + at) =
                make_uint2(Elem<T>::pack(v.x, v.y), Elem<T>::pack(v.z, v.w));
    }
    if (ctas > 1) cluster_sync();  // nobody leaves while others read its results
}

template <typename T, bool E8, int D, int NB>
static cudaError_t launch_short(const AttendArgs& a, const Scales& s, int ctas, cudaStream_t st) {
    using St = Steps<T, E8, D, NB>;
    int dev = 0;
    if (sm_count(&dev) < 1) return cudaErrorInvalidDevice;
    constexpr int ring = ShortCfg<D, NB>::slots * kAttWarps * St::UNIT, smem = ring + St::QBYTES;
    static_assert(ring / kAttWarps >= St::HEADS * (D + 4) * 4, "a warp's outputs fit its ring");
    static std::atomic<unsigned> ready;
    const auto kern = attend_short_kernel<T, E8, D, NB>;
    const cudaError_t e = allow_smem((const void*)kern, smem, ready, dev);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas, a.c.n_kv_heads * a.head_blocks, a.c.n_seqs);
    cfg.blockDim = dim3(kAttThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a, s);
}

template <typename T, bool E8>
static cudaError_t launch_short_dim(int dim, const AttendArgs& a, const Scales& s, int ctas, cudaStream_t st) {
    const int blocks = (a.block_heads + 7) / 8;
    if (dim == 256)
        return blocks == 1 ? launch_short<T, E8, 256, 1>(a, s, ctas, st) : launch_short<T, E8, 256, 2>(a, s, ctas, st);
    if (dim == 128)
        return blocks == 1 ? launch_short<T, E8, 128, 1>(a, s, ctas, st)
               : blocks == 2 ? launch_short<T, E8, 128, 2>(a, s, ctas, st) : launch_short<T, E8, 128, 3>(a, s, ctas, st);
    return blocks == 1 ? launch_short<T, E8, 64, 1>(a, s, ctas, st)
           : blocks == 2 ? launch_short<T, E8, 64, 2>(a, s, ctas, st) : launch_short<T, E8, 64, 3>(a, s, ctas, st);
}

// A cluster has as many CTAs as the row has tiles, up to 8 and to what the GPU holds
// at a time.  Past a few tiles a CTA the list is as fast or faster, and it balances mixed
// lengths; clusters that fill the GPU keep up longer, those of 16-bit values twice as
// many tiles, which have half the tokens and, being of a window, are alike in every row.
// In us, list / clusters, rows of equal lengths, group 8.  Codes, heads of 256: 2 rows of
// 1000 tokens, 1 tile a CTA, 9.3 / 8.1; 16 of 2000, 2, 11.1 / 12.3; 32 of 3000, 3 that fill
// the GPU, 17.1 / 15.5; 256 of 1000, 8, 31.8 / 26.2, of 4000, 32, 84.2 / 83.4; heads of 128:
// 16 of 2000, 2, 10.3 / 9.9; 256 of 500, 4, 16.3 / 13.7, of 2000, 16, 31.4 / 37.6; of 64: 8 of
// 3000, 3, 9.2 / 9.0; 512 of 1000, 8, 26.7 / 21.5.  16 bits: heads of 64, 512 of 1000, 16,
// 34.4 / 26.4; of 128, 256 of 500, 8, 18.8 / 15.7; of 256, 256 of 1000, 16, 46.8 / 41.8.
int short_ctas(const AttendArgs& a, int dim, bool e8) {
    const int64_t rows = (int64_t)a.c.n_seqs * a.c.n_kv_heads * a.head_blocks;
    if ((int64_t)a.c.n_kv_heads * a.head_blocks > 65535) return 0;   // of a grid's dimension
    const int64_t tiles = most_tiles(a.max_len, (e8 ? 32 : 16) * kAttWarps, a.window, a.sink);
    const int64_t room = (int64_t)sm_count() * short_per_sm(dim, (a.block_heads + 7) / 8);
    int ctas = 1;
    while (ctas < kShortCtas && ctas < tiles && rows * ctas * 2 <= room) ctas *= 2;
    const int64_t each = (tiles + ctas - 1) / ctas;
    const int64_t most = rows * ctas * 2 <= room ? (dim == 64 ? 3 : 2) : (dim == 128 ? 4 : 8) * (e8 ? 1 : 2);
    return each <= most ? ctas : 0;
}

cudaError_t launch_attend_short(int dtype, int dim, bool e8, const AttendArgs& a, const Scales& s, int ctas, cudaStream_t st) {
    if (dtype == MOE_W4_TYPE_BF16)
        return e8 ? launch_short_dim<__nv_bfloat16, true>(dim, a, s, ctas, st) : launch_short_dim<__nv_bfloat16, false>(dim, a, s, ctas, st);
    return e8 ? launch_short_dim<__half, true>(dim, a, s, ctas, st) : launch_short_dim<__half, false>(dim, a, s, ctas, st);
}

}  // namespace mw4
