// Shared by the operators of moe_w4_serving.h: the cache as the kernels see it,
// argument checks, exact division by a page size, and element types.
#pragma once
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "moe_w4_serving.h"

namespace mw4 {

// n / d for 0 <= n < 2^31 by a multiplication (the round-up method of Granlund
// and Montgomery, "Division by Invariant Integers using Multiplication", 1994):
// with s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1 the quotient is
// (mulhi(m, n) + n) >> s; the sum stays below 2^32 because n < 2^31.
struct FastDiv {
    uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d) {
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    return {d, (uint32_t)((((1ull << s) - d) << 32) / d + 1), s};
}
MW4_DEV uint32_t div_by(uint32_t n, const FastDiv& f) { return (__umulhi(f.m, n) + n) >> f.s; }

// The cache as kernels take it.  Offsets are 64-bit: a long cache passes 2^31
// elements.
struct KvView {
    const uint16_t* k;
    const uint16_t* v;
    int64_t page_stride, head_stride, slot_stride, table_stride;
    const int32_t* table;
    const int32_t* lens;
    FastDiv page;
    int num_pages, pages_per_seq, n_seqs, n_kv_heads;
};

// Element offset of token t of sequence b in head 0, or -1 where the block
// table names no page of the cache.
MW4_DEV int64_t kv_offset(const KvView& c, int b, int t) {
    const uint32_t p = div_by((uint32_t)t, c.page);
    if (p >= (uint32_t)c.pages_per_seq) return -1;
    const int page = c.table[b * c.table_stride + p];
    if ((unsigned)page >= (unsigned)c.num_pages) return -1;
    return page * c.page_stride + (int64_t)(t - p * c.page.d) * c.slot_stride;
}

MW4_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
MW4_DEV uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
MW4_DEV uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
MW4_DEV void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same in two halves, for what needs no order of memory: that all CTAs run.
MW4_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
MW4_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// This place of shared memory in CTA `rank` of the cluster.
MW4_DEV uint32_t at_rank(const void* p, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
MW4_DEV int ld_cluster(const int* p, int rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at_rank(p, rank)) : "memory");
    return v;
}
MW4_DEV int2 ld_cluster2(const int* p, int rank) {
    int2 v;
    asm volatile("ld.shared::cluster.v2.s32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at_rank(p, rank)) : "memory");
    return v;
}
// Two 16-bit floats in 32 bits, and as fp32.
template <typename T> struct Pair16;
template <> struct Pair16<__nv_bfloat16> {
    MW4_DEV static uint32_t pack(float a, float b) {
        __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&v);
    }
    MW4_DEV static float2 unpack(uint32_t u) { return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&u)); }
};
template <> struct Pair16<__half> {
    MW4_DEV static uint32_t pack(float a, float b) {
        __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&v);
    }
    MW4_DEV static float2 unpack(uint32_t u) { return __half22float2(*reinterpret_cast<__half2*>(&u)); }
};
constexpr float kLn2 = 0.693147180559945309f, kLog2e = 1.44269504088896341f;

inline bool misaligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

inline int check_cache(const moe_w4_kv_cache* c, bool need_lens) {
    if (!c) return MOE_W4_ERR_INVALID;
    if (c->n_seqs < 0 || c->n_kv_heads < 1 || c->page_size < 1 || c->num_pages < 1 || c->pages_per_seq < 1 ||
        c->table_stride < 0 || c->page_stride < 0 || c->head_stride < 0 || c->slot_stride < 0)
        return MOE_W4_ERR_INVALID;
    if (c->dtype != MOE_W4_TYPE_BF16 && c->dtype != MOE_W4_TYPE_FP16) return MOE_W4_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MOE_W4_ERR_UNSUPPORTED;
    if (c->n_seqs > MOE_W4_MAX_SEQS || c->n_kv_heads > 1024) return MOE_W4_ERR_UNSUPPORTED;
    if ((int64_t)c->pages_per_seq * c->page_size > (1 << 30)) return MOE_W4_ERR_UNSUPPORTED;
    if (((c->page_stride | c->head_stride | c->slot_stride) >> 3) > UINT32_MAX) return MOE_W4_ERR_UNSUPPORTED;
    if (c->n_seqs == 0) return MOE_W4_OK;
    if (!c->k || !c->v || !c->block_table || (need_lens && !c->seq_lens)) return MOE_W4_ERR_INVALID;
    if (misaligned(c->k, 16) || misaligned(c->v, 16) || c->page_stride % 8 || c->head_stride % 8 ||
        c->slot_stride % 8 || misaligned(c->block_table, 4) || misaligned(c->seq_lens, 4))
        return MOE_W4_ERR_ALIGN;
    return MOE_W4_OK;
}

inline int check_track(const moe_w4_kv_track* t, bool need_pos) {
    if (!t->weight || (need_pos && !t->pos) || t->slots < 0 || t->seq_stride < 0 || t->head_stride < 0)
        return MOE_W4_ERR_INVALID;
    if (misaligned(t->weight, 4) || misaligned(t->pos, 4)) return MOE_W4_ERR_ALIGN;
    return MOE_W4_OK;
}

inline int check_workspace(const void* ws, size_t bytes, size_t need) {
    return !ws || misaligned(ws, 256) || bytes < need ? MOE_W4_ERR_WORKSPACE : MOE_W4_OK;
}

inline KvView kv_view(const moe_w4_kv_cache& c) {
    return {static_cast<const uint16_t*>(c.k), static_cast<const uint16_t*>(c.v), c.page_stride, c.head_stride,
            c.slot_stride, c.table_stride, c.block_table, c.seq_lens, fast_div((uint32_t)c.page_size), c.num_pages,
            c.pages_per_seq, c.n_seqs, c.n_kv_heads};
}

// Bytes after the control header that have to be zero between calls, so that
// operators can share a workspace: the attention's arrival records, and the
// eviction's counter for each sequence.
constexpr int kRowSyncBytes = 8192, kSyncBytes = kRowSyncBytes + MOE_W4_MAX_SEQS * 4;

__host__ __device__ constexpr size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

// The current device and its SM count (asked once per device).
inline int sm_count(int* device = nullptr) {
    static std::atomic<int> cached[16];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
    if (device) *device = dev;
    if (dev < 16 && (n = cached[dev].load(std::memory_order_relaxed))) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 16) cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Lets a kernel take `bytes` of dynamic shared memory; the runtime is asked once
// per device.  `done` belongs to the kernel.
inline cudaError_t allow_smem(const void* kern, int bytes, std::atomic<unsigned>& done, int dev) {
    const unsigned bit = dev < 32 ? 1u << dev : 0u;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

inline int launched(cudaError_t e) {
    if (e == cudaSuccess) return MOE_W4_OK;
    cudaGetLastError();   // reported here; not left for the caller's next call
    return MOE_W4_ERR_LAUNCH;
}

}  // namespace mw4
