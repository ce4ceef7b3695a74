// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits x:
//   lse = m + log Z,  Z = sum exp(x - m),  m = max x
//   logprob(t) = x_t - lse,  entropy = log Z - sum exp(x - m) (x - m) / Z
//
// HBM bounds large calls in principle; each logit is read once, takes one
// exponential and about six instructions, and the warps wait about as much for
// those as for the copies (4096 x 49999 fp16, top 5: 82 us, 73% of the copy rate;
// without alternatives 86% of that time, the copies alone 71%).
// Latency bounds small ones (1 x 32000 fp32: 7.9 us; 16 x 131072 bf16, top 20: 9.7).
//
// Few rows: a row belongs to a cluster of 1 to 8 CTAs, each with a contiguous part.
// More rows than fit at once: single smaller CTAs of a resident grid take rows in
// turn.  A thread streams vectors of 16 bytes through slots of shared memory that
// only it uses, so nothing but its own copies is waited for, and the ring runs on
// into the CTA's next row while it finishes this one.  It keeps a reference maximum, Z and
// U = sum e (x - m), and its largest logit.
//
// The top k of a part: the k-th largest of the threads' maxima is a lower bound
// tau of the k-th largest logit.  A thread keeps the maximum of each quarter of
// its vectors, so only about k quarters have to be read again, from L2, all of
// them together by the whole CTA (a thread after the other it took 11 us a row
// for the top 20 of 49,999: each access waits behind the stream of loads); what
// reaches tau is listed, and the list, a few entries more than k, is sorted by
// warps.  Ties at tau and NaN can make the list too long or too short: paths of
// their own below, exact for every input.
#include "serving.cuh"

namespace mw4 {

struct LogprobArgs {
    const void* logits;
    int64_t row_stride;
    int n, vocab, top;
    const int32_t* targets;
    float* logprob;
    float* entropy;
    int32_t* top_index;
    float* top_logprob;
    unsigned int* status;
};

// Order of the alternatives: larger logit first, then the lower index; NaN
// after every number.  No logit has key 0.
MW4_DEV uint32_t logit_key(float x) { return isnan(x) ? 1u : order_key(x + 0.f); }
MW4_DEV float key_logit(uint32_t k) {
    return k == 1u ? NAN : __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
MW4_DEV uint64_t logit_word(float x, int i) { return ((uint64_t)logit_key(x) << 32) | (uint32_t)~i; }

constexpr int kLpVecs = 3;                                // vectors of a thread in a stage
constexpr int kLpStages = 2;
constexpr int kLpPerSm = 1024;                            // resident threads per SM
constexpr int kLpList = 256;                              // candidates listed before the paths for ties
constexpr int kLpMaxCluster = 8;
constexpr int kLpQuarters = 4;                            // maxima that a thread keeps
constexpr int kLpAgain = 4;                               // vectors that a thread re-reads at a time
constexpr float kLpLazy = 5.5f;                           // growth of the maximum before a rescale

template <typename T> struct Logit;
template <> struct Logit<float> {
    static constexpr int E = 4;   // of a 16-byte vector
    MW4_DEV static float one(const float* p) { return *p; }
    MW4_DEV static void split(const uint4& v, float2 (&x)[2]) {
        x[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
        x[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
};
template <> struct Logit<__nv_bfloat16> {
    static constexpr int E = 8;
    MW4_DEV static float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    MW4_DEV static float2 two(uint32_t u) { return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)); }
    MW4_DEV static void split(const uint4& v, float2 (&x)[4]) { x[0] = two(v.x); x[1] = two(v.y); x[2] = two(v.z); x[3] = two(v.w); }
};
template <> struct Logit<__half> {
    static constexpr int E = 8;
    MW4_DEV static float one(const __half* p) { return __half2float(*p); }
    MW4_DEV static float2 two(uint32_t u) { return __half22float2(*reinterpret_cast<__half2*>(&u)); }
    MW4_DEV static void split(const uint4& v, float2 (&x)[4]) { x[0] = two(v.x); x[1] = two(v.y); x[2] = two(v.z); x[3] = two(v.w); }
};

// two fp32 operations in one instruction
MW4_DEV uint64_t f2u(float2 v) { return *reinterpret_cast<uint64_t*>(&v); }
MW4_DEV float2 u2f(uint64_t v) { return *reinterpret_cast<float2*>(&v); }
MW4_DEV float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(f2u(a)), "l"(f2u(b)));
    return u2f(d);
}
MW4_DEV float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(f2u(a)), "l"(f2u(b)));
    return u2f(d);
}
MW4_DEV float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(f2u(a)), "l"(f2u(b)), "l"(f2u(c)));
    return u2f(d);
}
MW4_DEV float max_keeping_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

MW4_DEV float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
template <int N>
MW4_DEV float max_of(const float2 (&x)[N]) {
    float v = max3(x[0].x, x[0].y, x[1].x), w = x[1].y;
    if (N == 4) w = max3(max3(x[1].y, x[2 % N].x, x[2 % N].y), x[3 % N].x, x[3 % N].y);
    return fmaxf(v, w);
}

// Sums of a set of logits: Z = sum 2^y, U = sum 2^y y with y = (x - m) log2 e.
// An empty set, or one of nothing but -inf, has m = -inf and Z = U = 0.
struct Sums {
    float m, Z, U;
};
MW4_DEV void rebase(Sums& s, float m) {   // m >= s.m
    if (s.m == -INFINITY) {
        // nothing to move (Z keeps a NaN)
    } else if (m != s.m) {
        const float y = (s.m - m) * kLog2e, f = ex2(y);
        s.U = f == 0.f ? 0.f * s.Z : f * (s.U + s.Z * y);
        s.Z *= f;
    }
    s.m = m;
}
MW4_DEV Sums warp_join(Sums s) {
    float m = s.m;
#pragma unroll
    for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    rebase(s, m);
    s.Z = warp_sum(s.Z);
    s.U = warp_sum(s.U);
    return s;
}

// Bitonic networks over a warp, largest in lane 0.
template <typename V>
MW4_DEV V warp_sort(V v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j; j >>= 1) {
            const V o = __shfl_xor_sync(0xffffffffu, v, j);
            const bool larger = ((lane & j) == 0) == ((lane & k) == 0 || k == 32);
            v = larger ? (o > v ? o : v) : (o > v ? v : o);
        }
    return v;
}
// The 32 largest of two sorted lists, sorted.
template <typename V>
MW4_DEV V warp_merge(V a, V b) {
    const int lane = threadIdx.x & 31;
    const V r = __shfl_sync(0xffffffffu, b, 31 - lane);
    V v = r > a ? r : a;
#pragma unroll
    for (int j = 16; j; j >>= 1) {
        const V o = __shfl_xor_sync(0xffffffffu, v, j);
        v = (lane & j) == 0 ? (o > v ? o : v) : (o > v ? v : o);
    }
    return v;
}

MW4_DEV void st_cluster(uint32_t a, uint64_t v) { asm volatile("st.shared::cluster.u64 [%0], %1;" :: "r"(a), "l"(v) : "memory"); }
MW4_DEV void st_cluster(uint32_t a, float v) { asm volatile("st.shared::cluster.f32 [%0], %1;" :: "r"(a), "f"(v) : "memory"); }

// A CTA's part of a row: vectors [v0, v1) of the row's 16-byte aligned body,
// and for CTA 0 the logits before and after the body, one for each of the
// first threads.
template <typename T, int NT>
struct Part {
    const T* row;
    int head, v0, v1, scalar, count;   // scalar: this thread's logit outside the body, or -1; count: logits of the part
    MW4_DEV Part(const LogprobArgs& a, int r, int rank, int ctas) {
        constexpr int E = Logit<T>::E;
        row = static_cast<const T*>(a.logits) + r * a.row_stride;
        const int skew = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
        head = min(skew ? E - skew : 0, a.vocab);
        const int vecs = (a.vocab - head) / E, per = (vecs + ctas - 1) / ctas;
        v0 = min(vecs, rank * per);
        v1 = min(vecs, v0 + per);
        const int rest = a.vocab - vecs * E;   // head and tail together
        const int tid = threadIdx.x;
        scalar = rank == 0 && tid < rest ? (tid < head ? tid : tid + vecs * E) : -1;
        count = (v1 - v0) * E + (rank == 0 ? rest : 0);
    }
    // stages, and thus vectors of a thread, of a quarter
    MW4_DEV int quarter_chunks() const { return (chunks() + kLpQuarters - 1) / kLpQuarters; }
    MW4_DEV int chunks() const { return max(1, (v1 - v0 + (NT * kLpVecs) - 1) / (NT * kLpVecs)); }
    MW4_DEV const uint4* vec(int v) const { return reinterpret_cast<const uint4*>(row + head) + v; }
    MW4_DEV int index(int v) const { return head + v * Logit<T>::E; }
};

template <int NT>
struct LpShared {
    float lane_max[NT / 32][32];
    uint64_t sorted[NT / 32][32];
    uint64_t list[kLpList];
    float quarter_max[kLpQuarters][NT];
    uint16_t hits[kLpQuarters * NT];             // quarter and thread of the vectors to read again
    static constexpr int kCtas = NT == 256 ? kLpMaxCluster : 1;   // smaller CTAs come one to a row
    uint64_t part_words[kCtas][32];              // of the cluster's CTAs, in CTA 0; a cluster has one row
    float part_sums[kCtas][3];
    Sums sums[NT / 32];
    int warp_count[NT / 32];
    int count, hit_count;
    float tau;
};

// The kk largest words of a part by kk rounds over it.  Only for parts whose
// list is too long for another reason than ties, or short of kk because of NaN.
template <typename T, int NT>
__device__ __noinline__ uint64_t top_by_rounds(const Part<T, NT>& p, int kk, LpShared<NT>& sh) {
    constexpr int E = Logit<T>::E;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t last = ~0ull, mine = 0;
    for (int k = 0; k < kk; ++k) {
        uint64_t best = 0;
        auto see = [&](float x, int i) {
            const uint64_t w = logit_word(x, i);
            if (w < last && w > best) best = w;
        };
        if (p.scalar >= 0) see(Logit<T>::one(p.row + p.scalar), p.scalar);
        for (int v = p.v0 + tid; v < p.v1; v += NT) {
            float2 x[E / 2];
            Logit<T>::split(*p.vec(v), x);
            for (int j = 0; j < E / 2; ++j) {
                see(x[j].x, p.index(v) + 2 * j);
                see(x[j].y, p.index(v) + 2 * j + 1);
            }
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) {
            const uint64_t o = __shfl_xor_sync(0xffffffffu, best, off);
            best = o > best ? o : best;
        }
        __syncthreads();
        if (lane == 0) sh.sorted[warp][0] = best;
        __syncthreads();
        for (int w = 0; w < (NT / 32); ++w) best = sh.sorted[w][0] > best ? sh.sorted[w][0] : best;
        if (lane == k) mine = best;
        last = best;
    }
    return mine;
}

// Lists the logits of the part that are >= tau (> tau where strict).  Called by
// the whole CTA, which then has to meet before it reads the list.
template <typename T, int NT>
__device__ __noinline__ void list_from(const Part<T, NT>& p, float scalar, float tau, bool strict, LpShared<NT>& sh) {
    constexpr int E = Logit<T>::E;
    const int tid = threadIdx.x;
    auto see = [&](float x, int i) {
        if (strict ? x > tau : x >= tau) {
            const int at = atomicAdd(&sh.count, 1);
            if (at < kLpList) sh.list[at] = logit_word(x, i);
        }
    };
    if (p.scalar >= 0) see(scalar, p.scalar);
#pragma unroll
    for (int q = 0; q < kLpQuarters; ++q)
        if (strict ? sh.quarter_max[q][tid] > tau : sh.quarter_max[q][tid] >= tau)
            sh.hits[atomicAdd(&sh.hit_count, 1)] = (uint16_t)(q * NT + tid);
    __syncthreads();
    // Ties, as in a row that is masked with -inf but for a few logits: each of
    // these quarters holds one to list, so that the list would be too long.
    if (sh.hit_count > kLpList) {
        if (tid == 0) sh.count = sh.hit_count;
        return;
    }
    const int per = p.quarter_chunks() * kLpVecs;      // vectors of a thread in a quarter
    const int all = sh.hit_count * per;
    auto place = [&](int e) {                          // e-th of the vectors to read again
        const int hit = e / per, h = sh.hits[hit];
        return p.v0 + h % NT + (h / NT * per + e - hit * per) * NT;
    };
    // (a list that has grown too long is not read)
    for (int e0 = tid; e0 - tid < all && *(volatile int*)&sh.count <= kLpList; e0 += NT * kLpAgain) {
        uint4 v[kLpAgain];
        uint32_t there = 0, mask = 0;                  // logits that reach tau, by vector
#pragma unroll
        for (int k = 0; k < kLpAgain; ++k) {
            const int e = e0 + k * NT, at = e < all ? place(e) : p.v1;
            if (at < p.v1) {
                v[k] = *p.vec(at);
                there |= 1u << k;
            }
        }
#pragma unroll
        for (int k = 0; k < kLpAgain; ++k)
            if (there >> k & 1) {
                float2 x[E / 2];
                Logit<T>::split(v[k], x);
#pragma unroll
                for (int j = 0; j < E / 2; ++j)
                    mask |= (uint32_t)(strict ? x[j].x > tau : x[j].x >= tau) << (k * E + 2 * j) |
                            (uint32_t)(strict ? x[j].y > tau : x[j].y >= tau) << (k * E + 2 * j + 1);
            }
        for (; mask; mask &= mask - 1) {               // few: one copy of this code, from the cache
            const int bit = __ffs(mask) - 1, i = p.index(place(e0 + bit / E * NT)) + bit % E;
            see(Logit<T>::one(p.row + i), i);
        }
    }
}

// Adds to the list the `need` lowest-indexed logits of the body that equal tau
// (fewer if there are not so many), and all such logits outside it (at most 14).
template <typename T, int NT>
__device__ __noinline__ void list_ties(const Part<T, NT>& p, float tau, int need, LpShared<NT>& sh) {
    constexpr int E = Logit<T>::E;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (p.scalar >= 0) {
        const float x = Logit<T>::one(p.row + p.scalar);
        if (x == tau) sh.list[atomicAdd(&sh.count, 1)] = logit_word(x, p.scalar);
    }
    for (int base = p.v0; base < p.v1 && need > 0; base += NT) {
        const int v = base + tid;
        float2 x[E / 2];
        uint32_t eq = 0;
        if (v < p.v1) {
            Logit<T>::split(*p.vec(v), x);
#pragma unroll
            for (int j = 0; j < E / 2; ++j) eq |= (uint32_t)(x[j].x == tau) << (2 * j) | (uint32_t)(x[j].y == tau) << (2 * j + 1);
        }
        const int mine = __popc(eq);
        int incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        __syncthreads();
        if (lane == 31) sh.warp_count[warp] = incl;
        __syncthreads();
        int before = incl - mine, all = 0;
        for (int w = 0; w < (NT / 32); ++w) {
            before += w < warp ? sh.warp_count[w] : 0;
            all += sh.warp_count[w];
        }
        for (; eq && before < need; eq &= eq - 1, ++before)
            sh.list[atomicAdd(&sh.count, 1)] = logit_word(tau, p.index(v) + __ffs(eq) - 1);
        need -= all;
    }
}

// The kk largest words of a part, in lanes 0.. of warp 0.  Not inlined: its
// registers would make the streaming loop spill (4096 x 49999 fp16: 104 us).
template <typename T, int NT>
__device__ __noinline__ uint64_t part_top(const Part<T, NT>& p, float thread_max, float scalar, int kk, LpShared<NT>& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    sh.lane_max[warp][lane] = warp_sort(thread_max);
    if (tid == 0) sh.count = sh.hit_count = 0;
#pragma unroll
    for (int half = NT / 64; half; half >>= 1) {
        __syncthreads();
        if (warp < half) {
            const float v = warp_merge(sh.lane_max[warp][lane], sh.lane_max[warp + half][lane]);
            if (half > 1) sh.lane_max[warp][lane] = v;
            else if (lane == kk - 1) sh.tau = v;
        }
    }
    __syncthreads();
    const float tau = sh.tau;
    list_from(p, scalar, tau, false, sh);
    __syncthreads();
    int c = sh.count;
    if (c > kLpList) {   // many ties at tau: what exceeds it, then the first of them
        __syncthreads();
        if (tid == 0) sh.count = sh.hit_count = 0;
        __syncthreads();
        list_from(p, scalar, tau, true, sh);
        __syncthreads();
        c = sh.count;
        __syncthreads();
        if (c <= kLpList && c < kk) {
            list_ties(p, tau, kk - c, sh);
            __syncthreads();
            c = sh.count;
        }
    }
    if (c > kLpList || c < kk) return top_by_rounds(p, kk, sh);
    const int lists = min((NT / 32), (c + 31) / 32);
    uint64_t best = 0;
    if (warp < lists) {
        for (int at = warp * 32; at < c; at += NT) {
            const uint64_t s = warp_sort(at + lane < c ? sh.list[at + lane] : 0ull);
            best = at == warp * 32 ? s : warp_merge(best, s);
        }
        sh.sorted[warp][lane] = best;
    }
    if (lists > 1) {
        __syncthreads();
        if (warp == 0)
            for (int w = 1; w < lists; ++w) best = warp_merge(best, sh.sorted[w][lane]);
    }
    return lane < kk ? best : 0ull;
}

template <typename T, int NT>
__global__ void __launch_bounds__(NT, kLpPerSm / NT) token_logprobs_kernel(const LogprobArgs a) {
    extern __shared__ __align__(16) uint4 ring[];
    __shared__ LpShared<NT> sh;
    constexpr int E = Logit<T>::E;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster_rank(), ctas = (int)cluster_size();
    const int first = blockIdx.x / ctas, step = gridDim.x / ctas;
    // CTA 0's shared memory may be written by the others once it runs: all say so
    // here, and wait for it when they have their parts
    if (NT == 256 && ctas > 1) cluster_arrive();
    griddep_wait();

    // the next vector of this thread to load, and how many of its row are left
    int load_row = first, left = 0;
    const uint4* from = nullptr;
    auto load_part = [&]() {
        if (load_row < a.n) {
            const Part<T, NT> p(a, load_row, rank, ctas);
            from = p.vec(p.v0 + tid);
            left = p.v1 - p.v0 - tid;   // of the part, from this thread's on
        }
    };
    load_part();
    auto load = [&](int stage) {
        if (load_row < a.n) {
            uint4* to = &ring[stage * (NT * kLpVecs) + tid];
#pragma unroll
            for (int i = 0; i < kLpVecs; ++i)
                if (left > i * NT) cp_async_16(to + i * NT, from + i * NT);
            from += (NT * kLpVecs);
            left -= (NT * kLpVecs);
            if (left + tid <= 0) {   // the part is done: on to the next row's
                load_row += step;
                load_part();
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kLpStages; ++i) load(i);

    int stage = 0;
    for (int r = first; r < a.n; r += step) {
        const Part<T, NT> p(a, r, rank, ctas);
        float scalar = -INFINITY;
        if (p.scalar >= 0) scalar = Logit<T>::one(p.row + p.scalar);
        // what the end of the row needs from memory, asked for now
        int target = -1;
        float target_x = NAN;
        if (rank == 0 && tid == 0 && a.targets) {
            target = a.targets[r];
            if ((unsigned)target < (unsigned)a.vocab) target_x = Logit<T>::one(p.row + target);
        }
        Sums s{-INFINITY, 0.f, 0.f};
        float mine = -INFINITY, limit = -INFINITY;     // mine: of the present quarter
        int turns = p.quarter_chunks();
        float* quarter = &sh.quarter_max[0][tid];
        float2 Z = make_float2(0.f, 0.f), U = Z, minus = Z;
        for (int rest = p.v1 - p.v0 - tid, chunks = p.chunks(); chunks; --chunks, rest -= (NT * kLpVecs)) {
            cp_async_wait<kLpStages - 1>();
            const uint4* at = &ring[stage * (NT * kLpVecs) + tid];
#pragma unroll
            for (int i = 0; i < kLpVecs; ++i) {
                if (rest <= i * NT) break;
                float2 x[E / 2];
                Logit<T>::split(at[i * NT], x);
                const float vm = max_of(x);
                mine = fmaxf(mine, vm);
                // The reference follows the maximum when that has outgrown it by more than
                // kLpLazy, so that a rescale is rare; the sums stay far inside fp32's range.
                if (vm > limit) {
                    Sums t{s.m, Z.x + Z.y, U.x + U.y};
                    rebase(t, vm);
                    s.m = vm;
                    limit = vm + kLpLazy;
                    minus = make_float2(-vm, -vm);
                    Z = make_float2(t.Z, 0.f);
                    U = make_float2(t.U, 0.f);
                }
                const float2 l2e = make_float2(kLog2e, kLog2e);
#pragma unroll
                for (int j = 0; j < E / 2; ++j) {
                    float2 y = mul2(add2(x[j], minus), l2e);
                    // 2^-200 is 0: keeps 0 * -inf out of U; a NaN stays
                    y = make_float2(max_keeping_nan(y.x, -200.f), max_keeping_nan(y.y, -200.f));
                    const float2 e = make_float2(ex2(y.x), ex2(y.y));
                    Z = add2(Z, e);
                    U = fma2(e, y, U);
                }
            }
            load(stage);   // into the slots just read: nobody else reads them
            stage = stage == kLpStages - 1 ? 0 : stage + 1;
            if (--turns == 0) {
                *quarter = mine;
                quarter += NT;
                mine = -INFINITY;
                turns = p.quarter_chunks();
            }
        }
        float most = -INFINITY;
        while (quarter <= &sh.quarter_max[kLpQuarters - 1][tid]) {
            *quarter = mine;
            quarter += NT;
            mine = -INFINITY;
        }
#pragma unroll
        for (int q = 0; q < kLpQuarters; ++q) most = fmaxf(most, sh.quarter_max[q][tid]);
        s.Z = Z.x + Z.y;
        s.U = U.x + U.y;
        if (p.scalar >= 0) {
            if (scalar > s.m) rebase(s, scalar);
            const float y = max_keeping_nan((scalar - (s.m == -INFINITY ? 0.f : s.m)) * kLog2e, -200.f), e = ex2(y);
            s.Z += e;
            s.U += e * y;
            most = fmaxf(most, scalar);
        }
        s = warp_join(s);
        if (lane == 0) sh.sums[warp] = s;
        uint64_t word = 0;
        const int kk = min(a.top, p.count);
        if (kk) word = part_top(p, most, scalar, kk, sh);
        else __syncthreads();
        if (NT == 256 && ctas > 1) cluster_wait();
        if (warp == 0) {
            s = warp_join(lane < (NT / 32) ? sh.sums[lane] : Sums{-INFINITY, 0.f, 0.f});
            if (NT == 256 && ctas > 1) {
                st_cluster(at_rank(&sh.part_words[rank][lane], 0), word);
                if (lane < 3) st_cluster(at_rank(&sh.part_sums[rank][lane], 0), lane == 0 ? s.m : lane == 1 ? s.Z : s.U);
            }
        }
        if (NT == 256 && ctas > 1) cluster_sync();
        else __syncthreads();
        if (rank == 0 && warp == 0) {
            if (NT == 256 && ctas > 1) {
                const float* q = sh.part_sums[lane < ctas ? lane : 0];
                s = warp_join(lane < ctas ? Sums{q[0], q[1], q[2]} : Sums{-INFINITY, 0.f, 0.f});
                if (a.top)
                    for (int c = 1; c < ctas; ++c) word = warp_merge(word, sh.part_words[c][lane]);
            }
            // a NaN, +inf (x - m is NaN then), or nothing but -inf
            const bool none = s.m == -INFINITY || isnan(s.Z);
            const float logZ = none ? NAN : log2f(s.Z) * kLn2;
            // less m first: m + log Z would be rounded at the size of the logits
            auto logprob = [&](float x) { return (x - s.m) - logZ; };
            if (lane < a.top) {
                a.top_index[(int64_t)r * a.top + lane] = (int)~(uint32_t)word;
                a.top_logprob[(int64_t)r * a.top + lane] = logprob(key_logit((uint32_t)(word >> 32)));
            }
            if (lane == 0) {
                if (a.entropy) a.entropy[r] = logZ - s.U / s.Z * kLn2;
                if (a.targets) {
                    const bool in = (unsigned)target < (unsigned)a.vocab;
                    if (!in && target != -1) raise_status(a.status, MOE_W4_STATUS_BAD_INDEX);
                    a.logprob[r] = in ? logprob(target_x) : target == -1 ? 0.f : NAN;
                }
            }
        }
    }
}

template <typename T, int NT>
static cudaError_t launch_logprobs(const LogprobArgs& a, int ctas, int clusters, int dev, cudaStream_t st) {
    constexpr int smem = kLpStages * kLpVecs * NT * 16;
    static std::atomic<unsigned> ready;
    const cudaError_t e = allow_smem((const void*)token_logprobs_kernel<T, NT>, smem, ready, dev);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(clusters * ctas));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T, NT>, a);
}

// Few rows: CTAs of 256 threads, as many (up to 8) to a row as take three quarters
// of the SMs' places and still have a vector for every thread.  Clusters do not
// fit into every place (148 of 4 CTAs into 608; the rest would wait for a second
// turn) and spread unevenly when they nearly fill them: 152 x 131072 bf16 took
// 22.2 us with 4 CTAs a row, 15.8 with 2; 64 rows 13.4 with 8, 11.4 with 4.  Up to
// half instead: 200 rows 21.8 us against 19.2.  More rows than places: CTAs of
// 128 threads with a row each, whose row ends are shorter and overlap better
// (4096 x 49999 fp16: 82 us against 90; for 16 x 131072 bf16 it is the other way
// round, 12.0 against 10.3).
template <typename T>
static cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t st) {
    int dev = 0;
    const int sms = sm_count(&dev);
    if (sms < 1) return cudaErrorInvalidDevice;
    const int places = sms * (kLpPerSm / 256), vecs = a.vocab / Logit<T>::E;
    if (a.n > places) {
        const int most = sms * (kLpPerSm / 128);
        return launch_logprobs<T, 128>(a, 1, a.n < most ? a.n : most, dev, st);
    }
    int ctas = 1;
    while (ctas < kLpMaxCluster && a.n * ctas * 2 <= places / 4 * 3 && vecs >= 256 * ctas * 2) ctas *= 2;
    return launch_logprobs<T, 256>(a, ctas, a.n, dev, st);   // one row a cluster
}

}  // namespace mw4

using namespace mw4;

extern "C" int moe_w4_token_logprobs(int dtype, int n, int vocab, const void* logits, int64_t row_stride,
                                     const int32_t* targets, int top, float* logprob, float* entropy,
                                     int32_t* top_index, float* top_logprob, void* workspace, size_t ws_bytes,
                                     cudaStream_t stream) {
    if (n < 0 || vocab < 1 || row_stride < 0 || top < 0 || top > vocab) return MOE_W4_ERR_INVALID;
    if (dtype != MOE_W4_TYPE_BF16 && dtype != MOE_W4_TYPE_FP16 && dtype != MOE_W4_TYPE_FP32) return MOE_W4_ERR_UNSUPPORTED;
    if (top > MOE_W4_MAX_TOP || vocab > MOE_W4_MAX_VOCAB) return MOE_W4_ERR_UNSUPPORTED;
    if (n == 0) return MOE_W4_OK;
    if (!logits || !targets != !logprob || (top && (!top_index || !top_logprob)) || (n > 1 && row_stride < vocab))
        return MOE_W4_ERR_INVALID;
    const size_t size = dtype == MOE_W4_TYPE_FP32 ? 4 : 2;
    if (misaligned(logits, size) || misaligned(targets, 4) || misaligned(logprob, 4) || misaligned(entropy, 4) ||
        misaligned(top_index, 4) || misaligned(top_logprob, 4))
        return MOE_W4_ERR_ALIGN;
    const int r = check_workspace(workspace, ws_bytes, MOE_W4_CTRL_BYTES);
    if (r) return r;
    const LogprobArgs a{logits, row_stride, n, vocab, top, targets, logprob, entropy, top_index, top_logprob,
                        static_cast<unsigned int*>(workspace)};
    return launched(dtype == MOE_W4_TYPE_BF16 ? launch_logprobs<__nv_bfloat16>(a, stream)
                    : dtype == MOE_W4_TYPE_FP16 ? launch_logprobs<__half>(a, stream) : launch_logprobs<float>(a, stream));
}
