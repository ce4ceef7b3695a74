// The paged key-value cache: writing new tokens (append) and cutting sequences
// to a budget by accumulated attention weight (evict).
#include <climits>

#include "serving.cuh"

namespace mw4 {

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
struct AppendArgs {
    KvView c;
    const uint16_t* k_new;
    const uint16_t* v_new;
    int64_t k_stride, v_stride;
    const int32_t* seq;
    const int32_t* slot;
    const int32_t* pos;
    float* weight;
    int32_t* track_pos;
    int64_t track_seq, track_head;
    int slots, n, chunks;   // chunks: 16-byte pieces of a head's row
    unsigned int* status;
};

constexpr int kAppendThreads = 256;

// One thread per 16-byte piece of a (token, head) row: it copies that piece of
// the key and of the value.  Latency bounds it: four trips to memory one after the
// other (sequence, index, page number, data; the data's address needs only the
// token's number, but it is asked for when the place is known to be good) and a
// store (16 tokens: 2.4 us, 4096 tokens of 2 heads of 256: 3.8 us for 17 MB, 65% of
// the copy rate).
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs a) {
    griddep_wait();
    griddep_launch_dependents();   // the attention that follows may start to launch
    const int64_t at = (int64_t)blockIdx.x * kAppendThreads + threadIdx.x;
    const int per_token = a.c.n_kv_heads * a.chunks;
    const int i = (int)(at / per_token);
    if (i >= a.n) return;
    const int in = (int)(at - (int64_t)i * per_token);
    const int h = in / a.chunks, piece = in - h * a.chunks;
    const int b = a.seq ? a.seq[i] : i;
    bool ok = (unsigned)b < (unsigned)a.c.n_seqs;
    int t = 0;
    if (ok) {
        t = a.slot ? a.slot[i] : a.c.lens[b] - 1;
        if (!a.slot && t == -1) return;   // an idle sequence
        ok = t >= 0 && (!a.weight || t < a.slots);
    }
    const int64_t off = ok ? kv_offset(a.c, b, t) : -1;
    if (off < 0) {
        if (in == 0) raise_status(a.status, MOE_W4_STATUS_BAD_INDEX);
        return;
    }
    const int64_t from = (int64_t)h * a.chunks * 8 + piece * 8, to = off + h * a.c.head_stride + piece * 8;
    const uint4 kx = *reinterpret_cast<const uint4*>(a.k_new + i * a.k_stride + from);
    const uint4 vx = *reinterpret_cast<const uint4*>(a.v_new + i * a.v_stride + from);
    *reinterpret_cast<uint4*>(const_cast<uint16_t*>(a.c.k) + to) = kx;
    *reinterpret_cast<uint4*>(const_cast<uint16_t*>(a.c.v) + to) = vx;
    if (a.weight && piece == 0) {
        const int64_t e = b * a.track_seq + h * a.track_head + t;
        a.weight[e] = 0.f;
        if (a.track_pos) a.track_pos[e] = a.pos ? a.pos[i] : t;
    }
}

// ---------------------------------------------------------------------------
// evict
// ---------------------------------------------------------------------------
// A row is a (sequence, head) and belongs to a cluster of 1 to 8 CTAs, each with
// a contiguous range of its tokens:
//   - the budget-th largest key T by two or three histogram passes over the
//     key's digits, the CTAs' histograms added up through distributed shared
//     memory;
//   - which tokens stay (ties at T by index, ranks from the CTAs before), and
//     two lists in ascending order: places below the budget that are dropped,
//     tokens past it that are kept (as many);
//   - the lists' pairs, shared out among the CTAs: keys, values, weight and
//     position of the token move into the place.
// A token moves from an index >= budget to one below it, so no place is both
// read and written and any order is right.
// Bytes bound it in principle (weights read once, moved rows read and written);
// the chain of barriers does where few tokens move: 16 sequences of 4112 tokens to
// 4096, 2 heads: 11.0 us.  4 sequences of up to 32,768 to 8192, 8 heads of 128:
// 28 us, of which the selection takes 17 and the moves 8.
struct EvictArgs {
    KvView c;
    const float* weight;
    const int32_t* pos;
    const int32_t* seen;
    float* weight_out;
    int32_t* pos_out;
    int32_t* lens_out;
    int64_t track_seq, track_head;
    int budget, sink, recent, max_len, key_room;
    int32_t* holes;          // [row][budget]
    int32_t* movers;         // [row][budget]
    int32_t* moved;          // [row] pairs in the lists, written for every row, or NULL: the selecting CTAs move them too
    unsigned int* heads_in;  // [n_seqs] heads that have read the length; zero between calls
    unsigned int* status;
};

constexpr int kEvictThreads = 1024, kEvictManyThreads = 256;
constexpr int kEvictManyTokens = 6144;           // four CTAs' keys fit into an SM
constexpr int kEvictMaxCluster = 8;
constexpr int kDigits = 3;                       // 11 + 11 + 10 bits of the key
constexpr int kHistBins = 2048;                  // two bins a thread
constexpr int kKeyRoom = 40 * 1024;              // keys that a CTA holds in shared memory
// Weights in flight of a thread: 5120 tokens a CTA at a time.  A cache kept at a
// budget is a little longer than it when it is cut, and budgets are powers of two
// (4112 to 4096 tokens: 12.0 us with 4, 11.0 with 5, 11.3 with 8).
constexpr int kKeyUnroll = 5;
constexpr int kEvictUnroll = 4;                  // row pieces in flight of a thread
// Tokens of a row that the selecting CTAs move at most (as many as the lengths
// allow); more go to a kernel of their own on every SM.  2048 tokens kept of 16 x 8
// rows of 128: 64 moved 10.0 us inline and 14.1 with the kernel, 128 moved 11.7 and
// 14.6; of 2 rows of 256: 128 moved 12.6 and 12.0, 512 moved 22.0 and 12.4.
constexpr int64_t kInlineMoves = 128;
constexpr int kMovePairs = 64;                   // tokens moved at a time by a CTA

struct alignas(16) EvictShared {
    int hist[kDigits][kHistBins];
    int groups[kDigits][32]; // sums of 64 bins
    int64_t from[kMovePairs], to[kMovePairs];
    int warp_sums[32];
    int holes, movers;       // of this CTA
    int bin, above, in_bin, n;
};

// Sum over the warps before this one of the warps' values (uniform in a warp).
MW4_DEV int warps_before(int v, int* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) warp_sums[warp] = v;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[lane] : 0);
}

// The order in which a row's tokens are kept, as a 32-bit key: 0xffffffff for
// one that is kept by its position, the order-preserving bits of its weight
// otherwise, 0 for NaN.  order_key of a number lies strictly between (of -inf
// it is 0x007fffff, of +inf 0xff800000).
MW4_DEV uint32_t evict_key(const EvictArgs& a, float w, int p, int64_t oldest_recent) {
    if (p < a.sink || p >= oldest_recent) return 0xffffffffu;
    return isnan(w) ? 0u : order_key(w + 0.f);   // -0 + 0 = +0
}

// Moves the tokens of `count` <= kMovePairs pairs of a row's lists: one thread
// looks a pair's places up and moves its weight and position, then rows of LR
// lanes copy keys and values, kEvictUnroll pieces of a thread in flight.
template <int LR, int THREADS>
MW4_DEV void move_pairs(const EvictArgs& a, int b, int h, int64_t row, const int32_t* holes, const int32_t* movers, int count,
                        int64_t* sh_from, int64_t* sh_to) {
    const int tid = threadIdx.x;
    if (tid < count) {
        const int src = movers[tid], dst = holes[tid];
        const float w = a.weight[row + src];
        const int p = a.pos[row + src];
        int64_t from = kv_offset(a.c, b, src);
        const int64_t to = kv_offset(a.c, b, dst);
        if (from < 0 || to < 0) {
            raise_status(a.status, MOE_W4_STATUS_BAD_INDEX);
            from = -1;   // the whole move is left out: the place keeps its own token's weight and position too
        } else {
            a.weight_out[row + dst] = w;
            a.pos_out[row + dst] = p;
        }
        sh_from[tid] = from;
        sh_to[tid] = to;
    }
    __syncthreads();
    // keys of pair i are copy 2 i, its values copy 2 i + 1
    constexpr int PER = THREADS / LR;            // rows copied at a time
    const int64_t in_row = h * a.c.head_stride + tid % LR * 8;
    for (int x0 = tid / LR; x0 < 2 * count; x0 += PER * kEvictUnroll) {
        uint4 v[kEvictUnroll];
#pragma unroll
        for (int k = 0; k < kEvictUnroll; ++k) {
            const int x = x0 + k * PER;
            if (x < 2 * count && sh_from[x >> 1] >= 0)
                v[k] = *reinterpret_cast<const uint4*>((x & 1 ? a.c.v : a.c.k) + sh_from[x >> 1] + in_row);
        }
#pragma unroll
        for (int k = 0; k < kEvictUnroll; ++k) {
            const int x = x0 + k * PER;
            if (x < 2 * count && sh_from[x >> 1] >= 0)
                *reinterpret_cast<uint4*>(const_cast<uint16_t*>(x & 1 ? a.c.v : a.c.k) + sh_to[x >> 1] + in_row) = v[k];
        }
    }
    __syncthreads();
}

template <int LR, int NT>   // LR: lanes of a row of keys, head_dim / 8
__global__ void __launch_bounds__(NT, 1024 / NT) kv_evict_kernel(const EvictArgs a) {
    constexpr int WARPS = NT / 32;
    extern __shared__ uint32_t keys[];
    __shared__ EvictShared sh;
    griddep_wait();
    griddep_launch_dependents();
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank(), r = blockIdx.x / ctas;
    const int b = r / a.c.n_kv_heads, h = r % a.c.n_kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // one reading of the length for the whole cluster: its CTAs have to take the
    // same turns, whatever happens to the length meanwhile
    if (rank == 0 && tid == 0) {
        const int x = a.c.lens[b];
        if (x < 0 || x > a.max_len) raise_status(a.status, MOE_W4_STATUS_BAD_INDEX);
        sh.n = x < 0 ? 0 : min(x, a.max_len);
    }
    for (int i = tid; i < kDigits * kHistBins / 4; i += NT) reinterpret_cast<int4*>(sh.hist)[i] = make_int4(0, 0, 0, 0);
    auto sync = [&]() {
        if (ctas > 1) cluster_sync();
        else __syncthreads();
    };
    sync();
    const int n = ld_cluster(&sh.n, 0);
    const int64_t row = b * a.track_seq + h * a.track_head;
    const bool copies = a.weight_out != a.weight || a.pos_out != a.pos;
    // this CTA's tokens
    const int span = ((n + ctas - 1) / ctas + 31) & ~31;
    const int lo = min(n, rank * span), hi = min(n, lo + span);
    const bool cut = n > a.budget;
    const int64_t oldest_recent = (int64_t)a.seen[b] - a.recent;
    const bool held = span <= a.key_room;
    // the digit of a warp's keys where their higher bits are T's
    uint32_t T = 0, mask = 0;
    auto count = [&](int* hist, int shift, int bins, uint32_t x, bool in) {
        in = in && (x & mask) == T;
        const int bin = (x >> shift) & (bins - 1);
        // a warp whose tokens all fall into one bin adds once
        const uint32_t live = __ballot_sync(0xffffffffu, in);
        if (!live) return;
        const int first = __shfl_sync(0xffffffffu, bin, __ffs(live) - 1);
        if (__all_sync(0xffffffffu, !in || bin == first)) {
            if (lane == 0) atomicAdd(&hist[first], __popc(live));
        } else if (in) {
            atomicAdd(&hist[bin], 1);
        }
    };
    // Keys, counted by their first digit, and where the outputs are arrays of their
    // own, every token's weight and position at its old place: the tokens that move
    // are written after a barrier.
    if (cut || copies) {
        for (int j0 = lo + tid; j0 - tid < hi; j0 += NT * kKeyUnroll) {
            float w[kKeyUnroll];
            int p[kKeyUnroll];
#pragma unroll
            for (int k = 0; k < kKeyUnroll; ++k) {
                const int j = j0 + k * NT;
                w[k] = j < hi ? a.weight[row + j] : 0.f;
                p[k] = j < hi ? a.pos[row + j] : 0;
            }
#pragma unroll
            for (int k = 0; k < kKeyUnroll; ++k) {
                const int j = j0 + k * NT;
                if (cut) {
                    const uint32_t x = evict_key(a, w[k], p[k], oldest_recent);
                    if (held && j < hi) keys[j - lo] = x;
                    count(sh.hist[0], 21, kHistBins, x, j < hi);
                }
                if (copies && j < hi && j < a.budget) {
                    a.weight_out[row + j] = w[k];
                    a.pos_out[row + j] = p[k];
                }
            }
        }
    }
    auto key = [&](int j) { return held ? keys[j - lo] : evict_key(a, a.weight[row + j], a.pos[row + j], oldest_recent); };

    // T, the leading digits of the budget-th largest key: `above` keys have larger
    // ones, at least `budget` larger or the same.  It is done when exactly `budget`
    // have, as they mostly do after two digits, or when T is the whole key (ties).
    int above = 0, last = 0, last_bin = 0;
#pragma unroll 1
    for (int d = 0; cut; ++d) {
        const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bins = d == 2 ? 1024 : 2048;
        int* hist = sh.hist[d];
        if (d)
            for (int j0 = lo; j0 < hi; j0 += NT) {
                const int j = j0 + tid;
                count(hist, shift, bins, j < hi ? key(j) : 0, j < hi);
            }
        __syncthreads();
#pragma unroll
        for (int g = warp; g < 32; g += WARPS) {
            const int2 two = *reinterpret_cast<const int2*>(&hist[g * 64 + 2 * lane]);
            const int group = __reduce_add_sync(0xffffffffu, two.x + two.y);
            if (lane == 0) sh.groups[d][g] = group;
        }
        sync();
        if (warp == 0) {
            // the group of 64 bins with T's digit, counted from the top, then the bin:
            // two short trips to the other CTAs instead of all of their bins
            int at = 31, before = above;
#pragma unroll
            for (int level = 0; level < 2; ++level) {
                int2 part[kEvictMaxCluster];
#pragma unroll
                for (int q = 0; q < kEvictMaxCluster; ++q) {   // all asked for before the first is added
                    part[q] = make_int2(0, 0);
                    if (q < ctas) {
                        if (level == 0) part[q].y = ld_cluster(&sh.groups[d][31 - lane], q);
                        else part[q] = ld_cluster2(&hist[at * 64 + 62 - 2 * lane], q);
                    }
                }
                int y = 0, x = 0;   // this lane's group, or its two bins: y the higher one
#pragma unroll
                for (int q = 0; q < kEvictMaxCluster; ++q) {
                    y += part[q].y;
                    x += part[q].x;
                }
                int incl = y + x;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int o = __shfl_up_sync(0xffffffffu, incl, off);
                    if (lane >= off) incl += o;
                }
                const int mine = before + incl - y - x;   // keys above
                const int hit = __ffs(__ballot_sync(0xffffffffu, before + incl >= a.budget)) - 1 & 31;
                if (level == 0) {
                    at = 31 - hit;
                    before = __shfl_sync(0xffffffffu, mine, hit);
                } else if (lane == hit) {
                    const bool upper = mine + y >= a.budget;
                    sh.bin = at * 64 + 63 - 2 * lane - (upper ? 0 : 1);
                    sh.above = upper ? mine : mine + y;
                    sh.in_bin = upper ? y : x;
                }
            }
        }
        __syncthreads();
        last = d;
        last_bin = sh.bin;
        T |= (uint32_t)last_bin << shift;
        mask |= (uint32_t)(bins - 1) << shift;
        above = sh.above;
        if (d == kDigits - 1 || above + sh.in_bin == a.budget) break;
    }
    if (rank == 0 && tid == 0 && atomicAdd(&a.heads_in[b], 1u) == (unsigned)a.c.n_kv_heads - 1) {
        a.heads_in[b] = 0;
        a.lens_out[b] = min(n, a.budget);
    }
    if (!cut) {
        // Nothing moves.  The word has to say so: it holds what an earlier call, of any
        // operator, left in the workspace.
        if (a.moved && rank == 0 && tid == 0) a.moved[r] = 0;
        sync();   // CTA 0's memory stays until its length has been read
        return;
    }

    // Of the keys at T the first `ties` of the row stay.  A warp has a contiguous
    // range of tokens and counts, below and past the budget, those above T and those
    // at T; the places dropped and the tokens that move follow.
    const int ties = a.budget - above;
    const int wspan = (span / 32 + WARPS - 1) / WARPS * 32;
    const int j_lo = min(hi, lo + warp * wspan), j_hi = min(hi, j_lo + wspan), j_cut = min(max(a.budget, j_lo), j_hi);
    int above_in = 0, above_past = 0, at_in = 0, at_past = 0;
    for (int j = j_lo + lane; j < j_hi; j += 32) {
        const uint32_t x = key(j) & mask;
        above_in += x > T && j < a.budget;
        above_past += x > T && j >= a.budget;
        at_in += x == T && j < a.budget;
        at_past += x == T && j >= a.budget;
    }
    above_in = __reduce_add_sync(0xffffffffu, above_in);
    above_past = __reduce_add_sync(0xffffffffu, above_past);
    at_in = __reduce_add_sync(0xffffffffu, at_in);
    at_past = __reduce_add_sync(0xffffffffu, at_past);
    int e = lane < rank ? ld_cluster(&sh.hist[last][last_bin], lane) : 0;
    e = __reduce_add_sync(0xffffffffu, e) + warps_before(at_in + at_past, sh.warp_sums);
    const int stay = min(max(ties - e, 0), at_in + at_past), stay_in = min(stay, at_in);
    const int holes = j_cut - j_lo - above_in - stay_in, moved = above_past + stay - stay_in;
    int hole_at = warps_before(holes, sh.warp_sums), move_at = warps_before(moved, sh.warp_sums);
    if (warp == WARPS - 1 && lane == 0) {
        sh.holes = hole_at + holes;
        sh.movers = move_at + moved;
    }
    sync();
    const int all_holes = lane < ctas ? ld_cluster(&sh.holes, lane) : 0, all_moved = lane < ctas ? ld_cluster(&sh.movers, lane) : 0;
    hole_at += __reduce_add_sync(0xffffffffu, lane < rank ? all_holes : 0);
    move_at += __reduce_add_sync(0xffffffffu, lane < rank ? all_moved : 0);
    const int total = __reduce_add_sync(0xffffffffu, all_moved);
    int32_t* hole_list = a.holes + (int64_t)r * a.budget;
    int32_t* move_list = a.movers + (int64_t)r * a.budget;
    if (holes | moved)
        for (int j0 = j_lo; j0 < j_hi; j0 += 32) {
            const int j = j0 + lane;
            const uint32_t x = j < j_hi ? key(j) & mask : 0;
            const bool at = j < j_hi && x == T;
            const uint32_t before = (1u << lane) - 1, ats = __ballot_sync(0xffffffffu, at);
            const bool keep = j < j_hi && (x > T || (at && e + __popc(ats & before) < ties));
            e += __popc(ats);
            const bool hole = j < j_hi && !keep && j < a.budget, mover = keep && j >= a.budget;
            const uint32_t hs = __ballot_sync(0xffffffffu, hole), ms = __ballot_sync(0xffffffffu, mover);
            if (mover) move_list[move_at + __popc(ms & before)] = j;
            if (hole) hole_list[hole_at + __popc(hs & before)] = j;
            hole_at += __popc(hs);
            move_at += __popc(ms);
        }
    sync();   // the lists are written, and nobody reads this CTA's memory any more

    if (a.moved) {   // the moves are another kernel's
        if (rank == 0 && tid == 0) a.moved[r] = total;
        return;
    }
    const int share = (total + ctas - 1) / ctas, m_hi = min(total, (rank + 1) * share);
    for (int m0 = rank * share; m0 < m_hi; m0 += kMovePairs)
        move_pairs<LR, NT>(a, b, h, row, hole_list + m0, move_list + m0, min(kMovePairs, m_hi - m0), sh.from, sh.to);
}

// One CTA for kMovePairs pairs of a row's lists.
constexpr int kMoveThreads = 256;
template <int LR>
__global__ void __launch_bounds__(kMoveThreads) kv_evict_move_kernel(const EvictArgs a) {
    __shared__ int64_t from[kMovePairs], to[kMovePairs];
    griddep_wait();
    const int r = blockIdx.y, m0 = blockIdx.x * kMovePairs, count = min(kMovePairs, a.moved[r] - m0);
    if (count <= 0) return;
    const int b = r / a.c.n_kv_heads, h = r % a.c.n_kv_heads;
    const int64_t list = (int64_t)r * a.budget + m0;
    move_pairs<LR, kMoveThreads>(a, b, h, b * a.track_seq + h * a.track_head, a.holes + list, a.movers + list, count, from, to);
}

static size_t evict_rows(const moe_w4_kv_cache& c) { return (size_t)c.n_seqs * c.n_kv_heads; }
static size_t evict_list_bytes(const moe_w4_kv_cache& c, int budget) {
    return round_up(evict_rows(c) * (size_t)budget * 4, 256);
}
static size_t evict_bytes(const moe_w4_kv_cache& c, int budget) {
    return MOE_W4_CTRL_BYTES + kSyncBytes + 2 * evict_list_bytes(c, budget) + round_up(evict_rows(c) * 4, 256);
}

template <int LR>
static cudaError_t launch_evict(const EvictArgs& a, int rows, cudaStream_t st) {
    static std::atomic<unsigned> ready[2];
    int dev = 0;
    const int sms = sm_count(&dev);
    if (sms < 1) return cudaErrorInvalidDevice;
    // CTAs of a row: one up to 8192 tokens, where the barriers of a cluster cost more
    // than they save (16 x 4112 to 4096: 11.0 us, with two 12.7), then one per 4096,
    // up to 8 (4 x 16384 to 8192: 22.9 us; one per 8192: 26.6; one alone: 31.4), as
    // long as all are resident at once: 32 rows of 65,536 tokens took 38.7 us with 8
    // a row, in turns, 19.9 with 4; 32 rows of 32,768 to 8192 70 and 53 (but 24.7 and
    // 28.2 where only 8 of them have anything to cut).  Clusters of 8 do not reach
    // every SM (16 rows: 24.4 us, with 4 a row 19.5).
    int ctas = 1;
    while (ctas < kEvictMaxCluster && a.max_len > 8192 && a.max_len > ctas * 4096 &&
           rows * ctas * 2 <= (ctas * 2 < kEvictMaxCluster ? sms : sms / 4 * 3))
        ctas *= 2;
    // One CTA a row and more rows than SMs: smaller CTAs, four to an SM (512 rows of
    // 1000 tokens to 500: 35.6 -> 19.9 us; of 4112 to 4096: 35.2 -> 20.8).
    const bool many = ctas == 1 && rows > sms && a.max_len <= kEvictManyTokens;
    auto kern = many ? kv_evict_kernel<LR, kEvictManyThreads> : kv_evict_kernel<LR, kEvictThreads>;
    const cudaError_t e = allow_smem((const void*)kern, kKeyRoom * 4, ready[many], dev);
    if (e != cudaSuccess) return e;
    EvictArgs b = a;
    const int span = (int)((((int64_t)a.max_len + ctas - 1) / ctas + 31) & ~(int64_t)31);
    b.key_room = span < kKeyRoom ? span : kKeyRoom;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(rows * ctas));
    cfg.blockDim = dim3(many ? kEvictManyThreads : kEvictThreads);
    cfg.dynamicSmemBytes = (size_t)b.key_room * 4;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e2 = cudaLaunchKernelEx(&cfg, kern, b);
    if (e2 != cudaSuccess || !b.moved) return e2;
    const int most = a.budget < a.max_len - a.budget ? a.budget : a.max_len - a.budget;
    return launch_pdl(true, kv_evict_move_kernel<LR>, dim3((unsigned)((most + kMovePairs - 1) / kMovePairs), (unsigned)rows),
                      dim3(kMoveThreads), 0, st, b);
}

}  // namespace mw4

using namespace mw4;

extern "C" {

int moe_w4_kv_append(const moe_w4_kv_cache* c, const moe_w4_kv_track* track, int n, const void* k, int64_t k_stride,
                     const void* v, int64_t v_stride, const int32_t* seq, const int32_t* slot, const int32_t* pos,
                     void* workspace, size_t ws_bytes, cudaStream_t stream) {
    int r = check_cache(c, slot == nullptr);
    if (r) return r;
    if (n < 0 || k_stride < 0 || v_stride < 0) return MOE_W4_ERR_INVALID;
    if (n == 0 || c->n_seqs == 0) return MOE_W4_OK;
    if (!k || !v || (!seq && n != c->n_seqs)) return MOE_W4_ERR_INVALID;
    if (track && (r = check_track(track, false))) return r;
    if (misaligned(k, 16) || misaligned(v, 16) || k_stride % 8 || v_stride % 8 || misaligned(seq, 4) ||
        misaligned(slot, 4) || misaligned(pos, 4))
        return MOE_W4_ERR_ALIGN;
    if ((r = check_workspace(workspace, ws_bytes, MOE_W4_CTRL_BYTES))) return r;
    AppendArgs a{};
    a.c = kv_view(*c);
    a.k_new = static_cast<const uint16_t*>(k);
    a.v_new = static_cast<const uint16_t*>(v);
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.seq = seq;
    a.slot = slot;
    a.pos = pos;
    if (track) {
        a.weight = track->weight;
        a.track_pos = track->pos;
        a.track_seq = track->seq_stride;
        a.track_head = track->head_stride;
        a.slots = track->slots;
    }
    a.n = n;
    a.chunks = c->head_dim / 8;
    a.status = static_cast<unsigned int*>(workspace);
    const int64_t threads = (int64_t)n * c->n_kv_heads * a.chunks;
    const int64_t blocks = (threads + kAppendThreads - 1) / kAppendThreads;
    if (blocks > INT_MAX) return MOE_W4_ERR_UNSUPPORTED;
    return launched(launch_pdl(true, kv_append_kernel, dim3((unsigned)blocks), dim3(kAppendThreads), 0, stream, a));
}

size_t moe_w4_evict_workspace_size(const moe_w4_kv_cache* c, int budget, int max_len) {
    if (check_cache(c, false) != MOE_W4_OK || budget < 1 || max_len < 0) return 0;
    return evict_bytes(*c, budget < max_len ? budget : max_len < 1 ? 1 : max_len);
}

int moe_w4_kv_evict(const moe_w4_kv_cache* c, const moe_w4_kv_track* track, const int32_t* seen, int budget, int sink,
                    int recent, int max_len, int32_t* lens_out, float* weight_out, int32_t* pos_out, void* workspace,
                    size_t ws_bytes, cudaStream_t stream) {
    int r = check_cache(c, true);
    if (r) return r;
    if (!track || budget < 1 || sink < 0 || recent < 0 || (int64_t)sink + recent > budget || max_len < 0 ||
        (int64_t)max_len > (int64_t)c->pages_per_seq * c->page_size)
        return MOE_W4_ERR_INVALID;
    if (c->n_seqs == 0) return MOE_W4_OK;
    if ((r = check_track(track, true))) return r;
    if (!seen || !lens_out || !weight_out || !pos_out || max_len > track->slots) return MOE_W4_ERR_INVALID;
    if (misaligned(seen, 4) || misaligned(lens_out, 4) || misaligned(weight_out, 4) || misaligned(pos_out, 4))
        return MOE_W4_ERR_ALIGN;
    // places that a call can fill; a longer budget than any sequence cuts none
    const int places = budget < max_len ? budget : max_len < 1 ? 1 : max_len;
    if ((r = check_workspace(workspace, ws_bytes, evict_bytes(*c, places)))) return r;
    const size_t rows = evict_rows(*c);
    if (rows > 65535) return MOE_W4_ERR_UNSUPPORTED;
    EvictArgs a{};
    a.c = kv_view(*c);
    a.weight = track->weight;
    a.pos = track->pos;
    a.seen = seen;
    a.weight_out = weight_out;
    a.pos_out = pos_out;
    a.lens_out = lens_out;
    a.track_seq = track->seq_stride;
    a.track_head = track->head_stride;
    a.budget = places;
    a.sink = sink;
    a.recent = recent;
    a.max_len = max_len;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.heads_in = reinterpret_cast<unsigned int*>(ws + MOE_W4_CTRL_BYTES + kRowSyncBytes);
    a.holes = reinterpret_cast<int32_t*>(ws + MOE_W4_CTRL_BYTES + kSyncBytes);
    a.movers = reinterpret_cast<int32_t*>(ws + MOE_W4_CTRL_BYTES + kSyncBytes + evict_list_bytes(*c, places));
    a.status = reinterpret_cast<unsigned int*>(ws);
    const int64_t most = places < max_len - places ? places : max_len - places;
    if (most > kInlineMoves)
        a.moved = reinterpret_cast<int32_t*>(ws + MOE_W4_CTRL_BYTES + kSyncBytes + 2 * evict_list_bytes(*c, places));
    const cudaError_t e = c->head_dim == 64 ? launch_evict<8>(a, (int)rows, stream)
                          : c->head_dim == 128 ? launch_evict<16>(a, (int)rows, stream) : launch_evict<32>(a, (int)rows, stream);
    return launched(e);
}

}  // extern "C"
