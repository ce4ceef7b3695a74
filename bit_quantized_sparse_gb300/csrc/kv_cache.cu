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
// the key and of the value.
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs a) {
    griddep_wait();
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
struct EvictArgs {
    KvView c;
    const float* weight;
    const int32_t* pos;
    const int32_t* seen;
    float* weight_out;
    int32_t* pos_out;
    int32_t* lens_out;
    int64_t track_seq, track_head;
    int budget, sink, recent, max_len, key_room, chunks;
    int32_t* src;      // [row][budget] where the token of each place comes from
    int32_t* movers;   // [row][budget] kept tokens past the budget, ascending
    int32_t* kept;     // [row] tokens of the row after the cut
    unsigned int* status;
};

constexpr int kSelectThreads = 1024;
constexpr int kDigits = 3;                       // 11 + 11 + 10 bits of the key
constexpr int kHistBins = 2048;
constexpr int kKeyRoom = 48 * 1024;              // keys held in shared memory
constexpr int kMoveThreads = 256;

MW4_DEV int block_sum_1024(int v, int* warp_sums) {   // every thread gets the sum
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if (lane == 0) warp_sums[warp] = v;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, warp_sums[lane]);
}

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
MW4_DEV uint32_t evict_key(const EvictArgs& a, int64_t row, int j, int64_t oldest_recent) {
    const int p = a.pos[row + j];
    const float w = a.weight[row + j];
    if (p < a.sink || p >= oldest_recent) return 0xffffffffu;
    return isnan(w) ? 0u : order_key(w + 0.f);   // -0 + 0 = +0
}

// One CTA per (sequence, head): the budget-th largest key by three histogram
// passes over the key's digits, then the places it leaves and the tokens that
// fill them, in ascending order of both.
__global__ void __launch_bounds__(kSelectThreads) kv_evict_select_kernel(const EvictArgs a) {
    extern __shared__ uint32_t keys[];
    __shared__ int hist[kHistBins];
    __shared__ int warp_sums[32];
    __shared__ uint32_t sh_digit;
    __shared__ int sh_above;
    griddep_wait();
    const int b = blockIdx.x / a.c.n_kv_heads, h = blockIdx.x % a.c.n_kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int n = a.c.lens[b];
    if (n < 0 || n > a.max_len) {
        if (tid == 0) raise_status(a.status, MOE_W4_STATUS_BAD_INDEX);
        n = n < 0 ? 0 : a.max_len;
    }
    int32_t* src = a.src + (int64_t)blockIdx.x * a.budget;
    int32_t* movers = a.movers + (int64_t)blockIdx.x * a.budget;
    if (tid == 0) a.kept[blockIdx.x] = min(n, a.budget);
    if (n <= a.budget) {
        for (int j = tid; j < n; j += kSelectThreads) src[j] = j;
        return;
    }
    const int64_t row = b * a.track_seq + h * a.track_head;
    const int64_t oldest_recent = (int64_t)a.seen[b] - a.recent;
    const bool held = n <= a.key_room;
    if (held)
        for (int j = tid; j < n; j += kSelectThreads) keys[j] = evict_key(a, row, j, oldest_recent);
    auto key = [&](int j) { return held ? keys[j] : evict_key(a, row, j, oldest_recent); };

    // the largest key T with at least `budget` keys >= T; `above` keys are > T
    uint32_t prefix = 0, mask = 0;
    int above = 0;
    constexpr int shift_of[kDigits] = {21, 10, 0};
    constexpr int bits_of[kDigits] = {11, 11, 10};
#pragma unroll
    for (int d = 0; d < kDigits; ++d) {
        const int shift = shift_of[d], bins = 1 << bits_of[d];
        for (int i = tid; i < kHistBins; i += kSelectThreads) hist[i] = 0;
        __syncthreads();
        for (int j0 = 0; j0 < n; j0 += kSelectThreads) {
            const int j = j0 + tid;
            const uint32_t x = j < n ? key(j) : 0;
            const bool in = j < n && (x & mask) == prefix;
            const int bin = (x >> shift) & (bins - 1);
            // a warp whose tokens all fall into one bin adds once
            const uint32_t live = __ballot_sync(0xffffffffu, in);
            if (!live) continue;
            const int first = __shfl_sync(0xffffffffu, bin, __ffs(live) - 1);
            if (__all_sync(0xffffffffu, !in || bin == first)) {
                if (lane == 0) atomicAdd(&hist[first], __popc(live));
            } else if (in) {
                atomicAdd(&hist[bin], 1);
            }
        }
        __syncthreads();
        // thread t owns bins 2t and 2t + 1, counted from the top
        const int hi = hist[kHistBins - 1 - 2 * tid], lo = hist[kHistBins - 2 - 2 * tid];
        int incl = hi + lo;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        const int base = warps_before(__shfl_sync(0xffffffffu, incl, 31), warp_sums);
        const int before_hi = above + base + incl - hi - lo, before_lo = before_hi + hi;
        if (before_hi < a.budget && before_lo >= a.budget) { sh_digit = kHistBins - 1 - 2 * tid; sh_above = before_hi; }
        if (before_lo < a.budget && before_lo + lo >= a.budget) { sh_digit = kHistBins - 2 - 2 * tid; sh_above = before_lo; }
        __syncthreads();
        prefix |= sh_digit << shift;
        mask |= (uint32_t)(bins - 1) << shift;
        above = sh_above;
        __syncthreads();
    }
    const uint32_t T = prefix;
    const int ties = a.budget - above;   // of the keys equal to T the first `ties` stay

    // each warp owns a contiguous range of tokens, so that ranks follow the index
    const int span = (n + 32 * 32 - 1) / (32 * 32) * 32;
    const int j_lo = warp * span, j_hi = min(n, j_lo + span);
    int eq = 0;
    for (int j = j_lo + lane; j < j_hi; j += 32) eq += key(j) == T;
    eq = __reduce_add_sync(0xffffffffu, eq);
    const int eq_base = warps_before(eq, warp_sums);
    int holes = 0, moved = 0;
    for (int pass = 0; pass < 2; ++pass) {   // counts, then places
        int e = eq_base, hole_at = 0, move_at = 0;
        if (pass == 1) {
            hole_at = warps_before(holes, warp_sums);
            move_at = warps_before(moved, warp_sums);
        }
        for (int j0 = j_lo; j0 < j_hi; j0 += 32) {
            const int j = j0 + lane;
            const uint32_t x = j < j_hi ? key(j) : 0;
            const bool is_eq = j < j_hi && x == T;
            const uint32_t before = (1u << lane) - 1;
            const uint32_t eqs = __ballot_sync(0xffffffffu, is_eq);
            const bool keep = j < j_hi && (x > T || (is_eq && e + __popc(eqs & before) < ties));
            e += __popc(eqs);
            const bool hole = j < j_hi && !keep && j < a.budget, mover = keep && j >= a.budget;
            const uint32_t hs = __ballot_sync(0xffffffffu, hole), ms = __ballot_sync(0xffffffffu, mover);
            if (pass == 0) {
                holes += __popc(hs);
                moved += __popc(ms);
            } else {
                if (mover) movers[move_at + __popc(ms & before)] = j;
                // a hole notes its rank (negative) until the movers are known
                if (j < j_hi && j < a.budget) src[j] = hole ? -1 - (hole_at + __popc(hs & before)) : j;
                hole_at += __popc(hs);
                move_at += __popc(ms);
            }
        }
    }
    __syncthreads();
    for (int j = tid; j < a.budget; j += kSelectThreads) {
        const int s = src[j];
        if (s < 0) src[j] = movers[-1 - s];
    }
}

// One warp per 32 places of a row: their weights and positions, then the rows
// of keys and values that move.  A token moves from an index >= budget to one
// below it, so no place is both read and written and any order is right.
template <int LR>   // lanes of a row: head_dim / 8
__global__ void __launch_bounds__(kMoveThreads) kv_evict_move_kernel(const EvictArgs a) {
    __shared__ int2 list[kMoveThreads / 32][32];
    griddep_wait();
    const int r = blockIdx.y;
    const int b = r / a.c.n_kv_heads, h = r % a.c.n_kv_heads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kept = a.kept[r];
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) a.lens_out[b] = kept;
    const int j = blockIdx.x * kMoveThreads + threadIdx.x;
    int s = j;
    if (j < kept) {
        s = a.src[(int64_t)r * a.budget + j];
        const int64_t row = b * a.track_seq + h * a.track_head;
        const float w = a.weight[row + s];
        const int p = a.pos[row + s];
        a.weight_out[row + j] = w;
        a.pos_out[row + j] = p;
    }
    const bool moves = j < kept && s != j;
    const uint32_t ms = __ballot_sync(0xffffffffu, moves);
    if (moves) list[warp][__popc(ms & ((1u << lane) - 1))] = make_int2(s, j);
    __syncwarp();
    const int items = 2 * __popc(ms);   // a key row and a value row for each move
    constexpr int PER = 32 / LR;
    const int piece = lane % LR;
    for (int it = lane / LR; it < items; it += PER) {
        const int2 m = list[warp][it >> 1];
        const int64_t from = kv_offset(a.c, b, m.x), to = kv_offset(a.c, b, m.y);
        if (from < 0 || to < 0) {
            if (piece == 0) raise_status(a.status, MOE_W4_STATUS_BAD_INDEX);
            continue;
        }
        uint16_t* base = const_cast<uint16_t*>(it & 1 ? a.c.v : a.c.k) + h * a.c.head_stride + piece * 8;
        *reinterpret_cast<uint4*>(base + to) = *reinterpret_cast<const uint4*>(base + from);
    }
}

static size_t evict_rows(const moe_w4_kv_cache& c) { return (size_t)c.n_seqs * c.n_kv_heads; }
static size_t evict_list_bytes(const moe_w4_kv_cache& c, int budget) {
    return round_up(evict_rows(c) * (size_t)budget * 4, 256);
}
static size_t evict_bytes(const moe_w4_kv_cache& c, int budget) {
    return MOE_W4_CTRL_BYTES + kSyncBytes + 2 * evict_list_bytes(c, budget) + round_up(evict_rows(c) * 4, 256);
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
    a.key_room = max_len < kKeyRoom ? max_len : kKeyRoom;
    a.chunks = c->head_dim / 8;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const size_t list = evict_list_bytes(*c, places);
    a.src = reinterpret_cast<int32_t*>(ws + MOE_W4_CTRL_BYTES + kSyncBytes);
    a.movers = reinterpret_cast<int32_t*>(ws + MOE_W4_CTRL_BYTES + kSyncBytes + list);
    a.kept = reinterpret_cast<int32_t*>(ws + MOE_W4_CTRL_BYTES + kSyncBytes + 2 * list);
    a.status = reinterpret_cast<unsigned int*>(ws);
    const size_t smem = (size_t)a.key_room * 4;
    static std::atomic<unsigned> ready;
    int dev = 0;
    if (sm_count(&dev) < 1) return MOE_W4_ERR_LAUNCH;
    cudaError_t e = allow_smem((const void*)kv_evict_select_kernel, kKeyRoom * 4, ready, dev);
    if (e == cudaSuccess)
        e = launch_pdl(true, kv_evict_select_kernel, dim3((unsigned)rows), dim3(kSelectThreads), smem, stream, a);
    if (e == cudaSuccess) {
        auto kern = c->head_dim == 64 ? kv_evict_move_kernel<8>
                    : c->head_dim == 128 ? kv_evict_move_kernel<16> : kv_evict_move_kernel<32>;
        e = launch_pdl(true, kern, dim3((unsigned)((places + kMoveThreads - 1) / kMoveThreads), (unsigned)rows),
                       dim3(kMoveThreads), 0, stream, a);
    }
    return launched(e);
}

}  // extern "C"
