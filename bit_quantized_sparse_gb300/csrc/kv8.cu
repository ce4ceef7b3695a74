// The paged cache of 8-bit codes: writing tokens (append) and reading them back
// (also from a cache of 16-bit values).
#include "kv8.cuh"

namespace mw4 {

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
// A block of a head (up to 128 tokens) has one scale, so its new tokens are one piece of
// work: the largest magnitude, the scale, the codes, and they stay in registers
// between the one read and the one write.  The call's rows name sequences and
// indexes, in any order of blocks; a row that begins a run of consecutive indexes
// within a block leads it, and who finds it does the whole run.
//
// Bytes bound it (2 read and 1 written per value); for few rows the trips one
// after the other do: indexes, then page numbers and rows together, the scale of a
// block already begun, the store.  Three kernels by the block's tokens: 1, where rows
// have nothing to do with one another; to 16, which a warp holds, with other runs beside
// it; and to 128, whose runs of many rows take several warps.
//
// In us: 4096 tokens of 2 heads of 256, blocks of 1, 16, 64 and 128: 4.6, 4.4, 5.8 and 6.0
// for 12.6 MB; 11,963 of 8 heads of 64, blocks of 1, 2, 16 and 64: 10.9, 11.9, 10.3 and 14.7
// for 37 MB; 512 of 512 sequences, 8 heads of 128, blocks of 1, 16 and 64: 2.4, 3.0 and 3.5;
// 16 of 2 of 256: 2.2.  With a warp for each run or a CTA for each long block, one after
// the other: 11,963 in blocks of 1, 2 and 16 87.7, 46.7 and 11.2; 512 in blocks of 16 and
// 64 7.9 and 37.9.
struct Append8Args {
    KvView c;
    Scales s;
    const uint16_t* k_new;
    const uint16_t* v_new;
    int64_t k_stride, v_stride;
    const int32_t* seq;
    const int32_t* slot;
    int n, window, windows;   // rows; of a window; windows
    unsigned int* status;
    unsigned int* disorder;   // debug builds: not 0 where the rows' order is wrong
};

constexpr int kSingleThreads = 256, kRowsThreads = 128, kLongThreads = 256;
constexpr int kRows = 16, kRowsShift = 4;          // rows that a warp holds at a time: the largest block of its own
constexpr int kWindows = 6;                        // windows of a head's keys or values for each SM
constexpr int rows_warps(int dim) { return dim == 64 ? 32 : dim == 128 ? 24 : 16; }   // of an SM: registers hold their rows
constexpr int long_ctas(int dim) { return dim == 64 ? 4 : dim == 128 ? 3 : 2; }
constexpr int kLowest = -100, kHighest = 119;   // exponents of scales

template <typename T> constexpr uint32_t kInfinite = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;

// The bits of the largest finite magnitude of N times 8 values: they order like numbers,
// and those of infinities and NaN lie above.
template <typename T, int N>
MW4_DEV uint32_t largest_finite(const uint4 (&x)[N], int n) {
    uint32_t all = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (j >= n) break;
        all = __vmaxu2(__vmaxu2(__vmaxu2(all, x[j].x & 0x7fff7fffu), x[j].y & 0x7fff7fffu),
                       __vmaxu2(x[j].z & 0x7fff7fffu, x[j].w & 0x7fff7fffu));
    }
    const uint32_t top = max(all & 0xffffu, all >> 16);
    if (top < kInfinite<T>) return top;
    all = 0;                                               // rare: once more without them
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (j >= n) break;
        const uint32_t u[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t m = u[i] & 0x7fff7fffu;
            all = __vmaxu2(all, m & ~__vcmpgeu2(m, kInfinite<T> * 0x10001u));
        }
    }
    return max(all & 0xffffu, all >> 16);
}
template <typename T>
MW4_DEV uint32_t largest_finite(const uint4& x) {
    const uint4 one[1] = {x};
    return largest_finite<T>(one, 1);
}

// The sequence and index of row i: index -1 of an idle sequence, -2 for what is no index.
MW4_DEV void row_at(const Append8Args& a, int i, int& b, int& t) {
    b = a.seq ? a.seq[i] : i;
    t = a.slot ? max(a.slot[i], -2) : (unsigned)b < (unsigned)a.c.n_seqs ? max(a.c.lens[b], -1) - 1 : -2;
    if (a.slot && t == -1) t = -2;
}

// Debug builds: a block whose tokens are not consecutive rows would be several runs', each with its
// own scale.  Whether there is one takes a look at all rows (by CTAs beside the writing ones, 4096 tokens
// 4.5 -> 11.3 us), so the product does not ask; here such a call writes nothing.
MW4_DEV bool refused(const Append8Args& a) {
#ifdef MW4_DEBUG_CHECKS
    return *a.disorder;
#else
    (void)a;
    return false;
#endif
}
#ifdef MW4_DEBUG_CHECKS
__global__ void kv8_append_order_kernel(const Append8Args a) {
    const int i = (int)(blockIdx.x * blockDim.x + threadIdx.x);
    if (i >= a.n) return;
    int b, t, ob, ot;
    row_at(a, i, b, t);
    if ((unsigned)b >= (unsigned)a.c.n_seqs || t < 0) return;
    const int in_block = t & ((1 << a.s.shift) - 1);
    if (i > 0 && in_block > 0) {
        row_at(a, i - 1, ob, ot);
        if (ob == b && ot == t - 1) return;                // not a run's first
    }
    for (int j = 0; j < i; ++j) {
        row_at(a, j, ob, ot);
        if (ob == b && ot >= 0 && ot >> a.s.shift == t >> a.s.shift) {
            raise_status(a.status, MOE_W4_STATUS_BAD_INDEX);
            *a.disorder = 1;
            return;
        }
    }
}
#endif

// The exponent of the smallest power of two that brings `top` to 448 = 1.75 * 2^8 or below.
MW4_DEV int scale_exponent(float top) {
    const uint32_t u = __float_as_uint(top);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u);
    return max(kLowest, min(kHighest, e));   // (zero and subnormals lie below)
}

template <typename T>
MW4_DEV uint2 codes8(const uint4& x, float inv) {
    const float2 a = Pair16<T>::unpack(x.x), b = Pair16<T>::unpack(x.y), c = Pair16<T>::unpack(x.z), d = Pair16<T>::unpack(x.w);
    return make_uint2(codes_of(a.x * inv, a.y * inv) | codes_of(b.x * inv, b.y * inv) << 16,
                      codes_of(c.x * inv, c.y * inv) | codes_of(d.x * inv, d.y * inv) << 16);
}

// Two codes brought to a scale `ratio` times smaller.
MW4_DEV uint32_t recode(uint32_t two, float ratio) {
    const float2 f = Pair16<__half>::unpack(f16x2_of_codes((uint16_t)two));
    return codes_of(f.x * ratio, f.y * ratio);
}

// The exponent that a block's scale has, the scale made a power of two: up to the next
// where it is none, and one that is not positive and finite counts as the lowest.
MW4_DEV int exponent_of(float& before) {
    if (!(before > 0.f && before < INFINITY)) before = power2(kLowest);
    const uint32_t u = __float_as_uint(before);
    return max(kLowest, min(kHighest, (int)(u >> 23) - 127 + ((u & 0x7fffffu) != 0)));
}

// A block's tokens but `skip` .. `end` follow its scale, `ratio` times smaller; they lie beside
// one another.
MW4_DEV void follow(uint8_t* first, int64_t slot_stride, int block, int per16, int skip, int end, float ratio, int thread, int threads) {
    for (int i = thread; i < block * per16; i += threads) {
        const int token = i / per16, piece = i & (per16 - 1);
        if (token >= skip && token <= end) continue;
        uint4* at = reinterpret_cast<uint4*>(first + token * slot_stride + piece * 16);
        uint4 c = *at;
        uint32_t* word = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
        for (int k = 0; k < 4; ++k) word[k] = recode(word[k] & 0xffffu, ratio) | recode(word[k] >> 16, ratio) << 16;
        *at = c;
    }
}

// Blocks of one token have nothing to look for: a thread has 8 values of a token's key
// and the 8 of its value beside them, D / 8 lanes a head, and the largest magnitudes of
// both cross lanes together.
template <typename T>
__global__ void __launch_bounds__(kSingleThreads) kv8_append_single_kernel(const Append8Args a, int chunks, uint32_t pieces,
                                                                          uint64_t per_piece, FastDiv per_head) {
    griddep_wait();
    griddep_launch_dependents();
    if (refused(a)) return;
    const int64_t at = (int64_t)blockIdx.x * kSingleThreads + threadIdx.x;
    const uint64_t token = __umul64hi((uint64_t)at, per_piece);
    const bool on = token < (uint64_t)a.n;                 // a head's lanes agree
    const int i = on ? (int)token : 0;
    const uint32_t in = (uint32_t)(at - (int64_t)token * pieces);
    const int h = (int)div_by(in, per_head), piece = (int)in - h * chunks;
    int b = -1, t = -2, page = -1, in_page = 0;
    uint4 kx = make_uint4(0u, 0u, 0u, 0u), vx = kx;
    if (on) {
        row_at(a, i, b, t);
        const int64_t from = ((int64_t)h * chunks + piece) * 8;
        kx = *reinterpret_cast<const uint4*>(a.k_new + i * a.k_stride + from);
        vx = *reinterpret_cast<const uint4*>(a.v_new + i * a.v_stride + from);
    }
    if ((unsigned)b < (unsigned)a.c.n_seqs && t >= 0) {
        const uint32_t p = div_by((uint32_t)t, a.c.page);
        in_page = t - (int)(p * a.c.page.d);
        if (p < (uint32_t)a.c.pages_per_seq) page = a.c.table[b * a.c.table_stride + p];
    }
    const bool there = (unsigned)page < (unsigned)a.c.num_pages;
    if (on && !there && in == 0 && t != -1) raise_status(a.status, MOE_W4_STATUS_BAD_INDEX);
    uint32_t top = largest_finite<T>(kx) | largest_finite<T>(vx) << 16;
    for (int x = chunks >> 1; x; x >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, x));
    if (!there) return;
    const int ke = scale_exponent(Pair16<T>::unpack(top & 0xffffu).x), ve = scale_exponent(Pair16<T>::unpack(top >> 16).x);
    const int64_t to = page * a.c.page_stride + in_page * a.c.slot_stride + h * a.c.head_stride + piece * 8;
    *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(const_cast<uint16_t*>(a.c.k)) + to) = codes8<T>(kx, power2(-ke));
    *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(const_cast<uint16_t*>(a.c.v)) + to) = codes8<T>(vx, power2(-ve));
    if (piece == 0) {
        const int64_t e = page * a.s.page_stride + h * a.s.head_stride + in_page;
        a.s.k[e] = power2(ke);
        a.s.v[e] = power2(ve);
    }
}

// What a warp works for: a head's keys or values.
struct Side {
    int h, values;
    const uint16_t* src;      // a row's values of the head are `stride` apart
    int64_t stride;
    uint8_t* pool;
    float* scales;
    MW4_DEV Side(const Append8Args& a, int hv, int dim) : h(hv >> 1), values(hv & 1) {
        src = (values ? a.v_new : a.k_new) + h * dim;
        stride = values ? a.v_stride : a.k_stride;
        pool = reinterpret_cast<uint8_t*>(const_cast<uint16_t*>(values ? a.c.v : a.c.k));
        scales = values ? a.s.v : a.s.k;
    }
    MW4_DEV int64_t codes(const Append8Args& a, int page, int in_page) const {
        return page * a.c.page_stride + in_page * a.c.slot_stride + h * a.c.head_stride;
    }
    MW4_DEV float* scale(const Append8Args& a, int page, int in_page) const {
        return scales + page * a.s.page_stride + h * a.s.head_stride + (in_page >> a.s.shift);
    }
};

// A warp's rows, one a lane from the one before its window on.  A row follows on where its
// index is the next of the same block; a run is a row that does not and those that
// follow on from it.  The warp has the runs that the window's rows lead, up to 16 of them.
struct Rows {
    int b, t;                 // sequence and index
    int lead, last;           // first and last lane of the run, as far as lanes go
    bool leads, own;          // a row of the window that leads a run; one of such a run
    int entry, in_page;       // of a leader: what the block table says, the token's slot
    MW4_DEV Rows(const Append8Args& a, int row0, int block) : b(-1), t(-2), entry(-1), in_page(0) {
        const int lane = threadIdx.x & 31;
        const uint32_t i = (uint32_t)row0 - 1 + lane;      // past every row before the first
        const bool in = i < (uint32_t)a.n;
        if (in) row_at(a, (int)i, b, t);
        const int pb = __shfl_up_sync(0xffffffffu, b, 1), pt = __shfl_up_sync(0xffffffffu, t, 1);
        const bool on = lane > 0 && in && t > 0 && (t & (block - 1)) && pb == b && pt == t - 1;
        const unsigned starts = ~__ballot_sync(0xffffffffu, on), after = starts >> lane >> 1;
        lead = 31 - __clz(starts & (0xffffffffu >> (31 - lane)));
        last = after ? lane + __ffs(after) - 1 : 31;
        own = in && lead > 0 && lead <= a.window;
        leads = own && lane == lead;
        if (leads && (unsigned)b < (unsigned)a.c.n_seqs && t >= 0) {
            const uint32_t p = div_by((uint32_t)t, a.c.page);
            in_page = t - (int)(p * a.c.page.d);
            if (p < (uint32_t)a.c.pages_per_seq) entry = a.c.table[b * a.c.table_stride + p];
        }
    }
    // The page of the lane's run, -1 for none.
    MW4_DEV int page_of(const Append8Args& a, bool report) const {
        const bool good = (unsigned)entry < (unsigned)a.c.num_pages;
        if (leads && !good && t != -1 && report) raise_status(a.status, MOE_W4_STATUS_BAD_INDEX);   // (-1: an idle sequence)
        return __shfl_sync(0xffffffffu, good ? entry : -1, lead);
    }
};

// The runs of `mine` lanes, whole ones of up to 16 rows that lie within the lanes, by a warp,
// rows asked for before their pages are known:
// all those at a time that 16 rows hold, D / 8 lanes a row.  Rows' largest magnitudes go to
// a lane each, where the runs' come from a maximum over neighbours.
template <typename T, int D>
MW4_DEV void write_rows(const Append8Args& a, const Side& side, const Rows& rw, int row0, int block, bool mine, bool report) {
    constexpr int P = D / 8, RP = 32 / P, N = kRows / RP;  // lanes of a row, rows at a time, turns
    const int lane = threadIdx.x & 31, piece = lane % P, turn_row = lane / P;
    unsigned todo = __ballot_sync(0xffffffffu, mine);
#pragma unroll 1
    while (todo) {
        const int base = __ffs(todo) - 1;
        const unsigned batch = todo & __ballot_sync(0xffffffffu, rw.last < base + kRows), rows = batch >> base;
        todo &= ~batch;
        uint4 x[N];
        const uint16_t* from = side.src + (row0 - 1 + base + turn_row) * side.stride + piece * 8;
#pragma unroll
        for (int j = 0; j < N; ++j, from += RP * side.stride) {
            if (rows >> (j * RP) == 0) break;
            x[j] = make_uint4(0u, 0u, 0u, 0u);
            if (rows >> (j * RP + turn_row) & 1) x[j] = *reinterpret_cast<const uint4*>(from);
        }
        // where the rows go, and the scales of blocks already begun
        const int page = rw.page_of(a, report), first_in = __shfl_sync(0xffffffffu, rw.in_page, rw.lead);
        const int in_block = first_in & (block - 1);       // blocks divide pages
        const bool there = batch >> lane & 1 && page >= 0;
        const unsigned put = __ballot_sync(0xffffffffu, there) >> base;
        int64_t to = 0;                                    // of the row's codes
        float* scale = nullptr;
        float was = 0.f;
        if (there) {
            to = side.codes(a, page, first_in + lane - rw.lead);
            scale = side.scale(a, page, first_in);
            if (in_block) was = *scale;
        }
        uint32_t top = 0;                                  // bits of the largest of the lane's run
        const bool one = (rows & (rows + 1)) == 0 && __shfl_sync(0xffffffffu, rw.last, base) - base == __popc(rows) - 1;   // a single run
        if (one) {
            top = largest_finite<T>(x, (__popc(rows) + RP - 1) / RP);
            top = __reduce_max_sync(0xffffffffu, top);
        } else {
            const unsigned q = lane - base;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (rows >> (j * RP) == 0) break;
                uint32_t bits = largest_finite<T>(x[j]);
                if (P == 32) {
                    bits = __reduce_max_sync(0xffffffffu, bits);
                } else {
#pragma unroll
                    for (int m = P / 2; m; m >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, m));
                    bits = __shfl_sync(0xffffffffu, bits, q % RP * P);
                }
                if (q / RP == j) top = bits;
            }
#pragma unroll
            for (int m = 1; m < kRows; m <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, top, m);
                if (lane - m >= rw.lead) top = max(top, o);
            }
            top = __shfl_sync(0xffffffffu, top, rw.last);
        }
        int e = scale_exponent(Pair16<T>::unpack(top).x);
        if (in_block) e = max(e, exponent_of(was));
        const float now = power2(e), inv = power2(-e);
        const bool leads = there && lane == rw.lead;
#pragma unroll 1
        for (unsigned grown = __ballot_sync(0xffffffffu, leads && in_block && now != was); grown; grown &= grown - 1) {
            const int r = __ffs(grown) - 1;
            const int skip = __shfl_sync(0xffffffffu, in_block, r), end = skip + __shfl_sync(0xffffffffu, rw.last, r) - r;
            const int64_t first = __shfl_sync(0xffffffffu, to, r) - skip * a.c.slot_stride;
            follow(side.pool + first, a.c.slot_stride, block, D / 16, skip, end, __shfl_sync(0xffffffffu, was * inv, r), lane, 32);
        }
        uint8_t* at = side.pool + piece * 8;
        if (one) {
            const float by = __shfl_sync(0xffffffffu, inv, base);
            at += __shfl_sync(0xffffffffu, to, base) + turn_row * a.c.slot_stride;
#pragma unroll
            for (int j = 0; j < N; ++j, at += RP * a.c.slot_stride) {
                if (rows >> (j * RP) == 0) break;
                if (put >> (j * RP + turn_row) & 1) *reinterpret_cast<uint2*>(at) = codes8<T>(x[j], by);
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (rows >> (j * RP) == 0) break;
                const int r = (base + j * RP + turn_row) & 31;
                const int64_t off = __shfl_sync(0xffffffffu, to, r);
                const float by = __shfl_sync(0xffffffffu, inv, r);
                if (put >> (j * RP + turn_row) & 1) *reinterpret_cast<uint2*>(at + off) = codes8<T>(x[j], by);
            }
        }
        if (leads) *scale = now;
    }
}

// Blocks of 2 to 16 tokens: a warp a window.
template <typename T, int D>
__global__ void __launch_bounds__(kRowsThreads, rows_warps(D) * 32 / kRowsThreads) kv8_append_rows_kernel(const Append8Args a) {
    griddep_wait();
    griddep_launch_dependents();
    if (refused(a)) return;
    const int64_t item = (int64_t)blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5);
    const int per_window = 2 * a.c.n_kv_heads;
    const int w = (int)(item / per_window), hv = (int)(item - (int64_t)w * per_window);
    if (w >= a.windows) return;                            // whole warps
    const int block = 1 << a.s.shift, row0 = w * a.window;
    const Rows rows(a, row0, block);
    write_rows<T, D>(a, Side(a, hv, D), rows, row0, block, rows.own, hv == 0);
}

MW4_DEV void team_sync(int barrier, int threads) { asm volatile("bar.sync %0, %1;" :: "r"(barrier), "r"(threads) : "memory"); }

// A run of more rows than a warp holds, as its team sees it: found by one warp, once, so that
// all agree on it whatever happens to the indexes meanwhile.
struct Run {
    int row, count, page;     // first row, rows, page
    int in_page;              // the first token's slot
};

// Blocks of 32 to 128 tokens: a window for each warp of a CTA, which write their short runs
// themselves; the longer ones teams of as many warps as hold a block, in registers as well.
template <typename T, int D, int TEAM>
__global__ void __launch_bounds__(kLongThreads, long_ctas(D)) kv8_append_long_kernel(const Append8Args a) {
    constexpr int WARPS = kLongThreads / 32, P = D / 8, PIECES = kRows * P / 32;
    constexpr int TEAMS = WARPS / TEAM, THREADS = TEAM * 32;   // TEAM: warps, for blocks of 16 times as many tokens
    __shared__ float sh_top[2][WARPS];
    __shared__ Run sh_runs[WARPS][kRows];
    __shared__ int sh_found[WARPS];
    griddep_wait();
    griddep_launch_dependents();
    if (refused(a)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_window = 2 * a.c.n_kv_heads;
    const int w = blockIdx.x / per_window, hv = blockIdx.x - w * per_window;
    const int block = 1 << a.s.shift, row0 = min((w * WARPS + warp) * (int64_t)a.window, (int64_t)a.n);
    const Side side(a, hv, D);
    const Rows rows(a, row0, block);
    const bool is_short = rows.last < 31 && rows.last - rows.lead < kRows;
    int found = 0;
#pragma unroll 1
    for (unsigned left = __ballot_sync(0xffffffffu, rows.leads && !is_short); left; left &= left - 1) {
        const int page = rows.page_of(a, hv == 0);
        const int r = __ffs(left) - 1, end = __shfl_sync(0xffffffffu, rows.last, r);
        const int seq = __shfl_sync(0xffffffffu, rows.b, r), t0 = __shfl_sync(0xffffffffu, rows.t, r);
        Run run{row0 - 1 + r, end - r + 1, __shfl_sync(0xffffffffu, page, r), __shfl_sync(0xffffffffu, rows.in_page, r)};
        if (run.page < 0) continue;
        if (end == 31) {                                   // the lanes' rows end first
            const int room = min(block - (t0 & (block - 1)), a.n - run.row);
            while (run.count < room) {
                const int j = run.count + lane;
                int jb = -1, jt = -2;
                if (j < room) row_at(a, run.row + j, jb, jt);
                const unsigned on = __ballot_sync(0xffffffffu, j < room && jb == seq && jt == t0 + j);
                const int n = on == 0xffffffffu ? 32 : __ffs(~on) - 1;
                run.count += n;
                if (n < 32) break;
            }
        }
        if (lane == 0) sh_runs[warp][found] = run;
        ++found;
    }
    if (lane == 0) sh_found[warp] = found;
    write_rows<T, D>(a, side, rows, row0, block, rows.own && is_short, hv == 0);
    __syncthreads();
    const int team = warp / TEAM, thread = threadIdx.x % THREADS;
    int turn = 0, next = team;                             // of the team; runs before its next one
#pragma unroll 1
    for (int f = 0; f < WARPS; ++f) {
        const int runs = sh_found[f];
#pragma unroll 1
        for (; next < runs; next += TEAMS, ++turn) {
            const Run run = sh_runs[f][next];
            const int in_block = run.in_page & (block - 1), pieces = run.count * P;
            float* scale = side.scale(a, run.page, run.in_page);
            float before = in_block ? *scale : 0.f;
            uint4 x[PIECES];
#pragma unroll
            for (int j = 0; j < PIECES; ++j) {
                const int e = thread + j * THREADS;
                if (j * THREADS >= pieces) break;
                x[j] = make_uint4(0u, 0u, 0u, 0u);
                if (e < pieces) x[j] = *reinterpret_cast<const uint4*>(side.src + (run.row + e / P) * side.stride + e % P * 8);
            }
            const uint32_t bits = largest_finite<T>(x, (pieces + THREADS - 1) / THREADS);
            float top = Pair16<T>::unpack(__reduce_max_sync(0xffffffffu, bits)).x;
            if (lane == 0) sh_top[turn & 1][warp] = top;   // (two places in turn: nobody is two runs behind)
            team_sync(1 + team, THREADS);
#pragma unroll
            for (int j = 0; j < TEAM; ++j) top = fmaxf(top, sh_top[turn & 1][team * TEAM + j]);
            int e = scale_exponent(top);
            if (in_block) e = max(e, exponent_of(before));
            const float now = power2(e), inv = power2(-e);
            uint8_t* to = side.pool + side.codes(a, run.page, run.in_page);
            if (in_block && now != before)                 // the block's other tokens follow
                follow(to - in_block * a.c.slot_stride, a.c.slot_stride, block, D / 16, in_block, in_block + run.count - 1,
                       before * inv, thread, THREADS);
#pragma unroll
            for (int j = 0; j < PIECES; ++j) {
                const int e2 = thread + j * THREADS;
                if (j * THREADS >= pieces) break;
                if (e2 < pieces) *reinterpret_cast<uint2*>(to + e2 / P * a.c.slot_stride + e2 % P * 8) = codes8<T>(x[j], inv);
            }
            if (thread == 0) *scale = now;
        }
        next -= runs;
    }
}

template <typename T>
static cudaError_t launch_append8_single(const Append8Args& a, int dim, cudaStream_t st) {
    const uint32_t chunks = (uint32_t)dim / 8, pieces = chunks * (uint32_t)a.c.n_kv_heads;
    const int64_t ctas = ((int64_t)a.n * pieces + kSingleThreads - 1) / kSingleThreads;
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_pdl(true, kv8_append_single_kernel<T>, dim3((unsigned)ctas), dim3(kSingleThreads), 0, st, a, (int)chunks, pieces,
                      UINT64_MAX / pieces + 1, fast_div(chunks));
}
// Windows of as many rows, up to 16, as give every SM kWindows: more keep it busier but find
// fewer rows to take together (512 tokens of 512 sequences, 8 heads of 128, blocks of 2, with
// 4, 6, 8, 16 and 32 a SM: 3.6, 3.0, 3.0, 3.4 and 5.6 us; 4096 of 2 of 256, blocks of 16:
// 5.1, 5.1, 6.1, 6.2 and 6.7, before rows were asked for ahead of their pages).
template <typename T, int D>
static cudaError_t launch_append8_rows(Append8Args a, int sms, cudaStream_t st) {
    const bool few = a.s.shift <= kRowsShift;
    const int warps = (few ? kRowsThreads : kLongThreads) / 32;
    const int64_t sides = 2 * a.c.n_kv_heads, rows = a.n * sides / ((int64_t)sms * kWindows);
    a.window = rows < 1 ? 1 : rows < kRows ? (int)rows : kRows;
    a.windows = (a.n - 1) / a.window + 1;
    // a warp has a window of a side, or a CTA one of a side for each of its warps
    const int64_t ctas = few ? (a.windows * sides + warps - 1) / warps : (int64_t)((a.windows + warps - 1) / warps) * sides;
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    const auto kern = few ? kv8_append_rows_kernel<T, D> : a.s.shift == 5 ? kv8_append_long_kernel<T, D, 2>
                      : a.s.shift == 6 ? kv8_append_long_kernel<T, D, 4> : kv8_append_long_kernel<T, D, 8>;
    return launch_pdl(true, kern, dim3((unsigned)ctas), dim3(warps * 32), 0, st, a);
}
template <typename T>
static cudaError_t launch_append8(const Append8Args& a, int dim, cudaStream_t st) {
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
#ifdef MW4_DEBUG_CHECKS
    cudaError_t e = cudaMemsetAsync(a.disorder, 0, sizeof(*a.disorder), st);
    if (e == cudaSuccess) {
        kv8_append_order_kernel<<<(unsigned)((a.n - 1) / 256 + 1), 256, 0, st>>>(a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
#endif
    if (a.s.shift == 0) return launch_append8_single<T>(a, dim, st);
    return dim == 64 ? launch_append8_rows<T, 64>(a, sms, st)
           : dim == 128 ? launch_append8_rows<T, 128>(a, sms, st) : launch_append8_rows<T, 256>(a, sms, st);
}

// ---------------------------------------------------------------------------
// reading back
// ---------------------------------------------------------------------------
// A thread per 16 bytes of a token's row as it is written: 8 values of the key and of
// the value, code * scale rounded once.  Bytes bound it (1 read and 2 written per
// value); few tokens, three trips to memory.  16,384 tokens of 2 heads of 256: 9.1 us for
// 50 MB, 333 of 8 heads of 128 2.0 (a thread for 16 codes, whose two stores leave gaps
// between lanes: 9.8 and 2.3).
struct ReadArgs {
    KvView c;
    Scales s;
    uint16_t* k_out;
    uint16_t* v_out;
    int64_t k_stride, v_stride;
    const int32_t* seq;
    const int32_t* slot;
    int n, chunks;               // chunks: pieces of a head's row
    FastDiv per_head;            // chunks
    uint32_t pieces;             // of a token: n_kv_heads * chunks, at least 8
    uint64_t per_piece;          // 2^64 / pieces, rounded up: the high half of a product is a quotient below 2^47
    unsigned int* status;
};

constexpr int kReadThreads = 256;

template <typename T>
MW4_DEV uint32_t value_pair(uint32_t two, float scale) {
    const float2 f = Pair16<__half>::unpack(f16x2_of_codes((uint16_t)two));
    return Pair16<T>::pack(f.x * scale, f.y * scale);
}
template <typename T>
MW4_DEV uint4 values8(const uint2& c, float scale) {
    return make_uint4(value_pair<T>(c.x & 0xffffu, scale), value_pair<T>(c.x >> 16, scale),
                      value_pair<T>(c.y & 0xffffu, scale), value_pair<T>(c.y >> 16, scale));
}

// CODES: 8 codes a piece; else 8 values, copied.
template <typename T, bool CODES>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const ReadArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t at = (int64_t)blockIdx.x * kReadThreads + threadIdx.x;
    const uint64_t token = __umul64hi((uint64_t)at, a.per_piece);
    if (token >= (uint64_t)a.n) return;
    const int i = (int)token;
    const uint32_t in = (uint32_t)(at - (int64_t)i * a.pieces);
    const int h = (int)div_by(in, a.per_head), piece = (int)in - h * a.chunks;
    constexpr int W = 8;                         // values of a piece
    const int b = a.seq ? a.seq[i] : i;
    int t = -2;
    if ((unsigned)b < (unsigned)a.c.n_seqs) {
        t = a.slot ? a.slot[i] : max(a.c.lens[b], -1) - 1;
        if (a.slot && t < 0) t = -2;
    }
    int page = -1, in_page = 0;
    if (t >= 0) {
        const uint32_t p = div_by((uint32_t)t, a.c.page);
        in_page = t - (int)(p * a.c.page.d);
        if (p < (uint32_t)a.c.pages_per_seq) page = a.c.table[b * a.c.table_stride + p];
    }
    uint16_t* k_to = a.k_out + i * a.k_stride + ((int64_t)h * a.chunks + piece) * W;
    uint16_t* v_to = a.v_out + i * a.v_stride + ((int64_t)h * a.chunks + piece) * W;
    uint4 kx = make_uint4(0u, 0u, 0u, 0u), vx = kx;
    if ((unsigned)page < (unsigned)a.c.num_pages) {
        const int64_t from = page * a.c.page_stride + in_page * a.c.slot_stride + h * a.c.head_stride + piece * W;
        if (CODES) {
            const int64_t e = page * a.s.page_stride + h * a.s.head_stride + (in_page >> a.s.shift);
            const uint2 kc = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(a.c.k) + from);
            const uint2 vc = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(a.c.v) + from);
            const float ks = a.s.k[e], vs = a.s.v[e];
            kx = values8<T>(kc, ks);
            vx = values8<T>(vc, vs);
        } else {
            kx = *reinterpret_cast<const uint4*>(a.c.k + from);
            vx = *reinterpret_cast<const uint4*>(a.c.v + from);
        }
    } else if (in == 0 && t != -1) {
        raise_status(a.status, MOE_W4_STATUS_BAD_INDEX);
    }
    *reinterpret_cast<uint4*>(k_to) = kx;
    *reinterpret_cast<uint4*>(v_to) = vx;
}

// least: elements between tokens that must not overlap, as they are written.
static int check_tokens(const moe_w4_kv_tokens* t, const moe_w4_kv_cache& c, int64_t least) {
    if (!t || t->n < 0 || t->k_stride < 0 || t->v_stride < 0 || (t->n > 0 && (!t->k || !t->v || (!t->seq && t->n != c.n_seqs))) ||
        (t->n > 1 && (t->k_stride < least || t->v_stride < least)))
        return MOE_W4_ERR_INVALID;
    if (misaligned(t->k, 16) || misaligned(t->v, 16) || t->k_stride % 8 || t->v_stride % 8 || misaligned(t->seq, 4) ||
        misaligned(t->slot, 4))
        return MOE_W4_ERR_ALIGN;
    return check_workspace(t->workspace, t->ws_bytes, MOE_W4_CTRL_BYTES);
}

template <typename T, bool CODES>
static cudaError_t launch_read(const ReadArgs& a, cudaStream_t st) {
    const int64_t ctas = ((int64_t)a.n * a.pieces + kReadThreads - 1) / kReadThreads;
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_pdl(true, kv_read_kernel<T, CODES>, dim3((unsigned)ctas), dim3(kReadThreads), 0, st, a);
}

static int read_tokens(const moe_w4_kv_cache& c, const moe_w4_kv8_cache* c8, const moe_w4_kv_tokens* t, cudaStream_t stream) {
    const int r = check_tokens(t, c, (int64_t)c.n_kv_heads * c.head_dim);
    if (r) return r;
    if (t->n == 0) return MOE_W4_OK;   // (rows of a cache of no sequences are written all the same: zeros)
    ReadArgs a{};
    a.c = kv_view(c);
    if (c8) a.s = scales_of(*c8);
    a.k_out = static_cast<uint16_t*>(t->k);
    a.v_out = static_cast<uint16_t*>(t->v);
    a.k_stride = t->k_stride;
    a.v_stride = t->v_stride;
    a.seq = t->seq;
    a.slot = t->slot;
    a.n = t->n;
    a.chunks = c.head_dim / 8;
    a.per_head = fast_div((uint32_t)a.chunks);
    a.pieces = (uint32_t)(c.n_kv_heads * a.chunks);
    a.per_piece = UINT64_MAX / a.pieces + 1;
    a.status = &static_cast<Ctrl*>(t->workspace)->status;
    if (!c8) return launched(launch_read<__half, false>(a, stream));   // a copy, whatever the type
    return launched(c.dtype == MOE_W4_TYPE_BF16 ? launch_read<__nv_bfloat16, true>(a, stream) : launch_read<__half, true>(a, stream));
}

}  // namespace mw4

using namespace mw4;

extern "C" {

int moe_w4_kv8_append(const moe_w4_kv8_cache* c, const moe_w4_kv_tokens* t, cudaStream_t stream) {
    int r = check_cache8(c, t && !t->slot);
    if (r || (r = check_tokens(t, c->c, 0))) return r;
    if (t->n == 0 || c->c.n_seqs == 0) return MOE_W4_OK;
    Append8Args a{};
    a.c = kv_view(c->c);
    a.s = scales_of(*c);
    a.k_new = static_cast<const uint16_t*>(t->k);
    a.v_new = static_cast<const uint16_t*>(t->v);
    a.k_stride = t->k_stride;
    a.v_stride = t->v_stride;
    a.seq = t->seq;
    a.slot = t->slot;
    a.n = t->n;
    a.status = &static_cast<Ctrl*>(t->workspace)->status;
    a.disorder = &static_cast<Ctrl*>(t->workspace)->pad[kCtrlDisorderWord];
    return launched(c->c.dtype == MOE_W4_TYPE_BF16 ? launch_append8<__nv_bfloat16>(a, c->c.head_dim, stream)
                                                   : launch_append8<__half>(a, c->c.head_dim, stream));
}

int moe_w4_kv8_read(const moe_w4_kv8_cache* c, const moe_w4_kv_tokens* t, cudaStream_t stream) {
    const int r = check_cache8(c, t && !t->slot);
    return r ? r : read_tokens(c->c, c, t, stream);
}

int moe_w4_kv_read(const moe_w4_kv_cache* c, const moe_w4_kv_tokens* t, cudaStream_t stream) {
    const int r = check_cache(c, t && !t->slot);
    return r ? r : read_tokens(*c, nullptr, t, stream);
}

}  // extern "C"
