// Norms of queries and keys per head with the position rotation, in one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * w,  then pairs (a, b) of y turn:
//   a cos - b sin, b cos + a sin.
// Two bytes read and two written per value: HBM bounds it, and for the tokens of
// a decode batch the trips to memory do.
//
// A head's row of D values belongs to D / 8 lanes, and a lane has both partners of
// its pairs: by halves 4 values of each half (two loads of 8 bytes), interleaved 8
// in a row; where nothing turns, 8 in a row.  So only the sum of squares crosses
// lanes, and the row stays in registers between its one read and its one write.
// Arithmetic is in packed pairs of fp32: issue bounds it beside the bytes.
//
// The rows of a grid are whole tokens, so a thread keeps its head, its weights and
// its dimensions from one token to the next, and only pointers move.  The cosines
// and sines of a batch's tokens are worked out once a CTA, in shared memory, while
// the batch's rows arrive.
//
// 4096 tokens of 18 heads of 256, 64 of them turning: 15.9 us for 75 MB (a copy of
// them takes 12.3); 2501 tokens of 40 heads of 128: 12.4; 16 tokens: 1.9.  Slower:
// the batch after asked for before this one is worked on (29; registers cost a CTA),
// a warp for all of a token's heads and its angles in registers (16.3, 15.0 and 2.2).
//
// An angle is positions * turns modulo 2^64: the product's high 32 bits are the
// fraction of a turn, so that no position, however far, loses bits to a range
// reduction (with an fp32 angle 131,071 * 1 rad is off by 2^-8 rad).  Cosine and sine are
// those of half turns, to two steps of fp32; the fast ones (15.5 and 11.8 us) are off by
// 2^-21, which shows where a result is small.
#include "serving.cuh"
#include "moe_w4_longctx.h"

namespace mw4 {

constexpr int kRopeThreads = 256, kRopeCtas = 4;   // CTAs of an SM

struct RopeArgs {
    const uint16_t* x[2];      // queries, keys
    uint16_t* y[2];
    int64_t x_stride[2], y_stride[2];
    const uint16_t* w[2];      // or NULL
    const uint64_t* turns;
    const int32_t* axis;
    const int32_t* positions;
    int64_t pos_stride;
    int n, heads[2], pairs, axes, interleaved;
    FastDiv per_token, per_pair;   // heads[0] + heads[1], pairs
    int table_floats;              // of the cosines and sines of a batch
    int step;                      // tokens between a thread's rows
    float eps, offset, scale;
};

// Four values of a row: as packed pairs they multiply two at a time.
struct Four {
    float2 x, y;
};
template <typename T> MW4_DEV Four four_of(const uint2& u) { return {Pair16<T>::unpack(u.x), Pair16<T>::unpack(u.y)}; }
MW4_DEV Four mul(const Four& a, const Four& b) { return {__fmul2_rn(a.x, b.x), __fmul2_rn(a.y, b.y)}; }
MW4_DEV Four mul_add(const Four& a, const Four& b, const Four& c) { return {__ffma2_rn(a.x, b.x, c.x), __ffma2_rn(a.y, b.y, c.y)}; }
MW4_DEV Four all(float f) { return {make_float2(f, f), make_float2(f, f)}; }
// Evens and odds of 8 values, and back.
MW4_DEV void part(Four& a, Four& b) {
    const Four e = {make_float2(a.x.x, a.y.x), make_float2(b.x.x, b.y.x)}, o = {make_float2(a.x.y, a.y.y), make_float2(b.x.y, b.y.y)};
    a = e;
    b = o;
}
MW4_DEV void merge(Four& a, Four& b) {
    const Four p = {make_float2(a.x.x, b.x.x), make_float2(a.x.y, b.x.y)}, q = {make_float2(a.y.x, b.y.x), make_float2(a.y.y, b.y.y)};
    a = p;
    b = q;
}

// ROWS: rows of a thread in flight together, a batch.  PAIRED: pairs are interleaved.
template <typename T, int D, int ROWS, bool PAIRED>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int LR = D / 8;                          // lanes of a row
    constexpr int PASS = kRopeThreads / LR;            // rows that the CTA has at a time
    extern __shared__ __align__(16) float table[];     // once or twice: [rows][tokens of the CTA][cosines, sines][pairs]
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x % LR;
    const uint32_t heads = a.per_token.d, slot0 = blockIdx.x * PASS, slot = slot0 + threadIdx.x / LR;
    const int token0 = (int)div_by(slot0, a.per_token), span = (int)div_by(slot0 + PASS - 1, a.per_token) - token0 + 1;
    const int token = (int)div_by(slot, a.per_token), head = (int)(slot - token * heads), k = head >= a.heads[0];
    const bool turns = lane < a.pairs / 4;
    // a lane's two times four dimensions
    const int d1 = !PAIRED && turns ? 4 * lane : 8 * lane, d2 = !PAIRED && turns ? a.pairs + 4 * lane : 8 * lane + 4;
    const int64_t in_row = (int64_t)(head - (k ? a.heads[0] : 0)) * D + d1;
    const int64_t x_step = a.step * (k ? a.x_stride[1] : a.x_stride[0]), y_step = a.step * (k ? a.y_stride[1] : a.y_stride[0]);
    const uint16_t* x = (k ? a.x[1] : a.x[0]) + token * (k ? a.x_stride[1] : a.x_stride[0]) + in_row;
    uint16_t* y = (k ? a.y[1] : a.y[0]) + token * (k ? a.y_stride[1] : a.y_stride[0]) + in_row;
    Four wu = all(1.f), wv = all(1.f);
    const uint16_t* weight = k ? a.w[1] : a.w[0];
    if (weight) {
        wu = four_of<T>(*reinterpret_cast<const uint2*>(weight + d1));
        wv = four_of<T>(*reinterpret_cast<const uint2*>(weight + d2));
        const Four one = all(1.f), offset = all(a.offset);
        wu = mul_add(wu, one, offset);
        wv = mul_add(wv, one, offset);
    }
    // entry e of a batch's table: pair e % pairs of its row's and CTA's token
    const uint32_t count = (uint32_t)(ROWS * span * a.pairs);
    float* turn = table;
#pragma unroll 1
    for (int base = token0;; base += ROWS * a.step) {  // the batch's first token of the CTA
        const int mine = base + (token - token0);      // this thread's first
        uint2 x1[ROWS], x2[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i, x += x_step) {
            x1[i] = x2[i] = make_uint2(0u, 0u);
            if (mine + i * a.step < a.n) {
                x1[i] = *reinterpret_cast<const uint2*>(x);
                x2[i] = *reinterpret_cast<const uint2*>(x + (d2 - d1));
            }
        }
        for (uint32_t e = threadIdx.x; e < count; e += kRopeThreads) {   // while the rows are on their way
            // a shift where a division stood: 17.0 -> 15.4 us of 4096 tokens
            const uint32_t rt = div_by(e, a.per_pair);
            const int p = (int)(e - rt * a.pairs), i = span <= 2 ? (int)rt >> (span - 1) : (int)(rt / span), t = base + i * a.step + (int)rt - i * span;
            const int axis = a.axis ? max(0, min(a.axis[p], a.axes - 1)) : 0;
            const int pos = a.positions[axis * a.pos_stride + min(t, a.n - 1)];
            const uint64_t turned = (uint64_t)(int64_t)pos * a.turns[p];
            float* to = turn + 2 * (e - p) + p, sine, cosine;
            sincospif((float)(int32_t)(turned >> 32) * (1.f / 2147483648.f), &sine, &cosine);   // of -1 .. 1 half turns
            to[0] = cosine * a.scale;
            to[a.pairs] = sine * a.scale;
        }
        __syncthreads();                               // (the other table is free: everybody is past its last use)
        const float* cs = turn + 2 * (token - token0) * a.pairs + 4 * lane;
#pragma unroll
        for (int i = 0; i < ROWS; ++i, cs += 2 * span * a.pairs, y += y_step) {
            Four u = four_of<T>(x1[i]), v = four_of<T>(x2[i]);
            if (weight) {                              // (a row's lanes agree; its shuffles are their own)
                const Four sq = mul_add(u, u, mul(v, v));
                const float2 two = __fadd2_rn(sq.x, sq.y);
                float sum = two.x + two.y;
                const unsigned mask = LR == 32 ? 0xffffffffu : ((1u << (LR & 31)) - 1) << (threadIdx.x & 31 & ~(LR - 1));
#pragma unroll
                for (int off = LR / 2; off; off >>= 1) sum += __shfl_xor_sync(mask, sum, off);
                const Four inv = all(rsqrtf(sum * (1.f / D) + a.eps));
                u = mul(mul(u, inv), wu);
                v = mul(mul(v, inv), wv);
            }
            if (turns) {
                if (PAIRED) part(u, v);
                const float4 fc = *reinterpret_cast<const float4*>(cs), fs = *reinterpret_cast<const float4*>(cs + a.pairs);
                const Four c = {make_float2(fc.x, fc.y), make_float2(fc.z, fc.w)}, s = {make_float2(fs.x, fs.y), make_float2(fs.z, fs.w)};
                const Four minus = {make_float2(-fs.x, -fs.y), make_float2(-fs.z, -fs.w)};
                const Four p = mul_add(v, minus, mul(u, c)), q = mul_add(u, s, mul(v, c));
                u = p;
                v = q;
                if (PAIRED) merge(u, v);
            }
            if (mine + i * a.step < a.n) {
                *reinterpret_cast<uint2*>(y) = make_uint2(Pair16<T>::pack(u.x.x, u.x.y), Pair16<T>::pack(u.y.x, u.y.y));
                *reinterpret_cast<uint2*>(y + (d2 - d1)) = make_uint2(Pair16<T>::pack(v.x.x, v.x.y), Pair16<T>::pack(v.y.x, v.y.y));
            }
        }
        if (a.n - base <= ROWS * a.step) return;
        turn = turn == table ? table + a.table_floats : table;
    }
}

template <typename T, int D, int ROWS>
static cudaError_t launch_rope(RopeArgs a, cudaStream_t st) {
    constexpr int pass = kRopeThreads / (D / 8);
    const int64_t heads = a.per_token.d;
    // The grid's rows are those of `step` tokens, whole tokens to whole CTAs, so that a
    // thread keeps its head; and as many that all CTAs have equal numbers of batches.
    int64_t unit = pass;
    for (int64_t h = heads; unit > 1 && h % 2 == 0; h /= 2) unit /= 2;   // pass is a power of two
    const int64_t most = (int64_t)sm_count() * kRopeCtas * pass / heads / unit * unit, largest = most > unit ? most : unit;
    const int64_t batches = (a.n + largest * ROWS - 1) / (largest * ROWS);
    const int64_t step = ((a.n + batches * ROWS - 1) / (batches * ROWS) + unit - 1) / unit * unit;
    a.step = (int)step;
    const int64_t span = (pass - 1) / heads + 2 < pass ? (pass - 1) / heads + 2 : pass;   // tokens of a CTA's rows at most
    a.table_floats = (int)(ROWS * span * a.pairs * 2);   // 8192 at most (heads of 64, one a token)
    const size_t smem = (size_t)a.table_floats * sizeof(float) * (batches > 1 ? 2 : 1);
    const auto kern = a.interleaved ? qk_norm_rope_kernel<T, D, ROWS, true> : qk_norm_rope_kernel<T, D, ROWS, false>;
    static std::atomic<unsigned> ready[2];
    int dev = 0;
    sm_count(&dev);
    if (smem > 48 << 10) {
        const cudaError_t e = allow_smem((const void*)kern, 64 << 10, ready[a.interleaved ? 1 : 0], dev);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(true, kern, dim3((unsigned)(step * heads / pass)), dim3(kRopeThreads), smem, st, a);
}

template <typename T, int D>
static cudaError_t launch_rope_rows(const RopeArgs& a, cudaStream_t st) {
    // few rows are spread over the GPU, one of a thread
    const int64_t ctas = (int64_t)a.n * a.per_token.d / (kRopeThreads / (D / 8));
    return ctas < kRopeCtas * (int64_t)sm_count() ? launch_rope<T, D, 1>(a, st) : launch_rope<T, D, 4>(a, st);
}

template <typename T>
static cudaError_t launch_rope_dim(int dim, const RopeArgs& a, cudaStream_t st) {
    return dim == 64 ? launch_rope_rows<T, 64>(a, st) : dim == 128 ? launch_rope_rows<T, 128>(a, st) : launch_rope_rows<T, 256>(a, st);
}

}  // namespace mw4

using namespace mw4;

extern "C" int moe_w4_qk_norm_rope(const moe_w4_qk_call* call, cudaStream_t stream) {
    if (!call) return MOE_W4_ERR_INVALID;
    const moe_w4_qk_call& t = *call;
    const int dtype = t.dtype, n = t.n, head_dim = t.head_dim, n_q_heads = t.n_q_heads, n_k_heads = t.n_k_heads;
    const moe_w4_rope* rope = t.rope;
    const int32_t* positions = t.positions;
    const int64_t pos_stride = t.pos_stride;
    const float eps = t.eps;
    if (dtype != MOE_W4_TYPE_BF16 && dtype != MOE_W4_TYPE_FP16) return MOE_W4_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return MOE_W4_ERR_UNSUPPORTED;
    if (n < 0 || n_q_heads < 0 || n_k_heads < 0 || !(eps >= 0.f)) return MOE_W4_ERR_INVALID;
    if (n_q_heads > 65536 || n_k_heads > 65536) return MOE_W4_ERR_UNSUPPORTED;
    if (rope) {
        if (rope->pairs < 8 || rope->pairs % 8 || 2 * rope->pairs > head_dim || rope->axes < 1 || rope->axes > 8 || pos_stride < 0)
            return rope->pairs > 0 && rope->pairs % 8 ? MOE_W4_ERR_UNSUPPORTED : MOE_W4_ERR_INVALID;
        if (!rope->turns) return MOE_W4_ERR_INVALID;
        if (misaligned(rope->turns, 8) || misaligned(rope->axis, 4)) return MOE_W4_ERR_ALIGN;
    }
    const int64_t heads = (int64_t)n_q_heads + n_k_heads;
    if (n == 0 || heads == 0) return MOE_W4_OK;
    if (n * heads >= 1ll << 30) return MOE_W4_ERR_UNSUPPORTED;   // rows are counted with 32 bits
    if (rope && !positions) return MOE_W4_ERR_INVALID;
    if (rope && misaligned(positions, 4)) return MOE_W4_ERR_ALIGN;
    const void* x[2] = {t.q, t.k};
    void* y[2] = {t.q_out, t.k_out};
    const int64_t xs[2] = {t.q_stride, t.k_stride}, ys[2] = {t.qo_stride, t.ko_stride};
    const int count[2] = {n_q_heads, n_k_heads};
    RopeArgs a{};
    for (int i = 0; i < 2; ++i) {
        if (!count[i]) continue;
        if (!x[i] || !y[i] || (n > 1 && (xs[i] < 0 || ys[i] < (int64_t)count[i] * head_dim))) return MOE_W4_ERR_INVALID;
        if (x[i] == y[i] && n > 1 && xs[i] != ys[i]) return MOE_W4_ERR_INVALID;
        if (misaligned(x[i], 16) || misaligned(y[i], 16) || xs[i] % 8 || ys[i] % 8) return MOE_W4_ERR_ALIGN;
        a.x[i] = static_cast<const uint16_t*>(x[i]);
        a.y[i] = static_cast<uint16_t*>(y[i]);
        a.x_stride[i] = xs[i];
        a.y_stride[i] = ys[i];
    }
    if (misaligned(t.q_weight, 16) || misaligned(t.k_weight, 16)) return MOE_W4_ERR_ALIGN;
    a.w[0] = static_cast<const uint16_t*>(t.q_weight);
    a.w[1] = static_cast<const uint16_t*>(t.k_weight);
    a.n = n;
    a.heads[0] = n_q_heads;
    a.heads[1] = n_k_heads;
    a.per_token = fast_div((uint32_t)heads);
    a.eps = eps;
    a.offset = t.unit_offset ? 1.f : 0.f;
    if (rope) {
        a.turns = rope->turns;
        a.axis = rope->axis;
        a.positions = positions;
        a.pos_stride = pos_stride;
        a.pairs = rope->pairs;
        a.axes = rope->axes;
        a.interleaved = rope->interleaved;
        a.scale = rope->scale;
        a.per_pair = fast_div((uint32_t)rope->pairs);
    }
    return launched(dtype == MOE_W4_TYPE_BF16 ? launch_rope_dim<__nv_bfloat16>(head_dim, a, stream)
                                              : launch_rope_dim<__half>(head_dim, a, stream));
}

