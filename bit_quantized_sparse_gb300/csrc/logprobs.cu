// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits x:
//   lse = m + log Z,  Z = sum exp(x - m),  m = max x
//   logprob(t) = x_t - lse,  entropy = log Z - sum exp(x - m) (x - m) / Z
// Every logit is read once in principle: HBM bounds large calls.
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

template <typename T> MW4_DEV float to_float(T v);
template <> MW4_DEV float to_float<float>(float v) { return v; }
template <> MW4_DEV float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> MW4_DEV float to_float<__half>(__half v) { return __half2float(v); }

// Order of the alternatives: larger logit first, then the lower index; NaN
// after every number.  No logit has key 0.
MW4_DEV uint32_t logit_key(float x) { return isnan(x) ? 1u : order_key(x + 0.f); }
MW4_DEV uint64_t logit_word(float x, int i) { return ((uint64_t)logit_key(x) << 32) | (uint32_t)~i; }

constexpr int kRowThreads = 1024;

template <typename V, typename F>
MW4_DEV V block_reduce(V v, V* sh, F f) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 16; off; off >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, off));
    __syncthreads();
    if (lane == 0) sh[warp] = v;
    __syncthreads();
    v = sh[lane];
#pragma unroll
    for (int off = 16; off; off >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// One CTA per row.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) token_logprobs_kernel(const LogprobArgs a) {
    __shared__ float sh_f[32];
    __shared__ uint64_t sh_w[32];
    griddep_wait();
    const int row = blockIdx.x, tid = threadIdx.x;
    const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
    auto add = [](float p, float q) { return p + q; };
    float m = -INFINITY;
    int odd = 0;   // a NaN or +inf
    for (int i = tid; i < a.vocab; i += kRowThreads) {
        const float v = to_float(x[i]);
        m = fmaxf(m, v);
        odd |= isnan(v) || v == INFINITY;
    }
    m = block_reduce(m, sh_f, [](float p, float q) { return fmaxf(p, q); });
    odd = __syncthreads_or(odd);
    float Z = 0.f, U = 0.f;
    for (int i = tid; i < a.vocab; i += kRowThreads) {
        const float d = fmaxf(to_float(x[i]) - m, -200.f);   // exp is 0 below about -104
        const float e = __expf(d);
        Z += e;
        U += e * d;
    }
    Z = block_reduce(Z, sh_f, add);
    U = block_reduce(U, sh_f, add);
    const bool none = odd || m == -INFINITY;
    const float lse = none ? NAN : m + logf(Z);
    if (tid == 0) {
        if (a.entropy) a.entropy[row] = none ? NAN : logf(Z) - U / Z;
        if (a.targets) {
            const int t = a.targets[row];
            const bool in = (unsigned)t < (unsigned)a.vocab;
            if (!in && t != -1) raise_status(a.status, MOE_W4_STATUS_BAD_INDEX);
            a.logprob[row] = in ? to_float(x[t]) - lse : t == -1 ? 0.f : NAN;
        }
    }
    uint64_t last = ~0ull;
    for (int k = 0; k < a.top; ++k) {
        uint64_t best = 0;
        for (int i = tid; i < a.vocab; i += kRowThreads) {
            const uint64_t w = logit_word(to_float(x[i]), i);
            if (w < last && w > best) best = w;
        }
        best = block_reduce(best, sh_w, [](uint64_t p, uint64_t q) { return p > q ? p : q; });
        if (tid == 0) {
            const int i = (int)~(uint32_t)best;
            a.top_index[(int64_t)row * a.top + k] = i;
            a.top_logprob[(int64_t)row * a.top + k] = to_float(x[i]) - lse;
        }
        last = best;
    }
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
    LogprobArgs a{logits, row_stride, n, vocab, top, targets, logprob, entropy, top_index, top_logprob,
                  static_cast<unsigned int*>(workspace)};
    auto kern = dtype == MOE_W4_TYPE_BF16 ? token_logprobs_kernel<__nv_bfloat16>
                : dtype == MOE_W4_TYPE_FP16 ? token_logprobs_kernel<__half> : token_logprobs_kernel<float>;
    return launched(launch_pdl(true, kern, dim3(n), dim3(kRowThreads), 0, stream, a));
}
