// The cache of 8-bit codes as kernels see it, and its argument checks.
#pragma once
#include <cuda_fp8.h>

#include "moe_w4_longctx.h"
#include "serving.cuh"

namespace mw4 {

struct Scales {
    float* k;
    float* v;
    int64_t page_stride, head_stride;
    int shift;   // log2 of the block
};

// Strides and addresses of codes go in 16 bytes, so in elements they are multiples
// of 16; everything else is as for a cache of 16-bit values.
inline int check_cache8(const moe_w4_kv8_cache* c, bool need_lens) {
    if (!c) return MOE_W4_ERR_INVALID;
    const int r = check_cache(&c->c, need_lens);
    if (r) return r;
    if (c->block < 1 || c->scale_page_stride < 0 || c->scale_head_stride < 0) return MOE_W4_ERR_INVALID;
    if (c->block > 128 || (c->block & (c->block - 1)) || c->c.page_size % c->block) return MOE_W4_ERR_UNSUPPORTED;
    if (((c->c.page_stride | c->c.head_stride | c->c.slot_stride) >> 4) > UINT32_MAX) return MOE_W4_ERR_UNSUPPORTED;
    if (c->c.n_seqs == 0) return MOE_W4_OK;
    if (!c->k_scale || !c->v_scale) return MOE_W4_ERR_INVALID;
    if (c->c.page_stride % 16 || c->c.head_stride % 16 || c->c.slot_stride % 16 || misaligned(c->k_scale, 4) ||
        misaligned(c->v_scale, 4))
        return MOE_W4_ERR_ALIGN;
    return MOE_W4_OK;
}

inline Scales scales_of(const moe_w4_kv8_cache& c) {
    int shift = 0;
    while ((1 << shift) < c.block) ++shift;
    return {c.k_scale, c.v_scale, c.scale_page_stride, c.scale_head_stride, shift};
}

// 2^e, -126 <= e <= 127.
MW4_DEV float power2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// Two codes to two fp16, exact.
MW4_DEV uint32_t f16x2_of_codes(uint16_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}
// Two numbers to the nearest codes, the first in the low byte; past 448 they become 448, NaN stays.
MW4_DEV uint32_t codes_of(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace mw4
