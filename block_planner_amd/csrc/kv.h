// kv.h -- the 8-bit paged cache of keys and values: addressing, exponents of
// its power-of-two scales, and host checks shared by the kernels that write
// and read it (kv_plan.hip, kv_write.hip, kv_attn.hip).
#pragma once
#include "ht_internal.h"

namespace ht {

constexpr int kPage = HT_KV_PAGE;
constexpr int kMinExp = HT_KV_MIN_EXP;

// E of 2^(E-1) <= m < 2^E for a finite m >= 0, at least kMinExp (a subnormal
// m is below that anyway).
__device__ __forceinline__ int exp_of_max(float m) {
    return max(int(__float_as_uint(m) >> 23) - 126, kMinExp);
}

// E of a stored scale 2^(E-7), clamped to the range a write produces, so that
// a scale that was never written (zero, or any bits) stays harmless.
__device__ __forceinline__ int exp_of_scale(float s) {
    return min(max(int((__float_as_uint(s) >> 23) & 0xFFu) - 120, kMinExp), 128);
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

inline bool al4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
inline bool al16p(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Element size of an activation type, 0 for a type these calls do not take.
inline int act_size(int32_t t) { return t == HT_FP32 ? 4 : t == HT_BF16 ? 2 : 0; }

// Host check of one [T][heads][D] operand: strides wide enough and in whole
// 16-byte pieces, pointer aligned.  Strides may be in either order (heads
// inside rows or rows inside heads), so only their sizes are checked.
inline ht_status check_rows(const void *p, int64_t ld, int64_t hs, int64_t heads, int64_t D, int size) {
    if (!p) return HT_EINVAL;
    if (ld < D || (heads > 1 && hs < D)) return HT_ESHAPE;
    if (!al16p(p) || (ld * size) % 16 || (heads > 1 && (hs * size) % 16)) return HT_EALIGN;
    return HT_OK;
}

inline ht_status check_cache(const ht_kv_cache *c) {
    if (!c || !c->codes || !c->scales) return HT_EINVAL;
    if (c->n_pages <= 0 || c->n_pages * kPage >= (int64_t(1) << 31) || c->n_heads <= 0 || c->n_heads > 1024) return HT_ESHAPE;
    if (c->head_dim <= 0 || c->head_dim % 64 || c->head_dim > 256) return HT_ESHAPE;
    if (!al16p(c->codes) || !al16p(c->scales)) return HT_EALIGN;
    return HT_OK;
}

}  // namespace ht
