// rows.h -- rows of fp32 or bfloat16 values: loads and stores of 8 and 16-byte
// pieces, and the checks of 8-bit rows, shared by the norm (norm.hip), the
// linear that takes 8-bit rows (gemm_i8.hip) and the operators over logits.
#pragma once
#include "kv.h"

namespace ht {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

struct Row8 {
    float v[8];
};

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Two values rounded to nearest even by one instruction (NaN stays NaN).
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}
__device__ __forceinline__ uint16_t round_bf16(float v) { return __builtin_bit_cast(uint16_t, __bf16(v)); }

// 8 consecutive values, 16-byte aligned.
__device__ __forceinline__ void store8(float *p, const Row8 &r) {
    reinterpret_cast<f32x4 *>(p)[0] = f32x4{r.v[0], r.v[1], r.v[2], r.v[3]};
    reinterpret_cast<f32x4 *>(p)[1] = f32x4{r.v[4], r.v[5], r.v[6], r.v[7]};
}
__device__ __forceinline__ void store8(uint16_t *p, const Row8 &r) {
    *reinterpret_cast<u32x4 *>(p) = u32x4{pack_bf16(r.v[0], r.v[1]), pack_bf16(r.v[2], r.v[3]),
                                          pack_bf16(r.v[4], r.v[5]), pack_bf16(r.v[6], r.v[7])};
}

// K values of a row as a buffer: 8 of them per thread as two halves that start at
// columns lo and hi; what lies behind the row reads as zeros and is not written.
// The row's address is the same in every lane.  ONCE: not kept in the caches.
template <typename T>
struct RowBuf {
    __amdgpu_buffer_rsrc_t r;

    __device__ __forceinline__ RowBuf(const T *p, int K)
        : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<T *>(p), 0, K * int(sizeof(T)), 0x00020000)) {}

    template <bool WHOLE, bool ONCE>     // WHOLE: hi = lo + 4
    __device__ __forceinline__ Row8 load(int lo, int hi) const {
        constexpr int kAux = ONCE ? 2 : 0;
        if constexpr (sizeof(T) == 4) {
            const f32x4 a = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, 4 * lo, 0, kAux));
            const f32x4 b = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, 4 * hi, 0, kAux));
            return Row8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
        } else {
            u32x4 u;
            if constexpr (WHOLE) {
                u = __builtin_amdgcn_raw_buffer_load_b128(r, 2 * lo, 0, kAux);
            } else {
                const u32x2 a = __builtin_amdgcn_raw_buffer_load_b64(r, 2 * lo, 0, kAux), b = __builtin_amdgcn_raw_buffer_load_b64(r, 2 * hi, 0, kAux);
                u = u32x4{a.x, a.y, b.x, b.y};
            }
            return Row8{{bf_lo(u.x), bf_hi(u.x), bf_lo(u.y), bf_hi(u.y), bf_lo(u.z), bf_hi(u.z), bf_lo(u.w), bf_hi(u.w)}};
        }
    }
    template <bool WHOLE>
    __device__ __forceinline__ void store(int lo, int hi, const Row8 &o) const {
        if constexpr (sizeof(T) == 4) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{o.v[0], o.v[1], o.v[2], o.v[3]}), r, 4 * lo, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{o.v[4], o.v[5], o.v[6], o.v[7]}), r, 4 * hi, 0, 0);
        } else {
            const u32x4 u{pack_bf16(o.v[0], o.v[1]), pack_bf16(o.v[2], o.v[3]), pack_bf16(o.v[4], o.v[5]), pack_bf16(o.v[6], o.v[7])};
            if constexpr (WHOLE) {
                __builtin_amdgcn_raw_buffer_store_b128(u, r, 2 * lo, 0, 0);
            } else {
                __builtin_amdgcn_raw_buffer_store_b64(u32x2{u.x, u.y}, r, 2 * lo, 0, 0);
                __builtin_amdgcn_raw_buffer_store_b64(u32x2{u.z, u.w}, r, 2 * hi, 0, 0);
            }
        }
    }
};

// The value of lane ^ 16, lane ^ 32, by the swaps of rows of 16 and of halves.
__device__ __forceinline__ float row_xor16(float v) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(threadIdx.x & 16 ? r[0] : r[1]);
}
__device__ __forceinline__ float row_xor32(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(threadIdx.x & 32 ? r[0] : r[1]);
}

// Sum over a wavefront, the same on all lanes.
__device__ __forceinline__ float wave_sum(float v) {
    v = group_sum<16>(v);
    v += row_xor16(v);
    v += row_xor32(v);
    return v;
}

// Host check of a matrix of rows: ld >= K, pointer and stride in 16-byte pieces.
inline ht_status check_matrix(const void *p, int64_t ld, int64_t M, int64_t K, int size) {
    if (!p) return HT_EINVAL;
    if (M > 1 && ld < K) return HT_ESHAPE;
    if (!al16p(p) || (M > 1 && (ld * size) % 16)) return HT_EALIGN;
    return HT_OK;
}

inline int64_t q8_groups(int64_t M) { return (M + 15) / 16; }

inline ht_status check_q8_shape(int64_t M, int64_t K) {
    if (M < 0 || M > (int64_t(1) << 30) || K <= 0 || K % 64 || K > (1 << 20)) return HT_ESHAPE;
    return HT_OK;
}

inline ht_status check_q8(const ht_q8_rows *q) {
    if (!q || !q->codes || !q->scales) return HT_EINVAL;
    const ht_status st = check_q8_shape(q->M, q->K);
    if (st != HT_OK) return st;
    if (!al16p(q->codes) || !al16p(q->scales)) return HT_EALIGN;
    return HT_OK;
}

}  // namespace ht
