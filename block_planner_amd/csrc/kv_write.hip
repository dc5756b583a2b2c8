// kv_write.hip -- rows of keys and values quantised into the paged 8-bit
// cache, one power-of-two scale per page, head and K or V.
//
//   2^(E-1) <= max |x| < 2^E over the block,  code = clamp(rne(x 2^(7-E)), -127, 127)
//
// Scaling by a power of two is exact, so a code has one rounding and does not
// depend on the order of anything.  When appended rows raise E by d, older
// codes become rne(code 2^-d): E only grows, so all such halvings of an entry
// together add less than half a step of the final scale (1/4 + 1/8 + ...) to
// the half step of its own rounding.
//
// Bound by HBM for prompts (inputs in, one byte per entry out), by latency for
// single tokens.  The rows of one page (a run) are one workgroup's work per
// head and K or V, so the scale needs no exchange between workgroups.
// Workgroups find the runs in the slots themselves: a window of 64 rows is one
// ballot, and the `reps` workgroups of a window take its runs in turn (64
// single-token runs of a decode batch are 64 workgroups' work, a prompt's one
// or two runs per window leave the others to end at once).
#include "kv.h"

namespace ht {

namespace {

constexpr int kWriteThreads = 256;

struct WriteArgs {
    const void *x[2];
    int64_t ld[2], hs[2];
    const int32_t *slots;
    int8_t *codes;
    float *scales;
    int32_t T, n_slots, n_heads, reps;
};

template <typename X>
__device__ __forceinline__ f32x4 load_row4(const X *p);
template <>
__device__ __forceinline__ f32x4 load_row4<float>(const float *p) {
    return *reinterpret_cast<const f32x4 *>(p);
}
template <>
__device__ __forceinline__ f32x4 load_row4<uint16_t>(const uint16_t *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                 __uint_as_float(u.y & 0xFFFF0000u)};
}

__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u; }

// x f, f = 2^(7-E) (between 2^-121 and 2^67), rounded half to even and
// clamped; NaN gives 0.
__device__ __forceinline__ int quantise(float x, float f) {
    const float v = rintf(x * f);
    return v != v ? 0 : int(fminf(fmaxf(v, -127.f), 127.f));
}

// Byte of token t, dim d within a block.
template <int D>
__device__ __forceinline__ int k_byte(int t, int d) {
    return ((((t >> 4) * (D / 64) + (d >> 6)) * 4 + ((d >> 4) & 3)) * 16 + (t & 15)) * 16 + (d & 15);
}
__device__ __forceinline__ int v_byte(int t, int d) {
    return ((((d >> 4) * 4 + ((t >> 2) & 3)) * 16 + (d & 15)) * 4 + (t >> 4)) * 4 + (t & 3);
}

// Four codes scaled down by 2^-d (f = 2^-d), rounded half to even.
__device__ __forceinline__ uint32_t halve4(uint32_t w, float f) {
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) r |= (uint32_t(int(rintf(float(int8_t(w >> (8 * j))) * f))) & 0xFFu) << (8 * j);
    return r;
}

// One run: rows t0 .. t0 + n - 1 (slots off[0 .. n-1] of one page).
template <int D, typename X, bool V>
__device__ void write_run(const WriteArgs &a, int32_t t0, int n, int32_t page, int head, const uint8_t *off,
                          float *red, uint8_t *stage) {
    constexpr int kPerRow = D / 4, kRows = kWriteThreads / kPerRow;   // threads per row, rows per step
    constexpr int kUsed = kRows * kPerRow;                            // (D = 192: 240 of 256 threads)
    constexpr int kSteps = (kPage + kRows - 1) / kRows;
    constexpr int kBlock = kPage * D;
    const int tid = threadIdx.x, d = (tid % kPerRow) * 4, sub = tid / kPerRow;
    const X *x = static_cast<const X *>(a.x[V]) + int64_t(head) * a.hs[V] + d;
    const int64_t blk = (int64_t(page) * a.n_heads + head) * 2 + V;
    uint32_t *out = reinterpret_cast<uint32_t *>(a.codes + blk * kBlock);
    f32x4 v[kSteps];
    float top = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int i = s * kRows + sub;
        v[s] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (i < n && tid < kUsed) {
            v[s] = load_row4(x + (int64_t(t0) + i) * a.ld[V]);
#pragma unroll
            for (int j = 0; j < 4; ++j) top = fmaxf(top, finite(v[s][j]) ? fabsf(v[s][j]) : 0.f);
        }
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m));
    if ((tid & 63) == 0) red[tid >> 6] = top;
    const bool fresh = off[0] == 0;
    const int e_old = fresh ? kMinExp : exp_of_scale(a.scales[blk]);
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const int e = max(e_old, exp_of_max(top)), down = fresh ? 0 : e - e_old;
    const float f = pow2f(7 - e), fd = pow2f(max(-down, -126));
    if (tid == 0) a.scales[blk] = pow2f(e - 7);   // every thread has read the old one

    if (n <= 8) {
        // few rows: rewrite the block only if its scale grew, then store the new codes
        if (down > 0) {
            for (int w = tid; w < kBlock / 4; w += kWriteThreads) out[w] = halve4(out[w], fd);
            __syncthreads();
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int i = s * kRows + sub;
            if (s * kRows >= 8) break;
            if (i < n && tid < kUsed) {
                const int t = off[i];
                uint32_t q[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) q[j] = uint32_t(quantise(v[s][j], f)) & 0xFFu;
                if constexpr (V) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) reinterpret_cast<uint8_t *>(out)[v_byte(t, d + j)] = uint8_t(q[j]);
                } else {
                    out[k_byte<D>(t, d) / 4] = q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24);
                }
            }
        }
        return;
    }
    // many rows: the block in LDS, then out in whole lines
    uint32_t *st = reinterpret_cast<uint32_t *>(stage);
    if (n < kPage) {
        for (int w = tid; w < kBlock / 4; w += kWriteThreads) st[w] = down > 0 ? halve4(out[w], fd) : out[w];
        __syncthreads();
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int i = s * kRows + sub;
        if (i < n && tid < kUsed) {
            const int t = off[i];
            uint32_t q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = uint32_t(quantise(v[s][j], f)) & 0xFFu;
            if constexpr (V) {
#pragma unroll
                for (int j = 0; j < 4; ++j) stage[v_byte(t, d + j)] = uint8_t(q[j]);
            } else {
                st[k_byte<D>(t, d) / 4] = q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24);
            }
        }
    }
    __syncthreads();
    for (int w = tid; w < kBlock / 16; w += kWriteThreads)
        reinterpret_cast<uint4 *>(out)[w] = reinterpret_cast<const uint4 *>(stage)[w];
}

template <int D, typename XK, typename XV>
__global__ __launch_bounds__(kWriteThreads) void kv_write_kernel(WriteArgs a) {
    __shared__ float red[kWriteThreads / 64];
    __shared__ uint8_t off[kPage];
    __shared__ __align__(16) uint8_t stage[kPage * D];
    const int tid = threadIdx.x, lane = tid & 63;
    const int32_t w0 = int32_t(blockIdx.x / uint32_t(a.reps)) * 64;
    const int rep = int(blockIdx.x % uint32_t(a.reps));
    // the window's slots and the 64 after them (a run may end there); -1 where there is no row to write
    int32_t slot[2];
    uint64_t cont[2];   // bit i: row i belongs to the page of the row before it
    uint64_t lead = 0;  // bit i: row i starts a run
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t t = int64_t(w0) + 64 * j + lane;
        int32_t s = t < a.T ? a.slots[t] : -1, p = t > 0 && t <= a.T ? a.slots[t - 1] : -1;
        if (s < 0 || s >= a.n_slots) s = -1;
        if (p < 0 || p >= a.n_slots) p = -1;
        const bool same = s >= 0 && p >= 0 && s / kPage == p / kPage;
        slot[j] = s;
        cont[j] = __ballot(same);
        if (j == 0) lead = __ballot(s >= 0 && !same);
    }
    int nth = 0;
    for (; lead; lead &= lead - 1, ++nth) {
        if (nth % a.reps != rep) continue;
        const int i = __ffsll((unsigned long long)lead) - 1;
        // rows that continue the run, at most a page
        const uint64_t ahead = i == 63 ? cont[1] : (cont[0] >> (i + 1)) | (cont[1] << (63 - i));
        const int n = ahead == ~uint64_t(0) ? kPage : min(kPage, __ffsll((unsigned long long)~ahead));
        const int32_t s0 = __shfl(slot[0], i);
        __syncthreads();   // the run before has read off and stage
        if (tid < 64) {
            const int src = i + lane;
            const int32_t sa = __shfl(slot[0], src & 63), sb = __shfl(slot[1], src & 63);
            off[lane] = uint8_t((src < 64 ? sa : sb) & (kPage - 1));
        }
        __syncthreads();
        if (blockIdx.z == 0) write_run<D, XK, false>(a, w0 + i, n, s0 / kPage, int(blockIdx.y), off, red, stage);
        else write_run<D, XV, true>(a, w0 + i, n, s0 / kPage, int(blockIdx.y), off, red, stage);
    }
}

template <int D>
void launch_write(const WriteArgs &a, dim3 grid, bool kb, bool vb, hipStream_t s) {
    if (kb && vb) kv_write_kernel<D, uint16_t, uint16_t><<<grid, kWriteThreads, 0, s>>>(a);
    else if (kb) kv_write_kernel<D, uint16_t, float><<<grid, kWriteThreads, 0, s>>>(a);
    else if (vb) kv_write_kernel<D, float, uint16_t><<<grid, kWriteThreads, 0, s>>>(a);
    else kv_write_kernel<D, float, float><<<grid, kWriteThreads, 0, s>>>(a);
}

}  // namespace
}  // namespace ht

using namespace ht;

extern "C" ht_status ht_kv_write(const void *k, int64_t ldk, int64_t hsk, int32_t kt, const void *v, int64_t ldv,
                                 int64_t hsv, int32_t vt, int64_t T, const int32_t *slots, const ht_kv_cache *cache,
                                 ht_stream stream) {
    ht_status st = check_cache(cache);
    if (st != HT_OK) return st;
    if (!act_size(kt) || !act_size(vt)) return HT_EINVAL;
    if (T < 0 || T > (int64_t(1) << 30)) return HT_ESHAPE;
    if (T == 0) return HT_OK;
    if ((st = check_rows(k, ldk, hsk, cache->n_heads, cache->head_dim, act_size(kt))) != HT_OK) return st;
    if ((st = check_rows(v, ldv, hsv, cache->n_heads, cache->head_dim, act_size(vt))) != HT_OK) return st;
    if (!slots) return HT_EINVAL;
    if (!al4(slots)) return HT_EALIGN;
    WriteArgs a{{k, v}, {ldk, ldv}, {hsk, hsv}, slots, cache->codes, cache->scales, int32_t(T),
                int32_t(cache->n_pages * kPage), cache->n_heads, 64};
    // every run of a window its own workgroup while batches are small; from
    // 2048 rows (32 windows) a quarter of that, so that the workgroups that
    // find nothing stay few beside the ones that work
    if (T > 2048) a.reps = 16;
    const dim3 grid(uint32_t((T + 63) / 64) * uint32_t(a.reps), uint32_t(cache->n_heads), 2);
    hipStream_t s = hipStream_t(stream);
    const bool kb = kt == HT_BF16, vb = vt == HT_BF16;
    switch (cache->head_dim) {
    case 64: launch_write<64>(a, grid, kb, vb, s); break;
    case 128: launch_write<128>(a, grid, kb, vb, s); break;
    case 192: launch_write<192>(a, grid, kb, vb, s); break;
    default: launch_write<256>(a, grid, kb, vb, s); break;
    }
    HT_LAUNCH_CHECK();
    return HT_OK;
}
