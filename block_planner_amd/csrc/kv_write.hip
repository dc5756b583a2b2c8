// kv_write.hip -- rows of keys and values quantised into the paged 8-bit
// cache, one power-of-two scale per page, head and K or V.
//
//   2^(E-1) <= max |x| < 2^E over the block,  code = clamp(rne(x 2^(7-E)), -127, 127)
//
// Scaling by a power of two is exact, so a code has one rounding and does not
// depend on the order of anything.  When appended rows raise E by d, older
// codes become rne(code 2^-d): E only grows, so of an entry's roundings the last
// adds at most half a step of the final scale, the one before a quarter and so on
// (the entry's own is the first of them): less than one step together.
//
// Bound by HBM for prompts (inputs in, one byte per entry out), by latency for
// single tokens.  A run -- rows at consecutive slots of one page -- is the
// work of one workgroup (or, up to 8 rows, of one wavefront) per head and K or
// V, so the scale needs no exchange between workgroups.  Workgroups find the
// runs in the slots themselves: a window of 64 rows is one ballot, and the
// `reps` workgroups of a window take its runs in turn.
//
// Long runs: every thread owns whole 16-byte pieces of the block (K: 16 dims of
// a token, V: 16 tokens of a dim), loads the entries of its pieces straight
// into registers, and stores each piece at once; a piece the run covers in part
// is read, overlaid and stored by the same thread, so no LDS is needed.  12000
// rows of 8 x 128 (bf16 K, fp32 V): 22 us, 4.1 TB/s; 64 single rows: 4.4 us.
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
__device__ __forceinline__ u32x4 halve16(u32x4 w, float f) {
    return u32x4{halve4(w.x, f), halve4(w.y, f), halve4(w.z, f), halve4(w.w, f)};
}

__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return __uint_as_float(uint32_t(*p) << 16); }

// A run: rows row .. row + n - 1 at tokens first .. first + n - 1 of a page.
struct Run {
    int32_t row, page;
    int n, first;
};

// Scale of the block with the run in it: the exponent, and by how much older
// codes have to come down.
__device__ __forceinline__ int run_exponent(float top, float old_scale, bool fresh, int &down) {
    const int e_old = fresh ? kMinExp : exp_of_scale(old_scale);
    const int e = max(e_old, exp_of_max(top));
    down = fresh ? 0 : e - e_old;
    return e;
}

constexpr int kShort = 8;   // rows of a run that one wavefront takes

// A short run, by one wavefront: lane l holds dims DC * l .. DC * (l + 1) - 1 of every row.
template <int D, typename X, bool V>
__device__ __forceinline__ void write_short(const WriteArgs &a, const Run &r, int head) {
    constexpr int DC = D / 64;
    const int lane = threadIdx.x & 63, d = lane * DC;
    const X *x = static_cast<const X *>(a.x[V]) + int64_t(head) * a.hs[V] + int64_t(r.row) * a.ld[V] + d;
    const int64_t blk = (int64_t(r.page) * a.n_heads + head) * 2 + V;
    uint8_t *out = reinterpret_cast<uint8_t *>(a.codes + blk * (kPage * D));
    const float old_scale = a.scales[blk];
    float v[kShort][DC];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < kShort; ++i)
#pragma unroll
        for (int j = 0; j < DC; ++j) v[i][j] = i < r.n ? load1(x + i * a.ld[V] + j) : 0.f;
#pragma unroll
    for (int i = 0; i < kShort; ++i)
#pragma unroll
        for (int j = 0; j < DC; ++j) top = fmaxf(top, finite(v[i][j]) ? fabsf(v[i][j]) : 0.f);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m));
    int down;
    const int e = run_exponent(top, old_scale, r.first == 0, down);
    const float f = pow2f(7 - e);
    if (down > 0) {
        const float fd = pow2f(max(-down, -126));
        u32x4 *w = reinterpret_cast<u32x4 *>(out);
        for (int i = lane; i < kPage * D / 16; i += 64) w[i] = halve16(w[i], fd);
        // the new codes below overwrite bytes of these stores
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    if (lane == 0) a.scales[blk] = pow2f(e - 7);
#pragma unroll
    for (int i = 0; i < kShort; ++i) {
        if (i >= r.n) break;
        const int t = r.first + i;
        uint32_t q[DC];
#pragma unroll
        for (int j = 0; j < DC; ++j) q[j] = uint32_t(quantise(v[i][j], f)) & 0xFFu;
        if constexpr (!V && DC == 2) {
            *reinterpret_cast<uint16_t *>(out + k_byte<D>(t, d)) = uint16_t(q[0] | (q[1] << 8));
        } else if constexpr (!V && DC == 4) {
            *reinterpret_cast<uint32_t *>(out + k_byte<D>(t, d)) = q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24);
        } else {
#pragma unroll
            for (int j = 0; j < DC; ++j) out[V ? v_byte(t, d + j) : k_byte<D>(t, d + j)] = uint8_t(q[j]);
        }
    }
}

// A longer run, by the workgroup: DC pieces of 16 bytes per thread.
template <int D, typename X, bool V>
__device__ __forceinline__ void write_long(const WriteArgs &a, const Run &r, int head, float *red) {
    constexpr int DC = D / 64;
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const X *x = static_cast<const X *>(a.x[V]) + int64_t(head) * a.hs[V] + (int64_t(r.row) - r.first) * a.ld[V];
    const int64_t blk = (int64_t(r.page) * a.n_heads + head) * 2 + V;
    u32x4 *out = reinterpret_cast<u32x4 *>(a.codes + blk * (kPage * D));
    const float old_scale = a.scales[blk];
    const auto in_run = [&](int t) { return t >= r.first && t < r.first + r.n; };
    // tokens outside the run read its first row and count as zero: loads without branches, all in flight at once
    float v[DC][16];
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < DC; ++j) {
        if constexpr (V) {
            // dim 64 j + lane, tokens 16 b + 4 wv + i: a load is 64 dims of a token, a store four runs of 256 bytes
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int t = (i >> 2) * 16 + wv * 4 + (i & 3);
                v[j][i] = load1(x + (in_run(t) ? t : r.first) * a.ld[V] + 64 * j + lane);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (!in_run((i >> 2) * 16 + wv * 4 + (i & 3))) v[j][i] = 0.f;
        } else {
            // token 16 wv + lane % 16, dims 64 j + 16 (lane / 16) + 0 .. 15: a store is 1 KB
            const int t = wv * 16 + (lane & 15);
            const X *row = x + (in_run(t) ? t : r.first) * a.ld[V] + 16 * (lane >> 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 w = load_row4(row + 64 * j + 4 * i);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[j][4 * i + k] = in_run(t) ? w[k] : 0.f;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < DC; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, finite(v[j][i]) ? fabsf(v[j][i]) : 0.f);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m));
    if (lane == 0) red[wv] = top;
    __syncthreads();   // also: every thread has read the old scale
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    int down;
    const int e = run_exponent(top, old_scale, r.first == 0, down);
    const float f = pow2f(7 - e), fd = pow2f(max(-down, -126));
    if (tid == 0) a.scales[blk] = pow2f(e - 7);
#pragma unroll
    for (int j = 0; j < DC; ++j) {
        u32x4 w, mask;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            uint32_t c = 0, m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c |= (uint32_t(quantise(v[j][4 * b + i], f)) & 0xFFu) << (8 * i);
                if (in_run(V ? b * 16 + wv * 4 + i : wv * 16 + (lane & 15))) m |= 0xFFu << (8 * i);
            }
            w[b] = c;
            mask[b] = m;
        }
        // piece of (token, dims) or (dim, tokens) in the block's order
        u32x4 *p = out + (V ? (4 * j + (lane >> 4)) * 4 + wv : (wv * DC + j) * 4 + (lane >> 4)) * 16 + (lane & 15);
        const uint32_t all = mask.x & mask.y & mask.z & mask.w, any = mask.x | mask.y | mask.z | mask.w;
        if (all != 0xFFFFFFFFu) {
            if (any == 0 && down == 0) continue;
            const u32x4 old = *p;
            const u32x4 kept = down > 0 ? halve16(old, fd) : old;
            w = (w & mask) | (kept & ~mask);
        }
        *p = w;
    }
}

template <int D, typename XK, typename XV>
__global__ __launch_bounds__(kWriteThreads) void kv_write_kernel(WriteArgs a) {
    __shared__ float red[kWriteThreads / 64];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, head = int(blockIdx.y);
    const int32_t w0 = int32_t(blockIdx.x / uint32_t(a.reps)) * 64;
    const uint32_t rep = blockIdx.x & (uint32_t(a.reps) - 1);
    // the window's slots, the one before and the 64 after them (a run may end there); -1 where there is no row to write
    const int64_t t = int64_t(w0) + lane;
    int32_t s0 = a.slots[min(t, int64_t(a.T) - 1)], s1 = a.slots[min(t + 64, int64_t(a.T) - 1)];
    int32_t before = a.slots[max(w0 - 1, 0)];
    if (t >= a.T || s0 < 0 || s0 >= a.n_slots) s0 = -1;
    if (t + 64 >= a.T || s1 < 0 || s1 >= a.n_slots) s1 = -1;
    if (w0 == 0 || before < 0 || before >= a.n_slots) before = -1;
    const int32_t last = __shfl(s0, 63);
    int32_t p0 = __shfl_up(s0, 1), p1 = __shfl_up(s1, 1);
    if (lane == 0) { p0 = before; p1 = last; }
    const auto follows = [](int32_t s, int32_t p) { return s > 0 && p == s - 1 && (s & (kPage - 1)) != 0; };
    const uint64_t cont0 = __ballot(follows(s0, p0)), cont1 = __ballot(follows(s1, p1));   // row i goes on the run of i - 1
    // every lane's row as the start of a run: its length, its number among the window's runs
    const bool lead = s0 >= 0 && !follows(s0, p0);
    const uint64_t leads = __ballot(lead);
    const uint64_t ahead = lane == 63 ? cont1 : (cont0 >> (lane + 1)) | (cont1 << (63 - lane));
    const int n = ahead == ~uint64_t(0) ? kPage : __ffsll((unsigned long long)~ahead);
    const uint32_t nth = uint32_t(__popcll(leads & ((uint64_t(1) << lane) - 1)));
    const bool mine = lead && (nth & (uint32_t(a.reps) - 1)) == rep;   // reps: a power of two
    uint64_t longs = __ballot(mine && n > kShort);
    uint64_t shorts = __ballot(mine && n <= kShort && ((nth / uint32_t(a.reps)) & (kWriteThreads / 64 - 1)) == uint32_t(wv));
    const auto run_at = [&](uint64_t m) {
        const int i = __ffsll((unsigned long long)m) - 1;
        const int32_t s = __builtin_amdgcn_readlane(s0, i);
        return Run{w0 + i, s / kPage, __builtin_amdgcn_readlane(n, i), s & (kPage - 1)};
    };
    for (; shorts; shorts &= shorts - 1) {
        const Run r = run_at(shorts);
        if (blockIdx.z == 0) write_short<D, XK, false>(a, r, head);
        else write_short<D, XV, true>(a, r, head);
    }
    for (; longs; longs &= longs - 1) {
        const Run r = run_at(longs);
        if (blockIdx.z == 0) write_long<D, XK, false>(a, r, head, red);
        else write_long<D, XV, true>(a, r, head, red);
        __syncthreads();   // red has been read
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
    if (T < 0 || T > (int64_t(1) << 28)) return HT_ESHAPE;
    if (T == 0) return HT_OK;
    if ((st = check_rows(k, ldk, hsk, cache->n_heads, cache->head_dim, act_size(kt))) != HT_OK) return st;
    if ((st = check_rows(v, ldv, hsv, cache->n_heads, cache->head_dim, act_size(vt))) != HT_OK) return st;
    if (!slots) return HT_EINVAL;
    if (!al4(slots)) return HT_EALIGN;
    WriteArgs a{{k, v}, {ldk, ldv}, {hsk, hsv}, slots, cache->codes, cache->scales, int32_t(T),
                int32_t(cache->n_pages * kPage), cache->n_heads, 64};
    // about 2048 workgroups: all of a window's 64 possible runs in a workgroup
    // of their own while batches are small, and few that find no run beside a
    // prompt's (one or two runs per window)
    const int64_t base = (T + 63) / 64 * cache->n_heads * 2;
    a.reps = 1;
    while (a.reps < 64 && a.reps * base < 2048) a.reps *= 2;
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
