// qk_rope.hip -- the norm of every head of q and k and the rotation by
// position in one pass over them, and its backward pass.
//
//   n = x r w,  r = 1 / sqrt(mean(x^2) + eps);   (y_i, y_j) = R(a) (n_i, n_j)
//   backward, with g = R(-a) dy:  dx = r (w g - xhat mean(w g xhat)),  xhat = x r
//   (the same as r (w g) - x r^3 / D sum(w g x)),  dw = sum_rows g xhat.
//
// Bound by HBM: x in, y out (backward: dy and x in, dx out), a few tens of
// fp32 operations per 16 bytes.  8191 x 36 heads x 64, fp32 to bf16: 21 us, 5.3
// TB/s (part of it from the Infinity Cache); backward of 8192 x 40 x 128 in fp32:
// 85 us, 5.9 TB/s, + 5 us for the weights' partial sums; one token 3.1 us.
//
// A head's row is held by LPR lanes (8, 16 or 32 for D up to 64, 128, 256),
// 8 elements each in two groups of four chosen so that a lane holds both
// halves of its pairs: the rotation needs no exchange, and the norm's sum is
// one reduction within the row's lanes.  Rows of all tokens and heads are numbered through
// (q heads, then k heads, token by token); a workgroup takes a contiguous run
// of them, so any number of heads fills its lanes.  Sines and cosines are
// computed once per token and pair of a workgroup's run into LDS: the angle in
// fp64 turns, reduced to [-1/2, 1/2] there, then fp32 sine and cosine of pi
// times it; fp32 angles would lose the phase of far positions (position 10^5
// leaves 2^-7 of a radian).
#include "kv.h"

namespace ht {

namespace {

constexpr int kRopeThreads = 256;

struct RopeRows {
    const void *x;      // q or k
    const void *dy;     // backward: gradient of y
    void *y;            // forward: y; backward: dx
    int64_t ld, hs, ldd, hsd, ldy, hsy;
    const float *w;
};

struct RopeArgs {
    RopeRows q, k;
    const int32_t *positions;
    const double *inv_freq;
    float *dw_part;          // backward: [gridDim.x][2][D], or the result itself where one workgroup does it all
    float *dwq, *dwk;
    int64_t rows;            // T * (n_q + n_k)
    FastDiv heads;           // n_q + n_k
    int32_t n_q, D, half, interleaved, rows_per_wg, tokens_lds;
    float eps, inv_d;
};

template <typename T>
__device__ __forceinline__ f32x4 load4(const T *p);
template <>
__device__ __forceinline__ f32x4 load4<float>(const float *p) {
    return *reinterpret_cast<const f32x4 *>(p);
}
template <>
__device__ __forceinline__ f32x4 load4<uint16_t>(const uint16_t *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                 __uint_as_float(u.y & 0xFFFF0000u)};
}

template <typename T>
__device__ __forceinline__ void store4(T *p, f32x4 v);
template <>
__device__ __forceinline__ void store4<float>(float *p, f32x4 v) {
    *reinterpret_cast<f32x4 *>(p) = v;
}
template <>
__device__ __forceinline__ void store4<uint16_t>(uint16_t *p, f32x4 v) {
    uint2 u;
    u.x = uint32_t(f32_to_bf16_rne(v.x)) | (uint32_t(f32_to_bf16_rne(v.y)) << 16);
    u.y = uint32_t(f32_to_bf16_rne(v.z)) | (uint32_t(f32_to_bf16_rne(v.w)) << 16);
    *reinterpret_cast<uint2 *>(p) = u;
}

// Sum over the row's LPR lanes, the same on all of them.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
    v = group_sum<LPR < 16 ? LPR : 16>(v);
    if constexpr (LPR == 32) v += __shfl_xor(v, 16);
    return v;
}

// (a, b) rotated by (cos, sin); the pairs of a lane are (a[j], b[j]), or the
// neighbours within a and b where interleaved.
__device__ __forceinline__ void rotate(f32x4 &a, f32x4 &b, f32x4 c, f32x4 s, bool interleaved) {
    if (interleaved) {
        const f32x4 p = a, q = b;
        a.x = p.x * c.x - p.y * s.x;
        a.y = p.y * c.x + p.x * s.x;
        a.z = p.z * c.y - p.w * s.y;
        a.w = p.w * c.y + p.z * s.y;
        b.x = q.x * c.z - q.y * s.z;
        b.y = q.y * c.z + q.x * s.z;
        b.z = q.z * c.w - q.w * s.w;
        b.w = q.w * c.w + q.z * s.w;
    } else {
        const f32x4 p = a;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = p[j] * c[j] - b[j] * s[j];
            b[j] = b[j] * c[j] + p[j] * s[j];
        }
    }
}

// Cosines and sines of `n` tokens from t0 into LDS, [token][2][half].
__device__ __forceinline__ void fill_angles(const RopeArgs &a, float *cs, int64_t t0, int n) {
    for (int e = threadIdx.x; e < n * a.half; e += kRopeThreads) {
        const int t = e / a.half, i = e - t * a.half;
        double turn = double(a.positions[t0 + t]) * a.inv_freq[i] * 0.15915494309189533577;   // 1 / (2 pi)
        turn -= rint(turn);
        float s, c;
        sincospif(2.0f * float(turn), &s, &c);
        cs[(2 * t) * a.half + i] = c;
        cs[(2 * t + 1) * a.half + i] = s;
    }
}

template <bool ONCE, typename T>
__device__ __forceinline__ f32x4 load_row4(const T *p) {
    if constexpr (ONCE) return ld_stream_f4(reinterpret_cast<const float *>(p));   // T is float
    else return load4(p);
}

// BWD: 0 forward, 1 backward.  X: type of q, k (and dx); Y: type of y (and dy).
// ONCE: fp32 rows of more data than the 256 MB Infinity Cache are read with the
// hint not to keep them there: 503 MB forward 96 -> 81 us, backward 106 -> 90;
// 63 MB forward takes 15.9 us without the hint and 17.5 with it.
template <int LPR, typename X, typename Y, bool NORM, bool BWD, bool ONCE>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a) {
    extern __shared__ __align__(16) float cs[];
    constexpr int kRpw = 64 / LPR;                       // rows per wavefront
    constexpr int kStep = kRopeThreads / LPR;            // rows per workgroup and step
    const int lane = threadIdx.x & 63, l = lane & (LPR - 1);
    const int sub = (threadIdx.x >> 6) * kRpw + lane / LPR;
    const bool live = 8 * l < a.D;
    const bool rot = 4 * l < a.half;                     // this lane's elements are pairs
    // element offsets of the lane's two groups
    const int o0 = a.interleaved ? 8 * l : rot ? 4 * l : 2 * a.half + 8 * (l - a.half / 4);
    const int o1 = !a.interleaved && rot ? o0 + a.half : o0 + 4;
    f32x4 wq0 = {1.f, 1.f, 1.f, 1.f}, wq1 = wq0, wk0 = wq0, wk1 = wq0;
    if (NORM && live) {
        wq0 = load4(a.q.w + o0);
        wq1 = load4(a.q.w + o1);
        wk0 = load4(a.k.w + o0);
        wk1 = load4(a.k.w + o1);
    }
    f32x4 dq0 = {0.f, 0.f, 0.f, 0.f}, dq1 = dq0, dk0 = dq0, dk1 = dq0;   // this lane's part of dw

    const uint32_t H = a.heads.d;
    const int64_t r_first = int64_t(blockIdx.x) * a.rows_per_wg;
    const int64_t r_last = min(r_first + a.rows_per_wg, a.rows);
    // runs of rows whose tokens' angles fit the LDS
    for (int64_t r0 = r_first; r0 < r_last;) {
        const int64_t t0 = r0 / H;
        const int64_t r1 = min(r_last, (t0 + a.tokens_lds) * int64_t(H));
        if (r0 != r_first) __syncthreads();
        fill_angles(a, cs, t0, int((r1 - 1) / H - t0) + 1);
        __syncthreads();
        const uint32_t h0 = uint32_t(r0 - t0 * H);       // head of the run's first row
        for (int64_t r = r0 + sub; r < r1; r += kStep) {
            const uint32_t rel = h0 + uint32_t(r - r0);
            const uint32_t tl = fastdiv(rel, a.heads), h = rel - tl * H;
            const int64_t t = t0 + tl;
            const bool is_q = h < uint32_t(a.n_q);
            const RopeRows &m = is_q ? a.q : a.k;
            const int64_t hh = is_q ? h : h - a.n_q;
            f32x4 c = {1.f, 1.f, 1.f, 1.f}, s = {0.f, 0.f, 0.f, 0.f};
            if (rot) {
                c = *reinterpret_cast<const f32x4 *>(&cs[(2 * tl) * a.half + 4 * l]);
                s = *reinterpret_cast<const f32x4 *>(&cs[(2 * tl + 1) * a.half + 4 * l]);
            }
            f32x4 x0 = {0.f, 0.f, 0.f, 0.f}, x1 = x0, g0 = x0, g1 = x0;
            if (live) {
                if (!BWD || NORM) {
                    const X *x = static_cast<const X *>(m.x) + t * m.ld + hh * m.hs;
                    x0 = load_row4<ONCE>(x + o0);
                    x1 = load_row4<ONCE>(x + o1);
                }
                if (BWD) {
                    const Y *dy = static_cast<const Y *>(m.dy) + t * m.ldd + hh * m.hsd;
                    g0 = load_row4<ONCE && sizeof(Y) == 4>(dy + o0);
                    g1 = load_row4<ONCE && sizeof(Y) == 4>(dy + o1);
                }
            }
            float rn = 1.f;
            if constexpr (NORM) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) ss += x0[j] * x0[j] + x1[j] * x1[j];
                rn = 1.0f / sqrtf(row_sum<LPR>(ss) * a.inv_d + a.eps);
                x0 *= rn;
                x1 *= rn;
            }
            const f32x4 w0 = is_q ? wq0 : wk0, w1 = is_q ? wq1 : wk1;
            if constexpr (!BWD) {
                if constexpr (NORM) {
                    x0 *= w0;
                    x1 *= w1;
                }
                if (rot) rotate(x0, x1, c, s, a.interleaved != 0);
                if (live) {
                    Y *y = static_cast<Y *>(m.y) + t * m.ldy + hh * m.hsy;
                    store4(y + o0, x0);
                    store4(y + o1, x1);
                }
            } else {
                if (rot) rotate(g0, g1, c, -s, a.interleaved != 0);
                if constexpr (NORM) {
                    const f32x4 p0 = g0 * x0, p1 = g1 * x1;
                    if (is_q) { dq0 += p0; dq1 += p1; } else { dk0 += p0; dk1 += p1; }
                    float dot = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) dot += p0[j] * w0[j] + p1[j] * w1[j];
                    dot = row_sum<LPR>(dot) * a.inv_d;
                    g0 = (g0 * w0 - x0 * dot) * rn;
                    g1 = (g1 * w1 - x1 * dot) * rn;
                }
                if (live) {
                    X *y = static_cast<X *>(m.y) + t * m.ldy + hh * m.hsy;
                    store4(y + o0, g0);
                    store4(y + o1, g1);
                }
            }
        }
        r0 = r1;
    }
    if constexpr (BWD && NORM) {
        // sums of the workgroup: over the rows of a wavefront, then over the wavefronts, each in a fixed order
        __syncthreads();
        float *acc = cs;                                  // [4 wavefronts][2][LPR * 8]
        f32x4 v[4] = {dq0, dq1, dk0, dk1};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int d = LPR; d < 64; d <<= 1) v[i][j] += __shfl_xor(v[i][j], d);
        if (lane < LPR && live) {
            float *p = acc + (threadIdx.x >> 6) * 2 * a.D;
            *reinterpret_cast<f32x4 *>(p + o0) = v[0];
            *reinterpret_cast<f32x4 *>(p + o1) = v[1];
            *reinterpret_cast<f32x4 *>(p + a.D + o0) = v[2];
            *reinterpret_cast<f32x4 *>(p + a.D + o1) = v[3];
        }
        __syncthreads();
        for (int d = threadIdx.x; d < 2 * a.D; d += kRopeThreads) {
            float sum = 0.f;
            for (int w = 0; w < kRopeThreads / 64; ++w) sum += acc[w * 2 * a.D + d];
            if (gridDim.x > 1) a.dw_part[int64_t(blockIdx.x) * 2 * a.D + d] = sum;
            else (d < a.D ? a.dwq[d] : a.dwk[d - a.D]) = sum;
        }
    }
}

// dw from the workgroups' partial sums: 16 columns per workgroup, 64 threads
// per column over the partials in turn, then a tree: a fixed order.
__global__ __launch_bounds__(1024) void rope_dw_kernel(const float *part, int n, int D, float *dwq, float *dwk) {
    __shared__ float acc[64][17];
    const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
    const int d = int(blockIdx.x) * 16 + col;
    float s = 0.f;
#pragma unroll 8
    for (int i = row; i < n; i += 64) s += part[int64_t(i) * 2 * D + d];   // loads in flight together, added in order
    acc[row][col] = s;
    __syncthreads();
    for (int k = 32; k > 0; k >>= 1) {
        if (row < k) acc[row][col] += acc[row + k][col];
        __syncthreads();
    }
    if (row == 0) (d < D ? dwq[d] : dwk[d - D]) = acc[0][col];
}

template <int LPR, bool NORM, bool BWD>
void launch_rope(const RopeArgs &a, uint32_t grid, size_t lds, bool xb, bool yb, bool once, hipStream_t s) {
    if (xb && yb) rope_kernel<LPR, uint16_t, uint16_t, NORM, BWD, false><<<grid, kRopeThreads, lds, s>>>(a);
    else if (xb) rope_kernel<LPR, uint16_t, float, NORM, BWD, false><<<grid, kRopeThreads, lds, s>>>(a);
    else if (yb && once) rope_kernel<LPR, float, uint16_t, NORM, BWD, true><<<grid, kRopeThreads, lds, s>>>(a);
    else if (yb) rope_kernel<LPR, float, uint16_t, NORM, BWD, false><<<grid, kRopeThreads, lds, s>>>(a);
    else if (once) rope_kernel<LPR, float, float, NORM, BWD, true><<<grid, kRopeThreads, lds, s>>>(a);
    else rope_kernel<LPR, float, float, NORM, BWD, false><<<grid, kRopeThreads, lds, s>>>(a);
}

int lanes_per_row(int32_t D) { return D <= 64 ? 8 : D <= 128 ? 16 : 32; }

// Rows per workgroup and tokens whose angles it keeps in LDS at a time.
struct RopeShape {
    int32_t rows_per_wg, tokens;
    uint32_t grid;
};

RopeShape rope_shape(int64_t rows, int32_t H, int32_t D, int32_t half, bool bwd, int size) {
    const int step = kRopeThreads / lanes_per_row(D);
    // One step per workgroup while that gives few workgroups, then longer runs,
    // which share the angles of a token.  Backward, whose workgroups each leave a
    // partial sum of dw: 512 for fp32 input (8192 x 40 x 128: 106 us, with 1024
    // 109), 1024 for bf16, whose rows are half the bytes in flight (65 us, with
    // 512 94, with 2048 68).
    int64_t per = step;
    const int64_t want = !bwd ? 4096 : size == 4 ? 512 : 1024;
    if (rows > want * step) per = (rows + want * step - 1) / (want * step) * step;
    if (!bwd && per > 4 * step) per = 4 * step;
    while (rows / per >= (int64_t(1) << 22)) per *= 2;    // the launch's limit on threads
    int64_t tokens = (per + H - 2) / H + 1;               // most tokens a run of `per` rows touches
    const int64_t fit = (16 << 10) / (8 * half);          // 16 KiB of angles
    if (tokens > fit) tokens = fit;
    return RopeShape{int32_t(per), int32_t(tokens), uint32_t((rows + per - 1) / per)};
}

ht_status check_rope(int64_t T, int32_t n_q, int32_t n_k, int32_t D, int32_t rot) {
    if (T < 0 || n_q <= 0 || n_k < 0 || n_q > 4096 || n_k > 4096 || D <= 0 || D % 8 || D > 256 || rot < 0 || rot % 8 ||
        rot > D || T > (int64_t(1) << 36) || T * (int64_t(n_q) + n_k) >= (int64_t(1) << 40))
        return HT_ESHAPE;
    return HT_OK;
}

template <bool BWD>
ht_status run_rope(RopeArgs &a, int64_t T, int32_t n_q, int32_t n_k, int32_t D, int32_t rot, int32_t xt, int32_t yt,
                   hipStream_t s) {
    const bool norm = a.q.w != nullptr;
    a.rows = T * (int64_t(n_q) + n_k);
    a.heads = make_fastdiv(uint32_t(n_q + n_k));
    a.n_q = n_q;
    a.D = D;
    a.half = rot / 2;
    a.inv_d = 1.0f / float(D);
    const RopeShape sh = rope_shape(a.rows, n_q + n_k, D, a.half > 0 ? a.half : 4, BWD, act_size(xt));
    a.rows_per_wg = sh.rows_per_wg;
    a.tokens_lds = sh.tokens;
    size_t lds = size_t(sh.tokens) * 8 * size_t(a.half);
    if (BWD && norm) lds = lds > size_t(32) * D ? lds : size_t(32) * D;
    const bool xb = xt == HT_BF16, yb = yt == HT_BF16;
    const int lpr = lanes_per_row(D);
    const int64_t moved = a.rows * D * (act_size(xt) * (BWD && norm ? 2 : 1) + act_size(yt));
    const bool once = moved >= (int64_t(256) << 20);
    if (norm) {
        if (lpr == 8) launch_rope<8, true, BWD>(a, sh.grid, lds, xb, yb, once, s);
        else if (lpr == 16) launch_rope<16, true, BWD>(a, sh.grid, lds, xb, yb, once, s);
        else launch_rope<32, true, BWD>(a, sh.grid, lds, xb, yb, once, s);
    } else {
        if (lpr == 8) launch_rope<8, false, BWD>(a, sh.grid, lds, xb, yb, once, s);
        else if (lpr == 16) launch_rope<16, false, BWD>(a, sh.grid, lds, xb, yb, once, s);
        else launch_rope<32, false, BWD>(a, sh.grid, lds, xb, yb, once, s);
    }
    HT_LAUNCH_CHECK();
    if (BWD && norm && sh.grid > 1) {
        rope_dw_kernel<<<uint32_t(2 * D / 16), 1024, 0, s>>>(a.dw_part, int(sh.grid), D, a.dwq, a.dwk);
        HT_LAUNCH_CHECK();
    }
    return HT_OK;
}

}  // namespace
}  // namespace ht

using namespace ht;

#define HT_TRY(e)                       \
    do {                                \
        const ht_status st_ = (e);      \
        if (st_ != HT_OK) return st_;   \
    } while (0)

extern "C" ht_status ht_qk_norm_rope(const void *q, int64_t ldq, int64_t hsq, const void *k, int64_t ldk, int64_t hsk,
                                     int32_t xt, int64_t T, int32_t n_q, int32_t n_k, int32_t D, int32_t rot,
                                     int32_t interleaved, const int32_t *positions, const double *inv_freq,
                                     const float *wq, const float *wk, float eps, void *yq, int64_t ldyq,
                                     int64_t hsyq, void *yk, int64_t ldyk, int64_t hsyk, int32_t yt,
                                     ht_stream stream) {
    HT_TRY(check_rope(T, n_q, n_k, D, rot));
    if (!act_size(xt) || !act_size(yt) || (wq == nullptr) != (wk == nullptr) || !(eps >= 0.f)) return HT_EINVAL;
    if (T == 0) return HT_OK;
    HT_TRY(check_rows(q, ldq, hsq, n_q, D, act_size(xt)));
    HT_TRY(check_rows(yq, ldyq, hsyq, n_q, D, act_size(yt)));
    if (n_k) {
        HT_TRY(check_rows(k, ldk, hsk, n_k, D, act_size(xt)));
        HT_TRY(check_rows(yk, ldyk, hsyk, n_k, D, act_size(yt)));
    }
    if (rot && (!positions || !inv_freq)) return HT_EINVAL;
    if (!al4(positions) || !al16p(inv_freq) || !al16p(wq) || !al16p(wk)) return HT_EALIGN;
    RopeArgs a{};
    a.q = RopeRows{q, nullptr, yq, ldq, hsq, 0, 0, ldyq, hsyq, wq};
    a.k = RopeRows{k, nullptr, yk, ldk, hsk, 0, 0, ldyk, hsyk, wk};
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.interleaved = interleaved != 0;
    a.eps = eps;
    return run_rope<false>(a, T, n_q, n_k, D, rot, xt, yt, hipStream_t(stream));
}

extern "C" ht_status ht_qk_norm_rope_workspace(int64_t T, int32_t n_q, int32_t n_k, int32_t D, int32_t norm,
                                               size_t *bytes) {
    if (!bytes) return HT_EINVAL;
    HT_TRY(check_rope(T, n_q, n_k, D, 0));
    *bytes = 0;
    if (!norm || T == 0) return HT_OK;
    // the more workgroups of the two types of input
    const RopeShape sh = rope_shape(T * (int64_t(n_q) + n_k), n_q + n_k, D, 4, true, 2);
    if (sh.grid > 1) *bytes = size_t(sh.grid) * 2u * size_t(D) * sizeof(float);
    return HT_OK;
}

extern "C" ht_status ht_qk_norm_rope_backward(const void *dq, int64_t lddq, int64_t hsdq, const void *dk, int64_t lddk,
                                              int64_t hsdk, int32_t yt, const void *q, int64_t ldq, int64_t hsq,
                                              const void *k, int64_t ldk, int64_t hsk, int32_t xt, int64_t T,
                                              int32_t n_q, int32_t n_k, int32_t D, int32_t rot, int32_t interleaved,
                                              const int32_t *positions, const double *inv_freq, const float *wq,
                                              const float *wk, float eps, void *dxq, int64_t lddxq, int64_t hsdxq,
                                              void *dxk, int64_t lddxk, int64_t hsdxk, float *dwq, float *dwk,
                                              void *ws, size_t ws_bytes, ht_stream stream) {
    HT_TRY(check_rope(T, n_q, n_k, D, rot));
    if (!act_size(xt) || !act_size(yt) || (wq == nullptr) != (wk == nullptr) || !(eps >= 0.f)) return HT_EINVAL;
    const bool norm = wq != nullptr;
    if (norm && (!dwq || !dwk)) return HT_EINVAL;
    if (!al16p(dwq) || !al16p(dwk) || !al4(positions) || !al16p(inv_freq) || !al16p(wq) || !al16p(wk) || !al16p(ws))
        return HT_EALIGN;
    if (T > 0) {
        HT_TRY(check_rows(dq, lddq, hsdq, n_q, D, act_size(yt)));
        HT_TRY(check_rows(dxq, lddxq, hsdxq, n_q, D, act_size(xt)));
        if (norm) HT_TRY(check_rows(q, ldq, hsq, n_q, D, act_size(xt)));
        if (n_k) {
            HT_TRY(check_rows(dk, lddk, hsdk, n_k, D, act_size(yt)));
            HT_TRY(check_rows(dxk, lddxk, hsdxk, n_k, D, act_size(xt)));
            if (norm) HT_TRY(check_rows(k, ldk, hsk, n_k, D, act_size(xt)));
        }
        if (rot && (!positions || !inv_freq)) return HT_EINVAL;
        size_t need = 0;
        HT_TRY(ht_qk_norm_rope_workspace(T, n_q, n_k, D, norm, &need));
        if (need > 0 && (!ws || ws_bytes < need)) return HT_ESMALL;
    }
    if (T == 0) {   // no rows: the weights' gradients are zero (a sum over no partials)
        if (norm) {
            rope_dw_kernel<<<uint32_t(2 * D / 16), 1024, 0, hipStream_t(stream)>>>(nullptr, 0, D, dwq, dwk);
            HT_LAUNCH_CHECK();
        }
        return HT_OK;
    }
    RopeArgs a{};
    a.q = RopeRows{q, dq, dxq, ldq, hsq, lddq, hsdq, lddxq, hsdxq, wq};
    a.k = RopeRows{k, dk, dxk, ldk, hsk, lddk, hsdk, lddxk, hsdxk, wk};
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.dw_part = static_cast<float *>(ws);
    a.dwq = dwq;
    a.dwk = dwk;
    a.interleaved = interleaved != 0;
    a.eps = eps;
    return run_rope<true>(a, T, n_q, n_k, D, rot, xt, yt, hipStream_t(stream));
}
