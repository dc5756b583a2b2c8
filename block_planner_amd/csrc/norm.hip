// norm.hip -- the residual's addition and the root-mean-square norm between two
// layers in one pass, its output as the next linear takes it (fp32, bfloat16
// or 8-bit rows), its backward pass, and 8-bit rows read back.
//
//   h = x + res;  r = 1 / sqrt(mean(h^2) + eps);  y = h r w
//   backward, with g = w dy:  d = dh + r g - h r^3 / K sum(g h),
//   dw = sum over rows of dy h r.
//
// Bound by HBM: a few fp32 operations per 16 bytes.  A row is held in
// registers (8 consecutive values per thread and group), so its sum of squares
// costs no second read: by one wavefront up to 2048 columns (four rows per
// workgroup, no barrier), by 256 threads up to 8192, by 1024 above.
//   8192 x 4096 fp32 + fp32 -> bf16: 73 us, 6.5 TB/s;  one row: 2.5 us;
//   3001 x 2048 fp32 + bf16 -> 8 bits: 14.0 us (256 threads a row: the same);
//   backward, 8192 x 2048 fp32: 49 us, 4.6 of them for dw's parts.
// Loads and stores are the buffer's, which need no branch at a row's end: all of a
// row's are in flight at once (16384 x 4096 bf16 backward: 130 -> 111 us).
#include <type_traits>

#include "rows.h"

namespace ht {

namespace {

constexpr int64_t kNormMaxK = 32768;
constexpr int kQ8MinExp = -119;   // a block's scale, 2^(E-7), stays a normal number

struct NormArgs {
    const void *x, *res;
    void *h, *y;
    int64_t ldx, ldr, ldh, ldy;
    const float *w;
    uint8_t *codes;          // 8-bit rows, or null
    float *scales;
    int64_t M, Mp;           // Mp = 16 * groups
    int32_t K, y_bf16;
    float eps, inv_k;
};

__device__ __forceinline__ double wave_sum(double v) {
    v += dpp_f64<kDppXor1>(v);
    v += dpp_f64<kDppXor2>(v);
    v += dpp_f64<kDppHalfMirror>(v);
    v += dpp_f64<kDppMirror>(v);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

// Sum over the row's TPR threads (a wavefront, or the workgroup).
template <int TPR, typename F>
__device__ __forceinline__ F row_total(F v, F *part) {
    v = wave_sum(v);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) v += part[i];
    }
    return v;
}

// Largest over the 64-wide block's 8 lanes.
__device__ __forceinline__ uint32_t block_top(uint32_t v) {
    v = max(v, dpp_u32<kDppXor1>(v));
    v = max(v, dpp_u32<kDppXor2>(v));
    return max(v, dpp_u32<kDppHalfMirror>(v));
}
__device__ __forceinline__ uint64_t block_top(uint64_t v) {
    const auto other = [&](auto ctrl) {
        constexpr int kCtrl = decltype(ctrl)::value;
        return (uint64_t(dpp_u32<kCtrl>(uint32_t(v >> 32))) << 32) | dpp_u32<kCtrl>(uint32_t(v));
    };
    v = max(v, other(std::integral_constant<int, kDppXor1>{}));
    v = max(v, other(std::integral_constant<int, kDppXor2>{}));
    return max(v, other(std::integral_constant<int, kDppHalfMirror>{}));
}

// The row's 8 values h r w of one lane as codes; the 64-wide block's 8 lanes share
// the scale.  The codes are those of 64 bits (r is in 64 bits; in 32 the norm's
// rounding moves about one code in 10^5 across a border, by a whole step), worked
// out in 32 where that is certain (3001 x 2048 of fp32 + bf16: 14.0 us; all in 64
// bits 16.8; 32 alone 12.4).  A scaled value, of at most 128, is off by 4 steps of
// 2^-24, under 2^-14, so those within 2^-13 of a half are worked out again, and so are
// blocks whose largest value is within 16 steps of a power of two or far from 1, or
// whose r or w would make h r lose digits below fp32's normal numbers that the result
// still shows (2^-150 2^20 of a largest value of 2^-100: 2^-23 of a step).  The
// largest magnitude's bits, compared as whole numbers, tell a block that holds Inf or
// NaN too.
__device__ __forceinline__ void encode8(const Row8 &h, const Row8 &w, double r, const NormArgs &a, int64_t m, int col, bool live) {
    float y[8];
    const float rn = float(r);
    uint32_t top = 0, wtop = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        y[j] = h.v[j] * rn * w.v[j];
        top = max(top, __float_as_uint(y[j]) & 0x7FFFFFFFu);
        wtop = max(wtop, __float_as_uint(w.v[j]) & 0x7FFFFFFFu);
    }
    top = block_top(top);
    const uint32_t digits = top & 0x7FFFFFu;
    bool bad = false;
    int E = 7, q[8];
    // from 2^-100 to 2^100, not at a power of two: 32 bits give the exponent
    const bool sure = top >= 0x0D800000u && top < 0x71800000u && digits >= 16 && digits <= 0x7FFFEFu &&
                      wtop < 0x49800000u && rn >= 0x1p-100f;
    if (__all(!live || sure)) {
        if (live) E = int(top >> 23) - 126;                        // 2^(E-1) <= top < 2^E
        bool near = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = ldexpf(y[j], 7 - E), n = rintf(v);
            near = near || fabsf(v - n) > 0.5f - 0x1p-13f;
            q[j] = int(n);
        }
        if (__any(near)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = ldexpf(y[j], 7 - E);
                if (fabsf(v - rintf(v)) > 0.5f - 0x1p-13f) q[j] = int(rint(ldexp(double(h.v[j]) * r * double(w.v[j]), 7 - E)));
            }
        }
    } else {
        double z[8];
        uint64_t most = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            z[j] = double(h.v[j]) * r * double(w.v[j]);
            most = max(most, uint64_t(__double_as_longlong(z[j])) & 0x7FFFFFFFFFFFFFFFull);
        }
        most = block_top(most);
        bad = !(float(__longlong_as_double((long long)most)) <= 3.402823466e+38f);
        if (most > 0 && !bad) E = max(int(most >> 52) - 1022, kQ8MinExp);
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = bad ? 0 : int(rint(ldexp(z[j], 7 - E)));
    }
    if (!live) return;
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j >> 2] |= (uint32_t(min(max(q[j], -127), 127)) & 0xFFu) << (8 * (j & 3));
    const int64_t g = m >> 4;
    const uint32_t i = uint32_t(m) & 15u, kb = uint32_t(col) >> 6, e = uint32_t(col) & 63u;
    uint8_t *dst = a.codes + (g * (a.K / 64) + kb) * 1024 + 16u * (i + 16u * (e >> 4)) + (e & 15u);
    *reinterpret_cast<u32x2 *>(dst) = u32x2{c[0], c[1]};
    if (e == 0) a.scales[int64_t(kb) * a.Mp + m] = bad ? __builtin_nanf("") : ldexpf(1.0f, E - 7);
}

// The columns of a thread's group g of 8 in a row of TPR threads: 8 consecutive
// ones, or (QUAD, where an operand is fp32) 4 and 4 half the row's group further, so
// that a wavefront's 16-byte loads lie side by side: 8192 x 4096 fp32 -> bf16 88 ->
// 83 us.  ONCE: where the matrices are more than the 256 MB Infinity Cache they are
// not read with a view to the caches: 83 -> 73 (6.5 TB/s), 16384 x 4096 bf16 95 -> 83, but
// 49 -> 52 for a backward pass of 268 MB (stores with the same hint: slower).
template <int TPR, bool QUAD, bool ONCE>
struct Cols {
    static __device__ __forceinline__ int lo(int t, int g) { return QUAD ? 8 * TPR * g + 4 * t : 8 * (t + TPR * g); }
    static __device__ __forceinline__ int hi(int t, int g) { return lo(t, g) + (QUAD ? 4 * TPR : 4); }

    template <typename T>
    static __device__ __forceinline__ Row8 load(const RowBuf<T> &p, int t, int g) {
        return p.template load<!QUAD, ONCE>(lo(t, g), hi(t, g));
    }
    template <typename T>
    static __device__ __forceinline__ void store(const RowBuf<T> &p, const Row8 &r, int t, int g) {
        p.template store<!QUAD>(lo(t, g), hi(t, g), r);
    }
};

template <int TPR, int NV, typename X, typename R, bool RES, bool Q8, bool ONCE>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_kernel(NormArgs a) {
    using F = std::conditional_t<Q8, double, float>;
    constexpr bool kQuad = !Q8 && (sizeof(X) == 4 || (RES && sizeof(R) == 4));
    using In = Cols<TPR, kQuad, ONCE>;
    using Kept = Cols<TPR, kQuad, false>;
    constexpr int kRows = TPR >= 256 ? 1 : 256 / TPR;
    __shared__ F part[16];
    const int t = threadIdx.x & (TPR - 1);
    uint32_t b = blockIdx.x;
    // 8-bit rows: the 16 rows of a group share cache lines, so neighbouring
    // workgroups are placed on one XCD (workgroups go to the 8 XCDs in turn)
    if (Q8 && (gridDim.x & 7u) == 0) b = (b & 7u) * (gridDim.x >> 3) + (b >> 3);
    const int64_t m = int64_t(b) * kRows + __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
    if (m >= a.M) return;    // whole wavefronts (TPR = 64), never part of a workgroup that meets at a barrier
    const RowBuf<X> x(static_cast<const X *>(a.x) + m * a.ldx, a.K);
    const RowBuf<R> res(static_cast<const R *>(a.res) + m * a.ldr, a.K);
    const RowBuf<float> wb(a.w, a.K);
    Row8 v[NV];
    F ss = 0;
#pragma unroll
    for (int g = 0; g < NV; ++g) {
        v[g] = In::load(x, t, g);
        if constexpr (RES) {
            const Row8 r = In::load(res, t, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[g].v[j] += r.v[j];
        }
    }
    if constexpr (RES) {
        // the norm sees h as it is stored: the backward pass, which has h, differentiates what was computed
#pragma unroll
        for (int g = 0; g < NV; ++g) {
            if constexpr (sizeof(R) == 2) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[g].v[j] = __uint_as_float(uint32_t(round_bf16(v[g].v[j])) << 16);
            }
            if (a.h) Kept::store(RowBuf<R>(static_cast<R *>(a.h) + m * a.ldh, a.K), v[g], t, g);
        }
    }
#pragma unroll
    for (int g = 0; g < NV; ++g)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += F(v[g].v[j]) * F(v[g].v[j]);
    ss = row_total<TPR>(ss, part);
    const auto put = [&](int g, const Row8 &o) {
        if (a.y_bf16) Kept::store(RowBuf<uint16_t>(static_cast<uint16_t *>(a.y) + m * a.ldy, a.K), o, t, g);
        else Kept::store(RowBuf<float>(static_cast<float *>(a.y) + m * a.ldy, a.K), o, t, g);
    };
    if constexpr (Q8) {
        const double rn = 1.0 / sqrt(ss / a.K + double(a.eps));
#pragma unroll
        for (int g = 0; g < NV; ++g) {
            const int c = Kept::lo(t, g);
            const Row8 w = Kept::load(wb, t, g);
            if (a.y) {
                Row8 o;
#pragma unroll
                for (int j = 0; j < 8; ++j) o.v[j] = v[g].v[j] * float(rn) * w.v[j];
                put(g, o);
            }
            encode8(v[g], w, rn, a, m, c, c < a.K);
        }
    } else {
        const float rn = 1.0f / sqrtf(ss * a.inv_k + a.eps);
#pragma unroll
        for (int g = 0; g < NV; ++g) {
            const Row8 w = Kept::load(wb, t, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[g].v[j] = v[g].v[j] * rn * w.v[j];
            put(g, v[g]);
        }
    }
}

struct NormBwdArgs {
    const void *dy, *h, *dh;
    void *dres, *dx;         // in h's type; in the other type, or null
    int64_t lddy, ldh, lddh, lddres, lddx;
    const float *w;
    float *part;             // [gridDim.x][K], or dw itself where one workgroup does it all
    int64_t M;
    int32_t K;
    float eps, inv_k;
};

// A workgroup takes every gridDim.x-th set of rows and keeps its part of dw in
// registers; the parts are added by norm_dw_kernel in a fixed order, all in fp32: 16
// rows a part and then a tree, 1.1e-7 of dw's size off at 8192 rows.
template <int TPR, int NV, typename Y, typename H, bool ONCE>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_bwd_kernel(NormBwdArgs a) {
    constexpr bool kQuad = sizeof(Y) == 4 || sizeof(H) == 4;
    using In = Cols<TPR, kQuad, ONCE>;
    using Kept = Cols<TPR, kQuad, false>;
    constexpr int kRows = TPR >= 256 ? 1 : 256 / TPR;
    __shared__ float part[2][32];
    extern __shared__ __align__(16) float acc[];     // TPR = 64: [4][K]
    const int t = threadIdx.x & (TPR - 1);
    const int sub = __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
    const RowBuf<float> wb(a.w, a.K);
    Row8 w[NV], dw[NV];
#pragma unroll
    for (int g = 0; g < NV; ++g) {
        w[g] = Kept::load(wb, t, g);
        dw[g] = Row8{};
    }
    int at = 0;
    for (int64_t m0 = int64_t(blockIdx.x) * kRows; m0 < a.M; m0 += int64_t(gridDim.x) * kRows) {
        const int64_t m = m0 + sub;
        if (kRows > 1 && m >= a.M) break;            // a wavefront of its own: no barrier inside the loop
        const RowBuf<H> hp(static_cast<const H *>(a.h) + m * a.ldh, a.K);
        const RowBuf<Y> yp(static_cast<const Y *>(a.dy) + m * a.lddy, a.K);
        Row8 h[NV], dy[NV];
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int g = 0; g < NV; ++g) {
            h[g] = In::load(hp, t, g);
            dy[g] = In::load(yp, t, g);
        }
#pragma unroll
        for (int g = 0; g < NV; ++g)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ss += h[g].v[j] * h[g].v[j];
                dot += dy[g].v[j] * w[g].v[j] * h[g].v[j];
            }
        ss = wave_sum(ss);
        dot = wave_sum(dot);
        if constexpr (TPR > 64) {
            float *p = part[at];
            at ^= 1;                                 // two sets in turn: one barrier a row
            if ((threadIdx.x & 63) == 0) {
                p[threadIdx.x >> 6] = ss;
                p[16 + (threadIdx.x >> 6)] = dot;
            }
            __syncthreads();
            ss = dot = 0.f;
#pragma unroll
            for (int i = 0; i < TPR / 64; ++i) {
                ss += p[i];
                dot += p[16 + i];
            }
        }
        const float rn = 1.0f / sqrtf(ss * a.inv_k + a.eps);
        const float k = dot * a.inv_k * rn * rn;     // d = dh + r (g - h k)
#pragma unroll
        for (int g = 0; g < NV; ++g) {
            Row8 d;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[g].v[j] += dy[g].v[j] * (h[g].v[j] * rn);
                d.v[j] = rn * (dy[g].v[j] * w[g].v[j] - h[g].v[j] * k);
            }
            if (a.dh) {
                const Row8 e = In::load(RowBuf<H>(static_cast<const H *>(a.dh) + m * a.lddh, a.K), t, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) d.v[j] += e.v[j];
            }
            Kept::store(RowBuf<H>(static_cast<H *>(a.dres) + m * a.lddres, a.K), d, t, g);
            if (a.dx) {
                if constexpr (sizeof(H) == 4) Kept::store(RowBuf<uint16_t>(static_cast<uint16_t *>(a.dx) + m * a.lddx, a.K), d, t, g);
                else Kept::store(RowBuf<float>(static_cast<float *>(a.dx) + m * a.lddx, a.K), d, t, g);
            }
        }
    }
    float *out = a.part + int64_t(blockIdx.x) * a.K;
    if constexpr (kRows > 1) {
#pragma unroll
        for (int g = 0; g < NV; ++g) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = (j < 4 ? Kept::lo(t, g) : Kept::hi(t, g) - 4) + j;
                if (c < a.K) acc[sub * a.K + c] = dw[g].v[j];
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.K; c += 256) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < kRows; ++i) s += acc[i * a.K + c];
            out[c] = s;
        }
    } else {
#pragma unroll
        for (int g = 0; g < NV; ++g) Kept::store(RowBuf<float>(out, a.K), dw[g], t, g);
    }
}

// dw from the workgroups' parts: 16 columns per workgroup, 64 threads per
// column over the parts in turn, then a tree: a fixed order.
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float *part, int n, int K, float *dw) {
    __shared__ float acc[64][17];
    const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
    const int c = int(blockIdx.x) * 16 + col;
    float s = 0.f;
    if (c < K) {
#pragma unroll 8
        for (int i = row; i < n; i += 64) s += part[int64_t(i) * K + c];
    }
    acc[row][col] = s;
    __syncthreads();
    for (int k = 32; k > 0; k >>= 1) {
        if (row < k) acc[row][col] += acc[row + k][col];
        __syncthreads();
    }
    if (row == 0 && c < K) dw[c] = acc[0][col];
}

// 8-bit rows as the values they stand for: a wavefront turns one 1 KiB record
// (16 rows x 64 columns) round, each lane 16 codes of one row.  3001 x 2048: 6.3 us
// (18.5 MB, 2.9 TB/s: one pair of loads in flight per wavefront).
template <typename Y>
__global__ __launch_bounds__(256) void q8_values_kernel(const uint8_t *codes, const float *scales, int64_t M, int64_t Mp,
                                                        uint32_t KB, int64_t records, Y *y, int64_t ldy) {
    const int64_t rec = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (rec >= records) return;
    const uint32_t lane = threadIdx.x & 63;
    const int64_t g = rec / KB;
    const uint32_t kb = uint32_t(rec - g * KB);
    const int64_t m = 16 * g + (lane & 15u);
    if (m >= M) return;
    const u32x4 u = reinterpret_cast<const u32x4 *>(codes + rec * 1024)[lane];
    const float s = scales[int64_t(kb) * Mp + m];
    Y *p = y + m * ldy + 64u * kb + 16u * (lane >> 4);
    Row8 a, b;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        a.v[j] = float(int8_t(u[j >> 2] >> (8 * (j & 3)))) * s;
        b.v[j] = float(int8_t(u[2 + (j >> 2)] >> (8 * (j & 3)))) * s;
    }
    store8(p, a);
    store8(p + 8, b);
}

template <int TPR, int NV, bool Q8, bool ONCE>
void launch_norm_as(const NormArgs &a, int32_t xt, int32_t rt, hipStream_t s) {
    constexpr int kThreads = TPR > 256 ? TPR : 256, kRows = TPR >= 256 ? 1 : 256 / TPR;
    const uint32_t grid = uint32_t((a.M + kRows - 1) / kRows);
    const bool xb = xt == HT_BF16, rb = rt == HT_BF16;
    if (!a.res) {
        if (xb) norm_kernel<TPR, NV, uint16_t, float, false, Q8, ONCE><<<grid, kThreads, 0, s>>>(a);
        else norm_kernel<TPR, NV, float, float, false, Q8, ONCE><<<grid, kThreads, 0, s>>>(a);
    } else if (xb) {
        if (rb) norm_kernel<TPR, NV, uint16_t, uint16_t, true, Q8, ONCE><<<grid, kThreads, 0, s>>>(a);
        else norm_kernel<TPR, NV, uint16_t, float, true, Q8, ONCE><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (rb) norm_kernel<TPR, NV, float, uint16_t, true, Q8, ONCE><<<grid, kThreads, 0, s>>>(a);
        else norm_kernel<TPR, NV, float, float, true, Q8, ONCE><<<grid, kThreads, 0, s>>>(a);
    }
}

template <int TPR, int NV>
void launch_norm(const NormArgs &a, bool once, int32_t xt, int32_t rt, hipStream_t s) {
    if (a.codes) launch_norm_as<TPR, NV, true, false>(a, xt, rt, s);
    else if (once) launch_norm_as<TPR, NV, false, true>(a, xt, rt, s);
    else launch_norm_as<TPR, NV, false, false>(a, xt, rt, s);
}

template <int TPR, int NV, bool ONCE>
void launch_norm_bwd_as(const NormBwdArgs &a, uint32_t grid, int32_t yt, int32_t ht, hipStream_t s) {
    constexpr int kThreads = TPR > 256 ? TPR : 256, kRows = TPR >= 256 ? 1 : 256 / TPR;
    const size_t lds = kRows > 1 ? size_t(kRows) * size_t(a.K) * 4 : 0;
    const bool yb = yt == HT_BF16, hb = ht == HT_BF16;
    if (yb && hb) norm_bwd_kernel<TPR, NV, uint16_t, uint16_t, ONCE><<<grid, kThreads, lds, s>>>(a);
    else if (yb) norm_bwd_kernel<TPR, NV, uint16_t, float, ONCE><<<grid, kThreads, lds, s>>>(a);
    else if (hb) norm_bwd_kernel<TPR, NV, float, uint16_t, ONCE><<<grid, kThreads, lds, s>>>(a);
    else norm_bwd_kernel<TPR, NV, float, float, ONCE><<<grid, kThreads, lds, s>>>(a);
}

template <int TPR, int NV>
void launch_norm_bwd(const NormBwdArgs &a, bool once, uint32_t grid, int32_t yt, int32_t ht, hipStream_t s) {
    if (once) launch_norm_bwd_as<TPR, NV, true>(a, grid, yt, ht, s);
    else launch_norm_bwd_as<TPR, NV, false>(a, grid, yt, ht, s);
}

// The instance for K columns: threads per row and groups of 8 per thread.
#define HT_NORM_SHAPES(K, CALL)           \
    do {                                  \
        if (K <= 512) CALL(64, 1);        \
        else if (K <= 1024) CALL(64, 2);  \
        else if (K <= 2048) CALL(64, 4);  \
        else if (K <= 4096) CALL(256, 2); \
        else if (K <= 8192) CALL(256, 4); \
        else if (K <= 16384) CALL(1024, 2); \
        else CALL(1024, 4);               \
    } while (0)

// A call's matrices, `bytes` per entry together, are more than the Infinity Cache holds.
bool past_caches(int64_t M, int64_t K, int bytes) { return M * K * bytes > (int64_t(256) << 20); }

// Workgroups of the backward pass.  768 where h is bfloat16 and a row takes 256 threads
// of two groups: 16384 x 4096 bf16 95 us (512: 111, 1024: 99); fp32, 8192 x 4096: 94 (512: 90).
uint32_t norm_bwd_grid(int64_t M, int64_t K, bool bf16) {
    const int64_t rows = K <= 2048 ? 4 : 1, most = K > 8192 ? 256 : bf16 && K > 2048 && K <= 4096 ? 768 : 512;
    const int64_t sets = (M + rows - 1) / rows;
    return uint32_t(sets < most ? sets : most);
}

ht_status check_norm(int64_t M, int64_t K) {
    if (M < 0 || M > (int64_t(1) << 30) || K <= 0 || K % 8 || K > kNormMaxK) return HT_ESHAPE;
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

extern "C" ht_status ht_q8_bytes(int64_t M, int64_t K, size_t *codes, size_t *scales) {
    if (!codes || !scales) return HT_EINVAL;
    HT_TRY(check_q8_shape(M, K));
    *codes = size_t(q8_groups(M)) * size_t(K / 64) * 1024;
    *scales = size_t(q8_groups(M)) * size_t(K / 64) * 16 * sizeof(float);
    return HT_OK;
}

extern "C" ht_status ht_q8_values(const ht_q8_rows *q, void *y, int64_t ldy, int32_t yt, ht_stream stream) {
    if (!q || !act_size(yt)) return HT_EINVAL;
    HT_TRY(check_q8_shape(q->M, q->K));
    if (q->M == 0) return HT_OK;
    HT_TRY(check_q8(q));
    HT_TRY(check_matrix(y, ldy, q->M, q->K, act_size(yt)));
    const uint32_t KB = uint32_t(q->K / 64);
    const int64_t records = q8_groups(q->M) * KB;
    if ((records + 3) / 4 >= (int64_t(1) << 24)) return HT_ESHAPE;   // the launch's limit on threads
    const uint32_t grid = uint32_t((records + 3) / 4);
    const hipStream_t s = hipStream_t(stream);
    const uint8_t *codes = reinterpret_cast<const uint8_t *>(q->codes);
    const int64_t Mp = 16 * q8_groups(q->M);
    if (yt == HT_BF16) q8_values_kernel<<<grid, 256, 0, s>>>(codes, q->scales, q->M, Mp, KB, records, static_cast<uint16_t *>(y), ldy);
    else q8_values_kernel<<<grid, 256, 0, s>>>(codes, q->scales, q->M, Mp, KB, records, static_cast<float *>(y), ldy);
    HT_LAUNCH_CHECK();
    return HT_OK;
}

extern "C" ht_status ht_add_rms_norm(const void *x, int64_t ldx, int32_t xt, const void *res, int64_t ldr, int32_t rt,
                                     int64_t M, int64_t K, const float *w, float eps, void *h, int64_t ldh, void *y,
                                     int64_t ldy, int32_t yt, const ht_q8_rows *q, ht_stream stream) {
    HT_TRY(check_norm(M, K));
    if (!act_size(xt) || (res && !act_size(rt)) || (y && !act_size(yt)) || !(eps >= 0.f)) return HT_EINVAL;
    if (q && (q->M != M || q->K != K)) return HT_ESHAPE;
    if (M == 0) return HT_OK;
    if ((!y && !q) || (h && !res)) return HT_EINVAL;
    HT_TRY(check_matrix(x, ldx, M, K, act_size(xt)));
    if (res) HT_TRY(check_matrix(res, ldr, M, K, act_size(rt)));
    if (h) HT_TRY(check_matrix(h, ldh, M, K, act_size(rt)));
    if (y) HT_TRY(check_matrix(y, ldy, M, K, act_size(yt)));
    if (q) HT_TRY(check_q8(q));
    if (!w) return HT_EINVAL;
    if (!al16p(w)) return HT_EALIGN;
    if (M >= (int64_t(1) << 22)) return HT_ESHAPE;   // the launch's limit on threads (1024 a row)
    NormArgs a{};
    a.x = x;
    a.res = res;
    a.h = h;
    a.y = y;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldh = ldh;
    a.ldy = ldy;
    a.w = w;
    if (q) {
        a.codes = reinterpret_cast<uint8_t *>(q->codes);
        a.scales = q->scales;
    }
    a.M = M;
    a.Mp = 16 * q8_groups(M);
    a.K = int32_t(K);
    a.y_bf16 = yt == HT_BF16;
    a.eps = eps;
    a.inv_k = 1.0f / float(K);
    const hipStream_t s = hipStream_t(stream);
    const bool once = past_caches(M, K, act_size(xt) + (res ? act_size(rt) : 0) + (h ? act_size(rt) : 0) + (y ? act_size(yt) : 1));
#define HT_NORM_CALL(T, V) launch_norm<T, V>(a, once, xt, rt, s)
    HT_NORM_SHAPES(K, HT_NORM_CALL);
#undef HT_NORM_CALL
    HT_LAUNCH_CHECK();
    return HT_OK;
}

extern "C" ht_status ht_add_rms_norm_workspace(int64_t M, int64_t K, size_t *bytes) {
    if (!bytes) return HT_EINVAL;
    HT_TRY(check_norm(M, K));
    const uint32_t grid = norm_bwd_grid(M, K, true);     // the larger of both types'
    *bytes = grid > 1 ? size_t(grid) * size_t(K) * sizeof(float) : 0;
    return HT_OK;
}

extern "C" ht_status ht_add_rms_norm_backward(const void *dy, int64_t lddy, int32_t yt, const void *h, int64_t ldh,
                                              int32_t ht, const void *dh, int64_t lddh, int64_t M, int64_t K,
                                              const float *w, float eps, void *dres, int64_t lddres, void *dx,
                                              int64_t lddx, float *dw, void *ws, size_t ws_bytes, ht_stream stream) {
    HT_TRY(check_norm(M, K));
    if (!act_size(yt) || !act_size(ht) || !(eps >= 0.f) || !w || !dw) return HT_EINVAL;
    if (!al16p(w) || !al16p(dw) || !al16p(ws)) return HT_EALIGN;
    const hipStream_t s = hipStream_t(stream);
    if (M > 0) {
        const int size = act_size(ht);
        HT_TRY(check_matrix(dy, lddy, M, K, act_size(yt)));
        HT_TRY(check_matrix(h, ldh, M, K, size));
        if (dh) HT_TRY(check_matrix(dh, lddh, M, K, size));
        HT_TRY(check_matrix(dres, lddres, M, K, size));
        if (dx) HT_TRY(check_matrix(dx, lddx, M, K, 6 - size));
        size_t need = 0;
        HT_TRY(ht_add_rms_norm_workspace(M, K, &need));
        if (need && (!ws || ws_bytes < need)) return HT_ESMALL;
        const uint32_t grid = norm_bwd_grid(M, K, ht == HT_BF16);
        NormBwdArgs a{};
        a.dy = dy;
        a.h = h;
        a.dh = dh;
        a.dres = dres;
        a.dx = dx;
        a.lddy = lddy;
        a.ldh = ldh;
        a.lddh = lddh;
        a.lddres = lddres;
        a.lddx = lddx;
        a.w = w;
        a.part = grid > 1 ? static_cast<float *>(ws) : dw;
        a.M = M;
        a.K = int32_t(K);
        a.eps = eps;
        a.inv_k = 1.0f / float(K);
        const bool once = past_caches(M, K, act_size(yt) + (dh ? 3 : 2) * act_size(ht) + (dx ? 6 - act_size(ht) : 0));
#define HT_NORM_CALL(T, V) launch_norm_bwd<T, V>(a, once, grid, yt, ht, s)
        HT_NORM_SHAPES(K, HT_NORM_CALL);
#undef HT_NORM_CALL
        HT_LAUNCH_CHECK();
        if (grid == 1) return HT_OK;
        norm_dw_kernel<<<uint32_t((K + 15) / 16), 1024, 0, s>>>(static_cast<const float *>(ws), int(grid), int(K), dw);
    } else {
        norm_dw_kernel<<<uint32_t((K + 15) / 16), 1024, 0, s>>>(nullptr, 0, int(K), dw);   // no rows: zeros
    }
    HT_LAUNCH_CHECK();
    return HT_OK;
}
