// kv_attn.hip -- attention of a batch's query rows over the paged 8-bit cache.
//
//   o = sum_j w_j V_j / sum_j w_j,   w_j = 2^(x_j),   x_j = scale log2(e) q . K_j
//
// in one pass over the pages with a running maximum and sum.  A page's scales
// are powers of two, 2^(k) for K and 2^(v) for V: with codes c, K = c 2^k is a
// factor of the score and V = c 2^v an addend of the exponent, so that
// w_j V_j = 2^(x_j + v) c_j.  The maximum is that of y_j = x_j + v, the size of
// a token's contribution to o, and the weights go to the matrix cores as fp16
// relative to it (round to nearest; 11 bits for anything within 2^-26 of the
// largest contribution); the sum of the weights adds 2^(-v) times each page's.
// A heavy token with small values therefore does not push the others out of
// fp16's range.  Scores, maxima, sums and outputs are fp32.
//
// Rows of a request and the heads of a group that share a KV head are columns
// of one product, S^T = K Q^T, O^T = V^T P^T, so every page is read once per
// tile of columns.  Few columns (answers, drafts) and short calls:
// attn_decode_kernel, bound by HBM.  Many (prompts): attn_prompt_kernel, bound by
// the matrix and vector units.  A batch with both runs both, each on its
// requests.  Pages of one
// request are split over workgroups where that fills the card, and the
// partial results joined in their order: the result depends on the launch's
// hints by rounding only and is the same from run to run.
#include "kv.h"

namespace ht {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kAttnThreads = 256;
constexpr int kWaves = kAttnThreads / 64;
constexpr int64_t kJoinPages = 2, kWholePages = 24;
constexpr int kMaxSplits = 64;   // one per lane of the kernel that joins them
constexpr float kLog2e = 1.44269504088896341f;
// The weight of the running maximum, as handed to V: fp16 keeps 11 bits down to
// 2^-26 of it and has 2^-36 as its last bit.  The prompt kernel moves its
// maximum (and rescales its sums) only for a score kSlackLog2 above it: weights
// stay under 2^15.5, below fp16's 65504.
constexpr float kTopLog2 = 12.f, kSlackLog2 = 3.5f;
// Size of a maximum (log2 units) from which fp32 no longer holds a score, and its
// difference to the maximum plus kTopLog2, to the half unit that is left between
// 2^15.5 and 65504: the prompt kernel then takes the difference first.
constexpr float kFarLog2 = 0x1p20f;

struct AttnArgs {
    const uint16_t *q;
    const int8_t *codes;
    const float *scales;
    const int32_t *table, *cu_q, *kv_len;
    uint16_t *out;
    // results of splits, normalised, and the log2 of their weights' sums:
    // [splits][dec_rows][n_q] of the decode kernel's requests (rows by request,
    // dec_per_request each, or by T where that is 0), then [psplits][T][n_q]
    float *part, *lse;
    int64_t dec_rows, prompt_at;
    int32_t dec_per_request;
    int64_t ldq, hsq, ldo, hso, ldt, P;
    int32_t T, R, n_q, n_heads, group, n_pages, causal;
    int32_t splits, split_pages;     // of the decode kernel's requests
    int32_t psplits, psplit_pages;   // of the prompt kernel's
    int32_t prompt_from;             // columns from which a request is the prompt kernel's
    int64_t window;
    float scale_log2;   // |scale| * log2(e)
    float sign;         // of scale
};

// One request as the kernels see it: lengths clamped to the arrays.
struct Request {
    int32_t row0, rows, kv, p0, p1;   // pages [p0, p1) hold every token its rows may see
    int32_t splits, split_pages;
    bool prompt;                      // the prompt kernel's
};

// Columns (rows x heads of a group) of a request up to which the decode kernel
// takes it, where both kernels run.
constexpr int kDecodeCols = 32;
// Tiles of 16 columns times pages of a call up to which it runs alone (D <= 128),
// where requests are split.
constexpr int kDecodeVisits = 16384;

__device__ __forceinline__ Request load_request(const AttnArgs &a, int r) {
    Request q;
    q.row0 = min(max(a.cu_q[r], 0), a.T);
    q.rows = min(max(a.cu_q[r + 1] - q.row0, 0), a.T - q.row0);
    q.kv = int32_t(min(int64_t(max(a.kv_len[r], 0)), a.P * kPage));
    q.p1 = (q.kv + kPage - 1) / kPage;
    const int64_t first = a.window > 0 ? int64_t(q.kv) - q.rows + 1 - a.window : 0;   // first row's first token
    q.p0 = first > 0 ? min(int32_t(min(first / kPage, int64_t(q.p1))), q.p1) : 0;
    q.prompt = int64_t(q.rows) * a.group >= a.prompt_from;
    q.split_pages = q.prompt ? a.psplit_pages : a.split_pages;
    q.splits = min(max((q.p1 - q.p0 + q.split_pages - 1) / q.split_pages, 1), q.prompt ? a.psplits : a.splits);
    return q;
}

// Partial result of split 0 of a request's first row, head 0, and the step to the next split.
__device__ __forceinline__ int64_t partial_at(const AttnArgs &a, const Request &q, int r, int64_t &step) {
    step = (q.prompt ? int64_t(a.T) : a.dec_rows) * a.n_q;
    const int64_t row = q.prompt || a.dec_per_request == 0 ? q.row0 : int64_t(r) * a.dec_per_request;
    return (q.prompt ? a.prompt_at : 0) + row * a.n_q;
}

// Tokens row i of a request sees: [lo, hi).
__device__ __forceinline__ void row_range(const AttnArgs &a, const Request &q, int i, int &lo, int &hi) {
    const int64_t pos = int64_t(q.kv) - q.rows + i;
    hi = a.causal ? int(max(int64_t(0), min(int64_t(q.kv), pos + 1))) : q.kv;
    lo = a.window > 0 ? int(min(int64_t(q.kv), max(int64_t(0), pos + 1 - a.window))) : 0;
}

// Zeros for the rows of no request: those before the first request's by its
// workgroups, those past the last one's (a batch padded to a fixed number of rows)
// by the last one's, which know the border from their own lengths.
template <int D>
__device__ __forceinline__ void clear_rows(const AttnArgs &a, const Request &rq, int r, int head) {
    if (r != 0 && r != a.R - 1) return;
    const int32_t before = r == 0 ? rq.row0 : 0, last = r == a.R - 1 ? rq.row0 + rq.rows : a.T;
    if (before == 0 && last == a.T) return;
    const int64_t per = int64_t(a.n_q) * (D / 8), n = (before + int64_t(a.T - last)) * per;
    const int64_t wg = (int64_t(blockIdx.z) * gridDim.y + blockIdx.y) * a.n_heads + head;
    const int64_t step = int64_t(gridDim.z) * gridDim.y * a.n_heads * blockDim.x;
    for (int64_t i = wg * blockDim.x + threadIdx.x; i < n; i += step) {
        int64_t row = i / per;
        const int64_t in = i - row * per, h = in / (D / 8), d = in % (D / 8) * 8;
        if (row >= before) row += last - before;
        *reinterpret_cast<uint4 *>(a.out + row * a.ldo + h * a.hso + d) = uint4{0, 0, 0, 0};
    }
}

// Eight codes as fp16, exactly: a byte c + 128 under the exponent of 1024 is 1152 + c.
__device__ __forceinline__ f16x8 codes_to_f16(uint32_t w0, uint32_t w1) {
    union { uint32_t u[4]; f16x2 h[4]; f16x8 v; } r;
    const uint32_t b0 = w0 ^ 0x80808080u, b1 = w1 ^ 0x80808080u;
    r.u[0] = __builtin_amdgcn_perm(0x64646464u, b0, 0x04010400u);
    r.u[1] = __builtin_amdgcn_perm(0x64646464u, b0, 0x04030402u);
    r.u[2] = __builtin_amdgcn_perm(0x64646464u, b1, 0x04010400u);
    r.u[3] = __builtin_amdgcn_perm(0x64646464u, b1, 0x04030402u);
    const f16x2 bias = {_Float16(1152.f), _Float16(1152.f)};
#pragma unroll
    for (int i = 0; i < 4; ++i) r.h[i] -= bias;
    return r.v;
}

template <bool ONCE>
__device__ __forceinline__ i32x4 load_codes(const int8_t *p) {
    if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const i32x4 *>(p));
    else return *reinterpret_cast<const i32x4 *>(p);
}

// Larger of lane i's and lane i + 32's (i - 32's) value.
__device__ __forceinline__ float max_halves(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// 16 elements of a row of q as three int8 planes with n = rne(x 2^(22-E)) =
// 65536 p[0] + 256 p[1] + p[2]: exact for a bf16 entry of 2^-15 of the row's largest
// or more.  (Two planes lose the small channels beside a large one: one channel
// 200 times the rest left outputs off by twice their bound, 5000 times by seven.)
__device__ __forceinline__ void encode16(const uint16_t *x, float f, i32x4 *p) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint32_t a = 0, b = 0, c = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = int(rintf(__uint_as_float(uint32_t(x[4 * w + j]) << 16) * f));
            const int nb = (n + 128) >> 8, na = (nb + 128) >> 8;
            a |= (uint32_t(na) & 0xFFu) << (8 * j);
            b |= (uint32_t(nb) & 0xFFu) << (8 * j);   // nb - 256 na, modulo 256
            c |= (uint32_t(n) & 0xFFu) << (8 * j);
        }
        p[0][w] = int(a);
        p[1][w] = int(b);
        p[2][w] = int(c);
    }
}

// Columns (row of the request, head of the group) in tiles of 16; a
// workgroup's four wavefronts take the pages of its split in turn, each with
// a running maximum and sum of its own, joined through LDS at the end.
//
// Codes go from HBM straight into the operands of the MFMAs, which is what the
// cache's layout is for: K as int8 against q in three int8 planes (exact int32
// sums; converting K to fp16 would cost 5 vector operations per 4 codes), V to
// fp16 in registers.  The accumulator of S^T (16 tokens x 16 columns) holds 4
// tokens of a column per lane, and V's order of tokens makes two such blocks
// the B operand of P.V as they are.  Bound by HBM: 258 MB of 64 ragged requests
// in 53 us + 6 us for the join (4.8 TB/s), 683 MB of 3 x 120k tokens in 121 + 8
// (5.7 TB/s; a copy reaches 4.8).  A request of 17 pages takes 9 us, five page
// round trips per wavefront.
//
// ONCE: every code is read by one workgroup (one tile of columns), so the loads
// are hinted not to stay in the caches: 64 ragged requests of 32 x 128 heads 64
// -> 57 us, 3 x 120k tokens 137 -> 126; with a second tile, which finds the
// codes in the L2 without the hint, 16 x 7 rows over 3000 tokens 59 -> 65.
//
// Two wavefronts per SIMD are asked for up to D = 128: without, the compiler takes
// 284 registers there for the three planes' accumulators and one wavefront, with
// it 231.  The third plane costs 1% where HBM bounds (64 ragged requests 58.0 ->
// 58.6 us) and up to 7% where the matrix units do (short prompts at D = 256).
template <int DC, bool ONCE>
__global__ __launch_bounds__(kAttnThreads, DC <= 2 ? 2 : 1) void attn_decode_kernel(AttnArgs a) {
    constexpr int D = 64 * DC, NE = D / 16;
    __shared__ float s_o[kWaves][16][D + 4];
    __shared__ float s_m[kWaves][16], s_l[kWaves][16];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;
    const int r = int(blockIdx.x) / a.n_heads, head = int(blockIdx.x) % a.n_heads;
    const Request rq = load_request(a, r);
    const int split = int(blockIdx.y);
    clear_rows<D>(a, rq, r, head);
    if (rq.rows == 0 || rq.prompt || split >= rq.splits) return;
    const int pa = rq.p0 + split * rq.split_pages;
    const int pb = split == rq.splits - 1 ? rq.p1 : min(rq.p1, pa + rq.split_pages);
    const int n_cols = rq.rows * a.group;
    const int32_t *row_of_table = a.table + int64_t(r) * a.ldt;
    int64_t part_step;
    const int64_t part0 = partial_at(a, rq, r, part_step);

    for (int c0 = int(blockIdx.z) * 16; c0 < n_cols; c0 += int(gridDim.z) * 16) {
        const int c = c0 + col;
        const bool live = c < n_cols;
        const int qi = (live ? c : c0) / a.group, gh = (live ? c : c0) % a.group;
        const int t = rq.row0 + qi, hq = head * a.group + gh;
        int lo, hi;
        row_range(a, rq, qi, lo, hi);
        if (!live) hi = lo = 0;
        // q's row as int8 planes in registers
        i32x4 qp[DC][3];
        float qs;
        {
            const uint16_t *qx = a.q + int64_t(t) * a.ldq + int64_t(hq) * a.hsq + g * 16;
            union { uint4 u[2]; uint16_t h[16]; } x[DC];
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < DC; ++j) {
                x[j].u[0] = *reinterpret_cast<const uint4 *>(qx + 64 * j);
                x[j].u[1] = *reinterpret_cast<const uint4 *>(qx + 64 * j + 8);
#pragma unroll
                for (int i = 0; i < 16; ++i) top = max(top, uint32_t(x[j].h[i]) & 0x7FFFu);
            }
            top = max(top, uint32_t(__shfl_xor(int(top), 16)));
            top = max(top, uint32_t(__shfl_xor(int(top), 32)));
            const bool bad = top >= 0x7F80u;
            const int e = max(int(top >> 7) - 126, -100);
            const float f = bad ? 0.f : pow2f(22 - e) * a.sign;
#pragma unroll
            for (int j = 0; j < DC; ++j) {
                if (bad) {
                    qp[j][0] = qp[j][1] = qp[j][2] = i32x4{0, 0, 0, 0};
                } else {
                    encode16(x[j].h, f, qp[j]);
                }
            }
            qs = bad ? __uint_as_float(0x7FC00000u) : pow2f(e - 22) * a.scale_log2;
        }
        // pages any live column of the tile sees
        int lo_min = live ? lo : INT32_MAX, hi_max = hi, lo_max = live ? lo : 0, hi_min = live ? hi : INT32_MAX;
#pragma unroll
        for (int m = 1; m < 16; m <<= 1) {
            lo_min = min(lo_min, __shfl_xor(lo_min, m));
            lo_max = max(lo_max, __shfl_xor(lo_max, m));
            hi_min = min(hi_min, __shfl_xor(hi_min, m));
            hi_max = max(hi_max, __shfl_xor(hi_max, m));
        }
        const int p_first = max(pa, lo_min / kPage), p_last = min(pb, (hi_max + kPage - 1) / kPage);

        f32x4 o[NE];
#pragma unroll
        for (int e = 0; e < NE; ++e) o[e] = f32x4{0.f, 0.f, 0.f, 0.f};
        float m_run = -INFINITY, l_run = 0.f;
        // The wavefront's pages p_first + wv + 4 i: entry and scales of up to 64 of
        // them by a lane each, the codes a page ahead: K of the next page is loaded
        // when this page's scores are done, V when its values are added.
        i32x4 kf[4][DC];
        i32x4 vf[NE];
        const auto codes_of = [&](int id) {   // a page that is not there reads page 0 and is masked
            return a.codes + (int64_t(id < 0 ? 0 : id) * a.n_heads + head) * (2 * kPage * D) + lane * 16;
        };
        const auto load_k = [&](const int8_t *kp) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int j = 0; j < DC; ++j) kf[b][j] = load_codes<ONCE>(kp + (b * DC + j) * 1024);
        };
        const auto load_v = [&](const int8_t *kp) {
#pragma unroll
            for (int e = 0; e < NE; ++e) vf[e] = load_codes<ONCE>(kp + kPage * D + e * 1024);
        };
        for (int p_at = p_first + wv; p_at < p_last; p_at += 64 * kWaves) {
            const int mine = p_at + lane * kWaves, count = min(64, (p_last - p_at + kWaves - 1) / kWaves);
            int32_t entry = row_of_table[min(mine, p_last - 1)];
            if (entry < 0 || entry >= a.n_pages || mine >= p_last) entry = -1;
            const int64_t blk = (int64_t(max(entry, 0)) * a.n_heads + head) * 2;
            const float2 scale = *reinterpret_cast<const float2 *>(a.scales + blk);
            int id = __builtin_amdgcn_readlane(entry, 0);
            const int8_t *next = codes_of(id);
            load_k(next);
            load_v(next);
            for (int at = 0; at < count; ++at) {
                const int p = p_at + at * kWaves;
                const bool there = id >= 0;
                const float ks = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(scale.x), at));
                const float vs = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(scale.y), at));
                const int ev = exp_of_scale(vs) - 7;
                if (at + 1 < count) {
                    id = __builtin_amdgcn_readlane(entry, at + 1);
                    next = codes_of(id);
                }
                // scores of 16 tokens x 16 columns each, in the units of the codes
                const float f = qs * ks, ef = float(ev);
                float y[4][4];
                float top = -INFINITY;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    i32x4 s0 = {0, 0, 0, 0}, s1 = s0, s2 = s0;
#pragma unroll
                    for (int j = 0; j < DC; ++j) {
                        s0 = __builtin_amdgcn_mfma_i32_16x16x64_i8(kf[b][j], qp[j][0], s0, 0, 0, 0);
                        s1 = __builtin_amdgcn_mfma_i32_16x16x64_i8(kf[b][j], qp[j][1], s1, 0, 0, 0);
                        s2 = __builtin_amdgcn_mfma_i32_16x16x64_i8(kf[b][j], qp[j][2], s2, 0, 0, 0);
                    }
                    // |s1| <= 256 x 128 x 128 = 2^22: 256 s1 + s2 fits 32 bits
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        y[b][i] = fmaf(float(s0[i]), 0x1p16f, float(s1[i] * 256 + s2[i])) * f + ef;
                }
                if (at + 1 < count) load_k(next);
                const int j0 = p * kPage;
                if (!there || j0 < lo_max || j0 + kPage > hi_min) {
#pragma unroll
                    for (int b = 0; b < 4; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int j = j0 + b * 16 + g * 4 + i;
                            if (!there || j < lo || j >= hi) y[b][i] = -INFINITY;
                        }
                }
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = fmaxf(top, y[b][i]);
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                // the difference first: m_new - kTopLog2 would round to whole powers of two where scores are far from 0
                const float m_new = fmaxf(m_run, top), ref = m_new == -INFINITY ? 0.f : m_new;
                const float alpha = __builtin_amdgcn_exp2f(m_run == -INFINITY ? -INFINITY : m_run - m_new);
                m_run = m_new;
                float sum = 0.f;
                f16x8 pf[2];
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float w = __builtin_amdgcn_exp2f((y[b][i] - ref) + kTopLog2);
                        sum += w;
                        pf[b >> 1][(b & 1) * 4 + i] = _Float16(w);
                    }
                l_run = l_run * alpha + sum * pow2f(-ev);
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                    o[e] *= alpha;
                    const f16x8 v0 = codes_to_f16(uint32_t(vf[e].x), uint32_t(vf[e].y));
                    const f16x8 v1 = codes_to_f16(uint32_t(vf[e].z), uint32_t(vf[e].w));
                    o[e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf[0], o[e], 0, 0, 0);
                    o[e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf[1], o[e], 0, 0, 0);
                }
                if (at + 1 < count) load_v(next);
            }
        }
        // join: o[e][i] is dim 16 e + 4 g + i of column col
        l_run += __shfl_xor(l_run, 16);
        l_run += __shfl_xor(l_run, 32);
        __syncthreads();   // the tile before has been read
#pragma unroll
        for (int e = 0; e < NE; ++e) *reinterpret_cast<f32x4 *>(&s_o[wv][col][e * 16 + g * 4]) = o[e];
        if (g == 0) { s_m[wv][col] = m_run; s_l[wv][col] = l_run; }
        __syncthreads();
        for (int e = threadIdx.x; e < 16 * (D / 4); e += kAttnThreads) {
            const int cc = e / (D / 4), d = (e % (D / 4)) * 4;
            if (c0 + cc >= n_cols) continue;
            float m = s_m[0][cc];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) m = fmaxf(m, s_m[w][cc]);
            float l = 0.f;
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float mw = s_m[w][cc];
                const bool none = mw == -INFINITY && s_l[w][cc] == 0.f;
                const float x = none ? 0.f : __builtin_amdgcn_exp2f(mw == m ? 0.f : mw - m);
                l += s_l[w][cc] * x;
                v += *reinterpret_cast<const f32x4 *>(&s_o[w][cc][d]) * x;
            }
            const float inv = l == 0.f ? 0.f : 1.0f / l;
            v *= inv;
            const int tt = rq.row0 + (c0 + cc) / a.group, h = head * a.group + (c0 + cc) % a.group;
            if (rq.splits == 1) {
                uint2 u;
                u.x = uint32_t(f32_to_bf16_rne(v.x)) | (uint32_t(f32_to_bf16_rne(v.y)) << 16);
                u.y = uint32_t(f32_to_bf16_rne(v.z)) | (uint32_t(f32_to_bf16_rne(v.w)) << 16);
                *reinterpret_cast<uint2 *>(a.out + int64_t(tt) * a.ldo + int64_t(h) * a.hso + d) = u;
            } else {
                const int64_t at = part0 + split * part_step + int64_t((c0 + cc) / a.group) * a.n_q + h;
                *reinterpret_cast<f32x4 *>(a.part + at * D + d) = v;
                // kTopLog2 is in every l alike and cancels
                if (d == 0) a.lse[at] = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) + log2f(l);
            }
        }
    }
}

// Prompts: tiles of 32 columns per wavefront, 4 or 8 wavefronts, over all pages of a split.
//
// A page's codes are turned into fp16 (exactly) once per workgroup and put in
// LDS in the order in which the 32x32x16 fp16 MFMAs take them, K as their A
// operand of S^T = K Q^T, V as that of O^T += V^T P^T.  The accumulator of S^T
// holds, per lane, 4 + 4 tokens of a 16-token stretch of one column; V's
// operand takes its tokens in that same order, so the weights go from one
// product to the next in registers.  The next page is loaded into registers
// while this one is multiplied, and converted into the other LDS buffer after.
//
// 8192 rows of 32 x 128 heads: 561 us, 980 TFLOP/s (551 to 570 us on several
// cards), where a large library product reaches 1211.  The matrix units are busy
// 47% of the time that a compute unit has work, the vector units 53%: a 32x32x16
// product leaves room for about four vector instructions, and a page has eight
// per product (two exponentials, their sums, maxima and conversions).  At D = 64
// the same vector work meets half the products (vector units 63%, matrix units
// 30%): six windowed chunks take 127 us, 490 TFLOP/s, a third of it with most
// compute units idle, in the second round of 577 workgroups on 512 places.
template <int DC, int NW>
__global__ __launch_bounds__(64 * NW, DC <= 2 ? 2 : 1) void attn_prompt_kernel(AttnArgs a) {
    constexpr int D = 64 * DC, KS = D / 16, DB = D / 32, kCols = 32 * NW, kThr = 64 * NW;
    constexpr int kAhead = 4;                                            // operands read ahead of their product
    constexpr int kPieces = 4 * D, kPer = (kPieces + kThr - 1) / kThr;   // 16-byte pieces of K (and of V), per thread
    __shared__ f16x8 k_lds[2][kPage * D / 8], v_lds[2][kPage * D / 8];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, h = lane >> 5;
    const int r = int(blockIdx.x) / a.n_heads, head = int(blockIdx.x) % a.n_heads;
    const Request rq = load_request(a, r);
    const int split = int(blockIdx.y);
    if (a.prompt_from == 0) clear_rows<D>(a, rq, r, head);   // no decode kernel runs beside this one
    if (rq.rows == 0 || !rq.prompt || split >= rq.splits) return;
    const int pa = rq.p0 + split * rq.split_pages;
    const int pb = split == rq.splits - 1 ? rq.p1 : min(rq.p1, pa + rq.split_pages);
    const int n_cols = rq.rows * a.group, n_tiles = (n_cols + kCols - 1) / kCols;
    const int32_t *row_of_table = a.table + int64_t(r) * a.ldt;
    int64_t part_step;
    const int64_t part0 = partial_at(a, rq, r, part_step);

    // the last tiles first: under a causal mask they see the most
    for (int tile = n_tiles - 1 - int(blockIdx.z); tile >= 0; tile -= int(gridDim.z)) {
        const int c0 = tile * kCols, c = c0 + wv * 32 + col;
        const bool live = c < n_cols;
        const int qi = (live ? c : c0) / a.group, gh = (live ? c : c0) - qi * a.group;
        const int t = rq.row0 + qi, hq = head * a.group + gh;
        int lo, hi;
        row_range(a, rq, qi, lo, hi);
        if (!live) hi = lo = 0;
        // ranges of the tile and of this wavefront's columns (lo and hi never fall from row to row)
        int t_lo, t_hi, w_lo_max, w_hi_min, unused;
        row_range(a, rq, c0 / a.group, t_lo, unused);
        row_range(a, rq, (min(c0 + kCols, n_cols) - 1) / a.group, unused, t_hi);
        const int w_first = min(c0 + wv * 32, n_cols - 1), w_last = min(c0 + wv * 32 + 31, n_cols - 1);
        row_range(a, rq, w_first / a.group, unused, w_hi_min);
        row_range(a, rq, w_last / a.group, w_lo_max, unused);
        const int p_first = max(pa, t_lo / kPage), p_last = min(pb, (t_hi + kPage - 1) / kPage);

        // q's row as fp16, scaled by a power of two into fp16's normal range (exact but for
        // entries 2^-28 of the row's largest)
        f16x8 q[KS];
        float qs;
        {
            const uint16_t *qp = a.q + int64_t(t) * a.ldq + int64_t(hq) * a.hsq + h * 8;
            union { uint4 u; uint16_t x[8]; } x[KS];
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                x[k].u = *reinterpret_cast<const uint4 *>(qp + 16 * k);
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max(top, uint32_t(x[k].x[i]) & 0x7FFFu);
            }
            top = max(top, uint32_t(__shfl_xor(int(top), 32)));
            const bool bad = top >= 0x7F80u;
            const int e = max(int(top >> 7) - 126, -100);
            const float f = pow2f(14 - e) * a.sign;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    q[k][i] = bad ? _Float16(0.f) : _Float16(__uint_as_float(uint32_t(x[k].x[i]) << 16) * f);
            qs = bad ? __uint_as_float(0x7FC00000u) : pow2f(e - 14) * a.scale_log2;
        }

        u32x4 kr[kPer];
        uint2 vr[kPer][2];
        // Table entries are loaded a step before they are looked at, ahead of that
        // step's codes: waiting for an entry at once would wait for the codes too.
        const auto entry = [&](int p) { return row_of_table[min(p, p_last - 1)]; };
        const auto id_of = [&](int32_t e, int p) {
            const int32_t id = __builtin_amdgcn_readfirstlane(e);
            return p < p_last && id >= 0 && id < a.n_pages ? id : -1;
        };
        // a page that is not there reads page 0 and is masked
        const auto block_of = [&](int id) { return (int64_t(id < 0 ? 0 : id) * a.n_heads + head) * 2; };
        const auto scales_of = [&](int id) { return *reinterpret_cast<const float2 *>(a.scales + block_of(id)); };
        const auto load_k = [&](int id) {
            const int8_t *kp = a.codes + block_of(id) * (kPage * D);
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (kPieces % kThr == 0 || j * kThr + tid < kPieces)
                    kr[j] = *reinterpret_cast<const u32x4 *>(kp + (j * kThr + tid) * 16);
        };
        const auto load_v = [&](int id) {
            const int8_t *vp = a.codes + (block_of(id) + 1) * (kPage * D);
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                // two token groups g and g + 2 of a dim, half of their 16 tokens
                const int u = j * kThr + tid, m = u & 15, g = (u >> 4) & 1, half = (u >> 5) & 1, e = u >> 6;
                if (kPieces % kThr != 0 && u >= kPieces) break;
                const int8_t *v = vp + ((e * 4 + g) * 16 + m) * 16 + half * 8;
                vr[j][0] = *reinterpret_cast<const uint2 *>(v);
                vr[j][1] = *reinterpret_cast<const uint2 *>(v + 512);
            }
        };
        const auto store_k = [&](f16x8 *b) {   // 16 dims of a token: both halves of the lanes of one operand
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int u = j * kThr + tid, rr = u & 15, g = (u >> 4) & 3, cc = (u >> 6) % DC, aa = (u >> 6) / DC;
                if (kPieces % kThr != 0 && u >= kPieces) break;
                f16x8 *d = b + ((aa >> 1) * KS + cc * 4 + g) * 64 + (aa & 1) * 16 + rr;
                d[0] = codes_to_f16(kr[j].x, kr[j].y);
                d[32] = codes_to_f16(kr[j].z, kr[j].w);
            }
        };
        const auto store_v = [&](f16x8 *b) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int u = j * kThr + tid, m = u & 15, g = (u >> 4) & 1, half = (u >> 5) & 1, e = u >> 6;
                if (kPieces % kThr != 0 && u >= kPieces) break;
                f16x8 *d = b + ((e >> 1) * 4 + half * 2) * 64 + g * 32 + (e & 1) * 16 + m;
                d[0] = codes_to_f16(vr[j][0].x, vr[j][1].x);
                d[64] = codes_to_f16(vr[j][0].y, vr[j][1].y);
            }
        };
        const auto scores = [&](const f16x8 *kb, f32x16 *s) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    s[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kb[(b * KS + k) * 64 + lane], q[k], s[b], 0, 0, 0);
        };

        f32x16 o[DB];
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
        float m_run = -INFINITY, l_run = 0.f;
        int id0 = -1, id1 = -1, id2 = -1;   // pages p, p + 1, p + 2
        int32_t e3 = -1;                    // table entry of p + 3
        float2 sc = {0.f, 0.f}, sc1 = sc;   // scales of pages p, p + 1
        f32x16 s0[2], s1[2];
        // One page: its scores are in s; the next page's go to n while these
        // are turned into weights.  K is one page ahead of V in LDS.
        const auto page_step = [&](int p, f32x16 *s, f32x16 *n, int cur) {
            __syncthreads();   // K of p + 1 and V of p are in LDS; K of p and V of p - 1 have been read
            const int ev = exp_of_scale(sc.y) - 7;
            // above 0 (or NaN), so that a masked score, -inf, stays one
            float f = qs * sc.x == 0.f ? 0x1p-120f : qs * sc.x;
            const float ef = float(ev);
            const int j0 = p * kPage;
            if (id0 < 0 || j0 < w_lo_max || j0 + kPage > w_hi_min) {
                const int seen = id0 < 0 ? 0 : hi;
                if (id0 < 0) f = 1.f;   // page 0 stands in, and its scale may be anything
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int j = j0 + b * 32 + 8 * (i >> 2) + 4 * h + (i & 3);
                        if (j < lo || j >= seen) s[b][i] = -INFINITY;
                    }
            }
            float top = s[0][0];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
            const float m_new = fmaxf(m_run, max_halves(fmaf(top, f, ef)));
            if (__any(m_new > m_run + kSlackLog2)) {
                const float alpha = m_run == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m_run - m_new);
                l_run *= alpha;
#pragma unroll
                for (int d = 0; d < DB; ++d) o[d] *= alpha;
                m_run = m_new;
            }
            const float m = m_run == -INFINITY ? 0.f : m_run;
            float shift = ef - (m - kTopLog2);
            if (fabsf(m) > kFarLog2) {
                // the same rounding as m's, so that the largest score is at 0 and none far above (NaN stays)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float x = fmaf(s[b][i], f, ef) - m + kTopLog2;
                        s[b][i] = x > kTopLog2 + kSlackLog2 ? kTopLog2 + kSlackLog2 : x;
                    }
                f = 1.f;
                shift = 0.f;
            }
            // The next page's 2 KS products with this page's 32 weights between
            // them, then this page's 4 DB products with the conversions of the
            // pages behind: matrix and vector instructions side by side, operands
            // read kAhead products early.  The order is fixed here step by step
            // (left alone, the products come in one run and the rest after it).
            const f16x8 *kb = k_lds[cur ^ 1] + lane, *vb = v_lds[cur] + lane;
            f16x8 fr[kAhead];
            float sum = 0.f;
            f16x8 w[4];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) fr[i] = kb[((i & 1) * KS + (i >> 1)) * 64];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) n[b][i] = 0.f;
#pragma unroll
            for (int i = 0; i < 2 * KS; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                n[i & 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fr[i % kAhead], q[i >> 1], n[i & 1], 0, 0, 0);
                const int next = i + kAhead;
                if (next < 2 * KS) fr[i % kAhead] = kb[((next & 1) * KS + (next >> 1)) * 64];
                else fr[i % kAhead] = vb[((next - 2 * KS) % DB * 4 + (next - 2 * KS) / DB) * 64];
#pragma unroll
                for (int j = i * 32 / (2 * KS); j < (i + 1) * 32 / (2 * KS); ++j) {
                    const float x = __builtin_amdgcn_exp2f(s[j >> 4][j & 15] * f + shift);
                    sum += x;
                    w[j >> 3][j & 7] = _Float16(x);
                }
            }
            l_run += sum * pow2f(-ev);
#pragma unroll
            for (int i = 0; i < 4 * DB; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                const int at = (2 * KS + i) % kAhead, next = i + kAhead;
                o[i % DB] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fr[at], w[i / DB], o[i % DB], 0, 0, 0);
                if (next < 4 * DB) fr[at] = vb[(next % DB * 4 + next / DB) * 64];
                if (i == DB) store_k(k_lds[cur]);
                if (i == 2 * DB) store_v(v_lds[cur ^ 1]);
            }
            __builtin_amdgcn_sched_barrier(0);
            // the next step's codes, now that the registers are free
            id0 = id1;
            id1 = id2;
            id2 = id_of(e3, p + 3);
            e3 = entry(p + 4);
            load_k(id2);
            load_v(id1);
            sc = sc1;
            sc1 = scales_of(id1);
        };
        if (p_first < p_last) {
            const int32_t e0 = entry(p_first), e1 = entry(p_first + 1), e2 = entry(p_first + 2);
            e3 = entry(p_first + 3);
            id0 = id_of(e0, p_first);
            id1 = id_of(e1, p_first + 1);
            id2 = id_of(e2, p_first + 2);
            sc = scales_of(id0);
            sc1 = scales_of(id1);
            load_k(id0);
            load_v(id0);
            __syncthreads();   // the tile before has been read
            store_k(k_lds[0]);
            store_v(v_lds[0]);
            load_k(id1);
            store_k(k_lds[1]);
            load_k(id2);
            load_v(id1);
            __syncthreads();
            scores(k_lds[0], s0);
            for (int p = p_first; p < p_last; p += 2) {
                page_step(p, s0, s1, 0);
                if (p + 1 < p_last) page_step(p + 1, s1, s0, 1);
            }
        }
        const float l = l_run + __shfl_xor(l_run, 32);
        if (live) {
            const bool none = l == 0.f || hi <= lo;
            const float inv = 1.0f / l;
            const int64_t at = part0 + split * part_step + int64_t(qi) * a.n_q + hq;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f32x4 v = {o[d][4 * i] * inv, o[d][4 * i + 1] * inv, o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv};
                    if (none) v = f32x4{0.f, 0.f, 0.f, 0.f};
                    const int dim = d * 32 + 8 * i + 4 * h;
                    if (rq.splits == 1) {
                        uint2 u;
                        u.x = uint32_t(f32_to_bf16_rne(v.x)) | (uint32_t(f32_to_bf16_rne(v.y)) << 16);
                        u.y = uint32_t(f32_to_bf16_rne(v.z)) | (uint32_t(f32_to_bf16_rne(v.w)) << 16);
                        *reinterpret_cast<uint2 *>(a.out + int64_t(t) * a.ldo + int64_t(hq) * a.hso + dim) = u;
                    } else {
                        *reinterpret_cast<f32x4 *>(a.part + at * D + dim) = v;
                    }
                }
            if (rq.splits > 1 && h == 0)
                a.lse[at] = none ? -INFINITY : (m_run == -INFINITY ? 0.f : m_run) + log2f(l);
        }
    }
}

// Joins the splits of one request's rows, a workgroup per row and head: a
// result row is D / 4 lanes wide, so 4096 / D splits are read at once; each
// lane sums its splits in their order, then the groups are added in theirs.
template <int DC>
__global__ __launch_bounds__(kAttnThreads) void attn_join_kernel(AttnArgs a) {
    constexpr int D = 64 * DC, kLanes = D / 4, kGroups = kAttnThreads / kLanes;
    __shared__ float s_w[kMaxSplits];
    __shared__ f32x4 s_v[kGroups][kLanes];
    const int tid = threadIdx.x, lane = tid & 63, grp = tid / kLanes, d = tid % kLanes;
    const Request rq = load_request(a, int(blockIdx.x));
    if (rq.splits <= 1) return;
    const int64_t n = int64_t(rq.rows) * a.n_q;
    int64_t step;
    const int64_t first = partial_at(a, rq, int(blockIdx.x), step);
    for (int64_t i = blockIdx.y; i < n; i += gridDim.y) {
        const int64_t at = first + i;
        // weights of the splits (at most 64: one per lane), the same in every wavefront
        const float e = lane < rq.splits ? a.lse[at + lane * step] : -INFINITY;
        float m = e;
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) m = fmaxf(m, __shfl_xor(m, k));
        const float w = e == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(e - m);
        float l = w;
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) l += __shfl_xor(l, k);
        if (tid < 64) s_w[tid] = l == 0.f ? 0.f : w / l;
        __syncthreads();
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        if (grp < kGroups) {
            const f32x4 *p = reinterpret_cast<const f32x4 *>(a.part + at * D) + d;
#pragma unroll 4
            for (int s = grp; s < rq.splits; s += kGroups) {
                const float ws = s_w[s];
                const f32x4 x = p[s * step * (D / 4)];
                if (ws != 0.f) v += x * ws;   // what an empty split left there is not looked at (a NaN weight is)
            }
            s_v[grp][d] = v;
        }
        __syncthreads();
        if (grp == 0) {
#pragma unroll
            for (int k = 1; k < kGroups; ++k) v += s_v[k][d];
            uint2 u;
            u.x = uint32_t(f32_to_bf16_rne(v.x)) | (uint32_t(f32_to_bf16_rne(v.y)) << 16);
            u.y = uint32_t(f32_to_bf16_rne(v.z)) | (uint32_t(f32_to_bf16_rne(v.w)) << 16);
            const int64_t t = rq.row0 + i / a.n_q, h = i % a.n_q;
            *reinterpret_cast<uint2 *>(a.out + t * a.ldo + h * a.hso + 4 * d) = u;
        }
        __syncthreads();
    }
}

// The same for many rows: a group of D / 4 lanes per row and head, which goes
// through the splits one after the other with a running maximum.  A prompt call
// of 2300 rows of 32 heads x 64 in 2 splits: 158 us, with a workgroup per row and
// head 248.
template <int DC>
__global__ __launch_bounds__(kAttnThreads) void attn_join_rows_kernel(AttnArgs a) {
    constexpr int D = 64 * DC, kLanes = D / 4, kGroups = kAttnThreads / kLanes;
    const int grp = threadIdx.x / kLanes, d = threadIdx.x % kLanes;
    const Request rq = load_request(a, int(blockIdx.x));
    if (rq.splits <= 1 || grp >= kGroups) return;
    const int64_t n = int64_t(rq.rows) * a.n_q;
    int64_t step;
    const int64_t first = partial_at(a, rq, int(blockIdx.x), step);
    for (int64_t i = int64_t(blockIdx.y) * kGroups + grp; i < n; i += int64_t(gridDim.y) * kGroups) {
        const int64_t at = first + i;
        const f32x4 *p = reinterpret_cast<const f32x4 *>(a.part + at * D) + d;
        float m = -INFINITY, l = 0.f;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int s = 0; s < rq.splits; ++s) {
            const float e = a.lse[at + s * step];
            const f32x4 x = p[s * step * (D / 4)];
            if (e == -INFINITY) continue;   // an empty split
            const float top = fmaxf(m, e), old = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - top);
            const float w = __builtin_amdgcn_exp2f(e - top);   // NaN for a NaN row
            v = v * old + x * w;
            l = l * old + w;
            m = top;
        }
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        v *= inv;
        uint2 u;
        u.x = uint32_t(f32_to_bf16_rne(v.x)) | (uint32_t(f32_to_bf16_rne(v.y)) << 16);
        u.y = uint32_t(f32_to_bf16_rne(v.z)) | (uint32_t(f32_to_bf16_rne(v.w)) << 16);
        const int64_t t = rq.row0 + i / a.n_q, h = i % a.n_q;
        *reinterpret_cast<uint2 *>(a.out + t * a.ldo + h * a.hso + 4 * d) = u;
    }
}

struct AttnShape {
    int32_t splits, split_pages, psplits, psplit_pages;
    bool decode, prompt;   // kernels to run; one that runs alone takes every request
    int32_t waves;         // of the prompt kernel's workgroups
};

void set_splits(int64_t pages, int64_t per, int32_t &splits, int32_t &per_split) {
    if (per * kMaxSplits < pages) per = (pages + kMaxSplits - 1) / kMaxSplits;
    splits = per < pages ? int32_t((pages + per - 1) / per) : 1;
    per_split = int32_t(per > 0 ? per : 1);
}

// Splits of the decode kernel over `items` tiles of 16 columns: none up to
// kWholePages pages (a second launch costs more than its four wavefronts' six
// pages each), else about 4096 workgroups of 16 pages at least -- four per
// wavefront, which pay for the query's encoding before and the wavefronts' joining
// after (32 x 4000 tokens of 2 heads x 256: 32 us, with four pages 53) -- or of down
// to four where that leaves compute units empty.
void decode_splits(int64_t pages, int64_t items, AttnShape &s) {
    const int64_t fill = pages * items / 256, least = fill < 4 ? 4 : fill < 16 ? fill : 16;
    int64_t per = (pages * items + 4095) / 4096;
    if (per < least) per = least;
    set_splits(pages, pages <= kWholePages ? pages : per, s.splits, s.split_pages);
}

AttnShape attn_shape(int64_t T, int64_t R, int32_t n_heads, int32_t D, int32_t n_q, int64_t max_q, int64_t max_kv,
                     int64_t window) {
    // pages a request's rows look at: a window's rows and the pages it cuts at both ends
    int64_t pages = (max_kv + kPage - 1) / kPage;
    if (window > 0 && (window + max_q) / kPage + 2 < pages) pages = (window + max_q) / kPage + 2;
    const int64_t group = n_q / n_heads;
    AttnShape s{};
    // Up to kDecodeCols columns the decode kernel, and also for short prompts:
    // its 16 columns convert no page and come in as many workgroups as its tiles,
    // where the prompt kernel's few would walk the pages one after the other.
    // Split requests, which fill the card in any case, by tiles times pages; whole
    // ones by both kernels' times in us, fitted to 3070 shapes of 10 to 1500 rows
    // (standard errors 8 to 12%): the decode kernel's workgroups come in rounds of
    // 512 (256 above D = 128) that cost their pages and a start each, the prompt
    // kernel's walk all pages whatever their number.  Above D = 128, where a few
    // rounds are all, tiles times pages bound whole requests too.
    // Prompt kernel against decode kernel, us, rows of each request, heads / KV heads:
    //   D = 128  512, 8 / 1 20.0, 14.5;  1024, 8 / 1 27.1, 14.8;  1500, 8 / 1 30.8, 23.2;
    //            700, 32 / 8 34.6, 27.7;  512 of 1000, 32 / 8 33.4, 26.1;
    //            4 x 200, 32 / 8 18.2, 26.1;  4 x 300, 32 / 8 21.4, 36.6
    //   D = 256  512, 8 / 1 36.0, 14.7;  1024, 8 / 1 46.1, 31.4;  300, 32 / 8 28.5, 33.9;
    //            512, 32 / 8 37.2, 46.4;  4 x 200, 32 / 8 29.3, 69.7
    // and split: 64 rows of 4000, 4 times, 32 / 8 x 128 (16128 visits) 48, 51; 40 of
    // 4000, the same heads x 256 (5040 of 8192) 55.9, 40.3.
    const int64_t tiles = max_q > 0 ? (max_q * group + 15) / 16 : 1, items = R * n_heads * tiles;
    const double p = double(pages > 0 ? pages : 1);
    s.prompt = max_q * group > kDecodeCols;
    if (s.prompt && items <= 65536) {   // more are the prompt kernel's
        decode_splits(pages, items, s);
        const bool many = double(items) * p * (D > 128 ? D : 128) > 128.0 * kDecodeVisits;
        const double cols = double(R) * double(max_q * group) * n_heads / 128 / 512;   // prompt workgroups per place
        const double d_us = D > 128 ? 10 + items / 256.0 * (0.5 * p + 5) : 12 + items / 512.0 * (0.32 * p + 1);
        const double p_us = D > 128 ? 18 + p * (0.8 + 5.5 * cols) : 14 + p * (0.35 + 1.8 * cols);
        s.prompt = s.splits > 1 ? many : d_us > p_us || (D > 128 && many);
    }
    s.decode = !s.prompt || R > 1;
    decode_splits(pages, s.prompt ? R * n_heads * ((kDecodeCols + 15) / 16) : items, s);
    // 8 wavefronts share a page's conversion, 4 fill the card with fewer rows
    // and run two workgroups per compute unit out of step.  D = 128, 8 against 4,
    // us, by tiles of 256 columns times heads: 192 (4096 rows, 12 / 2 heads) 122.9,
    // 104.3; 256 (2048, 32 / 8) 77.6, 68.7; 512 (4096, 32 / 8) 165.1, 176.2; 640 (4096,
    // 40 / 40) 220.8, 208.8; 752 (3000, 64 / 8) 185.9, 186.0; 960 (6000, 40 / 40) 436.1,
    // 435.7; 1024 (8192, 32 / 8) 575.6, 595.3; 1504 (12000, 32 / 8) 1154, 1217; 4096
    // (16384, 64 / 8) 4265, 4447.  D = 64: 132 against 86 us a round of workgroups.
    s.waves = D == 128 && (T * group + 255) / 256 * n_heads >= 1024 ? 8 : 4;
    const int64_t cols = 32 * s.waves, ptiles = (T * group + cols - 1) / cols + (R - 1);
    // Splits of prompts: only into places for workgroups (two of 4 wavefronts or
    // one of 8 on each of 256 compute units) that would stay empty, by the pages
    // of each and kJoinPages a split for writing and joining its partial results.
    // Splitting more than fills the card loses: 596 workgroups' worth of rows and
    // heads with a window of 4096 took 130 us whole, 142 in 3 splits.
    const int64_t pitems = ptiles * n_heads, slots = s.waves == 8 ? 256 : 512;
    int64_t best = pages, want = 1;
    for (int64_t n = 2; n <= kMaxSplits && n * pitems <= slots && n * 2 <= pages; ++n) {
        const int64_t cost = (pages + n - 1) / n + kJoinPages * n;
        if (cost < best) { best = cost; want = n; }
    }
    set_splits(pages, (pages + want - 1) / want, s.psplits, s.psplit_pages);
    if (!s.prompt) s.psplits = 1;
    if (!s.decode) s.splits = 1;
    return s;
}

}  // namespace
}  // namespace ht

using namespace ht;

namespace {

ht_status check_attn(const ht_kv_cache *c, int64_t T, int64_t R, int32_t n_q, int64_t max_q, int64_t max_kv) {
    const ht_status st = check_cache(c);
    if (st != HT_OK) return st;
    if (T < 0 || T > (int64_t(1) << 30) || R <= 0 || R * c->n_heads > (int64_t(1) << 22) || R > (int64_t(1) << 22) ||
        n_q <= 0 || n_q > 4096 || n_q % c->n_heads || T * (n_q / c->n_heads) > (int64_t(1) << 30) || max_q < 0 ||
        max_kv < 0 || max_q > (int64_t(1) << 30) || max_kv > (int64_t(1) << 30))
        return HT_ESHAPE;
    return HT_OK;
}

// A window of 2^31 tokens or more keeps every token (and would overflow the sums it goes into): none.
int64_t clamp_window(int64_t window) { return window >= (int64_t(1) << 31) ? 0 : window; }

template <int DC>
ht_status run_attn(const AttnArgs &a, const AttnShape &sh, int64_t R, int64_t max_q, hipStream_t s) {
    const uint32_t x = uint32_t(R * a.n_heads);
    if (sh.prompt) {
        const int64_t cols = 32 * sh.waves, tiles = (max_q * a.group + cols - 1) / cols;
        const dim3 grid(x, uint32_t(sh.psplits), uint32_t(tiles > 8192 ? 8192 : tiles));
        if constexpr (DC == 2) {
            if (sh.waves == 8) attn_prompt_kernel<DC, 8><<<grid, 512, 0, s>>>(a);
        }
        if (sh.waves == 4) attn_prompt_kernel<DC, 4><<<grid, 256, 0, s>>>(a);
        HT_LAUNCH_CHECK();
    }
    if (sh.decode) {
        const int64_t cols = sh.prompt ? kDecodeCols : max_q * a.group, tiles = cols > 16 ? (cols + 15) / 16 : 1;
        const dim3 grid(x, uint32_t(sh.splits), uint32_t(tiles));
        if (tiles == 1) attn_decode_kernel<DC, true><<<grid, kAttnThreads, 0, s>>>(a);
        else attn_decode_kernel<DC, false><<<grid, kAttnThreads, 0, s>>>(a);
        HT_LAUNCH_CHECK();
    }
    if (sh.splits > 1 || sh.psplits > 1) {
        const int64_t rows = (sh.psplits > 1 || !sh.prompt ? max_q : kDecodeCols / a.group) * a.n_q;
        if (R * rows >= 4096) {   // more rows than the card takes workgroups at once
            const int64_t per = kAttnThreads / (16 * DC), y = (rows + per - 1) / per;
            attn_join_rows_kernel<DC><<<dim3(uint32_t(R), uint32_t(y < 4096 ? y : 4096)), kAttnThreads, 0, s>>>(a);
        } else {
            attn_join_kernel<DC><<<dim3(uint32_t(R), uint32_t(rows < 1 ? 1 : rows)), kAttnThreads, 0, s>>>(a);
        }
        HT_LAUNCH_CHECK();
    }
    return HT_OK;
}

// Where partial results of split rows go.  Where both kernels run, the decode
// kernel's requests have at most kDecodeCols columns each and rows of their own
// by request: T may be a prompt's thousands.
struct PartialShape {
    int64_t dec_rows, dec_total, total;   // rows per split; rows x heads x splits
    int32_t dec_per_request;
};

PartialShape partial_shape(const AttnShape &sh, int64_t T, int64_t R, int32_t n_q, int32_t n_heads) {
    PartialShape p{};
    const int32_t group = n_q / n_heads;
    p.dec_per_request = sh.prompt ? (kDecodeCols / group > 0 ? kDecodeCols / group : 1) : 0;
    p.dec_rows = sh.prompt ? R * p.dec_per_request : T;
    p.dec_total = sh.splits > 1 ? sh.splits * p.dec_rows * n_q : 0;
    p.total = p.dec_total + (sh.psplits > 1 ? sh.psplits * T * n_q : 0);
    return p;
}

}  // namespace

extern "C" ht_status ht_kv_attention_workspace(const ht_kv_cache *cache, int64_t T, int64_t R, int32_t n_q,
                                               int64_t max_q, int64_t max_kv, int64_t window, size_t *bytes) {
    if (!bytes) return HT_EINVAL;
    const ht_status st = check_attn(cache, T, R, n_q, max_q, max_kv);
    if (st != HT_OK) return st;
    if (window < 0) return HT_ESHAPE;
    const AttnShape sh = attn_shape(T, R, cache->n_heads, cache->head_dim, n_q, max_q, max_kv, clamp_window(window));
    const size_t rows = size_t(partial_shape(sh, T, R, n_q, cache->n_heads).total);
    *bytes = size_t(align256(rows * 4u)) + rows * size_t(cache->head_dim) * 4u;
    return HT_OK;
}

extern "C" ht_status ht_kv_attention_kernels(const ht_kv_cache *cache, int64_t T, int64_t R, int32_t n_q, int64_t max_q,
                                             int64_t max_kv, int64_t window, int32_t *info) {
    if (!info) return HT_EINVAL;
    const ht_status st = check_attn(cache, T, R, n_q, max_q, max_kv);
    if (st != HT_OK) return st;
    if (window < 0) return HT_ESHAPE;
    const AttnShape sh = attn_shape(T, R, cache->n_heads, cache->head_dim, n_q, max_q, max_kv, clamp_window(window));
    info[0] = sh.decode ? sh.splits : 0;
    info[1] = sh.prompt ? sh.psplits : 0;
    info[2] = sh.prompt ? sh.waves : 0;
    return HT_OK;
}

extern "C" ht_status ht_kv_attention(const uint16_t *q, int64_t ldq, int64_t hsq, int64_t T, int32_t n_q,
                                     const ht_kv_cache *cache, const int32_t *table, int64_t P, int64_t ldt,
                                     const int32_t *cu_q, const int32_t *kv_len, int64_t R, int64_t max_q,
                                     int64_t max_kv, float scale, int32_t causal, int64_t window, uint16_t *out,
                                     int64_t ldo, int64_t hso, void *ws, size_t ws_bytes, ht_stream stream) {
    ht_status st = check_attn(cache, T, R, n_q, max_q, max_kv);
    if (st != HT_OK) return st;
    if (P <= 0 || P > (int64_t(1) << 24) || ldt < P || window < 0) return HT_ESHAPE;
    window = clamp_window(window);
    if (!(scale == scale) || scale - scale != 0.f) return HT_EINVAL;
    if (T == 0) return HT_OK;
    if ((st = check_rows(q, ldq, hsq, n_q, cache->head_dim, 2)) != HT_OK) return st;
    if ((st = check_rows(out, ldo, hso, n_q, cache->head_dim, 2)) != HT_OK) return st;
    if (!table || !cu_q || !kv_len) return HT_EINVAL;
    if (!al4(table) || !al4(cu_q) || !al4(kv_len) || !al16p(ws)) return HT_EALIGN;
    size_t need = 0;
    if ((st = ht_kv_attention_workspace(cache, T, R, n_q, max_q, max_kv, window, &need)) != HT_OK) return st;
    if (need > 0 && (!ws || ws_bytes < need)) return HT_ESMALL;
    const AttnShape sh = attn_shape(T, R, cache->n_heads, cache->head_dim, n_q, max_q, max_kv, window);
    AttnArgs a{};
    a.q = q;
    a.codes = cache->codes;
    a.scales = cache->scales;
    a.table = table;
    a.cu_q = cu_q;
    a.kv_len = kv_len;
    a.out = out;
    a.lse = static_cast<float *>(ws);
    const PartialShape ps = partial_shape(sh, T, R, n_q, cache->n_heads);
    a.part = need > 0 ? a.lse + align256(size_t(ps.total) * 4u) / 4 : nullptr;
    a.dec_rows = ps.dec_rows;
    a.dec_per_request = ps.dec_per_request;
    a.prompt_at = ps.dec_total;
    a.ldq = ldq; a.hsq = hsq; a.ldo = ldo; a.hso = hso; a.ldt = ldt; a.P = P;
    a.T = int32_t(T);
    a.R = int32_t(R);
    a.n_q = n_q;
    a.n_heads = cache->n_heads;
    a.group = n_q / cache->n_heads;
    a.n_pages = int32_t(cache->n_pages);
    a.causal = causal != 0;
    a.splits = sh.splits;
    a.split_pages = sh.split_pages;
    a.window = window;
    a.prompt_from = !sh.prompt ? INT32_MAX : sh.decode ? kDecodeCols + 1 : 0;
    a.psplits = sh.psplits;
    a.psplit_pages = sh.psplit_pages;
    a.scale_log2 = (scale < 0.f ? -scale : scale) * kLog2e;
    a.sign = scale < 0.f ? -1.f : 1.f;
    hipStream_t s = hipStream_t(stream);
    switch (cache->head_dim) {
    case 64: return run_attn<1>(a, sh, R, max_q, s);
    case 128: return run_attn<2>(a, sh, R, max_q, s);
    case 192: return run_attn<3>(a, sh, R, max_q, s);
    default: return run_attn<4>(a, sh, R, max_q, s);
    }
}
