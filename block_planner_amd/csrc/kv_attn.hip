// kv_attn.hip -- attention of a batch's query rows over the paged 8-bit cache.
#include "kv.h"

namespace ht {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kAttnThreads = 256;
constexpr int kWaves = kAttnThreads / 64;
constexpr float kLog2e = 1.44269504088896341f;
// The largest weight handed to V is 2^14: fp16 keeps 11 bits down to 2^-28 of it.
constexpr float kTopLog2 = 14.f;

struct AttnArgs {
    const uint16_t *q;
    const int8_t *codes;
    const float *scales;
    const int32_t *table, *cu_q, *kv_len;
    uint16_t *out;
    float *part;        // [splits][T][n_q][D], normalised
    float *lse;         // [splits][T][n_q], log2 of the weights' sum
    int64_t ldq, hsq, ldo, hso, ldt, P;
    int32_t T, n_q, n_heads, group, n_pages, causal, splits, split_pages;
    int64_t window;
    float scale_log2;   // scale * log2(e)
};

// One request as the kernels see it: lengths clamped to the arrays.
struct Request {
    int32_t row0, rows, kv, p0, p1, splits;   // pages [p0, p1) hold every token its rows may see
};

__device__ __forceinline__ Request load_request(const AttnArgs &a, int r) {
    Request q;
    q.row0 = min(max(a.cu_q[r], 0), a.T);
    q.rows = min(max(a.cu_q[r + 1] - q.row0, 0), a.T - q.row0);
    q.kv = int32_t(min(int64_t(max(a.kv_len[r], 0)), a.P * kPage));
    q.p1 = (q.kv + kPage - 1) / kPage;
    const int64_t first = a.window > 0 ? int64_t(q.kv) - q.rows + 1 - a.window : 0;   // first row's first token
    q.p0 = first > 0 ? min(int32_t(min(first / kPage, int64_t(q.p1))), q.p1) : 0;
    q.splits = min(max((q.p1 - q.p0 + a.split_pages - 1) / a.split_pages, 1), a.splits);
    return q;
}

// Tokens row i of a request sees: [lo, hi).
__device__ __forceinline__ void row_range(const AttnArgs &a, const Request &q, int i, int &lo, int &hi) {
    const int64_t pos = int64_t(q.kv) - q.rows + i;
    hi = a.causal ? int(max(int64_t(0), min(int64_t(q.kv), pos + 1))) : q.kv;
    lo = a.window > 0 ? int(min(int64_t(q.kv), max(int64_t(0), pos + 1 - a.window))) : 0;
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

// 16 elements of a row of q as int8 planes hi, lo with n = rne(x 2^(14-E)) = 256 hi + lo.
__device__ __forceinline__ void encode16(const uint16_t *x, float f, i32x4 &hi, i32x4 &lo) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint32_t h = 0, l = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = int(rintf(__uint_as_float(uint32_t(x[4 * w + j]) << 16) * f));
            const int nh = (n + 128) >> 8, nl = n - (nh << 8);
            h |= (uint32_t(nh) & 0xFFu) << (8 * j);
            l |= (uint32_t(nl) & 0xFFu) << (8 * j);
        }
        hi[w] = int(h);
        lo[w] = int(l);
    }
}

// Columns (row of the request, head of the group) in tiles of 16; a
// workgroup's four wavefronts take the pages of its split in turn, each with
// a running maximum and sum of its own, joined through LDS at the end.
template <int DC>
__global__ __launch_bounds__(kAttnThreads) void attn_decode_kernel(AttnArgs a) {
    constexpr int D = 64 * DC, NE = D / 16;
    __shared__ float s_o[kWaves][16][D + 4];
    __shared__ float s_m[kWaves][16], s_l[kWaves][16];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;
    const int r = int(blockIdx.x) / a.n_heads, head = int(blockIdx.x) % a.n_heads;
    const Request rq = load_request(a, r);
    const int split = int(blockIdx.y);
    if (rq.rows == 0 || split >= rq.splits) return;
    const int pa = rq.p0 + split * a.split_pages;
    const int pb = split == rq.splits - 1 ? rq.p1 : min(rq.p1, pa + a.split_pages);
    const int n_cols = rq.rows * a.group;
    const int32_t *row_of_table = a.table + int64_t(r) * a.ldt;

    for (int c0 = int(blockIdx.z) * 16; c0 < n_cols; c0 += int(gridDim.z) * 16) {
        const int c = c0 + col;
        const bool live = c < n_cols;
        const int qi = (live ? c : c0) / a.group, gh = (live ? c : c0) % a.group;
        const int t = rq.row0 + qi, hq = head * a.group + gh;
        int lo, hi;
        row_range(a, rq, qi, lo, hi);
        if (!live) hi = lo = 0;
        // q's row as int8 planes in registers
        i32x4 qh[DC], ql[DC];
        float qs;
        {
            const uint16_t *qp = a.q + int64_t(t) * a.ldq + int64_t(hq) * a.hsq + g * 16;
            union { uint4 u[2]; uint16_t h[16]; } x[DC];
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < DC; ++j) {
                x[j].u[0] = *reinterpret_cast<const uint4 *>(qp + 64 * j);
                x[j].u[1] = *reinterpret_cast<const uint4 *>(qp + 64 * j + 8);
#pragma unroll
                for (int i = 0; i < 16; ++i) top = max(top, uint32_t(x[j].h[i]) & 0x7FFFu);
            }
            top = max(top, uint32_t(__shfl_xor(int(top), 16)));
            top = max(top, uint32_t(__shfl_xor(int(top), 32)));
            const bool bad = top >= 0x7F80u;
            const int e = max(int(top >> 7) - 126, -100);
            const float f = bad ? 0.f : pow2f(14 - e);
#pragma unroll
            for (int j = 0; j < DC; ++j) {
                if (bad) {
                    qh[j] = ql[j] = i32x4{0, 0, 0, 0};
                } else {
                    encode16(x[j].h, f, qh[j], ql[j]);
                }
            }
            qs = bad ? __uint_as_float(0x7FC00000u) : pow2f(e - 14) * a.scale_log2;
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
        for (int p = p_first + wv; p < p_last; p += kWaves) {
            const int32_t page = __builtin_amdgcn_readfirstlane(row_of_table[p]);
            if (page < 0 || page >= a.n_pages) continue;
            const int64_t blk = (int64_t(page) * a.n_heads + head) * 2;
            const int8_t *kp = a.codes + blk * (kPage * D) + lane * 16, *vp = kp + kPage * D;
            const float ks = a.scales[blk], vs = a.scales[blk + 1];
            const int ev = exp_of_scale(vs) - 7;
            i32x4 kf[4][DC];
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int j = 0; j < DC; ++j) kf[b][j] = *reinterpret_cast<const i32x4 *>(kp + (b * DC + j) * 1024);
            u32x4 vf[NE];
#pragma unroll
            for (int e = 0; e < NE; ++e) vf[e] = *reinterpret_cast<const u32x4 *>(vp + e * 1024);
            // scores of 16 tokens x 16 columns each, in the units of the codes
            const float f = qs * ks, ef = float(ev);
            float y[4][4];
            float top = -INFINITY;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                i32x4 sh = {0, 0, 0, 0}, sl = {0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < DC; ++j) {
                    sh = __builtin_amdgcn_mfma_i32_16x16x64_i8(kf[b][j], qh[j], sh, 0, 0, 0);
                    sl = __builtin_amdgcn_mfma_i32_16x16x64_i8(kf[b][j], ql[j], sl, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) y[b][i] = float(sh[i] * 256 + sl[i]) * f + ef;
            }
            const int j0 = p * kPage;
            if (j0 < lo_max || j0 + kPage > hi_min) {
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = j0 + b * 16 + g * 4 + i;
                        if (j < lo || j >= hi) y[b][i] = -INFINITY;
                    }
            }
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, y[b][i]);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float m_new = fmaxf(m_run, top), ref = m_new == -INFINITY ? 0.f : m_new - kTopLog2;
            const float alpha = __builtin_amdgcn_exp2f(m_run == -INFINITY ? -INFINITY : m_run - m_new);
            m_run = m_new;
            float sum = 0.f;
            f16x8 pf[2];
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float w = __builtin_amdgcn_exp2f(y[b][i] - ref);
                    sum += w;
                    pf[b >> 1][(b & 1) * 4 + i] = _Float16(w);
                }
            l_run = l_run * alpha + sum * pow2f(-ev);
#pragma unroll
            for (int e = 0; e < NE; ++e) {
                o[e] *= alpha;
                o[e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_to_f16(vf[e].x, vf[e].y), pf[0], o[e], 0, 0, 0);
                o[e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_to_f16(vf[e].z, vf[e].w), pf[1], o[e], 0, 0, 0);
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
                const float mw = s_m[w][cc], x = mw == -INFINITY && s_l[w][cc] == 0.f ? 0.f : __builtin_amdgcn_exp2f(mw == m ? 0.f : mw - m);
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
                const int64_t at = (int64_t(split) * a.T + tt) * a.n_q + h;
                *reinterpret_cast<f32x4 *>(a.part + at * D + d) = v;
                // kTopLog2 is in every l alike and cancels
                if (d == 0) a.lse[at] = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) + log2f(l);
            }
        }
    }
}

// Joins the splits of one request's rows, in their order: a wavefront per row and head.
template <int DC>
__global__ __launch_bounds__(kAttnThreads) void attn_join_kernel(AttnArgs a) {
    constexpr int D = 64 * DC;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const Request rq = load_request(a, int(blockIdx.x));
    if (rq.splits <= 1) return;
    const int64_t n = int64_t(rq.rows) * a.n_q;
    for (int64_t i = int64_t(blockIdx.y) * kWaves + wv; i < n; i += int64_t(gridDim.y) * kWaves) {
        const int64_t at = int64_t(rq.row0) * a.n_q + i, step = int64_t(a.T) * a.n_q;
        float m = -INFINITY;
        for (int s = 0; s < rq.splits; ++s) m = fmaxf(m, a.lse[at + s * step]);
        float l = 0.f, v[DC];
#pragma unroll
        for (int j = 0; j < DC; ++j) v[j] = 0.f;
        for (int s = 0; s < rq.splits; ++s) {
            const float e = a.lse[at + s * step];
            if (e == -INFINITY) continue;
            const float w = __builtin_amdgcn_exp2f(e - m);
            l += w;
#pragma unroll
            for (int j = 0; j < DC; ++j) v[j] += w * a.part[(at + s * step) * D + j * 64 + lane];
        }
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        const int64_t t = rq.row0 + i / a.n_q, h = i % a.n_q;
#pragma unroll
        for (int j = 0; j < DC; ++j)
            a.out[t * a.ldo + h * a.hso + j * 64 + lane] = f32_to_bf16_rne(v[j] * inv);
    }
}

struct AttnShape {
    int32_t splits, split_pages;
};

// Splits of the cached tokens: enough workgroups to fill the card a few times
// over, each with a few pages at least.
AttnShape attn_shape(int64_t T, int64_t R, int32_t n_heads, int32_t n_q, int64_t max_q, int64_t max_kv) {
    const int64_t pages = (max_kv + kPage - 1) / kPage;
    const int64_t tiles = max_q > 0 ? (max_q * (n_q / n_heads) + 15) / 16 : 1;
    const int64_t items = R * n_heads * tiles;
    AttnShape s{1, int32_t(pages > 0 ? pages : 1)};
    const int64_t want = (2048 + items - 1) / items;
    int64_t per = (pages + want - 1) / want;
    if (per < 4) per = 4;
    int64_t n = (pages + per - 1) / per;
    if (n > 64) { n = 64; per = (pages + n - 1) / n; n = (pages + per - 1) / per; }
    if (n > 1) { s.splits = int32_t(n); s.split_pages = int32_t(per); }
    (void)T;
    return s;
}

}  // namespace
}  // namespace ht

using namespace ht;

namespace {

ht_status check_attn(const ht_kv_cache *c, int64_t T, int64_t R, int32_t n_q, int64_t max_q, int64_t max_kv) {
    const ht_status st = check_cache(c);
    if (st != HT_OK) return st;
    if (T < 0 || T > (int64_t(1) << 30) || R <= 0 || R > (int64_t(1) << 20) || n_q <= 0 || n_q > 4096 ||
        n_q % c->n_heads || max_q < 0 || max_kv < 0 || max_q > (int64_t(1) << 30) || max_kv > (int64_t(1) << 30))
        return HT_ESHAPE;
    return HT_OK;
}

template <int DC>
ht_status run_attn(const AttnArgs &a, int64_t R, int64_t max_q, hipStream_t s) {
    const int64_t tiles = (max_q * a.group + 15) / 16;
    const dim3 grid(uint32_t(R * a.n_heads), uint32_t(a.splits), uint32_t(tiles < 1 ? 1 : tiles > 4096 ? 4096 : tiles));
    attn_decode_kernel<DC><<<grid, kAttnThreads, 0, s>>>(a);
    HT_LAUNCH_CHECK();
    if (a.splits > 1) {
        int64_t y = (max_q * a.n_q + kWaves - 1) / kWaves;
        attn_join_kernel<DC><<<dim3(uint32_t(R), uint32_t(y < 1 ? 1 : y > 1024 ? 1024 : y)), kAttnThreads, 0, s>>>(a);
        HT_LAUNCH_CHECK();
    }
    return HT_OK;
}

}  // namespace

extern "C" ht_status ht_kv_attention_workspace(const ht_kv_cache *cache, int64_t T, int64_t R, int32_t n_q,
                                               int64_t max_q, int64_t max_kv, size_t *bytes) {
    if (!bytes) return HT_EINVAL;
    const ht_status st = check_attn(cache, T, R, n_q, max_q, max_kv);
    if (st != HT_OK) return st;
    const AttnShape sh = attn_shape(T, R, cache->n_heads, n_q, max_q, max_kv);
    const size_t rows = size_t(sh.splits) * size_t(T) * size_t(n_q);
    *bytes = sh.splits > 1 ? size_t(align256(rows * 4u)) + rows * size_t(cache->head_dim) * 4u : 0;
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
    if (!(scale == scale) || scale - scale != 0.f) return HT_EINVAL;
    if (T == 0) return HT_OK;
    if ((st = check_rows(q, ldq, hsq, n_q, cache->head_dim, 2)) != HT_OK) return st;
    if ((st = check_rows(out, ldo, hso, n_q, cache->head_dim, 2)) != HT_OK) return st;
    if (!table || !cu_q || !kv_len) return HT_EINVAL;
    if (!al4(table) || !al4(cu_q) || !al4(kv_len) || !al16p(ws)) return HT_EALIGN;
    size_t need = 0;
    if ((st = ht_kv_attention_workspace(cache, T, R, n_q, max_q, max_kv, &need)) != HT_OK) return st;
    if (need > 0 && (!ws || ws_bytes < need)) return HT_ESMALL;
    const AttnShape sh = attn_shape(T, R, cache->n_heads, n_q, max_q, max_kv);
    AttnArgs a{};
    a.q = q;
    a.codes = cache->codes;
    a.scales = cache->scales;
    a.table = table;
    a.cu_q = cu_q;
    a.kv_len = kv_len;
    a.out = out;
    a.lse = static_cast<float *>(ws);
    a.part = sh.splits > 1 ? static_cast<float *>(ws) + align256(size_t(sh.splits) * size_t(T) * size_t(n_q) * 4u) / 4
                           : nullptr;
    a.ldq = ldq; a.hsq = hsq; a.ldo = ldo; a.hso = hso; a.ldt = ldt; a.P = P;
    a.T = int32_t(T);
    a.n_q = n_q;
    a.n_heads = cache->n_heads;
    a.group = n_q / cache->n_heads;
    a.n_pages = int32_t(cache->n_pages);
    a.causal = causal != 0;
    a.splits = sh.splits;
    a.split_pages = sh.split_pages;
    a.window = window;
    a.scale_log2 = scale * kLog2e;
    hipStream_t s = hipStream_t(stream);
    switch (cache->head_dim) {
    case 64: return run_attn<1>(a, R, max_q, s);
    case 128: return run_attn<2>(a, R, max_q, s);
    case 192: return run_attn<3>(a, R, max_q, s);
    default: return run_attn<4>(a, R, max_q, s);
    }
}
