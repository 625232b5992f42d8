// norm.cu -- the norm before the MoE layer and its backward.
//
// Forward, per row of cols values:
//   mu = mean(x) (0 without `center`: the RMS form), r = 1 / sqrt(mean((x - mu)^2) + eps),
//   xhat = (x - mu) r,  y = xhat w + b,
// and in the same pass, if asked for, y in 1 x 128 E4M3 codes (the operand of
// the experts' first product) and xhat in 1 x 128 codes (the checkpoint the
// backward reads in place of x).
// Backward, with a = dy + dy_add, g = a w, m1 = mean(g) (0 without `center`),
// m2 = mean(g xhat):
//   dx = r (g - m1 - xhat m2) + dx_add,  dw = sum_rows a xhat,  db = sum_rows a.
// Everything between the loads and the stores is fp32.
#include "common.cuh"

namespace moe {
namespace norm {

constexpr int MAX_COLS = 16384;

// ---- rows of bf16 or fp32, VEC elements at a time (16 bytes, or one element) ----
template <typename T, int VEC>
struct Vec;
template <>
struct Vec<uint16_t, 8> {
    typedef uint4 Raw;
    static __device__ __forceinline__ void get(const Raw &r, float (&f)[8]) { unpack_bf16x8(r, f); }
    static __device__ __forceinline__ Raw put(const float (&f)[8])
    {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                          pack_bf16x2(f[6], f[7]));
    }
};
template <>
struct Vec<float, 4> {
    typedef float4 Raw;
    static __device__ __forceinline__ void get(const Raw &r, float (&f)[4])
    {
        f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w;
    }
    static __device__ __forceinline__ Raw put(const float (&f)[4]) { return make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Vec<uint16_t, 1> {
    typedef uint16_t Raw;
    static __device__ __forceinline__ void get(const Raw &r, float (&f)[1]) { f[0] = bf16_bits_to_f32(r); }
    static __device__ __forceinline__ Raw put(const float (&f)[1])
    {
        return __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    }
};
template <>
struct Vec<float, 1> {
    typedef float Raw;
    static __device__ __forceinline__ void get(const Raw &r, float (&f)[1]) { f[0] = r; }
    static __device__ __forceinline__ Raw put(const float (&f)[1]) { return f[0]; }
};

template <typename T, int VEC>
__device__ __forceinline__ void load(const T *p, float (&f)[VEC])
{
    typedef typename Vec<T, VEC>::Raw Raw;
    Vec<T, VEC>::get(*reinterpret_cast<const Raw *>(p), f);      // may be the output's own memory: a plain load
}
template <typename T, int VEC>
__device__ __forceinline__ void store(T *p, const float (&f)[VEC])
{
    *reinterpret_cast<typename Vec<T, VEC>::Raw *>(p) = Vec<T, VEC>::put(f);
}

// VEC values of a weight (bf16 or fp32) from column c on; NULL gives `none`
template <int VEC>
__device__ __forceinline__ void load_weight(const void *w, bool f32, int c, float none, float (&f)[VEC])
{
    if (!w) {
#pragma unroll
        for (int i = 0; i < VEC; i++) f[i] = none;
    } else if (f32) {
        if (VEC == 1) {
            f[0] = __ldg(static_cast<const float *>(w) + c);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; i += 4) {
                const float4 v = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + c + i));
                f[i] = v.x, f[(i + 1) % VEC] = v.y, f[(i + 2) % VEC] = v.z, f[(i + 3) % VEC] = v.w;
            }
        }
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(w) + c;
        if (VEC == 1) {
            f[0] = bf16_bits_to_f32(__ldg(p));
        } else {
#pragma unroll
            for (int i = 0; i < VEC; i += 4) {
                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p + i));
                f[i] = __uint_as_float(v.x << 16), f[(i + 1) % VEC] = __uint_as_float(v.x & 0xFFFF0000u);
                f[(i + 2) % VEC] = __uint_as_float(v.y << 16), f[(i + 3) % VEC] = __uint_as_float(v.y & 0xFFFF0000u);
            }
        }
    }
}

// Sums of a and b over the warps of a row's group: shuffles, then the warps'
// parts added in warp order by every thread (the same bits in each).  `red`
// is this round's own buffer of the group; `bar` its named barrier (0: the
// whole CTA), `warps` of one: no exchange.
__device__ __forceinline__ void row_sums(float &a, float &b, float2 *red, int warps, int warp, int lane, int bar)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    if (warps == 1) return;
    if (lane == 0) red[warp] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(warps * 32) : "memory");
    a = b = 0.0f;
    for (int w = 0; w < warps; w++) {
        a += red[w].x;
        b += red[w].y;
    }
}

// ------------------------------------------------------------------ forward

struct Fwd {
    const void *x, *w, *b;
    void *y;
    float *mean, *rstd;
    uint8_t *y_q, *h_q;         // codes of y and of xhat, [rows, cols]
    float *y_s, *h_s;           // their scales, [rows, cols / 128]
    int64_t rows, ld_x, ld_y;
    int cols, warps;            // warps of a row (a divisor of the CTA's, or all of them)
    float eps;
    bool center, w_f32;
};

// VEC consecutive values of a row, 128 / VEC lanes a block, to codes
template <int VEC>
__device__ __forceinline__ void encode(const float (&v)[VEC], bool in, int lane, int64_t at, uint8_t *q, float *s)
{
    if constexpr (VEC >= 4) {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < VEC; i++) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
        for (int o = 64 / VEC; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        const float sc = block_scale(amax);
        if (!in) return;
        const float y = scale_recip(sc);
        const uint32_t lo = e4m3x4_div<2>(v[0], v[1], v[2], v[3], sc, y);
        if constexpr (VEC == 8)
            *reinterpret_cast<uint2 *>(q + at) = make_uint2(lo, e4m3x4_div<2>(v[4], v[5], v[6], v[7], sc, y));
        else
            *reinterpret_cast<uint32_t *>(q + at) = lo;
        if ((lane & (128 / VEC - 1)) == 0) s[at >> 7] = sc;
    }
}

// One row per group of warps, the row held in registers (EPT values a
// thread) from its one load to the stores.  The mean is taken twice: the sum
// of x - mu' with the first mean mu' gives what rounding left out of it, at
// no further exchange (it rides with the sum of squares).
template <typename T, int VEC, int EPT>
__global__ void __launch_bounds__(EPT == 8 ? 1024 : 512) norm_kernel(Fwd p)
{
    constexpr int VPT = EPT / VEC;
    __shared__ float2 red[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = warp / p.warps;
    const int64_t row = (int64_t)blockIdx.x * ((blockDim.x >> 5) / p.warps) + group;
    if (row >= p.rows) return;                         // only where a row is one warp: no barrier below
    const int t = threadIdx.x - group * p.warps * 32, nth = p.warps * 32;
    const T *x = static_cast<const T *>(p.x) + row * p.ld_x;
    const float inv_n = 1.0f / (float)p.cols;
    float v[VPT][VEC];
    float sum = 0.0f, sq = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int c = (t + i * nth) * VEC;
        if (c < p.cols) {
            load<T, VEC>(x + c, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; j++) v[i][j] = 0.0f;
        }
    }
    if (p.center) {
#pragma unroll
        for (int i = 0; i < VPT; i++) {
#pragma unroll
            for (int j = 0; j < VEC; j++) sum += v[i][j];
        }
        row_sums(sum, sq, red[0], p.warps, warp - group * p.warps, lane, 0);
    }
    const float mu = sum * inv_n;
    sum = sq = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const bool in = (t + i * nth) * VEC < p.cols;
#pragma unroll
        for (int j = 0; j < VEC; j++) {
            v[i][j] = in ? v[i][j] - mu : 0.0f;
            sum += v[i][j];
            sq = fmaf(v[i][j], v[i][j], sq);
        }
    }
    row_sums(sum, sq, red[1], p.warps, warp - group * p.warps, lane, 0);
    const float rest = p.center ? sum * inv_n : 0.0f;
    float var = fmaf(sq, inv_n, -rest * rest);
    if (var < 0.0f) var = 0.0f;                        // a NaN stays
    const float rstd = rsqrtf(var + p.eps);
    if (t == 0) {
        if (p.mean) p.mean[row] = mu + rest;
        if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int c = (t + i * nth) * VEC;
        const bool in = c < p.cols;
        float w[VEC], b[VEC], y[VEC];
#pragma unroll
        for (int j = 0; j < VEC; j++) v[i][j] = (v[i][j] - rest) * rstd;
        if (p.h_q) encode<VEC>(v[i], in, lane, row * p.cols + c, p.h_q, p.h_s);
        if (in) {
            load_weight<VEC>(p.w, p.w_f32, c, 1.0f, w);
            load_weight<VEC>(p.b, p.w_f32, c, 0.0f, b);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; j++) w[j] = b[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < VEC; j++) y[j] = fmaf(v[i][j], w[j], b[j]);
        if (in) store<T, VEC>(static_cast<T *>(p.y) + row * p.ld_y + c, y);
        if (p.y_q) encode<VEC>(y, in, lane, row * p.cols + c, p.y_q, p.y_s);
    }
}

// ----------------------------------------------------------------- backward

struct Bwd {
    const void *dy, *x, *dx_add, *w;
    const float *dy_add;        // [rows, cols]
    const uint8_t *h_q;         // xhat's codes and scales (then no x)
    const float *h_s;
    const float *mean, *rstd;
    void *dx;
    float *part;                // per CTA: cols sums of a xhat, cols sums of a
    int64_t rows, ld_dy, ld_x, ld_add, ld_dx;
    int cols, warps, groups;
    bool center, w_f32, want_w, want_b;
};

// Rows over groups of warps, grid-wide in turn; a thread owns the same EPT
// columns of every row of its group, so the sums over rows stay in registers
// until the CTA's last row.  Then the groups' sums are joined in group order
// through shared memory and leave as this CTA's part; reduce_kernel adds the
// parts in CTA order (no atomics: the same bits every time).
template <typename T, int VEC, int EPT, bool CKPT>
__global__ void __launch_bounds__(512) dnorm_kernel(Bwd p)
{
    constexpr int VPT = EPT / VEC;
    extern __shared__ float joined[];                  // [2][cols], groups > 1
    __shared__ float2 red[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = warp / p.warps, gw = warp - group * p.warps;
    const int t = threadIdx.x - group * p.warps * 32, nth = p.warps * 32;
    const float inv_n = 1.0f / (float)p.cols;
    float w[VPT][VEC], dw[VPT][VEC], db[VPT][VEC];
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int c = (t + i * nth) * VEC;
        if (c < p.cols) load_weight<VEC>(p.w, p.w_f32, c, 1.0f, w[i]);
#pragma unroll
        for (int j = 0; j < VEC; j++) {
            if (c >= p.cols) w[i][j] = 0.0f;
            dw[i][j] = db[i][j] = 0.0f;
        }
    }
    const int64_t step = (int64_t)gridDim.x * p.groups;
    int par = 0;
    for (int64_t row = (int64_t)blockIdx.x * p.groups + group; row < p.rows; row += step, par ^= 1) {
        const float rs = __ldg(p.rstd + row), mu = p.center && !CKPT ? __ldg(p.mean + row) : 0.0f;
        float g[VPT][VEC], h[VPT][VEC];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int c = (t + i * nth) * VEC;
            if (c < p.cols) {
                float a[VEC];
                load<T, VEC>(static_cast<const T *>(p.dy) + row * p.ld_dy + c, a);
                if (p.dy_add) {
#pragma unroll
                    for (int j = 0; j < VEC; j++) a[j] += __ldg(p.dy_add + row * p.cols + c + j);
                }
                if constexpr (CKPT) {
                    const float sc = __ldg(p.h_s + ((row * p.cols + c) >> 7));
#pragma unroll
                    for (int j = 0; j < VEC; j++) {
                        __nv_fp8_e4m3 q;
                        q.__x = __ldg(p.h_q + row * p.cols + c + j);
                        h[i][j] = (float)q * sc;
                    }
                } else {
                    load<T, VEC>(static_cast<const T *>(p.x) + row * p.ld_x + c, h[i]);
#pragma unroll
                    for (int j = 0; j < VEC; j++) h[i][j] = (h[i][j] - mu) * rs;
                }
#pragma unroll
                for (int j = 0; j < VEC; j++) {
                    g[i][j] = a[j] * w[i][j];
                    s1 += g[i][j];
                    s2 = fmaf(g[i][j], h[i][j], s2);
                    dw[i][j] = fmaf(a[j], h[i][j], dw[i][j]);
                    db[i][j] += a[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < VEC; j++) g[i][j] = h[i][j] = 0.0f;
            }
        }
        if (!p.dx) continue;
        // the buffer alternates by row: a warp a row ahead writes the other one
        row_sums(s1, s2, red[par] + group * p.warps, p.warps, gw, lane, group + 1);
        const float m1 = p.center ? s1 * inv_n : 0.0f, m2 = s2 * inv_n;
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int c = (t + i * nth) * VEC;
            if (c >= p.cols) continue;
            float d[VEC], add[VEC];
#pragma unroll
            for (int j = 0; j < VEC; j++) d[j] = rs * (g[i][j] - fmaf(h[i][j], m2, m1));
            if (p.dx_add) {
                load<T, VEC>(static_cast<const T *>(p.dx_add) + row * p.ld_add + c, add);
#pragma unroll
                for (int j = 0; j < VEC; j++) d[j] += add[j];
            }
            store<T, VEC>(static_cast<T *>(p.dx) + row * p.ld_dx + c, d);
        }
    }
    if (!p.want_w && !p.want_b) return;
    for (int gr = 0; gr < p.groups; gr++) {
        if (group == gr) {
#pragma unroll
            for (int i = 0; i < VPT; i++) {
#pragma unroll
                for (int j = 0; j < VEC; j++) {
                    const int c = (t + i * nth) * VEC + j;
                    if (c >= p.cols) continue;
                    if (gr) {
                        dw[i][j] = joined[c] + dw[i][j];
                        db[i][j] = joined[p.cols + c] + db[i][j];
                    }
                    if (gr + 1 < p.groups) {
                        joined[c] = dw[i][j];
                        joined[p.cols + c] = db[i][j];
                    } else {
                        float *out = p.part + (int64_t)blockIdx.x * 2 * p.cols;
                        out[c] = dw[i][j];
                        out[p.cols + c] = db[i][j];
                    }
                }
            }
        }
        if (p.groups > 1) __syncthreads();
    }
}

// dw and db: the CTAs' parts, 32 columns a CTA, eight runs of parts at a time
// joined in run order
__global__ void __launch_bounds__(256) reduce_kernel(const float *__restrict__ part, int parts, int cols, float *dw,
                                                     float *db)
{
    __shared__ float run[8][32];
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float *out = blockIdx.y ? db : dw;
    if (!out) return;
    float s = 0.0f;
    if (c < cols)
        for (int i = k; i < parts; i += 8) s += __ldg(part + ((int64_t)i * 2 + blockIdx.y) * cols + c);
    run[k][lane] = s;
    __syncthreads();
    if (k || c >= cols) return;
    for (int i = 1; i < 8; i++) s += run[i][lane];
    out[c] = s;
}

// ------------------------------------------------------------------- host

static bool overlap(const void *a, int64_t na, const void *b, int64_t nb)
{
    if (!a || !b) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// whether the rows of an output (elements es wide) lie over an input's other
// than row on row: a row would be written before another is read
static bool clash(const void *out, int64_t ld_out, const void *in, int64_t ld_in, int64_t rows, int cols, int es)
{
    if (!overlap(out, ((rows - 1) * ld_out + cols) * es, in, ((rows - 1) * ld_in + cols) * es)) return false;
    if (out == in) return rows > 1 && ld_out != ld_in;
    if (rows == 1 || ld_out != ld_in) return true;
    const int64_t off = ((int64_t)((intptr_t)out - (intptr_t)in) / es % ld_in + ld_in) % ld_in;
    return off < cols || ld_in - off < cols;             // two columns' ranges of one buffer are apart
}

static bool rows_aligned(const void *p, int64_t ld, int64_t rows, int es, int bytes)
{
    return (reinterpret_cast<uintptr_t>(p) % bytes) == 0 && (rows <= 1 || (ld * es) % bytes == 0);
}

static bool size_ok(int64_t rows, int64_t cols) { return rows >= 0 && rows < (1LL << 31) && cols >= 1 && cols <= MAX_COLS; }

// CTAs of the backward (their parts of dw and db are what the workspace holds)
static int bwd_ctas(int64_t rows, int groups)
{
    const int64_t n = (rows + groups - 1) / groups;
    return (int)(n < sm_count() ? n : sm_count());
}

template <int EPT>
static void fwd_launch(const Fwd &p, bool f32, bool vec, unsigned grid, int threads, cudaStream_t st)
{
    if (f32)
        vec ? norm_kernel<float, 4, EPT><<<grid, threads, 0, st>>>(p) : norm_kernel<float, 1, EPT><<<grid, threads, 0, st>>>(p);
    else
        vec ? norm_kernel<uint16_t, 8, EPT><<<grid, threads, 0, st>>>(p) : norm_kernel<uint16_t, 1, EPT><<<grid, threads, 0, st>>>(p);
}

template <int EPT>
static void bwd_launch(const Bwd &p, bool f32, bool vec, int grid, int threads, size_t smem, cudaStream_t st)
{
    if (p.h_q) {
        if (f32)
            dnorm_kernel<float, 4, EPT, true><<<grid, threads, smem, st>>>(p);
        else
            dnorm_kernel<uint16_t, 8, EPT, true><<<grid, threads, smem, st>>>(p);
    } else if (f32) {
        vec ? dnorm_kernel<float, 4, EPT, false><<<grid, threads, smem, st>>>(p)
            : dnorm_kernel<float, 1, EPT, false><<<grid, threads, smem, st>>>(p);
    } else {
        vec ? dnorm_kernel<uint16_t, 8, EPT, false><<<grid, threads, smem, st>>>(p)
            : dnorm_kernel<uint16_t, 1, EPT, false><<<grid, threads, smem, st>>>(p);
    }
}

} // namespace norm
} // namespace moe

using namespace moe;
using namespace moe::norm;

MOE_API moe_status moe_layer_norm(const void *x, int dtype, int64_t rows, int64_t cols, int64_t ld_x,
                                  const void *weight, const void *bias, int w_dtype, float eps, int center, void *y,
                                  int64_t ld_y, float *mean, float *rstd, uint8_t *y_q, float *y_s, uint8_t *xhat_q,
                                  float *xhat_s, void *stream)
{
    if (!size_ok(rows, cols) || dtype < 0 || dtype > 1 || w_dtype < 0 || w_dtype > 1 || !(eps >= 0.0f && eps < INFINITY) ||
        (rows > 1 && (ld_x < cols || ld_y < cols)))
        return MOE_ERR_SHAPE;
    if ((y_q || y_s || xhat_q || xhat_s) && cols % 128 != 0) return MOE_ERR_SHAPE;
    if (rows == 0) return MOE_OK;
    if (!x || !y || !y_q != !y_s || !xhat_q != !xhat_s) return MOE_ERR_NULL;
    const bool f32 = dtype == MOE_TYPE_F32;
    const int es = f32 ? 4 : 2, ws = w_dtype == MOE_TYPE_F32 ? 4 : 2;
    const auto aligned_to = [](const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
    if (!aligned_to(x, es) || !aligned_to(y, es) || !aligned_to(weight, ws) || !aligned_to(bias, ws)) return MOE_ERR_ALIGN;
    const int per = 16 / es;                             // values of a whole vector
    const bool vec = cols % per == 0 && rows_aligned(x, ld_x, rows, es, 16) && rows_aligned(y, ld_y, rows, es, 16) &&
                     aligned16(weight) && aligned16(bias);
    if ((y_q || xhat_q) && (!vec || !aligned16(y_q) || !aligned16(xhat_q))) return MOE_ERR_ALIGN;
    if (clash(y, ld_y, x, ld_x, rows, (int)cols, es)) return MOE_ERR_UNSUPPORTED;
    Fwd p{x, weight, bias, y, mean, rstd, y_q, xhat_q, y_s, xhat_s, rows, ld_x, ld_y, (int)cols, 1, eps,
          center != 0, w_dtype == MOE_TYPE_F32};
    // 8 values a thread where rows are few (a row's latency), 32 where there
    // are enough to fill the GPU; 16 in between
    const int ept = rows < sm_count() && cols <= 8192 ? 8 : cols > 8192 || rows >= 8 * sm_count() ? 32 : 16;
    const int nvec = (int)((cols + (vec ? per : 1) - 1) / (vec ? per : 1)), vpt = ept / (vec ? per : 1);
    p.warps = (nvec + 32 * vpt - 1) / (32 * vpt);
    const int per_cta = p.warps == 1 ? 4 : 1;
    const unsigned grid = (unsigned)((rows + per_cta - 1) / per_cta);
    const int threads = p.warps * per_cta * 32;
    cudaStream_t st = as_stream(stream);
    if (ept == 8) fwd_launch<8>(p, f32, vec, grid, threads, st);
    else if (ept == 16) fwd_launch<16>(p, f32, vec, grid, threads, st);
    else fwd_launch<32>(p, f32, vec, grid, threads, st);
    return launch_status();
}

MOE_API size_t moe_layer_norm_backward_workspace_size(int64_t rows, int64_t cols)
{
    if (!size_ok(rows, cols)) return 0;
    return (size_t)bwd_ctas(rows, 1) * 2 * (size_t)cols * sizeof(float);
}

MOE_API moe_status moe_layer_norm_backward(const void *dy, int dtype, int64_t rows, int64_t cols, int64_t ld_dy,
                                           const float *dy_add, const void *x, int64_t ld_x, const uint8_t *xhat_q,
                                           const float *xhat_s, const void *weight, int w_dtype, const float *mean,
                                           const float *rstd, int center, const void *dx_add, int64_t ld_add, void *dx,
                                           int64_t ld_dx, float *dweight, float *dbias, void *workspace,
                                           size_t workspace_bytes, void *stream)
{
    if (!size_ok(rows, cols) || dtype < 0 || dtype > 1 || w_dtype < 0 || w_dtype > 1) return MOE_ERR_SHAPE;
    if (rows > 1 && (ld_dy < cols || (x && ld_x < cols) || (dx_add && ld_add < cols) || (dx && ld_dx < cols)))
        return MOE_ERR_SHAPE;
    if ((xhat_q || xhat_s) && cols % 128 != 0) return MOE_ERR_SHAPE;
    cudaStream_t st = as_stream(stream);
    if (rows == 0) {
        if (dweight && cudaMemsetAsync(dweight, 0, (size_t)cols * 4, st) != cudaSuccess) return MOE_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, (size_t)cols * 4, st) != cudaSuccess) return MOE_ERR_CUDA;
        return MOE_OK;
    }
    if (!dy || !rstd || !x == !xhat_q || !xhat_q != !xhat_s || (center && x && !mean)) return MOE_ERR_NULL;
    if (dx_add && !dx) return MOE_ERR_NULL;
    const bool f32 = dtype == MOE_TYPE_F32;
    const int es = f32 ? 4 : 2, ws = w_dtype == MOE_TYPE_F32 ? 4 : 2;
    const auto aligned_to = [](const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
    if (!aligned_to(dy, es) || !aligned_to(x, es) || !aligned_to(dx_add, es) || !aligned_to(dx, es) ||
        !aligned_to(dy_add, 4) || !aligned_to(weight, ws))
        return MOE_ERR_ALIGN;
    const int per = 16 / es;
    const bool vec = cols % per == 0 && rows_aligned(dy, ld_dy, rows, es, 16) && (!x || rows_aligned(x, ld_x, rows, es, 16)) &&
                     (!dx_add || rows_aligned(dx_add, ld_add, rows, es, 16)) &&
                     (!dx || rows_aligned(dx, ld_dx, rows, es, 16)) && aligned16(dy_add) && aligned16(weight);
    if (xhat_q && (!vec || !aligned16(xhat_q))) return MOE_ERR_ALIGN;
    if (clash(dx, ld_dx, dy, ld_dy, rows, (int)cols, es) || clash(dx, ld_dx, x, ld_x, rows, (int)cols, es) ||
        clash(dx, ld_dx, dx_add, ld_add, rows, (int)cols, es) ||
        (dx && (overlap(dx, ((rows - 1) * ld_dx + cols) * es, dy_add, rows * cols * 4) ||
                overlap(dx, ((rows - 1) * ld_dx + cols) * es, xhat_q, rows * cols))))
        return MOE_ERR_UNSUPPORTED;
    const bool sums = dweight || dbias;
    if (sums && (!workspace || workspace_bytes < moe_layer_norm_backward_workspace_size(rows, cols)))
        return MOE_ERR_WORKSPACE;
    if (sums && !aligned16(workspace)) return MOE_ERR_ALIGN;
    if (!sums && !dx) return MOE_OK;
    Bwd p{dy, x, dx_add, weight, dy_add, xhat_q, xhat_s, mean, rstd, dx, static_cast<float *>(workspace),
          rows, ld_dy, ld_x, ld_add, ld_dx, (int)cols, 1, 1, center != 0, w_dtype == MOE_TYPE_F32, dweight != nullptr,
          dbias != nullptr};
    const int ept = cols > 8192 ? 32 : 16;
    const int unit = vec ? per : 1, nvec = (int)((cols + unit - 1) / unit), vpt = ept / unit;
    p.warps = (nvec + 32 * vpt - 1) / (32 * vpt);
    p.groups = 16 / p.warps;
    if (p.groups > 8) p.groups = 8;
    if (p.groups > rows) p.groups = (int)rows;
    const int grid = bwd_ctas(rows, p.groups);
    const size_t smem = p.groups > 1 ? (size_t)2 * cols * sizeof(float) : 0;
    if (ept == 16) bwd_launch<16>(p, f32, vec, grid, p.warps * p.groups * 32, smem, st);
    else bwd_launch<32>(p, f32, vec, grid, p.warps * p.groups * 32, smem, st);
    if (launch_status() != MOE_OK) return MOE_ERR_CUDA;
    if (sums) {
        reduce_kernel<<<dim3((unsigned)((cols + 31) / 32), 2), 256, 0, st>>>(p.part, grid, (int)cols, dweight, dbias);
        return launch_status();
    }
    return MOE_OK;
}
