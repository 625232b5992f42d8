// losses.cu -- the vocabulary losses of an RL training step: log-probabilities
// of given tokens with the entropy, and the clipped policy loss with a KL
// term together with its gradient in the logits.
//
// Every row t is one softmax over V logits l_v at temperature tau.  With
// k2 = log2(e) / tau and any shift c, t_v = (l_v - c) k2:
//   S = sum_v 2^t_v,  U = sum_v 2^t_v t_v,
//   log p_y = ln2 (t_y - log2 S),  H = ln2 (log2 S - U / S),
// and the gradient of w (pg + beta kl - eta H) / norm is
//   dl_v = coef (g 1[v = y] + 2^t_v / S (-g + eta (ln2 (t_v - log2 S) + H))).
// One shift per thread, the maximum so far, its sums rescaled when it grows;
// the threads' (c, S, U) are joined in a fixed order.  (l_v - c) k2 and not
// l_v k2 - c k2: the largest logit's t is then exactly 0.
#include "common.cuh"

#include <math.h>

namespace moe {

constexpr float LN2 = 0.693147180559945309f;
// where t multiplies 2^t it is held above this: 2^t is 0 there, and 0 times
// an infinite t (a masked logit) would be NaN
constexpr float TMIN = -16384.0f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// the sums of one part of a row, relative to the shift c (c = -inf: no logit
// above -inf so far, S = U = 0)
struct RowSum {
    float c, S, U;
};

// a and b joined: both moved to the larger shift
__device__ __forceinline__ RowSum join(const RowSum &a, const RowSum &b, float k2)
{
    if (b.c == -INFINITY && b.S == 0.0f) return a;
    if (a.c == -INFINITY && a.S == 0.0f) return b;
    const float c = fmaxf(a.c, b.c);
    const float da = fmaxf((a.c - c) * k2, TMIN), db = fmaxf((b.c - c) * k2, TMIN);
    const float fa = ex2(da), fb = ex2(db);
    RowSum r;
    r.c = c;
    r.S = a.S * fa + b.S * fb;
    r.U = (a.U + da * a.S) * fa + (b.U + db * b.S) * fb;
    return r;
}

template <typename T>
__device__ __forceinline__ float load_logit(const T *p);
template <>
__device__ __forceinline__ float load_logit<uint16_t>(const uint16_t *p) { return bf16_bits_to_f32(*p); }
template <>
__device__ __forceinline__ float load_logit<float>(const float *p) { return *p; }

__device__ __forceinline__ void store_grad(uint16_t *p, float v)
{
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    *p = *reinterpret_cast<const uint16_t *>(&b);
}
__device__ __forceinline__ void store_grad(float *p, float v) { *p = v; }

// one element of a thread's part of the row
__device__ __forceinline__ void add_logit(RowSum &s, float l, float k2)
{
    if (l > s.c) {
        if (s.S != 0.0f) {
            const float d = fmaxf((s.c - l) * k2, TMIN), f = ex2(d);
            s.U = (s.U + d * s.S) * f;
            s.S *= f;
        }
        s.c = l;
    }
    if (l == -INFINITY) return;
    const float t = (l - (s.c == -INFINITY ? 0.0f : s.c)) * k2;
    const float e = ex2(t);
    s.S += e;
    s.U = fmaf(e, fmaxf(t, TMIN), s.U);
}

struct PolicyArgs {
    const float *old_lp, *adv, *ref_lp, *w;
    float clip_lo, clip_hi, beta, eta, norm, grad_scale, inv_tau;
    int64_t ld_d;
    double *partial;     // [CTA][5]
};

// exp(q) - q - 1 without the cancellation near 0: its series for |q| < 1/2
__device__ __forceinline__ float kl_term(float q)
{
    if (fabsf(q) < 0.5f) {
        float p = 1.0f;
#pragma unroll
        for (int i = 10; i >= 3; i--) p = fmaf(q * (1.0f / i), p, 1.0f);
        return 0.5f * q * q * p;
    }
    return expf(q) - q - 1.0f;
}

template <typename T, bool POLICY>
__global__ void __launch_bounds__(512) token_rows_kernel(const T *logits, int64_t N, int64_t V,
                                                         int64_t ld, const void *__restrict__ targets, int t64,
                                                         float k2, float *__restrict__ logprobs,
                                                         float *__restrict__ entropy, T *dlogits, PolicyArgs a,
                                                         int32_t *dev_status)
{
    __shared__ RowSum s_part[16];
    __shared__ RowSum s_row;
    __shared__ double s_norm[16];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    double norm = 0.0;
    if (POLICY) {
        if (a.norm > 0.0f) {
            norm = a.norm;
        } else {
            double v = 0.0;
            for (int64_t i = tid; i < N; i += 512) v += a.w ? (double)a.w[i] : 1.0;
            for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            if (lane == 0) s_norm[warp] = v;
            __syncthreads();
            for (int i = 0; i < 16; i++) norm += s_norm[i];
        }
    }
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
    for (int64_t row = blockIdx.x; row < N; row += gridDim.x) {
        const int64_t y = t64 ? ((const int64_t *)targets)[row] : (int64_t)((const int32_t *)targets)[row];
        const float w = POLICY ? (a.w ? a.w[row] : 1.0f) : 1.0f;
        bool live = y >= 0 && y < V && w != 0.0f;
        if (y >= V && w != 0.0f && tid == 0) dev_flag(dev_status, MOE_DEV_BAD_IDS);
        const T *l = logits + row * ld;
        T *d = POLICY && dlogits ? dlogits + row * a.ld_d : nullptr;
        RowSum s = {-INFINITY, 0.0f, 0.0f};
        if (live) {
            for (int64_t i = tid; i < V; i += 512) add_logit(s, load_logit(l + i), k2);
            for (int o = 16; o; o >>= 1) {
                RowSum b;
                b.c = __shfl_xor_sync(0xFFFFFFFFu, s.c, o);
                b.S = __shfl_xor_sync(0xFFFFFFFFu, s.S, o);
                b.U = __shfl_xor_sync(0xFFFFFFFFu, s.U, o);
                s = (lane & o) ? join(b, s, k2) : join(s, b, k2);
            }
            if (lane == 0) s_part[warp] = s;
            __syncthreads();
            if (tid == 0) {
                s = s_part[0];
                for (int i = 1; i < 16; i++) s = join(s, s_part[i], k2);
                s_row = s;
            }
            __syncthreads();
            s = s_row;
            if (s.c == -INFINITY && s.S == 0.0f) {
                live = false;
                if (tid == 0) dev_flag(dev_status, MOE_DEV_BAD_IDS);
            }
        }
        float lp = 0.0f, H = 0.0f, A0 = 0.0f, B0 = 0.0f, gy = 0.0f;
        if (live) {
            const float ls = log2f(s.S);
            lp = LN2 * ((load_logit(l + y) - s.c) * k2 - ls);
            H = LN2 * (ls - s.U / s.S);
            if (POLICY) {
                const float A = a.adv[row];
                float dlt = lp - a.old_lp[row];
                dlt = dlt > 80.0f ? 80.0f : dlt;
                const float r = expf(dlt);
                const float rc = r < a.clip_lo ? a.clip_lo : (r > a.clip_hi ? a.clip_hi : r);
                const float p0 = -A * r, p1 = -A * rc;
                const bool clipped = p1 > p0;
                float g = clipped ? 0.0f : p0, kl = 0.0f;
                if (a.ref_lp) {
                    float q = a.ref_lp[row] - lp;
                    q = q > 80.0f ? 80.0f : q;
                    kl = kl_term(q);
                    g = fmaf(-a.beta, expm1f(q), g);
                }
                if (tid == 0) {
                    acc[0] += (double)w * (clipped ? p1 : p0);
                    acc[1] += (double)w * kl;
                    acc[2] += (double)w * H;
                    acc[3] += clipped ? (double)w : 0.0;
                }
                const float coef = norm != 0.0 ? (float)((double)w * a.grad_scale * a.inv_tau / norm) : 0.0f;
                gy = coef * g;
                A0 = coef * (-g + a.eta * (H - LN2 * ls)) / s.S;
                B0 = coef * a.eta * LN2 / s.S;
            }
        }
        if (tid == 0) {
            if (logprobs) logprobs[row] = lp;
            if (!POLICY && entropy) entropy[row] = H;
        }
        if (POLICY && d) {
            __syncthreads();
            for (int64_t i = tid; i < V; i += 512) {
                float v = 0.0f;
                if (live) {
                    const float t = (load_logit(l + i) - s.c) * k2;
                    v = ex2(t) * fmaf(B0, fmaxf(t, TMIN), A0);
                    if (i == y) v += gy;
                }
                store_grad(d + i, v);
            }
        }
    }
    if (POLICY && tid == 0)
        for (int i = 0; i < 4; i++) a.partial[(int64_t)blockIdx.x * 5 + i] = acc[i];
    if (POLICY && tid == 0) a.partial[(int64_t)blockIdx.x * 5 + 4] = norm;
}

__global__ void policy_stats_kernel(const double *__restrict__ partial, int ncta, float beta, float eta,
                                    float *__restrict__ stats)
{
    double m[4] = {0.0, 0.0, 0.0, 0.0};
    const double norm = partial[4];
    for (int c = 0; c < ncta; c++)
        for (int i = 0; i < 4; i++) m[i] += partial[(int64_t)c * 5 + i];
    for (int i = 0; i < 4; i++) m[i] = norm != 0.0 ? m[i] / norm : 0.0;
    stats[0] = (float)(m[0] + beta * m[1] - eta * m[2]);
    for (int i = 0; i < 4; i++) stats[1 + i] = (float)m[i];
    stats[5] = (float)norm;
}

static moe_status check_rows(const void *logits, int dtype, int64_t N, int64_t V, int64_t ld, const void *targets,
                             int target_bits, float temperature)
{
    if (N < 0 || V < 1 || N >= (1LL << 31) || V >= (1LL << 31) || ld < V) return MOE_ERR_SHAPE;
    if (dtype != MOE_LOGITS_BF16 && dtype != MOE_LOGITS_F32) return MOE_ERR_SHAPE;
    if (target_bits != 32 && target_bits != 64) return MOE_ERR_SHAPE;
    if (!isfinite(temperature) || !(temperature > 0.0f)) return MOE_ERR_SHAPE;
    if (N == 0) return MOE_OK;
    if (!logits || !targets) return MOE_ERR_NULL;
    const uintptr_t es = dtype == MOE_LOGITS_BF16 ? 2 : 4, ts = target_bits / 8;
    if ((uintptr_t)logits % es || (uintptr_t)targets % ts) return MOE_ERR_ALIGN;
    return MOE_OK;
}

constexpr int MAX_ROW_CTAS = 1024;
static unsigned row_grid(int64_t N)
{
    const int64_t g = 4LL * sm_count();
    const int64_t c = g < MAX_ROW_CTAS ? g : MAX_ROW_CTAS;
    return (unsigned)(N < c ? N : c);
}

} // namespace moe

using namespace moe;

MOE_API moe_status moe_token_logprobs(const void *logits, int logits_dtype, int64_t N, int64_t V, int64_t ld,
                                      const void *targets, int target_bits, float temperature, float *logprobs,
                                      float *entropy, int32_t *dev_status, void *stream)
{
    moe_status s = check_rows(logits, logits_dtype, N, V, ld, targets, target_bits, temperature);
    if (s != MOE_OK) return s;
    if (N == 0) return MOE_OK;
    if (!logprobs) return MOE_ERR_NULL;
    const float k2 = (float)(1.4426950408889634 / (double)temperature);
    PolicyArgs a = {};
    if (logits_dtype == MOE_LOGITS_BF16)
        token_rows_kernel<uint16_t, false><<<row_grid(N), 512, 0, as_stream(stream)>>>(
            (const uint16_t *)logits, N, V, ld, targets, target_bits == 64, k2, logprobs, entropy, nullptr, a,
            dev_status);
    else
        token_rows_kernel<float, false><<<row_grid(N), 512, 0, as_stream(stream)>>>(
            (const float *)logits, N, V, ld, targets, target_bits == 64, k2, logprobs, entropy, nullptr, a,
            dev_status);
    return launch_status();
}

MOE_API size_t moe_policy_loss_workspace_size(int64_t N, int64_t V)
{
    (void)N;
    (void)V;
    return sizeof(double) * 5 * MAX_ROW_CTAS;
}

MOE_API moe_status moe_policy_loss(const void *logits, int logits_dtype, int64_t N, int64_t V, int64_t ld,
                                   const void *targets, int target_bits, const float *old_logprobs,
                                   const float *advantages, const float *ref_logprobs, const float *weights,
                                   float temperature, float clip_low, float clip_high, float kl_coef,
                                   float entropy_coef, float norm, float grad_scale, float *stats, float *logprobs,
                                   void *dlogits, int64_t ld_d, void *workspace, size_t workspace_bytes,
                                   int32_t *dev_status, void *stream)
{
    moe_status s = check_rows(logits, logits_dtype, N, V, ld, targets, target_bits, temperature);
    if (s != MOE_OK) return s;
    const float c[6] = {clip_low, clip_high, kl_coef, entropy_coef, norm, grad_scale};
    for (float v : c)
        if (!isfinite(v)) return MOE_ERR_SHAPE;
    if (clip_low < 0.0f || clip_high < 0.0f || norm < 0.0f || (dlogits && ld_d < V)) return MOE_ERR_SHAPE;
    if (!stats) return MOE_ERR_NULL;
    cudaStream_t st = as_stream(stream);
    if (N > 0) {
        if (!old_logprobs || !advantages) return MOE_ERR_NULL;
        if (dlogits && (uintptr_t)dlogits % (logits_dtype == MOE_LOGITS_BF16 ? 2 : 4)) return MOE_ERR_ALIGN;
    }
    if (!workspace || workspace_bytes < moe_policy_loss_workspace_size(N, V)) return MOE_ERR_WORKSPACE;
    if (!aligned16(workspace)) return MOE_ERR_ALIGN;
    if (N == 0)
        return cudaMemsetAsync(stats, 0, 6 * sizeof(float), st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    PolicyArgs a = {old_logprobs, advantages, ref_logprobs, weights, 1.0f - clip_low, 1.0f + clip_high, kl_coef,
                    entropy_coef, norm, grad_scale, 1.0f / temperature, ld_d, (double *)workspace};
    const float k2 = (float)(1.4426950408889634 / (double)temperature);
    const unsigned g = row_grid(N);
    if (logits_dtype == MOE_LOGITS_BF16)
        token_rows_kernel<uint16_t, true><<<g, 512, 0, st>>>((const uint16_t *)logits, N, V, ld, targets,
                                                             target_bits == 64, k2, logprobs, nullptr,
                                                             (uint16_t *)dlogits, a, dev_status);
    else
        token_rows_kernel<float, true><<<g, 512, 0, st>>>((const float *)logits, N, V, ld, targets,
                                                          target_bits == 64, k2, logprobs, nullptr, (float *)dlogits,
                                                          a, dev_status);
    policy_stats_kernel<<<1, 1, 0, st>>>((const double *)workspace, (int)g, ref_logprobs ? kl_coef : 0.0f,
                                         entropy_coef, stats);
    return launch_status();
}
