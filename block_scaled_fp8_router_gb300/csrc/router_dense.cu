// router_dense.cu -- the router over all experts: the balance and z losses with
// per-expert counts and the gradient of the logits, and the entry points of
// the dense products (router_gemm.cu).
#include "router_dense.cuh"

#include <math.h>

namespace moe {

// ------------------------------------------------------------ balance loss

constexpr int MAX_BAL_CTAS = 1024;

// sequence of token t: the b with off[b] <= t < off[b+1], -1 if none (any
// contents of off give some b in [0, B) or -1)
__device__ __forceinline__ int seq_of(const int32_t *__restrict__ off, int B, int t)
{
    if (!off) return 0;
    int lo = 0, hi = B;                 // off[lo] <= t < off[hi], assumed sorted
    if (t < off[0] || t >= off[B]) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// counts[b, e] and n_b over the counted tokens; one thread per slot
__global__ void balance_count_kernel(const int32_t *__restrict__ ids, const uint8_t *__restrict__ mask,
                                     const int32_t *__restrict__ off, int T, int E, int k, int B,
                                     int32_t *__restrict__ counts, int32_t *__restrict__ nb,
                                     int32_t *__restrict__ dev_status)
{
    if (blockIdx.x == 0 && off)
        for (int b = threadIdx.x; b < B; b += blockDim.x)
            if (off[b] < 0 || off[b + 1] < off[b] || off[b + 1] > T) dev_flag(dev_status, MOE_DEV_ROWS);
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < (int64_t)T * k;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int t = (int)(i / k), j = (int)(i - (int64_t)t * k);
        const int b = seq_of(off, B, t);
        if (b < 0 || (mask && !mask[t])) continue;
        const int32_t e = ids[i];
        if (e >= 0 && e < E) atomicAdd(&counts[(int64_t)b * E + e], 1);
        if (j == 0) atomicAdd(&nb[b], 1);
    }
}

__device__ __forceinline__ float wsum(float v)
{
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ float wmax(float v)
{
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

struct BalanceArgs {
    const float *logits, *d_gates;
    const int32_t *ids, *off, *counts, *nb;
    const uint8_t *mask;
    int T, E, k, B, score_fn, renorm;
    float route_scale, alpha, zeta, grad_scale;
    float *d_logits;
    double *partial;    // [CTA][2]
    int32_t *dev_status;
};

// one warp per token, NV = ceil(E / 32) logits per lane
template <int NV>
__global__ void __launch_bounds__(256) balance_rows_kernel(BalanceArgs a)
{
    __shared__ double s_l[8][2];
    __shared__ int s_n, s_used;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) s_n = s_used = 0;
    __syncthreads();
    for (int b = threadIdx.x; b < a.B; b += 256) {
        atomicAdd(&s_n, a.nb[b]);
        if (a.nb[b] > 0) atomicAdd(&s_used, 1);
    }
    __syncthreads();
    const int n = s_n, used = s_used;
    double lb = 0.0, lz = 0.0;
    for (int64_t t = (int64_t)blockIdx.x * 8 + warp; t < a.T; t += (int64_t)gridDim.x * 8) {
        const int b = seq_of(a.off, a.B, (int)t);
        bool counted = b >= 0 && (!a.mask || a.mask[t]);
        const int32_t id = lane < a.k ? a.ids[t * a.k + lane] : -1 - lane;
        const float dg = a.d_gates && lane < a.k ? a.d_gates[t * a.k + lane] : 0.0f;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
        const bool bad = __any_sync(0xFFFFFFFFu, lane < a.k && (id < 0 || id >= a.E || same != (1u << lane)));
        if (bad && lane == 0) dev_flag(a.dev_status, MOE_DEV_BAD_IDS);
        const bool gate = !bad && __any_sync(0xFFFFFFFFu, dg != 0.0f);
        float l[NV], g[NV], m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int e = 32 * i + lane;
            l[i] = (counted || gate) && e < a.E ? a.logits[t * a.E + e] : -INFINITY;
            g[i] = 0.0f;
            m = fmaxf(m, l[i]);
        }
        m = wmax(m);
        const bool none = m == -INFINITY;   // NaN logits leave a NaN sum below
        float ex[NV], tot = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int e = 32 * i + lane;
            ex[i] = e < a.E ? expf(l[i] - (none ? 0.0f : m)) : 0.0f;
            tot += ex[i];
        }
        tot = wsum(tot);
        if (tot == 0.0f) counted = false;
        if (counted) {
            const float lse = m + logf(tot), it = 1.0f / tot;
            const int nbv = a.nb[b];
            const float fs = (float)((double)a.E / ((double)a.k * nbv));
            const float share = (float)((double)a.alpha / ((double)used * nbv));
            const int32_t *cnt = a.counts + (int64_t)b * a.E;
            float dot = 0.0f, S = 0.0f;
            if (a.score_fn == MOE_SCORE_SIGMOID) {
#pragma unroll
                for (int i = 0; i < NV; i++) S += 32 * i + lane < a.E ? 1.0f / (1.0f + expf(-l[i])) : 0.0f;
                S = 1.0f / wsum(S);
            }
            float f[NV], q[NV];
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int e = 32 * i + lane;
                f[i] = e < a.E ? fs * cnt[e] : 0.0f;
                q[i] = a.score_fn == MOE_SCORE_SIGMOID ? S / (1.0f + expf(-l[i])) : ex[i] * it;
                dot += e < a.E ? f[i] * q[i] : 0.0f;
            }
            dot = wsum(dot);
            const float cb = a.grad_scale * share, cz = a.grad_scale * 2.0f * a.zeta * lse / n;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                float sl = q[i];
                if (a.score_fn == MOE_SCORE_SIGMOID) sl = q[i] / (1.0f + expf(l[i]));
                g[i] = cb * sl * (f[i] - dot) + cz * (ex[i] * it);
            }
            if (lane == 0) {
                lb += (double)share * dot;
                lz += (double)lse * lse;
            }
        }
        if (!a.d_logits) continue;
        if (gate) {
            const float my = lane < a.k ? a.logits[t * a.E + id] : 0.0f;
            const bool mine = lane < a.k;
            float dl;
            if (a.score_fn == MOE_SCORE_SOFTMAX) {
                if (a.renorm) {
                    const float mm = wmax(mine ? my : -INFINITY);
                    const float e = mine ? expf(my - mm) : 0.0f;
                    const float p = e / wsum(e);
                    dl = p * (dg - wsum(dg * p));
                } else {
                    const float p = mine ? expf(my - m) / tot : 0.0f;
                    const float dot = wsum(dg * p);
                    dl = dg * p;
#pragma unroll
                    for (int i = 0; i < NV; i++) g[i] -= a.route_scale * dot * (ex[i] / tot);
                }
            } else {
                const float s = mine ? 1.0f / (1.0f + expf(-my)) : 0.0f;
                const float ds = mine ? s / (1.0f + expf(my)) : 0.0f;
                if (a.renorm) {
                    const float S = wsum(s), dot = wsum(dg * s);
                    dl = ds * ((dg - dot / S) / S);
                } else {
                    dl = ds * dg;
                }
            }
            dl *= a.route_scale;
            for (int j = 0; j < a.k; j++) {
                const int e = __shfl_sync(0xFFFFFFFFu, id, j);
                const float v = __shfl_sync(0xFFFFFFFFu, dl, j);
#pragma unroll
                for (int i = 0; i < NV; i++)
                    if (e == 32 * i + lane) g[i] += v;
            }
        }
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (32 * i + lane < a.E) a.d_logits[t * a.E + 32 * i + lane] = g[i];
    }
    if (lane == 0) {
        s_l[warp][0] = lb;
        s_l[warp][1] = lz;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        double v = 0.0;
        for (int i = 0; i < 8; i++) v += s_l[i][threadIdx.x];
        if (threadIdx.x == 1) v = n > 0 ? v * a.zeta / n : 0.0;
        a.partial[(int64_t)blockIdx.x * 2 + threadIdx.x] = v;
    }
}

__global__ void balance_losses_kernel(const double *__restrict__ partial, int ncta, float *__restrict__ losses)
{
    if (threadIdx.x >= 2) return;
    double v = 0.0;
    for (int c = 0; c < ncta; c++) v += partial[(int64_t)c * 2 + threadIdx.x];
    losses[threadIdx.x] = (float)v;
}

static bool aligned256(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

static moe_status check_dense(int T, int d, int E)
{
    if (T < 0 || d <= 0 || d % 128 != 0 || E < 1 || E > 1024) return MOE_ERR_SHAPE;
    return MOE_OK;
}

} // namespace moe

using namespace moe;

MOE_API size_t moe_router_logits_workspace_size(int T, int d, int E)
{
    return check_dense(T, d, E) == MOE_OK ? router_logits_workspace(T, d, E) : 0;
}

MOE_API moe_status moe_router_logits(const uint16_t *x, const uint16_t *w_router, int T, int d, int E, float *logits,
                                     void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    moe_status s = check_dense(T, d, E);
    if (s != MOE_OK) return s;
    if (T == 0) return MOE_OK;
    if (!x || !w_router || !logits) return MOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(w_router)) return MOE_ERR_ALIGN;
    if (!workspace || workspace_bytes < moe_router_logits_workspace_size(T, d, E)) return MOE_ERR_WORKSPACE;
    if (!aligned256(workspace)) return MOE_ERR_ALIGN;
    return router_logits(x, w_router, T, d, E, logits, workspace, dev_status, as_stream(stream));
}

MOE_API size_t moe_balance_loss_workspace_size(int T, int E, int B)
{
    (void)T; (void)E;
    return sizeof(double) * 2 * MAX_BAL_CTAS + sizeof(int32_t) * (size_t)(B > 0 ? B : 1);
}

MOE_API moe_status moe_balance_loss(const float *logits, const int32_t *topk_ids, const uint8_t *token_mask,
                                    const int32_t *seq_offsets, int T, int E, int k, int B, int score_fn, int renorm,
                                    float route_scale, float balance_coef, float z_coef, float grad_scale,
                                    const float *d_gates, int32_t *counts, float *losses, float *d_logits,
                                    void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    if (T < 0 || E < 1 || E > 1024 || k < 1 || k > 32 || k > E || B < 1 || B > 65535) return MOE_ERR_SHAPE;
    if (B > 1 && !seq_offsets) return MOE_ERR_SHAPE;
    if ((int64_t)T * k >= (1LL << 31)) return MOE_ERR_SHAPE;
    if (score_fn != MOE_SCORE_SOFTMAX && score_fn != MOE_SCORE_SIGMOID) return MOE_ERR_SHAPE;
    if (!isfinite(route_scale) || !isfinite(balance_coef) || !isfinite(z_coef) || !isfinite(grad_scale))
        return MOE_ERR_SHAPE;
    if (!counts || !losses) return MOE_ERR_NULL;
    if (T > 0 && (!logits || !topk_ids)) return MOE_ERR_NULL;
    if (!workspace || workspace_bytes < moe_balance_loss_workspace_size(T, E, B)) return MOE_ERR_WORKSPACE;
    if (!aligned256(workspace)) return MOE_ERR_ALIGN;
    cudaStream_t st = as_stream(stream);
    if (cudaMemsetAsync(counts, 0, sizeof(int32_t) * (size_t)B * E, st) != cudaSuccess) return MOE_ERR_CUDA;
    if (T == 0) return cudaMemsetAsync(losses, 0, 2 * sizeof(float), st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    double *partial = (double *)workspace;
    int32_t *nb = (int32_t *)(partial + 2 * MAX_BAL_CTAS);
    if (cudaMemsetAsync(nb, 0, sizeof(int32_t) * (size_t)B, st) != cudaSuccess) return MOE_ERR_CUDA;
    const int64_t slots = (int64_t)T * k;
    const int64_t cg = (slots + 255) / 256, cmax = 4LL * sm_count();
    balance_count_kernel<<<(unsigned)(cg < cmax ? cg : cmax), 256, 0, st>>>(topk_ids, token_mask, seq_offsets, T, E, k,
                                                                           B, counts, nb, dev_status);
    BalanceArgs a = {logits, d_gates, topk_ids, seq_offsets, counts, nb, token_mask, T, E, k, B, score_fn, renorm,
                     route_scale, balance_coef, z_coef, grad_scale, d_logits, partial, dev_status};
    const int64_t rg = ((int64_t)T + 7) / 8, rmax = 4LL * sm_count();
    int64_t g = rg < rmax ? rg : rmax;
    if (g > MAX_BAL_CTAS) g = MAX_BAL_CTAS;
    if (E <= 32) balance_rows_kernel<1><<<(unsigned)g, 256, 0, st>>>(a);
    else if (E <= 64) balance_rows_kernel<2><<<(unsigned)g, 256, 0, st>>>(a);
    else if (E <= 128) balance_rows_kernel<4><<<(unsigned)g, 256, 0, st>>>(a);
    else if (E <= 256) balance_rows_kernel<8><<<(unsigned)g, 256, 0, st>>>(a);
    else if (E <= 512) balance_rows_kernel<16><<<(unsigned)g, 256, 0, st>>>(a);
    else balance_rows_kernel<32><<<(unsigned)g, 256, 0, st>>>(a);
    balance_losses_kernel<<<1, 32, 0, st>>>(partial, (int)g, losses);
    return launch_status();
}

MOE_API size_t moe_router_backward_dense_workspace_size(int T, int d, int E)
{
    return check_dense(T, d, E) == MOE_OK ? router_backward_workspace(T, d, E) : 0;
}

MOE_API moe_status moe_router_backward_dense(const uint16_t *x, const uint16_t *w_router, const float *d_logits, int T,
                                             int d, int E, float *dx, float *dw_router, void *workspace,
                                             size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    moe_status s = check_dense(T, d, E);
    if (s != MOE_OK) return s;
    cudaStream_t st = as_stream(stream);
    if (dw_router && !aligned16(dw_router)) return MOE_ERR_ALIGN;
    if (T == 0) {
        if (!dw_router) return MOE_OK;
        return cudaMemsetAsync(dw_router, 0, sizeof(float) * (size_t)E * d, st) == cudaSuccess ? MOE_OK
                                                                                             : MOE_ERR_CUDA;
    }
    if (!dx && !dw_router) return MOE_OK;
    if (!d_logits || (dw_router && !x) || (dx && !w_router)) return MOE_ERR_NULL;
    if ((x && !aligned16(x)) || (w_router && !aligned16(w_router)) || (dx && !aligned16(dx))) return MOE_ERR_ALIGN;
    if (!workspace || workspace_bytes < moe_router_backward_dense_workspace_size(T, d, E)) return MOE_ERR_WORKSPACE;
    if (!aligned256(workspace)) return MOE_ERR_ALIGN;
    return router_backward(x, w_router, d_logits, T, d, E, dx, dw_router, workspace, dev_status, st);
}
