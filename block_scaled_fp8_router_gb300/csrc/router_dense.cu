// router_dense.cu -- the router over all experts: the balance and z losses with
// per-expert counts and the gradient of the logits, and the entry points of
// the dense products (router_gemm.cu).
#include "losses.cuh"
#include "router_dense.cuh"

#include <math.h>

namespace moe {

// ------------------------------------------------------------ balance loss
//
// The loss is linear in the probabilities once the counts are known:
//   sum_b sum_e f[b,e] P[b,e] / B' = sum_t share_b(t) dot_t, dot_t = sum_e f[b,e] q[t,e],
// and dot_t is what the gradient needs anyway:
//   softmax: d q.f / d l_e = q_e (f_e - dot),
//   sigmoid: d q.f / d l_e = q_e (1 - s_e) (f_e - dot), q = s / sum s.
// So one pass over the ids gives the counts and one pass over the logits the
// losses and the gradient: each logit is read once and its gradient written
// once.  balance_rows_kernel gives each token G lanes (8, 16 or 32, four
// experts of a 16-byte load each), each warp a run of consecutive tokens: f of
// the run's sequence stays in registers, the next token's loads are under way
// while this one is worked on.  The gates' k gradients go through a row of
// shared memory.  The losses are summed in two fp32 numbers per warp and joined by
// the CTA that finishes last, in order.
//
// Bound: the latency of dependent instructions at 16 warps an SM.  131072 x 256
// sigmoid with gates: 72 us, 3.7 TB/s read and written, 57% of the issue slots;
// no pipe is full (special functions 19%, FMA 32%, integer and logic 34%), and an
// issued instruction stands against 1.7 warps on fixed latencies, 1.1 on global
// and 0.9 on shared memory and the special functions.  8192 x 256 13.5 us in all,
// its two launches.

constexpr int HIST_MAX = 64;            // CTAs of the count when there is one sequence
constexpr int ROW_CTAS_MAX = 1024;

// workspace
struct BalWs {
    uint32_t done, pad[3];
    Sum2 loss[ROW_CTAS_MAX][2];
    int32_t hist[HIST_MAX][1024 + 1];   // one sequence: counts of each CTA's tokens, then the counted tokens
    int32_t nb[1];                      // several sequences: counted tokens of each
};

// sequence of token t: the b with off[b] <= t < off[b+1], -1 if none (any
// contents of off give some b in [0, B) or -1)
__device__ __forceinline__ int seq_of(const int32_t *__restrict__ off, int B, int t)
{
    if (!off) return 0;
    int lo = 0, hi = B;                 // off[lo] <= t < off[hi] for sorted offsets
    if (t < __ldg(off) || t >= __ldg(off + B)) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(off + mid) <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// first token after t that may be in another sequence than b
__device__ __forceinline__ int seq_end(const int32_t *__restrict__ off, int b, int t, int T)
{
    if (!off) return T;
    if (b < 0) return t + 1;
    const int e = __ldg(off + b + 1);
    return e > t ? (e < T ? e : T) : t + 1;
}

__global__ void balance_zero_kernel(int32_t *__restrict__ counts, int64_t n, int32_t *__restrict__ nb, int B, BalWs *ws)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, st = (int64_t)gridDim.x * blockDim.x;
    for (int64_t j = i; j < n; j += st) counts[j] = 0;
    for (int64_t j = i; j < B; j += st) nb[j] = 0;
    if (i == 0) ws->done = 0;
}

// counts of the tokens [t0, t1) of one CTA (1024 threads), a sequence at a
// time, in shared memory.  One sequence: the CTA's counts go to its row of
// ws->hist; several: they are added to counts and nb (zeroed before).
__global__ void __launch_bounds__(1024) balance_count_kernel(const int32_t *__restrict__ ids,
                                                             const uint8_t *__restrict__ mask,
                                                             const int32_t *__restrict__ off, int T, int E, int k, int B,
                                                             int32_t *counts, int32_t *nb, BalWs *ws,
                                                             int32_t *dev_status)
{
    __shared__ int32_t s_hist[1024 + 1];
    const int tid = threadIdx.x;
    const int t0 = (int)((int64_t)blockIdx.x * T / gridDim.x), t1 = (int)((int64_t)(blockIdx.x + 1) * T / gridDim.x);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = tid; i <= E; i += 1024) s_hist[i] = 0;
    __syncthreads();
    if (off && blockIdx.x == 0)
        for (int b = tid; b < B; b += 1024)
            if (off[b] < 0 || off[b + 1] < off[b] || off[b + 1] > T) dev_flag(dev_status, MOE_DEV_ROWS);
    const bool one = B == 1 && !off;
    const bool v4 = k % 4 == 0 && (reinterpret_cast<uintptr_t>(ids) & 15u) == 0;
    if (!one) asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int t = t0; t < t1;) {
        const int b = seq_of(off, B, t);
        int e1 = seq_end(off, b, t, T);
        e1 = e1 < t1 ? e1 : t1;
        if (b >= 0) {
            int32_t mine = 0;
            for (int i = t + tid; i < e1; i += 1024) {          // a token a thread
                if (mask && !__ldg(mask + i)) continue;
                mine++;
                const int32_t *p = ids + (int64_t)i * k;
                for (int j = 0; j < k; j += 8) {
                    int32_t e[8];
                    if (v4) {
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const int4 q = j + 4 * h < k ? __ldg(reinterpret_cast<const int4 *>(p + j + 4 * h))
                                                         : make_int4(-1, -1, -1, -1);
                            e[4 * h] = q.x;
                            e[4 * h + 1] = q.y;
                            e[4 * h + 2] = q.z;
                            e[4 * h + 3] = q.w;
                        }
                    } else {
#pragma unroll
                        for (int u = 0; u < 8; u++) e[u] = j + u < k ? __ldg(p + j + u) : -1;
                    }
#pragma unroll
                    for (int u = 0; u < 8; u++)
                        if ((uint32_t)e[u] < (uint32_t)E) atomicAdd(&s_hist[e[u]], 1);
                }
            }
            mine = __reduce_add_sync(0xFFFFFFFFu, mine);
            if ((tid & 31) == 0 && mine) atomicAdd(&s_hist[E], mine);
            __syncthreads();
            if (!one) {
                for (int i = tid; i < E; i += 1024)
                    if (s_hist[i]) {
                        atomicAdd(&counts[(int64_t)b * E + i], s_hist[i]);
                        s_hist[i] = 0;
                    }
                if (tid == 0) {
                    if (s_hist[E]) atomicAdd(&nb[b], s_hist[E]);
                    s_hist[E] = 0;
                }
                __syncthreads();
            }
        }
        t = e1;
    }
    if (one) {
        for (int i = tid; i <= E; i += 1024) ws->hist[blockIdx.x][i] = s_hist[i];
        if (blockIdx.x == 0 && tid == 0) ws->done = 0;
    }
}

struct BalanceArgs {
    const float *logits, *d_gates;
    const int32_t *ids, *off;
    const uint8_t *mask;
    int T, E, k, B, score_fn, renorm;
    float route_scale, alpha, zeta, grad_scale;
    int32_t *counts;
    float *losses, *d_logits;
    BalWs *ws;
    int32_t *nb;
    int nhist;         // CTAs whose counts to add up (one sequence); 0: this CTA, the only one, counts itself
    int vec;           // rows of four-expert vectors, 16-byte aligned
    int32_t *dev_status;
};

template <int G>
__device__ __forceinline__ float gsum(float v)
{
#pragma unroll
    for (int o = G / 2; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
template <int G>
__device__ __forceinline__ float gmax(float v)
{
#pragma unroll
    for (int o = G / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// the larger of the group's values; a NaN may count as the largest
template <int G>
__device__ __forceinline__ float gmaxf(float v)
{
    if (G < 32) return gmax<G>(v);
    const int i = __float_as_int(v), m = __reduce_max_sync(0xFFFFFFFFu, i ^ ((i >> 31) & 0x7FFFFFFF));
    return __int_as_float(m ^ ((m >> 31) & 0x7FFFFFFF));
}
template <int G>
__device__ __forceinline__ uint64_t gsum2(uint64_t v)
{
#pragma unroll
    for (int o = G / 2; o; o >>= 1) {
        float x, y;
        unpack2(v, x, y);
        v = add2(v, pack2(__shfl_xor_sync(0xFFFFFFFFu, x, o), __shfl_xor_sync(0xFFFFFFFFu, y, o)));
    }
    return v;
}
__device__ __forceinline__ float sum_pair(uint64_t v)
{
    float x, y;
    unpack2(v, x, y);
    return x + y;
}

// running sum with its error (Kahan): s - c is the sum; the limit on c, which
// has no effect while s is finite, lets a sum beyond fp32 stay infinite
__device__ __forceinline__ void kahan(float &s, float &c, float v)
{
    const float y = __fsub_rn(v, c), t = __fadd_rn(s, y);
    c = fminf(__fsub_rn(__fsub_rn(t, s), y), 0x1p126f);
    s = t;
}

// G lanes a token, NV vectors of four experts a lane (E <= 4 G NV), KS slots a
// lane (k <= G KS)
template <int G, int NV, int KS, int SCORE>
__global__ void __launch_bounds__(256) balance_rows_kernel(const BalanceArgs a)
{
    constexpr int NE = 4 * NV, NP = 2 * NV, EP = 4 * G * NV, GPW = 32 / G;
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    __shared__ __align__(16) float s_gate[256 / G][EP];    // zeros but for a token's k gates
    __shared__ int32_t s_cnt[1024 + 1];                    // one sequence: the counts, then n
    __shared__ int32_t s_n, s_used, s_last;
    __shared__ Sum2 s_sum[8][2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gl = lane & (G - 1), g = lane / G;
    const int E = a.E, k = a.k;
    float *grow = s_gate[tid / G];
    for (int i = tid; i < 256 / G * EP; i += 256) (&s_gate[0][0])[i] = 0.0f;
    if (tid == 0) s_n = s_used = 0;

    // this warp's tokens
    const int64_t nwarp = (int64_t)gridDim.x * 8;
    const int per = (int)((((int64_t)a.T + nwarp - 1) / nwarp + GPW - 1) / GPW * GPW);
    const int64_t w0l = ((int64_t)blockIdx.x * 8 + warp) * per;
    const int w0 = (int)(w0l < a.T ? w0l : a.T), w1 = a.T - w0 < per ? a.T : w0 + per;

    // the next token's logits, ids, gates' gradients and mask
    float ln[NE], dgn[KS];
    int32_t idn[KS];
    bool mn;
    auto load = [&](int t) {
        const float *p = a.logits + (int64_t)t * E;
        mn = t < w1 && (!a.mask || __ldg(a.mask + t) != 0);
#pragma unroll
        for (int u = 0; u < KS; u++) {
            const int j = gl + G * u;
            const bool mine = t < w1 && j < k;
            idn[u] = mine ? __ldg(a.ids + (int64_t)t * k + j) : -1;
            dgn[u] = mine && a.d_gates ? __ldg(a.d_gates + (int64_t)t * k + j) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int e = 4 * (G * i + gl);
            float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (t < w1) {
                if (a.vec) {
                    if (e < E) v = __ldg(reinterpret_cast<const float4 *>(p + e));
                } else {
                    if (e < E) v.x = __ldg(p + e);
                    if (e + 1 < E) v.y = __ldg(p + e + 1);
                    if (e + 2 < E) v.z = __ldg(p + e + 2);
                    if (e + 3 < E) v.w = __ldg(p + e + 3);
                }
            }
            ln[4 * i] = v.x;
            ln[4 * i + 1] = v.y;
            ln[4 * i + 2] = v.z;
            ln[4 * i + 3] = v.w;
        }
    };
    load(w0 + g);
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const bool one = a.B == 1 && !a.off;
    if (one) {
        if (a.nhist) {
            for (int e = tid; e <= E; e += 256) {
                int32_t v = 0;
#pragma unroll 16
                for (int c = 0; c < a.nhist; c++) v += __ldcg(&a.ws->hist[c][e]);
                s_cnt[e] = v;
            }
        } else {
            for (int e = tid; e <= E; e += 256) s_cnt[e] = 0;
            __syncthreads();
            for (int i = tid; i < a.T * k; i += 256) {
                const int t = i / k;
                if (a.mask && !a.mask[t]) continue;
                const int32_t e = __ldg(a.ids + i);
                if (e >= 0 && e < E) atomicAdd(&s_cnt[e], 1);
                if (i == t * k) atomicAdd(&s_cnt[E], 1);
            }
        }
        __syncthreads();
        if (blockIdx.x == 0)
            for (int e = tid; e < E; e += 256) a.counts[e] = s_cnt[e];
        if (tid == 0) {
            s_n = s_cnt[E];
            s_used = s_cnt[E] > 0;
        }
    } else {
        int32_t n = 0, u = 0;
        for (int b = tid; b < a.B; b += 256) {
            const int32_t v = __ldcg(a.nb + b);
            n += v;
            u += v > 0;
        }
        n = __reduce_add_sync(ALL, n);
        u = __reduce_add_sync(ALL, u);
        if (lane == 0) {
            atomicAdd(&s_n, n);
            atomicAdd(&s_used, u);
        }
    }
    __syncthreads();
    const float cz = s_n > 0 ? a.grad_scale * 2.0f * a.zeta / (float)s_n : 0.0f;

    float f[NE], share = 0.0f;
    int b = -1, send = 0;                // sequence of the tokens up to send
#pragma unroll
    for (int i = 0; i < NE; i++) f[i] = 0.0f;
    float lbs = 0.0f, lbc = 0.0f, lzs = 0.0f, lzc = 0.0f;
    for (int tb = w0; tb < w1; tb += GPW) {
        const int t = tb + g;
        const bool on = t < w1;
        float l[NE];
#pragma unroll
        for (int i = 0; i < NE; i++) l[i] = ln[i];
        int32_t id[KS];
        float dg[KS];
#pragma unroll
        for (int u = 0; u < KS; u++) {
            id[u] = idn[u];
            dg[u] = dgn[u];
        }
        const bool unmasked = mn;
        if (tb + GPW < w1) load(tb + GPW + g);
        if (on && t >= send) {
            b = seq_of(a.off, a.B, t);
            send = seq_end(a.off, b, t, a.T);
            if (b >= 0) {
                const int32_t nb = one ? s_cnt[E] : __ldcg(a.nb + b);
                const float n = (float)(nb > 0 ? nb : 1);
                const float fs = (float)E / ((float)k * n);
                share = a.alpha / ((float)(s_used > 0 ? s_used : 1) * n);
#pragma unroll
                for (int i = 0; i < NE; i++) {
                    const int e = 4 * (G * (i / 4) + gl) + (i & 3);
                    const int32_t c = e >= E ? 0 : one ? s_cnt[e] : __ldcg(a.counts + (int64_t)b * E + e);
                    f[i] = fs * (float)c;
                }
            }
        }
        bool counted = on && b >= 0 && unmasked;

        // the token's slots, gl + G u on this lane.  Each writes its number to
        // its expert's place in the group's row: one that finds another's
        // there has a repeated id
        bool bad = false, any = false;
#pragma unroll
        for (int u = 0; u < KS; u++) {
            const int j = gl + G * u;
            const bool mine = on && j < k;
            any |= dg[u] != 0.0f;
            if ((uint32_t)id[u] < (uint32_t)E) grow[id[u]] = __int_as_float(j);
            else bad |= mine;
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < KS; u++)
            if ((uint32_t)id[u] < (uint32_t)E) bad |= __float_as_int(grow[id[u]]) != gl + G * u;
        if (G == 32) {
            bad = __any_sync(ALL, bad);
            any = __any_sync(ALL, any);
        } else {
            const uint32_t gm = ((1u << (G & 31)) - 1u) << (G * g);
            bad = (__ballot_sync(ALL, bad) & gm) != 0;
            any = (__ballot_sync(ALL, any) & gm) != 0;
        }
        if (bad && gl == 0) dev_flag(a.dev_status, MOE_DEV_BAD_IDS);
        const bool gate = any && !bad;
        // a token that adds nothing may hold anything
        if (__any_sync(ALL, !(counted || gate))) {
#pragma unroll
            for (int i = 0; i < NE; i++) l[i] = counted || gate ? l[i] : 0.0f;
        }
        uint64_t l2[NP], e2[NP];
#pragma unroll
        for (int i = 0; i < NP; i++) l2[i] = pack2(l[2 * i], l[2 * i + 1]);

        float m = l[0];
#pragma unroll
        for (int i = 1; i < NE; i++) m = fmaxf(m, l[i]);
        m = gmaxf<G>(m);
        const float sh = m == -INFINITY ? 0.0f : m;
        const uint64_t sh2 = pack2(-sh, -sh), k2 = pack2(LOG2E, LOG2E);
        uint64_t acc = 0;
#pragma unroll
        for (int i = 0; i < NP; i++) {
            float x, y;
            unpack2(mul2(add2(l2[i], sh2), k2), x, y);
            e2[i] = pack2(ex2(x), ex2(y));
            acc = add2(acc, e2[i]);
        }
        float tot, S, dot;
        uint64_t s2[NP];                       // the scores' slopes, up to S
        if (SCORE == MOE_SCORE_SIGMOID) {
            const uint64_t nk2 = pack2(-LOG2E, -LOG2E), one2 = pack2(1.0f, 1.0f);
            uint64_t sa = 0, da = 0;
#pragma unroll
            for (int i = 0; i < NP; i++) {
                // e = exp(-l) up to 2^127, where s is 0; s = 1 / (1 + e), s (1 - s) = s (s e),
                // in this order: s s underflows where the slope is still about s
                float x, y;
                unpack2(mul2(l2[i], nk2), x, y);
                asm("min.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(127.0f));
                asm("min.NaN.f32 %0, %0, %1;" : "+f"(y) : "f"(127.0f));
                const uint64_t e = pack2(ex2(x), ex2(y));
                unpack2(add2(e, one2), x, y);
                const uint64_t s = pack2(rcp(x), rcp(y));
                sa = add2(sa, s);
                da = fma2(pack2(f[2 * i], f[2 * i + 1]), s, da);
                s2[i] = mul2(s, mul2(s, e));
            }
            if (m <= 0.0f) {
                // all scores e^m and less, and their sum underflows with them: up to
                // e^-m, s = a / (1 + a e^m) with a = e^(l - m), and 1 - s = 1 / (1 + a e^m)
                // (the branch costs ordinary tokens 75.8 -> 77.6 us at 131072 x 256, this
                // form for every token without a branch as much)
                const float em = ex2(sh * LOG2E);
                const uint64_t em2 = pack2(em, em);
                sa = da = 0;
#pragma unroll
                for (int i = 0; i < NP; i++) {
                    float x, y;
                    unpack2(fma2(e2[i], em2, one2), x, y);
                    const uint64_t r = pack2(rcp(x), rcp(y)), s = mul2(e2[i], r);
                    sa = add2(sa, s);
                    da = fma2(pack2(f[2 * i], f[2 * i + 1]), s, da);
                    s2[i] = mul2(s, r);
                }
            }
            tot = gsum<G>(sum_pair(acc));
            unpack2(gsum2<G>(pack2(sum_pair(sa), sum_pair(da))), S, dot);
            S = rcp(S);
        } else {
            uint64_t da = 0;
#pragma unroll
            for (int i = 0; i < NP; i++) {
                s2[i] = e2[i];
                da = fma2(pack2(f[2 * i], f[2 * i + 1]), e2[i], da);
            }
            unpack2(gsum2<G>(pack2(sum_pair(acc), sum_pair(da))), tot, dot);
            S = rcp(tot);
        }
        dot *= S;
        counted = counted && tot != 0.0f;
        const float it = rcp(tot), lse = fmaf(LN2, lg2(tot), sh);
        const float cb = counted ? a.grad_scale * share * S : 0.0f, cl = counted ? cz * lse * it : 0.0f;
        if (counted) {
            kahan(lbs, lbc, share * dot);
            kahan(lzs, lzc, lse * lse);
        }
        float go = 0.0f;                       // the full softmax's common part
        if (a.d_logits && __any_sync(ALL, gate)) {
            // through the gates: the chosen logits again (in L1), as the router's backward
            // (expf and rounded quotients: with few slots dg - sum dg p nearly cancels)
            float my[KS], dl[KS], sm = 0.0f, dt = 0.0f, mm = -INFINITY;
#pragma unroll
            for (int u = 0; u < KS; u++) {
                const bool mine = gate && gl + G * u < k;
                my[u] = mine ? __ldg(a.logits + (int64_t)t * E + id[u]) : -INFINITY;
                mm = fmaxf(mm, my[u]);
            }
            if (SCORE == MOE_SCORE_SOFTMAX) {
                mm = a.renorm ? gmaxf<G>(mm) : m;
#pragma unroll
                for (int u = 0; u < KS; u++) {
                    dl[u] = gate && gl + G * u < k ? expf(my[u] - mm) : 0.0f;
                    sm += dl[u];
                }
                sm = a.renorm ? gsum<G>(sm) : tot;
#pragma unroll
                for (int u = 0; u < KS; u++) {
                    dl[u] = div1(dl[u], sm);
                    dt = fmaf(dg[u], dl[u], dt);
                }
                dt = gsum<G>(dt);
#pragma unroll
                for (int u = 0; u < KS; u++) dl[u] *= a.renorm ? dg[u] - dt : dg[u];
                go = a.renorm || !gate ? 0.0f : a.route_scale * dt * it;
            } else {
                // renormalised gates depend on the scores' ratios: for low tokens, whose
                // scores are e^l and underflow, those of the logits moved up to -20 (1 - s
                // is 1 there too)
                const bool low = a.renorm && sh < -40.0f;
                const float l0 = low ? sh : 0.0f, l1 = low ? 20.0f : 0.0f;
                float ds[KS];
#pragma unroll
                for (int u = 0; u < KS; u++) {
                    const bool mine = gate && gl + G * u < k;
                    float e = expf(l1 - (my[u] - l0));
                    asm("min.NaN.f32 %0, %0, %1;" : "+f"(e) : "f"(0x1p126f));
                    const float s = mine ? div1(1.0f, 1.0f + e) : 0.0f;
                    ds[u] = e * s * s;
                    sm += s;
                    dt = fmaf(dg[u], s, dt);
                }
                if (a.renorm) {
                    unpack2(gsum2<G>(pack2(sm, dt)), sm, dt);
                    dt = div1(dt, sm);
                }
#pragma unroll
                for (int u = 0; u < KS; u++) dl[u] = ds[u] * (a.renorm ? div1(dg[u] - dt, sm) : dg[u]);
            }
#pragma unroll
            for (int u = 0; u < KS; u++)
                if (gate && gl + G * u < k) grow[id[u]] = a.route_scale * dl[u];
            __syncwarp();
        }
        if (a.d_logits) {
            float *o = a.d_logits + (int64_t)t * E;
            const uint64_t cb2 = pack2(cb, cb), cl2 = pack2(cl, cl), nd2 = pack2(-dot, -dot), ng2 = pack2(-go, -go);
            // (a token that is not counted has finite logits, or gates: no NaN from the zeros here)
            const uint64_t z2 = counted ? nd2 : 0;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int e = 4 * (G * i + gl);
                float4 gq = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (gate) gq = *reinterpret_cast<const float4 *>(grow + e);
                float v[4];
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int x = 2 * i + h;
                    uint64_t d = mul2(mul2(s2[x], cb2), add2(pack2(f[2 * x], f[2 * x + 1]), z2));
                    d = fma2(cl2, e2[x], d);
                    d = add2(d, h ? pack2(gq.z, gq.w) : pack2(gq.x, gq.y));
                    if (SCORE == MOE_SCORE_SOFTMAX) d = fma2(ng2, e2[x], d);
                    unpack2(d, v[2 * h], v[2 * h + 1]);
                }
                if (!on || e >= E) continue;
                if (a.vec) {
                    *reinterpret_cast<float4 *>(o + e) = make_float4(v[0], v[1], v[2], v[3]);
                } else {
#pragma unroll
                    for (int u = 0; u < 4; u++)
                        if (e + u < E) o[e + u] = v[u];
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < KS; u++)
            if ((uint32_t)id[u] < (uint32_t)E) grow[id[u]] = 0.0f;
        __syncwarp();
    }
    Sum2 lb = {gl == 0 ? lbs : 0.0f, gl == 0 ? -lbc : 0.0f}, lz = {gl == 0 ? lzs : 0.0f, gl == 0 ? -lzc : 0.0f};
    warp_sum2(lb);
    warp_sum2(lz);
    if (lane == 0) {
        s_sum[warp][0] = lb;
        s_sum[warp][1] = lz;
    }
    __syncthreads();
    if (tid < 2) {
        Sum2 v = s_sum[0][tid];
        for (int i = 1; i < 8; i++) add(v, s_sum[i][tid]);
        a.ws->loss[blockIdx.x][tid] = v;
        __threadfence();
    }
    if (gridDim.x > 1) {
        __syncthreads();
        if (tid == 0) s_last = atomicAdd(&a.ws->done, 1u) == gridDim.x - 1;
        __syncthreads();
        if (!s_last) return;
        __threadfence();
    } else {
        __syncthreads();
    }
    // the CTA that finishes last adds the CTAs' sums: warp 0 the balance loss, warp 1 z
    if (warp < 2) {
        Sum2 v = {0.0f, 0.0f};
        for (unsigned c = lane; c < gridDim.x; c += 32) {
            Sum2 o;
            o.hi = __ldcg(&a.ws->loss[c][warp].hi);
            o.lo = __ldcg(&a.ws->loss[c][warp].lo);
            add(v, o);
        }
        warp_sum2(v);
        if (lane == 0) a.losses[warp] = warp == 0 ? total(v) : s_n > 0 ? total(v) * (a.zeta / (float)s_n) : 0.0f;
    }
}

template <int G, int NV, int KS, int SCORE>
static cudaError_t launch_balance_k(const BalanceArgs &a, bool pdl, cudaStream_t st)
{
    // as many CTAs as the SMs hold at once (each warp's run of tokens is then
    // the same length), at least a token a group
    static const int per_sm = [] {
        int n = 0;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, balance_rows_kernel<G, NV, KS, SCORE>, 256, 0) ==
                           cudaSuccess && n > 0 ? n : 1;
    }();
    const int64_t need = ((int64_t)a.T * G / 32 + 8) / 8, cap = (int64_t)per_sm * sm_count();
    int64_t grid = need < cap ? need : cap;
    if (grid > ROW_CTAS_MAX) grid = ROW_CTAS_MAX;
    if (a.B == 1 && !a.off && a.nhist == 0) grid = 1;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(grid < 1 ? 1 : grid));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, balance_rows_kernel<G, NV, KS, SCORE>, a);
}

template <int G, int NV>
static cudaError_t launch_balance(const BalanceArgs &a, bool pdl, cudaStream_t st)
{
    constexpr int KS = 32 / G;
    if (a.score_fn == MOE_SCORE_SIGMOID)
        return a.k <= G ? launch_balance_k<G, NV, 1, MOE_SCORE_SIGMOID>(a, pdl, st)
                        : launch_balance_k<G, NV, KS, MOE_SCORE_SIGMOID>(a, pdl, st);
    return a.k <= G ? launch_balance_k<G, NV, 1, MOE_SCORE_SOFTMAX>(a, pdl, st)
                    : launch_balance_k<G, NV, KS, MOE_SCORE_SOFTMAX>(a, pdl, st);
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
    return sizeof(BalWs) + sizeof(int32_t) * (size_t)(B > 0 ? B : 1);
}

MOE_API moe_status moe_balance_loss(const float *logits, const int32_t *topk_ids, const uint8_t *token_mask,
                                    const int32_t *seq_offsets, int T, int E, int k, int B, int score_fn, int renorm,
                                    float route_scale, float balance_coef, float z_coef, float grad_scale,
                                    const float *d_gates, int32_t *counts, float *losses, float *d_logits,
                                    void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    if (T < 0 || E < 1 || E > 1024 || k < 1 || k > 32 || k > E || B < 1 || B > 65535) return MOE_ERR_SHAPE;
    if (B > 1 && !seq_offsets) return MOE_ERR_SHAPE;
    // (the kernels step through the tokens in strides of up to 1024, in 32 bits)
    if ((int64_t)T * k >= (1LL << 31) - 4096) return MOE_ERR_SHAPE;
    if (score_fn != MOE_SCORE_SOFTMAX && score_fn != MOE_SCORE_SIGMOID) return MOE_ERR_SHAPE;
    if (!isfinite(route_scale) || !isfinite(balance_coef) || !isfinite(z_coef) || !isfinite(grad_scale))
        return MOE_ERR_SHAPE;
    if (!counts || !losses) return MOE_ERR_NULL;
    if (T > 0 && (!logits || !topk_ids)) return MOE_ERR_NULL;
    if (!workspace || workspace_bytes < moe_balance_loss_workspace_size(T, E, B)) return MOE_ERR_WORKSPACE;
    if (!aligned256(workspace)) return MOE_ERR_ALIGN;
    cudaStream_t st = as_stream(stream);
    if (T == 0)
        return cudaMemsetAsync(counts, 0, sizeof(int32_t) * (size_t)B * E, st) == cudaSuccess &&
                       cudaMemsetAsync(losses, 0, 2 * sizeof(float), st) == cudaSuccess
                   ? MOE_OK
                   : MOE_ERR_CUDA;
    BalWs *ws = (BalWs *)workspace;
    BalanceArgs a = {logits, d_gates, topk_ids, seq_offsets, token_mask, T, E, k, B, score_fn, renorm, route_scale,
                     balance_coef, z_coef, grad_scale, counts, losses, d_logits, ws, ws->nb, 0, 0, dev_status};
    a.vec = E % 4 == 0 && aligned16(logits) && (!d_logits || aligned16(d_logits));
    const bool one = !seq_offsets;
    const int64_t slots = (int64_t)T * k;
    bool pdl = false;
    if (one) {
        // few tokens (eight a group): one CTA counts and goes through the rows;
        // else the counting CTAs' histograms are added up by the rows' CTAs
        if ((int64_t)T * (E <= 64 ? 8 : E <= 256 ? 16 : 32) > 2048) {
            const int64_t h = (slots + 2047) / 2048;
            a.nhist = (int)(h < HIST_MAX ? h : HIST_MAX);
            balance_count_kernel<<<a.nhist, 1024, 0, st>>>(topk_ids, token_mask, seq_offsets, T, E, k, B, counts, a.nb,
                                                           ws, dev_status);
            pdl = true;
        }
    } else {
        const int64_t nz = ((int64_t)B * E + 1023) / 1024, zmax = 2LL * sm_count();
        balance_zero_kernel<<<(unsigned)(nz < zmax ? nz : zmax), 1024, 0, st>>>(counts, (int64_t)B * E, a.nb, B, ws);
        if (cudaPeekAtLastError() != cudaSuccess) return launch_status();
        const int64_t h = (slots + 2047) / 2048, hmax = 2LL * sm_count();
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3((unsigned)(h < hmax ? h : hmax));
        cfg.blockDim = dim3(1024);
        cfg.stream = st;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, balance_count_kernel, topk_ids, token_mask, seq_offsets, T, E, k, B, counts, a.nb,
                               ws, dev_status) != cudaSuccess)
            return MOE_ERR_CUDA;
        pdl = true;
    }
    if (cudaPeekAtLastError() != cudaSuccess) return launch_status();
    cudaError_t e;
    // few lanes a token: a warp's reductions, gates and bookkeeping then serve
    // several tokens (131072 x 256 softmax: 76 us at 16 lanes, 82 at 32, 100
    // at 8, where the registers leave one CTA an SM; x 128: 33 at 16, 41 at 32)
    if (E <= 32) e = launch_balance<8, 1>(a, pdl, st);
    else if (E <= 64) e = launch_balance<8, 2>(a, pdl, st);
    else if (E <= 128) e = launch_balance<16, 2>(a, pdl, st);
    else if (E <= 256) e = launch_balance<16, 4>(a, pdl, st);
    else if (E <= 512) e = launch_balance<32, 4>(a, pdl, st);
    else e = launch_balance<32, 8>(a, pdl, st);
    return e == cudaSuccess ? launch_status() : MOE_ERR_CUDA;
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
