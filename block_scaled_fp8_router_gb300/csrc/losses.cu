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
// (l_v - c) k2 and not l_v k2 - c k2: the largest logit's t is then exactly 0.
//
// token_rows_kernel: one cluster of C CTAs per row.  A row's 16-byte vectors
// are dealt to the threads of the cluster, NV of them kept in registers from
// the one read to the gradient's write; a longer row goes through a ring of
// asynchronous copies in shared memory, and its gradient reads it again, mostly
// from L2 (a seventh misses at 131072 logits).  A warp takes its maximum, sums
// 2^t and 2^t t against it;
// the warps' sums are joined in shared memory, the CTAs' through one 16-byte
// message to every CTA of the cluster (st.async on an mbarrier), always in the
// same order.  So a row costs one CTA barrier, one exchange and one more CTA
// barrier, and several CTAs per SM keep HBM busy across them.
//
// Bound: HBM for long rows, one exponential a logit (two with a gradient) close
// behind.  Measured: log-probabilities of 8192 x 131072 bf16 0.30 ms (7.1
// TB/s read; 4096 x 131072 fp32 0.31), the gradient of 8192 rows, a quarter
// without weight, 0.61 ms (6.1 TB/s read once and written); short or few rows by
// latency, 7 x 50001 fp32 4.6 us, 256 x 32768 13 us (back to back in a CUDA graph).
#include "losses.cuh"

#include <math.h>

namespace moe {

// where t multiplies 2^t it is held above this: 2^t is 0 there, and 0 times
// an infinite t (a masked logit) would be NaN
constexpr float TMIN = -16384.0f;

// the sums of one part of a row, relative to the shift c (c = -inf: no logit
// above -inf, S = U = 0)
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

// joins over the lanes 0 .. n-1 of a warp (n a power of two), the same bits in
// each: the lower lane's sums always come first
__device__ __forceinline__ RowSum warp_join(RowSum s, int n, int lane, float k2)
{
    for (int o = 1; o < n; o <<= 1) {
        RowSum b;
        b.c = __shfl_xor_sync(0xFFFFFFFFu, s.c, o);
        b.S = __shfl_xor_sync(0xFFFFFFFFu, s.S, o);
        b.U = __shfl_xor_sync(0xFFFFFFFFu, s.U, o);
        s = (lane & o) ? join(b, s, k2) : join(s, b, k2);
    }
    return s;
}

// a 16-byte vector of logits: 8 bf16 or 4 fp32
template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
    static constexpr int W = 8;
    static constexpr uint32_t NINF = 0xFF80FF80u;
    static __device__ __forceinline__ float max(const uint4 &v)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        __nv_bfloat162 m[4];
#pragma unroll
        for (int i = 0; i < 4; i++) m[i] = *reinterpret_cast<const __nv_bfloat162 *>(&w[i]);
        const __nv_bfloat162 a = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
        return fmaxf(__low2float(a), __high2float(a));
    }
    // elements below -2^100 raised to it, NaN kept
    static __device__ __forceinline__ uint4 floor100(const uint4 &v)
    {
        const uint32_t lo = 0xF180F180u;
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; i++) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(lo));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // pair i (0 .. 3) as two fp32
    static __device__ __forceinline__ uint64_t pair(const uint4 &v, int i)
    {
        const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
        return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint4 make(const float *f)
    {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                          pack_bf16x2(f[6], f[7]));
    }
};
template <>
struct Vec<float> {
    static constexpr int W = 4;
    static constexpr uint32_t NINF = 0xFF800000u;
    static __device__ __forceinline__ float max(const uint4 &v)
    {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                     fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    static __device__ __forceinline__ uint4 floor100(const uint4 &v)
    {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float f = __uint_as_float(w[i]);
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(f) : "f"(-0x1p100f));
            w[i] = __float_as_uint(f);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ uint64_t pair(const uint4 &v, int i)
    {
        return i == 0 ? pack2(__uint_as_float(v.x), __uint_as_float(v.y))
                      : pack2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    static __device__ __forceinline__ uint4 make(const float *f)
    {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

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

// a vector at a row's ends, or past it: elements e .. e + W - 1 of the row,
// those outside [0, V) -inf
template <typename T>
__device__ __noinline__ uint4 load_ends(const T *l, int64_t V, int64_t e)
{
    constexpr int W = Vec<T>::W;
    float f[W];
#pragma unroll
    for (int u = 0; u < W; u++) f[u] = e + u >= 0 && e + u < V ? load_logit(l + e + u) : -INFINITY;
    return Vec<T>::make(f);
}

// a row as 16-byte vectors: vector j holds the elements W j - head .. + W - 1
// of the row, those outside [0, V) absent; vectors lo .. hi - 1 are whole
template <typename T>
struct Row {
    const T *l;
    const uint4 *base;
    int head, nvec, lo, hi;
    int64_t V;
    __device__ __forceinline__ Row(const T *p, int64_t n) : l(p), V(n)
    {
        constexpr int W = Vec<T>::W;
        head = (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
        base = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15u);
        nvec = (int)((n + head + W - 1) / W);
        lo = head > 0;
        hi = (int)((n + head) / W);
    }
    __device__ __forceinline__ bool inside(int j) const { return j >= lo && j < hi; }
    __device__ __forceinline__ uint4 load_edge(int j) const
    {
        return load_ends<T>(l, V, (int64_t)Vec<T>::W * j - head);
    }
    __device__ __forceinline__ uint4 load(int j) const
    {
        constexpr uint32_t NI = Vec<T>::NINF;
        uint4 v = make_uint4(NI, NI, NI, NI);
        if (inside(j))
            asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "l"(base + j)
                         : "memory");
        return v;
    }
};

struct PolicyArgs {
    const float *old_lp, *adv, *ref_lp, *w;
    float clip_lo, clip_hi, beta, eta;
    int64_t ld_d;
    struct Ws *ws;
    float num, norm;        // the gradient's scale is num / norm; norm 0: the rows' CTAs add up w; below: scale is in ws
};

// Up to this many weights each row's CTA adds them up itself, which saves a
// launch (256 rows of 32768: 28 us a call against 31, most of it the host's).
constexpr int64_t NORM_ROWS = 512;

// workspace: the weights' sum, and per row w pg, w kl, w H and w [clipped]
struct Ws {
    float norm, scale;      // scale = grad_scale / (norm temperature), 0 where norm is
    float pad[2];
    float4 row[1];
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

// sum of the weights in a fixed order
__global__ void __launch_bounds__(1024) policy_norm_kernel(const float *__restrict__ w, int64_t N, float num, Ws *ws)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ Sum2 s_v[32];
    const int tid = threadIdx.x;
    Sum2 v = {0.0f, 0.0f};
    for (int64_t i = tid; i < N; i += 8192) {
        float q[8];
#pragma unroll
        for (int u = 0; u < 8; u++) q[u] = i + 1024 * u < N ? __ldg(w + i + 1024 * u) : 0.0f;
#pragma unroll
        for (int u = 0; u < 8; u++) add(v, q[u]);
    }
    warp_sum2(v);
    if ((tid & 31) == 0) s_v[tid >> 5] = v;
    __syncthreads();
    if (tid >= 32) return;
    v = s_v[tid];
    warp_sum2(v);
    const float norm = total(v);
    if (tid == 0) {
        ws->norm = norm;
        ws->scale = norm != 0.0f ? num / norm : 0.0f;
    }
}

// the scale of the gradients, by a whole warp
__device__ __forceinline__ float grad_scale_of(const PolicyArgs &a, int64_t N, int lane)
{
    if (a.norm < 0.0f) return __ldcg(&a.ws->scale);
    float norm = a.norm;
    if (norm == 0.0f) {
        Sum2 v = {0.0f, 0.0f};
        for (int64_t i = lane; i < N; i += 256) {
            float q[8];
#pragma unroll
            for (int u = 0; u < 8; u++) q[u] = i + 32 * u < N ? __ldg(a.w + i + 32 * u) : 0.0f;
#pragma unroll
            for (int u = 0; u < 8; u++) add(v, q[u]);
        }
        warp_sum2(v);
        norm = total(v);
    }
    return norm != 0.0f ? a.num / norm : 0.0f;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank)
{
    uint32_t out;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(out) : "r"(addr), "r"(rank));
    return out;
}

constexpr int RING_DEPTH = 2;           // chunks of a thread in shared memory
constexpr uint64_t ROW_TIMEOUT_NS = 1000ull * 1000ull * 1000ull;

// what a row's gradient needs: dl_v = 2^t_v (A0 + B0 t_v), t_v = (l_v - c) k2, and
// gy, the whole of dl_y
struct RowGrad {
    float c, A0, B0, gy;
};

// whether t of a logit held above -2^100 is finite for the shift c, so that 2^t t
// needs no other care, and below -512, so that 2^t is still 0 (rows whose largest
// logit is beyond 2^99, or -inf, and temperatures below 1e-6 or above 1e27 take
// the slower form)
__device__ __forceinline__ bool plain_range(float c, float k2)
{
    return fabsf(c) < 0x1p99f && k2 > 0x1p-90f && k2 < 0x1p20f;
}

// sums of one vector against the shift c = -nc, two elements at a time
template <typename T, bool SLOW>
__device__ __forceinline__ void add_vec(uint4 v, uint64_t nc2, uint64_t k22, uint64_t &S, uint64_t &U)
{
    if (!SLOW) v = Vec<T>::floor100(v);
#pragma unroll
    for (int i = 0; i < Vec<T>::W / 2; i++) {
        uint64_t t = mul2(add2(Vec<T>::pair(v, i), nc2), k22);
        float t0, t1;
        unpack2(t, t0, t1);
        const uint64_t e = pack2(ex2(t0), ex2(t1));
        S = add2(S, e);
        if (SLOW) t = pack2(fmaxf(t0, TMIN), fmaxf(t1, TMIN));
        U = fma2(e, t, U);
    }
}

// adds NV vectors of a warp to its sums (all lanes hold the same shift)
template <typename T, int NV>
__device__ __forceinline__ void add_vecs(RowSum &s, const uint4 (&v)[NV], float k2)
{
    float m = s.c;
#pragma unroll
    for (int i = 0; i < NV; i++) m = fmaxf(m, Vec<T>::max(v[i]));
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (m > s.c) {
        if (s.c != -INFINITY) {
            const float d = fmaxf((s.c - m) * k2, TMIN), f = ex2(d);
            s.U = (s.U + d * s.S) * f;
            s.S *= f;
        }
        s.c = m;
    }
    const float nc = m == -INFINITY ? 0.0f : -m;
    const uint64_t nc2 = pack2(nc, nc), k22 = pack2(k2, k2);
    uint64_t S = pack2(s.S, 0.0f), U = pack2(s.U, 0.0f);
    if (plain_range(m, k2)) {
#pragma unroll
        for (int i = 0; i < NV; i++) add_vec<T, false>(v[i], nc2, k22, S, U);
    } else {
#pragma unroll
        for (int i = 0; i < NV; i++) add_vec<T, true>(v[i], nc2, k22, S, U);
    }
    float x, z;
    unpack2(S, x, z);
    s.S = x + z;
    unpack2(U, x, z);
    s.U = x + z;
}

// the gradient of one vector, t as in the sums
template <typename T, bool ETA>
__device__ __forceinline__ void grad_vec(const uint4 &v, const RowGrad &g, uint64_t k22, float *f)
{
    const uint64_t nc2 = pack2(-g.c, -g.c);
#pragma unroll
    for (int i = 0; i < Vec<T>::W / 2; i++) {
        const uint64_t t = mul2(add2(Vec<T>::pair(v, i), nc2), k22);
        float t0, t1;
        unpack2(t, t0, t1);
        const uint64_t e = pack2(ex2(t0), ex2(t1));
        uint64_t a = pack2(g.A0, g.A0);
        if (ETA) a = fma2(pack2(g.B0, g.B0), pack2(fmaxf(t0, TMIN), fmaxf(t1, TMIN)), a);
        unpack2(mul2(e, a), f[2 * i], f[2 * i + 1]);
    }
}

// Row blockIdx.x / C by a cluster of C CTAs of TH threads at most.  POLICY: the
// policy loss and its gradient (else log-probabilities and entropy); RING: that
// of a row with more than one chunk of NV vectors a thread; ETA: with an
// entropy bonus.  The CTAs an SM is to hold weigh rows in flight against
// registers: seven of 128 threads with a gradient in registers (8192 x 8192
// bf16 58 us, 65 at five; 8192 x 4096, 64 threads, 41 and 39).
template <typename T, int TH, int NV, bool RING, bool POLICY, bool ETA>
__global__ void __launch_bounds__(TH, TH == 256 ? (POLICY ? 3 : 4) : POLICY ? (RING ? 6 : 7) : 8)
    token_rows_kernel(const T *logits, int64_t N, int64_t V, int64_t ld, const void *__restrict__ targets, int t64,
                      float k2, int C, float *__restrict__ logprobs, float *__restrict__ entropy, T *dlogits,
                      const PolicyArgs a, int32_t *dev_status)
{
    constexpr int W = Vec<T>::W;
    __shared__ RowSum s_part[TH / 32];
    __shared__ float4 s_msg[8];
    __shared__ RowGrad s_grad;
    __shared__ int s_live;
    __shared__ uint64_t s_bar;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, nw = nt >> 5;
    const int64_t row = blockIdx.x / (unsigned)C;
    const int rank = C > 1 ? (int)cluster_rank() : 0;
    if (C > 1) {
        if (tid == 0) {
            mbar_init(&s_bar, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    const int64_t y = t64 ? ((const int64_t *)targets)[row] : (int64_t)((const int32_t *)targets)[row];
    const float w = POLICY && a.w ? a.w[row] : 1.0f;
    bool live = y >= 0 && y < V && w != 0.0f;
    if (y >= V && w != 0.0f && tid == 0 && rank == 0) dev_flag(dev_status, MOE_DEV_BAD_IDS);
    const Row<T> R(logits + row * ld, V);
    const int j0 = rank * nt + tid, dj = C * nt;   // my vectors: j0, j0 + dj, ...
    // The row in chunks of NV vectors a thread.  For a gradient, one chunk stays
    // in registers; of more, the next RING_DEPTH are on their way to the
    // thread's own places in shared memory (chunk c at c mod RING_DEPTH) while
    // one is worked on, and the gradient goes through them backward: the last
    // are still there, the others come again from L2.
    const int nch = POLICY && !RING ? 1 : (R.hi + NV * dj - 1) / (NV * dj);
    extern __shared__ uint4 s_ring[];
    uint4 raw[NV];
    // chunk c whole for every thread: no vector of it needs a look
    auto full = [&](int c) { return c * NV * dj >= R.lo && (c + 1) * NV * dj <= R.hi; };
    auto fetch = [&](int c) {            // always one group, empty outside 0 .. nch - 1
        if (c >= 0 && c < nch) {
            const uint32_t place = smem_u32(s_ring + (c % RING_DEPTH) * (NV * TH) + tid);
            const uint4 *src = R.base + (c * NV * dj + j0);
            auto copy = [&](int i) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(place + i * TH * 16), "l"(src + i * dj)
                             : "memory");
            };
            if (full(c)) {
#pragma unroll
                for (int i = 0; i < NV; i++) copy(i);
            } else {
#pragma unroll
                for (int i = 0; i < NV; i++)
                    if (R.inside((c * NV + i) * dj + j0)) copy(i);
            }
        }
        cp_async_commit();
    };
    auto load = [&](int c) {
        if (full(c)) {
            const uint4 *src = R.base + (c * NV * dj + j0);
#pragma unroll
            for (int i = 0; i < NV; i++)
                asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(raw[i].x), "=r"(raw[i].y), "=r"(raw[i].z), "=r"(raw[i].w)
                             : "l"(src + i * dj)
                             : "memory");
        } else {
#pragma unroll
            for (int i = 0; i < NV; i++) raw[i] = R.load((c * NV + i) * dj + j0);
        }
    };
    auto take = [&](int c) {             // chunk c to registers, absent vectors as -inf
        constexpr uint32_t NI = Vec<T>::NINF;
        cp_async_wait<RING_DEPTH - 1>();
        const uint4 *place = s_ring + (c % RING_DEPTH) * (NV * TH) + tid;
        if (full(c)) {
#pragma unroll
            for (int i = 0; i < NV; i++) raw[i] = place[i * TH];
        } else {
#pragma unroll
            for (int i = 0; i < NV; i++)
                raw[i] = R.inside((c * NV + i) * dj + j0) ? place[i * TH] : make_uint4(NI, NI, NI, NI);
        }
    };
    float lp = 0.0f, H = 0.0f;
    float4 st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (live) {
        if (RING) {
#pragma unroll
            for (int c = 0; c < RING_DEPTH; c++) fetch(c);
        } else {
            load(0);
        }
        const float ly = warp == 0 ? load_logit(R.l + y) : 0.0f;
        RowSum s = {-INFINITY, 0.0f, 0.0f};
        // the vectors at the row's two ends, one lane's each, if not whole
        if (R.lo > 0 || R.hi < R.nvec) {
            const bool first = R.lo > 0 && j0 == 0, last = R.hi < R.nvec && j0 == (R.nvec - 1) % dj;
            if (__any_sync(0xFFFFFFFFu, first || last)) {
                uint4 e[1];
                e[0] = R.load_edge(first ? 0 : R.nvec);
                add_vecs<T, 1>(s, e, k2);
                if (R.nvec > 1 || !(R.lo > 0)) {
                    e[0] = R.load_edge(last ? R.nvec - 1 : R.nvec);
                    add_vecs<T, 1>(s, e, k2);
                }
            }
        }
        for (int c = 0; c < nch; c++) {
            if (RING) {
                take(c);
                fetch(c + RING_DEPTH);
            } else if (c > 0) {
                load(c);
            }
            add_vecs<T, NV>(s, raw, k2);
        }
        for (int o = 16; o; o >>= 1) {
            s.S += __shfl_xor_sync(0xFFFFFFFFu, s.S, o);
            s.U += __shfl_xor_sync(0xFFFFFFFFu, s.U, o);
        }
        if (lane == 0) s_part[warp] = s;
        __syncthreads();
        if (warp == 0) {
            s = lane < nw ? s_part[lane] : RowSum{-INFINITY, 0.0f, 0.0f};
            s = warp_join(s, nw > C ? nw : C, lane, k2);     // lanes 0 .. C-1 all hold the CTA's
            if (C > 1) {
                // the peers have set up their barriers; lane r sends (c, S, U,
                // l_y) to CTA r.  l_y travels too so that it has been read
                // before any CTA can write the gradient over it
                asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
                if (lane == 0) mbar_arrive_expect_tx(&s_bar, 16 * C);
                if (lane < C)
                    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, "
                                 "%4}, [%5];" ::"r"(map_rank(smem_u32(&s_msg[rank]), lane)),
                                 "r"(__float_as_uint(s.c)), "r"(__float_as_uint(s.S)), "r"(__float_as_uint(s.U)),
                                 "r"(__float_as_uint(ly)), "r"(map_rank(smem_u32(&s_bar), lane))
                                 : "memory");
                if (!mbar_wait_bounded(&s_bar, 0, ROW_TIMEOUT_NS) && lane == 0) dev_flag(dev_status, MOE_DEV_TIMEOUT);
                __syncwarp();
                const float4 q = lane < C ? s_msg[lane] : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
                s = warp_join(RowSum{q.x, q.y, q.z}, C, lane, k2);
            }
            s.c = __shfl_sync(0xFFFFFFFFu, s.c, 0);
            s.S = __shfl_sync(0xFFFFFFFFu, s.S, 0);
            s.U = __shfl_sync(0xFFFFFFFFu, s.U, 0);
            if (s.c == -INFINITY && s.S == 0.0f) {       // no logit above -inf: not scored
                live = false;
                if (lane == 0 && rank == 0) dev_flag(dev_status, MOE_DEV_BAD_IDS);
            } else {
                const float ls = log2f(s.S);
                lp = LN2 * ((ly - s.c) * k2 - ls);
                H = LN2 * (ls - s.U / s.S);
                RowGrad g = {0.0f, 0.0f, 0.0f, 0.0f};
                if (POLICY) {
                    const float A = a.adv[row];
                    float dlt = lp - a.old_lp[row];
                    dlt = dlt > 80.0f ? 80.0f : dlt;
                    const float ratio = expf(dlt);
                    const float rc = ratio < a.clip_lo ? a.clip_lo : (ratio > a.clip_hi ? a.clip_hi : ratio);
                    const float p0 = -A * ratio, p1 = -A * rc;
                    const bool clipped = p1 > p0;
                    float gl = clipped ? 0.0f : p0, kl = 0.0f;
                    if (a.ref_lp) {
                        float u = a.ref_lp[row] - lp;
                        u = u > 80.0f ? 80.0f : u;
                        kl = kl_term(u);
                        gl = fmaf(-a.beta, expm1f(u), gl);
                    }
                    st = make_float4(w * (clipped ? p1 : p0), w * kl, w * H, clipped ? w : 0.0f);
                    asm volatile("griddepcontrol.wait;" ::: "memory");
                    const float coef = w * grad_scale_of(a, N, lane);
                    const float q = coef / s.S;
                    g.c = s.c;
                    g.B0 = q * a.eta * LN2;
                    g.A0 = q * (-gl + a.eta * (H - LN2 * ls));
                    const float ty = (ly - s.c) * k2;
                    g.gy = fmaf(ex2(ty), fmaf(g.B0, fmaxf(ty, TMIN), g.A0), coef * gl);
                }
                if (lane == 0) s_grad = g;
            }
            if (lane == 0) s_live = live;
        } else if (C > 1) {
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        }
    } else if (C > 1) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    if (POLICY && dlogits) {
        const bool was = live || (y >= 0 && y < V && w != 0.0f);   // the same for the whole cluster
        if (was) {
            __syncthreads();
            live = s_live != 0;
        }
        const RowGrad g = live ? s_grad : RowGrad{0.0f, 0.0f, 0.0f, 0.0f};
        const uint64_t k22 = pack2(k2, k2);
        T *d = dlogits + row * a.ld_d;
        // vector stores where the gradient's rows are aligned as the logits' are
        // (else elements: 4096 x 131072 bf16 1.15 ms against 0.36)
        const bool same = ((reinterpret_cast<uintptr_t>(d) ^ reinterpret_cast<uintptr_t>(R.l)) & 15u) == 0;
        uint4 *dv = reinterpret_cast<uint4 *>(reinterpret_cast<uintptr_t>(d) & ~(uintptr_t)15u);
        auto store = [&](int j, const float *f, bool whole) {
            if (whole && same) {
                __stcs(dv + j, Vec<T>::make(f));
            } else {
                const int64_t e = (int64_t)W * j - R.head;
#pragma unroll
                for (int u = 0; u < W; u++)
                    if (e + u >= 0 && e + u < V) store_grad(d + e + u, f[u]);
            }
        };
        const bool first = R.lo > 0 && j0 == 0;
        const bool last = R.hi < R.nvec && j0 == (R.nvec - 1) % dj && (R.nvec > 1 || R.lo == 0);
        if (live) {
            auto put = [&](int j, const uint4 &v, bool whole) {
                float f[W];
                grad_vec<T, ETA>(v, g, k22, f);
                store(j, f, whole);
            };
            if (first) put(0, R.load_edge(0), false);
            if (last) put(R.nvec - 1, R.load_edge(R.nvec - 1), false);
            for (int c = nch - 1; c >= 0; c--) {
                const int jc = c * NV * dj + j0;
                if (RING) {
                    take(c);
                    fetch(c - RING_DEPTH);
                }
                if (same && full(c)) {
                    uint4 *dst = dv + jc;
#pragma unroll
                    for (int i = 0; i < NV; i++) {
                        float f[W];
                        grad_vec<T, ETA>(raw[i], g, k22, f);
                        __stcs(dst + i * dj, Vec<T>::make(f));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < NV; i++)
                        if (R.inside(jc + i * dj)) put(jc + i * dj, raw[i], true);
                }
            }
            // the target's entry again, by the thread that has just written its vector
            if ((int)((y + R.head) / W) % dj == j0) store_grad(d + y, g.gy);
        } else {
            float f[W];
#pragma unroll
            for (int u = 0; u < W; u++) f[u] = 0.0f;
            if (first) store(0, f, false);
            if (last) store(R.nvec - 1, f, false);
            for (int j = j0; j < R.hi; j += dj)
                if (j >= R.lo) store(j, f, true);
        }
    }
    if (rank == 0 && tid == 0) {
        if (logprobs) logprobs[row] = lp;
        if (!POLICY && entropy) entropy[row] = H;
    }
    if (POLICY && rank == 0 && tid == 0) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        a.ws->row[row] = st;
    }
}

// the rows' parts, and the weights w where given, added in a fixed order
// (norm 0: the weights' sum; below: it is in ws)
__global__ void __launch_bounds__(1024) policy_stats_kernel(const Ws *__restrict__ ws, const float *__restrict__ w,
                                                            int64_t N, float norm, float beta, float eta,
                                                            float *__restrict__ stats)
{
    __shared__ Sum2 s_tot[32][5];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Sum2 v[5] = {};
    for (int64_t i = tid; i < N; i += 4096) {
        float4 q[4];
        float x[4];
#pragma unroll
        for (int u = 0; u < 4; u++) x[u] = w && i + 1024 * u < N ? __ldg(w + i + 1024 * u) : 0.0f;
#pragma unroll
        for (int u = 0; u < 4; u++)
            q[u] = i + 1024 * u < N ? ws->row[i + 1024 * u] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int u = 0; u < 4; u++) {
            add(v[0], q[u].x);
            add(v[1], q[u].y);
            add(v[2], q[u].z);
            add(v[3], q[u].w);
            add(v[4], x[u]);
        }
    }
#pragma unroll
    for (int i = 0; i < 5; i++) {
        warp_sum2(v[i]);
        if (lane == 0) s_tot[warp][i] = v[i];
    }
    __syncthreads();
    if (warp < 5) {
        Sum2 m = s_tot[lane][warp];
        warp_sum2(m);
        __syncwarp();
        if (lane == 0) s_tot[0][warp] = m;
    }
    __syncthreads();
    if (tid == 0) {
        if (norm == 0.0f) norm = total(s_tot[0][4]);
        else if (norm < 0.0f) norm = ws->norm;
        const float in = norm != 0.0f ? 1.0f / norm : 0.0f;
        const Sum2 pg = s_tot[0][0], kl = s_tot[0][1], H = s_tot[0][2], cl = s_tot[0][3];
        // pg + beta kl - eta H, the products' errors kept (no kl in it for beta 0,
        // where kl may be infinite)
        Sum2 l = pg;
        const float eh = -eta * H.hi;
        if (beta != 0.0f) {
            const float bk = beta * kl.hi;
            add(l, bk);
            l.lo += fmaf(beta, kl.hi, -bk) + beta * kl.lo;
        }
        add(l, eh);
        l.lo += fmaf(-eta, H.hi, -eh) - eta * H.lo;
        stats[0] = total(l) * in;
        stats[1] = total(pg) * in;
        stats[2] = total(kl) * in;
        stats[3] = total(H) * in;
        stats[4] = total(cl) * in;
        stats[5] = norm;
    }
}

// How a row is spread: threads of a CTA, CTAs of a cluster, vectors of a chunk.
// A CTA takes a warp per 256 vectors: up to four for log-probabilities (8192 x
// 16384 bf16: 50 us, 61 with eight warps, 58 with two), up to eight for
// gradients of rows beyond 2048 vectors or few in number (4096 x 10000: four
// warps 44 us, eight 53, where three rows an SM wait for their joins; 4096 x
// 32768: 100 and 96).  A longer row streams in even chunks of at most eight vectors a
// thread (chunks of eight and the rest: 4096 x 20000 bf16 gradients 91 us
// against 73, 4096 x 10000 log-probabilities 24 against 19: an absent vector
// costs its exponentials), one CTA a row where the rows fill the GPU: an
// exchange costs more than it saves (8192 x 131072 log-probabilities 0.30 ms,
// 0.34 with two CTAs, 0.60 with eight); two for the gradient of rows beyond
// 8192 vectors, so that the rows in work stay within L2 until they are read
// again (4096 x 131072: 0.32 ms against 0.37; but 4096 x 60000 0.16 with one,
// 0.19 with two).  More CTAs as rows get few, while each thread keeps a vector.
struct RowPlan {
    int threads, C, NV;
    bool ring;
};
static RowPlan row_plan(int64_t N, int64_t V, int w, bool aligned, bool policy)
{
    const int64_t nvec = (V + w - 1) / w + (aligned ? 0 : 1);
    RowPlan p = {32, policy && nvec > 8192 ? 2 : 1, 8, false};
    const int64_t fill = 4LL * sm_count();
    const int most = (policy && nvec > 2048) || 8 * N <= fill ? 256 : 128;
    while (p.threads < most && p.threads * 8 < nvec) p.threads *= 2;
    while (p.C < 8 && N * p.C * 2 <= fill && (int64_t)p.C * p.threads < nvec) p.C *= 2;
    const int64_t v = (nvec + p.C * p.threads - 1) / (p.C * p.threads), chunks = (v + 7) / 8;     // of a thread
    p.ring = policy && chunks > 1;                                  // (then there are 128 or 256 threads)
    p.NV = (int)((v + chunks - 1) / chunks);
    if (p.NV == 3) p.NV = 4;
    if (p.NV > 4 && (policy ? !p.ring : p.threads > 128)) p.NV += p.NV % 2;     // (no kernel of five or seven)
    return p;
}

template <typename T, int TH, int NV, bool RING, bool POLICY, bool ETA>
static cudaError_t launch_rows_nv(const RowPlan &p, const T *logits, int64_t N, int64_t V, int64_t ld,
                                  const void *targets, int t64, float k2, float *logprobs, float *entropy, T *dlogits,
                                  const PolicyArgs &a, int32_t *dev_status, cudaStream_t st)
{
    auto *kernel = token_rows_kernel<T, TH, NV, RING, POLICY, ETA>;
    constexpr int smem = RING ? RING_DEPTH * NV * TH * 16 : 0;
    if (RING) {
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = allow_smem((const void *)kernel, smem, done);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(N * p.C));
    cfg.blockDim = dim3(p.threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = POLICY && a.norm < 0.0f ? 2 : 1;     // after policy_norm_kernel
    return cudaLaunchKernelEx(&cfg, kernel, logits, N, V, ld, targets, t64, k2, p.C, logprobs, entropy, dlogits, a,
                              dev_status);
}

template <typename T, bool POLICY, bool ETA>
static cudaError_t launch_rows(const T *logits, int64_t N, int64_t V, int64_t ld, const void *targets, int t64,
                               float k2, float *logprobs, float *entropy, T *dlogits, const PolicyArgs &a,
                               int32_t *dev_status, cudaStream_t st)
{
    const bool aligned = aligned16(logits) && (N == 1 || ld % Vec<T>::W == 0);
    const RowPlan p = row_plan(N, V, Vec<T>::W, aligned, POLICY);
#define MOE_ROWS(TH, NV, RING)                                                                                        \
    launch_rows_nv<T, TH, NV, RING, POLICY, ETA>(p, logits, N, V, ld, targets, t64, k2, logprobs, entropy, dlogits,   \
                                                 a, dev_status, st)
#define MOE_ROWS_NV(TH)                                                                                               \
    p.NV == 1 ? MOE_ROWS(TH, 1, false)                                                                                \
    : p.NV == 2 ? MOE_ROWS(TH, 2, false)                                                                              \
    : p.NV == 4 ? MOE_ROWS(TH, 4, false)                                                                              \
    : p.NV == 6 ? MOE_ROWS(TH, 6, false)                                                                              \
                : MOE_ROWS(TH, 8, false)
#define MOE_ROWS_RING(TH)                                                                                             \
    p.NV == 5 ? MOE_ROWS(TH, 5, true)                                                                                 \
    : p.NV == 6 ? MOE_ROWS(TH, 6, true)                                                                               \
    : p.NV == 7 ? MOE_ROWS(TH, 7, true)                                                                               \
                : MOE_ROWS(TH, 8, true)
    if constexpr (POLICY) {
        if (p.ring) return p.threads > 128 ? (MOE_ROWS_RING(256)) : (MOE_ROWS_RING(128));
    } else if (p.NV == 5 || p.NV == 7) {
        return p.NV == 5 ? MOE_ROWS(128, 5, false) : MOE_ROWS(128, 7, false);
    }
    return p.threads > 128 ? (MOE_ROWS_NV(256)) : (MOE_ROWS_NV(128));
#undef MOE_ROWS_RING
#undef MOE_ROWS_NV
#undef MOE_ROWS
}

// log2(e) / temperature, infinite below 4.24e-39 (where every row would be NaN)
static float scale_of(float temperature) { return (float)(1.4426950408889634 / (double)temperature); }

static moe_status check_rows(const void *logits, int dtype, int64_t N, int64_t V, int64_t ld, const void *targets,
                             int target_bits, float temperature)
{
    if (N < 0 || V < 1 || N >= (1LL << 28) || V >= (1LL << 31) || ld < V) return MOE_ERR_SHAPE;
    if (dtype != MOE_LOGITS_BF16 && dtype != MOE_LOGITS_F32) return MOE_ERR_SHAPE;
    if (target_bits != 32 && target_bits != 64) return MOE_ERR_SHAPE;
    if (!isfinite(temperature) || !(temperature > 0.0f) || !isfinite(scale_of(temperature))) return MOE_ERR_SHAPE;
    if (N == 0) return MOE_OK;
    if (!logits || !targets) return MOE_ERR_NULL;
    const uintptr_t es = dtype == MOE_LOGITS_BF16 ? 2 : 4, ts = target_bits / 8;
    if ((uintptr_t)logits % es || (uintptr_t)targets % ts) return MOE_ERR_ALIGN;
    return MOE_OK;
}

static bool overlap(const void *a, int64_t na, const void *b, int64_t nb)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// whether the gradient's rows lie over the logits' in a way other than row on
// row: a row's CTAs would write what another row has yet to read
static bool rows_clash(const void *logits, int64_t ld, const void *d, int64_t ld_d, int64_t N, int64_t V, int64_t es)
{
    if (logits == d) return N > 1 && ld != ld_d;
    if (!d || ld != ld_d || !overlap(logits, ((N - 1) * ld + V) * es, d, ((N - 1) * ld + V) * es)) return false;
    const int64_t off = ((int64_t)((intptr_t)d - (intptr_t)logits) / es % ld + ld) % ld;
    return off < V || ld - off < V;
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
    const float k2 = scale_of(temperature);
    PolicyArgs a = {};
    cudaStream_t st = as_stream(stream);
    const int t64 = target_bits == 64;
    const cudaError_t e =
        logits_dtype == MOE_LOGITS_BF16
            ? launch_rows<uint16_t, false, false>((const uint16_t *)logits, N, V, ld, targets, t64, k2, logprobs,
                                                  entropy, nullptr, a, dev_status, st)
            : launch_rows<float, false, false>((const float *)logits, N, V, ld, targets, t64, k2, logprobs, entropy,
                                               nullptr, a, dev_status, st);
    return e == cudaSuccess ? launch_status() : MOE_ERR_CUDA;
}

MOE_API size_t moe_policy_loss_workspace_size(int64_t N, int64_t V)
{
    (void)V;
    return sizeof(Ws) + sizeof(float4) * (size_t)(N > 0 ? N : 0);
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
        const int es = logits_dtype == MOE_LOGITS_BF16 ? 2 : 4;
        if (dlogits && (uintptr_t)dlogits % es) return MOE_ERR_ALIGN;
        if (rows_clash(logits, ld, dlogits, ld_d, N, V, es)) return MOE_ERR_UNSUPPORTED;
    }
    if (!workspace || workspace_bytes < moe_policy_loss_workspace_size(N, V)) return MOE_ERR_WORKSPACE;
    if (!aligned16(workspace)) return MOE_ERR_ALIGN;
    // every CTA of a row reads its numbers, one of them writes the log-probability
    const float *in[4] = {old_logprobs, advantages, ref_logprobs, weights};
    for (const float *p : in)
        if (overlap(logprobs, 4 * N, p, 4 * N)) return MOE_ERR_UNSUPPORTED;
    if (overlap(logprobs, 4 * N, targets, target_bits / 8 * N)) return MOE_ERR_UNSUPPORTED;
    if (N == 0)
        return cudaMemsetAsync(stats, 0, 6 * sizeof(float), st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    Ws *ws = (Ws *)workspace;
    PolicyArgs a = {old_logprobs, advantages, ref_logprobs, weights, 1.0f - clip_low, 1.0f + clip_high, kl_coef,
                    entropy_coef, ld_d, ws, grad_scale * (1.0f / temperature), norm};
    const bool sum = norm == 0.0f && weights, first = sum && N > NORM_ROWS;
    if (!sum && norm == 0.0f) a.norm = (float)N;
    if (first) a.norm = -1.0f;
    const float k2 = scale_of(temperature);
    const int t64 = target_bits == 64;
    if (first) {
        policy_norm_kernel<<<1, 1024, 0, st>>>(weights, N, a.num, ws);
        if (cudaPeekAtLastError() != cudaSuccess) return launch_status();
    }
    cudaError_t e;
    if (logits_dtype == MOE_LOGITS_BF16)
        e = entropy_coef != 0.0f
                ? launch_rows<uint16_t, true, true>((const uint16_t *)logits, N, V, ld, targets, t64, k2, logprobs,
                                                    nullptr, (uint16_t *)dlogits, a, dev_status, st)
                : launch_rows<uint16_t, true, false>((const uint16_t *)logits, N, V, ld, targets, t64, k2, logprobs,
                                                     nullptr, (uint16_t *)dlogits, a, dev_status, st);
    else
        e = entropy_coef != 0.0f
                ? launch_rows<float, true, true>((const float *)logits, N, V, ld, targets, t64, k2, logprobs, nullptr,
                                                 (float *)dlogits, a, dev_status, st)
                : launch_rows<float, true, false>((const float *)logits, N, V, ld, targets, t64, k2, logprobs,
                                                  nullptr, (float *)dlogits, a, dev_status, st);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    policy_stats_kernel<<<1, 1024, 0, st>>>(ws, sum && !first ? weights : nullptr, N, a.norm,
                                            ref_logprobs ? kl_coef : 0.0f, entropy_coef, stats);
    return launch_status();
}
