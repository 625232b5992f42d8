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
//
// Both are bound by memory where there are many rows (8192 x 7168 bf16, GPU
// alone: forward 39 us = 6.0 TB/s, with both codes 63.5 us = 5.6 TB/s, backward
// from the codes with both additions 119-121 us = 5.4 TB/s; the measured copy
// has 6.8), by the exchanges of a row and its instructions where a value is one
// instruction each (rows without whole vectors: 2.2-3.6 TB/s).
#include <initializer_list>
#include <type_traits>

#include "losses.cuh"

namespace moe {
namespace norm {

constexpr int MAX_COLS = 16384;
constexpr int SMEM_MAX = 220 * 1024;

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

// Sums of a (and with `two` of b) over the warps of a row's group, the same
// bits in every thread: within the warp the lower half-warp ends up with a's
// sum and the upper one with b's (one exchange more than for a alone), the
// warps' parts meet in shared memory and are added the same way.  `red` is
// this exchange's own buffer, [2][32] floats, and `first` where the group's parts
// start in each; `bar` its named barrier (0: the whole CTA).  One warp: no
// exchange.
__device__ __forceinline__ void row_sums(float &a, float &b, bool two, float *red, int first, int warps, int warp,
                                         int lane, int bar)
{
    float v;
    if (two) {
        const bool up = lane & 16;
        v = (up ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, up ? a : b, 16);
    } else {
        v = a + __shfl_xor_sync(0xFFFFFFFFu, a, 16);
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (warps > 1) {
        const int l = lane & 15, k = (lane >> 4) * 32 + first;
        if (l == 0) red[k + warp] = v;                 // without `two` both halves hold the same sum
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(warps * 32) : "memory");
        v = l < warps ? red[k + l] : 0.0f;
        if (l + 16 < warps) v += red[k + l + 16];
#pragma unroll
        for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    }
    a = __shfl_sync(0xFFFFFFFFu, v, 0);
    if (two) b = __shfl_sync(0xFFFFFFFFu, v, 16);
}

// ---- rows on their way through shared memory ----
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src)
{
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

// the oldest of `stages` pending groups
__device__ __forceinline__ void wait_oldest(int stages)
{
    if (stages == 1) cp_async_wait<0>();
    else if (stages == 2) cp_async_wait<1>();
    else if (stages == 3) cp_async_wait<2>();
    else cp_async_wait<3>();
}

__device__ __forceinline__ void group_sync(int warps, int bar)
{
    if (warps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(warps * 32) : "memory");
}

// A row without whole vectors, copied as the 16-byte pieces it lies in, by
// all threads of its group (thread t of nth): column c lands at
// dst + (start & 15) + c * sizeof(T).  Bytes behind the row are not read; the
// piece it starts in may hold bytes of the row before, but where it would
// reach back beyond the tensor's first row the values are copied one by one.
// `pieces` is the same for every row (one more than the row may touch: zeros),
// so that nothing of another row stays behind this one.
// the most pieces that a row of that many bytes lies in
__host__ __device__ constexpr int odd_pieces(int bytes) { return (bytes + 14 + 15) / 16; }

template <typename T>
__device__ __forceinline__ void copy_odd(uint32_t dst, const T *base, int64_t at, int cols, int t, int nth)
{
    const char *start = reinterpret_cast<const char *>(base + at);
    const int shift = (int)(reinterpret_cast<uintptr_t>(start) & 15), bytes = shift + cols * (int)sizeof(T);
    const char *from = start - shift;
    const int pieces = odd_pieces(cols * (int)sizeof(T));
    int k = t;
    if (from < reinterpret_cast<const char *>(base)) {         // the first row, where the tensor starts off a boundary
        for (int c = t; c * (int)sizeof(T) < 16 - shift; c += nth) {                 // zeros behind a row that ends here
            const uint32_t to = dst + shift + c * (int)sizeof(T);
            if (sizeof(T) == 4) asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(c < cols ? reinterpret_cast<const uint32_t *>(start)[c] : 0u) : "memory");
            else asm volatile("st.shared.b16 [%0], %1;" ::"r"(to), "h"(c < cols ? reinterpret_cast<const uint16_t *>(start)[c] : (uint16_t)0) : "memory");
        }
        if (k == 0) k = nth;                                   // its first piece is done
    }
    for (; k < pieces; k += nth) {
        const int left = bytes - 16 * k;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16 * k), "l"(left > 0 ? from + 16 * k : from + 16),
                     "r"(left > 0 ? (left < 16 ? left : 16) : 0)
                     : "memory");
    }
}

template <typename T>
__device__ __forceinline__ int odd_shift(const T *base, int64_t at) { return (int)(reinterpret_cast<uintptr_t>(base + at) & 15); }

// VEC values to pairs; of single values two that lie 32 apart, the second one 0 where it is absent
template <typename T, int VEC>
__device__ __forceinline__ void pairs(const T *p, bool second, uint64_t (&v)[(VEC + 1) / 2])
{
    if constexpr (VEC == 1) {
        float a[1], b[1] = {0.0f};
        load<T, 1>(p, a);
        if (second) load<T, 1>(p + 32, b);
        v[0] = pack2(a[0], b[0]);
    } else {
        float f[VEC];
        load<T, VEC>(p, f);
#pragma unroll
        for (int j = 0; j < VEC / 2; j++) v[j] = pack2(f[2 * j], f[2 * j + 1]);
    }
}

// Zeros in shared memory behind the columns of a row (bytes from..to, both
// multiples of 4), once: a thread whose columns lie there reads them and needs
// no question (its stores do).  No row's copy writes there.
__device__ __forceinline__ void clear(uint8_t *p, int from, int to)
{
    for (int b = from + 4 * (int)threadIdx.x; b < to; b += 4 * (int)blockDim.x) *reinterpret_cast<uint32_t *>(p + b) = 0u;
}

// A weight in fp32 in shared memory (`none` where there is none), for a CTA
// that meets many rows: no conversion and no question of its type a row.
// Vectors of eight lie as two halves, so that a warp reads whole banks.  wide:
// the columns that the row's threads have together; zeros behind the last one.
template <int VEC, bool F32>
__device__ __forceinline__ void stage_weight_of(float *dst, const void *w, int cols, int wide)
{
    if constexpr (VEC == 1) {
#pragma unroll 8
        for (int c = threadIdx.x; c < cols; c += blockDim.x)
            dst[c] = F32 ? __ldg(static_cast<const float *>(w) + c) : bf16_bits_to_f32(__ldg(static_cast<const uint16_t *>(w) + c));
    } else {
#pragma unroll 4
        for (int q = threadIdx.x; q < cols >> 2; q += blockDim.x) {
            float4 f;
            if constexpr (F32) {
                f = __ldg(static_cast<const float4 *>(w) + q);
            } else {
                const uint2 v = __ldg(static_cast<const uint2 *>(w) + q);
                f = make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                                __uint_as_float(v.y & 0xFFFF0000u));
            }
            *reinterpret_cast<float4 *>(dst + (VEC == 8 ? (q >> 1) * 4 + (q & 1 ? wide >> 1 : 0) : 4 * q)) = f;
        }
    }
}
template <int VEC>
__device__ __forceinline__ void stage_weight(float *dst, const void *w, bool f32, int cols, int wide, float none)
{
    for (int c = (w ? cols : 0) + threadIdx.x; c < wide; c += blockDim.x)
        dst[VEC == 8 ? (c >> 3) * 4 + (c & 3) + (c & 4 ? wide >> 1 : 0) : c] = c < cols ? none : 0.0f;
    if (!w) return;
    if (f32) stage_weight_of<VEC, true>(dst, w, cols, wide);
    else stage_weight_of<VEC, false>(dst, w, cols, wide);
}
// the pairs of a vector from column c on (of single values c and c + 32)
template <int VEC>
__device__ __forceinline__ void staged_weight(const float *s, int c, int wide, uint64_t (&w)[(VEC + 1) / 2])
{
    if constexpr (VEC == 1) {
        w[0] = pack2(s[c], s[c + 32]);
    } else {
        const float4 a = *reinterpret_cast<const float4 *>(s + (VEC == 8 ? c >> 1 : c));
        w[0] = pack2(a.x, a.y);
        w[1] = pack2(a.z, a.w);
        if constexpr (VEC == 8) {
            const float4 b = *reinterpret_cast<const float4 *>(s + (wide >> 1) + (c >> 1));
            w[2] = pack2(b.x, b.y);
            w[3] = pack2(b.z, b.w);
        }
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
    int cols, wide;             // the row's columns, and those that its threads have together
    int warps, groups;          // warps of a row, rows that a CTA has at work
    int stages, stage_bytes;    // of a group's ring
    int weight_bytes;           // of the weights in shared memory
    float eps;
    bool center, w_f32;
};

// N values of each lane reduced (largest) over groups of G lanes, N <= G
// powers of two: value i is left in the lanes of the group whose number
// within it starts, in its log2(N) highest bits, with i.  Each step keeps
// half of the values: N - 1 + log2(G / N) shuffles, where a reduction of each
// takes N log2(G) (N = 4, G = 16: 5 against 16).
template <int N, int G>
__device__ __forceinline__ float scatter_max(float (&v)[N], int lane)
{
    int o = G / 2;
#pragma unroll
    for (int n = N / 2; n; n /= 2, o /= 2) {
        const bool hi = lane & o;
#pragma unroll
        for (int i = 0; i < n; i++)
            v[i] = fmaxf(hi ? v[n + i] : v[i], __shfl_xor_sync(0xFFFFFFFFu, hi ? v[i] : v[n + i], o));
    }
#pragma unroll
    for (; o; o /= 2) v[0] = fmaxf(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], o));
    return v[0];
}

// A thread's VPT vectors of a row to codes: a 128-block is one vector of
// 128 / VEC lanes.  Each scale is formed once, by the lanes that end up with
// its block's largest value.  c: the thread's first column; q, s: the row's.
template <int VEC, int VPT>
__device__ __forceinline__ void encode(const uint64_t (&v)[VPT][VEC / 2], int c, int cols, int lane, uint8_t *q, float *s)
{
    constexpr int G = 128 / VEC, EACH = G / VPT;               // lanes of a block; lanes that hold one block's value
    float m[VPT];
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        m[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < VEC / 2; j++) {
            float a, b;
            unpack2(v[i][j], a, b);
            m[i] = amax3(a, b, m[i]);
        }
    }
    const float sc = computed_scale(scatter_max<VPT, G>(m, lane)), y = computed_recip(sc);
    const int mine = (lane & (G - 1)) / EACH;                  // the vector whose scale this lane has
    const int c_mine = c - (lane & (G - 1)) * VEC + mine * 32 * VEC;
    if ((lane & (EACH - 1)) == 0 && c_mine < cols) s[c_mine >> 7] = sc;
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const float yi = __shfl_sync(0xFFFFFFFFu, y, (lane & ~(G - 1)) + i * EACH);
        if (c + i * 32 * VEC >= cols) continue;
        const uint64_t y2 = pack2(yi, yi);
        uint32_t w[VEC / 4];
#pragma unroll
        for (int k = 0; k < VEC / 4; k++) {
            float a, b, e, f;
            unpack2(mul2(v[i][2 * k], y2), a, b);
            unpack2(mul2(v[i][2 * k + 1], y2), e, f);
            w[k] = e4m3x4_pack(a, b, e, f);
        }
        if constexpr (VEC == 8) *reinterpret_cast<uint2 *>(q + c + i * 32 * VEC) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t *>(q + c + i * 32 * VEC) = w[0];
    }
}

// A row per group of warps, held in registers (EPT values a thread, two in
// each 64-bit pair) from its one reading to the stores.  A warp's vectors lie
// side by side, so a thread's addresses are one base and constants.  With
// RING the groups take rows in turn over the whole grid, and the next rows are
// on their way through a ring in shared memory (8192 x 7168 bf16: 40 us; one
// row a CTA at a time, 28 KB in flight an SM, 67); without, each group has one
// row, read straight to registers (one row of 7168: 2.8 us).  The mean is
// taken twice: the sum of x - mu' with the first mean mu' gives what rounding
// left out of it, at no further exchange (it rides with the sum of squares).
template <typename T, int VEC, int EPT, bool RING>
__global__ void __launch_bounds__(EPT == 8 ? 1024 : 512, EPT == 16 ? 2 : 1) norm_kernel(Fwd p)
{
    constexpr int N = VEC > 1 ? EPT / VEC : EPT / 2, H = VEC > 1 ? VEC / 2 : 1;      // vectors, or pairs of single values
    constexpr int STEP = VEC > 1 ? 32 * VEC : 64;              // columns from one to the next
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float red[2][64];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = warp / p.warps, gw = warp - group * p.warps;
    const int c = gw * 32 * EPT + lane * VEC;          // the thread's first column
    const float inv_n = 1.0f / (float)p.cols;
    const auto in = [&](int i) { return c + i * STEP < p.cols; };
    const auto in2 = [&](int i) { return c + i * STEP + 32 < p.cols; };              // a pair's second single value
    const int64_t first = (int64_t)blockIdx.x * p.groups + group, step = (int64_t)gridDim.x * p.groups;
    // RING: the weights, then the groups' rings
    float *sw = reinterpret_cast<float *>(ring), *sb = sw + p.wide;
    uint8_t *mine = ring + p.weight_bytes + group * p.stages * p.stage_bytes;
    const auto issue = [&](int64_t row, int stage) {
        if (row < p.rows) {
            const uint32_t dst = smem_u32(mine) + stage * p.stage_bytes;
            if constexpr (VEC > 1) {
                const T *src = static_cast<const T *>(p.x) + row * p.ld_x + c;
#pragma unroll
                for (int i = 0; i < N; i++)
                    if (in(i)) copy_async<16>(dst + c * (int)sizeof(T) + i * 512, src + i * STEP);
            } else {
                copy_odd<T>(dst, static_cast<const T *>(p.x), row * p.ld_x, p.cols, gw * 32 + lane, p.warps * 32);
            }
        }
        cp_async_commit();
    };
    int stage = 0, par = 0;
    if constexpr (RING) {
        for (int s = 0; s < p.stages; s++) issue(first + s * step, s);
        for (int s = 0; s < p.groups * p.stages; s++)
            clear(ring + p.weight_bytes + s * p.stage_bytes,
                  VEC == 1 ? 16 * odd_pieces(p.cols * (int)sizeof(T)) : p.cols * (int)sizeof(T), p.stage_bytes);
        stage_weight<VEC>(sw, p.w, p.w_f32, p.cols, p.wide, 1.0f);
        if (p.b) stage_weight<VEC>(sb, p.b, p.w_f32, p.cols, p.wide, 0.0f);
        __syncthreads();
    }
    for (int64_t row = first; row < p.rows; row += step, par ^= 1) {
        uint64_t v[N][H];
        {
            const T *x = static_cast<const T *>(p.x) + row * p.ld_x + c;
            if constexpr (RING) {
                wait_oldest(p.stages);
                const uint8_t *st = mine + stage * p.stage_bytes;
                if (VEC == 1) {
                    group_sync(p.warps, group + 1);        // the row's pieces were copied by others
                    st += odd_shift(static_cast<const T *>(p.x), row * p.ld_x);
                }
                x = reinterpret_cast<const T *>(st) + c;
            }
#pragma unroll
            for (int i = 0; i < N; i++) {
#pragma unroll
                for (int j = 0; j < H; j++) v[i][j] = 0;
                if (RING || in(i)) pairs<T, VEC>(x + i * STEP, RING || in2(i), v[i]);
            }
        }
        float sum = 0.0f, sq = 0.0f;
        if (p.center) {
            uint64_t s2 = 0;
#pragma unroll
            for (int i = 0; i < N; i++) {
#pragma unroll
                for (int j = 0; j < H; j++) s2 = add2(s2, v[i][j]);
            }
            unpack2(s2, sum, sq);
            sum += sq;
            sq = 0.0f;
            row_sums(sum, sq, false, red[0], group * p.warps, p.warps, gw, lane, group + 1);
        }
        const float mu = sum * inv_n;
        uint64_t s2 = 0, q2 = 0;
        if (p.center) {
#pragma unroll
            for (int i = 0; i < N; i++) {
                // absent columns stay 0
                const float m0 = in(i) ? -mu : 0.0f, m1 = VEC > 1 ? m0 : in2(i) ? -mu : 0.0f;
                const uint64_t m = pack2(m0, m1);
#pragma unroll
                for (int j = 0; j < H; j++) {
                    v[i][j] = add2(v[i][j], m);
                    s2 = add2(s2, v[i][j]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < N; i++) {
#pragma unroll
            for (int j = 0; j < H; j++) q2 = fma2(v[i][j], v[i][j], q2);
        }
        float a, b;
        unpack2(s2, a, b);
        sum = a + b;
        unpack2(q2, a, b);
        sq = a + b;
        // with one exchange a row the buffers alternate: a warp a row ahead writes the other one
        row_sums(sq, sum, p.center, red[p.center ? 1 : par], group * p.warps, p.warps, gw, lane, group + 1);
        if constexpr (RING) {
            if (VEC == 1 && p.warps == 1) __syncwarp();
            issue(row + p.stages * step, stage);           // the row is in registers (of others too: past their barrier)
        }
        if (RING && ++stage == p.stages) stage = 0;
        const float rest = p.center ? sum * inv_n : 0.0f;
        float var = fmaf(sq, inv_n, -rest * rest);
        if (var < 0.0f) var = 0.0f;                        // a NaN stays
        const float rstd = rsqrtf(var + p.eps);
        if (gw == 0 && lane == 0) {
            if (p.mean) p.mean[row] = mu + rest;
            if (p.rstd) p.rstd[row] = rstd;
        }
        const uint64_t r2 = pack2(rstd, rstd), c2 = pack2(-rest * rstd, -rest * rstd);
        if (p.center) {
#pragma unroll
            for (int i = 0; i < N; i++) {
#pragma unroll
                for (int j = 0; j < H; j++) v[i][j] = fma2(v[i][j], r2, c2);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) {
#pragma unroll
                for (int j = 0; j < H; j++) v[i][j] = mul2(v[i][j], r2);
            }
        }
        T *y = static_cast<T *>(p.y) + row * p.ld_y + c;
        if constexpr (VEC > 1) {
            const int64_t at = row * p.cols, at_s = row * (p.cols >> 7);
            if (p.h_q) encode<VEC, N>(v, c, p.cols, lane, p.h_q + at, p.h_s + at_s);
            const auto weigh = [&](auto biased) {
#pragma unroll
                for (int i = 0; i < N; i++) {
                    constexpr bool B = decltype(biased)::value;
                    uint64_t w[H] = {}, f2[H] = {};
                    float f[VEC];
                    if constexpr (RING) {
                        staged_weight<VEC>(sw, c + i * STEP, p.wide, w);
                        if (B) staged_weight<VEC>(sb, c + i * STEP, p.wide, f2);
                    } else if (in(i)) {
                        load_weight<VEC>(p.w, p.w_f32, c + i * STEP, 1.0f, f);
#pragma unroll
                        for (int j = 0; j < H; j++) w[j] = pack2(f[2 * j], f[2 * j + 1]);
                        if (B) {
                            load_weight<VEC>(p.b, p.w_f32, c + i * STEP, 0.0f, f);
#pragma unroll
                            for (int j = 0; j < H; j++) f2[j] = pack2(f[2 * j], f[2 * j + 1]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < H; j++) {
                        v[i][j] = B ? fma2(v[i][j], w[j], f2[j]) : mul2(v[i][j], w[j]);
                        unpack2(v[i][j], f[2 * j], f[2 * j + 1]);
                    }
                    if (in(i)) store<T, VEC>(y + i * STEP, f);
                }
            };
            if (p.b) weigh(std::true_type());
            else weigh(std::false_type());
            if (p.y_q) encode<VEC, N>(v, c, p.cols, lane, p.y_q + at, p.y_s + at_s);
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) {
                uint64_t w[1], f2[1] = {0};
                if constexpr (RING) {
                    staged_weight<1>(sw, c + i * STEP, p.wide, w);
                    if (p.b) staged_weight<1>(sb, c + i * STEP, p.wide, f2);
                } else if (in(i)) {
                    float a1[1], b1[1] = {0.0f};
                    load_weight<1>(p.w, p.w_f32, c + i * STEP, 1.0f, a1);
                    if (in2(i)) load_weight<1>(p.w, p.w_f32, c + i * STEP + 32, 1.0f, b1);
                    w[0] = pack2(a1[0], b1[0]);
                    load_weight<1>(p.b, p.w_f32, c + i * STEP, 0.0f, a1);
                    if (in2(i)) load_weight<1>(p.b, p.w_f32, c + i * STEP + 32, 0.0f, b1);
                    f2[0] = pack2(a1[0], b1[0]);
                }
                float lo[1], hi[1];
                unpack2(fma2(v[i][0], w[0], f2[0]), lo[0], hi[0]);
                if (in(i)) store<T, 1>(y + i * STEP, lo);
                if (in2(i)) store<T, 1>(y + i * STEP + 32, hi);
            }
        }
        if constexpr (!RING) break;
    }
    cp_async_wait<0>();
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
    int64_t ld_dy, ld_x, ld_add, ld_dx;
    int rows, cols, wide, warps, groups, stages;
    // a stage of a group in shared memory: dy, then x or the codes, the scales, dy_add (-1: not staged)
    int stage_bytes, at_x, at_s, at_dya, weight_bytes;
    bool center, w_f32, want_w, want_b;
};

// VEC codes of one block to fp32, times its scale
template <int VEC>
__device__ __forceinline__ void decode(const uint8_t *q, float s, uint64_t (&v)[VEC / 2])
{
    uint32_t w[VEC / 4];
    if constexpr (VEC == 8) {
        const uint2 r = *reinterpret_cast<const uint2 *>(q);
        w[0] = r.x, w[1] = r.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(q);
    }
    const uint64_t s2 = pack2(s, s);
#pragma unroll
    for (int i = 0; i < VEC / 4; i++) {
        float f[4];
        e4m3x4_unpack(w[i], f);
        v[2 * i] = mul2(pack2(f[0], f[1]), s2);
        v[2 * i + 1] = mul2(pack2(f[2], f[3]), s2);
    }
}

// Rows over groups of warps, grid-wide in turn; a thread owns the same EPT
// columns of every row of its group, so the sums over rows stay in registers
// until the CTA's last row.  Rows come through a ring in shared memory, whole
// vectors copied asynchronously by the thread that reads them, rows without
// as the pieces they lie in (and a barrier).  With KEEP a thread holds g and xhat of
// its columns from the row's means to dx; without (rows too long for that
// beside the sums) it reads them again.  FULL: with the rows' means and the sums
// of db; else the RMS form without.  At the end the groups' sums are
// joined in group order through shared memory and leave as this CTA's part;
// reduce_kernel adds the parts in CTA order (no atomics: the same bits every
// time).  8192 x 7168 bf16 from x: RMS 66 us (5.3 TB/s), FULL 79 (4.5: the
// instructions of one group of 14 warps an SM).  More threads at fewer
// registers (896 at 72) or two rows at a time spill, which next to 220 KB of
// shared memory costs 1.5 times the whole.
constexpr int BWD_THREADS = 512;                       // at up to 128 registers

// ADD: 0 without dy_add and dx_add; 1 with either or both, dy_add in the ring;
// 2 with dy_add read in place (fp32 rows too long for the ring with it).  One
// kernel that asked would hold the addresses beside the sums: 8192 x 7168 bf16
// from codes without either 67 us against 74, 4096 x 16384 from x 93 against 138,
// 8192 x 5001 88 against 102.  In the ring even where that leaves one stage: 4096 x
// 16384 bf16 220 us against 268-288 in place, 8192 x 5001 137 against 353.
template <typename T, int VEC, int EPT, bool CKPT, bool FULL, int ADD>
__global__ void __launch_bounds__(BWD_THREADS, 1) dnorm_kernel(Bwd p)
{
    // vectors, or pairs of single values 32 columns apart
    constexpr int N = VEC > 1 ? EPT / VEC : EPT / 2, H = (VEC + 1) / 2, STEP = VEC > 1 ? 32 * VEC : 64;
    constexpr bool KEEP = EPT == 16;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float red[2][64];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = warp / p.warps, gw = warp - group * p.warps;
    const int c = gw * 32 * EPT + lane * VEC, left = p.cols - c;       // the thread's first column, and those from there on
    const float inv_n = 1.0f / (float)p.cols;
    const int first = (int)blockIdx.x * p.groups + group, step = (int)gridDim.x * p.groups;
    float *sw = reinterpret_cast<float *>(ring);       // the weight, then the groups' rings
    uint8_t *mine = ring + p.weight_bytes + group * p.stages * p.stage_bytes;
    const uint32_t mine_u = smem_u32(mine);
    const int half = p.wide * 2;                       // bytes of the first halves of dy_add's vectors of eight
    const auto in = [&](int i) { return i * STEP < left; };
    const auto in2 = [&](int i) { return i * STEP + 32 < left; };      // a pair's second single value

    const auto issue = [&](int64_t row, int stage) {
        if constexpr (VEC == 1) {
            if (row < p.rows) {
                const uint32_t dst = mine_u + stage * p.stage_bytes;
                copy_odd<T>(dst, static_cast<const T *>(p.dy), row * p.ld_dy, p.cols, gw * 32 + lane, p.warps * 32);
                copy_odd<T>(dst + p.at_x, static_cast<const T *>(p.x), row * p.ld_x, p.cols, gw * 32 + lane, p.warps * 32);
                if (ADD == 1 && p.at_dya >= 0) copy_odd<float>(dst + p.at_dya, p.dy_add, row * p.cols, p.cols, gw * 32 + lane, p.warps * 32);
            }
        } else {
            if (row < p.rows) {
                const uint32_t dst = mine_u + stage * p.stage_bytes;
                const T *dy = static_cast<const T *>(p.dy) + row * p.ld_dy + c;
                const int64_t at = row * p.cols + c;
#pragma unroll
                for (int i = 0; i < N; i++)
                    if (in(i)) copy_async<16>(dst + c * (int)sizeof(T) + i * 512, dy + i * STEP);
                if constexpr (CKPT) {
                    const uint8_t *q = p.h_q + at;
                    const float *s = p.h_s + (at >> 7);
#pragma unroll
                    for (int i = 0; i < N; i++) {
                        if (!in(i)) continue;
                        copy_async<VEC>(dst + p.at_x + c + i * STEP, q + i * STEP);
                        if ((lane & (128 / VEC - 1)) == 0)
                            copy_async<4>(dst + p.at_s + (c >> 7) * 4 + i * STEP / 32, s + i * STEP / 128);
                    }
                } else {
                    const T *x = static_cast<const T *>(p.x) + row * p.ld_x + c;
#pragma unroll
                    for (int i = 0; i < N; i++)
                        if (in(i)) copy_async<16>(dst + p.at_x + c * (int)sizeof(T) + i * 512, x + i * STEP);
                }
                if (ADD == 1 && p.at_dya >= 0) {
                    const float *d = p.dy_add + at;
#pragma unroll
                    for (int i = 0; i < N; i++) {
                        if (!in(i)) continue;
                        copy_async<16>(dst + p.at_dya + c / VEC * 16 + i * 512, d + i * STEP);
                        if (VEC == 8) copy_async<16>(dst + p.at_dya + half + c / VEC * 16 + i * 512, d + i * STEP + 4);
                    }
                }
            }
        }
        cp_async_commit();
    };
    // vector i of the row: a = dy + dy_add and xhat = (x - mu) r, or from its codes.  dy, x: the row in shared memory
    const auto get = [&](int64_t row, const uint8_t *st, const T *dy, const T *x, int i, uint64_t rs2, uint64_t nmu2,
                         uint64_t (&a)[H], uint64_t (&h)[H]) {
        pairs<T, VEC>(dy + i * STEP, true, a);
        if constexpr (CKPT) {
            decode<VEC>(st + p.at_x + c + i * STEP,
                        *reinterpret_cast<const float *>(st + p.at_s + (c >> 7) * 4 + i * STEP / 32), h);
        } else {
            pairs<T, VEC>(x + i * STEP, true, h);
#pragma unroll
            for (int j = 0; j < H; j++) h[j] = mul2(FULL ? add2(h[j], nmu2) : h[j], rs2);
        }
        if (ADD == 1 && p.at_dya >= 0) {
            if constexpr (VEC > 1) {
#pragma unroll
                for (int k = 0; k < VEC / 4; k++) {
                    const float4 d = *reinterpret_cast<const float4 *>(st + p.at_dya + k * half + c / VEC * 16 + i * 512);
                    a[2 * k] = add2(a[2 * k], pack2(d.x, d.y));
                    a[2 * k + 1] = add2(a[2 * k + 1], pack2(d.z, d.w));
                }
            } else {
                const float *d = reinterpret_cast<const float *>(st + p.at_dya + odd_shift(p.dy_add, row * p.cols)) + c + i * STEP;
                a[0] = add2(a[0], pack2(d[0], d[32]));
            }
        } else if (ADD == 2 && p.dy_add && in(i)) {
            const float *d = p.dy_add + row * p.cols + c + i * STEP;
            if constexpr (VEC > 1) {
#pragma unroll
                for (int j = 0; j < H; j++) a[j] = add2(a[j], pack2(__ldg(d + 2 * j), __ldg(d + 2 * j + 1)));
            } else {
                a[0] = add2(a[0], pack2(__ldg(d), in2(i) ? __ldg(d + 32) : 0.0f));
            }
        }
    };
    const auto weights = [&](int i, uint64_t (&w)[H]) { staged_weight<VEC>(sw, c + i * STEP, p.wide, w); };

    uint64_t dw[N][H] = {}, db[FULL ? N : 1][H] = {};
    for (int s = 0; s < p.stages; s++) issue((int64_t)first + (int64_t)s * step, s);
    if (VEC == 1 || p.wide != p.cols) {
        const int row = VEC == 1 ? 16 * odd_pieces(p.cols * (int)sizeof(T)) : p.cols * (int)sizeof(T);
        for (int s = 0; s < p.groups * p.stages; s++) {
            uint8_t *st = ring + p.weight_bytes + s * p.stage_bytes;
            clear(st, row, p.at_x);
            clear(st, p.at_x + (CKPT ? p.cols : row), p.at_s);
            if (CKPT) clear(st, p.at_s + p.cols / 32, p.at_s + p.wide / 32);
            if (VEC == 1) {
                if (ADD == 1 && p.at_dya >= 0) clear(st, p.at_dya + 16 * odd_pieces(p.cols * 4), p.stage_bytes);
            } else if (ADD == 1 && p.at_dya >= 0) {    // of eights two halves
                clear(st, p.at_dya + p.cols * (VEC == 8 ? 2 : 4), p.at_dya + p.wide * (VEC == 8 ? 2 : 4));
                if (VEC == 8) clear(st, p.at_dya + half + p.cols * 2, p.at_dya + half + p.wide * 2);
            }
        }
    }
    stage_weight<VEC>(sw, p.w, p.w_f32, p.cols, p.wide, 1.0f);
    __syncthreads();
    float rs_next = 0.0f, mu_next = 0.0f;              // the next row's, loaded a row ahead
    const bool mean = FULL && !CKPT && p.center;
    if (first < p.rows) {
        rs_next = __ldg(p.rstd + first);
        if (mean) mu_next = __ldg(p.mean + first);
    }
    int par = 0, stage = 0;
    for (int64_t row = first; row < p.rows; row += step, par ^= 1) {
        const float rs = rs_next;
        const uint64_t rs2 = pack2(rs, rs), nmu2 = pack2(-mu_next, -mu_next);
        if (row + step < p.rows) {
            rs_next = __ldg(p.rstd + row + step);
            if (mean) mu_next = __ldg(p.mean + row + step);
        }
        typename Vec<T, VEC>::Raw add[N], more[VEC > 1 ? 1 : N];      // dx_add: on its way while the means are formed
        if (ADD && p.dx_add) {
            const T *src = static_cast<const T *>(p.dx_add) + row * p.ld_add + c;
#pragma unroll
            for (int i = 0; i < N; i++) {
                if (in(i)) add[i] = *reinterpret_cast<const typename Vec<T, VEC>::Raw *>(src + i * STEP);
                if (VEC == 1 && in2(i)) more[VEC > 1 ? 0 : i] = *reinterpret_cast<const typename Vec<T, VEC>::Raw *>(src + i * STEP + 32);
            }
            // the next row's as far as L2, a lane for each 128 bytes (8192 x 7168 from codes with both additions: 119 us
            // against 124; there is no room for it in the ring beside dy_add)
            if (row + step < p.rows && (lane & (VEC > 1 ? 7 : 31)) == 0) {
                const T *next = src + step * p.ld_add;
#pragma unroll
                for (int i = 0; i < N; i++) {
                    if (in(i)) asm volatile("prefetch.global.L2 [%0];" ::"l"(next + i * STEP));
                    if (VEC == 1 && sizeof(T) == 4 && in2(i)) asm volatile("prefetch.global.L2 [%0];" ::"l"(next + i * STEP + 32));
                }
            }
        }
        const uint8_t *st = mine + stage * p.stage_bytes;
        wait_oldest(p.stages);
        if (CKPT) __syncwarp();                        // a block's scale was copied by one of its lanes
        if (VEC == 1) group_sync(p.warps, group + 1);  // the row's pieces were copied by others
        const T *dy = reinterpret_cast<const T *>(st) + c, *x = reinterpret_cast<const T *>(st + p.at_x) + c;
        if (VEC == 1) {
            dy = reinterpret_cast<const T *>(st + odd_shift(static_cast<const T *>(p.dy), row * p.ld_dy)) + c;
            x = reinterpret_cast<const T *>(st + p.at_x + odd_shift(static_cast<const T *>(p.x), row * p.ld_x)) + c;
        }
        uint64_t g[KEEP ? N : 1][H], h[KEEP ? N : 1][H];
        uint64_t s1 = 0, s2 = 0;
#pragma unroll
        for (int i = 0; i < N; i++) {
            uint64_t (&hi)[H] = h[KEEP ? i : 0], (&gi)[H] = g[KEEP ? i : 0];
            uint64_t a[H], w[H];
            get(row, st, dy, x, i, rs2, nmu2, a, hi);
            weights(i, w);
#pragma unroll
            for (int j = 0; j < H; j++) {
                gi[j] = mul2(a[j], w[j]);
                if (FULL) s1 = add2(s1, gi[j]);
                s2 = fma2(gi[j], hi[j], s2);
                dw[i][j] = fma2(a[j], hi[j], dw[i][j]);
                if (FULL) db[i][j] = add2(db[i][j], a[j]);
            }
        }
        if (KEEP && VEC > 1) {
            if (CKPT) __syncwarp();
            issue(row + (int64_t)p.stages * step, stage);
        }
        if (p.dx) {
            float m1, m2, lo, up;
            unpack2(s1, lo, up);
            m1 = lo + up;
            unpack2(s2, lo, up);
            m2 = lo + up;
            // the buffer alternates by row: a warp a row ahead writes the other one
            row_sums(m2, m1, FULL, red[par], group * p.warps, p.warps, gw, lane, group + 1);
            m1 = FULL && p.center ? m1 * inv_n : 0.0f, m2 *= inv_n;
            const uint64_t nm1 = pack2(-m1, -m1), nm2 = pack2(-m2, -m2);
            T *dx = static_cast<T *>(p.dx) + row * p.ld_dx + c;
#pragma unroll
            for (int i = 0; i < N; i++) {
                uint64_t (&hi)[H] = h[KEEP ? i : 0], (&gi)[H] = g[KEEP ? i : 0];
                if (!KEEP) {
                    uint64_t w[H];
                    get(row, st, dy, x, i, rs2, nmu2, gi, hi);
                    weights(i, w);
#pragma unroll
                    for (int j = 0; j < H; j++) gi[j] = mul2(gi[j], w[j]);
                }
                constexpr int M = VEC > 1 ? VEC : 2;
                float f[M];
                if (ADD && p.dx_add) {
                    float d[M] = {};
                    if (in(i)) {
                        float r[VEC];
                        Vec<T, VEC>::get(add[i], r);
#pragma unroll
                        for (int j = 0; j < VEC; j++) d[j] = r[j];
                        if (VEC == 1 && in2(i)) {
                            Vec<T, VEC>::get(more[VEC > 1 ? 0 : i], r);
                            d[1] = r[0];
                        }
                    }
#pragma unroll
                    for (int j = 0; j < H; j++)
                        unpack2(fma2(fma2(hi[j], nm2, FULL ? add2(gi[j], nm1) : gi[j]), rs2, pack2(d[2 * j], d[2 * j + 1])),
                                f[2 * j], f[2 * j + 1]);
                } else {
#pragma unroll
                    for (int j = 0; j < H; j++)
                        unpack2(mul2(fma2(hi[j], nm2, FULL ? add2(gi[j], nm1) : gi[j]), rs2), f[2 * j], f[2 * j + 1]);
                }
                if constexpr (VEC > 1) {
                    if (in(i)) store<T, VEC>(dx + i * STEP, f);
                } else {
                    const float lo[1] = {f[0]}, hi1[1] = {f[1]};
                    if (in(i)) store<T, 1>(dx + i * STEP, lo);
                    if (in2(i)) store<T, 1>(dx + i * STEP + 32, hi1);
                }
            }
        }
        if (!KEEP || VEC == 1) {
            if (CKPT) __syncwarp();
            if (VEC == 1) group_sync(p.warps, group + 1);       // everyone has read the row
            issue(row + (int64_t)p.stages * step, stage);
        }
        if (++stage == p.stages) stage = 0;
    }
    if (!p.want_w && !p.want_b) return;
    cp_async_wait<0>();
    float *joined = sw + (p.weight_bytes >> 2);        // [2][cols], groups > 1
    for (int gr = 0; gr < p.groups; gr++) {
        if (p.groups > 1) __syncthreads();             // the first one: the ring is done with
        if (group != gr) continue;
        float *to = gr + 1 < p.groups ? joined : p.part + (int64_t)blockIdx.x * 2 * p.cols;
#pragma unroll
        for (int i = 0; i < N; i++) {
            if (!in(i)) continue;
            float w[2 * H], b[2 * H];
#pragma unroll
            for (int j = 0; j < H; j++) {
                unpack2(dw[i][j], w[2 * j], w[2 * j + 1]);
                if (FULL) unpack2(db[i][j], b[2 * j], b[2 * j + 1]);
            }
#pragma unroll
            for (int j = 0; j < (VEC > 1 ? VEC : 2); j++) {
                if (VEC == 1 && j && !in2(i)) continue;
                const int k = c + i * STEP + (VEC > 1 ? j : 32 * j);
                to[k] = gr ? joined[k] + w[j] : w[j];
                if (FULL) to[p.cols + k] = gr ? joined[p.cols + k] + b[j] : b[j];
            }
        }
    }
}

// dw and db: the CTAs' parts, 32 columns a CTA: warp k adds parts k, k + 32, ...
// of its lanes' columns, then the 32 warps' sums of column k (a fixed tree).
// blockIdx.y: dw, then db.
__global__ void __launch_bounds__(1024) reduce_kernel(const float *__restrict__ part, int parts, int cols, float *dw,
                                                      float *db)
{
    __shared__ float run[32][33];
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float *out = blockIdx.y || !dw ? db : dw;
    const float *from = part + (out == db ? cols : 0);
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 5
        for (int i = k; i < parts; i += 32) s += __ldg(from + (int64_t)i * 2 * cols + c);
    }
    run[k][lane] = s;
    __syncthreads();
    s = run[lane][k];
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane == 0 && (int)blockIdx.x * 32 + k < cols) out[blockIdx.x * 32 + k] = s;
}

// ------------------------------------------------------------------- host

static int64_t span(int64_t rows, int64_t ld, int64_t cols, int es) { return ((rows - 1) * ld + cols) * es; }

static bool aligned4(std::initializer_list<const void *> ps)
{
    uintptr_t bits = 0;
    for (const void *p : ps) bits |= reinterpret_cast<uintptr_t>(p);
    return bits % 4 == 0;
}

// whether the rows of an output (elements es wide) lie over an input's other
// than row on row: a row would be written before another is read
static bool clash(const void *out, int64_t ld_out, const void *in, int64_t ld_in, int64_t rows, int cols, int es)
{
    if (!overlap(out, span(rows, ld_out, cols, es), in, span(rows, ld_in, cols, es))) return false;
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

template <typename T, int VEC, int EPT, bool RING>
static cudaError_t fwd_launch(const Fwd &p, unsigned grid, int smem, cudaStream_t st)
{
    if (RING) {
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = allow_smem(reinterpret_cast<const void *>(norm_kernel<T, VEC, EPT, RING>), EPT == 16 ? SMEM_MAX / 2 : SMEM_MAX, done);
        if (e != cudaSuccess) return e;
    }
    norm_kernel<T, VEC, EPT, RING><<<grid, p.warps * p.groups * 32, smem, st>>>(p);
    return cudaGetLastError();
}

// The forward's plan.  Few rows (one a CTA and SM at most): 8 values a thread,
// read straight to registers, for a row's latency.  Else a ring: 16 values a
// thread, two CTAs an SM; 32 where a CTA would not hold the row else, and one
// CTA.  Groups as many as 512 threads hold, up to four stages each.
template <typename T, int VEC>
static cudaError_t fwd_plan(Fwd &p, cudaStream_t st)
{
    const int sms = sm_count(), es = sizeof(T);
    const int ept = p.cols > 8192 ? 32 : p.rows <= sms ? 8 : 16;
    p.warps = (p.cols + 32 * ept - 1) / (32 * ept);
    p.wide = p.warps * 32 * ept;
    p.groups = 1;
    p.stages = p.stage_bytes = 0;
    if (ept == 8) return fwd_launch<T, VEC, 8, false>(p, (unsigned)p.rows, 0, st);
    p.weight_bytes = p.wide * 4 * (p.b ? 2 : 1);
    const int per_sm = ept == 16 ? 2 : 1, room = SMEM_MAX / per_sm - p.weight_bytes;
    const int64_t each = (p.rows + sms * per_sm - 1) / (sms * per_sm);
    int groups = 16 / p.warps;
    if (groups > 8 && p.warps > 1) groups = 8;         // named barriers
    if (groups > each) groups = (int)each;
    p.stage_bytes = p.wide * es + (VEC == 1 ? 32 : 0);
    while (groups > 1 && 2 * groups * p.stage_bytes > room) groups--;
    p.groups = groups;
    p.stages = room / (groups * p.stage_bytes);
    if (p.stages > 4) p.stages = 4;
    const int64_t want = (p.rows + groups - 1) / groups;
    const unsigned grid = (unsigned)(want < (int64_t)sms * per_sm ? want : (int64_t)sms * per_sm);
    const int smem = p.weight_bytes + groups * p.stages * p.stage_bytes;
    return ept == 16 ? fwd_launch<T, VEC, 16, true>(p, grid, smem, st) : fwd_launch<T, VEC, 32, true>(p, grid, smem, st);
}

template <typename T, int VEC, int EPT, bool CKPT, bool FULL, int ADD>
static cudaError_t bwd_launch_add(const Bwd &p, int grid, int smem, cudaStream_t st)
{
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(dnorm_kernel<T, VEC, EPT, CKPT, FULL, ADD>), SMEM_MAX, done);
    if (e != cudaSuccess) return e;
    dnorm_kernel<T, VEC, EPT, CKPT, FULL, ADD><<<grid, p.warps * p.groups * 32, smem, st>>>(p);
    return cudaGetLastError();
}

template <typename T, int VEC, int EPT, bool CKPT, bool FULL>
static cudaError_t bwd_launch(const Bwd &p, int grid, int smem, cudaStream_t st)
{
    if (!p.dy_add && !p.dx_add) return bwd_launch_add<T, VEC, EPT, CKPT, FULL, 0>(p, grid, smem, st);
    if (EPT == 16 || !p.dy_add || p.at_dya >= 0) return bwd_launch_add<T, VEC, EPT, CKPT, FULL, 1>(p, grid, smem, st);
    return bwd_launch_add<T, VEC, EPT, CKPT, FULL, EPT == 16 ? 1 : 2>(p, grid, smem, st);       // 16 a thread: always room
}

template <typename T, int VEC, int EPT, bool CKPT>
static cudaError_t bwd_launch_bias(const Bwd &p, int grid, int smem, cudaStream_t st)
{
    return p.want_b || p.center ? bwd_launch<T, VEC, EPT, CKPT, true>(p, grid, smem, st) : bwd_launch<T, VEC, EPT, CKPT, false>(p, grid, smem, st);
}

template <typename T, int VEC>
static cudaError_t bwd_launch_for(const Bwd &p, int ept, int grid, int smem, cudaStream_t st)
{
    if constexpr (VEC > 1) {
        if (p.h_q)
            return ept == 16 ? bwd_launch_bias<T, VEC, 16, true>(p, grid, smem, st) : bwd_launch_bias<T, VEC, 32, true>(p, grid, smem, st);
    }
    return ept == 16 ? bwd_launch_bias<T, VEC, 16, false>(p, grid, smem, st) : bwd_launch_bias<T, VEC, 32, false>(p, grid, smem, st);
}

// The backward's plan: 16 values a thread (32 where a row has more than 512
// threads would hold), as many groups a CTA as its threads allow (fewer where
// rows are few, so that they spread over the SMs, and where each would not
// have two stages), up to four stages; dy_add is read in place where a row
// with it does not fit at all.
static int bwd_plan(Bwd &p, bool vec, int es, int &ept, int &smem)
{
    ept = p.cols > 8192 ? 32 : 16;
    p.warps = (p.cols + 32 * ept - 1) / (32 * ept);
    p.wide = p.warps * 32 * ept;
    int groups = BWD_THREADS / 32 / p.warps;
    const int64_t per_sm = ((int64_t)p.rows + sm_count() - 1) / sm_count();
    if (groups > 8) groups = 8;                        // named barriers, and the parts joined one after another
    if (groups > per_sm) groups = (int)per_sm;
    const auto lay = [&](bool dya) {
        const int row = p.wide * es + (vec ? 0 : 32);
        int n = row;
        p.at_x = n;
        n += p.h_q ? p.wide : row;
        p.at_s = n;
        if (p.h_q) n = (n + p.wide / 128 * 4 + 15) & ~15;
        p.at_dya = dya ? n : -1;
        if (dya) n += p.wide * 4 + (vec ? 0 : 32);
        p.stage_bytes = n;
    };
    p.weight_bytes = p.wide * 4;
    const int room = SMEM_MAX - p.weight_bytes;
    lay(p.dy_add != nullptr);
    if (p.stage_bytes > room) lay(false);
    while (groups > 1 && 2 * groups * p.stage_bytes > room) groups--;
    p.stages = room / (groups * p.stage_bytes);
    if (p.stages > 4) p.stages = 4;
    p.groups = groups;
    const int ring = groups * p.stages * p.stage_bytes, join = groups > 1 ? 2 * p.cols * (int)sizeof(float) : 0;
    smem = p.weight_bytes + (ring > join ? ring : join);
    return bwd_ctas(p.rows, groups);
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
    if (!aligned4({mean, rstd, y_s, xhat_s})) return MOE_ERR_ALIGN;
    const Span in_x{x, span(rows, ld_x, cols, es)}, in_w{weight, cols * ws}, in_b{bias, cols * ws};
    const int64_t codes = rows * cols, scales = rows * (cols / 128) * 4;
    const Span out_y{y, span(rows, ld_y, cols, es)};
    const Span outs[] = {{mean, rows * 4}, {rstd, rows * 4}, {y_q, codes}, {y_s, scales}, {xhat_q, codes}, {xhat_s, scales}};
    if (clash(y, ld_y, x, ld_x, rows, (int)cols, es) || overlap_any({out_y}, {in_w, in_b}) ||
        overlap_any(outs, {in_x, in_w, in_b, out_y}) || overlap_each(outs))
        return MOE_ERR_UNSUPPORTED;
    Fwd p{x, weight, bias, y, mean, rstd, y_q, xhat_q, y_s, xhat_s, rows, ld_x, ld_y, (int)cols, 0, 1, 1, 0, 0, 0, eps,
          center != 0, w_dtype == MOE_TYPE_F32};
    cudaStream_t st = as_stream(stream);
    const cudaError_t e = f32 ? (vec ? fwd_plan<float, 4>(p, st) : fwd_plan<float, 1>(p, st))
                              : (vec ? fwd_plan<uint16_t, 8>(p, st) : fwd_plan<uint16_t, 1>(p, st));
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
    if (!aligned4({mean, rstd, xhat_s, dweight, dbias})) return MOE_ERR_ALIGN;
    if (clash(dx, ld_dx, dy, ld_dy, rows, (int)cols, es) || clash(dx, ld_dx, x, ld_x, rows, (int)cols, es) ||
        clash(dx, ld_dx, dx_add, ld_add, rows, (int)cols, es) ||
        overlap_any({{dx, span(rows, ld_dx, cols, es)}}, {{dy_add, rows * cols * 4}, {xhat_q, rows * cols}}))
        return MOE_ERR_UNSUPPORTED;
    const bool sums = dweight || dbias;
    if (sums && (!workspace || workspace_bytes < moe_layer_norm_backward_workspace_size(rows, cols)))
        return MOE_ERR_WORKSPACE;
    if (sums && !aligned16(workspace)) return MOE_ERR_ALIGN;
    if (!sums && !dx) return MOE_OK;
    const Span sums_w{dweight, cols * 4}, sums_b{dbias, cols * 4},
        parts{sums ? workspace : nullptr, (int64_t)moe_layer_norm_backward_workspace_size(rows, cols)},
        in_w{weight, cols * ws}, in_m{center && x ? mean : nullptr, rows * 4}, in_r{rstd, rows * 4},
        in_s{xhat_s, rows * (cols / 128) * 4};
    const Span outs[] = {{dx, span(rows, ld_dx, cols, es)}, sums_w, sums_b, parts};
    if (overlap_each(outs) || overlap_any(outs, {in_w, in_m, in_r, in_s}) ||
        overlap_any({sums_w, sums_b, parts}, {{dy, span(rows, ld_dy, cols, es)}, {x, span(rows, ld_x, cols, es)},
                    {dx_add, span(rows, ld_add, cols, es)}, {dy_add, rows * cols * 4}, {xhat_q, rows * cols}}))
        return MOE_ERR_UNSUPPORTED;
    Bwd p{dy, x, dx_add, weight, dy_add, xhat_q, xhat_s, mean, rstd, dx, static_cast<float *>(workspace),
          ld_dy, ld_x, ld_add, ld_dx, (int)rows, (int)cols, 0, 1, 1, 0, 0, 0, 0, 0, 0, center != 0, w_dtype == MOE_TYPE_F32,
          dweight != nullptr, dbias != nullptr};
    int ept, smem;
    const int grid = bwd_plan(p, vec, es, ept, smem);
    const cudaError_t e = f32 ? (vec ? bwd_launch_for<float, 4>(p, ept, grid, smem, st) : bwd_launch_for<float, 1>(p, ept, grid, smem, st))
                              : (vec ? bwd_launch_for<uint16_t, 8>(p, ept, grid, smem, st) : bwd_launch_for<uint16_t, 1>(p, ept, grid, smem, st));
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    if (!sums) return MOE_OK;
    reduce_kernel<<<dim3((unsigned)((cols + 31) / 32), dweight && dbias ? 2 : 1), 1024, 0, st>>>(p.part, grid, (int)cols,
                                                                                               dweight, dbias);
    return launch_status();
}
