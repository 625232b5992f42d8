// ckpt.cu -- the SwiGLU backward from pre-activations kept in 8 bits.
//
// GEMM1's pre-activations h are the largest thing a layer keeps from forward
// to backward; moe_grouped_ffn_fp8_ckpt keeps them as 1 x 128 E4M3 codes and
// fp32 scales (2.06 bytes a pair of gate and up, where fp32 takes 8).  This
// file reads them back.  Per element, with g = code * scale, u likewise,
// a = d_act and sg = 1 / (1 + e^-g):
//   d_up = a g sg,  d_gate = a u (sg + g sg (1 - sg)),  act = g sg u,
// and everything the gradient products read leaves in one pass over h and
// d_act: dh in 1 x 128 codes along 2F (the dgrad operand), dh and act in
// 128 x 1 codes along the expert's rows, channel-major (the weight gradients'
// operands), and <d_act, act>, which over the gate is the gate's gradient:
// d_act = W2^T (gate dy), so <d_act, act> = gate <dy, W2 act>.
#include "losses.cuh"

namespace moe {
namespace ckpt {

struct Args {
    const uint16_t *d_act;      // [rows, F] bf16
    const uint8_t *h_q;         // [rows, 2F]
    const float *h_s;           // [rows, 2F / 128]
    const int32_t *offsets, *pad;
    uint8_t *dh_q, *dhT_q, *actT_q;
    float *dh_s, *dhT_s, *actT_s;
    float *dots;                // [rows, F / 128]: <d_act, act> over each block of columns
    int64_t rows, ld;
    int F, E;
};

constexpr int TILE = 128;       // rows and columns of a tile
constexpr int WARPS = 8;        // each with 16 of the rows; a lane four columns
constexpr int RW = TILE / WARPS;

// 2^64 brings the reciprocal of a subnormal scale into range
constexpr float LIFT = 0x1p64f;

// A block scale's reciprocal; `lift` says that the values are multiplied by
// LIFT first.  A code is E4M3(v RN(1 / s)), as the act codes of GEMM1.
__device__ __forceinline__ float recip(float s, bool &lift)
{
    lift = s < 0x1p-126f;
    return __frcp_rn(lift ? s * LIFT : s);
}

// four codes (value 0 in the low byte), two at a time to fp32, times the scale
__device__ __forceinline__ void decode4(uint32_t q, uint64_t s2, uint64_t (&v)[2])
{
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(q >> (16 * i)), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        v[i] = mul2(pack2(f.x, f.y), s2);
    }
}

// one row's four columns: a (bf16), gate and up codes -> d_gate, d_up, act,
// two columns in each 64-bit pair
__device__ __forceinline__ void swiglu4(uint2 a, uint32_t gq, uint32_t uq, float gs, float us, uint64_t (&dg)[2],
                                        uint64_t (&du)[2], uint64_t (&act)[2])
{
    uint64_t g[2], u[2];
    decode4(gq, pack2(gs, gs), g);
    decode4(uq, pack2(us, us), u);
    const uint32_t aw[2] = {a.x, a.y};
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint64_t a2 = pack2(__uint_as_float(aw[i] << 16), __uint_as_float(aw[i] & 0xFFFF0000u));
        float t0, t1;
        unpack2(mul2(g[i], pack2(-LOG2E, -LOG2E)), t0, t1);
        unpack2(add2(pack2(ex2(t0), ex2(t1)), pack2(1.0f, 1.0f)), t0, t1);
        const uint64_t sg = pack2(rcp(t0), rcp(t1));
        const uint64_t p = mul2(g[i], sg);                                    // silu
        const uint64_t rest = fma2(sg, pack2(-1.0f, -1.0f), pack2(1.0f, 1.0f));
        du[i] = mul2(a2, p);
        dg[i] = mul2(mul2(a2, u[i]), fma2(p, rest, sg));
        act[i] = mul2(p, u[i]);
    }
}

__device__ __forceinline__ float amax4(const uint64_t (&v)[2])
{
    float a, b, c, d;
    unpack2(v[0], a, b);
    unpack2(v[1], c, d);
    return fmaxf(fmaxf(fabsf(a), fabsf(b)), fmaxf(fabsf(c), fabsf(d)));
}

// the warp's largest of non-negative numbers (their bits order as integers do)
__device__ __forceinline__ float warp_max(float v)
{
    return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v)));
}

__device__ __forceinline__ uint32_t encode4(const uint64_t (&v)[2], float y, bool lift)
{
    float f[4];
    unpack2(mul2(v[0], pack2(lift ? LIFT : 1.0f, lift ? LIFT : 1.0f)), f[0], f[1]);
    unpack2(mul2(v[1], pack2(lift ? LIFT : 1.0f, lift ? LIFT : 1.0f)), f[2], f[3]);
    return (uint32_t)pack_e4m3x2(f[0] * y, f[1] * y) | ((uint32_t)pack_e4m3x2(f[2] * y, f[3] * y) << 16);
}

// shared memory of the column side: the codes of 3 x 128 channels, 128 rows each
constexpr int CODES = 3 * TILE * TILE;
constexpr int SMEM_COL = CODES + 3 * TILE * 2 * (int)sizeof(float);

// One 128 x 128 tile of (rows, columns of F): with COL the rows of one padded
// 128-row block of an expert, else any 128 rows.  Lane l of warp w holds
// columns 4 l .. 4 l + 3 of rows 16 w .. 16 w + 15 as they came from memory
// (one 32-bit register a pair of gate and up with its d_act), so the two
// passes over them (largest values, then codes) recompute rather than keep
// three fp32 numbers each.  A row's largest value is one warp reduction; its
// scales are formed by one lane each.  The columns' largest values go through
// shared memory.  A lane's sixteen codes of a channel are the 16-byte piece w
// of its row of the code tile (at piece w ^ (l & 7): no bank conflicts either
// way), and a channel leaves as one 128-byte run.
template <bool ROW, bool COL>
__global__ void __launch_bounds__(WARPS * 32, 2) swiglu_ckpt_kernel(Args p)
{
    extern __shared__ __align__(16) uint8_t sm[];
    float *red = reinterpret_cast<float *>(sm);                   // [WARPS][3][TILE], before the codes take its place
    float *col_y = reinterpret_cast<float *>(sm + CODES);         // [3][TILE] reciprocals, then which are lifted
    __shared__ int64_t s_r0, s_rend;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nb = p.F >> 7;
    const int64_t kb = blockIdx.x / nb;
    const int cb = blockIdx.x - (int)kb * nb;
    int64_t r0 = kb * TILE, rend = p.rows;
    if (COL) {
        if (kb * TILE >= p.pad[p.E] || kb * TILE >= p.ld) return;
        if (threadIdx.x == 0) s_r0 = s_rend = 0;
        __syncthreads();
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
            const int32_t p0 = __ldg(p.pad + e), p1 = __ldg(p.pad + e + 1);
            if (p0 <= kb * TILE && kb * TILE < p1) {
                s_r0 = __ldg(p.offsets + e) + (kb * TILE - p0);
                s_rend = __ldg(p.offsets + e + 1);
            }
        }
        __syncthreads();
        r0 = s_r0;
        rend = s_rend < p.rows ? s_rend : p.rows;
        if (r0 < 0) rend = 0;
    }
    const int64_t row0 = r0 + warp * RW;
    const int c0 = 4 * lane;
    uint2 a[RW];
    uint32_t gq[RW], uq[RW];
#pragma unroll
    for (int i = 0; i < RW; i++) {
        const int64_t r = row0 + i;
        a[i] = make_uint2(0u, 0u);
        gq[i] = uq[i] = 0u;
        if (r < rend) {
            a[i] = __ldcs(reinterpret_cast<const uint2 *>(p.d_act + r * p.F + cb * TILE + c0));
            gq[i] = __ldcs(reinterpret_cast<const uint32_t *>(p.h_q + r * 2 * p.F + cb * TILE + c0));
            uq[i] = __ldcs(reinterpret_cast<const uint32_t *>(p.h_q + r * 2 * p.F + p.F + cb * TILE + c0));
        }
    }
    // lane 2 i + 0 / 1 holds row i's gate / up scale
    float hs = 0.0f;
    if (row0 + (lane >> 1) < rend) hs = __ldg(p.h_s + (row0 + (lane >> 1)) * 2 * nb + (lane & 1) * nb + cb);

    float cm[3][4] = {};                                          // the lane's columns: largest d_gate, d_up, act
    float rm = 0.0f, dot = 0.0f;                                  // lane 2 i + 0 / 1: row i's largest d_gate / d_up; lane i: its dot
#pragma unroll
    for (int i = 0; i < RW; i++) {
        uint64_t dg[2], du[2], act[2];
        swiglu4(a[i], gq[i], uq[i], __shfl_sync(0xFFFFFFFFu, hs, 2 * i), __shfl_sync(0xFFFFFFFFu, hs, 2 * i + 1), dg,
                du, act);
        if (ROW) {
            const float mg = warp_max(amax4(dg)), mu = warp_max(amax4(du));
            if ((lane >> 1) == i) rm = lane & 1 ? mu : mg;
        }
        if (COL) {
#pragma unroll
            for (int j = 0; j < 2; j++) {
                float x, y;
                unpack2(dg[j], x, y);
                cm[0][2 * j] = fmaxf(cm[0][2 * j], fabsf(x));
                cm[0][2 * j + 1] = fmaxf(cm[0][2 * j + 1], fabsf(y));
                unpack2(du[j], x, y);
                cm[1][2 * j] = fmaxf(cm[1][2 * j], fabsf(x));
                cm[1][2 * j + 1] = fmaxf(cm[1][2 * j + 1], fabsf(y));
                unpack2(act[j], x, y);
                cm[2][2 * j] = fmaxf(cm[2][2 * j], fabsf(x));
                cm[2][2 * j + 1] = fmaxf(cm[2][2 * j + 1], fabsf(y));
            }
        }
        if (p.dots) {
            const float a0 = __uint_as_float(a[i].x << 16), a1 = __uint_as_float(a[i].x & 0xFFFF0000u);
            const float a2 = __uint_as_float(a[i].y << 16), a3 = __uint_as_float(a[i].y & 0xFFFF0000u);
            float x, y, z, w;
            unpack2(act[0], x, y);
            unpack2(act[1], z, w);
            float s = fmaf(a0, x, a1 * y) + fmaf(a2, z, a3 * w);
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
            if (lane == i) dot = s;
        }
    }
    if (p.dots && lane < RW && row0 + lane < rend) p.dots[(row0 + lane) * nb + cb] = dot;
    float ry = 0.0f;
    bool rlift = false;
    if (ROW) {
        const float s = block_scale(rm);
        ry = recip(s, rlift);
        if (row0 + (lane >> 1) < rend) p.dh_s[(row0 + (lane >> 1)) * 2 * nb + (lane & 1) * nb + cb] = s;
    }
    const unsigned rl = __ballot_sync(0xFFFFFFFFu, rlift);
    float cy[3][4];
    unsigned cl = 0;
    if (COL) {
#pragma unroll
        for (int k = 0; k < 3; k++)
            *reinterpret_cast<float4 *>(red + (warp * 3 + k) * TILE + c0) = make_float4(cm[k][0], cm[k][1], cm[k][2], cm[k][3]);
        __syncthreads();
        for (int c = threadIdx.x; c < 3 * TILE; c += WARPS * 32) {
            float m = red[c];
#pragma unroll
            for (int w = 1; w < WARPS; w++) m = fmaxf(m, red[w * 3 * TILE + c]);
            const float s = block_scale(m);
            bool lift;
            col_y[c] = recip(s, lift);
            col_y[3 * TILE + c] = lift ? 1.0f : 0.0f;
            const int k = c >> 7, ch = cb * TILE + (c & 127);
            if (k == 2) {
                if (p.actT_s) p.actT_s[kb * p.F + ch] = s;
            } else if (p.dhT_s) {
                p.dhT_s[kb * 2 * p.F + k * p.F + ch] = s;
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; k++) {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                cy[k][j] = col_y[k * TILE + c0 + j];
                if (col_y[3 * TILE + k * TILE + c0 + j] != 0.0f) cl |= 1u << (4 * k + j);
            }
        }
    }
    // the second pass starts from what was loaded: without this the compiler
    // keeps the first one's results and spills them
#pragma unroll
    for (int i = 0; i < RW; i++) asm volatile("" : "+r"(a[i].x), "+r"(a[i].y), "+r"(gq[i]), "+r"(uq[i]));
    uint32_t words[3][4][RW / 4];
#pragma unroll
    for (int i4 = 0; i4 < RW; i4 += 4) {
        float v[3][4][4];                                          // [array][column][row]
#pragma unroll
        for (int ii = 0; ii < 4; ii++) {
            const int i = i4 + ii;
            uint64_t dg[2], du[2], act[2];
            swiglu4(a[i], gq[i], uq[i], __shfl_sync(0xFFFFFFFFu, hs, 2 * i), __shfl_sync(0xFFFFFFFFu, hs, 2 * i + 1),
                    dg, du, act);
            if (ROW) {
                const float yg = __shfl_sync(0xFFFFFFFFu, ry, 2 * i), yu = __shfl_sync(0xFFFFFFFFu, ry, 2 * i + 1);
                if (row0 + i < rend) {
                    uint8_t *q = p.dh_q + (row0 + i) * 2 * p.F + cb * TILE + c0;
                    *reinterpret_cast<uint32_t *>(q) = encode4(dg, yg, rl >> (2 * i) & 1);
                    *reinterpret_cast<uint32_t *>(q + p.F) = encode4(du, yu, rl >> (2 * i + 1) & 1);
                }
            }
            if (COL) {
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    unpack2(dg[j], v[0][2 * j][ii], v[0][2 * j + 1][ii]);
                    unpack2(du[j], v[1][2 * j][ii], v[1][2 * j + 1][ii]);
                    unpack2(act[j], v[2][2 * j][ii], v[2][2 * j + 1][ii]);
                }
            }
        }
        if (COL) {
#pragma unroll
            for (int k = 0; k < 3; k++) {
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    float *x = v[k][j];
                    if (cl) {
                        const float f = cl >> (4 * k + j) & 1 ? LIFT : 1.0f;
#pragma unroll
                        for (int ii = 0; ii < 4; ii++) x[ii] *= f;
                    }
                    const float y = cy[k][j];
                    words[k][j][i4 / 4] = (uint32_t)pack_e4m3x2(x[0] * y, x[1] * y) |
                                          ((uint32_t)pack_e4m3x2(x[2] * y, x[3] * y) << 16);
                }
            }
        }
    }
    if (!COL) return;
    uint4 *tile = reinterpret_cast<uint4 *>(sm);                   // [3 * TILE channels][8 pieces]
#pragma unroll
    for (int k = 0; k < 3; k++) {
#pragma unroll
        for (int j = 0; j < 4; j++)
            tile[(k * TILE + c0 + j) * 8 + (warp ^ (lane & 7))] =
                make_uint4(words[k][j][0], words[k][j][1], words[k][j][2], words[k][j][3]);
    }
    __syncthreads();
#pragma unroll 4
    for (int u = threadIdx.x; u < 3 * TILE * 8; u += WARPS * 32) {
        const int c = u >> 3, piece = u & 7;
        const int k = c >> 7, cc = c & 127;
        const uint4 w = tile[c * 8 + (piece ^ (cc >> 2 & 7))];
        uint8_t *base = k == 2 ? p.actT_q : p.dhT_q;
        if (base)
            *reinterpret_cast<uint4 *>(base + ((int64_t)(k & 1) * p.F + cb * TILE + cc) * p.ld + kb * TILE + 16 * piece) = w;
    }
}

// d_gates[slot]: the blocks' dots of the slot's row in order, over its gate; 0
// for a slot without a row and for a gate of 0 (its row of d_act holds
// nothing, and every gate function's slope is 0 there)
__global__ void __launch_bounds__(256) gate_kernel(const float *__restrict__ dots, const float *__restrict__ gates,
                                                   const int32_t *__restrict__ slot_to_sorted, int64_t slots,
                                                   int64_t rows, const int32_t *__restrict__ routed, int nb,
                                                   float *__restrict__ d_gates)
{
    if (routed && __ldg(routed) < rows) rows = __ldg(routed);      // expert_offsets[E]
    const int64_t p = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
    if (p >= slots) return;
    const int32_t r = __ldg(slot_to_sorted + p);
    const float g = __ldg(gates + p);
    float s = 0.0f;
    if (r >= 0 && r < rows && g != 0.0f) {
        for (int b = 0; b < nb; b++) s += __ldg(dots + (int64_t)r * nb + b);
        s = __fdiv_rn(s, g);
    }
    d_gates[p] = s;
}

template <bool ROW, bool COL>
static cudaError_t launch(const Args &p, int64_t blocks, cudaStream_t st)
{
    constexpr int smem = COL ? SMEM_COL : 0;
    if (COL) {
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = allow_smem(reinterpret_cast<const void *>(swiglu_ckpt_kernel<ROW, COL>), smem, done);
        if (e != cudaSuccess) return e;
    }
    swiglu_ckpt_kernel<ROW, COL><<<(unsigned)(blocks * (p.F / TILE)), WARPS * 32, smem, st>>>(p);
    return cudaGetLastError();
}

} // namespace ckpt
} // namespace moe

using namespace moe;
using namespace moe::ckpt;

MOE_API size_t moe_swiglu_backward_ckpt_workspace_size(int64_t rows, int F)
{
    if (rows < 0 || F <= 0) return 0;
    return (size_t)rows * (F / 128) * sizeof(float);
}

MOE_API moe_status moe_swiglu_backward_ckpt(const uint16_t *d_act, const uint8_t *h_q, const float *h_s, int64_t rows,
                                            int F, const float *gates, const int32_t *slot_to_sorted, int64_t slots,
                                            uint8_t *dh_q, float *dh_s, float *d_gates, const int32_t *expert_offsets,
                                            const int32_t *pad, int E, int64_t max_pad, uint8_t *dhT_q, float *dhT_s,
                                            uint8_t *actT_q, float *actT_s, void *workspace, size_t workspace_bytes,
                                            void *stream)
{
    const bool col = dhT_q || dhT_s || actT_q || actT_s;
    if (rows < 0 || rows >= (1LL << 31) || F <= 0 || F % 128 != 0 || slots < 0 || slots >= (1LL << 31)) return MOE_ERR_SHAPE;
    if (col && (E < 1 || E > 1024 || max_pad < 0 || max_pad % 128 != 0)) return MOE_ERR_SHAPE;
    if ((col ? max_pad / 128 : (rows + 127) / 128) * (F / 128) >= (1LL << 31)) return MOE_ERR_SHAPE;
    if (!dh_q != !dh_s || !dhT_q != !dhT_s || !actT_q != !actT_s) return MOE_ERR_NULL;
    if (col && (!expert_offsets || !pad)) return MOE_ERR_NULL;
    if (d_gates && slots && (!gates || !slot_to_sorted)) return MOE_ERR_NULL;
    if (rows && (dh_q || col || d_gates) && (!d_act || !h_q || !h_s)) return MOE_ERR_NULL;
    if (!aligned16(d_act) || !aligned16(h_q) || !aligned16(dh_q) || !aligned16(dhT_q) || !aligned16(actT_q))
        return MOE_ERR_ALIGN;
    if (!dh_q && !col && !(d_gates && slots)) return MOE_OK;
    const bool dots = d_gates && slots && rows;
    if (dots && (!workspace || workspace_bytes < moe_swiglu_backward_ckpt_workspace_size(rows, F))) return MOE_ERR_WORKSPACE;
    if (dots && !aligned16(workspace)) return MOE_ERR_ALIGN;
    cudaStream_t st = as_stream(stream);
    float *ws = dots ? static_cast<float *>(workspace) : nullptr;
    Args p{d_act, h_q, h_s, expert_offsets, pad, dh_q, dhT_q, actT_q, dh_s, dhT_s, actT_s, ws, rows, max_pad, F, E};
    const int64_t blocks = col ? max_pad / 128 : (rows + 127) / 128;
    if (blocks && (dh_q || col || dots)) {
        const cudaError_t e = dh_q ? (col ? launch<true, true>(p, blocks, st) : launch<true, false>(p, blocks, st))
                                   : (col ? launch<false, true>(p, blocks, st) : launch<false, false>(p, blocks, st));
        if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
    if (d_gates && slots)
        gate_kernel<<<(unsigned)((slots + 255) / 256), 256, 0, st>>>(ws, gates, slot_to_sorted, slots, rows,
                                                                    col ? expert_offsets + E : nullptr, F / 128, d_gates);
    else if (!blocks)
        return MOE_OK;
    return launch_status();
}
