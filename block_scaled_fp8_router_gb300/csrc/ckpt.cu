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
#include <type_traits>

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
    int64_t rows;
    int ld, F, E;
};

constexpr int TILE = 128;       // rows and columns of a tile
constexpr int WARPS = 16;       // each with eight of the rows; a lane four columns
constexpr int RW = TILE / WARPS;
constexpr int THREADS = WARPS * 32;
constexpr int MAX_E = 1024;

// One row's four columns: a (bf16), gate and up codes -> d_gate, d_up, act,
// two columns in each 64-bit pair, and a act summed into dot.  g below is
// minus the gate, and the reciprocal gives -sg, so that silu p = (-g)(-sg)
// takes no sign, and p - p sg comes out of one fused multiply-add, exact where
// sg is next to 1.
__device__ __forceinline__ void swiglu4(uint2 a, uint32_t gq, uint32_t uq, float gs, float us, uint64_t (&dg)[2],
                                        uint64_t (&du)[2], uint64_t (&act)[2], uint64_t &dot)
{
    float gc[4], uc[4];
    e4m3x4_unpack(gq, gc);
    e4m3x4_unpack(uq, uc);
    const uint32_t aw[2] = {a.x, a.y};
    const uint64_t gs2 = pack2(-gs, -gs), us2 = pack2(us, us);
    dot = 0;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint64_t g = mul2(pack2(gc[2 * i], gc[2 * i + 1]), gs2), u = mul2(pack2(uc[2 * i], uc[2 * i + 1]), us2);
        const uint64_t a2 = pack2(__uint_as_float(aw[i] << 16), __uint_as_float(aw[i] & 0xFFFF0000u));
        float t0, t1;
        unpack2(g, t0, t1);
        const uint64_t nsg = pack2(rcp(-1.0f - ex2(t0 * LOG2E)), rcp(-1.0f - ex2(t1 * LOG2E)));
        const uint64_t p = mul2(g, nsg);                                      // silu
        du[i] = mul2(a2, p);
        dg[i] = mul2(mul2(a2, u), sub2(fma2(p, nsg, p), nsg));
        act[i] = mul2(p, u);
        dot = fma2(a2, act[i], dot);
    }
}

__device__ __forceinline__ float amax4(const uint64_t (&v)[2])
{
    float a, b, c, d;
    unpack2(v[0], a, b);
    unpack2(v[1], c, d);
    return amax3(amax3(a, b, c), d, 0.0f);
}

// the warp's largest of non-negative numbers (their bits order as integers do)
__device__ __forceinline__ float warp_max(float v)
{
    return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v)));
}

// products by pairs beside the columns' codes (65536 x 2048: 313 us against
// 315), one by one without them (145 against 151)
template <bool PAIRS>
__device__ __forceinline__ uint32_t encode4(const uint64_t (&v)[2], float y)
{
    float a, b, c, d;
    if (PAIRS) {
        const uint64_t y2 = pack2(y, y);
        unpack2(mul2(v[0], y2), a, b);
        unpack2(mul2(v[1], y2), c, d);
        return e4m3x4_pack(a, b, c, d);
    }
    unpack2(v[0], a, b);
    unpack2(v[1], c, d);
    return e4m3x4_pack(a * y, b * y, c * y, d * y);
}

// eight sums of a warp's lanes, sum i left in every lane with lane / 4 = i:
// each step keeps half of the sums
__device__ __forceinline__ float sums8(const float (&v)[8], int lane)
{
    float a[4], b[2], c;
    const bool h4 = lane & 16, h3 = lane & 8, h2 = lane & 4;
#pragma unroll
    for (int i = 0; i < 4; i++)
        a[i] = (h4 ? v[4 + i] : v[i]) + __shfl_xor_sync(0xFFFFFFFFu, h4 ? v[i] : v[4 + i], 16);
#pragma unroll
    for (int i = 0; i < 2; i++)
        b[i] = (h3 ? a[2 + i] : a[i]) + __shfl_xor_sync(0xFFFFFFFFu, h3 ? a[i] : a[2 + i], 8);
    c = (h2 ? b[1] : b[0]) + __shfl_xor_sync(0xFFFFFFFFu, h2 ? b[0] : b[1], 4);
    c += __shfl_xor_sync(0xFFFFFFFFu, c, 2);
    return c + __shfl_xor_sync(0xFFFFFFFFu, c, 1);
}

// sixteen / four bytes to shared memory, asynchronously; `in` false: zeros, and
// nothing is read
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool in)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}

// shared memory: two stages of a tile as it comes from memory (a row's 128
// columns of d_act, gate codes and up codes are 512 bytes; then each warp's
// scales), then for the column side the codes of 3 x 128 channels of 128 rows,
// the warps' largest values of a channel, the reciprocals, and the experts'
// maps
constexpr int ROW_BYTES = 4 * TILE;
constexpr int SCALES = TILE * ROW_BYTES;
constexpr int STAGE = SCALES + TILE * 8;
constexpr int CODES = 3 * TILE * TILE;
constexpr int RED = WARPS * 3 * TILE * 4;
constexpr int SMEM_ROW = 2 * STAGE;
constexpr int SMEM_COL = 2 * STAGE + CODES + RED + 3 * TILE * 4 + 2 * (MAX_E + 1) * 4;
static_assert(SMEM_COL <= 227 * 1024, "shared memory of a tile");

// The rows of padded block kb: the first one, and the end of those that are
// there (not behind it where there are none): those of the expert with
// pad[e] <= 128 kb < pad[e + 1]
struct Rows {
    int64_t first, end;
};
__device__ __forceinline__ Rows block_rows(const int32_t *pad, const int32_t *off, int E, int64_t kb, int64_t rows)
{
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pad[mid] <= kb * TILE) lo = mid;
        else hi = mid;
    }
    const int64_t in = kb * TILE - pad[lo];                    // the block's place among the expert's rows
    const int64_t first = off[lo] + in;
    const int64_t end = off[lo + 1] < rows ? off[lo + 1] : rows;
    return {first, in < 0 || first < 0 ? first : end};         // in front of the expert's rows, or of all rows: empty
}

// the blocks that the maps name (no more than E experts of these rows or ld can have); those behind ld give their
// rows' outputs only
__device__ __forceinline__ int blocks_named(int P, int E, int64_t rows, int ld)
{
    const int most = max((int)((rows + TILE - 1) / TILE) + E, ld / TILE);
    return P <= 0 ? 0 : min(P / TILE, most);
}

struct Where {
    int kb, cb;                 // the tile
    int row;                    // the warp's first row
    int n;                      // how many of its eight are there
};

// Tiles of 128 rows x 128 columns of F, a contiguous run of them for each CTA
// (one per SM): with COL the rows of a tile are a padded 128-row block of one
// expert, else any 128 rows.  Warp w has rows 8 w .. 8 w + 7; it copies them
// asynchronously two tiles ahead into shared memory of its own (a row is one
// instruction: lanes 0-15 its d_act, 16-23 its gate and 24-31 its up codes,
// whose rows are all 2 F bytes apart).  Lane l takes columns 4 l .. 4 l + 3
// and holds their d_gate, d_up and act in registers from there on (96 of
// them; 65536 x 2048 of 256 experts: 316 us, where two passes that each
// recomputed them from the codes took 598).  A row's largest
// value is one warp reduction, its scale is formed by one lane.  The columns'
// largest values meet in shared memory.  A lane's eight codes of a channel
// are an 8-byte piece of the channel's row of the code tile (piece w at
// w ^ (l & 15): no bank conflicts either way); a channel leaves as one
// 128-byte run.
// With COL neither memory nor issue is full (47% and 59%): the sixteen warps
// go in step between two barriers a tile and wait together; 316 us of 196 that
// the bytes need (the five codes a pair alone take 15 clocks of a scheduler's
// conversions a warp).  ROW alone 138-143 us = 5.8-6.0 TB/s.
template <bool ROW, bool COL>
__global__ void __launch_bounds__(THREADS, 1) swiglu_ckpt_kernel(Args p)
{
    extern __shared__ __align__(16) uint8_t sm[];
    uint8_t *codes = sm + 2 * STAGE;
    float *red = reinterpret_cast<float *>(codes + CODES);              // [WARPS][3][TILE]
    float *col_y = red + WARPS * 3 * TILE;                              // [3][TILE]
    int32_t *s_pad = reinterpret_cast<int32_t *>(col_y + 3 * TILE), *s_off = s_pad + MAX_E + 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nb = p.F >> 7, c0 = 4 * lane;
    int blocks = (int)((p.rows + TILE - 1) / TILE);
    if (COL) {
        for (int e = tid; e <= p.E; e += THREADS) {
            s_pad[e] = __ldg(p.pad + e);
            s_off[e] = __ldg(p.offsets + e);
        }
        __syncthreads();
        blocks = blocks_named(s_pad[p.E], p.E, p.rows, p.ld);
    }
    // this CTA's tiles: the same number each, the first ones one more
    const int total = blocks * nb, each = total / (int)gridDim.x, more = total - each * (int)gridDim.x;
    const int t0 = (int)blockIdx.x * each + ((int)blockIdx.x < more ? (int)blockIdx.x : more);
    const int t1 = t0 + each + ((int)blockIdx.x < more ? 1 : 0);
    // the warp's rows of a stage; this lane's piece of a row, there and in memory
    const uint32_t stage0 = smem_u32(sm) + warp * RW * ROW_BYTES + lane * 16;
    const uint8_t *piece = lane < 16 ? reinterpret_cast<const uint8_t *>(p.d_act) + lane * 16
                                     : p.h_q + (lane < 24 ? (lane - 16) * 16 : p.F + (lane - 24) * 16);
    const int piece_tile = lane < 16 ? 2 * TILE : TILE;
    const uint32_t scale0 = smem_u32(sm) + SCALES + warp * RW * 8 + lane * 4;

    int f_kb = t0 / nb, f_cb = t0 - f_kb * nb, f_t = t0;               // the tile that is fetched next
    int k_r0 = 0, k_n = 0, k_at = -1;                                  // its block's first row and rows
    auto fetch = [&](int stage) -> Where {
        Where w{f_kb, f_cb, 0, 0};
        if (f_t < t1) {
            if (f_kb != k_at) {
                k_at = f_kb;
                int64_t r0 = (int64_t)f_kb * TILE, rend = p.rows;
                if (COL) {
                    const Rows b = block_rows(s_pad, s_off, p.E, f_kb, p.rows);
                    r0 = b.first, rend = b.end;
                }
                k_n = rend <= r0 ? 0 : rend - r0 < TILE ? (int)(rend - r0) : TILE;
                k_r0 = k_n ? (int)r0 : 0;
            }
            w.row = k_r0 + warp * RW;
            w.n = k_n - warp * RW < RW ? k_n - warp * RW : RW;
            const uint8_t *src = piece + (int64_t)w.row * 2 * p.F + f_cb * piece_tile;
#pragma unroll
            for (int i = 0; i < RW; i++, src += 2 * p.F) copy16(stage0 + stage * STAGE + i * ROW_BYTES, src, i < w.n);
            if (lane < 2 * RW)
                copy4(scale0 + stage * STAGE, p.h_s + (int64_t)(w.row + (lane >> 1)) * 2 * nb + (lane & 1) * nb + f_cb,
                      (lane >> 1) < w.n);
            f_t++;
            if (++f_cb == nb) f_cb = 0, f_kb++;
        }
        cp_async_commit();
        return w;
    };
    // A tile's codes leave while the next tile is at work (no barrier of their
    // own: the next tile's first one has every code in place, its second one
    // every code read).  Sixteen bytes a thread, eight threads a channel, 64
    // channels at a time: channel tid / 8 + 64 i of the tile's 3 x 128, whose
    // lane's l & 15 was this warp's number.
    Where before{-1, 0, 0, 0};
    const auto leave = [&] {
        if (before.kb < 0 || (int64_t)before.kb * TILE >= p.ld) return;
        const int ch = tid >> 3, pc = tid & 7;
        const uint8_t *src = codes + ch * TILE + (((2 * pc) ^ warp) & ~1) * 8;
        const int64_t off = (int64_t)(before.cb * TILE + ch) * p.ld + before.kb * TILE + 16 * pc;
        const auto one = [&](uint8_t *q, int i) {
            uint4 w = *reinterpret_cast<const uint4 *>(src + i * 64 * TILE);
            if (warp & 1) w = make_uint4(w.z, w.w, w.x, w.y);
            *reinterpret_cast<uint4 *>(q) = w;
        };
        const int64_t half = 64 * (int64_t)p.ld;
        if (p.dhT_q) {
            uint8_t *q = p.dhT_q + off, *u = q + (int64_t)p.F * p.ld;
            one(q, 0);
            one(q + half, 1);
            one(u, 2);
            one(u + half, 3);
        }
        if (p.actT_q) {
            one(p.actT_q + off, 4);
            one(p.actT_q + off + half, 5);
        }
    };
    Where now = fetch(0), next = fetch(1);
    int stage = 0;
    for (int t = t0; t < t1; t++, stage ^= 1) {
        cp_async_wait<1>();
        __syncwarp();
        const uint8_t *st = sm + stage * STAGE + warp * RW * ROW_BYTES;
        const float2 *hs = reinterpret_cast<const float2 *>(sm + stage * STAGE + SCALES) + warp * RW;
        uint64_t v[3][RW][2];
        float rm = 0.0f, dots[RW];
#pragma unroll
        for (int i = 0; i < RW; i++) {
            uint64_t dot;
            const float2 s = hs[i];
            swiglu4(*reinterpret_cast<const uint2 *>(st + i * ROW_BYTES + lane * 8),
                    *reinterpret_cast<const uint32_t *>(st + i * ROW_BYTES + 2 * TILE + lane * 4),
                    *reinterpret_cast<const uint32_t *>(st + i * ROW_BYTES + 3 * TILE + lane * 4), s.x, s.y, v[0][i],
                    v[1][i], v[2][i], dot);
            float x, y;
            unpack2(dot, x, y);
            dots[i] = x + y;
            if (ROW) {
                const float mg = warp_max(amax4(v[0][i])), mu = warp_max(amax4(v[1][i]));
                if ((lane >> 1) == i) rm = lane & 1 ? mu : mg;
            }
        }
        const Where at = now;
        now = next;
        __syncwarp();                                                  // the warp has read the stage
        next = fetch(stage);
        if (p.dots) {
            const float d = sums8(dots, lane);
            if ((lane & 3) == 0 && (lane >> 2) < at.n) p.dots[(int64_t)(at.row + (lane >> 2)) * nb + at.cb] = d;
        }
        if (COL) {
#pragma unroll
            for (int k = 0; k < 3; k++) {
                float m[4] = {};
#pragma unroll
                for (int i = 0; i < RW; i += 2) {
#pragma unroll
                    for (int j = 0; j < 2; j++) {
                        float x0, y0, x1, y1;
                        unpack2(v[k][i][j], x0, y0);
                        unpack2(v[k][i + 1][j], x1, y1);
                        m[2 * j] = amax3(x0, x1, m[2 * j]);
                        m[2 * j + 1] = amax3(y0, y1, m[2 * j + 1]);
                    }
                }
                *reinterpret_cast<float4 *>(red + (warp * 3 + k) * TILE + c0) = make_float4(m[0], m[1], m[2], m[3]);
            }
            __syncthreads();
            if (tid < 3 * TILE) {
                float m = red[tid];
#pragma unroll
                for (int w = 1; w < WARPS; w++) m = fmaxf(m, red[w * 3 * TILE + tid]);
                const float s = computed_scale(m);
                col_y[tid] = computed_recip(s);
                const int k = tid >> 7, ch = at.cb * TILE + (tid & 127);
                if ((int64_t)at.kb * TILE >= p.ld) {
                } else if (k == 2) {
                    if (p.actT_s) p.actT_s[(int64_t)at.kb * p.F + ch] = s;
                } else if (p.dhT_s) {
                    p.dhT_s[(int64_t)at.kb * 2 * p.F + k * p.F + ch] = s;
                }
            }
            leave();
        }
        if (ROW) {
            // computed_scale's value by block_scale's code: its branch keeps the encoding behind it apart from what is
            // before (65536 x 2048, this side alone: 139 us against 153 in one piece)
            const float s = fmaxf(block_scale(rm), 0x1p-126f), ry = computed_recip(s);
            if ((lane >> 1) < at.n) p.dh_s[(int64_t)(at.row + (lane >> 1)) * 2 * nb + (lane & 1) * nb + at.cb] = s;
            uint8_t *q = p.dh_q + (int64_t)at.row * 2 * p.F + at.cb * TILE + c0, *q2 = q + p.F;
#pragma unroll
            for (int i = 0; i < RW; i++, q += 2 * p.F, q2 += 2 * p.F) {
                const uint32_t g = encode4<COL>(v[0][i], __shfl_sync(0xFFFFFFFFu, ry, 2 * i));
                const uint32_t u = encode4<COL>(v[1][i], __shfl_sync(0xFFFFFFFFu, ry, 2 * i + 1));
                if (i < at.n) {
                    *reinterpret_cast<uint32_t *>(q) = g;
                    *reinterpret_cast<uint32_t *>(q2) = u;
                }
            }
        }
        if (COL) {
            __syncthreads();                                           // the reciprocals; the last tile's codes were read
#pragma unroll
            for (int k = 0; k < 3; k++) {
                const float4 y4 = *reinterpret_cast<const float4 *>(col_y + k * TILE + c0);
                const uint64_t y[2] = {pack2(y4.x, y4.y), pack2(y4.z, y4.w)};
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    uint32_t lo[2], hi[2];                             // the two columns' eight codes
#pragma unroll
                    for (int i = 0; i < RW; i += 4) {
                        float a[4], b[4];
#pragma unroll
                        for (int r = 0; r < 4; r++) unpack2(mul2(v[k][i + r][j], y[j]), a[r], b[r]);
                        lo[i / 4] = e4m3x4_pack(a[0], a[1], a[2], a[3]);
                        hi[i / 4] = e4m3x4_pack(b[0], b[1], b[2], b[3]);
                    }
                    uint2 *dst = reinterpret_cast<uint2 *>(codes + (k * TILE + c0 + 2 * j) * TILE) + (warp ^ (lane & 15));
                    dst[0] = make_uint2(lo[0], lo[1]);
                    dst[TILE / 8] = make_uint2(hi[0], hi[1]);
                }
            }
            before = at;
        }
    }
    if (COL) {
        __syncthreads();
        leave();
    }
    cp_async_wait<0>();
}

// Whether a row's dots were written: whether the block in which its expert has
// the row is named and holds it.
__device__ __forceinline__ bool row_formed(int64_t r, int64_t rows, const int32_t *__restrict__ off,
                                           const int32_t *__restrict__ pad, int E, int ld)
{
    int lo = 0, hi = E;                                            // off[lo] <= r < off[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= r) lo = mid;
        else hi = mid;
    }
    const int64_t at = pad[lo] + (r - off[lo]);
    if (at < 0 || at / TILE >= blocks_named(pad[E], E, rows, ld)) return false;
    const Rows b = block_rows(pad, off, E, at / TILE, rows);
    return r >= b.first && r < b.first + TILE && r < b.end;
}

constexpr int GATE_THREADS = 256, GATE_SLOTS = GATE_THREADS / 16;

// d_gates[slot]: the blocks' dots of the slot's row, sixteen lanes a slot (a
// fixed tree), over its gate; 0 for a slot whose row has no dots and for a
// gate of 0 (its row of d_act holds nothing, and every gate function's slope
// is 0 there).  With maps (off, pad) a CTA first sees whether they leave out
// no row in front of off[E], as those of a dispatch do; else each row is
// looked up, so that whatever the maps are, nothing is read that this call
// did not write (looking up every row: 82 us for 24576 x 1408 with every operand against
// 79, 323 for 65536 x 2048 against 314).
__global__ void __launch_bounds__(GATE_THREADS) gate_kernel(const float *__restrict__ dots,
                                                            const float *__restrict__ gates,
                                                            const int32_t *__restrict__ slot_to_sorted, int64_t slots,
                                                            int64_t rows, const int32_t *__restrict__ off,
                                                            const int32_t *__restrict__ pad, int E, int ld, int nb,
                                                            float *__restrict__ d_gates)
{
    const int lane = threadIdx.x & 15;
    int64_t end = rows;
    bool whole = true;
    if (off) {
        const int32_t P = __ldg(pad + E), A = __ldg(off + E);
        bool ok = P % TILE == 0 && P / TILE <= blocks_named(P, E, rows, ld);
        for (int e = threadIdx.x; e < E; e += GATE_THREADS) {
            const int64_t o0 = __ldg(off + e), o1 = __ldg(off + e + 1), p0 = __ldg(pad + e), p1 = __ldg(pad + e + 1);
            ok = ok && o0 <= o1 && p1 - p0 >= o1 - o0 && p0 % TILE == 0 && (e || (o0 == 0 && p0 == 0));
        }
        whole = __syncthreads_and(ok);
        if (A < end) end = A;
    }
    for (int64_t p0 = blockIdx.x * (int64_t)GATE_SLOTS; p0 < slots; p0 += gridDim.x * (int64_t)GATE_SLOTS) {
        const int64_t p = p0 + (threadIdx.x >> 4);
        const int32_t r = p < slots ? __ldg(slot_to_sorted + p) : -1;
        const float g = p < slots ? __ldg(gates + p) : 0.0f;
        const bool in = r >= 0 && g != 0.0f && (whole ? r < end : r < rows && row_formed(r, rows, off, pad, E, ld));
        float s = 0.0f;
        if (in)
            for (int b = lane; b < nb; b += 16) s += __ldg(dots + (int64_t)r * nb + b);
#pragma unroll
        for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (lane == 0 && p < slots) d_gates[p] = in ? __fdiv_rn(s, g) : 0.0f;
    }
}

template <bool ROW, bool COL>
static cudaError_t launch(const Args &p, int64_t blocks, cudaStream_t st)
{
    constexpr int smem = COL ? SMEM_COL : SMEM_ROW;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(swiglu_ckpt_kernel<ROW, COL>), smem, done);
    if (e != cudaSuccess) return e;
    const int64_t tiles = blocks * (p.F / TILE), sms = sm_count();
    swiglu_ckpt_kernel<ROW, COL><<<(unsigned)(tiles < sms ? tiles : sms), THREADS, smem, st>>>(p);
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
    int64_t blocks = (rows + 127) / 128;                          // at most
    if (col) {
        blocks += rows ? E : 0;
        if (max_pad / 128 > blocks) blocks = max_pad / 128;
    }
    if (blocks * (F / 128) >= (1LL << 31) || max_pad >= (1LL << 31)) return MOE_ERR_SHAPE;
    if (!dh_q != !dh_s || !dhT_q != !dhT_s || !actT_q != !actT_s) return MOE_ERR_NULL;
    if (col && (!expert_offsets || !pad)) return MOE_ERR_NULL;
    if (d_gates && slots && (!gates || !slot_to_sorted)) return MOE_ERR_NULL;
    if (rows && (dh_q || col || d_gates) && (!d_act || !h_q || !h_s)) return MOE_ERR_NULL;
    if (!aligned16(d_act) || !aligned16(h_q) || !aligned16(dh_q) || !aligned16(dhT_q) || !aligned16(actT_q))
        return MOE_ERR_ALIGN;
    for (const void *v : {(const void *)h_s, (const void *)dh_s, (const void *)dhT_s, (const void *)actT_s,
                          (const void *)gates, (const void *)slot_to_sorted, (const void *)d_gates,
                          (const void *)expert_offsets, (const void *)pad})
        if (reinterpret_cast<uintptr_t>(v) % 4) return MOE_ERR_ALIGN;
    if (!dh_q && !col && !(d_gates && slots)) return MOE_OK;
    const bool dots = d_gates && slots && rows;
    if (dots && (!workspace || workspace_bytes < moe_swiglu_backward_ckpt_workspace_size(rows, F))) return MOE_ERR_WORKSPACE;
    if (dots && !aligned16(workspace)) return MOE_ERR_ALIGN;
    const Span outs[] = {{dh_q, rows * 2 * F}, {dh_s, rows * (F / 128) * 8}, {dhT_q, max_pad * 2 * F},
                         {dhT_s, max_pad / 128 * 2 * F * 4}, {actT_q, max_pad * F}, {actT_s, max_pad / 128 * F * 4},
                         {d_gates, slots * 4},
                         {dots ? workspace : nullptr, (int64_t)moe_swiglu_backward_ckpt_workspace_size(rows, F)}};
    const Span ins[] = {{d_act, rows * F * 2}, {h_q, rows * 2 * F}, {h_s, rows * (F / 128) * 8},
                        {d_gates ? gates : nullptr, slots * 4}, {d_gates ? slot_to_sorted : nullptr, slots * 4},
                        {col ? expert_offsets : nullptr, (E + 1) * 4}, {col ? pad : nullptr, (E + 1) * 4}};
    if (overlap_any(outs, ins) || overlap_each(outs)) return MOE_ERR_UNSUPPORTED;
    cudaStream_t st = as_stream(stream);
    float *ws = dots ? static_cast<float *>(workspace) : nullptr;
    Args p{d_act, h_q, h_s, expert_offsets, pad, dh_q, dhT_q, actT_q, dh_s, dhT_s, actT_s, ws, rows, (int)max_pad, F, E};
    if (blocks && (dh_q || col || dots)) {
        const cudaError_t e = dh_q ? (col ? launch<true, true>(p, blocks, st) : launch<true, false>(p, blocks, st))
                                   : (col ? launch<false, true>(p, blocks, st) : launch<false, false>(p, blocks, st));
        if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
    if (d_gates && slots) {
        const int64_t each = (slots + GATE_SLOTS - 1) / GATE_SLOTS, most = (int64_t)sm_count() * 8;
        gate_kernel<<<(unsigned)(each < most ? each : most), GATE_THREADS, 0, st>>>(
            ws, gates, slot_to_sorted, slots, rows, col ? expert_offsets : nullptr, pad, E, (int)max_pad, F / 128, d_gates);
    } else if (!blocks) {
        return MOE_OK;
    }
    return launch_status();
}
