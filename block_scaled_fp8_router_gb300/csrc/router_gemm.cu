// router_gemm.cu -- the dense products of the router on the tensor cores, all
// of 24 significant bits: every expert's logit x W_r^T, and from dense logit
// gradients dl the input gradient dl W_r and the weight gradient dl^T x.
//
// x and W_r are bf16, so their products are exact in fp32.  dl is fp32: it is
// cut once into three bf16 parts by truncation (hi + mid + lo = dl exactly,
// 8 significant bits each), and every K block is multiplied part by part
// against the same B tile, three MMAs for one.
//
// The tensor core's running sum truncates: a chain of MMAs on one accumulator
// drifts toward zero by about half a unit in the last place per step.  So a
// chain stays within CHUNK K blocks; the epilogue warps add each chunk to
// fp32 registers, rounding to nearest (two or more TMEM buffers, so that the
// next chunk's MMAs run meanwhile).  That is 16 additions in a row for the
// logits and 48 for the three parts.  Norm of the error against 64 bits, and an
// fp32 product's: logits of 8192 x 7168 x 256 2.4e-7 (8.8e-7), dx 8.3e-7 (2.9e-7;
// its whole sum is one chain), dW_r 8.2e-7 (1.6e-6); 4093 x 2048 x 64: 2.3e-7
// (3.9e-7), 1.1e-7 (1.4e-7), 8.2e-7 (5.2e-7).  Shorter chains truncate less;
// of two blocks they cost dW_r 65 -> 71 us.
//
// One persistent CTA per SM: eight epilogue warps, a producer warp (TMA,
// 128-byte swizzle) and an MMA warp.  A tiles (one part, 16 KB) and B tiles
// have rings of their own, so that a part's place is free again after its own
// four MMAs.  The work is the list of K blocks of all output tiles, cut into
// equal runs of blocks, one run per CTA (whole tiles where there are many): a
// CTA has at most one tile begun by another and one that another ends, which
// go to its two fp32 slots in the workspace; reduce_kernel adds a tile's slots
// in order.  The launches are chained programmatically (a kernel sets itself
// up while the one before it ends).
//
// Bound: a block of four MMAs of 128 x 256 x 16 needs 512 clocks and takes 730 to
// 830, one of twelve 1536 and 1960 or, over two SMs, 1820.  For the logits the
// counters show no full unit (tensor pipe 44%, L2 to shared memory 25% of its
// peak over all SMs, HBM 42%, issue 21%); which wait makes up the rest of a
// block's time they do not show.  Measured at 8192 x 7168 x 256: logits 36 us
// (0.83 PFLOP/s), both gradients 119 us (0.51 PFLOP/s of fp32 products, three
// times that in MMAs); 4093 x 2048 x 64: 9 and 20 us.
#include "tcgen05.cuh"
#include "router_dense.cuh"

namespace moe {
namespace rg {

using namespace ffn;

constexpr int TM = 128;                   // tile rows
constexpr int KB = 64;                    // K block: 128 bytes of bf16
constexpr int CHUNK = 4;                  // K blocks per accumulator chain
constexpr int A_TILE = TM * KB * 2;       // 16 KB
constexpr int GEMM_EPI = 8;               // epilogue warps
constexpr int GEMM_PRODUCER = 8, GEMM_MMA = 9;
constexpr int GEMM_THREADS = 10 * 32;
constexpr int MAX_CTAS = 160;
constexpr int SLOT_COLS = 256;
constexpr size_t SLOT_FLOATS = (size_t)TM * SLOT_COLS;

// BOTH: DW's tiles by the first CTAs, DX's by the others, in one launch
enum Mode { LOGITS, DX, DW, BOTH };

// CL = 2: a pair of CTAs takes two row tiles of one column tile.  Each loads its
// own A tile and half of the B tile; one thread of the first CTA issues MMAs of
// 256 rows over both SMs (cta_group::2), each accumulating its 128 rows.
template <Mode MODE, int BN, int CL>
struct Cfg {
    static constexpr int P = MODE == LOGITS ? 1 : 3;              // parts of A
    static constexpr bool A_MN = MODE == DW, B_MN = MODE != LOGITS;  // (BOTH: A as the CTA's product has it)
    static constexpr int B_TILE = BN / CL * KB * 2;               // this CTA's share
    // places of the rings, 192 KB in all at most: a block needs one B and P A tiles
    static constexpr int NB = B_TILE == 32768 ? (P == 3 ? 3 : 4) : B_TILE == 16384 ? (P == 3 ? 4 : 6) : 8;
    static constexpr int NA = P == 3 ? (B_TILE == 32768 ? 6 : 8) : (B_TILE == 32768 ? 4 : B_TILE == 16384 ? 6 : 8);
    static constexpr int BUFS = BN == 256 ? 2 : 4;                // accumulators in tensor memory
    static constexpr int WCOLS = BN / 2;                          // columns of one epilogue warp
};

template <Mode MODE, int BN, int CL>
struct Smem {
    using C = Cfg<MODE, BN, CL>;
    uint8_t a[C::NA][A_TILE];
    uint8_t b[C::NB][C::B_TILE];
    float stage[GEMM_EPI][32 * 32];       // a warp's 32 x 32 sub-tile for its TMA store
    uint64_t afull[C::NA], aempty[C::NA];
    uint64_t bfull[C::NB], bempty[C::NB];
    uint64_t tfull[C::BUFS], tempty[C::BUFS];
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort_flag;
};

struct Params {
    int M, N;
    int nkb;                  // K blocks of a tile
    int n_tiles;              // tiles along N
    int64_t blocks;           // K blocks in all
    int gran;                 // cuts fall on multiples of this many blocks
    int split;                // CTAs that share a tile's K blocks
    int first;                // BOTH: CTAs of this product, the grid's first
    float *c;                 // [M, N]
    int direct_tma;           // whole tiles may be stored through tm_c
    int32_t *dev_status;
};

// first K block of run c (a CTA's, or a cluster's)
__host__ __device__ __forceinline__ int64_t run_begin(int64_t blocks, int gran, int ctas, int64_t c)
{
    return c * (blocks / gran) / ctas * gran;
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *tm, int x, int y, int z, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
                 "%3, %4}], [%5];" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *tm, int x, int y, int z, int w,
                                            uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
                 "%3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
                 : "memory");
}

// ---- the pair's forms (cta_group::2) ----
// loads to this CTA that complete at a barrier of the pair's first CTA (bar:
// its shared::cluster address)
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *tm, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
                 "[%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void *dst, const CUtensorMap *tm, int x, int y, int z, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
                 "[%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(void *dst, const CUtensorMap *tm, int x, int y, int z, int w,
                                                 uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
                 "[%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
                 : "memory");
}
// arrive at the barrier at this place in both CTAs when the MMAs so far are done
__device__ __forceinline__ void mma_commit_pair(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_u32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}
// this barrier's address in the pair's first CTA
__device__ __forceinline__ uint32_t first_cta(const uint64_t *bar)
{
    uint32_t out;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(out) : "r"(smem_u32(bar)));
    return out;
}
__device__ __forceinline__ void arrive_remote(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *tm, const void *src, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(tm)),
                 "r"(x), "r"(y), "r"(smem_u32(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// bf16 x bf16 -> fp32
__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// MN-major operand tile: 64-element (128-byte) groups along M/N, each [64 k
// rows][128 bytes] with the 128-byte swizzle.  Leading offset 8192 B from
// group to group, stride offset 1024 B from 8 k rows to the next 8.
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t saddr)
{
    uint64_t desc = 0;
    desc |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    desc |= (uint64_t)(8192u >> 4) << 16;
    desc |= (uint64_t)(1024u >> 4) << 32;
    desc |= (uint64_t)1 << 46;
    desc |= (uint64_t)2 << 61;
    return desc;
}

// fp32 accumulate, A = B = bf16, majorness bits 15 / 16 (1 = MN-major)
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// true in one thread of the (converged) warp
__device__ __forceinline__ bool elect_one()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// waits (each bounded) until the last of the n uses of each place of a ring is
// complete at its barrier
__device__ __forceinline__ void drain(uint64_t *full, int size, uint32_t n)
{
    for (int i = 0; i < size && (uint32_t)i < n; i++) {
        const uint32_t last = n - 1 - ((n - 1 - i) % size);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&full[i], (last / size) & 1) && globaltimer_ns() - t0 < TIMEOUT_NS) {}
    }
}

// SPLIT: a cluster of p.split CTAs per tile, each a share of its K blocks; the
// partial tiles meet in shared memory (CL = 1)
template <Mode MODE, int BN, int CL, bool SPLIT>
__global__ void __launch_bounds__(GEMM_THREADS, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_b0,
                const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_slots,
                const __grid_constant__ CUtensorMap tm_b1, const __grid_constant__ Params p0,
                const __grid_constant__ Params p1)
{
    using C = Cfg<MODE, BN, CL>;
    extern __shared__ uint8_t smem_raw[];
    Smem<MODE, BN, CL> &s =
        *reinterpret_cast<Smem<MODE, BN, CL> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    static_assert(CL == 1 || !SPLIT, "one or the other");
    static_assert(MODE != BOTH || SPLIT, "clusters for DW");
    // BOTH: CTAs below p1.first take DW (p1, A through tm_slots, B through
    // tm_b1) in clusters of p1.split, the others DX (p0), in the same clusters
    // but each on its own tiles
    const bool second = MODE == BOTH && (int)blockIdx.x < p1.first;
    const Params &p = second ? p1 : p0;
    const CUtensorMap &tm_a = second ? tm_slots : tm_a0, &tm_b = second ? tm_b1 : tm_b0;
    const bool a_mn = MODE == BOTH ? second : C::A_MN, split = MODE == BOTH ? second : SPLIT;
    static_assert(sizeof(s.a) + sizeof(s.b) >= (size_t)TM * BN * 4, "a partial tile fits the rings");
    const int rank = CL > 1 ? (int)(blockIdx.x % CL) : 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NA; i++) {
            mbar_init(&s.afull[i], 1);
            mbar_init(&s.aempty[i], 1);
        }
        for (int i = 0; i < C::NB; i++) {
            mbar_init(&s.bfull[i], 1);
            mbar_init(&s.bempty[i], 1);
        }
        for (int i = 0; i < C::BUFS; i++) {
            mbar_init(&s.tfull[i], 1);
            mbar_init(&s.tempty[i], CL * GEMM_EPI);
        }
        mbar_init(&s.mma_done, 1);
        s.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == GEMM_MMA) {
        if (CL > 1) tmem_alloc_pair(&s.tmem_base, TMEM_COLS);
        else tmem_alloc(&s.tmem_base, TMEM_COLS);
    }
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    if (CL > 1)      // both CTAs barriers are set up
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    tc_fence_after();
    // everything before this overlaps the kernel before; nothing it wrote is
    // read, and nothing written, before it has ended
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t tmem = s.tmem_base;
    volatile int *abort_flag = &s.abort_flag;
    int64_t b0, b1;
    const int share = split ? (int)(blockIdx.x % (unsigned)p.split) : 0;
    if (split) {
        const int64_t t0 = (int64_t)(blockIdx.x / (unsigned)p.split) * p.nkb;
        b0 = t0 + (int64_t)p.nkb * share / p.split;
        b1 = t0 + (int64_t)p.nkb * (share + 1) / p.split;
    } else {
        const int first = MODE == BOTH ? p1.first : 0;
        b0 = run_begin(p.blocks, p.gran, (gridDim.x - first) / CL, (blockIdx.x - first) / CL);
        b1 = run_begin(p.blocks, p.gran, (gridDim.x - first) / CL, (blockIdx.x - first) / CL + 1);
    }

    if (warp == GEMM_PRODUCER) {
        if (lane == 0) {
            uint32_t ja = 0, jb = 0;
            bool ok = true;
            int tile = (int)(b0 / p.nkb), kb = (int)(b0 - (int64_t)tile * p.nkb);
            int mt = tile / p.n_tiles, nt = tile - mt * p.n_tiles;
            mt = mt * CL + rank;
            for (int64_t b = b0; ok && b < b1; b++) {
                const int sb = jb % C::NB;
                if (!wait_or_abort(&s.bempty[sb], ((jb / C::NB) & 1) ^ 1, abort_flag, p.dev_status)) break;
                if (rank == 0) mbar_arrive_expect_tx(&s.bfull[sb], CL * C::B_TILE);
                const int bt = nt * CL + rank;           // this CTA's share of the column tile
                if (CL > 1) {
                    const uint32_t bar = first_cta(&s.bfull[sb]);
                    if (C::B_MN) tma_load_3d_pair(s.b[sb], &tm_b, 0, kb * KB, bt * (BN / CL / 64), bar);
                    else tma_load_2d_pair(s.b[sb], &tm_b, kb * KB * 2, bt * (BN / CL), bar);
                } else {
                    if (C::B_MN) tma_load_3d(s.b[sb], &tm_b, 0, kb * KB, bt * (BN / 64), &s.bfull[sb]);
                    else tma_load_2d(s.b[sb], &tm_b, kb * KB * 2, bt * BN, &s.bfull[sb]);
                }
                jb++;
#pragma unroll
                for (int q = C::P - 1; q >= 0; q--) {
                    const int sa = ja % C::NA;
                    if (!wait_or_abort(&s.aempty[sa], ((ja / C::NA) & 1) ^ 1, abort_flag, p.dev_status)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(&s.afull[sa], CL * A_TILE);
                    if (CL > 1) {
                        const uint32_t bar = first_cta(&s.afull[sa]);
                        if (a_mn) tma_load_4d_pair(s.a[sa], &tm_a, 0, kb * KB, mt * (TM / 64), q, bar);
                        else tma_load_3d_pair(s.a[sa], &tm_a, kb * KB * 2, mt * TM, q, bar);
                    } else {
                        if (a_mn) tma_load_4d(s.a[sa], &tm_a, 0, kb * KB, mt * (TM / 64), q, &s.afull[sa]);
                        else tma_load_3d(s.a[sa], &tm_a, kb * KB * 2, mt * TM, q, &s.afull[sa]);
                    }
                    ja++;
                }
                if (++kb == p.nkb) {
                    kb = 0;
                    if (++nt == p.n_tiles) {
                        nt = 0;
                        mt += CL;
                    }
                }
            }
            // no copy may still be in flight when the CTA exits (the pair's
            // copies all complete at the first CTA's barriers)
            if (rank == 0) {
                drain(s.afull, C::NA, ja);
                drain(s.bfull, C::NB, jb);
            }
            // nor an arrival at this CTA's barriers from the other
            if (CL > 1 && !*abort_flag) {
                drain(s.aempty, C::NA, ja);
                drain(s.bempty, C::NB, jb);
            }
        }
        __syncwarp();
    } else if (warp == GEMM_MMA) {
        // the whole warp goes through the loop (addresses and descriptors stay
        // in uniform registers), one elected thread issues
        if (rank == 0) {
            const uint32_t IDESC = idesc_bf16(CL * TM, BN, a_mn, C::B_MN);
            auto commit = [](uint64_t *bar) {
                if (CL > 1) mma_commit_pair(bar);
                else mma_commit(bar);
            };
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                return __all_sync(0xFFFFFFFFu, wait_or_abort(bar, parity, abort_flag, p.dev_status));
            };
            const bool leader = elect_one();
            const uint64_t A_STEP = a_mn ? 2048 >> 4 : 32 >> 4;
            constexpr uint64_t B_STEP = C::B_MN ? 2048 >> 4 : 32 >> 4;
            const uint32_t a0 = smem_u32(s.a[0]), bb0 = smem_u32(s.b[0]);
            const uint64_t adesc0 = a_mn ? sw128_desc_mn(a0) : sw128_desc(a0);
            const uint64_t bdesc0 = C::B_MN ? sw128_desc_mn(bb0) : sw128_desc(bb0);
            int sa = 0, sb = 0, buf = 0;                 // places in the rings, and their phases
            uint32_t pa = 0, pb = 0, pt = 1;
            int in_chunk = 0, kb = (int)(b0 % p.nkb);
            bool ok = true;
            for (int left = (int)(b1 - b0); ok && left > 0; left--) {
                if ((in_chunk == 0 && !wait(&s.tempty[buf], pt)) || !wait(&s.bfull[sb], pb)) break;
                const uint64_t bdesc = bdesc0 + (uint64_t)sb * (C::B_TILE >> 4);
#pragma unroll
                for (int q = C::P - 1; q >= 0; q--) {      // the small parts first
                    if (!wait(&s.afull[sa], pa)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t adesc = adesc0 + (uint64_t)sa * (A_TILE >> 4);
                    if (leader) {
#pragma unroll
                        for (int ks = 0; ks < KB / 16; ks++) {
                            const uint32_t add = in_chunk > 0 || q < C::P - 1 || ks > 0;
                            if (CL > 1)
                                mma_bf16_pair(tmem + buf * BN, adesc + A_STEP * ks, bdesc + B_STEP * ks, IDESC, add);
                            else
                                mma_bf16(tmem + buf * BN, adesc + A_STEP * ks, bdesc + B_STEP * ks, IDESC, add);
                        }
                        commit(&s.aempty[sa]);
                    }
                    __syncwarp();
                    if (++sa == C::NA) {
                        sa = 0;
                        pa ^= 1;
                    }
                }
                if (!ok) break;
                in_chunk++;
                if (++kb == p.nkb) kb = 0;
                const bool end = in_chunk == CHUNK || kb == 0 || left == 1;
                if (leader) {
                    commit(&s.bempty[sb]);
                    if (end) commit(&s.tfull[buf]);
                }
                __syncwarp();
                if (++sb == C::NB) {
                    sb = 0;
                    pb ^= 1;
                }
                if (end) {
                    in_chunk = 0;
                    if (++buf == C::BUFS) {
                        buf = 0;
                        pt ^= 1;
                    }
                }
            }
            if (leader) commit(&s.mma_done);
            __syncwarp();
        }
        // (the second CTA too: the arrival at its barrier has then come)
        if (lane == 0) {
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(&s.mma_done, 0) && globaltimer_ns() - t0 < 4 * TIMEOUT_NS) {}
        }
        __syncwarp();
    } else {
        // warp (q, half): TMEM lanes 32q .. 32q+31 (tile rows), columns WCOLS half ..
        const int q = warp & 3, half = warp >> 2;
        const uint32_t lane_addr = (uint32_t)(q * 32) << 16;
        float *stg = s.stage[warp];
        uint32_t jc = 0;
        bool aborted = false;
        for (int64_t b = b0; b < b1 && !aborted;) {
            const int tile = (int)(b / p.nkb), kb0 = (int)(b - (int64_t)tile * p.nkb);
            const int mp = tile / p.n_tiles, nt = tile - mp * p.n_tiles, mt = mp * CL + rank;
            const int64_t left = b1 - b;
            const int n = (int)(left < p.nkb - kb0 ? left : p.nkb - kb0);   // K blocks of this tile here
            float acc[C::WCOLS];
#pragma unroll
            for (int i = 0; i < C::WCOLS; i++) acc[i] = 0.0f;
            for (int k = 0; k < n; k += CHUNK, jc++) {
                const int buf = jc % C::BUFS;
                if (!wait_or_abort(&s.tfull[buf], (jc / C::BUFS) & 1, abort_flag, p.dev_status)) {
                    aborted = true;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < C::WCOLS / 16; h++) {
                    float v[16];
                    tmem_ld16(tmem + lane_addr + buf * BN + C::WCOLS * half + 16 * h, v);
#pragma unroll
                    for (int i = 0; i < 16; i++) acc[16 * h + i] += v[i];
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CL > 1) arrive_remote(first_cta(&s.tempty[buf]));
                    else mbar_arrive(&s.tempty[buf]);
                }
            }
            if (aborted) break;
            if (split) {
                // this CTA's partial tile over the rings, which nothing uses any
                // more: row r's 16-byte chunk c at chunk c ^ (r & 15)
                float4 *part = reinterpret_cast<float4 *>(s.a) + (32 * q + lane) * (BN / 4);
#pragma unroll
                for (int i = 0; i < C::WCOLS / 4; i++)
                    part[(C::WCOLS / 4 * half + i) ^ (lane & 15)] =
                        make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
                break;
            }
            const bool whole = n == p.nkb;
            const int row0 = mt * TM + 32 * q;
            const bool slot0 = b == b0;
#pragma unroll
            for (int h = 0; h < C::WCOLS / 32; h++) {
                const int col_t = C::WCOLS * half + 32 * h, col0 = nt * BN + col_t;
                if (row0 >= p.M || col0 >= p.N) break;
                if (whole && !p.direct_tma) {
                    if (row0 + lane < p.M)
                        for (int i = 0; i < 32; i++)
                            if (col0 + i < p.N) p.c[(int64_t)(row0 + lane) * p.N + col0 + i] = acc[32 * h + i];
                    continue;
                }
                // the previous store has read the staging tile
                if (lane == 0) bulk_wait_read_all();
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; i++)
                    *reinterpret_cast<float4 *>(stg + lane * 32 + 4 * (i ^ (lane & 7))) =
                        make_float4(acc[32 * h + 4 * i], acc[32 * h + 4 * i + 1], acc[32 * h + 4 * i + 2],
                                    acc[32 * h + 4 * i + 3]);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    if (whole)
                        tma_store_2d_evict_first(&tm_c, stg, col0, row0);
                    else
                        tma_store_2d(&tm_slots, stg, col_t, ((int)blockIdx.x * 2 + (slot0 ? 0 : 1)) * TM + 32 * q);
                }
            }
            b += n;
        }
        // the stores have read their staging tiles (they are complete when the
        // grid is)
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    __syncwarp();
    if constexpr (SPLIT) {
        // every CTA's partial tile is there: each adds up a share of the rows,
        // the partial tiles in order of K
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        const int tile = (int)(blockIdx.x / (unsigned)p.split), mt = tile / p.n_tiles, nt = tile - mt * p.n_tiles;
        const int r0 = TM * share / p.split, r1 = min(TM * (share + 1) / p.split, p.M - mt * TM);
        const uint32_t base = smem_u32(s.a);
        for (int i = r0 * (BN / 4) + threadIdx.x; split && i < r1 * (BN / 4) && !*abort_flag; i += GEMM_THREADS) {
            const int r = i / (BN / 4), c = i % (BN / 4), col = nt * BN + 4 * c;
            if (col >= p.N) continue;
            const uint32_t at = base + (uint32_t)(r * (BN / 4) + (c ^ (r & 15))) * 16;
            float4 v[8];
#pragma unroll
            for (int u = 0; u < 8; u++) {
                v[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (u < p.split) {
                    uint32_t a;
                    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(at), "r"(u));
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(v[u].x), "=f"(v[u].y), "=f"(v[u].z), "=f"(v[u].w)
                                 : "r"(a));
                }
            }
#pragma unroll
            for (int u = 1; u < 8; u++) {
                v[0].x += v[u].x;
                v[0].y += v[u].y;
                v[0].z += v[u].z;
                v[0].w += v[u].w;
            }
            float *o = p.c + (int64_t)(mt * TM + r) * p.N + col;
            if (p.direct_tma) {
                *reinterpret_cast<float4 *>(o) = v[0];
            } else {
                const float x[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
                for (int u = 0; u < 4; u++)
                    if (col + u < p.N) o[u] = x[u];
            }
        }
        __syncwarp();
    }
    if (CL > 1 || SPLIT)      // no CTA leaves while another may still use its memory or barriers
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp == GEMM_MMA) {
        if (CL > 1) tmem_dealloc_pair(tmem, TMEM_COLS);
        else tmem_dealloc(tmem, TMEM_COLS);
    }
}

// C tiles that several CTAs have parts of: the parts added in order of K.
// grid (tile, row group of 8), 256 threads, four columns each
template <int BN>
__global__ void __launch_bounds__(256) reduce_kernel(const float *__restrict__ slots, Params p, int ctas, int cl)
{
    __shared__ int s_slot[MAX_CTAS];
    // ctas: runs; cl CTAs each, for the row tiles mp cl .. mp cl + cl - 1
    const int tile = blockIdx.x / cl, mp = tile / p.n_tiles, nt = tile - mp * p.n_tiles;
    const int rank = blockIdx.x % cl, mt = mp * cl + rank;
    const int64_t k0 = (int64_t)tile * p.nkb, k1 = k0 + p.nkb;
    const int64_t ub = p.blocks / p.gran;
    const int c0 = (int)(((k0 / p.gran + 1) * ctas - 1) / ub), c1 = (int)((((k1 - 1) / p.gran + 1) * ctas - 1) / ub);
    const int rows = min(8, p.M - mt * TM - 8 * (int)blockIdx.y), cols = min(BN, p.N - nt * BN), n = c1 - c0 + 1;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (n == 1 || rows <= 0) return;
    for (int i = threadIdx.x; i < n; i += 256)
        s_slot[i] = 2 * ((c0 + i) * cl + rank) + (run_begin(p.blocks, p.gran, ctas, c0 + i) >= k0 ? 0 : 1);
    __syncthreads();
    const int tc = threadIdx.x % (BN / 4), tr = threadIdx.x / (BN / 4);
    if (4 * tc >= cols) return;
    for (int r = tr; r < rows; r += 256 / (BN / 4)) {
        const float *src = slots + (size_t)(8 * blockIdx.y + r) * SLOT_COLS + 4 * tc;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int c = 0; c < n; c += 8) {
            float4 v[8];
#pragma unroll
            for (int u = 0; u < 8; u++)
                v[u] = c + u < n ? __ldcs(reinterpret_cast<const float4 *>(src + (size_t)s_slot[c + u] * SLOT_FLOATS))
                                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int u = 0; u < 8; u++) {
                acc.x += v[u].x;
                acc.y += v[u].y;
                acc.z += v[u].z;
                acc.w += v[u].w;
            }
        }
        float *o = p.c + (int64_t)(mt * TM + 8 * blockIdx.y + r) * p.N + nt * BN + 4 * tc;
        if (p.direct_tma) {
            *reinterpret_cast<float4 *>(o) = acc;
        } else {
            const float v[4] = {acc.x, acc.y, acc.z, acc.w};
            for (int i = 0; i < 4; i++)
                if (4 * tc + i < cols) o[i] = v[i];
        }
    }
}

__device__ __forceinline__ float rest(float v, float part)
{
    const float r = v - part;
    return r == r ? r : 0.0f;
}

// dl [T, E] fp32 -> parts [3][T][Ep] bf16 by truncation, zeros in columns E ..
// Ep - 1; one thread per eight columns
__global__ void __launch_bounds__(256) split_kernel(const float *__restrict__ dl, int T, int E, int Ep,
                                                    uint16_t *__restrict__ parts)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int per = Ep / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)T * per) return;
    const int64_t t = i / per;
    const int e = 8 * (int)(i - t * per);
    float v[8];
    if (e + 8 <= E && (E & 3) == 0 && (reinterpret_cast<uintptr_t>(dl) & 15u) == 0) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(dl + t * E + e));
        const float4 b = __ldg(reinterpret_cast<const float4 *>(dl + t * E + e) + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int u = 0; u < 8; u++) v[u] = e + u < E ? __ldg(dl + t * E + e + u) : 0.0f;
    }
    const int64_t plane = (int64_t)T * Ep;
    // infinities and NaN are their first part (NaN made quiet: a low payload
    // would be cut off).  A part that comes out 0 where dl is not is the least
    // bf16 of dl's sign, 2^-133: 0 times an infinity of x or W_r would be a NaN
    // beside the other parts' infinity, this gives the same infinity
    uint32_t least[8];
#pragma unroll
    for (int u = 0; u < 8; u++) {
        v[u] = v[u] == v[u] ? v[u] : __uint_as_float(0x7FC00000u);
        least[u] = (__float_as_uint(v[u]) & 0x80000000u) | (v[u] != 0.0f ? 0x00010000u : 0u);
    }
#pragma unroll
    for (int q = 0; q < 3; q++) {
        uint32_t w[8];
#pragma unroll
        for (int u = 0; u < 8; u++) {
            w[u] = __float_as_uint(v[u]) & 0xFFFF0000u;
            v[u] = rest(v[u], __uint_as_float(w[u]));
            if ((w[u] & 0x7FFFFFFFu) == 0) w[u] = least[u];
        }
        *reinterpret_cast<uint4 *>(parts + q * plane + t * Ep + e) =
            make_uint4((w[0] >> 16) | w[1], (w[2] >> 16) | w[3], (w[4] >> 16) | w[5], (w[6] >> 16) | w[7]);
    }
}

// ------------------------------------------------------------------- host

static inline int pad64(int v) { return (v + 63) / 64 * 64; }

// clusters of 2, 4 or 8 of these CTAs (one fills an SM) that the device holds
// at once: SMs come in groups of uneven size, so fewer than SMs / size
static int clusters_at_once(int size)
{
    static const struct Held {
        int n[4];
        Held()
        {
            constexpr size_t smem = sizeof(Smem<LOGITS, 256, 1>) + 1024;
            auto *kernel = gemm_kernel<LOGITS, 256, 1, true>;
            const bool ok =
                cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess;
            for (int i = 1; i < 4; i++) {
                cudaLaunchConfig_t cfg = {};
                cudaLaunchAttribute attr[1];
                attr[0].id = cudaLaunchAttributeClusterDimension;
                attr[0].val.clusterDim.x = 1 << i;
                attr[0].val.clusterDim.y = 1;
                attr[0].val.clusterDim.z = 1;
                cfg.gridDim = dim3(1 << i);
                cfg.blockDim = dim3(GEMM_THREADS);
                cfg.dynamicSmemBytes = smem;
                cfg.attrs = attr;
                cfg.numAttrs = 1;
                if (!ok || cudaOccupancyMaxActiveClusters(&n[i], kernel, &cfg) != cudaSuccess || n[i] < 1) n[i] = 1;
            }
            cudaGetLastError();
        }
    } held;
    return held.n[size == 2 ? 1 : size == 4 ? 2 : 3];
}

// How the work is cut, by an estimate in clocks.  A K block takes parts x 2 BN
// clocks on the tensor cores and about 400 more (measured: 128 clocks per MMA
// of N = 256, 960 per block of four, 1960 per block of twelve), and 700 at
// least, where a CTA's share of HBM is slower.  Whole tiles; or a cluster of 2, 4 or 8 CTAs per
// tile (about 4000 clocks for the exchange; 8192 x 7168 x 256 logits 40 us
// against 44 cut into runs); or all blocks cut into equal runs (about 16000
// for the slots and their reduction: only long sums, weight gradients of
// thousands of tokens, win by it: 65 us against 79 at 8192 x 7168 x 256).
struct Plan {
    int cl, split, runs, gran, m_tiles, n_tiles, nkb;     // m_tiles: groups of cl row tiles
    int64_t blocks;
    bool slots;          // some tile is cut into runs
    int bn;              // columns of a tile
    int64_t clocks;
};

static Plan plan_bn(int M, int N, int K, int bn, int parts)
{
    Plan r;
    r.bn = bn;
    const int rows = (M + TM - 1) / TM;
    r.n_tiles = (N + bn - 1) / bn;
    r.nkb = (K + KB - 1) / KB;
    int sms = sm_count();
    if (sms > MAX_CTAS) sms = MAX_CTAS;
    const int64_t t = 2 * bn * parts + 400 > 700 ? 2 * bn * parts + 400 : 700;
    const int64_t tiles1 = (int64_t)rows * r.n_tiles;
    int64_t best = (tiles1 + sms - 1) / sms * r.nkb * t;
    int kind = 1;                                          // whole tiles
    for (int s = 2; s <= 8 && s <= r.nkb; s *= 2) {
        const int64_t cap = clusters_at_once(s);
        const int64_t e = (tiles1 + cap - 1) / cap * ((r.nkb + s - 1) / s * t + 4000);
        if (e < best) {
            best = e;
            kind = s;
        }
    }
    const int64_t cut = tiles1 * r.nkb * t / sms + 16000;
    if (cut < best && r.nkb > 1) {
        best = cut;
        kind = 0;
    }
    r.split = kind > 1 ? kind : 1;
    // pairs of row tiles (two-SM MMAs) for long work where few tiles are
    // wasted: 8192 x 7168 x 256 backward 125 us against 129, but dx of 5000 x
    // 4096 x 128 29 us against 25
    r.cl = kind <= 1 && best > 50000 && bn >= 128 && rows > 1 && (rows % 2 == 0 || rows >= 7) ? 2 : 1;
    r.m_tiles = (rows + r.cl - 1) / r.cl;
    const int64_t tiles = (int64_t)r.m_tiles * r.n_tiles;
    const int most = sms / r.cl > 0 ? sms / r.cl : 1;
    r.blocks = tiles * r.nkb;
    r.gran = kind == 0 ? 1 : r.nkb;
    const int64_t units = kind == 0 ? (r.blocks + CHUNK - 1) / CHUNK : tiles;
    r.runs = kind > 1 ? (int)(tiles * kind) : (int)(units < most ? units : most);
    r.slots = kind == 0;
    r.clocks = best;
    return r;
}

// the tile width by the same estimate: narrower tiles where wide ones are too
// few for the SMs
static Plan plan(Mode mode, int M, int N, int K)
{
    const int parts = mode == LOGITS ? 1 : 3;
    Plan r = plan_bn(M, N, K, 256, parts);
    for (int bn = 128; bn >= (mode == LOGITS ? 64 : 128); bn /= 2) {
        const Plan q = plan_bn(M, N, K, bn, parts);
        if (q.clocks < r.clocks || N <= bn) r = q;
    }
    return r;
}

static size_t slots_bytes(const Plan &r) { return r.slots ? (size_t)r.runs * r.cl * 2 * SLOT_FLOATS * sizeof(float) : 0; }


// [parts][rows][k] bf16, k contiguous: box 64 k x box_rows rows of one part
static bool map_k_major(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap *m, const void *base, uint64_t k,
                        uint64_t rows, uint64_t parts, uint32_t box_rows)
{
    const cuuint64_t dims[3] = {k * 2, rows, parts};
    const cuuint64_t strides[2] = {k * 2, k * 2 * rows};
    const cuuint32_t box[3] = {128, box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [parts][k rows][mn] bf16, mn contiguous (a multiple of 64), as (128 bytes,
// k, 64-element group, part): box 64 k rows x `groups` groups of one part
static bool map_mn_major(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap *m, const void *base, uint64_t mn,
                         uint64_t k, uint64_t parts, uint32_t groups, int rank)
{
    const cuuint64_t dims[4] = {128, k, mn / 64, parts};
    const cuuint64_t strides[3] = {mn * 2, 128, mn * 2 * k};
    const cuuint32_t box[4] = {128, KB, groups, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T>
struct Same {
    using type = T;
};

// a launch that may begin while the kernel before it on the stream ends (pdl:
// that kernel is one of this file's, which lets it)
template <typename... Args>
static cudaError_t launch_chained(void (*kernel)(Args...), dim3 grid, int cluster, int threads, size_t smem, bool pdl,
                                  cudaStream_t st, typename Same<Args>::type... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

static Params params(const Plan &pl, float *c, int M, int N, int32_t *dev_status)
{
    Params p;
    p.M = M;
    p.N = N;
    p.nkb = pl.nkb;
    p.n_tiles = pl.n_tiles;
    p.blocks = pl.blocks;
    p.gran = pl.gran;
    p.split = pl.split;
    p.first = 0;
    p.c = c;
    p.direct_tma = N % 4 == 0 && aligned16(c);
    p.dev_status = dev_status;
    return p;
}

// the maps of A ([parts][rows][k] for logits and dx, [parts][k][rows] for dW_r)
// and of one CTA's share of B ([N][K] for logits, else [K][N])
static bool map_a(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap *m, Mode mode, const void *a, int M, int K)
{
    if (mode == DW) return map_mn_major(enc, m, a, pad64(M), K, 3, TM / 64, 4);
    return map_k_major(enc, m, a, mode == DX ? pad64(K) : K, M, mode == DX ? 3 : 1, TM);
}
static bool map_b(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap *m, Mode mode, const void *b, int N, int K, int share)
{
    return mode == LOGITS ? make_map(enc, m, b, (uint64_t)K * 2, N, share) : map_mn_major(enc, m, b, N, K, 1, share / 64, 3);
}

static PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static const auto enc = encode_fn();      // the driver's: looked up once
    return enc;
}

template <Mode MODE, int BN, int CL, bool SPLIT>
static cudaError_t start(int ctas, int cluster, const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &c,
                         const CUtensorMap &slots, const CUtensorMap &b1, const Params &p0, const Params &p1, bool pdl,
                         cudaStream_t st)
{
    constexpr size_t smem = sizeof(Smem<MODE, BN, CL>) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory");
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem((const void *)gemm_kernel<MODE, BN, CL, SPLIT>, (int)smem, done);
    if (e != cudaSuccess) return e;
    return launch_chained(gemm_kernel<MODE, BN, CL, SPLIT>, dim3(ctas), cluster, GEMM_THREADS, smem, pdl, st, a, b, c,
                          slots, b1, p0, p1);
}

template <Mode MODE, int BN, int CL, bool SPLIT>
static moe_status launch_cl(const Plan &pl, const void *a, const void *b, float *c, int M, int N, int K, float *slots,
                            int32_t *dev_status, bool pdl, cudaStream_t st)
{
    const auto enc = encoder();
    if (!enc) return MOE_ERR_CUDA;
    const Params p = params(pl, c, M, N, dev_status);
    const int ctas = pl.runs * CL;
    CUtensorMap ma, mb, mc, ms;
    if (!map_a(enc, &ma, MODE, a, M, K) || !map_b(enc, &mb, MODE, b, N, K, BN / CL)) return MOE_ERR_CUDA;
    mc = ms = ma;                         // where not used
    if (!SPLIT && p.direct_tma && !make_map_f32_store(enc, &mc, c, (uint64_t)N, (uint64_t)M)) return MOE_ERR_CUDA;
    if (pl.slots && !make_map_f32_store(enc, &ms, slots, SLOT_COLS, (uint64_t)ctas * 2 * TM)) return MOE_ERR_CUDA;
    if (start<MODE, BN, CL, SPLIT>(ctas, SPLIT ? pl.split : CL, ma, mb, mc, ms, mb, p, p, pdl, st) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (pl.slots && launch_chained(reduce_kernel<BN>, dim3((unsigned)(pl.m_tiles * pl.n_tiles * CL), TM / 8), 1, 256, 0,
                                   true, st, (const float *)slots, p, pl.runs, CL) != cudaSuccess)
        return MOE_ERR_CUDA;
    return launch_status();
}

// dx and dW_r in one launch where neither fills the GPU for long: clusters of
// pw.split CTAs on dW_r's tiles, the other CTAs on whole tiles of dx, all
// resident at once.  False where two launches are estimated to be shorter.
// Measured, one launch against two (split_kernel included): 4093 x 2048 x 64
// 23.6 us against 30, 5000 x 4096 x 128 39.5 against 49, 4096 x 5120 x 160 48
// against 60, 1 x 2048 x 64 11 against 13; dW_r alone, which keeps the same cut
// so that its bits do not depend on what else is asked for, 31.7 against 25.5
// at 5000 x 4096 x 128.
static bool plan_both(int T, int d, int E, Plan *px, Plan *pw, int *first, int *ctas)
{
    int64_t best = plan(DX, T, d, E).clocks + plan(DW, E, d, T).clocks;
    bool found = false;
    for (int bn = 256; bn >= 128; bn /= 2)
        for (int s = 1; s <= 8; s *= 2) {
            Plan x = plan_bn(T, d, E, bn, 3), w = plan_bn(E, d, T, bn, 3);
            const int64_t tx = (int64_t)((T + TM - 1) / TM) * x.n_tiles, tw = (int64_t)((E + TM - 1) / TM) * w.n_tiles;
            const int64_t cap = (s == 1 ? sm_count() : clusters_at_once(s)) * (int64_t)s;
            int64_t nx = (cap - tw * s) / s * s;
            if (s > w.nkb || nx < s) continue;
            if (nx > (tx + s - 1) / s * s) nx = (tx + s - 1) / s * s;
            const int64_t t = 6 * bn + 400;
            const int64_t cw = (w.nkb + s - 1) / s * t + (s > 1 ? 4000 : 0), cx = (tx + nx - 1) / nx * (x.nkb * t + 600);
            if ((cw > cx ? cw : cx) >= best) continue;
            best = cw > cx ? cw : cx;
            found = true;
            x.cl = w.cl = 1;
            x.m_tiles = (T + TM - 1) / TM;
            w.m_tiles = (E + TM - 1) / TM;
            x.blocks = tx * x.nkb;
            w.blocks = tw * w.nkb;
            x.gran = x.nkb;
            w.gran = w.nkb;
            x.split = 1;
            w.split = s;
            x.slots = w.slots = false;
            x.runs = (int)(tx < sm_count() ? tx : sm_count());     // on its own
            w.runs = (int)(tw * s);
            *px = x;
            *pw = w;
            *first = (int)(tw * s);
            *ctas = (int)(tw * s + nx);
        }
    return found;
}

template <int BN>
static moe_status launch_both(const Plan &px, const Plan &pw, int first, int ctas, const uint16_t *parts,
                              const uint16_t *x, const uint16_t *w, int T, int d, int E, float *dx, float *dw,
                              int32_t *dev_status, cudaStream_t st)
{
    const auto enc = encoder();
    if (!enc) return MOE_ERR_CUDA;
    CUtensorMap xa, xb, xc, wa, wb;
    if (!map_a(enc, &xa, DX, parts, T, E) || !map_b(enc, &xb, DX, w, d, E, BN) ||
        !make_map_f32_store(enc, &xc, dx, (uint64_t)d, (uint64_t)T) || !map_a(enc, &wa, DW, parts, E, T) ||
        !map_b(enc, &wb, DW, x, d, T, BN))
        return MOE_ERR_CUDA;
    const Params p0 = params(px, dx, T, d, dev_status);
    Params p1 = params(pw, dw, E, d, dev_status);
    p1.first = first;
    return start<BOTH, BN, 1, true>(ctas, pw.split, xa, xb, xc, wa, wb, p0, p1, true, st) == cudaSuccess
               ? launch_status()
               : MOE_ERR_CUDA;
}

template <Mode MODE, int BN>
static moe_status launch_bn(const Plan &pl, const void *a, const void *b, float *c, int M, int N, int K, float *slots,
                            int32_t *dev_status, bool pdl, cudaStream_t st)
{
    if (pl.split > 1) return launch_cl<MODE, BN, 1, true>(pl, a, b, c, M, N, K, slots, dev_status, pdl, st);
    if constexpr (BN >= 128) {
        if (pl.cl == 2) return launch_cl<MODE, BN, 2, false>(pl, a, b, c, M, N, K, slots, dev_status, pdl, st);
    }
    return launch_cl<MODE, BN, 1, false>(pl, a, b, c, M, N, K, slots, dev_status, pdl, st);
}

template <Mode MODE>
static moe_status launch(const Plan &pl, const void *a, const void *b, float *c, int M, int N, int K, float *slots,
                         int32_t *dev_status, bool pdl, cudaStream_t st)
{
    if (pl.bn == 256) return launch_bn<MODE, 256>(pl, a, b, c, M, N, K, slots, dev_status, pdl, st);
    if constexpr (MODE == LOGITS) {
        if (pl.bn == 64) return launch_bn<MODE, 64>(pl, a, b, c, M, N, K, slots, dev_status, pdl, st);
    }
    return launch_bn<MODE, 128>(pl, a, b, c, M, N, K, slots, dev_status, pdl, st);
}

static size_t align_up(size_t v) { return (v + 255) & ~(size_t)255; }

} // namespace rg

size_t router_logits_workspace(int T, int d, int E)
{
    using namespace rg;
    return 256 + slots_bytes(plan(LOGITS, T, E, d));
}

moe_status router_logits(const uint16_t *x, const uint16_t *w, int T, int d, int E, float *logits, void *ws,
                         int32_t *dev_status, cudaStream_t st)
{
    return rg::launch<rg::LOGITS>(rg::plan(rg::LOGITS, T, E, d), x, w, logits, T, E, d, (float *)ws, dev_status, false, st);
}

size_t router_backward_workspace(int T, int d, int E)
{
    using namespace rg;
    const size_t sx = slots_bytes(plan(DX, T, d, E)), sw = slots_bytes(plan(DW, E, d, T));
    return 256 + align_up((size_t)3 * T * pad64(E) * 2) + (sx > sw ? sx : sw);
}

moe_status router_backward(const uint16_t *x, const uint16_t *w, const float *dl, int T, int d, int E, float *dx,
                           float *dw, void *ws, int32_t *dev_status, cudaStream_t st)
{
    using namespace rg;
    const int Ep = pad64(E);
    uint16_t *parts = (uint16_t *)ws;
    float *slots = (float *)((uint8_t *)ws + align_up((size_t)3 * T * Ep * 2));
    const int64_t n = (int64_t)T * (Ep / 8);
    split_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(dl, T, E, Ep, parts);
    moe_status s = launch_status();
    Plan px, pw;
    int first, ctas;
    if (s != MOE_OK) return s;
    // (one output alone is summed in the same order as beside the other)
    if (!plan_both(T, d, E, &px, &pw, &first, &ctas)) {
        px = plan(DX, T, d, E);
        pw = plan(DW, E, d, T);
    } else if (dx && dw) {
        return px.bn == 256
                   ? launch_both<256>(px, pw, first, ctas, parts, x, w, T, d, E, dx, dw, dev_status, st)
                   : launch_both<128>(px, pw, first, ctas, parts, x, w, T, d, E, dx, dw, dev_status, st);
    }
    if (dx) s = launch<DX>(px, parts, w, dx, T, d, E, slots, dev_status, true, st);
    if (s == MOE_OK && dw) s = launch<DW>(pw, parts, x, dw, E, d, T, slots, dev_status, true, st);
    return s;
}

} // namespace moe
