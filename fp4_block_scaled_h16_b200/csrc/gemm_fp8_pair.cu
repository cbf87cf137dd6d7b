// gemm_fp8_pair.cu -- the FP8 block-scaled GEMM (fp4_fp8_block_gemm) for
// outputs large enough to fill the GPU with 256 x 256 tiles:
//
//   C[i, j] = sum_kc sA[kc, i] sB[kc, j or j / 128] P_kc[i, j],
//   P_kc[i, j] = sum_{k in chunk kc of 128} qA[i, k] qB[j, k].
//
// An FP32 scale per 128-K chunk cannot ride in the tensor core's accumulator,
// so every chunk is a partial product of its own, promoted in binary32
// registers: acc += (sA sB) P.  The partial of a chunk is 256 x 256 over a CTA
// pair (tcgen05.mma cta_group::2 kind::f8f6f4, four of K = 32), 128 x 256 per
// CTA: 256 TMEM columns, so all 512 columns hold two partials and the tensor
// core fills one while eight warps promote the other.
//
// What bounds it: the hand-over of the two partials.  A chunk is 512 tensor
// cycles (520 measured with the promotion left out); with it, 790, because a
// partial is busy for its MMAs (512), until the promotion warps see them
// complete (240), until those have read it (about 500) and until the issuer
// sees that (200), and only two fit in TMEM.  What was tried against that, per
// chunk of 256 columns: halves of 128 columns with four partials, 1480 (the
// N = 128 MMA takes 1.2 times its share, and every hand-over costs the issuer
// and each warp as much as a whole chunk's), 850 with an issuer per half; tiles
// of 160 columns with three partials, 800 for each 160; 16 promotion warps of 64
// columns, 815.  Single CTAs with 128 x 256 tiles, persistent like these, hand over
// sooner but load 48 KB per chunk and SM instead of 32: 203 and 602 us for the two
// products below.  One thread needs about 800 cycles for a chunk's two waits, four
// MMAs and two commits beside a busy promotion, so two issuers take turns.  With
// 1 x 128 blocks of B the promotion's product per element more makes it 1040.
// QKV Fprop 8192 x 6144 x 4096: 196 us, 2100 TFLOP/s (0.63 of twice the bf16
// burst rate); Wgrad 4096 x 14336 x 8192 in f32: 584 us, 1650 TFLOP/s (570 to 632
// from run to run, by the clocks that the power limit leaves).
//
// Roles (both CTAs, 384 threads, persistent over pair tiles, one CTA per SM):
//   warp 0   TMA producer: this CTA's 128 rows of A and 128 lines of B per
//            chunk, and the chunk's scales of its rows (and of the tile's
//            columns) into a longer ring, all counted on the leader's barrier;
//   warps 1, 2  (warp 1: TMEM) in the leader, one thread each issues the MMAs
//            of both CTAs for every other chunk;
//   warps 4-11  promotion, 32 rows x 128 columns each (128 accumulators and 64
//            columns in flight per thread; setmaxnreg moves registers of warps
//            0-3 here), then the output: 32-row x 128-byte boxes in swizzled
//            shared memory and TMA stores.
// No load uses cluster multicast.  Every wait is bounded; one that runs out
// sets the device error word to FP4_ERR_TIMEOUT, and before either CTA exits
// the leader settles every load either CTA issued, as in gemm_pair.cu.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "internal.h"
#include "sm100.cuh"

namespace fp4 {

namespace {

constexpr int PM = 256, PN = 256;        // tile of a CTA pair
constexpr int BK = 128;                  // K elements (bytes) per stage: one scale chunk
constexpr int MMA_WARPS = 2;
constexpr int PROMO_WARPS = 8;
constexpr int NUM_THREADS = 128 + 32 * PROMO_WARPS;
// registers per thread: at launch, of warps 0-3, and of the promotion warps
constexpr int REGS_LAUNCH = 168, REGS_LEAD = 56, REGS_PROMO = 224;
static_assert(128 * REGS_LEAD + 32 * PROMO_WARPS * REGS_PROMO <= NUM_THREADS * REGS_LAUNCH, "register split");
constexpr int COLS = PN / (PROMO_WARPS / 4);         // columns of the tile per promotion warp
constexpr int STAGES = 5;
// Ring of scale slots, without barriers of its own: a stage is refilled once its
// MMAs are done; those were issued once the promotion had read the partial two
// chunks before, and so was past the scales of the chunk before that one (their
// values are in its sums by then: mbar_arrive_cluster_relaxed).
constexpr int SC_SLOTS = 8;
static_assert(SC_SLOTS >= STAGES + 3, "scales are read before their slot is refilled");
constexpr uint32_t A_BYTES = 128 * BK, B_BYTES = 128 * BK;
constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;
constexpr uint32_t SC_BYTES = 128 * 4 + PN * 4;      // scales of 128 rows and of 256 columns
constexpr uint32_t EPI_BUF = 4096;       // per promotion warp: one 32-row x 128-byte box of C
constexpr uint32_t SMEM = STAGES * STAGE_BYTES + PROMO_WARPS * EPI_BUF + SC_SLOTS * SC_BYTES + 512 + 1024;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t DRAIN_LIMIT = 1u << 22;
constexpr unsigned int ERR_TIMEOUT = 7u;
static_assert(SMEM <= 232448u, "shared memory");

struct PairParams {
    const float* sb;          // [chunks, lpb] (128 x 128 blocks)
    int64_t lpb;
    void* c;
    int64_t ldc;
    int M, N, chunks;
    int odd_n;                // N ends inside a 16-byte chunk of a row of C
    int tiles_m, tiles_n;
    uint32_t wait_limit;
    unsigned int* err;
};

__device__ __forceinline__ void raise_timeout(const PairParams& p, volatile int* abort_flag) {
    *abort_flag = 1;
    atomicExch(p.err, ERR_TIMEOUT);
}

// M = 256 E4M3 MMA over the pair: rows 0-127 of A and D in the leader, 128-255
// in the peer; B's first 128 lines from the leader's shared memory, the rest
// from the peer's
__device__ __forceinline__ void mma_f8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, {%5, %5, %5, %5, %5, %5, %5, %5}, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(0u)
                 : "memory");
}

// VEC: B's scales are one per line (1 x 128 blocks), else one per 128 lines
template <bool VEC, bool OUT_BF16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NUM_THREADS, 1)
gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                     const __grid_constant__ CUtensorMap tmC, const PairParams p) {
    // bytes of one fill of a stage and its scale slot, per CTA
    constexpr uint32_t FILL_BYTES = STAGE_BYTES + 512u + (VEC ? PN * 4u : 0u);
    extern __shared__ uint8_t smem_raw[];
    // 1024-byte aligned base, at the same offset in both CTAs
    const uint32_t raw = sm100::smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t* epi_bufs = smem + STAGES * STAGE_BYTES;
    uint8_t* sc_ring = epi_bufs + PROMO_WARPS * EPI_BUF;
    uint64_t* full = reinterpret_cast<uint64_t*>(sc_ring + SC_SLOTS * SC_BYTES);
    uint64_t* empty = full + STAGES;
    uint64_t* pfull = empty + STAGES;
    uint64_t* pempty = pfull + 2;
    uint64_t* drain = pempty + 2;
    uint64_t* peer_done = drain + MMA_WARPS;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(peer_done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile uint32_t* peer_fills = reinterpret_cast<volatile uint32_t*>(tmem_slot + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = sm100::cluster_rank();
    const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);
    const int tiles = p.tiles_m * p.tiles_n;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            sm100::mbar_init(&full[s], 1);
            sm100::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            sm100::mbar_init(&pfull[b], 1);
            sm100::mbar_init(&pempty[b], 2 * PROMO_WARPS);
        }
        for (int w = 0; w < MMA_WARPS; ++w) sm100::mbar_init(&drain[w], 1);
        sm100::mbar_init(peer_done, 1);
        *abort_flag = 0;
        *peer_fills = 0;
        sm100::fence_barrier_init();
        sm100::prefetch_tmap(&tmA);
        sm100::prefetch_tmap(&tmB);
        sm100::prefetch_tmap(&tmC);
    }
    if (warp == 1) {
        sm100::tmem_alloc_pair(tmem_slot, TMEM_COLS);
        sm100::tmem_relinquish_pair();
    }
    sm100::tc_fence_before();
    sm100::cluster_sync();        // both CTAs' barriers initialised before any load signals them
    sm100::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_LEAD));
        if (warp == 0) {
            // -------------------------------------------------------- producer
            if (sm100::elect_one()) {
                int stage = 0, slot = 0;
                uint32_t phase = 0;
                uint32_t fills = 0;
                bool ok = true;
                for (int u = pair; u < tiles && ok; u += pairs) {
                    int tm_, tn_;
                    tile_coords(u, p.tiles_m, p.tiles_n, tm_, tn_);
                    const int n0 = tn_ * PN;
                    const int ma = tm_ * PM + 128 * (int)rank;       // this CTA's rows of A
                    const int nb = n0 + 128 * (int)rank;             // ... and lines of B
                    for (int kc = 0; kc < p.chunks; ++kc) {
                        if (!sm100::mbar_wait(&empty[stage], phase ^ 1u, p.wait_limit, abort_flag)) {
                            raise_timeout(p, abort_flag);
                            ok = false;
                            break;
                        }
                        uint8_t* st = smem + stage * STAGE_BYTES;
                        uint8_t* sc = sc_ring + slot * SC_BYTES;
                        const uint32_t bar = sm100::cluster_addr(&full[stage], 0);
                        if (rank == 0) sm100::mbar_arrive_expect_tx(&full[stage], 2 * FILL_BYTES);
                        sm100::tma_load_2d_pair(st, &tmA, kc * BK, ma, bar);
                        sm100::tma_load_2d_pair(st + A_BYTES, &tmB, kc * BK, nb, bar);
                        sm100::tma_load_2d_pair(sc, &tmSA, ma, kc, bar);
                        if (VEC) sm100::tma_load_2d_pair(sc + 512, &tmSB, n0, kc, bar);
                        ++fills;
                        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                        if (++slot == SC_SLOTS) slot = 0;
                    }
                }
                if (rank == 1) {
                    // report the fills to the leader, whose barriers count their bytes
                    sm100::st_cluster_u32(sm100::cluster_addr(const_cast<uint32_t*>(peer_fills), 0), fills);
                    sm100::mbar_arrive_cluster(sm100::cluster_addr(peer_done, 0));
                } else {
                    // after a timeout the two producers may have filled different
                    // numbers of stages: complete the bookkeeping of every fill
                    // either CTA issued, then wait for the last phase of each stage
                    uint32_t pf = fills;
                    if (sm100::mbar_wait_cluster(peer_done, 0, DRAIN_LIMIT, nullptr)) pf = *peer_fills;
                    else raise_timeout(p, abort_flag);
                    const uint32_t lf = fills;
                    for (uint32_t i = lf; i < pf; ++i) {          // the peer's half only: expect it
                        const uint32_t s = i % STAGES;
                        if (i >= (uint32_t)STAGES)
                            sm100::mbar_wait(&full[s], ((i - STAGES) / STAGES) & 1u, DRAIN_LIMIT, nullptr);
                        sm100::mbar_arrive_expect_tx(&full[s], FILL_BYTES);
                    }
                    for (uint32_t i = pf; i < lf; ++i) {          // this CTA's half only: the peer's never comes
                        const uint32_t s = i % STAGES;
                        if (i >= (uint32_t)STAGES)
                            sm100::mbar_wait(&full[s], ((i - STAGES) / STAGES) & 1u, DRAIN_LIMIT, nullptr);
                        sm100::mbar_complete_tx(&full[s], FILL_BYTES);
                    }
                    const uint32_t last = lf > pf ? lf : pf;
                    for (int s = 0; s < STAGES; ++s)
                        if (last > (uint32_t)s)
                            sm100::mbar_wait(&full[s], ((last - 1u - s) / STAGES) & 1u, DRAIN_LIMIT, nullptr);
                }
            }
            __syncwarp();
        } else if (warp <= MMA_WARPS) {
            // -------------------------------------------------------- MMA issuers (leader)
            if (rank == 0 && sm100::elect_one()) {
                constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(PN >> 3) << 17) | ((uint32_t)(PM >> 4) << 24);
                int stage = 0, pb = 0, turn = 0;
                uint32_t phase = 0, pphase = 0;
                bool ok = true, issued = false;
                for (int u = pair; u < tiles && ok; u += pairs) {
                    for (int kc = 0; kc < p.chunks; ++kc) {
                        if (turn == warp - 1) {
                            if (!sm100::mbar_wait(&full[stage], phase, p.wait_limit, abort_flag) ||
                                !sm100::mbar_wait(&pempty[pb], pphase ^ 1u, p.wait_limit, abort_flag)) {
                                raise_timeout(p, abort_flag);
                                ok = false;
                                break;
                            }
                            sm100::tc_fence_after();
                            const uint32_t st = sm100::smem_u32(smem + stage * STAGE_BYTES);
                            const uint64_t da = sm100::desc_sw128(st), db = sm100::desc_sw128(st + A_BYTES);
                            // descriptor addresses count 16 bytes: 32 bytes of K per step
#pragma unroll
                            for (int kk = 0; kk < BK / 32; ++kk)
                                mma_f8_pair(tmem + PN * pb, da + 2 * kk, db + 2 * kk, idesc, kk > 0 ? 1u : 0u);
                            issued = true;
                            sm100::tc_commit_pair_both(&pfull[pb]);      // both CTAs' rows of the partial ready
                            sm100::tc_commit_pair_both(&empty[stage]);   // both CTAs' stage free
                        }
                        if (++turn == MMA_WARPS) turn = 0;
                        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                        if (++pb == 2) { pb = 0; pphase ^= 1u; }
                    }
                }
                if (issued) {
                    sm100::tc_commit_pair_local(&drain[warp - 1]);
                    sm100::mbar_wait(&drain[warp - 1], 0, DRAIN_LIMIT, nullptr);
                }
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_PROMO));
        // ------------------------------------------------------------ promotion and output
        constexpr int BOX_COLS = OUT_BF16 ? 64 : 32;    // 128 bytes of a row of C
        const int q = warp & 3;                         // TMEM lane quarter of this warp
        const int cg = (warp - 4) >> 2;                 // which COLS columns of the tile
        uint8_t* buf = epi_bufs + (warp - 4) * EPI_BUF;
        const uint32_t buf_s = sm100::smem_u32(buf);
        const uint32_t leader_pempty = sm100::cluster_addr(pempty, 0);
        int slot = 0, pb = 0;
        uint32_t pphase = 0;
        bool ok = true, seen = false;
        for (int u = pair; u < tiles && ok; u += pairs) {
            int tm_, tn_;
            tile_coords(u, p.tiles_m, p.tiles_n, tm_, tn_);
            const int n0 = tn_ * PN + cg * COLS;
            const int row0 = tm_ * PM + 128 * (int)rank + 32 * q;
            // block scales of B: one value per chunk for this warp's 128 columns
            // (columns past N take the last block's; they are not stored)
            const int nblk = VEC ? 0 : min(n0 / 128, (int)p.lpb - 1);
            float sb32 = 0.0f;       // lane l: the scale of chunk 32 (kc / 32) + l
            float2 acc[COLS / 2];
#pragma unroll
            for (int c = 0; c < COLS / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
            for (int kc = 0; kc < p.chunks; ++kc) {
                if (!VEC && (kc & 31) == 0) sb32 = __ldg(p.sb + min(kc + lane, p.chunks - 1) * p.lpb + nblk);
                const float sb = VEC ? 1.0f : __shfl_sync(0xffffffffu, sb32, kc & 31);
                if (!__all_sync(0xffffffffu, seen) &&
                    !__all_sync(0xffffffffu, sm100::mbar_wait(&pfull[pb], pphase, p.wait_limit, abort_flag))) {
                    if (lane == 0) raise_timeout(p, abort_flag);
                    ok = false;
                    break;
                }
                sm100::tc_fence_after();
                const uint32_t base = tmem + ((uint32_t)(32 * q) << 16) + PN * pb + cg * COLS;
                // the chunk's scales landed before its MMAs ran
                const float* sc = reinterpret_cast<const float*>(sc_ring + slot * SC_BYTES);
                const float sa = sc[32 * q + lane];
                float s = VEC ? sa : __fmul_rn(sa, sb);
                const float4* sbv = reinterpret_cast<const float4*>(sc + 128 + cg * COLS);
                // 64 columns in flight at a time
#pragma unroll
                for (int g = 0; g < COLS / 64; ++g) {
                    uint32_t r[2][32];
                    sm100::tmem_ld32(base + 64 * g, r[0]);
                    sm100::tmem_ld32(base + 64 * g + 32, r[1]);
                    sm100::tmem_ld_wait_on(r[0]);
                    sm100::tmem_ld_wait_on(r[1]);
                    if (g == COLS / 64 - 1) {
                        sm100::tc_fence_before();
                        __syncwarp();
                        // the tensor core may refill this partial
                        if (lane == 0) sm100::mbar_arrive_cluster_relaxed(leader_pempty + 8u * (uint32_t)pb);
                        pb ^= 1;
                        if (pb == 0) pphase ^= 1u;
                        seen = sm100::mbar_test_wait(&pfull[pb], pphase);    // the next chunk's, ahead of the sums
                    }
                    const float2 s2 = make_float2(s, s);
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const uint32_t* v = &r[c >> 3][4 * (c & 7)];
                        // the scales' product first: it lies in the range of binary32,
                        // a partial times one of them need not
                        float2 w0 = s2, w1 = s2;
                        if (VEC) {
                            const float4 w = sbv[16 * g + c];
                            w0 = __fmul2_rn(make_float2(w.x, w.y), s2);
                            w1 = __fmul2_rn(make_float2(w.z, w.w), s2);
                        }
                        acc[32 * g + 2 * c] = __ffma2_rn(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), w0,
                                                         acc[32 * g + 2 * c]);
                        acc[32 * g + 2 * c + 1] = __ffma2_rn(make_float2(__uint_as_float(v[2]), __uint_as_float(v[3])),
                                                             w1, acc[32 * g + 2 * c + 1]);
                    }
                }
                if (++slot == SC_SLOTS) slot = 0;
            }
            if (!ok) break;
            // rows row0 .. row0 + 31 (lane = row), columns n0 .. n0 + 127
#pragma unroll
            for (int b = 0; b < COLS / BOX_COLS; ++b) {
                if (p.odd_n && n0 + (b + 1) * BOX_COLS > p.N) {
                    // a TMA store clips a row at 16 bytes, so a box in which C
                    // ends inside a 16-byte chunk is written by the lanes
                    if (row0 + lane < p.M) {
#pragma unroll
                        for (int e = 0; e < BOX_COLS; ++e) {
                            const int i = b * BOX_COLS + e;
                            const float v = (i & 1) ? acc[i / 2].y : acc[i / 2].x;
                            const int64_t at = (int64_t)(row0 + lane) * p.ldc + n0 + i;
                            if (n0 + i < p.N) {
                                if (OUT_BF16) static_cast<__nv_bfloat16*>(p.c)[at] = __float2bfloat16_rn(v);
                                else static_cast<float*>(p.c)[at] = v;
                            }
                        }
                    }
                    continue;
                }
                if (lane == 0) sm100::bulk_wait_read0();        // the previous box has left the buffer
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 8; ++c) {                    // 16-byte chunk c of this lane's row
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (OUT_BF16) {
                            const float2 v = acc[(b * BOX_COLS + 8 * c + 2 * e) / 2];
                            const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
                            w[e] = *reinterpret_cast<const uint32_t*>(&h);
                        } else {
                            const float2 v = acc[(b * BOX_COLS + 4 * c + e) / 2];
                            w[e] = __float_as_uint((e & 1) ? v.y : v.x);
                        }
                    }
                    sm100::st_shared_v4(buf_s + lane * 128 + ((c ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
                }
                sm100::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && row0 < p.M && n0 + b * BOX_COLS < p.N) {
                    sm100::tma_store_2d(&tmC, buf, n0 + b * BOX_COLS, row0);
                    sm100::bulk_commit();
                }
            }
        }
        if (lane == 0) sm100::bulk_wait0();     // this warp's stores are complete before the CTA leaves
        __syncwarp();
    }

    // neither CTA frees its TMEM or leaves while the leader's MMAs or either
    // CTA's loads may still touch it
    sm100::tc_fence_before();
    sm100::cluster_sync();
    if (warp == 1) {
        __syncwarp();
        sm100::tc_fence_after();
        sm100::tmem_dealloc_pair(tmem, TMEM_COLS);
    }
}

// 2-D map over 1 x 128 scales [chunks, lines]: boxes of `box` lines of one chunk, zeros past the last line
bool make_scale_map(CUtensorMap* m, const float* scales, int64_t chunks, int64_t lines, int box) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)lines, (cuuint64_t)chunks};
    cuuint64_t strides[1] = {(cuuint64_t)(lines * 4)};
    cuuint32_t boxes[2] = {(cuuint32_t)box, 1u};
    cuuint32_t estr[2] = {1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float*>(scales), dims, strides, boxes, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool VEC, bool OUT_BF16>
cudaError_t run_pair(const Fp8GemmArgs& g, cudaStream_t s) {
    static PerDeviceOnce setup;
    static int max_pairs[kOnceDevices] = {};
    int dev = 0;
    const cudaError_t attr_err = setup.run([](int d) {
        cudaError_t e = cudaFuncSetAttribute(gemm_fp8_pair_kernel<VEC, OUT_BF16>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * 512);
        cfg.blockDim = dim3(NUM_THREADS);
        cfg.dynamicSmemBytes = SMEM;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, gemm_fp8_pair_kernel<VEC, OUT_BF16>, &cfg);
        if (e != cudaSuccess) return e;
        max_pairs[d] = n;
        return n > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
    }, &dev);
    if (attr_err != cudaSuccess) return attr_err;
    CUtensorMap ta, tb, tsa, tsb, tc;
    const int64_t chunks = (g.K + BK - 1) / BK;
    if (!make_fp8_map(&ta, g.a_codes, g.M, g.K, g.lda, 128) || !make_fp8_map(&tb, g.b_codes, g.N, g.K, g.ldb, 128) ||
        !make_scale_map(&tsa, g.a_scales, chunks, fp8_scale_lines(g.M, 1), 128) ||
        !make_scale_map(&tsb, VEC ? g.b_scales : g.a_scales, chunks, fp8_scale_lines(VEC ? g.N : g.M, 1), PN) ||
        !make_c_map(&tc, g.c, OUT_BF16, g.M, g.N, g.ldc))
        return cudaErrorInvalidValue;
    PairParams p{};
    p.sb = g.b_scales;
    p.lpb = fp8_scale_lines(g.N, g.b_lines);
    p.M = (int)g.M;
    p.N = (int)g.N;
    p.c = g.c;
    p.ldc = g.ldc;
    p.odd_n = (g.N * (OUT_BF16 ? 2 : 4)) % 16 != 0;
    p.chunks = (int)chunks;
    p.tiles_m = (int)((g.M + PM - 1) / PM);
    p.tiles_n = (int)((g.N + PN - 1) / PN);
    p.wait_limit = g.wait_limit;
    p.err = device_error_word();
    const int tiles = p.tiles_m * p.tiles_n;
    const int pairs = tiles < max_pairs[dev] ? tiles : max_pairs[dev];
    gemm_fp8_pair_kernel<VEC, OUT_BF16><<<2 * pairs, NUM_THREADS, SMEM, s>>>(ta, tb, tsa, tsb, tc, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gemm_fp8_pair(const Fp8GemmArgs& g, cudaStream_t s) {
    if (g.b_lines == 1) return g.out_bf16 ? run_pair<true, true>(g, s) : run_pair<true, false>(g, s);
    return g.out_bf16 ? run_pair<false, true>(g, s) : run_pair<false, false>(g, s);
}

}  // namespace fp4
