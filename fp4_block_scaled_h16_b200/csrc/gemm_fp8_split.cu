// gemm_fp8_split.cu -- the FP8 block-scaled GEMM (fp4_fp8_block_gemm) for few
// rows of A, or for outputs too small to fill the GPU with the tiles of
// gemm_fp8_pair.cu:
//
//   C[i, j] = sum_kc sA[kc, i] sB[kc, j or j / 128] P_kc[i, j],
//   P_kc[i, j] = sum_{k in chunk kc of 128} qA[i, k] qB[j, k].
//
// With few tokens the call is bound by reading the weight B once.  So the
// roles are swapped: a tile is 128 lines of B (the M of the MMA, one TMEM lane
// each) by NT rows of A (its N, 16 to 64), two CTAs per SM.  Beyond 64 rows a
// tile is 128 rows of A (the lanes) by 256 lines of B, or 192.  K is split over a
// cluster of up to eight CTAs.  Each 128-K chunk is four kind::f8f6f4 MMAs into
// one of several TMEM buffers; four warps (eight for 256 lines) promote it,
// acc += P (sA sB), in binary32 registers, because an FP32 scale per chunk
// cannot ride in the tensor core's accumulator.  The partial tiles of a cluster are added
// in rank order through distributed shared memory, so the result does not
// depend on timing and no workspace or second launch is needed.
//
// One token, N = 6144, K = 4096: 9.2 us, 25 MB of weights out of HBM at 2750 GB/s,
// and 7.5 us where they lie in L2 (as in the comparisons at the kernel); about
// half of it is the launch, the first loads' latency and the sum over the
// cluster.  333 x 4096 x 14336: 33 us, 1190 TFLOP/s, on 48 clusters of two (the
// GPU holds 45 of three).  A chunk takes 0.42 us there, of which the loads alone
// would take 0.33 (264 MB out of L2 for all tiles, 14 TB/s) and the MMAs alone
// 0.28; 9 us are the launch, the first loads and the sum over the cluster, 2.6 of
// them at the rate of distributed shared memory.  Tiles of 128 x 128 with two CTAs
// per SM: 40 us.
//
// Roles: warp 0 TMA producer, warp 1 MMA issuer (and TMEM), warps 2-5
// promotion; for 256 lines of B two issuers, and promotion by warps 4-11 with
// the registers of warps 0-3 (setmaxnreg).  All warps write the output.  Every wait is bounded; one that runs out
// sets the device error word to FP4_ERR_TIMEOUT, and the CTA lets its copies
// and MMAs in flight land and frees TMEM before it leaves.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "internal.h"
#include "sm100.cuh"

namespace fp4 {

namespace {

constexpr int LANES = 128;               // the tile's side on the TMEM lanes
constexpr int BK = 128;                  // K elements (bytes) per stage: one scale chunk
constexpr int MAX_RANKS = 8;             // CTAs of a cluster, which share a tile's K
constexpr uint32_t DRAIN_LIMIT = 1u << 22;
constexpr unsigned int ERR_TIMEOUT = 7u;

template <int NT>
struct SCfg {
    static constexpr bool WIDE = NT > 64;
    static constexpr int MMA_WARPS = WIDE ? 2 : 1;        // issuers, which take the chunks in turn
    static constexpr int FIRST = WIDE ? 4 : 2;            // first promotion warp
    static constexpr int PROMO_WARPS = WIDE ? 8 : 4;
    static constexpr int THREADS = 32 * (FIRST + PROMO_WARPS);
    static constexpr int WC = NT / (PROMO_WARPS / 4);     // columns of the N side per promotion warp
    static constexpr int CTAS = WIDE ? 1 : 2;             // per SM
    static constexpr uint32_t L_BYTES = LANES * BK;
    static constexpr uint32_t N_BYTES = NT * BK;
    static constexpr uint32_t SN_BYTES = NT * 4;          // scales of the tile's N side
    static constexpr uint32_t SL_BYTES = LANES * 4;       // ... and of its lanes
    static constexpr uint32_t STAGE_BYTES = L_BYTES + N_BYTES;
    static constexpr uint32_t SC_BYTES = SN_BYTES + SL_BYTES;
    static constexpr uint32_t EXTRA = 1024 + 512;         // alignment, barriers
    static constexpr int PBUF = WIDE ? 2 : 4;             // TMEM buffers of NT columns
    // Scales have a longer ring, without barriers of its own, so that a stage is
    // free when its MMAs are done: they were issued once the promotion had read the
    // partial PBUF chunks before, and so was past the scales of the chunk before that
    // (their values are in its sums by then: mbar_arrive_cluster_relaxed).
    static constexpr int STAGES =
        (int)((232448u / CTAS - 1024u - EXTRA - (PBUF + 1) * SC_BYTES) / (STAGE_BYTES + SC_BYTES));
    static constexpr int SC_SLOTS = STAGES + PBUF + 1;
    // the partial tile, over the stages: rows of C (NT lines of A, or 128), padded
    // so that eight rows' 16-byte chunks differ in bank
    static constexpr int RED_PITCH = (WIDE ? NT : LANES) + 4;
    static constexpr uint32_t RED_BYTES = (WIDE ? LANES : NT) * RED_PITCH * 4;
    static constexpr uint32_t SMEM = STAGES * STAGE_BYTES + SC_SLOTS * SC_BYTES + EXTRA;
    static constexpr uint32_t PSTRIDE = WIDE ? 256 : NT;    // TMEM columns from buffer to buffer
    static constexpr uint32_t TMEM_COLS = PBUF * PSTRIDE;
    static_assert(RED_BYTES <= STAGES * STAGE_BYTES, "the partial tile fits over the ring");
    static_assert(TMEM_COLS >= 32 && TMEM_COLS * CTAS <= 512, "TMEM of an SM's CTAs");
};

struct SplitParams {
    const float* sa;          // [chunks, lpa]
    const float* sb;          // [chunks, lpb]
    int64_t lpa, lpb;
    void* c;
    int64_t ldc;
    int M, N, chunks;
    int lane_tile0, n_tile0;  // the first tile of a launch
    uint32_t wait_limit;
    unsigned int* err;
};

__device__ __forceinline__ void raise_timeout(const SplitParams& p, volatile int* abort_flag) {
    *abort_flag = 1;
    atomicExch(p.err, ERR_TIMEOUT);
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t caddr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(caddr) : "memory");
    return v;
}

// four columns of C from element `at` (a multiple of 4 columns into a row), `n` of them inside C
template <bool OUT_BF16>
__device__ __forceinline__ void put4(void* c, int64_t at, const float4& v, int n) {
    const float x[4] = {v.x, v.y, v.z, v.w};
    if (OUT_BF16) {
        __nv_bfloat16* d = static_cast<__nv_bfloat16*>(c) + at;
        if (n >= 4) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
            *reinterpret_cast<uint2*>(d) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                      *reinterpret_cast<const uint32_t*>(&hi));
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (e < n) d[e] = __float2bfloat16_rn(x[e]);
        }
    } else {
        float* d = static_cast<float*>(c) + at;
        if (n >= 4) {
            *reinterpret_cast<float4*>(d) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (e < n) d[e] = x[e];
        }
    }
}

// barrier of all threads, reached from different branches
template <int THREADS>
__device__ __forceinline__ void all_roles() {
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// The sum over the ranks of a cluster of their partial tiles `red`, in rank order,
// for the rows of C that are this rank's.  RANKS is a bound on `ranks`; eight loads
// are in flight per thread, because a load from another CTA waits long
// (one by one 333 x 4096 x 512 takes 9.6 us, 9.0 this way).
template <int SPANS, int PITCH, int WARPS, bool OUT_BF16>
struct Reduce {
    template <int RANKS>
    static __device__ __forceinline__ void rows(const SplitParams& p, const float* red, int rank, int ranks, int rows,
                                                int cols, int64_t at0) {
        constexpr int U = 8 / RANKS;                 // (row, span) steps of a warp at a time
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        for (int i = warp; rank + i / SPANS * ranks < rows; i += U * WARPS) {
            float4 part[U][RANKS];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = i + u * WARPS, row = rank + k / SPANS * ranks, col = k % SPANS * 128 + 4 * lane;
                const bool in = row < rows && col < cols;
                const float* at = red + row * PITCH + col;
#pragma unroll
                for (int r = 0; r < RANKS; ++r) {
                    if (!in || r >= ranks) continue;
                    if (RANKS == 1) part[u][r] = *reinterpret_cast<const float4*>(at);
                    else part[u][r] = ld_cluster_v4(sm100::cluster_addr(at, (uint32_t)r));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = i + u * WARPS, row = rank + k / SPANS * ranks, col = k % SPANS * 128 + 4 * lane;
                if (row >= rows || col >= cols) continue;
                float4 v = part[u][0];
#pragma unroll
                for (int r = 1; r < RANKS; ++r)
                    if (r < ranks) {
                        v.x += part[u][r].x;
                        v.y += part[u][r].y;
                        v.z += part[u][r].z;
                        v.w += part[u][r].w;
                    }
                put4<OUT_BF16>(p.c, at0 + (int64_t)row * p.ldc + col, v, cols - col);
            }
        }
    }
};

// SWAP: lanes are lines of B and the N side rows of A, else the reverse.
// VEC: B's scales are one per line (1 x 128 blocks), else one per 128 lines.
template <int NT, bool SWAP, bool VEC, bool OUT_BF16>
__global__ void __launch_bounds__(SCfg<NT>::THREADS, SCfg<NT>::CTAS)
gemm_fp8_split_kernel(const __grid_constant__ CUtensorMap tmL, const __grid_constant__ CUtensorMap tmN,
                      const SplitParams p) {
    using G = SCfg<NT>;
    constexpr bool LANE_VEC = !SWAP || VEC;          // a scale per lane
    constexpr bool N_VEC = SWAP || VEC;              // a scale per column of the N side
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = sm100::smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t* sc_ring = smem + G::STAGES * G::STAGE_BYTES;
    uint64_t* full = reinterpret_cast<uint64_t*>(sc_ring + G::SC_SLOTS * G::SC_BYTES);
    uint64_t* empty = full + G::STAGES;
    uint64_t* pfull = empty + G::STAGES;
    uint64_t* pempty = pfull + G::PBUF;
    uint64_t* drain = pempty + G::PBUF;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + G::MMA_WARPS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)blockIdx.x, ranks = (int)gridDim.x;      // the cluster spans the x dimension
    const int l0 = (p.lane_tile0 + (int)blockIdx.y) * LANES, t0 = (p.n_tile0 + (int)blockIdx.z) * NT;
    const int kc0 = (int)((int64_t)p.chunks * rank / ranks), kc1 = (int)((int64_t)p.chunks * (rank + 1) / ranks);

    // one thread's loads of chunk kc
    auto fill = [&](int kc, int stage, int slot) {
        const int64_t lpl = SWAP ? p.lpb : p.lpa, lpn = SWAP ? p.lpa : p.lpb;
        // lines past M and N lie in the scale rows' padding to 128
        const uint32_t sn_bytes = !N_VEC ? 0u : (uint32_t)min((int64_t)NT, lpn - t0) * 4u;
        uint8_t* st = smem + stage * G::STAGE_BYTES;
        uint8_t* sc = sc_ring + slot * G::SC_BYTES;
        sm100::mbar_arrive_expect_tx(&full[stage],
                                     G::L_BYTES + G::N_BYTES + sn_bytes + (LANE_VEC ? G::SL_BYTES : 0u));
        sm100::tma_load_2d(st, &tmL, kc * BK, l0, &full[stage]);
        sm100::tma_load_2d(st + G::L_BYTES, &tmN, kc * BK, t0, &full[stage]);
        if (N_VEC) sm100::bulk_load(sc, (SWAP ? p.sa : p.sb) + kc * lpn + t0, sn_bytes, &full[stage]);
        if (LANE_VEC) sm100::bulk_load(sc + G::SN_BYTES, (SWAP ? p.sb : p.sa) + kc * lpl + l0, G::SL_BYTES, &full[stage]);
    };
    // the first stages are on their way before TMEM is allocated (one token, N =
    // 6144, K = 4096 7.5 -> 7.3 us); with 256 lines of B that costs the promotion
    // registers (333 x 4096 x 14336 32.7 -> 34.3 us)
    const int ahead = G::WIDE ? 0 : min(G::STAGES, kc1 - kc0);

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::STAGES; ++s) {
            sm100::mbar_init(&full[s], 1);
            sm100::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < G::PBUF; ++b) {
            sm100::mbar_init(&pfull[b], 1);
            sm100::mbar_init(&pempty[b], G::PROMO_WARPS);
        }
        for (int w = 0; w < G::MMA_WARPS; ++w) sm100::mbar_init(&drain[w], 1);
        *abort_flag = 0;
        sm100::fence_barrier_init();
        for (int k = 0; k < ahead; ++k) fill(kc0 + k, k, k);
    }
    if (warp == 1) {
        sm100::tmem_alloc(tmem_slot, G::TMEM_COLS);
        sm100::tmem_relinquish();
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    float* red = reinterpret_cast<float*>(smem);             // the partial tile: [rows of C][columns]
    const int rows = min(SWAP ? NT : LANES, p.M - (SWAP ? t0 : l0));
    const int cols = min(SWAP ? LANES : NT, p.N - (SWAP ? l0 : t0));
    if constexpr (G::WIDE) {         // 384 threads x 168 registers at launch = 128 x 64 + 256 x 216
        if (warp < G::FIRST) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    }
    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (sm100::elect_one()) {
            int stage = ahead % G::STAGES, slot = ahead;
            uint32_t phase = ahead / G::STAGES, fills = ahead;
            for (int kc = kc0 + ahead; kc < kc1; ++kc) {
                if (!sm100::mbar_wait(&empty[stage], phase ^ 1u, p.wait_limit, abort_flag)) {
                    raise_timeout(p, abort_flag);
                    break;
                }
                fill(kc, stage, slot);
                ++fills;
                if (++slot == G::SC_SLOTS) slot = 0;
                if (++stage == G::STAGES) { stage = 0; phase ^= 1u; }
            }
            for (int s = 0; s < G::STAGES; ++s)
                if (fills > (uint32_t)s)
                    sm100::mbar_wait(&full[s], ((fills - 1u - s) / G::STAGES) & 1u, DRAIN_LIMIT, nullptr);
        }
        __syncwarp();
    } else if (warp < G::FIRST) {
        // ------------------------------------------------------------ MMA issuers
        if (warp <= G::MMA_WARPS && sm100::elect_one()) {
            int stage = 0, pb = 0, turn = 0;
            uint32_t phase = 0, pphase = 0;
            bool issued = false;
            constexpr uint32_t idesc = sm100::idesc_f8_e4m3(NT);
            for (int kc = kc0; kc < kc1; ++kc) {
                if (G::MMA_WARPS == 1 || turn == warp - 1) {
                    if (!sm100::mbar_wait(&full[stage], phase, p.wait_limit, abort_flag) ||
                        !sm100::mbar_wait(&pempty[pb], pphase ^ 1u, p.wait_limit, abort_flag)) {
                        raise_timeout(p, abort_flag);
                        break;
                    }
                    sm100::tc_fence_after();
                    const uint32_t st = sm100::smem_u32(smem + stage * G::STAGE_BYTES);
                    // descriptor addresses count 16 bytes: 32 bytes of K per step
                    const uint64_t dl = sm100::desc_sw128(st), dn = sm100::desc_sw128(st + G::L_BYTES);
#pragma unroll
                    for (int kk = 0; kk < BK / 32; ++kk)
                        sm100::mma_f8(tmem + G::PSTRIDE * pb, dl + 2 * kk, dn + 2 * kk, idesc, kk > 0 ? 1u : 0u);
                    issued = true;
                    sm100::tc_commit(&pfull[pb]);
                    sm100::tc_commit(&empty[stage]);
                }
                if (++turn == G::MMA_WARPS) turn = 0;
                if (++stage == G::STAGES) { stage = 0; phase ^= 1u; }
                if (++pb == G::PBUF) { pb = 0; pphase ^= 1u; }
            }
            if (issued) {
                sm100::tc_commit(&drain[warp - 1]);
                sm100::mbar_wait(&drain[warp - 1], 0, DRAIN_LIMIT, nullptr);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ promotion
        const int q = warp & 3;                     // TMEM lane quarter of this warp
        const int n0 = (warp - G::FIRST) / 4 * G::WC;      // its first column of the N side
        float2 acc[G::WC / 2];
#pragma unroll
        for (int c = 0; c < G::WC / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
        int slot = 0, pb = 0;
        uint32_t pphase = 0;
        bool seen = false;
        // columns past N take the last block's scale; they are not stored
        const float* sb_block = p.sb + (VEC ? 0 : min((int64_t)(SWAP ? l0 : t0 + n0) / 128, p.lpb - 1));
        float sb32 = 0.0f;                          // lane l: the block scale of chunk kc0 + 32 i + l
        for (int kc = kc0; kc < kc1; ++kc) {
            if (!VEC && ((kc - kc0) & 31) == 0) sb32 = __ldg(sb_block + min(kc + lane, kc1 - 1) * p.lpb);
            if (!__all_sync(0xffffffffu, seen) &&
                !__all_sync(0xffffffffu, sm100::mbar_wait(&pfull[pb], pphase, p.wait_limit, abort_flag))) {
                if (lane == 0) raise_timeout(p, abort_flag);
                break;
            }
            sm100::tc_fence_after();
            // the chunk's scales landed before its MMAs ran
            const float* sn = reinterpret_cast<const float*>(sc_ring + slot * G::SC_BYTES);
            float s = LANE_VEC ? sn[NT + 32 * q + lane] : 1.0f;
            if (!VEC) s = __fmul_rn(s, __shfl_sync(0xffffffffu, sb32, (kc - kc0) & 31));
            const uint32_t base = tmem + ((uint32_t)(32 * q) << 16) + G::PSTRIDE * pb + n0;
            constexpr int W = G::WC < 32 ? 16 : 32;             // columns per TMEM load
            constexpr int F = G::WC % 96 == 0 ? 3 : (G::WC > W ? 2 : 1);   // loads in flight
#pragma unroll
            for (int c0 = 0; c0 < G::WC; c0 += F * W) {
                uint32_t r[F][W];
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    if constexpr (W == 16) sm100::tmem_ld16(base + c0 + f * W, r[f]);
                    else sm100::tmem_ld32(base + c0 + f * W, r[f]);
                }
#pragma unroll
                for (int f = 0; f < F; ++f) sm100::tmem_ld_wait_on(r[f]);
                if (c0 + F * W == G::WC) {
                    sm100::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) sm100::mbar_arrive_cluster_relaxed(sm100::smem_u32(&pempty[pb]));
                    if (++pb == G::PBUF) { pb = 0; pphase ^= 1u; }
                    seen = sm100::mbar_test_wait(&pfull[pb], pphase);    // the next chunk's, ahead of the sums
                }
#pragma unroll
                for (int c = 0; c < F * W; c += 4) {
                    float2 w0 = make_float2(s, s), w1 = w0;
                    if (N_VEC) {
                        const float4 v = *reinterpret_cast<const float4*>(sn + n0 + c0 + c);
                        w0 = __fmul2_rn(make_float2(v.x, v.y), w0);
                        w1 = __fmul2_rn(make_float2(v.z, v.w), w1);
                    }
                    const uint32_t* v = &r[c / W][c % W];
                    float2* d = &acc[(c0 + c) / 2];
                    d[0] = __ffma2_rn(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), w0, d[0]);
                    d[1] = __ffma2_rn(make_float2(__uint_as_float(v[2]), __uint_as_float(v[3])), w1, d[1]);
                }
            }
            if (++slot == G::SC_SLOTS) slot = 0;
        }
        // every load and MMA of this CTA has completed once all roles are here, so
        // the partial tile may take the ring's place
        sm100::tc_fence_before();
        all_roles<G::THREADS>();
        const int l = 32 * q + lane;
        if (SWAP) {
#pragma unroll
            for (int c = 0; c < G::WC; ++c)
                if (c < rows) red[c * G::RED_PITCH + l] = (c & 1) ? acc[c / 2].y : acc[c / 2].x;
        } else if (l < rows) {
#pragma unroll
            for (int c = 0; c < G::WC; c += 4)
                *reinterpret_cast<float4*>(red + l * G::RED_PITCH + n0 + c) =
                    make_float4(acc[c / 2].x, acc[c / 2].y, acc[c / 2 + 1].x, acc[c / 2 + 1].y);
        }
    }
    if (warp < G::FIRST) {
        sm100::tc_fence_before();
        all_roles<G::THREADS>();
    }
    if (ranks > 1) sm100::cluster_sync();
    else __syncthreads();
    // the ranks of a cluster share the rows of C; a warp takes 128 columns of a
    // row at a time, four per thread
    const int64_t at0 = (int64_t)(SWAP ? t0 : l0) * p.ldc + (SWAP ? l0 : t0);
    using Red = Reduce<(SWAP ? LANES : NT + 127) / 128, G::RED_PITCH, G::THREADS / 32, OUT_BF16>;
    if (ranks == 1) Red::template rows<1>(p, red, rank, ranks, rows, cols, at0);
    else if (ranks == 2) Red::template rows<2>(p, red, rank, ranks, rows, cols, at0);
    else if (ranks <= 4) Red::template rows<4>(p, red, rank, ranks, rows, cols, at0);
    else Red::template rows<8>(p, red, rank, ranks, rows, cols, at0);
    if (ranks > 1) sm100::cluster_sync();                    // no CTA leaves while another reads its tile
    if (warp == 1) {
        __syncwarp();
        sm100::tc_fence_after();
        sm100::tmem_dealloc(tmem, G::TMEM_COLS);
    }
}

// launches the product, or only tells what it would cost
template <int NT, bool SWAP, bool VEC, bool OUT_BF16>
cudaError_t run_split(const Fp8GemmArgs& g, cudaStream_t s, int64_t* cost = nullptr) {
    using G = SCfg<NT>;
    static PerDeviceOnce setup;
    static int max_clusters[kOnceDevices][MAX_RANKS + 1] = {};   // resident at once, one CTA per SM, by cluster size
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(G::THREADS);
    cfg.dynamicSmemBytes = G::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int dev = 0;
    const cudaError_t attr_err = setup.run([&](int d) {
        cudaError_t e = cudaFuncSetAttribute(gemm_fp8_split_kernel<NT, SWAP, VEC, OUT_BF16>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)G::SMEM);
        for (int r = 1; r <= MAX_RANKS && e == cudaSuccess; ++r) {
            attr.val.clusterDim.x = (unsigned)r;
            cfg.gridDim = dim3((unsigned)r * 512);
            e = cudaOccupancyMaxActiveClusters(&max_clusters[d][r], gemm_fp8_split_kernel<NT, SWAP, VEC, OUT_BF16>, &cfg);
        }
        return e;
    }, &dev);
    if (attr_err != cudaSuccess) return attr_err;
    const int64_t lanes = SWAP ? g.N : g.M, cols = SWAP ? g.M : g.N;
    const int64_t tiles = ((lanes + LANES - 1) / LANES) * ((cols + NT - 1) / NT);
    const int64_t chunks = (g.K + BK - 1) / BK;
    // K is split as far as all clusters are resident at once, with two chunks per
    // CTA at least: one token, N = 6144, K = 4096 takes 14.1, 9.5, 8.4, 7.7 and 7.3
    // us with 1 to 5 ranks, and 11.1 with 6, which do not all fit
    int ranks = 1;
    for (int r = 2; r <= MAX_RANKS; ++r)
        if (tiles <= G::CTAS * max_clusters[dev][r] && chunks >= 2 * r) ranks = r;
    if (cost) {                             // columns of all chunks that the busiest SM promotes
        *cost = (tiles * ranks + num_sms() - 1) / num_sms() * ((chunks + ranks - 1) / ranks) * NT;
        return cudaSuccess;
    }
    CUtensorMap ta, tb;
    if (!make_fp8_map(&ta, g.a_codes, g.M, g.K, g.lda, SWAP ? NT : LANES) ||
        !make_fp8_map(&tb, g.b_codes, g.N, g.K, g.ldb, SWAP ? LANES : NT))
        return cudaErrorInvalidValue;
    SplitParams p{};
    p.sa = g.a_scales;
    p.sb = g.b_scales;
    p.lpa = fp8_scale_lines(g.M, 1);
    p.lpb = fp8_scale_lines(g.N, g.b_lines);
    p.c = g.c;
    p.ldc = g.ldc;
    p.M = (int)g.M;
    p.N = (int)g.N;
    p.chunks = (int)chunks;
    p.wait_limit = g.wait_limit;
    p.err = device_error_word();
    attr.val.clusterDim.x = (unsigned)ranks;
    // one launch, unless a side has more tiles than a grid has lines
    constexpr int MAX_LINES = 65535;
    const int lane_tiles = (int)((lanes + LANES - 1) / LANES), n_tiles = (int)((cols + NT - 1) / NT);
    for (p.n_tile0 = 0; p.n_tile0 < n_tiles; p.n_tile0 += MAX_LINES)
        for (p.lane_tile0 = 0; p.lane_tile0 < lane_tiles; p.lane_tile0 += MAX_LINES) {
            cfg.gridDim = dim3((unsigned)ranks, (unsigned)min(lane_tiles - p.lane_tile0, MAX_LINES),
                               (unsigned)min(n_tiles - p.n_tile0, MAX_LINES));
            const cudaError_t e = cudaLaunchKernelEx(&cfg, gemm_fp8_split_kernel<NT, SWAP, VEC, OUT_BF16>,
                                                     SWAP ? tb : ta, SWAP ? ta : tb, p);
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

template <int NT, bool SWAP>
cudaError_t run_nt(const Fp8GemmArgs& g, cudaStream_t s) {
    if (g.b_lines == 1)
        return g.out_bf16 ? run_split<NT, SWAP, true, true>(g, s) : run_split<NT, SWAP, true, false>(g, s);
    return g.out_bf16 ? run_split<NT, SWAP, false, true>(g, s) : run_split<NT, SWAP, false, false>(g, s);
}

// With 1 x 128 blocks of B the promotion, one product per element more, bounds a
// chunk, not its loads, so tiles of 192 lines gain where they spread over more SMs:
// 333 x 4096 x 14336 44.1 -> 36.2 us, 512 x 6144 x 4096 28.0 -> 23.3, but 300 x
// 6144 x 4096 20.2 -> 23.8 where they leave no room to split K.  (With 128 x 128
// blocks they load more for the same product: 33.2 -> 36.3 us for the first.)
template <bool OUT_BF16>
cudaError_t run_vec(const Fp8GemmArgs& g, cudaStream_t s) {
    int64_t c192 = 0, c256 = 0;
    cudaError_t e = run_split<192, false, true, OUT_BF16>(g, s, &c192);
    if (e == cudaSuccess) e = run_split<256, false, true, OUT_BF16>(g, s, &c256);
    if (e != cudaSuccess) return e;
    return 8 * c192 <= 9 * c256 ? run_split<192, false, true, OUT_BF16>(g, s) : run_split<256, false, true, OUT_BF16>(g, s);
}

}  // namespace

cudaError_t launch_gemm_fp8_split(const Fp8GemmArgs& g, cudaStream_t s) {
    if (g.M <= 16) return run_nt<16, true>(g, s);
    if (g.M <= 32) return run_nt<32, true>(g, s);
    if (g.M <= 64) return run_nt<64, true>(g, s);
    if (g.b_lines == 1) return g.out_bf16 ? run_vec<true>(g, s) : run_vec<false>(g, s);
    return g.out_bf16 ? run_split<256, false, false, true>(g, s) : run_split<256, false, false, false>(g, s);
}

}  // namespace fp4
