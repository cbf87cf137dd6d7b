// gemm_fp8_split.cu -- the FP8 block-scaled GEMM (fp4_fp8_block_gemm) for few
// rows of A, or for outputs too small to fill the GPU with the tiles of
// gemm_fp8_pair.cu:
//
//   C[i, j] = sum_kc sA[kc, i] sB[kc, j or j / 128] P_kc[i, j],
//   P_kc[i, j] = sum_{k in chunk kc of 128} qA[i, k] qB[j, k].
//
// With few tokens the call is bound by reading the weight B once.  So the
// roles are swapped: a tile is 128 lines of B (the M of the MMA, one TMEM lane
// each) by NT rows of A (its N, 16 to 128), K is split over a cluster of S
// CTAs, and each CTA streams its share of B through a ring of 16 KB boxes, all
// of them in flight at once for the usual shares.  Each 128-K chunk is four
// kind::f8f6f4 MMAs into one of several TMEM buffers; four warps (one per lane
// quarter) promote it, acc += P (sA sB), in binary32 registers, because an FP32
// scale per chunk cannot ride in the tensor core's accumulator.  The S partial
// tiles are then added in rank order through distributed shared memory, so the
// result does not depend on timing and no workspace or second launch is needed.
//
// Roles (192 threads): warp 0 TMA producer, warp 1 MMA issuer (and TMEM),
// warps 2-5 promotion and output.  Every wait is bounded; one that runs out
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

constexpr int LINES = 128;               // lines of B per tile
constexpr int BK = 128;                  // K elements (bytes) per stage: one scale chunk
constexpr int NUM_THREADS = 192;
constexpr int PROMO_WARPS = 4;
constexpr uint32_t DRAIN_LIMIT = 1u << 22;
constexpr unsigned int ERR_TIMEOUT = 7u;

template <int NT>
struct SCfg {
    static constexpr uint32_t B_BYTES = LINES * BK;
    static constexpr uint32_t A_BYTES = NT * BK;
    static constexpr uint32_t SA_BYTES = NT * 4;          // scales of the A rows
    static constexpr uint32_t SB_BYTES = LINES * 4;       // scales of the B lines (1 x 128 blocks)
    static constexpr uint32_t STAGE_BYTES = (B_BYTES + A_BYTES + SA_BYTES + SB_BYTES + 1023) / 1024 * 1024;
    static constexpr int FIT = (int)((232448u - 1024u - 512u) / STAGE_BYTES);
    static constexpr int STAGES = FIT > 8 ? 8 : FIT;
    static constexpr uint32_t RED_BYTES = NT * LINES * 4; // this CTA's partial tile, over the stages
    static constexpr uint32_t SMEM = STAGES * STAGE_BYTES + 1024 + 512;
    static constexpr int PBUF = 4;                        // TMEM buffers of NT columns
    static constexpr uint32_t TMEM_COLS = PBUF * NT < 32 ? 32 : PBUF * NT;
    static_assert(RED_BYTES <= STAGES * STAGE_BYTES, "the partial tile fits over the ring");
    static_assert((TMEM_COLS & (TMEM_COLS - 1)) == 0 && TMEM_COLS <= 512, "TMEM allocation");
};

struct SplitParams {
    const float* sa;          // [chunks, lpa]
    const float* sb;          // [chunks, lpb]
    int64_t lpa, lpb;
    void* c;
    int64_t ldc;
    int M, N, chunks;
    uint32_t wait_limit;
    unsigned int* err;
};

__device__ __forceinline__ void raise_timeout(const SplitParams& p, volatile int* abort_flag) {
    *abort_flag = 1;
    atomicExch(p.err, ERR_TIMEOUT);
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t caddr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(caddr) : "memory");
    return v;
}

template <bool OUT_BF16>
__device__ __forceinline__ void put(void* c, int64_t at, float v) {
    if (OUT_BF16) static_cast<__nv_bfloat16*>(c)[at] = __float2bfloat16_rn(v);
    else static_cast<float*>(c)[at] = v;
}

// VEC: B's scales are one per line (1 x 128 blocks), else one per 128 lines
template <int NT, bool VEC, bool OUT_BF16>
__global__ void __launch_bounds__(NUM_THREADS, 1)
gemm_fp8_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const SplitParams p) {
    using G = SCfg<NT>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = sm100::smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::STAGES * G::STAGE_BYTES);
    uint64_t* empty = full + G::STAGES;
    uint64_t* pfull = empty + G::STAGES;
    uint64_t* pempty = pfull + G::PBUF;
    uint64_t* drain = pempty + G::PBUF;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)blockIdx.x, ranks = (int)gridDim.x;      // the cluster spans the x dimension
    const int n0 = (int)blockIdx.y * LINES, m0 = (int)blockIdx.z * NT;
    const int kc0 = (int)((int64_t)p.chunks * rank / ranks), kc1 = (int)((int64_t)p.chunks * (rank + 1) / ranks);

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::STAGES; ++s) {
            sm100::mbar_init(&full[s], 1);
            sm100::mbar_init(&empty[s], 1 + PROMO_WARPS);   // the MMAs, and the readers of the scales
        }
        for (int b = 0; b < G::PBUF; ++b) {
            sm100::mbar_init(&pfull[b], 1);
            sm100::mbar_init(&pempty[b], PROMO_WARPS);
        }
        sm100::mbar_init(drain, 1);
        *abort_flag = 0;
        sm100::fence_barrier_init();
        sm100::prefetch_tmap(&tmA);
        sm100::prefetch_tmap(&tmB);
    }
    if (warp == 1) {
        sm100::tmem_alloc(tmem_slot, G::TMEM_COLS);
        sm100::tmem_relinquish();
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    float acc[NT];
    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (sm100::elect_one()) {
            int stage = 0;
            uint32_t phase = 0, fills = 0;
            for (int kc = kc0; kc < kc1; ++kc) {
                if (!sm100::mbar_wait(&empty[stage], phase ^ 1u, p.wait_limit, abort_flag)) {
                    raise_timeout(p, abort_flag);
                    break;
                }
                uint8_t* st = smem + stage * G::STAGE_BYTES;
                sm100::mbar_arrive_expect_tx(&full[stage],
                                             G::B_BYTES + G::A_BYTES + G::SA_BYTES + (VEC ? G::SB_BYTES : 0u));
                sm100::tma_load_2d(st, &tmB, kc * BK, n0, &full[stage]);
                sm100::tma_load_2d(st + G::B_BYTES, &tmA, kc * BK, m0, &full[stage]);
                // lines past M and N lie in the scale rows' padding to 128
                sm100::bulk_load(st + G::B_BYTES + G::A_BYTES, p.sa + kc * p.lpa + m0, G::SA_BYTES, &full[stage]);
                if (VEC)
                    sm100::bulk_load(st + G::B_BYTES + G::A_BYTES + G::SA_BYTES, p.sb + kc * p.lpb + n0, G::SB_BYTES,
                                     &full[stage]);
                ++fills;
                if (++stage == G::STAGES) { stage = 0; phase ^= 1u; }
            }
            for (int s = 0; s < G::STAGES; ++s)
                if (fills > (uint32_t)s)
                    sm100::mbar_wait(&full[s], ((fills - 1u - s) / G::STAGES) & 1u, DRAIN_LIMIT, nullptr);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (sm100::elect_one()) {
            int stage = 0, pb = 0;
            uint32_t phase = 0, pphase = 0;
            bool issued = false;
            constexpr uint32_t idesc = sm100::idesc_f8_e4m3(NT);
            for (int kc = kc0; kc < kc1; ++kc) {
                if (!sm100::mbar_wait(&full[stage], phase, p.wait_limit, abort_flag) ||
                    !sm100::mbar_wait(&pempty[pb], pphase ^ 1u, p.wait_limit, abort_flag)) {
                    raise_timeout(p, abort_flag);
                    break;
                }
                sm100::tc_fence_after();
                const uint32_t st = sm100::smem_u32(smem + stage * G::STAGE_BYTES);
#pragma unroll
                for (int kk = 0; kk < BK / 32; ++kk)
                    sm100::mma_f8(tmem + NT * pb, sm100::desc_sw128(st + 32 * kk),
                                  sm100::desc_sw128(st + G::B_BYTES + 32 * kk), idesc, kk > 0 ? 1u : 0u);
                issued = true;
                sm100::tc_commit(&empty[stage]);
                sm100::tc_commit(&pfull[pb]);
                if (++stage == G::STAGES) { stage = 0; phase ^= 1u; }
                if (++pb == G::PBUF) { pb = 0; pphase ^= 1u; }
            }
            if (issued) {
                sm100::tc_commit(drain);
                sm100::mbar_wait(drain, 0, DRAIN_LIMIT, nullptr);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ promotion
        const int q = warp & 3;                     // TMEM lane quarter of this warp
#pragma unroll
        for (int c = 0; c < NT; ++c) acc[c] = 0.0f;
        int stage = 0, pb = 0;
        uint32_t phase = 0, pphase = 0;
        const float* sb_block = p.sb + (VEC ? 0 : n0 / 128);
        float sb_next = (VEC || kc0 >= kc1) ? 0.0f : __ldg(sb_block + kc0 * p.lpb);
        for (int kc = kc0; kc < kc1; ++kc) {
            float sb = sb_next;
            if (!VEC && kc + 1 < kc1) sb_next = __ldg(sb_block + (kc + 1) * p.lpb);
            const bool ok = sm100::mbar_wait(&pfull[pb], pphase, p.wait_limit, abort_flag) &&
                            sm100::mbar_wait(&full[stage], phase, p.wait_limit, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) raise_timeout(p, abort_flag);
                break;
            }
            sm100::tc_fence_after();
            const float* sa = reinterpret_cast<const float*>(smem + stage * G::STAGE_BYTES + G::B_BYTES + G::A_BYTES);
            if (VEC) sb = sa[NT + 32 * q + lane];
            const uint32_t base = tmem + ((uint32_t)(32 * q) << 16) + NT * pb;
#pragma unroll
            for (int c0 = 0; c0 < NT; c0 += 16) {
                uint32_t r[16];
                sm100::tmem_ld16(base + c0, r);
                sm100::tmem_ld_wait_on(r);
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    acc[c0 + c] = __fmaf_rn(__uint_as_float(r[c]), __fmul_rn(sa[c0 + c], sb), acc[c0 + c]);
            }
            sm100::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                sm100::mbar_arrive(&pempty[pb]);
                sm100::mbar_arrive(&empty[stage]);
            }
            if (++stage == G::STAGES) { stage = 0; phase ^= 1u; }
            if (++pb == G::PBUF) { pb = 0; pphase ^= 1u; }
        }
    }

    // every load and MMA of this CTA has completed once all roles are here, so
    // the partial tile may take the ring's place
    sm100::tc_fence_before();
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);             // [NT][128]
    const int tokens = min(NT, p.M - m0);
    if (warp >= 2) {
        const int q = warp & 3;
        const int line = 32 * q + lane;
        const int64_t at = (int64_t)m0 * p.ldc + n0 + line;
        if (ranks == 1) {
            if (n0 + line < p.N) {
#pragma unroll
                for (int c = 0; c < NT; ++c)
                    if (c < tokens) put<OUT_BF16>(p.c, at + c * p.ldc, acc[c]);
            }
        } else {
#pragma unroll
            for (int c = 0; c < NT; ++c)
                if (c < tokens) red[c * LINES + line] = acc[c];
        }
    }
    if (ranks > 1) {
        sm100::cluster_sync();
        if (warp >= 2) {
            const int line = 32 * (warp & 3) + lane;
            const bool in_n = n0 + line < p.N;
            for (int c = rank; c < tokens; c += ranks) {
                float v = 0.0f;
                for (int r = 0; r < ranks; ++r)
                    v += ld_cluster_f32(sm100::cluster_addr(red + c * LINES + line, (uint32_t)r));
                if (in_n) put<OUT_BF16>(p.c, (int64_t)(m0 + c) * p.ldc + n0 + line, v);
            }
        }
        sm100::cluster_sync();                               // no CTA leaves while another reads its tile
    }
    if (warp == 1) {
        __syncwarp();
        sm100::tc_fence_after();
        sm100::tmem_dealloc(tmem, G::TMEM_COLS);
    }
}

template <int NT, bool VEC, bool OUT_BF16>
cudaError_t run_split(const Fp8GemmArgs& g, int ranks, cudaStream_t s) {
    using G = SCfg<NT>;
    static PerDeviceOnce setup;
    const cudaError_t attr_err = setup.run([](int) {
        return cudaFuncSetAttribute(gemm_fp8_split_kernel<NT, VEC, OUT_BF16>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)G::SMEM);
    });
    if (attr_err != cudaSuccess) return attr_err;
    CUtensorMap ta, tb;
    if (!make_fp8_map(&ta, g.a_codes, g.M, g.K, g.lda, NT) || !make_fp8_map(&tb, g.b_codes, g.N, g.K, g.ldb, LINES))
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
    p.chunks = (int)((g.K + BK - 1) / BK);
    p.wait_limit = g.wait_limit;
    p.err = device_error_word();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ranks, (unsigned)((g.N + LINES - 1) / LINES), (unsigned)((g.M + NT - 1) / NT));
    cfg.blockDim = dim3(NUM_THREADS);
    cfg.dynamicSmemBytes = G::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)ranks;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gemm_fp8_split_kernel<NT, VEC, OUT_BF16>, ta, tb, p);
}

template <int NT>
cudaError_t run_nt(const Fp8GemmArgs& g, int ranks, cudaStream_t s) {
    if (g.b_lines == 1)
        return g.out_bf16 ? run_split<NT, true, true>(g, ranks, s) : run_split<NT, true, false>(g, ranks, s);
    return g.out_bf16 ? run_split<NT, false, true>(g, ranks, s) : run_split<NT, false, false>(g, ranks, s);
}

}  // namespace

cudaError_t launch_gemm_fp8_split(const Fp8GemmArgs& g, cudaStream_t s) {
    const int nt = g.M <= 16 ? 16 : (g.M <= 32 ? 32 : (g.M <= 64 ? 64 : 128));
    const int64_t tiles = ((g.N + LINES - 1) / LINES) * ((g.M + nt - 1) / nt);
    const int64_t chunks = (g.K + BK - 1) / BK;
    // K is split while the tiles alone leave SMs idle, two chunks per CTA at least
    int ranks = 1;
    while (ranks < 8 && tiles * ranks * 2 <= num_sms() && chunks >= 4 * ranks) ranks *= 2;
    switch (nt) {
    case 16: return run_nt<16>(g, ranks, s);
    case 32: return run_nt<32>(g, ranks, s);
    case 64: return run_nt<64>(g, ranks, s);
    default: return run_nt<128>(g, ranks, s);
    }
}

}  // namespace fp4
