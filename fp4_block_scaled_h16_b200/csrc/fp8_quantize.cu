// fp8_quantize.cu -- E4M3 codes with one FP32 scale per block of 128 elements
// along K (fp4_fp8_block_quantize), the operands of the FP8 block-scaled GEMM.
//
// A block is 128 consecutive elements of one line (activations, gradients) or
// of 128 lines (weights): a scale s = RN(m / 448) from the block's largest
// magnitude m, and codes E4M3_rne(448 x / m) (fp8_block.cuh).
//
// What bounds it: HBM.  Per element 2 B (bf16) or 4 B (f32) are read and 1 B
// is written per axis.  A CTA of 256 threads takes 128 x 128 tiles: the rows of a
// tile are one 1 x 128 block each, its columns one 128 x 1 block each, and the
// tile one 128 x 128 block, so a single read serves both axes.  A tile lands by
// TMA with the 128-byte swizzle (zeros past the edges, which change no maximum),
// in bf16 while the tile before it is worked on; rows are read as 16-byte chunks
// and columns as 4-byte words, both free of bank conflicts; the codes of either
// axis are staged swizzled in shared memory and leave by one TMA store of 128
// lines x 128 bytes, in whole 128-byte lines.
// 8192 x 4096 bf16, both axes: 26.5 us, 5150 GB/s, 0.80 of the measured copy rate
// (28.0 with a tile per CTA and three CTAs per SM); 4096 x 14336 f32 in 128 x 128
// blocks, both axes: 63 us, 0.87.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "fp8_block.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace fp4 {

namespace {

constexpr int TILE = 128;
constexpr int THREADS = 256;
constexpr uint32_t OUT_BYTES = TILE * TILE;                 // one axis' codes of a tile
constexpr uint32_t DRAIN_LIMIT = 1u << 22;
constexpr unsigned int ERR_TIMEOUT = 7u;                    // FP4_ERR_TIMEOUT

// bf16 tiles are small enough to have the next one on its way in two CTAs per
// SM; f32 takes one tile per CTA
template <bool BF16>
constexpr int IN_STAGES = BF16 ? 2 : 1;

struct Fp8QuantParams {
    int64_t rows, cols;
    int tiles_c;                 // tiles across the columns
    int tiles;
    float* scales_rows;          // [ceil(cols / 128), lp_rows]
    float* scales_cols;          // [ceil(rows / 128), lp_cols]
    uint8_t* codes_rows;
    uint8_t* codes_cols;
    int64_t ld_rows, ld_cols;
    int64_t lp_rows, lp_cols;    // lines of a scale row: padded lines, or line blocks
    uint32_t wait_limit;
    unsigned int* err;
};

__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) {
    const uint32_t ab = b & 0x7FFF7FFFu;
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                     *reinterpret_cast<const __nv_bfloat162*>(&ab));
    return *reinterpret_cast<const uint32_t*>(&m);
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// the tile's staged codes (lines line0.., K k0..) without a byte past `lines` or K
__device__ void store_clipped(const uint8_t* staged, uint8_t* codes, int64_t ld, int64_t line0, int64_t lines,
                              int64_t k0, int64_t K) {
    const uint32_t base = sm100::smem_u32(staged);
    for (int i = threadIdx.x; i < TILE * 8; i += THREADS) {
        const int line = i >> 3, chunk = i & 7;
        const int64_t k = k0 + 16 * chunk;
        if (line0 + line >= lines || k >= K) continue;
        const uint4 v = ld_shared_v4(base + line * 128 + ((chunk ^ (line & 7)) << 4));
        uint8_t* dst = codes + (line0 + line) * ld + k;
        if (k + 16 <= K) {
            *reinterpret_cast<uint4*>(dst) = v;
        } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int b = 0; b < 16; ++b)
                if (k + b < K) dst[b] = (uint8_t)(w[b >> 2] >> (8 * (b & 3)));
        }
    }
}

// BF16: input type (else f32); LINES: 1 or 128 lines per block
template <bool BF16, int LINES, bool ROWS, bool COLS>
__global__ void __launch_bounds__(THREADS, 2)
fp8_block_quantize_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_rows,
                          const __grid_constant__ CUtensorMap tm_cols, const Fp8QuantParams p) {
    constexpr int ES = BF16 ? 2 : 4;
    constexpr int BOX_COLS = 128 / ES;                      // columns of a 128-byte box row
    constexpr int BOXES = TILE / BOX_COLS;
    constexpr uint32_t BOX_BYTES = TILE * 128;
    constexpr int WORDS = TILE * TILE * ES / 4 / THREADS;   // 32-bit words of the tile per thread
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = sm100::smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    constexpr int STAGES = IN_STAGES<BF16>;
    uint8_t* out_r = smem + STAGES * BOXES * BOX_BYTES;
    uint8_t* out_c = out_r + (ROWS ? OUT_BYTES : 0);
    float* part = reinterpret_cast<float*>(out_c + (COLS ? OUT_BYTES : 0));   // [4][128] column maxima, or 8 warps'
    uint64_t* full = reinterpret_cast<uint64_t*>(part + 4 * TILE);

    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    auto load_tile = [&](int tile, int stage) {
        const int r = tile / p.tiles_c * TILE, c = tile % p.tiles_c * TILE;
        sm100::mbar_arrive_expect_tx(&full[stage], BOXES * BOX_BYTES);
#pragma unroll
        for (int b = 0; b < BOXES; ++b)
            sm100::tma_load_2d(smem + (stage * BOXES + b) * BOX_BYTES, &tm_x, c + b * BOX_COLS, r, &full[stage]);
    };
    if (t == 0) {
        for (int s = 0; s < STAGES; ++s) sm100::mbar_init(&full[s], 1);
        sm100::fence_barrier_init();
        load_tile((int)blockIdx.x, 0);
    }
    // ---- rows: thread t takes half a row (64 columns) of row t / 2
    const int row = t >> 1, half = t & 1;
    // ---- columns: a warp takes one box (bf16: of 64 columns, a pair per lane)
    // and a group of rows, WORDS rows per thread
    const int box = warp & (BOXES - 1), rgroup = warp / BOXES;
    const int ccol = box * BOX_COLS + (BF16 ? 2 * lane : lane);      // first column of this lane
    constexpr int RGROUPS = 8 / BOXES;

    int stage = 0;
    uint32_t phase = 0;
    for (int tile_i = (int)blockIdx.x; tile_i < p.tiles; tile_i += (int)gridDim.x) {
        const int tr = tile_i / p.tiles_c, tc = tile_i % p.tiles_c;
        const int row0 = tr * TILE, col0 = tc * TILE;
        const uint32_t in_s = sm100::smem_u32(smem + stage * BOXES * BOX_BYTES);
        if (t == 0) sm100::bulk_wait_read0();           // the previous tile's codes have left the staging buffers
        __syncthreads();                                // and every thread has read its input
        if (STAGES > 1 && t == 0 && tile_i + (int)gridDim.x < p.tiles) load_tile(tile_i + (int)gridDim.x, stage ^ 1);
        if (!sm100::mbar_wait(&full[stage], phase, p.wait_limit, nullptr)) {
            atomicExch(p.err, ERR_TIMEOUT);
            if (t == 0) sm100::mbar_wait(&full[stage], phase, DRAIN_LIMIT, nullptr);   // the tile lands before the CTA leaves
        }
        uint32_t w[WORDS];

        auto load_row = [&]() {
#pragma unroll
            for (int c = 0; c < WORDS / 4; ++c) {
                // chunk order differs between the two halves so that they meet no bank twice
                const int cc = (BF16 ? c : (c & 7)) ^ (4 * half);
                const int bx = BF16 ? half : 2 * half + (c >> 3);
                const uint4 v = ld_shared_v4(in_s + bx * BOX_BYTES + row * 128 + ((cc ^ (row & 7)) << 4));
                w[4 * c] = v.x; w[4 * c + 1] = v.y; w[4 * c + 2] = v.z; w[4 * c + 3] = v.w;
            }
        };
        auto load_col = [&]() {
#pragma unroll
            for (int r = 0; r < WORDS; ++r) {
                const int rr = rgroup * WORDS + r;
                w[r] = ld_shared_u32(in_s + box * BOX_BYTES + rr * 128 + (((lane >> 2) ^ (rr & 7)) << 4) + (lane & 3) * 4);
            }
        };
        // maximum magnitude of the words held: one value (f32), or a pair (bf16)
        auto max_words = [&](float& lo, float& hi) {
            if (BF16) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < WORDS; ++i) m = abs_max2(m, w[i]);
                lo = bf16_lo(m);
                hi = bf16_hi(m);
            } else {
                float m = 0.0f;
#pragma unroll
                for (int i = 0; i < WORDS; ++i) m = fmaxf(m, fabsf(__uint_as_float(w[i])));
                lo = hi = m;
            }
        };
        Fp8Block tile;
        if (LINES == 128) {
            load_row();
            float lo, hi;
            max_words(lo, hi);
            const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(lo, hi)));
            if (lane == 0) part[warp] = __uint_as_float(m);
            __syncthreads();
            float mm = part[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) mm = fmaxf(mm, part[i]);
            tile = fp8_block(mm);
            if (t == 0) {
                if (ROWS) p.scales_rows[(int64_t)tc * p.lp_rows + tr] = tile.s;
                if (COLS) p.scales_cols[(int64_t)tr * p.lp_cols + tc] = tile.s;
            }
        }
        if (ROWS) {
            Fp8Block b = tile;
            if (LINES == 1) {
                load_row();
                float lo, hi;
                max_words(lo, hi);
                float m = fmaxf(lo, hi);
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                b = fp8_block(m);
                if (half == 0 && row0 + row < p.rows) p.scales_rows[(int64_t)tc * p.lp_rows + row0 + row] = b.s;
            }
            // 64 codes of the row: four 16-byte chunks (of 16 columns each)
            const uint32_t dst = sm100::smem_u32(out_r) + row * 128;
            uint32_t q[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (BF16)
                    q[i] = fp8_codes4(make_float2(bf16_lo(w[2 * i]), bf16_hi(w[2 * i])),
                                      make_float2(bf16_lo(w[2 * i + 1]), bf16_hi(w[2 * i + 1])), b);
                else
                    q[i] = fp8_codes4(make_float2(__uint_as_float(w[4 * i]), __uint_as_float(w[4 * i + 1])),
                                      make_float2(__uint_as_float(w[4 * i + 2]), __uint_as_float(w[4 * i + 3])), b);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // the order in which load_row took the 16-byte chunks, undone: two
                // input chunks (bf16) or four (f32) make one chunk of codes
                const int at = BF16 ? (i ^ (2 * half)) : ((i & 2) | ((i & 1) ^ half));
                sm100::st_shared_v4(dst + (((4 * half + at) ^ (row & 7)) << 4), q[4 * i], q[4 * i + 1], q[4 * i + 2],
                                    q[4 * i + 3]);
            }
        }
        if (COLS) {
            load_col();
            Fp8Block b0 = tile, b1 = tile;
            if (LINES == 1) {
                float lo, hi;
                max_words(lo, hi);
                part[rgroup * TILE + ccol] = lo;
                if (BF16) part[rgroup * TILE + ccol + 1] = hi;
                __syncthreads();
                float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
                for (int i = 0; i < RGROUPS; ++i) {
                    m0 = fmaxf(m0, part[i * TILE + ccol]);
                    if (BF16) m1 = fmaxf(m1, part[i * TILE + ccol + 1]);
                }
                b0 = fp8_block(m0);
                if (BF16) b1 = fp8_block(m1);
                if (rgroup == 0) {
                    float* sc = p.scales_cols + (int64_t)tr * p.lp_cols + col0 + ccol;
                    if (col0 + ccol < p.cols) sc[0] = b0.s;
                    if (BF16 && col0 + ccol + 1 < p.cols) sc[1] = b1.s;
                }
            }
            const uint32_t dst = sm100::smem_u32(out_c);
#pragma unroll
            for (int i = 0; i < WORDS / 16; ++i) {              // 16 rows: one 16-byte chunk per column
                const int chunk = rgroup * (WORDS / 16) + i;
                uint32_t q0[4], q1[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t* v = &w[16 * i + 4 * e];
                    if (BF16) {
                        q0[e] = fp8_codes4(make_float2(bf16_lo(v[0]), bf16_lo(v[1])), make_float2(bf16_lo(v[2]), bf16_lo(v[3])), b0);
                        q1[e] = fp8_codes4(make_float2(bf16_hi(v[0]), bf16_hi(v[1])), make_float2(bf16_hi(v[2]), bf16_hi(v[3])), b1);
                    } else {
                        q0[e] = fp8_codes4(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])),
                                           make_float2(__uint_as_float(v[2]), __uint_as_float(v[3])), b0);
                    }
                }
                if (BF16) {
                    // lanes 4-7 of each eight write their odd column first, so that
                    // eight lanes meet eight different chunk positions
                    const bool odd = (lane & 4) != 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t a = odd ? q1[e] : q0[e], b = odd ? q0[e] : q1[e];
                        q0[e] = a;
                        q1[e] = b;
                    }
                    const int ca = ccol + (odd ? 1 : 0), cb = ccol + (odd ? 0 : 1);
                    sm100::st_shared_v4(dst + ca * 128 + ((chunk ^ (ca & 7)) << 4), q0[0], q0[1], q0[2], q0[3]);
                    sm100::st_shared_v4(dst + cb * 128 + ((chunk ^ (cb & 7)) << 4), q1[0], q1[1], q1[2], q1[3]);
                } else {
                    sm100::st_shared_v4(dst + ccol * 128 + ((chunk ^ (ccol & 7)) << 4), q0[0], q0[1], q0[2], q0[3]);
                }
            }
        }
        sm100::fence_proxy_async_smem();
        __syncthreads();
        // a TMA store clips a line at 16 bytes, so a tile that ends inside a
        // 16-byte chunk is written by the threads
        const bool odd_r = ROWS && col0 + TILE > p.cols && (p.cols & 15);
        const bool odd_c = COLS && row0 + TILE > p.rows && (p.rows & 15);
        if (odd_r) store_clipped(out_r, p.codes_rows, p.ld_rows, row0, p.rows, col0, p.cols);
        if (odd_c) store_clipped(out_c, p.codes_cols, p.ld_cols, col0, p.cols, row0, p.rows);
        if (t == 0) {
            if (ROWS && !odd_r) sm100::tma_store_2d(&tm_rows, out_r, col0, row0);
            if (COLS && !odd_c) sm100::tma_store_2d(&tm_cols, out_c, row0, col0);
            sm100::bulk_commit();
        }
        if (STAGES > 1) {
            stage ^= 1;
            if (stage == 0) phase ^= 1u;
        }
    }
    if (t == 0) sm100::bulk_wait_read0();           // shared memory is read before the CTA leaves
}

template <bool BF16, int LINES, bool ROWS, bool COLS>
cudaError_t run_quantize(const CUtensorMap& tx, const CUtensorMap& trow, const CUtensorMap& tcol,
                         const Fp8QuantParams& p, cudaStream_t s) {
    constexpr uint32_t smem = IN_STAGES<BF16> * TILE * TILE * (BF16 ? 2 : 4) + (ROWS ? OUT_BYTES : 0) + (COLS ? OUT_BYTES : 0) +
                              4 * TILE * 4 + 16 + 1024;
    static PerDeviceOnce setup;
    const cudaError_t e = setup.run([](int) {
        return cudaFuncSetAttribute(fp8_block_quantize_kernel<BF16, LINES, ROWS, COLS>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    const int resident = 2 * num_sms();
    const int grid = BF16 && p.tiles > resident ? resident : p.tiles;
    fp8_block_quantize_kernel<BF16, LINES, ROWS, COLS><<<grid, THREADS, smem, s>>>(tx, trow, tcol, p);
    return cudaGetLastError();
}

template <bool BF16, int LINES>
cudaError_t run_axes(const CUtensorMap& tx, const CUtensorMap& trow, const CUtensorMap& tcol, const Fp8QuantParams& p,
                     bool rows, bool cols, cudaStream_t s) {
    if (rows && cols) return run_quantize<BF16, LINES, true, true>(tx, trow, tcol, p, s);
    if (rows) return run_quantize<BF16, LINES, true, false>(tx, trow, tcol, p, s);
    return run_quantize<BF16, LINES, false, true>(tx, trow, tcol, p, s);
}

// 2-D map of 128-byte-swizzled boxes, 128 bytes x 128 lines
bool make_box_map(CUtensorMap* m, const void* x, CUtensorMapDataType type, int es, int64_t lines, int64_t K,
                  int64_t pitch) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)lines};
    cuuint64_t strides[1] = {(cuuint64_t)(pitch * es)};
    cuuint32_t box[2] = {(cuuint32_t)(128 / es), 128u};
    cuuint32_t estr[2] = {1u, 1u};
    return fn(m, type, 2, const_cast<void*>(x), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

}  // namespace

bool make_fp8_map(CUtensorMap* m, const uint8_t* codes, int64_t lines, int64_t K, int64_t pitch, int box_lines) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)lines};
    cuuint64_t strides[1] = {(cuuint64_t)pitch};
    cuuint32_t box[2] = {128u, (cuuint32_t)box_lines};
    cuuint32_t estr[2] = {1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, cudaStream_t s) {
    const bool rows = a.codes_rows != nullptr, cols = a.codes_cols != nullptr;
    CUtensorMap tx, trow, tcol;
    if (!make_box_map(&tx, a.x, a.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                      a.bf16 ? 2 : 4, a.rows, a.cols, a.ld))
        return cudaErrorInvalidValue;
    if (rows && !make_fp8_map(&trow, a.codes_rows, a.rows, a.cols, a.ld_rows, 128)) return cudaErrorInvalidValue;
    if (cols && !make_fp8_map(&tcol, a.codes_cols, a.cols, a.rows, a.ld_cols, 128)) return cudaErrorInvalidValue;
    if (!rows) trow = tcol;
    if (!cols) tcol = trow;
    Fp8QuantParams p{};
    p.rows = a.rows;
    p.cols = a.cols;
    p.tiles_c = (int)((a.cols + TILE - 1) / TILE);
    p.codes_rows = a.codes_rows;
    p.codes_cols = a.codes_cols;
    p.ld_rows = a.ld_rows;
    p.ld_cols = a.ld_cols;
    p.scales_rows = a.scales_rows;
    p.scales_cols = a.scales_cols;
    p.lp_rows = fp8_scale_lines(a.rows, a.block_lines);
    p.lp_cols = fp8_scale_lines(a.cols, a.block_lines);
    p.wait_limit = a.wait_limit;
    p.err = device_error_word();
    p.tiles = (int)(p.tiles_c * ((a.rows + TILE - 1) / TILE));
    if (a.block_lines == 1)
        return a.bf16 ? run_axes<true, 1>(tx, trow, tcol, p, rows, cols, s)
                      : run_axes<false, 1>(tx, trow, tcol, p, rows, cols, s);
    return a.bf16 ? run_axes<true, 128>(tx, trow, tcol, p, rows, cols, s)
                  : run_axes<false, 128>(tx, trow, tcol, p, rows, cols, s);
}

}  // namespace fp4
