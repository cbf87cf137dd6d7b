// norm_residual.cu -- the norms around a block, fused with its gate and the
// residual update (fp4_norm_residual), and their gradients
// (fp4_norm_residual_backward).  With o the block's output and h the stream:
//
//   n1 = o rstd1,  rstd1 = 1 / sqrt(mean(o^2) + eps)      (with w_post)
//   r  = n1 w_post, or o                                  (without)
//   h' = h + alpha g r                                    (rounded to its type)
//   n2 = h' rstd2,  y = n2 w_pre                          (with w_pre)
//
// and, for the gradients dy of y and dhin of h':
//
//   a   = dy w_pre
//   dh' = dhin + rstd2 (a - n2 mean(a n2)),   dw_pre = sum_rows dy n2
//   dr  = alpha dh',   dgate = sum_group dr r
//   b   = g dr w_post,                        dw_post = sum_rows g dr n1
//   do  = rstd1 (b - n1 mean(b n1)), or g dr
//
// Both are bound by HBM: in bf16 the forward call reads o and h and writes h'
// and y (8 B per element, 7 with FP8 codes for y), the backward call reads dy,
// dhin, h' and o and writes dh' and do (12 B).  Every tensor crosses once: a
// CTA holds a whole row in registers, 8 elements (16 bytes of bf16) per vector
// and VPT vectors per thread, so the row statistics cost no second read, and the
// next row's vectors are on their way while a row is worked on.  The products of
// weights, gate and alpha that a column needs are kept in shared memory, where a
// thread reads and writes only its own columns'.  All sums are binary32; h' is
// rounded before its norm, because the stored h' is what the next block and the
// backward call see.
//
// 8192 x 4096 in bf16, both weights and a gate: forward 50 us (5400 GB/s; 46 us
// without a gate), backward with its sums 76 us (5310 GB/s); without w_post, FP8
// codes for y, 44 us (5370 GB/s).  What
// is left to the copy rate is the block sums' barrier between a row's loads and its
// stores, and in the backward call the arithmetic of the three sums.  One row 3.6
// us; a backward call adds a second launch, 6 us at least.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "fp8_block.cuh"
#include "internal.h"

namespace fp4 {

namespace {

constexpr int VEC = 8;                   // elements per vector
constexpr int PAIRS = VEC / 2;
constexpr float TINY_EPS = 0x1p-96f;

// a vector as it is in memory: one (bf16) or two (fp32) 16-byte words
template <bool BF16>
struct Raw {
    uint4 w[BF16 ? 1 : 2];
};

// the first `n` elements of a vector (8 or more: all; 0 or fewer: none), the others zero
template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_raw(const void* p, int n) {
    Raw<BF16> r;
    if (n >= VEC) {
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) r.w[i] = static_cast<const uint4*>(p)[i];
    } else {
        uint32_t v[BF16 ? 4 : 8];
#pragma unroll
        for (int i = 0; i < (BF16 ? 4 : 8); ++i) v[i] = 0u;
#pragma unroll
        for (int e = 0; e < VEC - 1; ++e)
            if (e < n) {
                if (BF16) v[e / 2] |= (uint32_t)static_cast<const uint16_t*>(p)[e] << (16 * (e & 1));
                else v[BF16 ? 0 : e] = static_cast<const uint32_t*>(p)[e];
            }
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) r.w[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
    return r;
}

// A vector of a row that is not its matrix's last, for 0 < n: the row's pitch is a
// multiple of 16 bytes, so the words that hold its first n elements can be read
// whole; what lies behind the row is cut off by clip() before use.  Loads under a
// branch per vector kept the next row's from being in flight together: backward
// 4771 x 8191 161 us, 8192 columns 77.
template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_words(const char* row, uint32_t off, int n) {
    Raw<BF16> r;
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i)         // words without an element: the row's first, clipped
        r.w[i] = *reinterpret_cast<const uint4*>(row + (n > 4 * i ? off + 16 * i : 0u));
    return r;
}

// the vector with its elements from the n-th on as zeros
template <bool BF16>
__device__ __forceinline__ Raw<BF16> clip(Raw<BF16> r, int n) {
    if (n >= VEC) return r;
    uint32_t* const w = &r.w[0].x;
#pragma unroll
    for (int i = 0; i < (BF16 ? 4 : 8); ++i) {
        const int left = BF16 ? n - 2 * i : 2 * (n - i);         // halves of the word that stay
        w[i] = left >= 2 ? w[i] : (left == 1 ? w[i] & 0xffffu : 0u);
    }
    return r;
}

template <bool BF16>
__device__ __forceinline__ Raw<BF16> zero_raw() {
    Raw<BF16> r;
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) r.w[i] = make_uint4(0u, 0u, 0u, 0u);
    return r;
}

template <bool BF16>
__device__ __forceinline__ void widen(const Raw<BF16>& r, float2 (&v)[PAIRS]) {
    if constexpr (BF16) {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) v[i] = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[2 * i] = make_float2(__uint_as_float(r.w[i].x), __uint_as_float(r.w[i].y));
            v[2 * i + 1] = make_float2(__uint_as_float(r.w[i].z), __uint_as_float(r.w[i].w));
        }
    }
}

// rounded to the stored type (bf16: to nearest even)
template <bool BF16>
__device__ __forceinline__ Raw<BF16> narrow(const float2 (&v)[PAIRS]) {
    Raw<BF16> r;
    if constexpr (BF16) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(v[i].x, v[i].y);
            w[i] = *reinterpret_cast<const uint32_t*>(&x);
        }
        r.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            r.w[i] = make_uint4(__float_as_uint(v[2 * i].x), __float_as_uint(v[2 * i].y), __float_as_uint(v[2 * i + 1].x),
                                __float_as_uint(v[2 * i + 1].y));
    }
    return r;
}

template <bool BF16>
__device__ __forceinline__ void store_raw(void* p, int n, const Raw<BF16>& r) {
    if (n >= VEC) {
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) static_cast<uint4*>(p)[i] = r.w[i];
    } else {
        const uint32_t v[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[BF16 ? 0 : 1].x, r.w[BF16 ? 0 : 1].y,
                               r.w[BF16 ? 0 : 1].z, r.w[BF16 ? 0 : 1].w};
#pragma unroll
        for (int e = 0; e < VEC - 1; ++e)
            if (e < n) {
                if (BF16) static_cast<uint16_t*>(p)[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
                else static_cast<uint32_t*>(p)[e] = v[e];
            }
    }
}

// A float per column in shared memory, a thread's vector as two 16-byte words a
// whole plane apart, so that neighbouring threads meet no bank twice.
struct Columns {
    float4* at;             // [2][vectors of the CTA]
    int stride;             // vectors of the CTA
    __device__ __forceinline__ void get(int i, float2 (&v)[PAIRS]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 w = at[h * stride + i];
            v[2 * h] = make_float2(w.x, w.y);
            v[2 * h + 1] = make_float2(w.z, w.w);
        }
    }
    __device__ __forceinline__ void set(int i, const float2 (&v)[PAIRS]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            at[h * stride + i] = make_float4(v[2 * h].x, v[2 * h].y, v[2 * h + 1].x, v[2 * h + 1].y);
    }
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// a row that starts `row_off` elements into p, the same for the whole CTA, and
// in it the vector at byte `off`
template <bool BF16>
__device__ __forceinline__ const char* row_at(const void* p, int64_t row_off) {
    return static_cast<const char*>(p) + row_off * (BF16 ? 2 : 4);
}
template <bool BF16>
__device__ __forceinline__ char* row_at(void* p, int64_t row_off) {
    return static_cast<char*>(p) + row_off * (BF16 ? 2 : 4);
}

// the factor alpha g w_post of a vector's columns for gate row `grp`
template <bool BF16>
__device__ __forceinline__ void branch_factor(const void* w_post, const void* gate, int64_t ldg, float alpha,
                                              int64_t grp, uint32_t off, int n, float2 (&f)[PAIRS]) {
#pragma unroll
    for (int e = 0; e < PAIRS; ++e) f[e] = both(alpha);
    float2 v[PAIRS];
    if (w_post) {
        widen<BF16>(load_raw<BF16>(row_at<BF16>(w_post, 0) + off, n), v);
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) f[e] = __fmul2_rn(f[e], v[e]);
    }
    if (gate) {
        widen<BF16>(load_raw<BF16>(row_at<BF16>(gate, grp * ldg) + off, n), v);
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) f[e] = __fmul2_rn(f[e], v[e]);
    }
}

// sums of up to four values over the CTA, in a fixed order; every thread gets
// them.  `part` alternates between two buffers from call to call, so one barrier
// is enough.
__device__ __forceinline__ float4 block_sum(float4 v, float4* part, int tid, int warps) {
    float2 lo = make_float2(v.x, v.y), hi = make_float2(v.z, v.w);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        lo = __fadd2_rn(lo, make_float2(__shfl_xor_sync(0xffffffffu, lo.x, d), __shfl_xor_sync(0xffffffffu, lo.y, d)));
        hi.x += __shfl_xor_sync(0xffffffffu, hi.x, d);
    }
    if ((tid & 31) == 0) part[tid >> 5] = make_float4(lo.x, lo.y, hi.x, 0.0f);
    __syncthreads();
    float4 s = part[0];
    lo = make_float2(s.x, s.y);
    for (int w = 1; w < warps; ++w) {
        const float4 t = part[w];
        lo = __fadd2_rn(lo, make_float2(t.x, t.y));
        s.z += t.z;
    }
    return make_float4(lo.x, lo.y, s.z, 0.0f);
}
__device__ __forceinline__ float block_sum(float v, float* part, int tid, int warps) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if ((tid & 31) == 0) part[tid >> 5] = v;
    __syncthreads();
    float s = part[0];
    for (int w = 1; w < warps; ++w) s += part[w];
    return s;
}

// 1 / sqrt(mean + eps) over a row that the CTA holds in registers.  TINY: where that
// mean lies so low that squares were lost to binary32's lower end, they are summed
// again from values times 2^96, whose squares are normal numbers.
template <bool TINY, int VPT>
__device__ __forceinline__ float rstd_of(const float2 (&v)[VPT][PAIRS], float cols, float eps, float (&part)[2][32],
                                         int& turn, int tid, int warps) {
    float2 s2 = both(0.0f);
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) s2 = __ffma2_rn(v[k][e], v[k][e], s2);
    float m = __fadd_rn(__fdiv_rn(block_sum(s2.x + s2.y, part[turn], tid, warps), cols), eps);
    turn ^= 1;
    if (TINY && m < TINY_EPS) {              // the same in every thread
        s2 = both(0.0f);
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int e = 0; e < PAIRS; ++e) {
                const float2 x = __fmul2_rn(v[k][e], both(0x1p96f));
                s2 = __ffma2_rn(x, x, s2);
            }
        m = __fadd_rn(__fdiv_rn(block_sum(s2.x + s2.y, part[turn], tid, warps), cols), eps * 0x1p96f * 0x1p96f);
        turn ^= 1;
        return __frcp_rn(__fsqrt_rn(m)) * 0x1p96f;
    }
    return __frcp_rn(__fsqrt_rn(m));
}

// FULL: the row is exactly the CTA's vectors, none of them partial or empty.
// POST: the block output is normalised; RES: there is one.  TINY: eps lies below
// TINY_EPS, so that a row's mean square may, too.  Any other eps keeps mean + eps
// above it, and takes forms without the second sum, whose registers spill (fp32
// 4096 x 4096 54 us, 67 with it).
template <bool BF16, int VPT, int THREADS, bool FULL, bool RES, bool POST, bool TINY>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 1 : (VPT == 1 ? 4 : 3))
norm_residual_kernel(const NormArgs a) {
    constexpr uint32_t BYTES = VEC * (BF16 ? 2 : 4);
    extern __shared__ float4 columns[];
    __shared__ float part[2][32];
    const int tid = (int)threadIdx.x, T = (int)blockDim.x, cols = (int)a.cols, vecs = T * VPT, warps = T >> 5;
    const Columns w_pre{columns, vecs}, factor{columns + 2 * vecs, vecs};
    int n[VPT];                               // elements of this thread's vectors inside the row
    uint32_t off[VPT];                        // and where they start
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        n[k] = FULL ? VEC : cols - VEC * (tid + k * T);
        off[k] = BYTES * (uint32_t)(tid + k * T);
    }
    Raw<BF16> hr[VPT], orw[VPT];
    auto fetch = [&](int64_t row) {
        const char* h = row_at<BF16>(a.h, row * a.ldh);
        const char* o = row_at<BF16>(a.o, row * a.ldo);
        if (!FULL && row + 1 < a.rows) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                hr[k] = load_words<BF16>(h, off[k], n[k]);
                if (RES) orw[k] = load_words<BF16>(o, off[k], n[k]);
            }
            return;
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            hr[k] = n[k] > 0 ? load_raw<BF16>(h + off[k], n[k]) : zero_raw<BF16>();
            if (RES) orw[k] = n[k] > 0 ? load_raw<BF16>(o + off[k], n[k]) : zero_raw<BF16>();
        }
    };
    int64_t grp = -1;
    int turn = 0;
    // Neighbouring CTAs take neighbouring rows (8192 x 4096 43.9 us, 47.1 with a run
    // of rows per CTA), but with a gate a run per CTA, so that the gate row seldom
    // changes (3589 x 5348 in groups of 156 rows 63 us, 103 the other way).
    const int64_t step = a.gate ? 1 : gridDim.x;
    const int64_t row_end = a.gate ? a.rows * (blockIdx.x + 1) / gridDim.x : a.rows;
    int64_t row = a.gate ? a.rows * blockIdx.x / gridDim.x : blockIdx.x;
    if (row < row_end) fetch(row);
    if (a.w_pre) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (n[k] <= 0) continue;
            float2 v[PAIRS];
            widen<BF16>(load_raw<BF16>(row_at<BF16>(a.w_pre, 0) + off[k], n[k]), v);
            w_pre.set(tid + k * T, v);
        }
    }
    for (; row < row_end; row += step) {
        float2 h[VPT][PAIRS], o[VPT][PAIRS];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            widen<BF16>(FULL ? hr[k] : clip<BF16>(hr[k], n[k]), h[k]);
            if (RES) widen<BF16>(FULL ? orw[k] : clip<BF16>(orw[k], n[k]), o[k]);
        }
        if (row + step < row_end) fetch(row + step);
        if (RES) {
            const int64_t g = a.gate ? row / a.per : 0;
            if (g != grp) {
                grp = g;
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    float2 f[PAIRS];
                    if (n[k] <= 0) continue;
                    branch_factor<BF16>(a.w_post, a.gate, a.ldg, a.alpha, grp, off[k], n[k], f);
                    factor.set(tid + k * T, f);
                }
            }
            float rstd = 1.0f;
            if (POST) {
                rstd = rstd_of<TINY>(o, (float)cols, a.eps, part, turn, tid, warps);
                if (tid == 0) a.rstd_post[row] = rstd;
            }
            char* h_out = row_at<BF16>(a.h_out, row * a.ldho);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if (n[k] <= 0) continue;
                float2 f[PAIRS];
                factor.get(tid + k * T, f);
#pragma unroll
                for (int e = 0; e < PAIRS; ++e) {
                    if (POST) o[k][e] = __fmul2_rn(o[k][e], both(rstd));
                    h[k][e] = __ffma2_rn(o[k][e], f[e], h[k][e]);
                }
                const Raw<BF16> r = narrow<BF16>(h[k]);
                store_raw<BF16>(h_out + off[k], n[k], r);
                if (BF16) widen<BF16>(r, h[k]);
            }
        }
        if (!a.w_pre) continue;
        const float rstd = rstd_of<TINY>(h, (float)cols, a.eps, part, turn, tid, warps);
        if (tid == 0) a.rstd_pre[row] = rstd;
        char* y_out = row_at<BF16>(a.y, row * a.ldy);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const bool live = n[k] > 0;
            float2 f[PAIRS];
#pragma unroll
            for (int e = 0; e < PAIRS; ++e) f[e] = both(0.0f);
            if (live) w_pre.get(tid + k * T, f);
            // y = RN(RN(h' rstd) w): h' rstd lies near 1, where h' w may pass binary32
            // although y does not
            auto product = [&](float2 (&y)[PAIRS]) {
#pragma unroll
                for (int e = 0; e < PAIRS; ++e) y[e] = __fmul2_rn(__fmul2_rn(h[k][e], both(rstd)), f[e]);
            };
            if (a.y && live) {
                float2 y[PAIRS];
                product(y);
                store_raw<BF16>(y_out + off[k], n[k], narrow<BF16>(y));
            }
            if (a.codes) {
                // a block of 128 columns is 16 lanes' vectors; its codes follow from
                // h' w alone, because rstd is common to the block (for bf16 exact, so
                // that ties of y stay ties)
                auto block_max = [&](const float2 (&v)[PAIRS]) {
                    float m = 0.0f;
#pragma unroll
                    for (int e = 0; e < PAIRS; ++e) m = fmaxf(m, fmaxf(fabsf(v[e].x), fabsf(v[e].y)));
#pragma unroll
                    for (int d = 8; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                    return m;
                };
                float2 t[PAIRS];
#pragma unroll
                for (int e = 0; e < PAIRS; ++e) t[e] = __fmul2_rn(h[k][e], f[e]);
                float m = block_max(t), times = rstd;
                const bool far = !(m >= 0x1p-100f && m <= 0x1p100f);
                if (__any_sync(0xffffffffu, far)) {     // 448 / m or h' w pass binary32: the codes of y itself
                    if (far) {
                        product(t);
                        times = 1.0f;
                    }
                    m = block_max(t);
                }
                const Fp8Block b = fp8_block(m, times);
                if (live) {
                    const int i = tid + k * T;
                    if ((tid & 15) == 0) a.scales[(int64_t)(i >> 4) * a.lp + row] = b.s;
                    const uint2 q = make_uint2(fp8_codes4(t[0], t[1], b), fp8_codes4(t[2], t[3], b));
                    uint8_t* dst = a.codes + row * a.ldc + VEC * i;
                    if (n[k] >= VEC) {
                        *reinterpret_cast<uint2*>(dst) = q;
                    } else {                 // 4, 2 and 1 codes
                        const uint32_t b = n[k] & 4 ? q.y : q.x;
                        if (n[k] & 4) *reinterpret_cast<uint32_t*>(dst) = q.x;
                        dst += n[k] & 4;
                        if (n[k] & 2) *reinterpret_cast<uint16_t*>(dst) = (uint16_t)b;
                        dst += n[k] & 2;
                        if (n[k] & 1) *dst = (uint8_t)(b >> (n[k] & 2 ? 16 : 0));
                    }
                }
            }
        }
    }
}

// ------------------------------------------------------------------ backward

// One CTA takes work items in turn: a run of rows inside one gate group.  Over
// an item it sums T = sum dh' n1 per column (n1 = o without w_post), from which
// at its end both dgate = alpha w_post T and dw_post's share, alpha g T, follow.
// dw_pre and dw_post run over all of a CTA's items.  Partial sums go to the
// workspace and are added in a fixed order by norm_reduce_kernel, so results do
// not depend on timing.  Columns past the row are zeros all the way and are only
// left out of the stores.
//
// Four vectors per thread (beyond 8192 columns), or two of fp32, do not fit the
// registers in this form: there a row is read twice, the second time out of L2, to
// which it comes while the row before is worked on, and the sums are in shared
// memory (4096 x 4096 in fp32 91 us, 96 in registers with spills).  Rows beyond 8192
// columns always take 512 threads, of which whole warps have fewer than four vectors.
//
// FULL as above.  PARTS: which parts of the operator are there, or -1 to ask the
// arguments.
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

constexpr int PART_PRE = 1, PART_RES = 2, PART_POST = 4;
template <bool BF16, int VPT, int THREADS, bool FULL, int PARTS>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 1 : (THREADS == 128 ? 4 : (VPT == 1 ? 3 : 2)))
norm_residual_backward_kernel(const NormBwdArgs a) {
    constexpr uint32_t BYTES = VEC * (BF16 ? 2 : 4);
    constexpr bool BIG = VPT == 4 || (VPT == 2 && !BF16);
    constexpr int KEPT = BIG ? 1 : VPT;       // vectors whose A, n1, n2 and sums stay in registers
    const bool pre = PARTS < 0 ? a.w_pre != nullptr : (PARTS & PART_PRE) != 0;
    const bool res = PARTS < 0 ? a.o != nullptr : (PARTS & PART_RES) != 0;
    const bool has_post = PARTS < 0 ? a.w_post != nullptr : (PARTS & PART_POST) != 0;
    extern __shared__ float4 columns[];
    __shared__ float4 part[2][32];
    const int tid = (int)threadIdx.x, T = (int)blockDim.x, cols = (int)a.cols, vecs = T * VPT, warps = T >> 5;
    // BIG (see above): the second and third plane hold the sums of dw_pre and of the item
    const Columns factor{columns, vecs}, plane1{columns + 2 * vecs, vecs}, plane2{columns + 4 * vecs, vecs};
    const Columns w_pre = plane1, post = plane2, sum_pre = plane1, sum_item = plane2;
    const float inv_cols = 1.0f / (float)cols;
    int n[VPT];                               // elements of this thread's vectors inside the row
    uint32_t off[VPT];                        // and where they start
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        n[k] = FULL ? VEC : cols - VEC * (tid + k * T);
        off[k] = BYTES * (uint32_t)(tid + k * T);
    }
    constexpr int SLOTS = BIG ? 2 : VPT;      // vectors as loaded; BIG: the next one while one is worked on
    Raw<BF16> r_dhin[SLOTS], r_dy[SLOTS], r_h[SLOTS], r_o[SLOTS];
    float rstd2n = 0.0f, rstd1n = 1.0f;
    auto fetch_vector = [&](int64_t row, int k) {
        const int j = k % SLOTS;
        if (!FULL && row + 1 < a.rows) {
            r_dhin[j] = a.dh_in ? load_words<BF16>(row_at<BF16>(a.dh_in, row * a.lddhi), off[k], n[k]) : zero_raw<BF16>();
            if (pre) {
                r_dy[j] = load_words<BF16>(row_at<BF16>(a.dy, row * a.lddy), off[k], n[k]);
                r_h[j] = load_words<BF16>(row_at<BF16>(a.h, row * a.ldh), off[k], n[k]);
            }
            if (res) r_o[j] = load_words<BF16>(row_at<BF16>(a.o, row * a.ldo), off[k], n[k]);
            return;
        }
        r_dhin[j] = a.dh_in ? load_raw<BF16>(row_at<BF16>(a.dh_in, row * a.lddhi) + off[k], n[k]) : zero_raw<BF16>();
        if (pre) {
            r_dy[j] = load_raw<BF16>(row_at<BF16>(a.dy, row * a.lddy) + off[k], n[k]);
            r_h[j] = load_raw<BF16>(row_at<BF16>(a.h, row * a.ldh) + off[k], n[k]);
        }
        if (res) r_o[j] = load_raw<BF16>(row_at<BF16>(a.o, row * a.ldo) + off[k], n[k]);
    };
    auto fetch_rstd = [&](int64_t row) {
        if (pre) rstd2n = a.rstd_pre[row];
        if (has_post) rstd1n = a.rstd_post[row];
    };
    auto fetch = [&](int64_t row) {
        fetch_rstd(row);
#pragma unroll
        for (int k = 0; k < VPT; ++k) fetch_vector(row, k);
    };
    // the row on its way to L2
    auto ahead = [&](int64_t row, bool there) {
        if (!there || (tid & (128 / (int)BYTES - 1))) return;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (n[k] <= 0) continue;
            if (a.dh_in) prefetch_l2(row_at<BF16>(a.dh_in, row * a.lddhi) + off[k]);
            if (pre) {
                prefetch_l2(row_at<BF16>(a.dy, row * a.lddy) + off[k]);
                prefetch_l2(row_at<BF16>(a.h, row * a.ldh) + off[k]);
            }
            if (res) prefetch_l2(row_at<BF16>(a.o, row * a.ldo) + off[k]);
        }
    };
    // A = dhin + rstd2 a, n2, n1 and d = a of vector k, from the row as loaded
    float rstd2 = 0.0f, rstd1 = 1.0f;
    auto form = [&](int k, float2 (&A)[PAIRS], float2 (&n2)[PAIRS], float2 (&n1)[PAIRS], float2 (&d)[PAIRS],
                    float2 (&dy)[PAIRS]) {
        widen<BF16>(FULL ? r_dhin[k % SLOTS] : clip<BF16>(r_dhin[k % SLOTS], n[k]), A);
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) n2[e] = n1[e] = d[e] = dy[e] = both(0.0f);
        if (res) widen<BF16>(FULL ? r_o[k % SLOTS] : clip<BF16>(r_o[k % SLOTS], n[k]), n1);
        if (pre) {
            widen<BF16>(FULL ? r_h[k % SLOTS] : clip<BF16>(r_h[k % SLOTS], n[k]), n2);
            widen<BF16>(FULL ? r_dy[k % SLOTS] : clip<BF16>(r_dy[k % SLOTS], n[k]), dy);
            if (BIG) widen<BF16>(load_raw<BF16>(row_at<BF16>(a.w_pre, 0) + off[k], n[k]), d);
            else w_pre.get(tid + k * T, d);
#pragma unroll
            for (int e = 0; e < PAIRS; ++e) {
                n2[e] = __fmul2_rn(n2[e], both(rstd2));
                d[e] = __fmul2_rn(dy[e], d[e]);
                A[e] = __ffma2_rn(d[e], both(rstd2), A[e]);
            }
        }
        if (has_post) {
#pragma unroll
            for (int e = 0; e < PAIRS; ++e) n1[e] = __fmul2_rn(n1[e], both(rstd1));
        }
    };
    // the rows of item `it`
    auto bounds = [&](int64_t it, int64_t& grp, int64_t& first, int64_t& last) {
        grp = it / a.nseg;
        first = grp * a.per + (it - grp * a.nseg) * a.seg_rows;
        last = min(min(first + a.seg_rows, (grp + 1) * a.per), a.rows);
    };
    int turn = 0;
    int64_t grp = 0, row = 0, last = 0;
    int64_t item = blockIdx.x;
    if (item < a.items) {
        bounds(item, grp, row, last);
        if (!BIG && row < last) fetch(row);      // on its way before the weights are read
    }
    float2 acc_pre[KEPT][PAIRS];
    float* const post_row = has_post ? a.post_part + (int64_t)blockIdx.x * a.pitch : nullptr;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int i = tid + k * T;
        float2 v[PAIRS];
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) v[e] = both(0.0f);
        if (BIG) {
            sum_pre.set(i, v);
            if (has_post && n[k] > 0) store_raw<false>(post_row + VEC * i, n[k], narrow<false>(v));
        } else {
#pragma unroll
            for (int e = 0; e < PAIRS; ++e) acc_pre[BIG ? 0 : k][e] = v[e];
            post.set(i, v);
            if (pre) {
                widen<BF16>(load_raw<BF16>(row_at<BF16>(a.w_pre, 0) + off[k], n[k]), v);
                w_pre.set(i, v);
            }
        }
    }
    for (; item < a.items; item += gridDim.x) {
        int64_t grp_next = 0, row_next = 0, last_next = 0;
        if (item + gridDim.x < a.items) bounds(item + gridDim.x, grp_next, row_next, last_next);
        float2 acc[KEPT][PAIRS];                   // sum dh' n1
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            float2 f[PAIRS];
#pragma unroll
            for (int e = 0; e < PAIRS; ++e) {
                f[e] = both(0.0f);
                if (!BIG) acc[BIG ? 0 : k][e] = f[e];
            }
            if (BIG) sum_item.set(tid + k * T, f);
            if (!res || (BIG && n[k] <= 0)) continue;
            branch_factor<BF16>(has_post ? a.w_post : nullptr, a.gate, a.ldg, a.alpha, grp, off[k], n[k], f);
            factor.set(tid + k * T, f);
        }
        for (; row < last; ++row) {
            if (BIG) {
                fetch_rstd(row);
                fetch_vector(row, 0);
                ahead(row + 1 < last ? row + 1 : row_next, row + 1 < last || row_next < last_next);
            }
            rstd2 = rstd2n;
            rstd1 = rstd1n;
            // with dh' = A - rstd2 n2 c1, both means follow from three sums of one
            // pass: c1 = mean(a n2), c2 = mean(b n1) = mean(u A) - c1 rstd2 mean(u n2),
            // u = alpha g w_post n1
            float2 A[KEPT][PAIRS], n2[KEPT][PAIRS], n1[KEPT][PAIRS];
            float2 s0 = both(0.0f), s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int i = tid + k * T, j = BIG ? 0 : k;
                if (BIG && k + 1 < VPT) fetch_vector(row, k + 1);
                if (BIG && n[k] <= 0) continue;
                float2 d[PAIRS], dy[PAIRS];
                form(k, A[j], n2[j], n1[j], d, dy);
                if (pre) {
                    float2 sum[PAIRS];
                    if (BIG) sum_pre.get(i, sum);
#pragma unroll
                    for (int e = 0; e < PAIRS; ++e) {
                        if (BIG) sum[e] = __ffma2_rn(dy[e], n2[j][e], sum[e]);
                        else acc_pre[j][e] = __ffma2_rn(dy[e], n2[j][e], acc_pre[j][e]);
                        s0 = __ffma2_rn(d[e], n2[j][e], s0);
                    }
                    if (BIG) sum_pre.set(i, sum);
                }
                if (has_post) {
                    float2 f[PAIRS];
                    factor.get(i, f);
#pragma unroll
                    for (int e = 0; e < PAIRS; ++e) {
                        const float2 u = __fmul2_rn(f[e], n1[j][e]);
                        s1 = __ffma2_rn(u, A[j][e], s1);
                        s2 = __ffma2_rn(u, n2[j][e], s2);
                    }
                }
            }
            if (BIG) {
                fetch_vector(row, 0);
            } else {
                if (row + 1 < last) fetch(row + 1);
                else if (row_next < last_next) fetch(row_next);
            }
            float c1 = 0.0f, c2 = 0.0f;
            if (pre || has_post) {
                const float4 sums = block_sum(make_float4(s0.x + s0.y, s1.x + s1.y, s2.x + s2.y, 0.0f), part[turn], tid,
                                              warps);
                turn ^= 1;
                c1 = rstd2 * (sums.x * inv_cols);
                c2 = (sums.y - c1 * sums.z) * inv_cols;
            }
            char* dh_out = row_at<BF16>(a.dh, row * a.lddh);
            char* do_out = row_at<BF16>(a.d_o, row * a.lddo);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int i = tid + k * T, j = BIG ? 0 : k;
                if (BIG && k + 1 < VPT) fetch_vector(row, k + 1);
                if (BIG && n[k] <= 0) continue;
                if (BIG) {
                    float2 d[PAIRS], dy[PAIRS];
                    form(k, A[j], n2[j], n1[j], d, dy);
                }
                if (pre) {
#pragma unroll
                    for (int e = 0; e < PAIRS; ++e) A[j][e] = __ffma2_rn(n2[j][e], both(-c1), A[j][e]);      // dh'
                }
                if (n[k] > 0) store_raw<BF16>(dh_out + off[k], n[k], narrow<BF16>(A[j]));
                if (!res) continue;
                float2 f[PAIRS], sum[PAIRS];
                factor.get(i, f);
                if (BIG) sum_item.get(i, sum);
#pragma unroll
                for (int e = 0; e < PAIRS; ++e) {
                    if (BIG) sum[e] = __ffma2_rn(A[j][e], n1[j][e], sum[e]);
                    else acc[j][e] = __ffma2_rn(A[j][e], n1[j][e], acc[j][e]);
                    f[e] = __fmul2_rn(A[j][e], f[e]);                                    // b, or do itself
                    if (has_post) f[e] = __fmul2_rn(__ffma2_rn(n1[j][e], both(-c2), f[e]), both(rstd1));
                }
                if (BIG) sum_item.set(i, sum);
                if (n[k] > 0) store_raw<BF16>(do_out + off[k], n[k], narrow<BF16>(f));
            }
        }
        if (a.gate || has_post) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int i = tid + k * T;
                if (n[k] <= 0) continue;
                float2 f[PAIRS], sum[PAIRS];
                if (BIG) {
                    sum_item.get(i, sum);
                } else {
#pragma unroll
                    for (int e = 0; e < PAIRS; ++e) sum[e] = acc[BIG ? 0 : k][e];
                }
                if (has_post) {
                    float2 p[PAIRS];
                    branch_factor<BF16>(nullptr, a.gate, a.ldg, a.alpha, grp, off[k], n[k], f);
                    if (BIG) widen<false>(load_raw<false>(post_row + VEC * i, n[k]), p);
                    else post.get(i, p);
#pragma unroll
                    for (int e = 0; e < PAIRS; ++e) p[e] = __ffma2_rn(f[e], sum[e], p[e]);
                    if (BIG) store_raw<false>(post_row + VEC * i, n[k], narrow<false>(p));
                    else post.set(i, p);
                }
                if (a.gate) {
                    branch_factor<BF16>(has_post ? a.w_post : nullptr, nullptr, 0, a.alpha, 0, off[k], n[k], f);
#pragma unroll
                    for (int e = 0; e < PAIRS; ++e) f[e] = __fmul2_rn(f[e], sum[e]);
                    float* dst = a.gate_part + item * a.gate_pitch + VEC * i;
                    if (a.gate_pitch % 4 == 0) {
                        store_raw<false>(dst, n[k], narrow<false>(f));
                    } else {                 // dgate itself, with an odd row pitch
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            if (e < n[k]) dst[e] = (e & 1) ? f[e / 2].y : f[e / 2].x;
                    }
                }
            }
        }
        grp = grp_next;
        row = row_next;
        last = last_next;
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int i = tid + k * T;
        if (n[k] <= 0) continue;
        float2 v[PAIRS];
        if (pre) {
            if (BIG) {
                sum_pre.get(i, v);
            } else {
#pragma unroll
                for (int e = 0; e < PAIRS; ++e) v[e] = acc_pre[BIG ? 0 : k][e];
            }
            store_raw<false>(a.pre_part + (int64_t)blockIdx.x * a.pitch + VEC * i, n[k], narrow<false>(v));
        }
        if (has_post && !BIG) {
            post.get(i, v);
            store_raw<false>(post_row + VEC * i, n[k], narrow<false>(v));
        }
    }
}

// out[g][c] = sum over p < n of part[g * n + p][c], in a fixed order; the jobs
// dw_pre, dw_post and dgate (one per group) along the grid's y
__global__ void __launch_bounds__(256) norm_reduce_kernel(const NormBwdArgs a, int ctas) {
    __shared__ float4 sums[32][9];
    const int job = (int)blockIdx.y, quad = (int)threadIdx.x & 7, y = (int)threadIdx.x >> 3;
    const float* part;
    float* out;
    int64_t n = ctas;
    if (a.w_pre && job == 0) {
        part = a.pre_part;
        out = a.dw_pre;
    } else if (a.w_post && job == (a.w_pre ? 1 : 0)) {
        part = a.post_part;
        out = a.dw_post;
    } else {
        const int64_t g = job - (a.w_pre ? 1 : 0) - (a.w_post ? 1 : 0);
        n = a.nseg;
        part = a.gate_part + g * n * a.pitch;
        out = a.dgate + g * a.cols;
    }
    // 32 columns, four per thread; every 32nd line per thread, then over the threads
    const int64_t c = (int64_t)blockIdx.x * 32 + 4 * quad;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < a.cols) {
#pragma unroll 4
        for (int64_t p = y; p < n; p += 32) {
            const float4 w = *reinterpret_cast<const float4*>(part + p * a.pitch + c);
            v.x += w.x;
            v.y += w.y;
            v.z += w.z;
            v.w += w.w;
        }
    }
    sums[y][quad] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        const int col = (int)threadIdx.x;
        const float* s = reinterpret_cast<const float*>(&sums[0][0]) + col;
        float t = s[0];
        for (int i = 1; i < 32; ++i) t += s[i * 36];
        if ((int64_t)blockIdx.x * 32 + col < a.cols) out[(int64_t)blockIdx.x * 32 + col] = t;
    }
}

// vectors per thread and threads for a row of `cols` elements.  Two vectors per
// thread up to 4096 columns leave registers for three CTAs of 256 threads per SM:
// norm 8192 x 4096 52.9 us at the time, against 67.6 with one vector and 512
// threads, 58.9 with two CTAs per SM and 66.4 with four, which spill.
void shape_of(int64_t cols, int& vpt, int& threads) {
    const int64_t nvec = (cols + VEC - 1) / VEC;
    vpt = nvec <= 256 ? 1 : (nvec <= 1024 ? 2 : 4);
    threads = (int)(((nvec + vpt - 1) / vpt + 31) / 32 * 32);
}

// CTAs of the backward kernel, which have a line of partial sums each: three per SM
// with up to 256 threads of one vector, two with two, one beyond 4096 columns, as
// many as the SM holds at once (4364 x 2034 47 us at the time, 57 with two).  Rows
// of up to 1024 columns have a form of 128 threads with all their registers and
// take up to 512 threads per SM: 16, 8, 4 and 4 CTAs of 32, 64, 96 and 128.  The SM
// would hold more, but with 768 threads the longer sum over the lines costs more
// than the rows gain (1031 x 1003 12.2 us against 14.1).  The SMs are a B200's and
// not asked for, so that the workspace's size and the order of the sums follow from
// the sizes alone.
constexpr int64_t BWD_SMS = 148;
int64_t norm_bwd_limit(int64_t cols) {
    int vpt, threads;
    shape_of(cols, vpt, threads);
    if (threads > 256) return BWD_SMS;
    return vpt == 1 && threads > 128 ? 3 * BWD_SMS : 2 * BWD_SMS * (256 / threads);
}
int64_t norm_bwd_ctas(const NormBwdArgs& a) {
    const int64_t limit = norm_bwd_limit(a.cols);
    return a.items < limit ? a.items : limit;
}

template <bool BF16, int VPT, int THREADS, bool FULL, bool TINY, bool RES, bool POST>
cudaError_t run_norm(const NormArgs& a, int threads, cudaStream_t s) {
    static PerDeviceOnce setup;
    static int per_sm[kOnceDevices][17] = {};
    constexpr auto kernel = norm_residual_kernel<BF16, VPT, THREADS, FULL, RES, POST, TINY>;
    const auto smem = [](int t) { return (size_t)t * VPT * VEC * sizeof(float) * (RES ? 2 : 1); };
    int dev = 0;
    const cudaError_t e = setup.run([&](int d) {
        cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem(THREADS));
        for (int w = 1; w <= THREADS / 32 && err == cudaSuccess; ++w) {
            int n = 0;
            err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, 32 * w, smem(32 * w));
            per_sm[d][w] = n < 1 ? 1 : n;
        }
        return err;
    }, &dev);
    if (e != cudaSuccess) return e;
    const int64_t cap = (int64_t)num_sms() * per_sm[dev][threads / 32];
    const unsigned grid = (unsigned)(a.rows < cap ? a.rows : cap);
    kernel<<<grid, threads, smem(threads), s>>>(a);
    return cudaGetLastError();
}

template <bool BF16, int VPT, int THREADS, bool FULL, bool TINY>
cudaError_t run_norm_parts(const NormArgs& a, int threads, cudaStream_t s) {
    if (!a.o) return run_norm<BF16, VPT, THREADS, FULL, TINY, false, false>(a, threads, s);
    return a.w_post ? run_norm<BF16, VPT, THREADS, FULL, TINY, true, true>(a, threads, s)
                    : run_norm<BF16, VPT, THREADS, FULL, TINY, true, false>(a, threads, s);
}

template <bool BF16, int VPT, int THREADS, bool FULL, int PARTS>
cudaError_t run_norm_bwd(const NormBwdArgs& a, int threads, cudaStream_t s) {
    static PerDeviceOnce setup;
    constexpr auto kernel = norm_residual_backward_kernel<BF16, VPT, THREADS, FULL, PARTS>;
    const auto smem = [](int t) { return (size_t)t * VPT * VEC * sizeof(float) * 3; };
    cudaError_t e = setup.run([&](int) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem(THREADS));
    });
    if (e != cudaSuccess) return e;
    const int ctas = (int)norm_bwd_ctas(a);
    kernel<<<ctas, threads, smem(threads), s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t jobs = (a.w_pre ? 1 : 0) + (a.w_post ? 1 : 0) + ((a.gate && a.nseg > 1) ? a.groups : 0);
    if (jobs == 0) return cudaSuccess;
    norm_reduce_kernel<<<dim3((unsigned)((a.cols + 31) / 32), (unsigned)jobs), 256, 0, s>>>(a, ctas);
    return cudaGetLastError();
}

template <bool BF16, int VPT, int THREADS, bool FULL>
cudaError_t run_norm_bwd_parts(const NormBwdArgs& a, int threads, cudaStream_t s) {
    // the usual blocks compiled for themselves
    if (a.w_pre && a.o && a.w_post)
        return run_norm_bwd<BF16, VPT, THREADS, FULL, PART_PRE | PART_RES | PART_POST>(a, threads, s);
    if (a.w_pre && a.o) return run_norm_bwd<BF16, VPT, THREADS, FULL, PART_PRE | PART_RES>(a, threads, s);
    return run_norm_bwd<BF16, VPT, THREADS, FULL, -1>(a, threads, s);
}

template <bool BF16, int VPT, int THREADS>
cudaError_t launch_shape(const NormArgs& a, int threads, cudaStream_t s) {
    if (a.eps < TINY_EPS) return run_norm_parts<BF16, VPT, THREADS, false, true>(a, threads, s);
    return a.cols == (int64_t)threads * VPT * VEC ? run_norm_parts<BF16, VPT, THREADS, true, false>(a, threads, s)
                                                  : run_norm_parts<BF16, VPT, THREADS, false, false>(a, threads, s);
}
template <bool BF16, int VPT, int THREADS>
cudaError_t launch_shape(const NormBwdArgs& a, int threads, cudaStream_t s) {
    return a.cols == (int64_t)threads * VPT * VEC ? run_norm_bwd_parts<BF16, VPT, THREADS, true>(a, threads, s)
                                                  : run_norm_bwd_parts<BF16, VPT, THREADS, false>(a, threads, s);
}

template <bool BF16, class Args>
cudaError_t launch_columns(const Args& a, cudaStream_t s) {
    int vpt, threads;
    shape_of(a.cols, vpt, threads);
    if constexpr (std::is_same<Args, NormBwdArgs>::value)
        if (threads <= 128) return launch_shape<BF16, 1, 128>(a, threads, s);
    if (vpt == 1) return launch_shape<BF16, 1, 256>(a, threads, s);
    if (vpt == 4) return launch_shape<BF16, 4, 512>(a, std::is_same<Args, NormBwdArgs>::value ? 512 : threads, s);
    return threads <= 256 ? launch_shape<BF16, 2, 256>(a, threads, s) : launch_shape<BF16, 2, 512>(a, threads, s);
}

}  // namespace

void norm_bwd_plan(NormBwdArgs& a) {
    a.groups = a.gate ? (a.rows + a.per - 1) / a.per : 1;
    if (!a.gate) a.per = a.rows;
    // segments per group: as many as fill one to four rounds of the CTAs, whichever
    // leaves the busiest CTA the fewest rows, an item's own time counted as two
    const int64_t limit = norm_bwd_limit(a.cols);
    int64_t nseg = 1, best = (a.groups + limit - 1) / limit * (a.per + 2);
    for (int64_t k = 1; k <= 4; ++k) {
        int64_t n = k * limit / a.groups;
        if (n > a.per) n = a.per;
        if (n <= nseg) continue;
        const int64_t cost = (n * a.groups + limit - 1) / limit * ((a.per + n - 1) / n + 2);
        if (cost < best) {
            best = cost;
            nseg = n;
        }
    }
    a.seg_rows = (a.per + nseg - 1) / nseg;
    a.nseg = (a.per + a.seg_rows - 1) / a.seg_rows;
    a.items = a.groups * a.nseg;
    a.pitch = (a.cols + 3) / 4 * 4;
}

size_t norm_bwd_workspace(const NormBwdArgs& a) {
    const int64_t ctas = norm_bwd_ctas(a);
    const int64_t lines = (a.w_pre ? ctas : 0) + (a.w_post ? ctas : 0) + ((a.gate && a.nseg > 1) ? a.items : 0);
    return (size_t)lines * (size_t)a.pitch * sizeof(float);
}

cudaError_t launch_norm(const NormArgs& a, bool bf16, cudaStream_t s) {
    return bf16 ? launch_columns<true>(a, s) : launch_columns<false>(a, s);
}

cudaError_t launch_norm_bwd(NormBwdArgs a, bool bf16, float* workspace, cudaStream_t s) {
    const int64_t ctas = norm_bwd_ctas(a);
    a.pre_part = workspace;
    a.post_part = a.pre_part + (a.w_pre ? ctas * a.pitch : 0);
    // one item per group: its sums are dgate's row
    a.gate_part = a.nseg > 1 ? a.post_part + (a.w_post ? ctas * a.pitch : 0) : a.dgate;
    a.gate_pitch = a.nseg > 1 ? a.pitch : a.cols;
    return bf16 ? launch_columns<true>(a, s) : launch_columns<false>(a, s);
}

}  // namespace fp4
