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
// and VPT vectors per thread, so the row statistics cost no second read.  All
// sums are binary32; h' is rounded before its norm, because the stored h' is
// what the next block and the backward call see.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "internal.h"

namespace fp4 {

namespace {

constexpr int VEC = 8;                   // elements per vector

template <bool BF16>
__device__ __forceinline__ void load8(const void* base, int64_t row_off, int i, int cols, float (&v)[VEC]) {
    const int c0 = VEC * i;
    if (BF16) {
        const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(base) + row_off + c0;
        if (c0 + VEC <= cols) {
            const uint4 w = *reinterpret_cast<const uint4*>(p);
            v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
            v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[e] = c0 + e < cols ? __bfloat162float(p[e]) : 0.0f;
        }
    } else {
        const float* p = static_cast<const float*>(base) + row_off + c0;
        if (c0 + VEC <= cols) {
            const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[e] = c0 + e < cols ? p[e] : 0.0f;
        }
    }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* base, int64_t row_off, int i, int cols, const float (&v)[VEC]) {
    const int c0 = VEC * i;
    if (BF16) {
        __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + row_off + c0;
        if (c0 + VEC <= cols) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
                w[e] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (c0 + e < cols) p[e] = __float2bfloat16_rn(v[e]);
        }
    } else {
        float* p = static_cast<float*>(base) + row_off + c0;
        if (c0 + VEC <= cols) {
            *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (c0 + e < cols) p[e] = v[e];
        }
    }
}

// sums of N values over the CTA, in a fixed order; every thread gets them.
// `part` alternates between two buffers from call to call, so one barrier is enough.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*part)[32]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], d);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = (int)(blockDim.x >> 5);
    if (lane == 0)
#pragma unroll
        for (int n = 0; n < N; ++n) part[n][warp] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        float s = 0.0f;
        for (int w = 0; w < warps; ++w) s += part[n][w];
        v[n] = s;
    }
}

__device__ __forceinline__ float rstd_of(float sum, float cols, float eps) {
    return __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(sum, cols), eps)));
}

template <bool BF16, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 256 : 512)
norm_residual_kernel(const NormArgs a) {
    __shared__ float part[2][1][32];
    const int T = (int)blockDim.x, cols = (int)a.cols;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float h[VPT][VEC];
#pragma unroll
        for (int k = 0; k < VPT; ++k) load8<BF16>(a.h, row * a.ldh, (int)threadIdx.x + k * T, cols, h[k]);
        if (a.o) {
            float o[VPT][VEC];
#pragma unroll
            for (int k = 0; k < VPT; ++k) load8<BF16>(a.o, row * a.ldo, (int)threadIdx.x + k * T, cols, o[k]);
            float rstd = 1.0f;
            if (a.w_post) {
                float ss[1] = {0.0f};
#pragma unroll
                for (int k = 0; k < VPT; ++k)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) ss[0] = fmaf(o[k][e], o[k][e], ss[0]);
                block_sum<1>(ss, part[turn]);
                turn ^= 1;
                rstd = rstd_of(ss[0], (float)cols, a.eps);
                if (threadIdx.x == 0) a.rstd_post[row] = rstd;
            }
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int i = (int)threadIdx.x + k * T;
                if (VEC * i >= cols) continue;
                float w[VEC];
                if (a.w_post) {
                    load8<BF16>(a.w_post, 0, i, cols, w);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) o[k][e] = o[k][e] * rstd * w[e];
                }
                if (a.gate) {
                    load8<BF16>(a.gate, row / a.per * a.ldg, i, cols, w);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) o[k][e] *= w[e];
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    h[k][e] = fmaf(a.alpha, o[k][e], h[k][e]);
                    if (BF16) h[k][e] = __bfloat162float(__float2bfloat16_rn(h[k][e]));
                }
                store8<BF16>(a.h_out, row * a.ldho, i, cols, h[k]);
            }
        }
        if (!a.w_pre) continue;
        float ss[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int e = 0; e < VEC; ++e) ss[0] = fmaf(h[k][e], h[k][e], ss[0]);
        block_sum<1>(ss, part[turn]);
        turn ^= 1;
        const float rstd = rstd_of(ss[0], (float)cols, a.eps);
        if (threadIdx.x == 0) a.rstd_pre[row] = rstd;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int i = (int)threadIdx.x + k * T;
            const bool live = VEC * i < cols;
            float y[VEC];
            if (live) load8<BF16>(a.w_pre, 0, i, cols, y);
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[e] = live ? h[k][e] * rstd * y[e] : 0.0f;
            if (a.y && live) store8<BF16>(a.y, row * a.ldy, i, cols, y);
            if (a.codes) {
                // a block of 128 columns is 16 lanes' vectors
                float m = 0.0f;
#pragma unroll
                for (int e = 0; e < VEC; ++e) m = fmaxf(m, fabsf(y[e]));
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                float s = __fdiv_rn(m, 448.0f);
                s = s >= 1.17549435e-38f ? s : 1.0f;
                const float r = __frcp_rn(s);
                if (live) {
                    if ((threadIdx.x & 15) == 0) a.scales[(int64_t)(i >> 4) * a.lp + row] = s;
                    uint16_t q[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                            : "=h"(q[e]) : "f"(__fmul_rn(y[2 * e + 1], r)), "f"(__fmul_rn(y[2 * e], r)));
                    uint8_t* dst = a.codes + row * a.ldc + VEC * i;
                    if (VEC * i + VEC <= cols) {
                        *reinterpret_cast<uint2*>(dst) = make_uint2((uint32_t)q[0] | ((uint32_t)q[1] << 16),
                                                                    (uint32_t)q[2] | ((uint32_t)q[3] << 16));
                    } else {
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            if (VEC * i + e < cols) dst[e] = (uint8_t)(q[e >> 1] >> (8 * (e & 1)));
                    }
                }
            }
        }
    }
}

// ------------------------------------------------------------------ backward

// One CTA takes work items in turn: a run of rows inside one gate group, whose
// dgate sums end with the item.  The sums for dw_pre and dw_post run over all
// of a CTA's items.  Partial sums go to the workspace and are added in a fixed
// order by norm_reduce_kernel, so results do not depend on timing.
template <bool BF16, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 256 : 512)
norm_residual_backward_kernel(const NormBwdArgs a) {
    __shared__ float part[2][3][32];
    const int T = (int)blockDim.x, cols = (int)a.cols;
    const float inv_cols = 1.0f / (float)cols;
    int turn = 0;
    float acc_pre[VPT][VEC], acc_post[VPT][VEC];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc_pre[k][e] = acc_post[k][e] = 0.0f;
    for (int64_t item = blockIdx.x; item < a.items; item += gridDim.x) {
        const int64_t grp = item / a.nseg, seg = item % a.nseg;
        const int64_t first = grp * a.per + seg * a.seg_rows;
        int64_t last = first + a.seg_rows;
        if (last > (grp + 1) * a.per) last = (grp + 1) * a.per;
        if (last > a.rows) last = a.rows;
        float acc_gate[VPT][VEC];
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc_gate[k][e] = 0.0f;
        for (int64_t row = first; row < last; ++row) {
            const float rstd2 = a.w_pre ? a.rstd_pre[row] : 0.0f, rstd1 = a.w_post ? a.rstd_post[row] : 1.0f;
            // A = dhin + rstd2 dy w_pre, n2, o and u = alpha g w_post n1: with
            // dh' = A - rstd2 n2 c1, both means follow from three sums of one pass:
            // c1 = mean(a n2), c2 = mean(b n1) = mean(u A) - c1 mean(u rstd2 n2)
            float A[VPT][VEC], n2[VPT][VEC], o[VPT][VEC];
            float sums[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int i = (int)threadIdx.x + k * T;
#pragma unroll
                for (int e = 0; e < VEC; ++e) A[k][e] = n2[k][e] = o[k][e] = 0.0f;
                if (VEC * i >= cols) continue;
                if (a.dh_in) load8<BF16>(a.dh_in, row * a.lddhi, i, cols, A[k]);
                if (a.o) load8<BF16>(a.o, row * a.ldo, i, cols, o[k]);
                if (a.w_pre) {
                    float dy[VEC], w[VEC];
                    load8<BF16>(a.dy, row * a.lddy, i, cols, dy);
                    load8<BF16>(a.h, row * a.ldh, i, cols, n2[k]);
                    load8<BF16>(a.w_pre, 0, i, cols, w);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        n2[k][e] *= rstd2;
                        acc_pre[k][e] = fmaf(dy[e], n2[k][e], acc_pre[k][e]);
                        const float d = dy[e] * w[e];
                        sums[0] = fmaf(d, n2[k][e], sums[0]);
                        A[k][e] = fmaf(rstd2, d, A[k][e]);
                    }
                }
                if (a.w_post) {
                    float w[VEC], g[VEC];
                    load8<BF16>(a.w_post, 0, i, cols, w);
                    if (a.gate) load8<BF16>(a.gate, grp * a.ldg, i, cols, g);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float u = a.alpha * (a.gate ? g[e] : 1.0f) * w[e] * (o[k][e] * rstd1);
                        sums[1] = fmaf(u, A[k][e], sums[1]);
                        sums[2] = fmaf(u, rstd2 * n2[k][e], sums[2]);
                    }
                }
            }
            block_sum<3>(sums, part[turn]);
            turn ^= 1;
            const float c1 = sums[0] * inv_cols, c2 = (sums[1] - c1 * sums[2]) * inv_cols;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int i = (int)threadIdx.x + k * T;
                if (VEC * i >= cols) continue;
                float dh[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) dh[e] = fmaf(-rstd2 * c1, n2[k][e], A[k][e]);
                store8<BF16>(a.dh, row * a.lddh, i, cols, dh);
                if (!a.o) continue;
                float w[VEC], g[VEC], d[VEC];
                if (a.w_post) load8<BF16>(a.w_post, 0, i, cols, w);
                if (a.gate) load8<BF16>(a.gate, grp * a.ldg, i, cols, g);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float dr = a.alpha * dh[e], gr = a.gate ? g[e] * dr : dr;
                    const float n1 = o[k][e] * rstd1;
                    if (a.gate) acc_gate[k][e] = fmaf(dr, a.w_post ? n1 * w[e] : o[k][e], acc_gate[k][e]);
                    if (a.w_post) {
                        acc_post[k][e] = fmaf(gr, n1, acc_post[k][e]);
                        d[e] = rstd1 * (gr * w[e] - n1 * c2);
                    } else {
                        d[e] = gr;
                    }
                }
                store8<BF16>(a.d_o, row * a.lddo, i, cols, d);
            }
        }
        if (a.gate) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int i = (int)threadIdx.x + k * T;
                if (a.gate_pitch % 4 == 0) {
                    store8<false>(a.gate_part, item * a.gate_pitch, i, cols, acc_gate[k]);
                } else {                 // dgate itself, with an odd row pitch
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (VEC * i + e < cols) a.gate_part[item * a.gate_pitch + VEC * i + e] = acc_gate[k][e];
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int i = (int)threadIdx.x + k * T;
        if (a.w_pre) store8<false>(a.pre_part, (int64_t)blockIdx.x * a.pitch, i, cols, acc_pre[k]);
        if (a.w_post) store8<false>(a.post_part, (int64_t)blockIdx.x * a.pitch, i, cols, acc_post[k]);
    }
}

// out[g][c] = sum over p < n of part[g * n + p][c], in a fixed order; the jobs
// dw_pre, dw_post and dgate (one per group) along the grid's y
__global__ void __launch_bounds__(256) norm_reduce_kernel(const NormBwdArgs a, int ctas) {
    __shared__ float s[8][33];
    int job = (int)blockIdx.y;
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
    const int64_t c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    const int y = threadIdx.x >> 5;
    float v = 0.0f;
    if (c < a.cols)
        for (int64_t p = y; p < n; p += 8) v += part[p * a.pitch + c];
    s[y][threadIdx.x & 31] = v;
    __syncthreads();
    if (y == 0 && c < a.cols) {
        for (int i = 1; i < 8; ++i) v += s[i][threadIdx.x];
        out[c] = v;
    }
}

// vectors per thread and threads for a row of `cols` elements
void shape_of(int64_t cols, int& vpt, int& threads) {
    const int64_t nvec = (cols + VEC - 1) / VEC;
    vpt = nvec <= 256 ? 1 : (nvec <= 1024 ? 2 : 4);
    threads = (int)(((nvec + vpt - 1) / vpt + 31) / 32 * 32);
}

template <bool BF16, int VPT>
cudaError_t run_norm(const NormArgs& a, int threads, cudaStream_t s) {
    static PerDeviceOnce setup;
    static int per_sm[kOnceDevices][17] = {};
    int dev = 0;
    cudaError_t e = setup.run([](int d) {
        for (int w = 1; w <= 16; ++w) {
            int n = 0;
            const cudaError_t err =
                cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, norm_residual_kernel<BF16, VPT>, 32 * w, 0);
            if (err != cudaSuccess) return err;
            per_sm[d][w] = n < 1 ? 1 : n;
        }
        return cudaSuccess;
    }, &dev);
    if (e != cudaSuccess) return e;
    const int64_t cap = (int64_t)num_sms() * per_sm[dev][threads / 32];
    const unsigned grid = (unsigned)(a.rows < cap ? a.rows : cap);
    norm_residual_kernel<BF16, VPT><<<grid, threads, 0, s>>>(a);
    return cudaGetLastError();
}

template <bool BF16, int VPT>
cudaError_t run_norm_bwd(const NormBwdArgs& a, int threads, cudaStream_t s) {
    const int ctas = (int)(a.items < NORM_BWD_CTAS ? a.items : NORM_BWD_CTAS);
    norm_residual_backward_kernel<BF16, VPT><<<ctas, threads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t jobs = (a.w_pre ? 1 : 0) + (a.w_post ? 1 : 0) + ((a.gate && a.nseg > 1) ? a.groups : 0);
    if (jobs == 0) return cudaSuccess;
    norm_reduce_kernel<<<dim3((unsigned)((a.cols + 31) / 32), (unsigned)jobs), 256, 0, s>>>(a, ctas);
    return cudaGetLastError();
}

}  // namespace

void norm_bwd_plan(NormBwdArgs& a) {
    a.groups = a.gate ? (a.rows + a.per - 1) / a.per : 1;
    if (!a.gate) a.per = a.rows;
    // segments per group: enough items for every CTA, each of at least one row
    int64_t nseg = (NORM_BWD_CTAS + a.groups - 1) / a.groups;
    if (nseg > a.per) nseg = a.per;
    a.seg_rows = (a.per + nseg - 1) / nseg;
    a.nseg = (a.per + a.seg_rows - 1) / a.seg_rows;
    a.items = a.groups * a.nseg;
    a.pitch = (a.cols + 3) / 4 * 4;
}

size_t norm_bwd_workspace(const NormBwdArgs& a) {
    const int64_t ctas = a.items < NORM_BWD_CTAS ? a.items : NORM_BWD_CTAS;
    const int64_t lines = (a.w_pre ? ctas : 0) + (a.w_post ? ctas : 0) + ((a.gate && a.nseg > 1) ? a.items : 0);
    return (size_t)lines * (size_t)a.pitch * sizeof(float);
}

cudaError_t launch_norm(const NormArgs& a, bool bf16, cudaStream_t s) {
    int vpt, threads;
    shape_of(a.cols, vpt, threads);
    switch (vpt) {
    case 1: return bf16 ? run_norm<true, 1>(a, threads, s) : run_norm<false, 1>(a, threads, s);
    case 2: return bf16 ? run_norm<true, 2>(a, threads, s) : run_norm<false, 2>(a, threads, s);
    default: return bf16 ? run_norm<true, 4>(a, threads, s) : run_norm<false, 4>(a, threads, s);
    }
}

cudaError_t launch_norm_bwd(NormBwdArgs a, bool bf16, float* workspace, cudaStream_t s) {
    const int64_t ctas = a.items < NORM_BWD_CTAS ? a.items : NORM_BWD_CTAS;
    a.pre_part = workspace;
    a.post_part = a.pre_part + (a.w_pre ? ctas * a.pitch : 0);
    // one item per group: its sums are dgate's row
    a.gate_part = a.nseg > 1 ? a.post_part + (a.w_post ? ctas * a.pitch : 0) : a.dgate;
    a.gate_pitch = a.nseg > 1 ? a.pitch : a.cols;
    int vpt, threads;
    shape_of(a.cols, vpt, threads);
    switch (vpt) {
    case 1: return bf16 ? run_norm_bwd<true, 1>(a, threads, s) : run_norm_bwd<false, 1>(a, threads, s);
    case 2: return bf16 ? run_norm_bwd<true, 2>(a, threads, s) : run_norm_bwd<false, 2>(a, threads, s);
    default: return bf16 ? run_norm_bwd<true, 4>(a, threads, s) : run_norm_bwd<false, 4>(a, threads, s);
    }
}

}  // namespace fp4
