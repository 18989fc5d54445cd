// zdmmv_norm.cu -- zdmmv_add_rmsnorm_q8_0: the root-mean-square norm with the
// residual's addition, quantized to the Q8_0 blocks that the DMMV reads.
//
//   s = x + r,  y = (s * (1 / sqrt(mean(s^2) + eps))) * w,  blocks of 32: d = max|y| / 127, q = round(y / d)
//
// A row is read once and held in its threads' registers between the sum of
// squares and the quantization: T threads (whole warps) with V float4 each, eight
// neighbouring threads a block. Bound by memory with many rows (4 + 4 bytes in,
// 4 + 34/32 out, 2 with y, a value): 4096 x 4096 takes 40.2 us, 93% of the copy rate.
// By latency with few: then V = 1, as many
// threads as the row has float4 (8 x 4096: 2.8 us, 1 x 2048: 2.1 us).
#include <cmath>

#include "zdmmv_kv.cuh"

namespace zdmmv {
namespace {

struct NormArgs {
    const float *x, *r, *w;
    float *out;
    uint8_t *xq;
    __half *y;
    int64_t rows, x_stride, r_stride;
    int32_t cols;
    float eps;
};

constexpr int kNormMaxCols = 32768;
constexpr int kNormFewRows = 304;  // up to two rows an SM

// blockDim.x = T threads a row; blockDim.y rows a CTA.
template <int V> __global__ void __launch_bounds__(1024) add_rmsnorm_kernel(NormArgs a) {
    extern __shared__ __align__(16) uint8_t staged[];  // the rows' Q8_0 blocks
    __shared__ float part[32];
    const int tid = threadIdx.x, T = blockDim.x, lane = tid & 31, warps = T >> 5;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < a.rows;
    const int n4 = a.cols / 4;
    block_op_wait();
    block_op_release();
    float4 s[V];
    if (live) {
        const float4 *x = reinterpret_cast<const float4 *>(a.x + row * a.x_stride);
        const float4 *r = reinterpret_cast<const float4 *>(a.r + row * a.r_stride);
        float4 u[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int i = tid + k * T;
            s[k] = u[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < n4) {
                s[k] = x[i];
                if (a.r) u[k] = r[i];
            }
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (a.r) {
                s[k].x += u[k].x; s[k].y += u[k].y; s[k].z += u[k].z; s[k].w += u[k].w;
            }
            const int i = tid + k * T;
            if (a.out && i < n4) reinterpret_cast<float4 *>(a.out + row * a.cols)[i] = s[k];
        }
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) s[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // the weights' loads run beside the reduction (of 8 float4 they would cost spills, and wait)
    const auto weight = [&](int i) {
        return a.w && i < n4 ? reinterpret_cast<const float4 *>(a.w)[i] : make_float4(1.f, 1.f, 1.f, 1.f);
    };
    float4 ws[V <= 4 ? V : 1];
    if constexpr (V <= 4) {
#pragma unroll
        for (int k = 0; k < V; ++k) ws[k] = weight(tid + k * T);
    }
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) ss += (s[k].x * s[k].x + s[k].y * s[k].y) + (s[k].z * s[k].z + s[k].w * s[k].w);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (warps > 1) {  // uniform: T is the CTA's
        const int first = threadIdx.y * warps;
        if (lane == 0) part[first + (tid >> 5)] = ss;
        __syncthreads();
        ss = lane < warps ? part[first + lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(a.cols)), a.eps)));
    const int row_bytes = a.cols / kQK * 34;
    uint8_t *mine = staged + threadIdx.y * row_bytes;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int i = tid + k * T;
        if ((i & ~31) >= n4) break;  // whole warps: the 8 lanes of a block exchange its maximum
        float4 v = s[k], w;
        if constexpr (V <= 4) w = ws[k];
        else w = weight(i);
        v.x = __fmul_rn(__fmul_rn(v.x, rstd), w.x);
        v.y = __fmul_rn(__fmul_rn(v.y, rstd), w.y);
        v.z = __fmul_rn(__fmul_rn(v.z, rstd), w.z);
        v.w = __fmul_rn(__fmul_rn(v.w, rstd), w.w);
        unsigned short db;
        const uint32_t q = quantize_q8_0_quad(v, db);
        if (i >= n4) break;
        if (a.xq) {
            uint16_t *blk = reinterpret_cast<uint16_t *>(mine + i / 8 * 34);
            blk[1 + 2 * (i & 7)] = static_cast<uint16_t>(q);
            blk[2 + 2 * (i & 7)] = static_cast<uint16_t>(q >> 16);
            if ((i & 7) == 0) blk[0] = db;
        }
        if (a.y && live) {
            const float d = __half2float(__ushort_as_half(db));
            const __half2 lo = __floats2half2_rn(d * static_cast<int8_t>(q), d * static_cast<int8_t>(q >> 8));
            const __half2 hi = __floats2half2_rn(d * static_cast<int8_t>(q >> 16), d * static_cast<int8_t>(q >> 24));
            uint2 both;
            both.x = *reinterpret_cast<const uint32_t *>(&lo);
            both.y = *reinterpret_cast<const uint32_t *>(&hi);
            reinterpret_cast<uint2 *>(a.y + row * a.cols)[i] = both;
        }
    }
    if (!a.xq) return;
    // the CTA's rows are one stretch of bytes: out of shared memory in the widest words its start allows
    __syncthreads();
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * blockDim.y;
    const int bytes = static_cast<int>(min(static_cast<int64_t>(blockDim.y), a.rows - row0)) * row_bytes;
    uint8_t *dst = a.xq + row0 * row_bytes;
    const int t = threadIdx.y * T + tid, n = T * blockDim.y;
    const uint32_t align = static_cast<uint32_t>(row0 * row_bytes) & 15u;
    if (align == 0) {
        for (int i = t; i < bytes / 16; i += n) reinterpret_cast<uint4 *>(dst)[i] = reinterpret_cast<const uint4 *>(staged)[i];
        for (int i = bytes / 16 * 8 + t; i < bytes / 2; i += n)
            reinterpret_cast<uint16_t *>(dst)[i] = reinterpret_cast<const uint16_t *>(staged)[i];
    } else if ((align & 3u) == 0) {
        for (int i = t; i < bytes / 4; i += n) reinterpret_cast<uint32_t *>(dst)[i] = reinterpret_cast<const uint32_t *>(staged)[i];
        if (t == 0 && (bytes & 2)) reinterpret_cast<uint16_t *>(dst)[bytes / 2 - 1] = reinterpret_cast<const uint16_t *>(staged)[bytes / 2 - 1];
    } else {
        for (int i = t; i < bytes / 2; i += n)
            reinterpret_cast<uint16_t *>(dst)[i] = reinterpret_cast<const uint16_t *>(staged)[i];
    }
}

template <int V> cudaError_t launch_norm(const NormArgs &a, int threads, int rows_per_cta, cudaStream_t st) {
    const size_t smem = a.xq ? static_cast<size_t>(rows_per_cta) * (a.cols / kQK) * 34 : 0;
    const cudaError_t e = smem_limit_raised<&add_rmsnorm_kernel<V>>();
    if (e != cudaSuccess) return e;
    const int64_t ctas = (a.rows + rows_per_cta - 1) / rows_per_cta;
    return launch_block_op(add_rmsnorm_kernel<V>, dim3(static_cast<unsigned>(ctas)), dim3(threads, rows_per_cta), smem, st, a);
}

}  // namespace
}  // namespace zdmmv

using namespace zdmmv;

extern "C" zdmmv_status zdmmv_add_rmsnorm_q8_0(const zdmmv_rmsnorm_args *args, zdmmv_stream_t stream) {
    if (!args) return ZDMMV_ERR_NULL;
    const zdmmv_rmsnorm_args &g = *args;
    if (g.rows < 0 || g.rows > 0x7fffffff || g.cols <= 0 || g.cols % kQK || g.cols > kNormMaxCols ||
        !(g.eps > 0.0f) || !std::isfinite(g.eps))
        return ZDMMV_ERR_SHAPE;
    if (g.rows == 0) return ZDMMV_OK;
    if (!g.x || (!g.out && !g.xq && !g.y)) return ZDMMV_ERR_NULL;
    if (g.x_stride < g.cols || (g.residual && g.residual_stride < g.cols)) return ZDMMV_ERR_SHAPE;
    // out may only take the place of an input whose rows lie as its own do
    if ((g.out == g.x && g.x_stride != g.cols) || (g.out && g.out == g.residual && g.residual_stride != g.cols))
        return ZDMMV_ERR_SHAPE;
    if (kv_misaligned(g.x, 16) || kv_misaligned(g.residual, 16) || kv_misaligned(g.weight, 16) ||
        kv_misaligned(g.out, 16) || kv_misaligned(g.xq, 16) || kv_misaligned(g.y, 8) || g.x_stride % 4 ||
        (g.residual && g.residual_stride % 4))
        return ZDMMV_ERR_ALIGN;
    NormArgs a{g.x, g.residual, g.weight, g.out, static_cast<uint8_t *>(g.xq), static_cast<__half *>(g.y), g.rows,
               g.x_stride, g.residual_stride, static_cast<int32_t>(g.cols), g.eps};
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // Few rows: a thread a float4, up to 1024 of them. Many: up to four float4 a thread, so that a CTA of about 256
    // threads holds enough loads in flight and several CTAs share an SM.
    const int n4 = a.cols / 4;
    const int most = a.rows <= kNormFewRows ? 1024 : 256;
    int v = 1;
    while (v < 4 && n4 > v * most) v *= 2;
    if (n4 > v * 1024) v = 8;
    const int threads = ((n4 + v - 1) / v + 31) / 32 * 32;
    const int rows_per_cta = a.rows <= kNormFewRows ? 1 : (threads >= 256 ? 1 : 256 / threads);
    cudaError_t e;
    switch (v) {
    case 1: e = launch_norm<1>(a, threads, rows_per_cta, st); break;
    case 2: e = launch_norm<2>(a, threads, rows_per_cta, st); break;
    case 4: e = launch_norm<4>(a, threads, rows_per_cta, st); break;
    default: e = launch_norm<8>(a, threads, rows_per_cta, st); break;
    }
    return e == cudaSuccess ? ZDMMV_OK : ZDMMV_ERR_CUDA;
}
