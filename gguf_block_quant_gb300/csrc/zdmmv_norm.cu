// zdmmv_norm.cu -- zdmmv_add_rmsnorm_q8_0: the root-mean-square norm with the
// residual's addition, quantized to the Q8_0 blocks that the DMMV reads.
//
//   s = x + r,  y = (s * (1 / sqrt(mean(s^2) + eps))) * w,  blocks of 32: d = max|y| / 127, q = round(y / d)
//
// One CTA per row; the sums are kept in shared memory between the two passes.
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

constexpr int kNormThreads = 256;
constexpr int kNormMaxCols = 32768;

__global__ void __launch_bounds__(kNormThreads) add_rmsnorm_kernel(NormArgs a) {
    extern __shared__ float4 s4[];
    __shared__ float part[kNormThreads / 32];
    block_op_wait();
    block_op_release();
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float4 *x = reinterpret_cast<const float4 *>(a.x + row * a.x_stride);
    const float4 *r = a.r ? reinterpret_cast<const float4 *>(a.r + row * a.r_stride) : nullptr;
    float4 *out = a.out ? reinterpret_cast<float4 *>(a.out + row * a.cols) : nullptr;
    const int n4 = a.cols / 4;
    float ss = 0.0f;
    for (int i = tid; i < n4; i += kNormThreads) {
        float4 v = x[i];
        if (r) {
            const float4 u = r[i];
            v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
        if (out) out[i] = v;
        s4[i] = v;
        ss += v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
    }
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int k = 0; k < kNormThreads / 32; ++k) ss += part[k];
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(a.cols)), a.eps)));
    // eight lanes a block of 32; the loop count is uniform over the warp
    for (int i0 = warp * 32; i0 < n4; i0 += kNormThreads) {
        const int i = i0 + lane;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n4) {
            v = s4[i];
            const float4 w = a.w ? reinterpret_cast<const float4 *>(a.w)[i] : make_float4(1.f, 1.f, 1.f, 1.f);
            v.x = __fmul_rn(__fmul_rn(v.x, rstd), w.x);
            v.y = __fmul_rn(__fmul_rn(v.y, rstd), w.y);
            v.z = __fmul_rn(__fmul_rn(v.z, rstd), w.z);
            v.w = __fmul_rn(__fmul_rn(v.w, rstd), w.w);
        }
        unsigned short db;
        const uint32_t q = quantize_q8_0_quad(v, db);
        if (i >= n4) continue;
        if (a.xq) {
            uint8_t *blk = a.xq + (row * (a.cols / kQK) + i / 8) * 34;
            uint16_t *dst = reinterpret_cast<uint16_t *>(blk + 2 + 4 * (i & 7));
            dst[0] = static_cast<uint16_t>(q);
            dst[1] = static_cast<uint16_t>(q >> 16);
            if ((i & 7) == 0) *reinterpret_cast<unsigned short *>(blk) = db;
        }
        if (a.y) {
            const float d = __half2float(__ushort_as_half(db));
            __half2 *y = reinterpret_cast<__half2 *>(a.y + row * a.cols + 4 * i);
            y[0] = __floats2half2_rn(d * static_cast<int8_t>(q), d * static_cast<int8_t>(q >> 8));
            y[1] = __floats2half2_rn(d * static_cast<int8_t>(q >> 16), d * static_cast<int8_t>(q >> 24));
        }
    }
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
    const size_t smem = static_cast<size_t>(g.cols) * 4;
    if (smem > 47 * 1024 &&
        cudaFuncSetAttribute(add_rmsnorm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxCols * 4) !=
            cudaSuccess)
        return ZDMMV_ERR_CUDA;
    return launch_block_op(add_rmsnorm_kernel, dim3(static_cast<unsigned>(g.rows)), kNormThreads, smem,
                           reinterpret_cast<cudaStream_t>(stream), a) == cudaSuccess
               ? ZDMMV_OK
               : ZDMMV_ERR_CUDA;
}
