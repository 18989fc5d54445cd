// zdmmv_attn.cu -- zdmmv_attn_q4_0: attention over the paged 4-bit cache.
//
//   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale * (q . k_t) - m),  m the running maximum
//
// One CTA per (new token, query head): tile by tile, the warps form the tile's 16
// scores, then every thread updates its dimensions of the sum over V.
#include <cmath>

#include "zdmmv_kv.cuh"

namespace zdmmv {
namespace {

struct AttnArgs {
    KvView c;
    const float *q;
    const int32_t *q_start, *kv_len;
    float *out;
    int32_t *status;
    int64_t q_stride;
    int32_t n_tok, n_q_heads, max_q_len, max_kv_len, window;
    float scale;
};

constexpr int kThreads = 128;

template <int NB> __global__ void __launch_bounds__(kThreads) attn_kernel(AttnArgs a) {
    using G = KvGeom<NB>;
    __shared__ float q[G::kDim];
    __shared__ float score[kKvSlab];
    block_op_wait();
    block_op_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int head = blockIdx.x % a.n_q_heads;
    const int item = blockIdx.x / a.n_q_heads;
    const int seq = item / a.max_q_len, i = item % a.max_q_len;
    int q0 = a.q_start[seq], q1 = a.q_start[seq + 1];
    const int len = a.kv_len[seq];
    bool bad = q0 < 0 || q1 < q0 || q1 > a.n_tok || q1 - q0 > a.max_q_len || len < 0 || len > a.max_kv_len ||
               len > static_cast<int64_t>(a.c.max_pages) * a.c.page_tokens;
    q0 = max(q0, 0);
    q1 = min(q1, a.n_tok);
    if (i >= q1 - q0) return;
    const int64_t row = q0 + i;
    const int end = bad ? 0 : max(0, len - (q1 - q0 - 1 - i));
    const int low = a.window > 0 ? max(0, end - a.window) : 0;
    const int kvh = head / (a.n_q_heads / a.c.n_kv_heads);
    for (int e = tid; e < G::kDim; e += kThreads) q[e] = a.q[row * a.q_stride + static_cast<int64_t>(head) * G::kDim + e];
    __syncthreads();
    float m = -INFINITY, l = 0.0f, o[2] = {0.0f, 0.0f};
    for (int t0 = low / kKvSlab * kKvSlab; t0 < end; t0 += kKvSlab) {
        const int page = a.c.table[static_cast<int64_t>(seq) * a.c.max_pages + t0 / a.c.page_tokens];
        if (page < 0 || page >= a.c.n_pages) {
            bad = true;
            break;
        }
        const uint8_t *tile = a.c.pages + page * a.c.page_bytes +
                              static_cast<int64_t>(kvh * (a.c.page_tokens / kKvSlab) + t0 % a.c.page_tokens / kKvSlab) * G::kTileBytes;
        const __half *ks = reinterpret_cast<const __half *>(tile + G::kKScaleAt);
        const __half *vs = reinterpret_cast<const __half *>(tile + G::kVScaleAt);
        for (int r = warp; r < kKvSlab; r += kThreads / 32) {
            float s = 0.0f;
            for (int w = lane; w < NB * 4; w += 32) {
                const uint32_t code = reinterpret_cast<const uint32_t *>(tile)[G::k_word(r, w / 4, w % 4)];
                const float d = __half2float(ks[G::scale_half(r, w / 4)]);
                float part = 0.0f;
                for (int j = 0; j < 8; ++j) part += q[w * 8 + j] * (static_cast<float>((code >> (4 * j)) & 15) - 8.0f);
                s += d * part;
            }
            for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
            if (lane == 0) score[r] = t0 + r >= low && t0 + r < end ? s * a.scale : -INFINITY;
        }
        __syncthreads();
        float top = m;
        for (int r = 0; r < kKvSlab; ++r) top = fmaxf(top, score[r]);
        const float keep = m == -INFINITY ? 0.0f : expf(m - top);
        m = top;
        l *= keep;
        o[0] *= keep;
        o[1] *= keep;
        for (int r = 0; r < kKvSlab; ++r) {
            if (score[r] == -INFINITY) continue;
            const float p = expf(score[r] - m);
            l += p;
            for (int k = 0; k < 2; ++k) {
                const int e = tid + k * kThreads;
                if (e >= G::kDim) continue;
                const uint32_t code = reinterpret_cast<const uint16_t *>(tile + G::kVAt)[G::v_half(r, e / kQK, e % kQK / 4)];
                const float v = __half2float(vs[G::scale_half(r, e / kQK)]) *
                                (static_cast<float>((code >> (4 * (e % 4))) & 15) - 8.0f);
                o[k] += p * v;
            }
        }
        __syncthreads();
    }
    if (bad && tid == 0 && a.status) *a.status = 1;
    for (int k = 0; k < 2; ++k) {
        const int e = tid + k * kThreads;
        if (e < G::kDim)
            a.out[(row * a.n_q_heads + head) * G::kDim + e] = bad ? __int_as_float(0x7fffffff) : (l > 0.0f ? o[k] / l : 0.0f);
    }
}

template <int NB> cudaError_t launch_attn(const AttnArgs &a, cudaStream_t st) {
    const int64_t ctas = static_cast<int64_t>(a.c.n_seq) * a.max_q_len * a.n_q_heads;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_block_op(attn_kernel<NB>, dim3(static_cast<unsigned>(ctas)), kThreads, 0, st, a);
}

}  // namespace
}  // namespace zdmmv

using namespace zdmmv;

extern "C" {

size_t zdmmv_attn_q4_0_workspace_bytes(const zdmmv_kv_cache *cache, int n_q_heads, int max_q_len, int max_kv_len) {
    (void)cache; (void)n_q_heads; (void)max_q_len; (void)max_kv_len;
    return 0;
}

zdmmv_status zdmmv_attn_q4_0(const zdmmv_kv_cache *cache, const zdmmv_attn_args *args, zdmmv_stream_t stream) {
    if (!args) return ZDMMV_ERR_NULL;
    AttnArgs a{};
    const zdmmv_status st = kv_check(cache, &a.c);
    if (st != ZDMMV_OK) return st;
    const zdmmv_attn_args &g = *args;
    if (g.n_tok < 0 || g.n_q_heads < 1 || g.n_q_heads > 65535 || g.n_q_heads % cache->n_kv_heads || g.max_q_len < 1 ||
        g.max_kv_len < 0 || g.window < 0 || !std::isfinite(g.scale))
        return ZDMMV_ERR_SHAPE;
    if (g.n_tok == 0) return ZDMMV_OK;
    if (!g.q || !g.q_start || !g.kv_len || !g.out) return ZDMMV_ERR_NULL;
    if (g.q_stride < static_cast<int64_t>(g.n_q_heads) * cache->head_dim) return ZDMMV_ERR_SHAPE;
    if (kv_misaligned(g.q, 16) || kv_misaligned(g.out, 16) || kv_misaligned(g.workspace, 16) ||
        kv_misaligned(g.q_start, 4) || kv_misaligned(g.kv_len, 4) || kv_misaligned(g.status_dev, 4) || g.q_stride % 4)
        return ZDMMV_ERR_ALIGN;
    const size_t need = zdmmv_attn_q4_0_workspace_bytes(cache, g.n_q_heads, g.max_q_len, g.max_kv_len);
    if (need && !g.workspace) return ZDMMV_ERR_NULL;
    if (g.workspace_bytes < need) return ZDMMV_ERR_SIZE;
    a.q = g.q; a.q_start = g.q_start; a.kv_len = g.kv_len; a.out = g.out; a.status = g.status_dev;
    a.q_stride = g.q_stride;
    a.n_tok = g.n_tok; a.n_q_heads = g.n_q_heads; a.max_q_len = g.max_q_len; a.max_kv_len = g.max_kv_len;
    a.window = g.window; a.scale = g.scale;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
    switch (kv_blocks(cache->head_dim)) {
    case 2: e = launch_attn<2>(a, s); break;
    case 3: e = launch_attn<3>(a, s); break;
    case 4: e = launch_attn<4>(a, s); break;
    case 6: e = launch_attn<6>(a, s); break;
    case 8: e = launch_attn<8>(a, s); break;
    }
    return e == cudaSuccess ? ZDMMV_OK : ZDMMV_ERR_CUDA;
}

}  // extern "C"
