// zdmmv_kv.cu -- the paged 4-bit cache's geometry and zdmmv_kv_append_q4_0: the
// position rotation of q and k, and k and v quantized to Q4_0 into their pages.
#include "zdmmv_kv.cuh"

namespace zdmmv {

int kv_blocks(int head_dim) {
    switch (head_dim) {
    case 64: case 96: case 128: case 192: case 256: return head_dim / kQK;
    default: return 0;
    }
}

namespace {
bool kv_geometry_ok(int page_tokens, int n_kv_heads, int head_dim) {
    return kv_blocks(head_dim) != 0 && page_tokens >= kKvSlab && page_tokens <= 1024 && page_tokens % kKvSlab == 0 &&
           n_kv_heads >= 1 && n_kv_heads <= 1024;
}
}  // namespace

zdmmv_status kv_check(const zdmmv_kv_cache *c, KvView *out) {
    if (!c) return ZDMMV_ERR_NULL;
    if (!kv_geometry_ok(c->page_tokens, c->n_kv_heads, c->head_dim) || c->n_pages < 1 || c->n_seq < 1 ||
        c->max_pages < 1)
        return ZDMMV_ERR_SHAPE;
    if (!c->pages || !c->page_table) return ZDMMV_ERR_NULL;
    if (kv_misaligned(c->pages, 16) || kv_misaligned(c->page_table, 4)) return ZDMMV_ERR_ALIGN;
    out->pages = static_cast<uint8_t *>(c->pages);
    out->table = c->page_table;
    out->n_pages = c->n_pages;
    out->page_bytes = static_cast<int64_t>(zdmmv_kv_page_bytes(c->page_tokens, c->n_kv_heads, c->head_dim));
    out->n_seq = c->n_seq;
    out->max_pages = c->max_pages;
    out->page_tokens = c->page_tokens;
    out->n_kv_heads = c->n_kv_heads;
    return ZDMMV_OK;
}

namespace {

struct AppendArgs {
    KvView c;
    const float *k, *v, *q;
    const int32_t *seq, *pos;
    const float *rope;
    float *q_out;
    __half *k_val, *v_val;
    int32_t *status;
    int64_t k_stride, v_stride, q_stride, rope_rows;
    int32_t n_tok, n_q_heads, rot_dim, halves;
};

constexpr int kAppendWarps = 4;

// One warp per (token, head) of q, k and v: lane l holds the four dimensions
// 4l .. 4l+3 of each pass of 128. All of a head is loaded before any of it is
// stored, so q_out may be q.
template <int NB>
__global__ void __launch_bounds__(kAppendWarps * 32) kv_append_kernel(AppendArgs a) {
    using G = KvGeom<NB>;
    constexpr int kPass = (G::kDim + 127) / 128;
    block_op_wait();
    block_op_release();
    const int lane = threadIdx.x & 31;
    const int heads = a.n_q_heads + 2 * a.c.n_kv_heads;
    const int64_t job = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
    const int64_t tok = job / heads;
    if (tok >= a.n_tok) return;
    int head = static_cast<int>(job - tok * heads);
    const int kind = head < a.n_q_heads ? 0 : (head < a.n_q_heads + a.c.n_kv_heads ? 1 : 2);  // q, k, v
    head -= kind == 0 ? 0 : (kind == 1 ? a.n_q_heads : a.n_q_heads + a.c.n_kv_heads);
    const int pos = a.pos[tok], seq = a.seq[tok];
    // where the token goes; bad: outside what the cache and the rotation table have
    bool bad = false;
    uint8_t *tile = nullptr;
    int r = 0;
    if (pos >= 0) {
        const int slot = pos / a.c.page_tokens, in = pos - slot * a.c.page_tokens;
        bad = seq < 0 || seq >= a.c.n_seq || slot >= a.c.max_pages || (a.rot_dim > 0 && pos >= a.rope_rows);
        if (!bad) {
            const int page = a.c.table[static_cast<int64_t>(seq) * a.c.max_pages + slot];
            bad = page < 0 || page >= a.c.n_pages;
            r = in % kKvSlab;
            tile = a.c.pages + page * a.c.page_bytes +
                   static_cast<int64_t>(head * (a.c.page_tokens / kKvSlab) + in / kKvSlab) * G::kTileBytes;
        }
    }
    if (bad && lane == 0 && a.status) *a.status = 1;
    const float *src = kind == 0 ? a.q + tok * a.q_stride : (kind == 1 ? a.k + tok * a.k_stride : a.v + tok * a.v_stride);
    src += static_cast<int64_t>(head) * G::kDim;
    float v[kPass][4];
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
        const int e0 = p * 128 + 4 * lane;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = e0 + i;
            v[p][i] = 0.0f;
            if (e >= G::kDim) continue;
            if (pos < 0 || bad) {
                v[p][i] = bad ? __int_as_float(0x7fffffff) : 0.0f;
            } else if (kind == 2 || e >= a.rot_dim) {
                v[p][i] = src[e];
            } else {
                const int half = a.rot_dim / 2;
                const bool second = a.halves ? e >= half : (e & 1) != 0;
                const int pair = a.halves ? (second ? e - half : e) : e / 2;
                const int other = a.halves ? (second ? e - half : e + half) : e ^ 1;
                const float c = a.rope[static_cast<int64_t>(pos) * a.rot_dim + pair];
                const float s = a.rope[static_cast<int64_t>(pos) * a.rot_dim + half + pair];
                const float own = src[e], oth = src[other];
                v[p][i] = second ? __fadd_rn(__fmul_rn(oth, s), __fmul_rn(own, c))
                                 : __fsub_rn(__fmul_rn(own, c), __fmul_rn(oth, s));
            }
        }
    }
    __syncwarp();
    if (kind == 0) {
        float *dst = a.q_out + (tok * a.n_q_heads + head) * G::kDim;
#pragma unroll
        for (int p = 0; p < kPass; ++p) {
            const int e0 = p * 128 + 4 * lane;
            if (e0 < G::kDim) *reinterpret_cast<float4 *>(dst + e0) = make_float4(v[p][0], v[p][1], v[p][2], v[p][3]);
        }
        return;
    }
    __half *val = kind == 1 ? a.k_val : a.v_val;
    if (val) val += (tok * a.c.n_kv_heads + head) * G::kDim;
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
        const int e0 = p * 128 + 4 * lane;
        const bool in = e0 < G::kDim;
        // the first value of the largest magnitude, over the block's 8 lanes
        float m = v[p][0];
        int at = e0;
#pragma unroll
        for (int i = 1; i < 4; ++i)
            if (fabsf(v[p][i]) > fabsf(m)) { m = v[p][i]; at = e0 + i; }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            const float om = __shfl_xor_sync(0xffffffffu, m, o);
            const int oat = __shfl_xor_sync(0xffffffffu, at, o);
            if (fabsf(om) > fabsf(m) || (fabsf(om) == fabsf(m) && oat < at)) { m = om; at = oat; }
        }
        const float d = m / -8.0f;
        const float id = d != 0.0f ? 1.0f / d : 0.0f;
        const __half dh = __float2half_rn(d);
        uint32_t code[4], packed = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = static_cast<int>(__fadd_rn(__fmul_rn(v[p][i], id), 8.5f));
            code[i] = c < 0 ? 0 : (c > 15 ? 15 : c);
            packed |= code[i] << (4 * i);
        }
        const int b = e0 / kQK, g = (e0 % kQK) / 4;
        const uint32_t upper = __shfl_down_sync(0xffffffffu, packed, 1);
        if (tile && !bad && in) {
            __half *scales = reinterpret_cast<__half *>(tile + (kind == 1 ? G::kKScaleAt : G::kVScaleAt));
            if (g == 0) scales[G::scale_half(r, b)] = dh;
            if (kind == 1) {
                if ((g & 1) == 0) reinterpret_cast<uint32_t *>(tile)[G::k_word(r, b, g / 2)] = packed | (upper << 16);
            } else {
                reinterpret_cast<uint16_t *>(tile + G::kVAt)[G::v_half(r, b, g)] = static_cast<uint16_t>(packed);
            }
        }
        if (val && in) {
            const float df = __half2float(dh);
#pragma unroll
            for (int i = 0; i < 4; i += 2)
                *reinterpret_cast<__half2 *>(val + e0 + i) =
                    __floats2half2_rn(df * (static_cast<float>(code[i]) - 8.0f), df * (static_cast<float>(code[i + 1]) - 8.0f));
        }
    }
}

template <int NB> cudaError_t launch_append(const AppendArgs &a, cudaStream_t st) {
    const int64_t jobs = static_cast<int64_t>(a.n_tok) * (a.n_q_heads + 2 * a.c.n_kv_heads);
    const int64_t ctas = (jobs + kAppendWarps - 1) / kAppendWarps;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_block_op(kv_append_kernel<NB>, dim3(static_cast<unsigned>(ctas)), kAppendWarps * 32, 0, st, a);
}

}  // namespace
}  // namespace zdmmv

using namespace zdmmv;

extern "C" {

size_t zdmmv_kv_page_bytes(int page_tokens, int n_kv_heads, int head_dim) {
    if (!kv_geometry_ok(page_tokens, n_kv_heads, head_dim)) return 0;
    return static_cast<size_t>(page_tokens / kKvSlab) * n_kv_heads * 18 * head_dim;
}

zdmmv_status zdmmv_kv_append_q4_0(const zdmmv_kv_cache *cache, const zdmmv_kv_append_args *args,
                                  zdmmv_stream_t stream) {
    if (!args) return ZDMMV_ERR_NULL;
    AppendArgs a{};
    const zdmmv_status st = kv_check(cache, &a.c);
    if (st != ZDMMV_OK) return st;
    const zdmmv_kv_append_args &g = *args;
    const int64_t kv = static_cast<int64_t>(cache->n_kv_heads) * cache->head_dim;
    const int64_t qn = static_cast<int64_t>(g.n_q_heads) * cache->head_dim;
    if (g.n_tok < 0 || g.rot_dim < 0 || g.rot_dim % 2 || g.rot_dim > cache->head_dim ||
        (g.rope_style != ZDMMV_ROPE_PAIRS && g.rope_style != ZDMMV_ROPE_HALVES) ||
        (g.rot_dim > 0 && g.rope_rows < 1) || g.n_q_heads < 0 || g.n_q_heads > 65535 || (g.q != nullptr) != (g.n_q_heads > 0))
        return ZDMMV_ERR_SHAPE;
    if (g.n_tok == 0) return ZDMMV_OK;
    if (!g.k || !g.v || !g.seq || !g.pos || (g.rot_dim > 0 && !g.rope) || (g.q && !g.q_out)) return ZDMMV_ERR_NULL;
    if (g.k_stride < kv || g.v_stride < kv || (g.q && g.q_stride < qn)) return ZDMMV_ERR_SHAPE;
    if (g.q && g.q_out == g.q && g.q_stride != qn) return ZDMMV_ERR_SHAPE;
    if (kv_misaligned(g.k, 16) || kv_misaligned(g.v, 16) || kv_misaligned(g.q, 16) || kv_misaligned(g.q_out, 16) ||
        kv_misaligned(g.rope, 16) || kv_misaligned(g.k_val, 8) || kv_misaligned(g.v_val, 8) || kv_misaligned(g.seq, 4) ||
        kv_misaligned(g.pos, 4) || kv_misaligned(g.status_dev, 4) || g.k_stride % 4 || g.v_stride % 4 ||
        (g.q && g.q_stride % 4))
        return ZDMMV_ERR_ALIGN;
    a.k = g.k; a.v = g.v; a.q = g.q;
    a.seq = g.seq; a.pos = g.pos; a.rope = g.rope;
    a.q_out = g.q_out;
    a.k_val = static_cast<__half *>(g.k_val);
    a.v_val = static_cast<__half *>(g.v_val);
    a.status = g.status_dev;
    a.k_stride = g.k_stride; a.v_stride = g.v_stride; a.q_stride = g.q_stride; a.rope_rows = g.rope_rows;
    a.n_tok = g.n_tok; a.n_q_heads = g.n_q_heads; a.rot_dim = g.rot_dim; a.halves = g.rope_style == ZDMMV_ROPE_HALVES;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
    switch (kv_blocks(cache->head_dim)) {
    case 2: e = launch_append<2>(a, s); break;
    case 3: e = launch_append<3>(a, s); break;
    case 4: e = launch_append<4>(a, s); break;
    case 6: e = launch_append<6>(a, s); break;
    case 8: e = launch_append<8>(a, s); break;
    }
    return e == cudaSuccess ? ZDMMV_OK : ZDMMV_ERR_CUDA;
}

}  // extern "C"
