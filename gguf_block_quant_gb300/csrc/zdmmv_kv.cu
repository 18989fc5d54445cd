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

constexpr int64_t kManyWarps = 152 * 64;  // as many (token, head) pairs as the device holds warps
constexpr int kAppendWarps = 4;

// The rotation of four neighbouring dimensions e0 .. e0+3 of a head at `src`: their cosines and sines, the partner
// dimensions, and which half of its pair each is. Every product and sum is rounded by itself (no fused multiply-add), so
// that the result is the same wherever it is computed.
struct Turn {
    float c[4], s[4];  // sign of s: minus for a pair's first dimension, whose result is x cos - partner sin
};

// FAST: four neighbouring dimensions are all rotated or none, and their partners and angles are neighbours too (pairs:
// rot_dim a multiple of 4; halves: rot_dim a multiple of 8), so everything is 128-bit loads.
template <bool FAST>
__device__ __forceinline__ Turn load_turn(const AppendArgs &a, int pos, int e0) {
    Turn t;
    const int half = a.rot_dim / 2;
    const float *row = a.rope + static_cast<int64_t>(pos) * a.rot_dim;
    if constexpr (FAST) {
        if (a.halves) {
            const bool second = e0 >= half;
            const int p = second ? e0 - half : e0;
            const float4 c = *reinterpret_cast<const float4 *>(row + p), s = *reinterpret_cast<const float4 *>(row + half + p);
            const float sign = second ? 1.0f : -1.0f;
            t.c[0] = c.x; t.c[1] = c.y; t.c[2] = c.z; t.c[3] = c.w;
            t.s[0] = sign * s.x; t.s[1] = sign * s.y; t.s[2] = sign * s.z; t.s[3] = sign * s.w;
        } else {
            const float2 c = *reinterpret_cast<const float2 *>(row + e0 / 2), s = *reinterpret_cast<const float2 *>(row + half + e0 / 2);
            t.c[0] = t.c[1] = c.x; t.c[2] = t.c[3] = c.y;
            t.s[0] = -s.x; t.s[1] = s.x; t.s[2] = -s.y; t.s[3] = s.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = e0 + i;
            t.c[i] = 1.0f;
            t.s[i] = 0.0f;
            if (e >= a.rot_dim) continue;
            const bool second = a.halves ? e >= half : (e & 1) != 0;
            const int p = a.halves ? (second ? e - half : e) : e / 2;
            t.c[i] = row[p];
            t.s[i] = second ? row[half + p] : -row[half + p];
        }
    }
    return t;
}
template <bool FAST>
__device__ __forceinline__ void load_head(const AppendArgs &a, const float *src, int e0, bool turned, float (&v)[4], float (&o)[4]) {
    const float4 x = *reinterpret_cast<const float4 *>(src + e0);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    o[0] = v[1]; o[1] = v[0]; o[2] = v[3]; o[3] = v[2];
    if (!turned || !a.halves) return;
    const int half = a.rot_dim / 2;
    if constexpr (FAST) {
        const float4 y = *reinterpret_cast<const float4 *>(src + (e0 >= half ? e0 - half : e0 + half));
        o[0] = y.x; o[1] = y.y; o[2] = y.z; o[3] = y.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = e0 + i;
            if (e < a.rot_dim) o[i] = src[e >= half ? e - half : e + half];
        }
    }
}

// One warp per token and HEADS neighbouring heads of its q, k and v: lane l holds the four dimensions 4l .. 4l+3 of each
// pass of 128, loads them for all its heads before it stores any (so q_out may be q), and keeps the token's cosines and
// sines for all of them. Bound by memory for prompts (HEADS = 4: four heads' loads in flight), by latency for a few
// tokens (HEADS = 1: as many warps as heads).
template <int NB, int HEADS, bool FAST>
__global__ void __launch_bounds__(kAppendWarps * 32) kv_append_kernel(AppendArgs a) {
    using G = KvGeom<NB>;
    constexpr int kPass = (G::kDim + 127) / 128;
    const int lane = threadIdx.x & 31;
    const int heads = a.n_q_heads + 2 * a.c.n_kv_heads;
    const int groups = (heads + HEADS - 1) / HEADS;
    const int64_t job = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
    const int64_t tok = job / groups;
    const int h0 = static_cast<int>(job - tok * groups) * HEADS;
    block_op_wait();
    block_op_release();
    if (tok >= a.n_tok) return;
    const int pos = a.pos[tok], seq = a.seq[tok];
    // where the token goes; bad: outside what the cache and the rotation table have
    const int slot = pos / a.c.page_tokens, in = pos - slot * a.c.page_tokens;
    const bool pad = pos < 0;
    bool bad = !pad && (seq < 0 || seq >= a.c.n_seq || slot >= a.c.max_pages || (a.rot_dim > 0 && pos >= a.rope_rows));
    const int page = pad || bad ? 0 : a.c.table[static_cast<int64_t>(seq) * a.c.max_pages + slot];
    if (page < 0 || page >= a.c.n_pages) bad = true;
    if (bad && lane == 0 && a.status) *a.status = 1;
    const bool ok = !pad && !bad;
    uint8_t *tiles = a.c.pages + (ok ? page : 0) * a.c.page_bytes + static_cast<int64_t>(in / kKvSlab) * G::kTileBytes;
    const int64_t head_bytes = static_cast<int64_t>(a.c.page_tokens / kKvSlab) * G::kTileBytes;
    const int r = in % kKvSlab;
    const float fill = bad ? __int_as_float(0x7fffffff) : 0.0f;
    float v[HEADS][kPass][4], o[HEADS][kPass][4];
    Turn turn[kPass];
#pragma unroll
    for (int u = 0; u < HEADS; ++u)
#pragma unroll
        for (int p = 0; p < kPass; ++p) {
            const int head = h0 + u, kvh = head - a.n_q_heads, e0 = p * 128 + 4 * lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[u][p][i] = fill;
            if (!ok || e0 >= G::kDim || head >= heads) continue;
            const float *src = kvh < 0 ? a.q + tok * a.q_stride + static_cast<int64_t>(head) * G::kDim
                               : (kvh < a.c.n_kv_heads ? a.k + tok * a.k_stride + static_cast<int64_t>(kvh) * G::kDim
                                                       : a.v + tok * a.v_stride + static_cast<int64_t>(kvh - a.c.n_kv_heads) * G::kDim);
            load_head<FAST>(a, src, e0, e0 < a.rot_dim && kvh < a.c.n_kv_heads, v[u][p], o[u][p]);
        }
#pragma unroll
    for (int p = 0; p < kPass; ++p)
        if (ok && p * 128 + 4 * lane < a.rot_dim) turn[p] = load_turn<FAST>(a, pos, p * 128 + 4 * lane);
    __syncwarp();
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
        const int head = h0 + u, kvh = head - a.n_q_heads;
        if (head >= heads) break;
#pragma unroll
        for (int p = 0; p < kPass; ++p) {
            const int e0 = p * 128 + 4 * lane;
            const bool inside = e0 < G::kDim;
            float (&x)[4] = v[u][p];
            if (ok && e0 < a.rot_dim && kvh < a.c.n_kv_heads) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (FAST || e0 + i < a.rot_dim) x[i] = __fadd_rn(__fmul_rn(x[i], turn[p].c[i]), __fmul_rn(o[u][p][i], turn[p].s[i]));
            }
            if (kvh < 0) {
                if (inside)
                    *reinterpret_cast<float4 *>(a.q_out + (tok * a.n_q_heads + head) * G::kDim + e0) = make_float4(x[0], x[1], x[2], x[3]);
                continue;
            }
            const bool is_k = kvh < a.c.n_kv_heads;
            const int h = is_k ? kvh : kvh - a.c.n_kv_heads;
            // the first value of the largest magnitude, over the block's 8 lanes
            float m = x[0];
            int at = e0;
#pragma unroll
            for (int i = 1; i < 4; ++i)
                if (fabsf(x[i]) > fabsf(m)) { m = x[i]; at = e0 + i; }
#pragma unroll
            for (int s = 1; s < 8; s <<= 1) {
                const float om = __shfl_xor_sync(0xffffffffu, m, s);
                const int oat = __shfl_xor_sync(0xffffffffu, at, s);
                if (fabsf(om) > fabsf(m) || (fabsf(om) == fabsf(m) && oat < at)) { m = om; at = oat; }
            }
            const float d = m / -8.0f;
            const float id = d != 0.0f ? 1.0f / d : 0.0f;
            const __half dh = __float2half_rn(d);
            uint32_t code[4], packed = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = static_cast<int>(__fadd_rn(__fmul_rn(x[i], id), 8.5f));
                code[i] = c < 0 ? 0 : (c > 15 ? 15 : c);
                packed |= code[i] << (4 * i);
            }
            const int b = e0 / kQK, g = (e0 % kQK) / 4;
            const uint32_t upper = __shfl_down_sync(0xffffffffu, packed, 1);
            if (!inside) continue;
            if (ok) {
                uint8_t *tile = tiles + h * head_bytes;
                __half *scales = reinterpret_cast<__half *>(tile + (is_k ? G::kKScaleAt : G::kVScaleAt));
                if (g == 0) scales[G::scale_half(r, b)] = dh;
                if (is_k) {
                    if ((g & 1) == 0) reinterpret_cast<uint32_t *>(tile)[G::k_word(r, b, g / 2)] = packed | (upper << 16);
                } else {
                    reinterpret_cast<uint16_t *>(tile + G::kVAt)[G::v_half(r, b, g)] = static_cast<uint16_t>(packed);
                }
            }
            __half *val = is_k ? a.k_val : a.v_val;
            if (val) {
                const float df = __half2float(dh);
                __half2 w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    w[i] = __floats2half2_rn(df * (static_cast<float>(code[2 * i]) - 8.0f), df * (static_cast<float>(code[2 * i + 1]) - 8.0f));
                *reinterpret_cast<uint2 *>(val + (tok * a.c.n_kv_heads + h) * G::kDim + e0) = *reinterpret_cast<uint2 *>(w);
            }
        }
    }
}

template <int NB, int HEADS, bool FAST> cudaError_t launch_append_as(const AppendArgs &a, cudaStream_t st) {
    const int heads = a.n_q_heads + 2 * a.c.n_kv_heads;
    const int64_t jobs = static_cast<int64_t>(a.n_tok) * ((heads + HEADS - 1) / HEADS);
    const int64_t ctas = (jobs + kAppendWarps - 1) / kAppendWarps;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_block_op(kv_append_kernel<NB, HEADS, FAST>, dim3(static_cast<unsigned>(ctas)), dim3(kAppendWarps * 32), 0, st, a);
}
template <int NB> cudaError_t launch_append(const AppendArgs &a, cudaStream_t st) {
    const bool fast = a.rot_dim % (a.halves ? 8 : 4) == 0;
    const int64_t warps = static_cast<int64_t>(a.n_tok) * (a.n_q_heads + 2 * a.c.n_kv_heads);
    if (warps > kManyWarps) return fast ? launch_append_as<NB, 4, true>(a, st) : launch_append_as<NB, 4, false>(a, st);
    return fast ? launch_append_as<NB, 1, true>(a, st) : launch_append_as<NB, 1, false>(a, st);
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
