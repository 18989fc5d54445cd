// zdmmv_attn_weights.cu -- zdmmv_attn_weights_q4_0: what the query rows of a call give each cached token,
//
//   out_t = keep before_t + sum_c exp(scale (q_c . k_t) - lse_c)      over the columns c (query rows of the kv head) that see t,
//
// from the keys alone: half of the cache's bytes, and no product with V.
//
// The scores are formed as in the narrow kernel of zdmmv_attn.cuh (A = a tile's 16 tokens of codes, B = four columns' upper and
// lower parts; a product's C holds a column's two sums side by side), so that they agree with those that lse was made of. Every
// tile belongs to one warp, which goes over all columns, four at a time, and adds up its tokens' weights in a fixed order:
// nothing is joined, no atomics. Up to kBlockCols columns the parts of q lie in shared memory once; more columns come in blocks
// of as many, between which the weights wait in shared memory.
// The keys go from the cache to registers (they lie there in the order of the fragments): a lane's 128-bit loads of a tile run a
// tile ahead of the products.
#include <algorithm>
#include <cmath>

#include "zdmmv_attn.cuh"
#include "zdmmv_internal.h"

namespace zdmmv {
namespace {

constexpr int kWeightWarps = 8, kWeightThreads = kWeightWarps * 32;
constexpr int kBlockCols = 64;       // columns whose parts of q lie in shared memory at once
constexpr int kMostChunk = 512;      // tiles of a CTA with several blocks of columns: their weights take 32 KB
constexpr int kAllCols = 0x7fffff00; // a column tile of all columns

struct WeightArgs {
    AttnArgs a;            // out, the workspace's and the split's fields unused
    FastDiv by_chunks;
    const float *lse_in, *before;
    float *out;
    int64_t before_stride, out_stride;  // between kv heads
    int32_t chunks, chunk;              // CTAs of an item, tiles of one
    float keep;
};

template <int N, int W> __device__ __forceinline__ void ldg_words(const uint8_t *at, int step, uint32_t (&w)[N]) {
#pragma unroll
    for (int c = 0; c < N / W; ++c) {
        const uint8_t *p = at + c * step;
        if constexpr (W == 4) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p));
            w[4 * c] = x.x; w[4 * c + 1] = x.y; w[4 * c + 2] = x.z; w[4 * c + 3] = x.w;
        } else if constexpr (W == 2) {
            const uint2 x = __ldg(reinterpret_cast<const uint2 *>(p));
            w[2 * c] = x.x; w[2 * c + 1] = x.y;
        } else {
            w[c] = __ldg(reinterpret_cast<const uint32_t *>(p));
        }
    }
}
// A lane's part of a tile's keys: of the tokens g and g + 8 the codes of 8 dimensions of every block, and the scales.
template <int NB> struct Keys {
    uint32_t code[2][NB], scale[2][NB];
    __device__ void load(const uint8_t *tile, int lane) {
        using G = KvGeom<NB>;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            ldg_words<NB, G::kVec>(tile + (h * NB * 32 + lane * G::kVec) * 4, 128 * G::kVec, code[h]);
            ldg_words<NB, G::kVec>(tile + G::kKScaleAt + ((lane >> 3) + 4 * h) * NB * 4, 4 * G::kVec, scale[h]);
        }
    }
};

template <int NB> __global__ void __launch_bounds__(kWeightThreads, 2) attn_weights_kernel(WeightArgs w) {
    using G = KvGeom<NB>;
    const AttnArgs &a = w.a;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 sh_exp[kBlockCols];  // p = exp2(x * score + y)
    __shared__ int2 sh_see[kBlockCols];    // first token that a column sees, and the one after the last
    __shared__ int sh_low, sh_end;
    uint2 *q_sm = reinterpret_cast<uint2 *>(smem);                                     // [group of 4][2 NB][lane]
    float *wait_sm = reinterpret_cast<float *>(smem + kBlockCols / 4 * 2 * NB * 256);  // weights between blocks of columns
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    block_op_wait();
    block_op_release();
    const int item = w.by_chunks.div(blockIdx.x), chunk = w.by_chunks.mod(blockIdx.x, item);
    const int seq = a.by_heads.div(item), kvh = a.by_heads.mod(item, seq);
    const AttnRange r = attn_range<true>(a, seq, 0, kAllCols);
    if (r.bad) {
        if (tid == 0 && a.status) *a.status = 1;
        return;
    }
    const int tiles = (r.len + kKvSlab - 1) / kKvSlab, first = chunk * w.chunk, last = min(tiles, first + w.chunk);
    if (first >= last) return;
    const int base = r.len - r.n, columns = r.n * a.group;
    const bool tree = a.seen != nullptr;
    const float *before = w.before ? w.before + static_cast<int64_t>(item) * w.before_stride : nullptr;
    float *out = w.out + static_cast<int64_t>(item) * w.out_stride;
    const int32_t *table = a.c.table + static_cast<int64_t>(seq) * a.c.max_pages;
    const uint8_t *head = a.c.pages + static_cast<int64_t>(kvh) * static_cast<int>(a.by_page_tiles.d) * G::kTileBytes;
    const uint32_t pick = (g & 1) ? 0x7632u : 0x5410u;  // the token's half of two words of scales

    for (int col0 = 0;; col0 += kBlockCols) {
        const int cols = max(0, min(kBlockCols, columns - col0)), groups = (cols + 3) / 4;
        const bool last_block = col0 + kBlockCols >= columns;
        if (col0 > 0) __syncthreads();  // the block before is done with
        if (tid == 0) {
            sh_low = 0;
            sh_end = r.len;
        }
        __syncthreads();
        for (int grp = warp; grp < groups; grp += kWeightWarps) {
            float v[NB][8], top = 0.0f, up, down;
            const int col = col0 + 4 * grp + g / 2, i = a.by_group.div(col);
            load_q<NB>(a, r, kvh, col, t, v);
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(v[b][k]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            q_unit(top, a.scale_log2, up, down);
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t f[4];
                    split_h2(v[b][2 * h] * up, v[b][2 * h + 4] * up, f[0], f[1]);
                    split_h2(v[b][2 * h + 1] * up * 0.0625f, v[b][2 * h + 5] * up * 0.0625f, f[2], f[3]);
                    q_sm[(grp * 2 * NB + 2 * b + h) * 32 + lane] = (g & 1) ? make_uint2(f[1], f[3]) : make_uint2(f[0], f[2]);
                }
            if (t == 0 && (g & 1) == 0) {
                const int at = 4 * grp + g / 2;
                // a column that is none adds 2^-infinity
                float2 e = make_float2(0.0f, -INFINITY);
                int2 see = make_int2(0, r.len);
                if (i < r.n) {
                    const float lse = w.lse_in[static_cast<int64_t>(r.q0 + i) * a.n_q_heads + kvh * a.group + (col - i * a.group)];
                    e = make_float2(fmaxf(fabsf(a.scale_log2) * down, 1e-37f), -1.44269504088896340736f * lse);
                    if (tree) {
                        see.x = tree_low(a, r, i);
                        atomicMin(&sh_end, base);
                    } else {
                        see.y = max(0, r.len - (r.n - 1 - i));
                        see.x = a.window > 0 ? max(0, see.y - a.window) : 0;
                        atomicMin(&sh_end, see.y);
                    }
                    atomicMax(&sh_low, see.x);
                }
                sh_exp[at] = e;
                sh_see[at] = see;
            }
        }
        __syncthreads();
        const int low_max = sh_low, end_min = sh_end;

        // the warp's tiles are first + warp + 8 k; a lane looks up every 32nd one's page
        const uint8_t *src = nullptr;
        bool wrong = false;
        const auto look = [&](int k0) {
            const int tile = first + warp + kWeightWarps * (k0 + lane);
            src = nullptr;
            wrong = false;
            if (tile < last && tile >= r.slab0 && tile < r.slab0 + r.slabs && columns > 0) {
                const int slot = a.by_page_tiles.div(tile), page = table[slot];
                wrong = page < 0 || page >= a.c.n_pages;
                if (wrong && a.status) *a.status = 1;
                if (!wrong)
                    src = head + page * a.c.page_bytes + static_cast<int64_t>(a.by_page_tiles.mod(tile, slot)) * G::kTileBytes;
            }
        };
        const auto source = [&](int k) {
            return reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), k & 31));
        };
        Keys<NB> keys;
        look(0);
        const uint8_t *now = source(0);
        bool skip = __shfl_sync(0xffffffffu, wrong ? 1 : 0, 0) != 0;
        if (now) keys.load(now, lane);
        for (int k = 0, tile = first + warp; tile < last; ++k, tile += kWeightWarps) {
            const int t0 = tile * kKvSlab, tok = t0 + g + ((t & 1) ? 8 : 0);  // the token that lanes t = 0 and 1 store
            uint32_t f[NB][8];
            float dd[NB][2];
            const bool some = now != nullptr, left = skip;
            if (some) {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    uint32_t k0[4], k1[4];
                    code_pairs(keys.code[0][b], kCodeMagic, k0);
                    code_pairs(keys.code[1][b], kCodeMagic, k1);
                    f[b][0] = k0[0]; f[b][1] = k1[0]; f[b][2] = k0[1]; f[b][3] = k1[1];
                    f[b][4] = k0[2]; f[b][5] = k1[2]; f[b][6] = k0[3]; f[b][7] = k1[3];
                    const float2 d = f2_parts(f2_half2(__byte_perm(keys.scale[0][b], keys.scale[1][b], pick)));
                    dd[b][0] = d.x;
                    dd[b][1] = d.y;
                }
            }
            if (tile + kWeightWarps < last) {
                if (((k + 1) & 31) == 0) look(k + 1);
                now = source(k + 1);
                skip = __shfl_sync(0xffffffffu, wrong ? 1 : 0, (k + 1) & 31) != 0;
                if (now) keys.load(now, lane);
            }
            float s0 = 0.0f, s1 = 0.0f;  // tokens t0 + g and t0 + g + 8
            if (some) {
                const bool masked = t0 < low_max || t0 + kKvSlab > end_min;
                for (int grp = 0; grp < groups; ++grp) {
                    float x0 = 0.0f, x1 = 0.0f;
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const uint2 q0 = q_sm[(grp * 2 * NB + 2 * b) * 32 + lane], q1 = q_sm[(grp * 2 * NB + 2 * b + 1) * 32 + lane];
                        const uint32_t a0[4] = {f[b][0], f[b][1], f[b][2], f[b][3]}, a1[4] = {f[b][4], f[b][5], f[b][6], f[b][7]};
                        float c[4];
                        mma_first(c, a0, q0.x, q0.y);
                        mma_acc(c, a1, q1.x, q1.y);
                        x0 = fmaf(dd[b][0], c[0] + c[1], x0);
                        x1 = fmaf(dd[b][1], c[2] + c[3], x1);
                    }
                    const float2 e = sh_exp[4 * grp + t];
                    float p0 = exp2_approx(fmaf(x0, e.x, e.y)), p1 = exp2_approx(fmaf(x1, e.x, e.y));
                    if (masked) {
                        const int2 see = sh_see[4 * grp + t];
                        const int i = a.by_group.div(col0 + 4 * grp + t);
                        const uint32_t bits = tree && i < r.n ? tree_bits(a, r, i, t0) : ~0u;
                        if (t0 + g < see.x || t0 + g >= see.y || !(bits >> g & 1u)) p0 = 0.0f;
                        if (t0 + g + 8 < see.x || t0 + g + 8 >= see.y || !(bits >> (g + 8) & 1u)) p1 = 0.0f;
                    }
                    s0 += p0;
                    s1 += p1;
                }
                s0 += __shfl_xor_sync(0xffffffffu, s0, 1);
                s1 += __shfl_xor_sync(0xffffffffu, s1, 1);
                s0 += __shfl_xor_sync(0xffffffffu, s0, 2);
                s1 += __shfl_xor_sync(0xffffffffu, s1, 2);
            }
            if (t < 2 && tok < r.len && !left) {
                float s = t == 0 ? s0 : s1;
                float *rest = wait_sm + (tile - first) * kKvSlab + (tok - t0);
                if (col0 > 0) s += *rest;
                if (!last_block) *rest = s;
                else out[tok] = before && tok < base ? fmaf(w.keep, before[tok], s) : s;
            }
        }
        if (last_block) break;
    }
}

template <int NB> cudaError_t launch_weights(const WeightArgs &w, int64_t items, int64_t columns, cudaStream_t st) {
    const cudaError_t e = smem_limit_raised<&attn_weights_kernel<NB>>();
    if (e != cudaSuccess) return e;
    const size_t smem = static_cast<size_t>(std::min<int64_t>(kBlockCols, columns + 3) / 4) * 2 * NB * 256 +
                        (columns > kBlockCols ? static_cast<size_t>(w.chunk) * kKvSlab * 4 : 0);
    return launch_block_op(&attn_weights_kernel<NB>, dim3(static_cast<unsigned>(items * w.chunks)), dim3(kWeightThreads), smem, st, w);
}

}  // namespace
}  // namespace zdmmv

using namespace zdmmv;

extern "C" {

zdmmv_status zdmmv_attn_weights_q4_0(const zdmmv_kv_cache *cache, const zdmmv_attn_weights_args *args, zdmmv_stream_t stream) {
    if (!args) return ZDMMV_ERR_NULL;
    WeightArgs w{};
    AttnArgs &a = w.a;
    const zdmmv_status st = kv_check(cache, &a.c);
    if (st != ZDMMV_OK) return st;
    const zdmmv_attn_weights_args &g = *args;
    if (g.n_tok < 0 || g.n_q_heads < 1 || g.n_q_heads > 65535 || g.n_q_heads % cache->n_kv_heads || g.max_q_len < 1 ||
        g.max_kv_len < 0 || g.window < 0 || !std::isfinite(g.scale) || !std::isfinite(g.keep))
        return ZDMMV_ERR_SHAPE;
    if (g.seen && (g.seen_words < 1 || g.seen_words > kMostSeenWords || static_cast<int64_t>(g.seen_words) * 32 < g.max_q_len))
        return ZDMMV_ERR_SHAPE;
    const int group = g.n_q_heads / cache->n_kv_heads;
    const int64_t columns = static_cast<int64_t>(std::min(g.max_q_len, std::max(1, g.n_tok))) * group;
    const int64_t items = static_cast<int64_t>(a.c.n_seq) * a.c.n_kv_heads;
    const int64_t tiles = (static_cast<int64_t>(std::min(g.max_kv_len, kMostAttnTokens)) + kKvSlab - 1) / kKvSlab;
    if (columns > kAllCols || items > 0x7fffff00) return ZDMMV_ERR_SHAPE;
    if (g.max_kv_len == 0) return ZDMMV_OK;
    if (!g.q_start || !g.kv_len || !g.out || (g.n_tok > 0 && (!g.q || !g.lse))) return ZDMMV_ERR_NULL;
    if ((g.n_tok > 0 && g.q_stride < static_cast<int64_t>(g.n_q_heads) * cache->head_dim) || g.out_stride < g.max_kv_len ||
        (g.before && g.before_stride < g.max_kv_len) || (g.before == g.out && g.before_stride != g.out_stride))
        return ZDMMV_ERR_SHAPE;
    if (kv_misaligned(g.q, 16) || g.q_stride % 4 || kv_misaligned(g.q_start, 4) || kv_misaligned(g.kv_len, 4) || kv_misaligned(g.lse, 4) ||
        kv_misaligned(g.seen, 4) || kv_misaligned(g.before, 4) || kv_misaligned(g.out, 4) || kv_misaligned(g.status_dev, 4))
        return ZDMMV_ERR_ALIGN;
    a.q = g.q; a.q_start = g.q_start; a.kv_len = g.kv_len; a.status = g.status_dev;
    a.q_stride = g.q_stride;
    a.n_tok = g.n_tok; a.n_q_heads = g.n_q_heads; a.group = group;
    a.max_q_len = g.max_q_len; a.max_kv_len = std::min(g.max_kv_len, kMostAttnTokens);
    a.window = attn_window(g.window, g.max_kv_len);
    a.scale_log2 = g.scale * 1.44269504088896340736f;
    a.by_heads = FastDiv::of(cache->n_kv_heads);
    a.by_group = FastDiv::of(group);
    a.by_page_tiles = FastDiv::of(cache->page_tokens / kKvSlab);
    a.seen = g.seen; a.seen_words = g.seen_words;
    w.lse_in = g.lse; w.before = g.before; w.out = g.out;
    w.before_stride = g.before_stride; w.out_stride = g.out_stride; w.keep = g.keep;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return ZDMMV_ERR_CUDA;
    // as many CTAs as run at once, or four times that for several sequences, whose lengths may differ
    const int64_t want = static_cast<int64_t>(sms) * 2 * (a.c.n_seq > 1 ? 4 : 1);
    int64_t chunk = std::max<int64_t>(kWeightWarps, (items * tiles + want - 1) / want);
    chunk = (chunk + kWeightWarps - 1) / kWeightWarps * kWeightWarps;
    if (columns > kBlockCols) chunk = std::min<int64_t>(chunk, kMostChunk);
    const int64_t chunks = (tiles + chunk - 1) / chunk;
    if (items * chunks > 0x7fffff00) return ZDMMV_ERR_SHAPE;
    w.chunk = static_cast<int32_t>(chunk);
    w.chunks = static_cast<int32_t>(chunks);
    w.by_chunks = FastDiv::of(w.chunks);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
    switch (kv_blocks(cache->head_dim)) {
    case 2: e = launch_weights<2>(w, items, columns, s); break;
    case 3: e = launch_weights<3>(w, items, columns, s); break;
    case 4: e = launch_weights<4>(w, items, columns, s); break;
    case 6: e = launch_weights<6>(w, items, columns, s); break;
    case 8: e = launch_weights<8>(w, items, columns, s); break;
    }
    return e == cudaSuccess ? ZDMMV_OK : ZDMMV_ERR_CUDA;
}

}  // extern "C"
