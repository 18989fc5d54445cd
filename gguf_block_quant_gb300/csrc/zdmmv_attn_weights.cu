// zdmmv_attn_weights.cu -- zdmmv_attn_weights_q4_0: what the query rows of a call give each cached token,
//
//   out_t = keep before_t + sum_c exp(min(0, scale (q_c . k_t) - lse_c))      over the columns c (query rows of the kv head) that see t,
//
// from the keys alone: half of the cache's bytes, and no product with V. A token belongs to one warp (or thread), which goes over
// all columns in a fixed order: nothing is joined, no atomics on sums.
//
// Few columns (decoding, small trees): attn_weights_kernel, on mma.sync. Many (prompts, drafted tokens of grouped heads):
// attn_weights_tall_kernel, on tcgen05.
#include <algorithm>
#include <cmath>

#include "zdmmv_attn_prompt.cuh"
#include "zdmmv_internal.h"

namespace zdmmv {
namespace {

constexpr int kWeightWarps = 8, kWeightThreads = kWeightWarps * 32;
constexpr int kBlockCols = 64;       // columns of a block of q, and most of the kernel for few
constexpr int kAllCols = 0x7fffff00; // a column tile of all columns

struct WeightArgs {
    AttnArgs a;            // out, the workspace's and the split's fields unused
    FastDiv by_items;      // kv heads of sequences
    const float *lse_in, *before;
    float *out;
    int64_t before_stride, out_stride;  // between kv heads
    uint8_t *images;                    // the tall kernel's blocks of q
    FastDiv by_blocks;                  // ... of an item, at most
    int32_t chunks;                     // the tall kernel's CTAs of an item
    float keep;
};

// How a column's product with a key becomes its weight, p = exp2(min(0, x * product + y)), and which tokens it sees. The minimum
// changes roundings alone while |lse| is small: a row's lse is no less than any of its scores. A large lse's own step is a part
// of the exponent that counts (2^-24 of |lse|, four times over with the products by ln 2 and its inverse), and a score is off by up
// to 2^-19 of its products' magnitudes, here and in the kernel that made lse. From 2^20 on y is therefore raised by 2^-17 of what
// |y| has beyond that, from 2^21 on more than all of it together where the largest score's products hardly cancel (where they do, the
// bound is far from what happens): a token that has all of a row's weight then gets it, whichever way its score was rounded.
struct Column {
    float x, y;
    int low, end;
};
__device__ __forceinline__ Column column_of(const WeightArgs &w, const AttnRange &r, int kvh, int col, float lse, float down) {
    const AttnArgs &a = w.a;
    const int i = a.by_group.div(col);
    // one that is none adds 2^-infinity, and where tokens are masked at all it sees none: a key may be no number. (A product of
    // -infinity is one here too.)
    if (i >= r.n) return {1e-37f, -INFINITY, 0, 0};
    Column c;
    c.x = fmaxf(fabsf(a.scale_log2) * down, 1e-37f);
    c.y = -1.44269504088896340736f * lse;
    c.y += fminf(fmaxf(0.0f, (fabsf(c.y) - 1048576.0f) * 0x1p-17f), 1e34f);  // what is no number or infinite stays so
    if (a.seen) {
        c.low = tree_low(a, r, i);
        c.end = r.len;
    } else {
        c.end = max(0, r.len - (r.n - 1 - i));
        c.low = a.window > 0 ? max(0, c.end - a.window) : 0;
    }
    return c;
}
__device__ __forceinline__ float weight_of(float e) {  // a key that is no number has a weight that is none
    float x;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(e), "f"(0.0f));
    return exp2_approx(x);
}
__device__ __forceinline__ const float *column_lse(const WeightArgs &w, const AttnRange &r, int kvh, int col) {
    const int i = w.a.by_group.div(col);
    return w.lse_in + static_cast<int64_t>(r.q0 + i) * w.a.n_q_heads + kvh * w.a.group + (col - i * w.a.group);
}
// The cache tiles low .. end-1 of a sequence whose tokens' sums a call has to write: all, or, where sums stay in place and
// unscaled, those that a row sees.
__device__ __forceinline__ void tiles_of(const WeightArgs &w, const AttnRange &r, int &low, int &end) {
    low = 0;
    end = r.bad ? 0 : (r.len + kKvSlab - 1) / kKvSlab;
    if (w.keep == 1.0f && w.before == w.out) low = min(r.slab0, end);
}

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

__device__ __forceinline__ void cp_async_16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void cp_async_4(uint32_t to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// ------------------------------------------------------------------ few columns
// The scores are formed as in the narrow kernel of zdmmv_attn.cuh (A = a tile's 16 tokens of codes, B = four columns' upper and
// lower parts; a product's C holds a column's two sums side by side), so that they agree with those that lse was made of. The
// steps (16 tiles, a pair for each warp) of all kv heads of all sequences one after another are a row, of which every CTA of a
// grid that fills the device (two an SM; heads past 128 dimensions mostly have room for one, and the stretches then run in two rounds) takes
// an equal stretch, whatever the lengths. A warp keeps the next pairs' keys, and their tokens'
// earlier sums, on their way into its own ring in shared memory; a pair's 32 sums end up one in each lane.
// ONE: up to four columns, whose parts of q stay in registers.
// One token of 32 heads over 130975 tokens of 8 kv heads of 128: 20.0 us, 4.2 TB/s, 63% of the copy rate; 48 sequences of up to
// 16384 45.6 us, 3.8 TB/s. Four warps a scheduler keep 57% of the issue slots busy (207 instructions a tile, 72 of them the codes'
// conversion, two the weight's bound), and the start, lengths, pages, the first keys and q, is four latencies one after another, of some 4 us;
// of several sequences each kv head is such a start, as the rings run empty there. Over 131072 tokens of heads of 256 41.5 us,
// one CTA an SM. Measured, over 130975, against 19.7 before the bound: loads a tile
// ahead into registers, the earlier sums read where they are used, 33.2; rings of four single tiles 28.8; three CTAs an SM, with
// 80 registers a thread, 21.6; four places a ring 19.8 (and 45.2), five 20.1; q asked for before the pages, which it costs spills, 32.6.
constexpr int kWeightStages = 3;
template <int NB> constexpr int kPairBytes = 2 * 9 * NB * kQK + 2 * kKvSlab * 4;
template <int NB> constexpr size_t kWeightRing = static_cast<size_t>(kWeightWarps) * kWeightStages * kPairBytes<NB>;
constexpr int kWeightCtas = 2;  // an SM

template <int NB, bool ONE> __global__ void __launch_bounds__(kWeightThreads, kWeightCtas) attn_weights_kernel(WeightArgs w) {
    using G = KvGeom<NB>;
    const AttnArgs &a = w.a;
    constexpr int kKeyBytes = 9 * G::kDim;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Column sh_col[kBlockCols];
    __shared__ int sh_low, sh_end, sh_scan[kWeightWarps], sh_seq, sh_from;
    __shared__ uint32_t sh_magic;
    uint2 *q_sm = reinterpret_cast<uint2 *>(smem + kWeightRing<NB>);  // [group of 4][2 NB][lane]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_addr(smem) + warp * (kWeightStages * kPairBytes<NB>);
    if (tid == 0) sh_magic = kCodeMagic;
    block_op_wait();
    block_op_release();
    const int heads = a.c.n_kv_heads, n_seq = a.c.n_seq;
    const auto steps_of = [&](int seq) {
        const AttnRange r = attn_range<true>(a, seq, 0, kAllCols);
        int low, end;
        tiles_of(w, r, low, end);
        if (r.bad && blockIdx.x == 0 && a.status) *a.status = 1;
        return (end - low + kStepTiles - 1) / kStepTiles;
    };
    // this CTA's stretch of the row, and the sequence that it begins in
    int64_t at, last;
    {
        int64_t total = 0;
        int kept = 0;
        for (int s0 = 0; s0 < n_seq; s0 += kWeightThreads) {
            const int n = s0 + tid < n_seq ? steps_of(s0 + tid) * heads : 0;
            if (s0 == 0) kept = n;
            int all;
            (void)AttnWalk::upto(n, sh_scan, all);
            total += all;
            __syncthreads();
        }
        const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total);
        if (blockIdx.x >= ctas) return;
        at = total * blockIdx.x / ctas;
        last = total * (blockIdx.x + 1) / ctas;
        for (int64_t s0 = 0, before = 0;; s0 += kWeightThreads) {
            const int seq = static_cast<int>(s0) + tid, n = s0 == 0 ? kept : (seq < n_seq ? steps_of(seq) * heads : 0);
            int all;
            const int64_t from = before + AttnWalk::upto(n, sh_scan, all) - n;
            if (n > 0 && at >= from && at < from + n) {
                sh_seq = seq;
                sh_from = static_cast<int>(at - from);
            }
            before += all;
            __syncthreads();
            if (at < before) break;
        }
    }
    int seq = sh_seq, inside = sh_from;  // the step of the sequence's steps
    const uint32_t magic = lds32(smem_addr(&sh_magic));
    const uint32_t pick = (g & 1) ? 0x7632u : 0x5410u;  // the token's half of two words of scales

    while (true) {
        const AttnRange r = attn_range<true>(a, seq, 0, kAllCols);
        int low, end;
        tiles_of(w, r, low, end);
        const int steps = (end - low + kStepTiles - 1) / kStepTiles;
        if (inside >= steps * heads) {  // the next sequence, as long as the stretch has steps of one
            ++seq;
            inside = 0;
            continue;
        }
        const int kvh = inside / steps, step = inside - kvh * steps;
        const int n_steps = static_cast<int>(min(static_cast<int64_t>(steps - step), last - at));
        const int first = low + step * kStepTiles, stop = min(end, first + n_steps * kStepTiles);
        const int base = r.len - r.n, columns = r.n * a.group, groups = (columns + 3) / 4;
        const int seen0 = r.slab0, seen1 = columns > 0 ? r.slab0 + r.slabs : 0;  // tiles that a column sees
        const bool tree = a.seen != nullptr;
        const int64_t item = static_cast<int64_t>(seq) * heads + kvh;
        const float *before = w.before ? w.before + item * w.before_stride : nullptr;
        float *out = w.out + item * w.out_stride;
        const int32_t *table = a.c.table + static_cast<int64_t>(seq) * a.c.max_pages;
        const uint8_t *head = a.c.pages + static_cast<int64_t>(kvh) * static_cast<int>(a.by_page_tiles.d) * G::kTileBytes;

        // the warp's pairs are tiles first + 2 (warp + 8 k); lanes 2 j and 2 j + 1 look up every 16th one's pages
        const uint8_t *src = nullptr;
        uint32_t bad_now = 0, bad_next = 0;  // bad pages of 16 pairs, those in use and those asked for
        const auto ask = [&](int k) {
            const int tile = first + 2 * (warp + kWeightWarps * k);
            if (tile < stop) {
                if ((k & 15) == 0) {
                    const int mine = tile + 2 * kWeightWarps * (lane >> 1) + (lane & 1);
                    src = nullptr;
                    bool wrong = false;
                    if (mine < stop && mine >= seen0 && mine < seen1) {
                        const int slot = a.by_page_tiles.div(mine), page = table[slot];
                        wrong = page < 0 || page >= a.c.n_pages;
                        if (wrong && a.status) *a.status = 1;
                        if (!wrong)
                            src = head + page * a.c.page_bytes + static_cast<int64_t>(a.by_page_tiles.mod(mine, slot)) * G::kTileBytes;
                    }
                    bad_next = __ballot_sync(0xffffffffu, wrong);
                }
                const int s = lane >> 4, l = lane & 15;  // half a warp for a tile
                const uint8_t *from = reinterpret_cast<const uint8_t *>(
                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), 2 * (k & 15) + s));
                const uint32_t stage = ring + (k % kWeightStages) * kPairBytes<NB>, to = stage + s * kKeyBytes + 16 * l;
                if (from) {
#pragma unroll
                    for (int c = 0; c < NB; ++c) cp_async_16(to + 256 * c, from + 16 * l + 256 * c);
                    if (l < 2 * NB) cp_async_16(to + G::kCodeBytes, from + 16 * l + G::kKScaleAt);
                }
                const int tok = tile * kKvSlab + lane;
                if (before && tok < base) cp_async_4(stage + 2 * kKeyBytes + 4 * lane, before + tok);
            }
            cp_async_commit();
        };
#pragma unroll
        for (int k = 0; k < kWeightStages - 1; ++k) ask(k);

        __syncthreads();  // the segment before is done with q and its columns
        if (tid == 0) {
            sh_low = 0;
            sh_end = tree ? base : r.len;
        }
        __syncthreads();
        for (int grp = warp; grp < groups; grp += kWeightWarps) {
            float v[NB][8], top = 0.0f, up, down;
            const int col = 4 * grp + g / 2;
            const bool lead = t == 0 && (g & 1) == 0;
            const float lse = lead && col < columns ? *column_lse(w, r, kvh, col) : 0.0f;
            // a column that is none has another's q: its products with an infinite key are no NaN where that one's are none
            load_q<NB>(a, r, kvh, col < columns ? col : 4 * grp, t, v);
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
            if (lead) {
                const Column c = column_of(w, r, kvh, col, lse, down);
                if (col < columns) {
                    atomicMin(&sh_end, c.end);
                    atomicMax(&sh_low, c.low);
                }
                sh_col[col] = c;
            }
        }
        __syncthreads();
        const int low_max = sh_low, end_min = sh_end;
        uint2 qf[ONE ? 2 * NB : 1];
        Column mine{0.0f, -INFINITY, 0, 0};
        if constexpr (ONE) {
            if (groups > 0) mine = sh_col[t];
#pragma unroll
            for (int k = 0; k < 2 * NB; ++k) qf[k] = groups > 0 ? q_sm[k * 32 + lane] : make_uint2(0, 0);
        }

        for (int k = 0, tile = first + 2 * warp; tile < stop; ++k, tile += kStepTiles) {
            cp_async_wait<kWeightStages - 2>();
            __syncwarp();  // all lanes' copies of pair k are there, and all are done with the place before
            ask(k + kWeightStages - 1);
            if ((k & 15) == 0) bad_now = bad_next;
            const uint32_t stage = ring + (k % kWeightStages) * kPairBytes<NB>;
            const int t0 = tile * kKvSlab;
            float p[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};  // by tile: tokens g and g + 8
            if (tile + 1 >= seen0 && tile < seen1) {
                const bool masked = t0 < low_max || t0 + 2 * kKvSlab > end_min;
                // ... of one column of a group of four
                const auto weigh = [&](int s, int grp, const Column &c, float x0, float x1) {
                    float p0 = weight_of(fmaf(x0, c.x, c.y)), p1 = weight_of(fmaf(x1, c.x, c.y));
                    if (masked) {
                        const int i = a.by_group.div(4 * grp + t), tok = t0 + kKvSlab * s + g;
                        const uint32_t bits = tree && i < r.n ? tree_bits(a, r, i, t0 + kKvSlab * s) : ~0u;
                        if (tok < c.low || tok >= c.end || !(bits >> g & 1u)) p0 = 0.0f;
                        if (tok + 8 < c.low || tok + 8 >= c.end || !(bits >> (g + 8) & 1u)) p1 = 0.0f;
                    }
                    p[s][0] += p0;
                    p[s][1] += p1;
                };
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const uint32_t keys = stage + s * kKeyBytes;
                    uint32_t kw[2][NB], dk[2][NB];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        lds_words<NB, G::kVec>(keys + (h * NB * 32 + lane * G::kVec) * 4, 128 * G::kVec, kw[h]);
                        lds_words<NB, G::kVec>(keys + G::kCodeBytes + ((lane >> 3) + 4 * h) * NB * 4, 4 * G::kVec, dk[h]);
                    }
                    uint32_t f[ONE ? 1 : NB][8];
                    float2 dd[ONE ? 1 : NB];
                    const auto block = [&](int b, uint32_t (&x)[8], float2 &d) {
                        uint32_t k0[4], k1[4];
                        code_pairs(kw[0][b], magic, k0);
                        code_pairs(kw[1][b], magic, k1);
                        x[0] = k0[0]; x[1] = k1[0]; x[2] = k0[1]; x[3] = k1[1];
                        x[4] = k0[2]; x[5] = k1[2]; x[6] = k0[3]; x[7] = k1[3];
                        d = f2_parts(f2_half2(__byte_perm(dk[0][b], dk[1][b], pick)));
                    };
                    const auto score = [&](const uint32_t (&x)[8], float2 d, uint2 q0, uint2 q1, float &x0, float &x1) {
                        const uint32_t a0[4] = {x[0], x[1], x[2], x[3]}, a1[4] = {x[4], x[5], x[6], x[7]};
                        float c[4];
                        mma_first(c, a0, q0.x, q0.y);
                        mma_acc(c, a1, q1.x, q1.y);
                        x0 = fmaf(d.x, c[0] + c[1], x0);
                        x1 = fmaf(d.y, c[2] + c[3], x1);
                    };
                    if constexpr (ONE) {
                        float x0 = 0.0f, x1 = 0.0f;
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            block(b, f[0], dd[0]);
                            score(f[0], dd[0], qf[2 * b], qf[2 * b + 1], x0, x1);
                        }
                        weigh(s, 0, mine, x0, x1);
                    } else {
#pragma unroll
                        for (int b = 0; b < NB; ++b) block(b, f[b], dd[b]);
                        for (int grp = 0; grp < groups; ++grp) {
                            float x0 = 0.0f, x1 = 0.0f;
#pragma unroll
                            for (int b = 0; b < NB; ++b)
                                score(f[b], dd[b], q_sm[(grp * 2 * NB + 2 * b) * 32 + lane], q_sm[(grp * 2 * NB + 2 * b + 1) * 32 + lane], x0, x1);
                            weigh(s, grp, sh_col[4 * grp + t], x0, x1);
                        }
                    }
                }
            }
            // over the four columns' lanes: lane t has tile t / 2, tokens g and g + 8 by t % 2
            const bool upper = t & 2, odd = t & 1;
            const float r0 = (upper ? p[1][0] : p[0][0]) + __shfl_xor_sync(0xffffffffu, upper ? p[0][0] : p[1][0], 2);
            const float r1 = (upper ? p[1][1] : p[0][1]) + __shfl_xor_sync(0xffffffffu, upper ? p[0][1] : p[1][1], 2);
            const float sum = (odd ? r1 : r0) + __shfl_xor_sync(0xffffffffu, odd ? r0 : r1, 1);
            const int own = (upper ? kKvSlab : 0) + (odd ? 8 : 0) + g, tok = t0 + own;
            if (tok < r.len && !(bad_now >> (2 * (k & 15) + (upper ? 1 : 0)) & 1u))
                out[tok] = before && tok < base ? fmaf(w.keep, __uint_as_float(lds32(stage + 2 * kKeyBytes + 4 * own)), sum) : sum;
        }
        cp_async_wait<0>();
        at += n_steps;
        inside += n_steps;
        if (at >= last) break;
    }
}

// ------------------------------------------------------------------ more columns
// S = K Q^T on tcgen05: a CTA takes 128 tokens of a kv head, the 128 rows of D, and goes over all columns, 64 at a time, so that
// a thread has one token's products with 32 columns in registers and adds their weights up by itself.
//  * K is the A operand, in tensor memory for the CTA's life, Q the B operand, in shared memory (rows of 128 bytes swizzled by
//    128 bytes), each in two fp16 parts (k exactly, q to 22 bits; zdmmv_attn_prompt.cuh): 3 D/16 products a block.
//  * Every CTA of a kv head needs all of its q: weights_q_kernel makes the operands (and what each column needs to become a
//    weight) once, in the workspace, as they lie in shared memory, and the CTAs bring them with one bulk copy a block, two
//    blocks ahead. (Each CTA turning q into operands by itself: 141 us where this took 46, 700 of 1000 instructions a block.)
//  * One lane starts a block's products while all threads take the weights of the block before; D is double. Two CTAs an SM
//    (heads of up to 128 dimensions) fill each other's gaps.
// Where a token has a scale of 2^13 or more, the 128 tokens' operand is in units of 16, as there.
// 256 tokens of 32 heads over 8192 of 8 kv heads of 128 (1024 columns, 512 CTAs): 49.1 us, the tensor cores 44% busy, of which
// weights_q_kernel and the start take 6 (4 with lengths, pages and keys loaded before the wait for that kernel, where nothing says that
// what the kernels before it wrote can be seen), the weights' bound 1. A block's 24 products are 816 cycles; two CTAs' blocks take 2200
// and more, as the next block's products wait for the weights of the one before (D is double, not triple), and 512 CTAs are 1.7 rounds of
// 304 places. On mma.sync 199 us.
constexpr int kTallTokens = 128, kTallSlots = 3;
template <int NB> struct TallGeom {
    static constexpr int kDim = NB * kQK, kChunks = (NB + 1) / 2;  // of 64 dimensions
    static constexpr uint32_t kKChunk = kTallTokens * 128, kQChunk = kBlockCols * 128;
    static constexpr uint32_t kKPart = kChunks * kKChunk, kQPart = kChunks * kQChunk;
    // a block of q in the workspace: the operand's parts, the columns' (x, y) by two, what they see, and of it the latest first
    // token, the earliest end, the earliest first token and the latest end
    static constexpr uint32_t kExpAt = 2 * kQPart, kSeeAt = kExpAt + kBlockCols * 8, kBothAt = kSeeAt + kBlockCols * 8;
    static constexpr uint32_t kImage = kBothAt + 16, kSlot = (kImage + 1023) / 1024 * 1024;
    static constexpr size_t kSmem = kTallSlots * kSlot + 1024;  // aligned to 1024; before the blocks of q, K
    static_assert(2 * kKPart <= kTallSlots * kSlot, "K's rows");
    static constexpr int kCtas = NB <= 4 ? 2 : 1;
    static constexpr uint32_t kTm = NB <= 4 ? 256 : 512, kTmD = kDim;  // K's columns, then twice 64 of D
    static_assert(kTmD + 2 * kBlockCols <= kTm, "tensor memory");
};
// Blocks of a call's q: sequence s's first is number q0 group / 64 + s, which leaves room for all of those before it.
__device__ __forceinline__ int64_t first_block(const WeightArgs &w, const AttnRange &r, int seq) {
    return static_cast<int64_t>(r.q0) * w.a.group / kBlockCols + seq;
}
int64_t weight_blocks(int n_seq, int n_tok, int group) { return static_cast<int64_t>(n_tok) * group / kBlockCols + n_seq; }
template <int NB> __device__ __forceinline__ uint8_t *block_image(const WeightArgs &w, int64_t block, int kvh) {
    return w.images + (block * w.a.c.n_kv_heads + kvh) * TallGeom<NB>::kImage;
}

// A CTA makes a block: whole rows by a warp, four dimensions a lane of each 128.
template <int NB> __global__ void __launch_bounds__(kWeightThreads) weights_q_kernel(WeightArgs w) {
    using T = TallGeom<NB>;
    constexpr int D = T::kDim, kPasses = (D + 127) / 128, kPerWarp = kBlockCols / kWeightWarps;
    const AttnArgs &a = w.a;
    __shared__ int4 sh_both;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    block_op_wait();
    block_op_release();
    const int item = w.by_blocks.div(blockIdx.x), block = w.by_blocks.mod(blockIdx.x, item);
    const int seq = a.by_heads.div(item), kvh = a.by_heads.mod(item, seq);
    const AttnRange r = attn_range<true>(a, seq, 0, kAllCols);
    const int columns = r.n * a.group, col0 = block * kBlockCols + warp * kPerWarp;
    if (r.bad || block * kBlockCols >= columns) return;
    float4 x[kPerWarp][kPasses];
#pragma unroll
    for (int j = 0; j < kPerWarp; ++j) {
        const int col = col0 + j, i = a.by_group.div(col);
        const float *q = a.q + static_cast<int64_t>(r.q0 + (i < r.n ? i : 0)) * a.q_stride +
                         static_cast<int64_t>(kvh * a.group + (i < r.n ? col - i * a.group : 0)) * D + 4 * lane;
#pragma unroll
        for (int p = 0; p < kPasses; ++p)
            x[j][p] = i < r.n && 128 * p + 4 * lane < D ? __ldg(reinterpret_cast<const float4 *>(q + 128 * p)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float lse = lane < kPerWarp && col0 + lane < columns ? __ldg(column_lse(w, r, kvh, col0 + lane)) : 0.0f;
    if (tid == 0) {
        sh_both = make_int4(0, a.seen ? r.len - r.n : r.len, r.len, 0);
    }
    __syncthreads();
    uint8_t *image = block_image<NB>(w, first_block(w, r, seq) + block, kvh);
    float up[kPerWarp], mine = 0.0f;
#pragma unroll
    for (int j = 0; j < kPerWarp; ++j) {
        float top = 0.0f, down;
#pragma unroll
        for (int p = 0; p < kPasses; ++p)
            top = fmaxf(fmaxf(fmaxf(top, fabsf(x[j][p].x)), fmaxf(fabsf(x[j][p].y), fabsf(x[j][p].z))), fabsf(x[j][p].w));
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        q_unit(top, a.scale_log2, up[j], down);
        if (lane == j) mine = down;
    }
    if (lane < kPerWarp) {
        const int at = warp * kPerWarp + lane;
        const Column c = column_of(w, r, kvh, col0 + lane, lse, mine);
        float *e = reinterpret_cast<float *>(image + T::kExpAt) + 4 * (at / 2) + (at & 1);  // two columns' x, then their y
        e[0] = c.x;
        e[2] = c.y;
        reinterpret_cast<int2 *>(image + T::kSeeAt)[at] = make_int2(c.low, c.end);
        if (col0 + lane < columns) {
            atomicMax(&sh_both.x, c.low);
            atomicMin(&sh_both.y, c.end);
            atomicMin(&sh_both.z, c.low);
            atomicMax(&sh_both.w, c.end);
        }
    }
#pragma unroll
    for (int j = 0; j < kPerWarp; ++j) {
        const int to = warp * kPerWarp + j;  // the operand's row
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            const float4 v = x[j][p];
            const bool odd = lane & 1;
            const float o0 = __shfl_xor_sync(0xffffffffu, odd ? v.x : v.z, 1), o1 = __shfl_xor_sync(0xffffffffu, odd ? v.y : v.w, 1);
            uint2 hi, lo;  // dimensions 0 4 1 5, or 2 6 3 7, of 8
            split_h2((odd ? o0 : v.x) * up[j], (odd ? v.z : o0) * up[j], hi.x, lo.x);
            split_h2((odd ? o1 : v.y) * up[j], (odd ? v.w : o1) * up[j], hi.y, lo.y);
            if (128 * p + 4 * lane < D) {
                const int t8 = 16 * p + (lane >> 1);
                uint8_t *at = image + (t8 >> 3) * T::kQChunk + to * 128 + (((t8 & 7) ^ (to & 7)) << 4) + (lane & 1) * 8;
                *reinterpret_cast<uint2 *>(at) = hi;
                *reinterpret_cast<uint2 *>(at + T::kQPart) = lo;
            }
        }
    }
    __syncthreads();
    if (tid == 0) *reinterpret_cast<int4 *>(image + T::kBothAt) = sh_both;
}

template <int NB> __global__ void __launch_bounds__(kWeightThreads, TallGeom<NB>::kCtas) attn_weights_tall_kernel(WeightArgs w) {
    using G = KvGeom<NB>;
    using T = TallGeom<NB>;
    constexpr int D = G::kDim;
    const AttnArgs &a = w.a;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int sh_skip[kWeightWarps], sh_dead;
    __shared__ float sh_sum[kTallTokens];
    __shared__ __align__(8) uint64_t bar[kTallSlots + 3];  // by slot: its block of q has come; by block % 2: its products are done; all are
    __shared__ uint32_t sh_tm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, half = warp >> 2;
    block_op_wait();  // before any load: what an early start may look at of the kernels before weights_q_kernel is said nowhere
    block_op_release();
    // the last tokens of the sequences, whose columns are masked, first
    const int back = w.by_items.div(blockIdx.x), item = w.by_items.mod(blockIdx.x, back), chunk = w.chunks - 1 - back;
    const int seq = a.by_heads.div(item), kvh = a.by_heads.mod(item, seq);
    const AttnRange r = attn_range<true>(a, seq, 0, kAllCols);
    const int first = chunk * kTallTokens, live = r.bad ? 0 : r.len - first;  // tokens from `live` on are none
    if (r.bad && tid == 0 && a.status) *a.status = 1;
    if (live <= 0) return;
    const int base = r.len - r.n, columns = r.n * a.group, blocks = (columns + kBlockCols - 1) / kBlockCols;
    const bool tree = a.seen != nullptr;
    const int row = (warp & 3) * 32 + lane, tok = first + row;  // this thread's token, with half of a block's columns
    float *out = w.out + static_cast<int64_t>(item) * w.out_stride + tok;
    const bool had = w.before != nullptr && tok < base && half == 0;
    const float earlier = had ? w.before[static_cast<int64_t>(item) * w.before_stride + tok] : 0.0f;
    constexpr int kSlabs = kTallTokens / kKvSlab;
    if (columns == 0 || chunk * kSlabs >= r.slab0 + r.slabs || (chunk + 1) * kSlabs <= r.slab0) {  // nobody sees them
        if (half == 0 && row < live) *out = had ? w.keep * earlier : 0.0f;
        return;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh_tm)), "n"(T::kTm) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 0) {
        for (int k = 0; k < kTallSlots + 3; ++k) mbar_init(&bar[k], 1);
        fence_barrier_init();
        sh_dead = 0;
    }
    const uint32_t slots = (smem_addr(smem) + 1023u) & ~1023u;
    uint8_t *slot_mem = smem + (slots - smem_addr(smem));

    // K: a cache tile a warp, as rows in shared memory, whence each thread puts half of its token's row into tensor memory
    float unit;
    {
        const int slab = chunk * kSlabs + warp;
        const uint8_t *src = nullptr;
        bool wrong = false;
        if (slab >= r.slab0 && slab < r.slab0 + r.slabs) {  // of the others, which every column masks, the pages may be gone
            const int slot = a.by_page_tiles.div(slab), page = a.c.table[static_cast<int64_t>(seq) * a.c.max_pages + slot];
            if (page >= 0 && page < a.c.n_pages)
                src = a.c.pages + page * a.c.page_bytes +
                      (static_cast<int64_t>(kvh) * static_cast<int>(a.by_page_tiles.d) + a.by_page_tiles.mod(slab, slot)) * G::kTileBytes;
            else wrong = true;
        }
        if (lane == 0) {
            sh_skip[warp] = wrong;
            if (wrong && a.status) *a.status = 1;
        }
        uint32_t code[2][NB], scale[2][NB], any = 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int b = 0; b < NB; ++b) code[u][b] = scale[u][b] = 0;
            if (src) {
                ldg_words<NB, G::kVec>(src + (u * NB * 32 + lane * G::kVec) * 4, 128 * G::kVec, code[u]);
                ldg_words<NB, G::kVec>(src + G::kKScaleAt + ((lane >> 3) + 4 * u) * NB * 4, 4 * G::kVec, scale[u]);
            }
            const int tok0 = 16 * warp + 8 * u + 2 * (lane >> 3);
            const uint32_t alive = (tok0 < live ? 0x4000u : 0u) | (tok0 + 1 < live ? 0x40000000u : 0u);
#pragma unroll
            for (int b = 0; b < NB; ++b) any |= scale[u][b] & scale[u][b] << 1 & scale[u][b] << 2 & alive;
        }
        const bool units = __syncthreads_or(any != 0);
        unit = units ? 16.0f : 1.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int mine = 16 * warp + 8 * u + (lane >> 2);
            const uint32_t pick = mine >= live ? 0x4444u : ((lane & 4) ? 0x3232u : 0x1010u);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                scale[u][b] = __byte_perm(scale[u][b], 0, pick);
                if (units) scale[u][b] = h2_mul(scale[u][b], 0x2C002C00u);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                // odd rows begin with the other block of a chunk, so that 8 lanes' stores meet 8 different banks
                const int o = (b ^ 1) < NB ? b ^ 1 : b;
                const bool other = o != b && (mine & 1);
                const int c = (((b & 1) ^ (other ? 1 : 0)) * 4 + (lane & 3)) ^ (mine & 7);
                PromptFeed<NB>::put(other ? code[u][o] : code[u][b], other ? scale[u][o] : scale[u][b], kCodeMagic,
                                    slots + (b >> 1) * T::kKChunk + mine * 128 + c * 16);
            }
        }
    }
    tm_before_sync();
    __syncthreads();
    tm_after_sync();
    const uint32_t tm = sh_tm, rows = tm + (static_cast<uint32_t>(warp & 3) << 21);  // the warp's 32 rows
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        const int e = half * (D / 16) + k;  // 8 dimensions
        const uint32_t from = slots + (e >> 3) * T::kKChunk + row * 128 + (((e & 7) ^ (row & 7)) << 4);
        const uint4 hi = lds128(from), lo = lds128(from + T::kKPart);
        tm_store4(rows + 16 * (e >> 1) + 4 * (e & 1), hi.x, hi.y, hi.z, hi.w);
        tm_store4(rows + 16 * (e >> 1) + 8 + 4 * (e & 1), lo.x, lo.y, lo.z, lo.w);
    }
    tm_stored();
    tm_before_sync();
    fence_proxy_async_smem();
    __syncthreads();
    tm_after_sync();

    const int64_t block0 = first_block(w, r, seq);
    const uint64_t policy = l2_evict_last_policy();
    const auto ask = [&](int block) {
        const int s = block % kTallSlots;
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(&bar[s], T::kImage);
        bulk_copy_g2s(slot_mem + s * T::kSlot, block_image<NB>(w, block0 + block, kvh), T::kImage, &bar[s], policy);
    };
    bool dead = false;  // a wait gave up: no more waits, but every barrier of threads is met; the result is NaN
    int asked = 0;      // tid 0: blocks that were asked for
    const auto wait = [&](int which, int parity) {
        if (!dead && !mbar_wait(&bar[which], parity)) {
            atomicOr(a.fault, 1u);
            dead = true;
        }
        __syncwarp();
    };
    uint64_t total2 = 0;
    const auto weigh = [&](int block) {
        const uint8_t *image = slot_mem + block % kTallSlots * T::kSlot;
        const float4 *exps = reinterpret_cast<const float4 *>(image + T::kExpAt) + half * (kBlockCols / 4);
        const int4 both = *reinterpret_cast<const int4 *>(image + T::kBothAt);
        if (first >= both.w || first + kTallTokens <= both.z) return;  // no column sees a token of the CTA's
        uint32_t s[2][16];
        const uint32_t at = rows + T::kTmD + (block & 1) * kBlockCols + half * (kBlockCols / 2);
        tm_load(at, s[0]);
        tm_load(at + 16, s[1]);
        tm_loaded(s);
        const bool masked = first < both.x || first + kTallTokens > both.y;
        const uint64_t unit2 = f2(unit, unit);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float4 e = exps[k];
            const float2 y = f2_parts(f2_fma(f2_mul(f2(__uint_as_float(s[k / 8][2 * k % 16]), __uint_as_float(s[k / 8][2 * k % 16 + 1])), unit2),
                                             f2(e.x, e.y), f2(e.z, e.w)));
            s[k / 8][2 * k % 16] = __float_as_uint(weight_of(y.x));
            s[k / 8][2 * k % 16 + 1] = __float_as_uint(weight_of(y.y));
        }
        if (masked) {
            const int2 *see = reinterpret_cast<const int2 *>(image + T::kSeeAt) + half * (kBlockCols / 2);
            if (tree) {
                const int col0 = block * kBlockCols + half * (kBlockCols / 2);
                int was = -1;
                bool bit = true;
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const int i = a.by_group.div(col0 + k);
                    if (i != was) bit = tok < base || (i < r.n && tok < r.len && (tree_bits(a, r, i, tok) & 1u));
                    was = i;
                    const int2 c = see[k];
                    if (tok < c.x || tok >= c.y || !bit) s[k / 16][k % 16] = 0;
                }
            } else {
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const int2 c = see[k];
                    if (tok < c.x || tok >= c.y) s[k / 16][k % 16] = 0;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) total2 = f2_add(total2, f2(__uint_as_float(s[k / 8][2 * k % 16]), __uint_as_float(s[k / 8][2 * k % 16 + 1])));
    };
    if (tid == 0)
        for (; asked < min(kTallSlots, blocks); ++asked) ask(asked);
#pragma unroll 1
    for (int block = 0; block <= blocks; ++block) {
        if (block < blocks && warp == 0) {
            wait(block % kTallSlots, block / kTallSlots & 1);
            if (one_lane() && !dead) {
                const uint64_t q = tm_operand(slots + block % kTallSlots * T::kSlot, T::kQChunk);
                tm_mma_parts<tm_kind(kBlockCols, false), D / 16, T::kQPart>(tm + T::kTmD + (block & 1) * kBlockCols, tm, q,
                                                                            [](int k) { return (k >> 2) * T::kQChunk + (k & 3) * 32u; });
                tm_commit(&bar[kTallSlots + (block & 1)]);
            }
            __syncwarp();
        }
        if (block > 0) {
            // a barrier for each half of D: the next block's products may be done before a slow warp looks
            wait(kTallSlots + (block - 1 & 1), block - 1 >> 1 & 1);
            tm_after_sync();
            weigh(block - 1);
            tm_before_sync();
        }
        __syncthreads();  // D of the block before is read, and so is its slot
        tm_after_sync();
        if (tid == 0 && block > 0 && asked < blocks && !dead) ask(asked++);
    }
    // after a wait that gave up: leave only when the products and the copies that were started are done, as far as they will be
    if (warp == 0 && __any_sync(0xffffffffu, dead)) {
        if (one_lane()) tm_commit(&bar[kTallSlots + 2]);
        (void)mbar_wait(&bar[kTallSlots + 2], 0);
        if (tid == 0)
            for (int k = max(0, asked - kTallSlots); k < asked; ++k) (void)mbar_wait(&bar[k % kTallSlots], k / kTallSlots & 1);
        __syncwarp();
    }
    if (dead) sh_dead = 1;
    const float2 both = f2_parts(total2);
    if (half == 1) sh_sum[row] = both.x + both.y;
    __syncthreads();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(T::kTm));
    if (half == 0 && row < live && !sh_skip[row / kKvSlab]) {
        float sum = both.x + both.y + sh_sum[row];
        if (sh_dead) sum = __int_as_float(0x7fffffff);
        *out = had ? fmaf(w.keep, earlier, sum) : sum;
    }
}

// More columns than kBlockCols take the tall kernel, and more than kTallFrom where all its CTAs run at once (its second launch, and
// a CTA's start, cost it as much as eight groups of four columns): 8 heads of 128 over 1000 tokens, tall and few, 28 columns 8.8 us and 7.9,
// 32 8.9 and 8.4, 36 8.9 and 9.5, 48 8.6 and 11.0, and over 64000 48 columns 67.0 and 49.7, 64 67.1 and 62.8; of 192 dimensions 28
// columns 10.2 and 9.5, 36 10.2 and 11.7; of 256, where the other kernel has one CTA an SM, 28 11.2 and 12.4.
constexpr int kFewCols = 24;  // up to which no rule takes the tall kernel: no workspace
template <int NB> constexpr int kTallFrom = NB < 8 ? 32 : kFewCols;
template <int NB> bool weights_tall(int64_t columns, int64_t items, int64_t max_kv_len, int sms) {
    return columns > kBlockCols || (columns > kTallFrom<NB> && items * ((max_kv_len + kTallTokens - 1) / kTallTokens) <= TallGeom<NB>::kCtas * sms);
}
size_t weights_bytes(int head_dim, int n_seq, int n_kv_heads, int group, int n_tok, int max_q_len) {
    if (static_cast<int64_t>(std::min(max_q_len, n_tok)) * group <= kFewCols) return 0;
    const int64_t images = weight_blocks(n_seq, n_tok, group) * n_kv_heads;
    switch (kv_blocks(head_dim)) {
    case 2: return images * TallGeom<2>::kImage;
    case 3: return images * TallGeom<3>::kImage;
    case 4: return images * TallGeom<4>::kImage;
    case 6: return images * TallGeom<6>::kImage;
    default: return images * TallGeom<8>::kImage;
    }
}

template <int NB, bool ONE> cudaError_t launch_few(const WeightArgs &w, int64_t items, int64_t columns, int sms, cudaStream_t st) {
    const cudaError_t e = smem_limit_raised<&attn_weights_kernel<NB, ONE>>();
    if (e != cudaSuccess) return e;
    constexpr int kStep = kStepTiles * kKvSlab;
    const int64_t steps = items * ((w.a.max_kv_len + kStep - 1) / kStep), ctas = static_cast<int64_t>(kWeightCtas) * sms;
    const size_t smem = kWeightRing<NB> + static_cast<size_t>((columns + 3) / 4) * 2 * NB * 256;
    return launch_block_op(&attn_weights_kernel<NB, ONE>, dim3(static_cast<unsigned>(std::min(steps, ctas))), dim3(kWeightThreads), smem, st, w);
}
template <int NB> cudaError_t launch_weights(WeightArgs w, int64_t items, int64_t columns, int sms, cudaStream_t st) {
    const int64_t most = w.a.max_kv_len;
    if (weights_tall<NB>(columns, items, most, sms)) {
        cudaError_t e = smem_limit_raised<&attn_weights_tall_kernel<NB>>();
        if (e != cudaSuccess) return e;
        const int64_t blocks = (columns + kBlockCols - 1) / kBlockCols;
        w.by_blocks = FastDiv::of(static_cast<int32_t>(blocks));
        e = launch_block_op(&weights_q_kernel<NB>, dim3(static_cast<unsigned>(items * blocks)), dim3(kWeightThreads), 0, st, w);
        if (e != cudaSuccess) return e;
        const int64_t chunks = (most + kTallTokens - 1) / kTallTokens;
        w.chunks = static_cast<int32_t>(chunks);
        w.by_items = FastDiv::of(static_cast<int32_t>(items));
        return launch_block_op(&attn_weights_tall_kernel<NB>, dim3(static_cast<unsigned>(items * chunks)), dim3(kWeightThreads),
                               TallGeom<NB>::kSmem, st, w);
    }
    return columns <= 4 ? launch_few<NB, true>(w, items, columns, sms, st) : launch_few<NB, false>(w, items, columns, sms, st);
}

}  // namespace
}  // namespace zdmmv

using namespace zdmmv;

extern "C" {

size_t zdmmv_attn_weights_q4_0_workspace_bytes(const zdmmv_kv_cache *cache, int n_q_heads, int n_tok, int max_q_len) {
    KvView c{};
    if (kv_check(cache, &c) != ZDMMV_OK || n_q_heads < 1 || n_q_heads > 65535 || n_q_heads % c.n_kv_heads || n_tok < 0 || max_q_len < 1)
        return 0;
    return weights_bytes(cache->head_dim, c.n_seq, c.n_kv_heads, n_q_heads / c.n_kv_heads, n_tok, max_q_len);
}

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
    // 128 tokens of a kv head are a CTA of the tall kernel; a step of the other is 256
    const int64_t steps = items * ((static_cast<int64_t>(g.max_kv_len) + kTallTokens - 1) / kTallTokens);
    if (columns > kAllCols || steps > 0x7fffff00 || items * ((columns + kBlockCols - 1) / kBlockCols) > 0x7fffff00) return ZDMMV_ERR_SHAPE;
    if (g.max_kv_len == 0) return ZDMMV_OK;
    if (!g.q_start || !g.kv_len || !g.out || (g.n_tok > 0 && (!g.q || !g.lse))) return ZDMMV_ERR_NULL;
    if ((g.n_tok > 0 && g.q_stride < static_cast<int64_t>(g.n_q_heads) * cache->head_dim) || g.out_stride < g.max_kv_len ||
        (g.before && g.before_stride < g.max_kv_len) || (g.before == g.out && g.before_stride != g.out_stride))
        return ZDMMV_ERR_SHAPE;
    if (kv_misaligned(g.q, 16) || g.q_stride % 4 || kv_misaligned(g.q_start, 4) || kv_misaligned(g.kv_len, 4) || kv_misaligned(g.lse, 4) ||
        kv_misaligned(g.seen, 4) || kv_misaligned(g.before, 4) || kv_misaligned(g.out, 4) || kv_misaligned(g.status_dev, 4) || kv_misaligned(g.workspace, 16))
        return ZDMMV_ERR_ALIGN;
    const size_t need = weights_bytes(cache->head_dim, a.c.n_seq, a.c.n_kv_heads, group, g.n_tok, g.max_q_len);
    if (need && !g.workspace) return ZDMMV_ERR_NULL;
    if (g.workspace_bytes < need) return ZDMMV_ERR_SIZE;
    w.images = static_cast<uint8_t *>(g.workspace);
    a.fault = current_fault_word();
    if (!a.fault) return ZDMMV_ERR_CUDA;
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
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
    switch (kv_blocks(cache->head_dim)) {
    case 2: e = launch_weights<2>(w, items, columns, sms, s); break;
    case 3: e = launch_weights<3>(w, items, columns, sms, s); break;
    case 4: e = launch_weights<4>(w, items, columns, sms, s); break;
    case 6: e = launch_weights<6>(w, items, columns, sms, s); break;
    case 8: e = launch_weights<8>(w, items, columns, sms, s); break;
    }
    return e == cudaSuccess ? ZDMMV_OK : ZDMMV_ERR_CUDA;
}

}  // extern "C"
