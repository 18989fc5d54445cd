// zdmmv_attn.cuh -- attention over the paged 4-bit cache (zdmmv_attn_q4_0).
//
//   out_c = sum_t p_ct v_t / sum_t p_ct,   p_ct = exp2(s_ct - max),   s_ct = log2(e) scale (q_c . k_t)
//
// A COLUMN c is one query row: a new token's head. The columns of one kv head (the
// heads of its group times the sequence's new tokens) read the same K and V, so a
// CTA takes 8, 16, 32 or 64 of them and streams the kv head's tiles once.
//
// The arithmetic, on mma.sync m16n8k16 (fp16 in, fp32 sums):
//  * A code n (0..15) under the bits of 1024 is the fp16 number 1024 + n, or
//    1024 + 16 n one nibble higher; less 1032 or 1152 it is n - 8 or 16 (n - 8),
//    exactly. The factor 16 is taken out of the other operand (scores) or the
//    result. (The bare nibbles are fp16 subnormals and would do without the
//    subtraction, but the tensor cores keep 8 bits less of such products: 7e-6 of
//    the result instead of 4e-7.)
//  * Scores: A = q, rows 0..7 the columns' upper fp16 parts and rows 8..15 their
//    lower parts (q = hi + lo to 22 bits, scaled by a power of two so that neither
//    part is subnormal where it counts), B = 8 tokens' codes of half a block. Two
//    MMAs make a block's sum for 8 tokens; then s += d_k * (hi + lo) in fp32,
//    block by block.
//  * The C fragment of the scores holds, per lane, a column's two neighbouring
//    tokens: exactly the B fragment of the product with V (columns x tokens), so
//    p goes from one MMA to the next in its registers.
//  * Product with V: A = the codes' dimensions x 16 tokens. V's scales are per
//    (token, block): x = p * d_v, split into two
//    fp16 parts again. p is kept in units of 2^sx, sx such that x <= 2^14 for the
//    largest |d_v| met: with fp16's lowest unit at 2^-24 every x is then exact to
//    2^-38 of the largest.
//
// Work: grid (kv head of a sequence and column tile) x (split of its tokens); a
// producer warp copies tiles (one bulk copy each) into a ring, the consumer warps
// split a stage's tiles among them (WC = 1) or the columns (WC = 4). Each warp has
// its own running maximum and sums; they are joined once, at the end, through
// shared memory, and the splits by attn_join_kernel.
#pragma once

#include "zdmmv_kv.cuh"

namespace zdmmv {

struct AttnArgs {
    KvView c;
    const float *q;
    const int32_t *q_start, *kv_len;
    float *out;
    float *part;        // partial sums [item][split][column][dim], then float2 (max, sum) [item][split][column]
    float2 *part_ml;
    int32_t *status;
    uint32_t *fault;
    int64_t q_stride;
    int32_t n_tok, n_q_heads, group, max_q_len, max_kv_len, window;
    int32_t n_ct;       // column tiles of a kv head of a sequence
    int32_t n_split, chunk;  // most splits, tiles of a split
    int32_t stages;
    int32_t wc;         // warps that split the columns (the others split the tokens)
    float scale_log2;
};

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = kAttnWarps * 32 + 32;
constexpr int kAttnBarBytes = 256;
constexpr int kAttnMaxStages = 8;

// Tiles of a pipeline stage: about 18 KB.
template <int NB> struct AttnStage {
    static constexpr int kTiles = NB <= 2 ? 16 : (NB <= 4 ? 8 : 4);
    static constexpr int kBytes = kTiles * KvGeom<NB>::kTileBytes;
};

// What a CTA (and the join) works on, from the lengths on the device.
struct AttnRange {
    int q0, n;       // first row of the sequence, its new tokens (as far as they lie in 0..n_tok)
    int len;
    bool bad;
    int slab0, slabs;  // tiles that any column of the column tile sees
    __device__ int splits(int chunk) const { return slabs <= chunk ? 1 : (slabs + chunk - 1) / chunk; }
};
__device__ __forceinline__ AttnRange attn_range(const AttnArgs &a, int seq, int ct, int cols) {
    AttnRange r;
    const int q0 = a.q_start[seq], q1 = a.q_start[seq + 1];
    r.len = a.kv_len[seq];
    r.bad = q0 < 0 || q1 < q0 || q1 > a.n_tok || q1 - q0 > a.max_q_len || r.len < 0 || r.len > a.max_kv_len ||
            r.len > static_cast<int64_t>(a.c.max_pages) * a.c.page_tokens;
    r.q0 = min(max(q0, 0), a.n_tok);
    r.n = max(0, min(q1, a.n_tok) - r.q0);
    const int i0 = ct * cols / a.group, i1 = min(r.n - 1, (ct * cols + cols - 1) / a.group);
    const int end = max(0, r.len - (r.n - 1 - i1));
    const int low = a.window > 0 ? max(0, r.len - (r.n - 1 - i0) - a.window) : 0;
    r.slab0 = low / kKvSlab;
    r.slabs = r.bad ? 0 : max(0, (end + kKvSlab - 1) / kKvSlab - r.slab0);
    return r;
}

__device__ __forceinline__ void mma_acc(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t h2_add(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// hi + lo = (x, y) to 22 bits, as two fp16 pairs
__device__ __forceinline__ void split_h2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack_h2(x, y);
    lo = pack_h2(x - half_lo(hi), y - half_hi(hi));
}

// The 8 codes of a word as exact fp16 pairs: n - 8 of the nibbles 0 and 4, 16 (n - 8) of 1 and 5, n - 8 of 2 and 6,
// 16 (n - 8) of 3 and 7.
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t (&f)[4]) {
    constexpr uint32_t kMagic = 0x64006400u, kM1032 = 0xE408E408u, kM1152 = 0xE480E480u;
    const uint32_t w8 = w >> 8;
    f[0] = h2_add((w & 0x000F000Fu) | kMagic, kM1032);
    f[1] = h2_add((w & 0x00F000F0u) | kMagic, kM1152);
    f[2] = h2_add((w8 & 0x000F000Fu) | kMagic, kM1032);
    f[3] = h2_add((w8 & 0x00F000F0u) | kMagic, kM1152);
}

// NB words of a lane: NB / W vectors of W words, `step` bytes apart.
template <int NB, int W> __device__ __forceinline__ void lds_words(uint32_t at, uint32_t step, uint32_t (&w)[NB]) {
#pragma unroll
    for (int c = 0; c < NB / W; ++c) {
        const uint32_t p = at + c * step;
        if constexpr (W == 4) {
            const uint4 v = lds128(p);
            w[4 * c] = v.x; w[4 * c + 1] = v.y; w[4 * c + 2] = v.z; w[4 * c + 3] = v.w;
        } else if constexpr (W == 2) {
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[2 * c]), "=r"(w[2 * c + 1]) : "r"(p));
        } else {
            w[c] = lds32(p);
        }
    }
}

__device__ __forceinline__ void attn_consumer_barrier() {
    asm volatile("bar.sync 1, %0;" ::"n"(kAttnWarps * 32) : "memory");
}

template <int NB, int NT>
__global__ void __launch_bounds__(kAttnThreads, NB * NT <= 4 ? 3 : (NB * NT <= 8 ? 2 : 1)) attn_kernel(AttnArgs a) {
    using G = KvGeom<NB>;
    using S = AttnStage<NB>;
    constexpr int D = G::kDim;
    constexpr bool kQReg = NB * NT <= 8;  // q's fragments in registers, else in shared memory
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float sh_m[kAttnWarps][NT * 8], sh_l[kAttnWarps][NT * 8];
    __shared__ int sh_bad;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem);
    uint64_t *empty = full + kAttnMaxStages;
    uint8_t *ring = smem + kAttnBarBytes;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cols = 8 * NT * a.wc;  // columns of the CTA
    if (tid == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kAttnWarps);
        }
        sh_bad = 0;
        fence_barrier_init();
    }
    __syncthreads();
    block_op_wait();
    block_op_release();

    const int item = blockIdx.x, split = blockIdx.y;
    const int ct = item % a.n_ct;
    const int kvh = item / a.n_ct % a.c.n_kv_heads;
    const int seq = item / a.n_ct / a.c.n_kv_heads;
    const AttnRange r = attn_range(a, seq, ct, cols);
    if (ct * cols >= r.n * a.group) return;
    const int n_splits = r.splits(a.chunk);
    if (split >= n_splits) return;
    const int first = r.slab0 + split * a.chunk;                        // tiles first .. last-1
    const int last = min(r.slab0 + r.slabs, first + a.chunk);
    const int n_stages = (last - first + S::kTiles - 1) / S::kTiles;

    if (warp == kAttnWarps) {
        // ------------------------------------------------------- producer
        const uint64_t policy = l2_evict_first_policy();
        const int page_tiles = a.c.page_tokens / kKvSlab;
        const int32_t *table = a.c.table + static_cast<int64_t>(seq) * a.c.max_pages;
        const int64_t head_at = static_cast<int64_t>(kvh) * page_tiles * G::kTileBytes;
        int slab = first + lane;  // the lane's tile of the stage
        int page = lane < S::kTiles && slab < last ? table[slab / page_tiles] : 0;
        bool ok = true;
        int st = 0;
        for (; st < n_stages; ++st) {
            const int s = st % a.stages;
            const bool mine = lane < S::kTiles && slab < last;
            const bool bad_page = mine && (page < 0 || page >= a.c.n_pages);
            const int use = bad_page ? 0 : page;
            const uint8_t *src = a.c.pages + use * a.c.page_bytes + head_at +
                                 static_cast<int64_t>(slab % page_tiles) * G::kTileBytes;
            slab += S::kTiles;
            page = lane < S::kTiles && slab < last ? table[slab / page_tiles] : 0;  // the next stage's, ahead of time
            if (st >= a.stages) {
                if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], static_cast<uint32_t>(st / a.stages - 1) & 1u))) {
                    ok = false;
                    break;
                }
                fence_proxy_async_smem();
            }
            const bool any_bad = __any_sync(0xffffffffu, bad_page);
            if (lane == 0) {
                if (any_bad) {
                    sh_bad = 1;
                    if (a.status) *a.status = 1;
                }
                const int n = min(S::kTiles, last - first - st * S::kTiles);
                mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(n) * G::kTileBytes);
            }
            __syncwarp();
            if (mine) bulk_copy_g2s(ring + s * S::kBytes + lane * G::kTileBytes, src, G::kTileBytes, &full[s], policy);
        }
        if (!ok && lane == 0) atomicOr(a.fault, 1u);
        // leave only when the copies into this CTA's shared memory have landed
        for (int k = max(0, st - a.stages); k < st; ++k)
            (void)mbar_wait(&full[k % a.stages], static_cast<uint32_t>(k / a.stages) & 1u);
        return;
    }

    // ---------------------------------------------------------- consumers
    const int g = lane >> 2, t = lane & 3;
    const int wc = warp % a.wc, wt = warp / a.wc, n_wt = kAttnWarps / a.wc;
    const int col0 = ct * cols + wc * 8 * NT;  // the warp's first column

    // q's fragments: column g of each group of 8, this lane's 8 dimensions 8t.. of every block
    uint32_t qf[kQReg ? NT : 1][kQReg ? 2 * NB : 1][4];
    uint4 *q_sm = reinterpret_cast<uint4 *>(ring + a.stages * S::kBytes) + warp * (NT * 2 * NB * 32) + lane;
    float qs[NT];
    int end[NT], low[NT];
    int end_min = r.len, low_max = 0, len = r.len;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int col = col0 + 8 * nt + g;
        const int i = col / a.group;
        const bool valid = i < r.n;
        end[nt] = valid ? max(0, r.len - (r.n - 1 - i)) : r.len;
        low[nt] = valid && a.window > 0 ? max(0, end[nt] - a.window) : 0;
        end_min = min(end_min, end[nt]);
        low_max = max(low_max, low[nt]);
        const float *q = a.q + static_cast<int64_t>(r.q0 + (valid ? i : 0)) * a.q_stride +
                         static_cast<int64_t>(kvh * a.group + (valid ? col - i * a.group : 0)) * D + 8 * t;
        float v[NB][8];
        float top = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
            if (valid) {
                x = *reinterpret_cast<const float4 *>(q + b * kQK);
                y = *reinterpret_cast<const float4 *>(q + b * kQK + 4);
            }
            v[b][0] = x.x; v[b][1] = x.y; v[b][2] = x.z; v[b][3] = x.w;
            v[b][4] = y.x; v[b][5] = y.y; v[b][6] = y.z; v[b][7] = y.w;
#pragma unroll
            for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(v[b][k]));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^e brings the column's largest magnitude into [2^13, 2^14)
        int e = 13 - (static_cast<int>(__float_as_uint(top) >> 23) - 127);
        e = min(100, max(-100, e));
        const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        qs[nt] = a.scale_log2 * down;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[b][k] *= up;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // k slots: the codes at bits 0 and 16 of the (shifted) word, then those at bits 4 and 20
                uint4 f;
                split_h2(v[b][2 * h], v[b][2 * h + 4], f.x, f.y);
                split_h2(v[b][2 * h + 1] * 0.0625f, v[b][2 * h + 5] * 0.0625f, f.z, f.w);
                if constexpr (kQReg) {
                    qf[nt][2 * b + h][0] = f.x; qf[nt][2 * b + h][1] = f.y;
                    qf[nt][2 * b + h][2] = f.z; qf[nt][2 * b + h][3] = f.w;
                } else {
                    q_sm[(nt * 2 * NB + 2 * b + h) * 32] = f;
                }
            }
        }
    }
    // tiles outside low_max .. end_min need masks (warp-uniform)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        end_min = min(end_min, __shfl_xor_sync(0xffffffffu, end_min, o));
        low_max = max(low_max, __shfl_xor_sync(0xffffffffu, low_max, o));
    }
    __syncwarp();

    float o[NT][2 * NB][4], m[NT], l[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt] = -INFINITY;
        l[nt] = 0.0f;
#pragma unroll
        for (int k = 0; k < 2 * NB; ++k) o[nt][k][0] = o[nt][k][1] = o[nt][k][2] = o[nt][k][3] = 0.0f;
    }
    int sx = 38;           // p is in units of 2^sx ...
    uint32_t cap = 0x0001;  // ... |d_v| <= 2^(14 - sx), as an fp16 number: here 2^-24
    bool dead = false;

    for (int st = 0; st < n_stages; ++st) {
        const int s = st % a.stages;
        if (!__all_sync(0xffffffffu, mbar_wait(&full[s], static_cast<uint32_t>(st / a.stages) & 1u))) {
            if (lane == 0) atomicOr(a.fault, 1u);
            dead = true;
            break;
        }
        const int n_tiles = min(S::kTiles, last - first - st * S::kTiles);
        for (int k = wt; k < n_tiles; k += n_wt) {
            const int t0 = (first + st * S::kTiles + k) * kKvSlab;
            const uint32_t tile = smem_addr(ring + s * S::kBytes + k * G::kTileBytes);
            // ------------------------------------------------ scores
            float sc[NT][4];  // column g, tokens 2t, 2t+1, 8+2t, 8+2t+1
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t kw[NB], dk[NB];
                lds_words<NB, G::kVec>(tile + (h * NB * 32 + lane * G::kVec) * 4, 128 * G::kVec, kw);
                lds_words<NB, G::kVec>(tile + G::kKScaleAt + (t + 4 * h) * NB * 4, 4 * G::kVec, dk);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) sc[nt][2 * h] = sc[nt][2 * h + 1] = 0.0f;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    uint32_t kc[4];
                    code_pairs(kw[b], kc);
                    const float d0 = half_lo(dk[b]), d1 = half_hi(dk[b]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        if constexpr (kQReg) {
                            mma_acc(c, qf[nt][2 * b], kc[0], kc[1]);
                            mma_acc(c, qf[nt][2 * b + 1], kc[2], kc[3]);
                        } else {
                            const uint4 f0 = q_sm[(nt * 2 * NB + 2 * b) * 32], f1 = q_sm[(nt * 2 * NB + 2 * b + 1) * 32];
                            const uint32_t a0[4] = {f0.x, f0.y, f0.z, f0.w}, a1[4] = {f1.x, f1.y, f1.z, f1.w};
                            mma_acc(c, a0, kc[0], kc[1]);
                            mma_acc(c, a1, kc[2], kc[3]);
                        }
                        sc[nt][2 * h] = fmaf(d0, c[0] + c[2], sc[nt][2 * h]);
                        sc[nt][2 * h + 1] = fmaf(d1, c[1] + c[3], sc[nt][2 * h + 1]);
                    }
                }
            }
            // ------------------------------------------------ V's scales, masks
            uint32_t dv[2][NB];
            lds_words<NB, G::kVec>(tile + G::kVScaleAt + t * NB * 4, 4 * G::kVec, dv[0]);
            lds_words<NB, G::kVec>(tile + G::kVScaleAt + (t + 4) * NB * 4, 4 * G::kVec, dv[1]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[nt][i] *= qs[nt];
            if (t0 + kKvSlab > end_min || t0 < low_max) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = t0 + 2 * t + (i & 1) + 8 * (i >> 1);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        if (tok < low[nt] || tok >= end[nt]) sc[nt][i] = -INFINITY;
                    // a token past the sequence's may hold anything, NaN among it: its V counts for nothing
                    if (tok >= len) {
#pragma unroll
                        for (int b = 0; b < NB; ++b) dv[i >> 1][b] &= (i & 1) ? 0x0000ffffu : 0xffff0000u;
                    }
                }
            }
            // ------------------------------------------------ the unit of p: largest |d_v| so far
            uint32_t big = 0;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                // magnitudes of fp16 numbers order like their bits
                big = __vmaxu2(big, dv[0][b] & 0x7fff7fffu);
                big = __vmaxu2(big, dv[1][b] & 0x7fff7fffu);
            }
            big = max(big & 0xffffu, big >> 16);
            if (__any_sync(0xffffffffu, big > cap)) {
                big = __reduce_max_sync(0xffffffffu, big);
                // the power of two at or above it
                const float f = half_lo(min(big, 0x7bffu));
                const int ex = static_cast<int>((__float_as_uint(f) + 0x7fffffu) >> 23) - 127;
                const int to = 14 - ex;
                const float keep = __uint_as_float(static_cast<uint32_t>(max(0, to - sx + 127)) << 23);
                sx = to;
                cap = ex >= 16 ? 0x7fffu : __half_as_ushort(__float2half_rn(__uint_as_float(static_cast<uint32_t>(ex + 127) << 23)));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    l[nt] *= keep;
#pragma unroll
                    for (int j = 0; j < 2 * NB; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[nt][j][i] *= keep;
                }
            }
            // ------------------------------------------------ softmax
            bool grow = false;
            float top[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                top[nt] = fmaxf(fmaxf(sc[nt][0], sc[nt][1]), fmaxf(sc[nt][2], sc[nt][3]));
                top[nt] = fmaxf(top[nt], __shfl_xor_sync(0xffffffffu, top[nt], 1));
                top[nt] = fmaxf(top[nt], __shfl_xor_sync(0xffffffffu, top[nt], 2));
                grow |= top[nt] > m[nt];
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float to = fmaxf(m[nt], top[nt]);
                    const float keep = to > m[nt] ? exp2_approx(m[nt] - to) : 1.0f;  // 0 where nothing was seen before
                    m[nt] = to;
                    l[nt] *= keep;
                    const float k0 = __shfl_sync(0xffffffffu, keep, 8 * t), k1 = __shfl_sync(0xffffffffu, keep, 8 * t + 4);
#pragma unroll
                    for (int j = 0; j < 2 * NB; ++j) {
                        o[nt][j][0] *= k0; o[nt][j][2] *= k0;
                        o[nt][j][1] *= k1; o[nt][j][3] *= k1;
                    }
                }
            }
            float p[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float base = m[nt] == -INFINITY ? 0.0f : m[nt] - static_cast<float>(sx);
#pragma unroll
                for (int i = 0; i < 4; ++i) p[nt][i] = exp2_approx(sc[nt][i] - base);
                l[nt] += (p[nt][0] + p[nt][1]) + (p[nt][2] + p[nt][3]);
            }
            // ------------------------------------------------ product with V
            uint32_t vw[2][NB];
            lds_words<NB, G::kVec>(tile + G::kVAt + lane * G::kVec * 4, 128 * G::kVec, vw[0]);
            lds_words<NB, G::kVec>(tile + G::kVAt + (NB * 32 + lane * G::kVec) * 4, 128 * G::kVec, vw[1]);
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                uint32_t f0[4], f1[4];  // dimensions 4g, 4g+1 and 4g+2, 4g+3 of the block
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t vc[4];
                    code_pairs(vw[h][j], vc);
                    f0[2 * h] = vc[0]; f0[2 * h + 1] = vc[1];
                    f1[2 * h] = vc[2]; f1[2 * h + 1] = vc[3];
                }
                const float d0 = half_lo(dv[0][j]), d1 = half_hi(dv[0][j]), d2 = half_lo(dv[1][j]), d3 = half_hi(dv[1][j]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint32_t hi0, lo0, hi1, lo1;
                    split_h2(p[nt][0] * d0, p[nt][1] * d1, hi0, lo0);
                    split_h2(p[nt][2] * d2, p[nt][3] * d3, hi1, lo1);
                    mma_acc(o[nt][2 * j], f0, hi0, hi1);
                    mma_acc(o[nt][2 * j + 1], f1, hi0, hi1);
                    mma_acc(o[nt][2 * j], f0, lo0, lo1);
                    mma_acc(o[nt][2 * j + 1], f1, lo0, lo1);
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
    }

    // ------------------------------------------------ join the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        l[nt] += __shfl_xor_sync(0xffffffffu, l[nt], 1);
        l[nt] += __shfl_xor_sync(0xffffffffu, l[nt], 2);
        m[nt] -= static_cast<float>(sx);  // the maximum in p's unit
        if (t == 0) {
            sh_m[warp][8 * nt + g] = m[nt];
            sh_l[warp][8 * nt + g] = dead ? __int_as_float(0x7fffffff) : l[nt];
        }
    }
    attn_consumer_barrier();  // every warp is done with the ring
    float *sum = reinterpret_cast<float *>(ring);  // [warp][column of the warp][D]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = 8 * nt + 2 * t + h;
            float top = -INFINITY;
            for (int w = 0; w < n_wt; ++w) top = fmaxf(top, sh_m[w * a.wc + wc][c]);
            f[h] = top == -INFINITY ? 0.0f : exp2_approx(sh_m[warp][c] - top);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float *dst = sum + (warp * NT * 8 + 8 * nt + 2 * t + h) * D + 4 * g;
            const float one = f[h], sixteenth = f[h] * 0.0625f;
#pragma unroll
            for (int j = 0; j < NB; ++j)
                *reinterpret_cast<float4 *>(dst + j * kQK) =
                    make_float4(o[nt][2 * j][h] * one, o[nt][2 * j][2 + h] * sixteenth, o[nt][2 * j + 1][h] * one,
                                o[nt][2 * j + 1][2 + h] * sixteenth);
        }
    }
    attn_consumer_barrier();
    const bool bad = r.bad || sh_bad;
    if (r.bad && tid == 0 && a.status) *a.status = 1;
    constexpr int kQuads = D / 4;
    for (int k = tid; k < cols * kQuads; k += kAttnWarps * 32) {
        const int c = k / kQuads, e = 4 * (k % kQuads);
        const int w0 = c / (8 * NT), wcol = c % (8 * NT);
        const int col = ct * cols + c;
        if (col >= r.n * a.group) break;
        float top = -INFINITY, ls = 0.0f;
        for (int w = 0; w < n_wt; ++w) top = fmaxf(top, sh_m[w * a.wc + w0][wcol]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < n_wt; ++w) {
            const int ww = w * a.wc + w0;
            ls += sh_l[ww][wcol] * (top == -INFINITY ? 1.0f : exp2_approx(sh_m[ww][wcol] - top));
            const float4 x = *reinterpret_cast<const float4 *>(sum + (ww * NT * 8 + wcol) * D + e);
            acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
        }
        if (bad) ls = __int_as_float(0x7fffffff);
        if (n_splits == 1) {
            const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
            const int i = col / a.group;
            float *dst = a.out + (static_cast<int64_t>(r.q0 + i) * a.n_q_heads + kvh * a.group + (col - i * a.group)) * D + e;
            *reinterpret_cast<float4 *>(dst) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        } else {
            const int64_t at = (static_cast<int64_t>(item) * a.n_split + split) * cols + c;
            *reinterpret_cast<float4 *>(a.part + at * D + e) = acc;
            if (e == 0) a.part_ml[at] = make_float2(top, ls);
        }
    }
}

// Joins the splits of a column: out = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s, in the splits' order. One CTA
// a column; groups of D/4 threads take every n-th split.
constexpr int kJoinThreads = 128;
template <int NB> __global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(AttnArgs a, int cols) {
    constexpr int D = NB * kQK, kQuads = D / 4, kGroups = kJoinThreads / kQuads;
    __shared__ float4 sum[kGroups][kQuads];
    __shared__ float sum_l[kGroups];
    block_op_wait();
    block_op_release();
    const int item = blockIdx.x, c = blockIdx.y;
    const int ct = item % a.n_ct;
    const int kvh = item / a.n_ct % a.c.n_kv_heads;
    const int seq = item / a.n_ct / a.c.n_kv_heads;
    const AttnRange r = attn_range(a, seq, ct, cols);
    const int col = ct * cols + c;
    const int n = r.splits(a.chunk);
    if (n == 1 || col >= r.n * a.group) return;
    const int64_t at = static_cast<int64_t>(item) * a.n_split * cols + c;
    float top = -INFINITY;
    for (int s = 0; s < n; ++s) top = fmaxf(top, a.part_ml[at + static_cast<int64_t>(s) * cols].x);
    const int grp = threadIdx.x / kQuads, e = threadIdx.x % kQuads;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float ls = 0.0f;
    if (grp < kGroups) {
        for (int s = grp; s < n; s += kGroups) {
            const int64_t p = at + static_cast<int64_t>(s) * cols;
            const float2 ml = a.part_ml[p];
            const float f = top == -INFINITY ? 0.0f : exp2_approx(ml.x - top);
            const float4 x = *reinterpret_cast<const float4 *>(a.part + p * D + 4 * e);
            ls += f * ml.y;
            acc.x += f * x.x; acc.y += f * x.y; acc.z += f * x.z; acc.w += f * x.w;
        }
        sum[grp][e] = acc;
        if (e == 0) sum_l[grp] = ls;
    }
    __syncthreads();
    if (grp != 0) return;
    for (int k = 1; k < kGroups; ++k) {
        const float4 x = sum[k][e];
        acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
        ls += sum_l[k];
    }
    const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
    const int i = col / a.group;
    float *dst = a.out + (static_cast<int64_t>(r.q0 + i) * a.n_q_heads + kvh * a.group + (col - i * a.group)) * D + 4 * e;
    *reinterpret_cast<float4 *>(dst) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
}

// ------------------------------------------------------------------ host side
struct AttnPlan {
    int nt, wc;           // column groups of 8 a warp, warps that split the columns
    int n_ct, cols;       // column tiles, columns of a tile
    int64_t items;        // kv heads of sequences x column tiles
    int chunk, n_split;   // tiles of a split, most splits
    int max_split;        // an upper bound of n_split that only grows with max_kv_len (the workspace's)
};

template <int NB> cudaError_t launch_attn(AttnArgs a, const AttnPlan &p, cudaStream_t st);
extern template cudaError_t launch_attn<2>(AttnArgs, const AttnPlan &, cudaStream_t);
extern template cudaError_t launch_attn<3>(AttnArgs, const AttnPlan &, cudaStream_t);
extern template cudaError_t launch_attn<4>(AttnArgs, const AttnPlan &, cudaStream_t);
extern template cudaError_t launch_attn<6>(AttnArgs, const AttnPlan &, cudaStream_t);
extern template cudaError_t launch_attn<8>(AttnArgs, const AttnPlan &, cudaStream_t);

#ifdef ZDMMV_ATTN_INSTANTIATE
template <int NB, int NT> cudaError_t launch_attn_nt(const AttnArgs &a, const AttnPlan &p, cudaStream_t st) {
    constexpr bool kQReg = NB * NT <= 8;
    const size_t ring = static_cast<size_t>(a.stages) * AttnStage<NB>::kBytes + (kQReg ? 0 : kAttnWarps * NT * 2 * NB * 512);
    const size_t join = static_cast<size_t>(kAttnWarps) * NT * 8 * NB * kQK * 4;
    const size_t smem = kAttnBarBytes + (ring > join ? ring : join);
    cudaError_t e = cudaFuncSetAttribute(attn_kernel<NB, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    e = launch_block_op(attn_kernel<NB, NT>, dim3(static_cast<unsigned>(p.items), p.n_split), kAttnThreads, smem, st, a);
    if (e != cudaSuccess || p.n_split == 1) return e;
    return launch_block_op(attn_join_kernel<NB>, dim3(static_cast<unsigned>(p.items), p.cols), kJoinThreads, 0, st, a,
                           p.cols);
}
template <int NB> cudaError_t launch_attn(AttnArgs a, const AttnPlan &p, cudaStream_t st) {
    a.stages = 3;
    return p.nt == 1 ? launch_attn_nt<NB, 1>(a, p, st) : launch_attn_nt<NB, 2>(a, p, st);
}
#endif

}  // namespace zdmmv
