// zdmmv_attn.cuh -- attention over the paged 4-bit cache (zdmmv_attn_q4_0).
//
//   out_c = sum_t p_ct v_t / sum_t p_ct,   p_ct = exp2(s_ct - max),   s_ct = log2(e) scale (q_c . k_t)
//
// A COLUMN c is one query row: a new token's head. The columns of one kv head (the
// heads of its group times the sequence's new tokens) read the same K and V, so a
// CTA takes 4 to 128 of them and streams the kv head's tiles once. More than 16 columns
// with heads of up to 128 dimensions: zdmmv_attn_prompt.cuh. Else:
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
//  * Product with V: A = the codes' dimensions x 16 tokens, B = x = p * d_v (V's
//    scales are per token and block) in two fp16 parts, formed in fp16: with p =
//    ph + pl, xh = ph * d_v rounded, xl = pl * d_v + (ph * d_v - xh), whose bracket
//    one fma gives exactly. p is in units of 2^-13, so that x is an fp16 number while
//    |d_v| < 7: half of fp16's lowest unit, 2^-24, is then 2^-38 of the largest p.
//    32 tokens of which one has a larger scale take x = p * d_v in fp32 instead,
//    split in the unit of each column's and block's largest x, so that large values
//    cost neither other blocks nor other tokens their precision, and infinities and
//    NaN no column that does not see them.
//
// Work. Up to 16 columns a kv head of a sequence (decoding): the ITEMS (sequence, kv head) one after another are a row of
// STEPS of 16 tiles (a pair for each of a CTA's 8 warps), and every CTA of a grid that fills the device once takes an
// equal stretch of them, whatever the lengths: parts of an item at the stretch's ends, whole items between. Each warp has
// its own ring of two slots (a pair of tiles each, one bulk copy a tile), its own running maximum and its own sums; they
// are joined at the item's end through shared memory, and an item's parts by the CTA that finishes last (through the
// workspace). More columns: the grid is (column tile of an item) x (split of its tokens), the warps split the
// columns and share a ring.
//
// What it reaches. One sequence of 130975 tokens, 8 kv heads of 128, 4 columns (the narrow kernel): 36.2 us, 61% of the
// copy rate, of which some 12 us are the kernel's ends; at 2^20 tokens 220 us, 81%. 64 sequences of up to 16384 tokens:
// 98.0 us (64%). The narrow kernel is bound by its instructions as much as by memory (issue 61%, ALU 47% at 131K tokens).
#pragma once

#include <type_traits>

#include "zdmmv_kv.cuh"

namespace zdmmv {

struct AttnArgs {
    KvView c;
    FastDiv by_ct, by_heads, by_group, by_page_tiles, by_split;
    const float *q;
    const int32_t *q_start, *kv_len;
    float *out;
    uint32_t *count;    // parts of an item that have stored their sums (0 between calls)
    float *part;        // parts' sums [part][column][dim], then float2 (max, sum) [part][column]
    float2 *part_ml;
    int32_t *status;
    uint32_t *fault;
    int64_t q_stride;
    int32_t n_tok, n_q_heads, group, max_q_len, max_kv_len, window;
    int32_t n_ct;       // column tiles of a kv head of a sequence
    int32_t n_split, chunk;  // the grid's form: most splits, tiles of a split of the longest sequence; else 0
    int32_t round;      // ... whose length is a multiple of this power of two
    int32_t wc;         // warps that split the columns (the others split the tokens)
    float scale_log2;
};

constexpr int kAttnWarps = 8, kAttnThreads = kAttnWarps * 32;
constexpr int kWalker = kAttnThreads - 1;    // the thread that finds the CTA's next segment
constexpr int kStepTiles = 2 * kAttnWarps;  // tiles of a step: a ring slot for each warp
// The wide kernel's forms: own rings (up to 16 columns), a shared ring (17 to 64), a shared ring whose codes the CTA turns
// into fragments once for all its warps (more: prompts).
enum AttnForm { kOwn = 0, kShared = 1, kPrompt = 2 };
// Ring slots (a pair of tiles) of a CTA: two a warp; of the shared rings as many where they fit.
__host__ __device__ constexpr int attn_slots(int nb, int form) { return form == kOwn || (form == kShared && nb < 8) ? 16 : 8; }
// Heads of up to kTallBlocks blocks with more than kTallColumns columns take the form on tcgen05 (zdmmv_attn_prompt.cuh)
// instead of the shared and the prompt form: 8 sequences of 4000 tokens with 64 columns, 8 heads of 128, 99 us with the
// shared form and 46 with that; one of 60000 with 24 columns 88 and 66; 20 columns over 2000 16.5 and 14.1; 1024 columns over
// 8192 292 with the prompt form and 82.
constexpr int kTallBlocks = 4, kTallColumns = 16;
// Groups of 8 columns a warp of the prompt form: two, one where the shared memory does not hold q and the fragments of two.
__host__ __device__ constexpr int attn_prompt_nt(int nb) { return nb < 8 ? 2 : 1; }
// CTAs of the forms without a shared ring that run on an SM at once.
__host__ __device__ constexpr int attn_ctas_per_sm(int nb, int nt) { return nb * nt <= 4 ? 2 : 1; }
// Whether the warps' sums have shared memory of their own, so that the next item's tiles can come while they are joined.
__host__ __device__ constexpr bool attn_sums_apart(int nb, int nt, int form) { return form == kOwn && nb * nt < 16; }
constexpr int kAttnBarBytes = 256;  // two barriers a slot
constexpr float kAttnUnit = 13.0f;  // p is in units of 2^-kAttnUnit
// From scores of some size on (in powers of two) a float's step is a part of p that counts: p is then of the rounded score less
// the maximum, not of both in one fma, which would leave the largest score's own rounding in the exponent of every p: below
// 2^(1/32) of it at 2^20 (of the products here), below 2^(1/4) at 2^23 (tcgen05), 2^64 at 2^30.
constexpr float kHugeScore = 1048576.0f, kHugeScoreTall = 8388608.0f;
__device__ __forceinline__ bool score_huge(float m, float from) { return fabsf(m) >= from && m != -INFINITY; }
constexpr int kJoinAhead = 16;

// What a CTA (and the join) works on, from the lengths on the device.
struct AttnRange {
    int q0, n;       // first row of the sequence, its new tokens (as far as they lie in 0..n_tok)
    int len;
    bool bad;
    int slab0, slabs;  // tiles that any column of the column tile sees
};
__device__ __forceinline__ AttnRange attn_range(const AttnArgs &a, int seq, int ct, int cols) {
    AttnRange r;
    const int q0 = a.q_start[seq], q1 = a.q_start[seq + 1];
    r.len = a.kv_len[seq];
    r.bad = q0 < 0 || q1 < q0 || q1 > a.n_tok || q1 - q0 > a.max_q_len || r.len < 0 || r.len > a.max_kv_len ||
            r.len > static_cast<int64_t>(a.c.max_pages) * a.c.page_tokens;
    r.q0 = min(max(q0, 0), a.n_tok);
    r.n = max(0, min(q1, a.n_tok) - r.q0);
    const int i0 = a.by_group.div(ct * cols), i1 = min(r.n - 1, a.by_group.div(ct * cols + cols - 1));
    const int end = max(0, r.len - (r.n - 1 - i1));
    const int low = a.window > 0 ? max(0, r.len - (r.n - 1 - i0) - a.window) : 0;
    r.slab0 = low / kKvSlab;
    r.slabs = r.bad ? 0 : max(0, (end + kKvSlab - 1) / kKvSlab - r.slab0);
    return r;
}

// One CTA's share of an item: tiles first .. last-1, and where its sums go where others share the item.
struct AttnSeg {
    AttnRange r;
    int seq, kvh, ct;
    int first, last;
    int parts;           // CTAs that share the item
    int counter;         // ... their counter
    int mine, part0, part_step;  // this CTA's part; part s of the item is part0 (s = 0) or rest + s * part_step
    int rest;
    bool some;           // false: there is no such segment
    bool whole;          // the CTA has all of the item ...
    int base, steps;     // ... whose steps these are
    __device__ int part(int s) const { return s == 0 ? part0 : rest + s * part_step; }
};

// The grid's form, (item) x (split): the CTA's part of its item, tiles in equal stretches of kMinChunk or more; false where
// there is none. (Splitting each of several sequences by its own length cuts the short ones up for nothing: 22.4 instead of
// 15 us for 8 sequences of 3 to 8191 tokens and 16 heads.)
constexpr int kMinChunk = kStepTiles;
__device__ __forceinline__ bool attn_grid_seg(const AttnArgs &a, int cols, AttnSeg &g) {
    const int item = blockIdx.x, split = blockIdx.y;
    const int sh = a.by_ct.div(item);
    g.ct = a.by_ct.mod(item, sh);
    g.seq = a.by_heads.div(sh);
    g.kvh = a.by_heads.mod(sh, g.seq);
    g.r = attn_range(a, g.seq, g.ct, cols);
    if (g.ct * cols >= g.r.n * a.group) return false;
    // the host's chunk is for the longest sequence that the call allows; a single one is split by its own length
    const int chunk = a.c.n_seq > 1 ? a.chunk : max(kMinChunk, (a.by_split.div(g.r.slabs + a.n_split - 1) + a.round - 1) & -a.round);
    g.parts = max(1, (g.r.slabs + chunk - 1) / chunk);
    if (split >= g.parts) return false;
    g.first = g.r.slab0 + split * chunk;
    g.last = min(g.r.slab0 + g.r.slabs, g.first + chunk);
    g.counter = item;
    g.part0 = g.rest = item * a.n_split;
    g.part_step = 1;
    g.mine = g.part0 + split;
    return true;
}

// Decoding of several sequences: the CTA's stretch of the row of steps. It lies in shared memory, as the segments do (the main loop has no
// registers to spare).
struct AttnWalk {
    int ctas, each, more;  // CTAs that have steps; `each` and in all `more` besides, evenly spread
    float per_step;        // ctas / steps
    int snap;              // a stretch's end this near an item's moves there: a part of so few steps costs more than it evens
    int at, end;           // the CTA's steps
    int seq, kvh, base, steps;  // the item that holds step `at`: its first step, its steps
    AttnRange r;

    __device__ static int steps_of(const AttnRange &r) { return r.n == 0 ? 0 : max(1, (r.slabs + kStepTiles - 1) / kStepTiles); }
    __device__ int cut(int c) const { return c * each + c * more / ctas; }  // where CTA c's stretch begins, before snapping
    // ... after it; a cut inside the item of steps first .. first + n - 1 may move
    __device__ int snapped(int cut, int first, int n) const {
        if (cut <= first || cut >= first + n) return cut;
        return cut - first <= snap ? first : (first + n - cut <= snap ? first + n : cut);
    }
    __device__ int holder(int step) const {  // the CTA whose stretch holds a step, before snapping
        int c = min(ctas - 1, static_cast<int>(static_cast<float>(step) * per_step));
        while (cut(c) > step) --c;
        while (cut(c + 1) <= step) ++c;
        return c;
    }

    // Steps up to and with this thread's, of one value a thread of the CTA; `all` those of the whole CTA. scan: shared
    // memory for kAttnWarps ints, free again after the next barrier.
    __device__ static int upto(int w, int *scan, int &all) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, w, k);
            if (lane >= k) w += o;
        }
        if (lane == 31) scan[warp] = w;
        __syncthreads();
        all = 0;
#pragma unroll
        for (int k = 0; k < kAttnWarps; ++k) {
            if (k < warp) w += scan[k];
            all += scan[k];
        }
        return w;
    }
    // For all threads: fills *to, in shared memory, and is false in all where the CTA has nothing to do. scan: shared memory
    // for kAttnWarps ints.
    __device__ static bool begin(const AttnArgs &a, int cols, int *scan, AttnWalk *to) {
        const int tid = threadIdx.x, me = blockIdx.x, heads = a.c.n_kv_heads, n_seq = a.c.n_seq;
        // the sequences 256 at a time, one a thread; the first 256 are kept (beyond, they are looked at once more)
        AttnRange r{};
        int n = 0, all = 0;
        if (tid < n_seq) {
            r = attn_range(a, tid, 0, cols);
            n = steps_of(r);
        }
        int last = upto(n * heads, scan, all), total = all;
        for (int s0 = kAttnThreads; s0 < n_seq; s0 += kAttnThreads) {
            int more_all;
            __syncthreads();
            (void)upto(s0 + tid < n_seq ? steps_of(attn_range(a, s0 + tid, 0, cols)) * heads : 0, scan, more_all);
            total += more_all;
        }
        AttnWalk w;
        w.ctas = min(static_cast<int>(gridDim.x), total);
        if (me >= w.ctas) return false;
        w.each = total / w.ctas;
        w.more = total - w.each * w.ctas;
        w.per_step = static_cast<float>(w.ctas) / static_cast<float>(total);
        // a part costs its CTA about as much as a step and a half
        w.snap = min(2, w.each / 3);
        const int at = w.cut(me), end = w.cut(me + 1);
        // the threads whose sequences hold the stretch's ends snap them
        for (int s0 = 0, before = 0;;) {
            const int from = before + last - n * heads;
            if (n > 0 && end > from && end <= from + n * heads) {
                const int k = (end - 1 - from) / n;
                to->end = w.snapped(end, from + k * n, n);
            }
            if (n > 0 && at >= from && at < from + n * heads) {
                const int k = (at - from) / n;
                w.at = w.snapped(at, from + k * n, n);
                w.seq = s0 + tid;
                w.kvh = k;
                w.base = from + k * n;
                w.steps = n;
                to->ctas = w.ctas; to->each = w.each; to->more = w.more; to->snap = w.snap; to->per_step = w.per_step;
                to->at = w.at; to->seq = w.seq; to->kvh = w.kvh; to->base = w.base; to->steps = w.steps; to->r = r;
            }
            before += all;
            if (end <= before) break;
            s0 += kAttnThreads;
            r = AttnRange{};
            n = 0;
            if (s0 + tid < n_seq) {
                r = attn_range(a, s0 + tid, 0, cols);
                n = steps_of(r);
            }
            __syncthreads();
            last = upto(n * heads, scan, all);
        }
        __syncthreads();
        return to->at < to->end;
    }
    // For one thread: the next segment, but for share()'s fields.
    __device__ void next(const AttnArgs &a, int cols, AttnSeg &g) {
        g.some = at < end;
        if (!g.some) return;
        if (at == base + steps) {
            base = at;
            if (++kvh == a.c.n_kv_heads) {
                kvh = 0;
                do {
                    r = attn_range(a, ++seq, 0, cols);
                    steps = steps_of(r);
                } while (steps == 0);  // `end` is within the steps of all, so a sequence with some follows
            }
        }
        const int k0 = at - base, k1 = min(steps, k0 + end - at);
        g.r = r;
        g.seq = seq;
        g.kvh = kvh;
        g.ct = 0;
        g.first = r.slab0 + k0 * kStepTiles;
        g.last = min(r.slab0 + r.slabs, r.slab0 + k1 * kStepTiles);
        g.parts = 1;
        g.base = base;
        g.steps = steps;
        g.whole = k0 == 0 && k1 == steps;
        at += k1 - k0;
    }
    // ... and these: who else has parts of the segment's item.
    __device__ void share(AttnSeg &g) const {
        if (!g.whole) {
            const int base = g.base, steps = g.steps;
            // the first and the last CTA that have a step of the item
            int c0 = holder(base), c1 = holder(base + steps - 1);
            while (snapped(cut(c0 + 1), base, steps) <= base) ++c0;
            while (snapped(cut(c1), base, steps) >= base + steps) --c1;
            // a CTA has at most two parts: of the item it starts with, and of the one that it leaves to the next CTA
            g.parts = c1 - c0 + 1;
            g.counter = c0;
            g.part0 = 2 * c0 + 1;
            g.rest = 2 * c0;
            g.part_step = 2;
            g.mine = g.part(static_cast<int>(blockIdx.x) - c0);
        }
    }
};

__device__ __forceinline__ void mma_acc(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void sts128(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint32_t h2_add(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t h2_neg(uint32_t a) {
    uint32_t d;
    asm("neg.f16x2 %0, %1;" : "=r"(d) : "r"(a));
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
// 16 (n - 8) of 3 and 7. `magic` is 1024 in both halves, loaded from shared memory so that it stays in a register: the
// mask is then the one immediate of a three-input logic operation (two constants take two operations).
constexpr uint32_t kCodeMagic = 0x64006400u;
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t magic, uint32_t (&f)[4]) {
    constexpr uint32_t kM1032 = 0xE408E408u, kM1152 = 0xE480E480u;
    const uint32_t w8 = w >> 8;
    f[0] = h2_add((w & 0x000F000Fu) | magic, kM1032);
    f[1] = h2_add((w & 0x00F000F0u) | magic, kM1152);
    f[2] = h2_add((w8 & 0x000F000Fu) | magic, kM1032);
    f[3] = h2_add((w8 & 0x00F000F0u) | magic, kM1152);
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

// Two fp32 operations in one instruction (each half rounded as the scalar one; but a product that an f2_add takes may become one
// fma with it, .rn or not: where that matters, the scalar intrinsics).
__device__ __forceinline__ uint64_t f2(float x, float y) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ float2 f2_parts(uint64_t v) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
    return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t f2_half2(uint32_t w) {
    uint64_t d;
    asm("{\n\t.reg .b16 a, b;\n\t.reg .f32 x, y;\n\t"
        "mov.b32 {a, b}, %1;\n\tcvt.f32.f16 x, a;\n\tcvt.f32.f16 y, b;\n\tmov.b64 %0, {x, y};\n\t}"
        : "=l"(d)
        : "r"(w));
    return d;
}
// hi + lo = x to 22 bits, as two fp16 pairs
__device__ __forceinline__ void split_f2(uint64_t x, uint32_t &hi, uint32_t &lo) {
    const float2 v = f2_parts(x);
    hi = pack_h2(v.x, v.y);
    const float2 r = f2_parts(f2_fma(f2_half2(hi), f2(-1.0f, -1.0f), x));
    lo = pack_h2(r.x, r.y);
}

// The fp32 values of a query row (column `col` of the kv head) that a lane of index t holds: dimensions 8t .. 8t+7 of
// every block; zeros where the column is none.
template <int NB>
__device__ __forceinline__ void load_q(const AttnArgs &a, const AttnRange &r, int kvh, int col, int t, float (&v)[NB][8]) {
    const int i = a.by_group.div(col);
    const bool valid = i < r.n;
    const float *q = a.q + static_cast<int64_t>(r.q0 + (valid ? i : 0)) * a.q_stride +
                     static_cast<int64_t>(kvh * a.group + (valid ? col - i * a.group : 0)) * (NB * kQK) + 8 * t;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (valid) {
            x = *reinterpret_cast<const float4 *>(q + b * kQK);
            y = *reinterpret_cast<const float4 *>(q + b * kQK + 4);
        }
        v[b][0] = x.x; v[b][1] = x.y; v[b][2] = x.z; v[b][3] = x.w;
        v[b][4] = y.x; v[b][5] = y.y; v[b][6] = y.z; v[b][7] = y.w;
    }
}

// 2^e that brings a column's largest magnitude into [2^13, 2^14), with the scale's sign (up), and 2^-e (down).
__device__ __forceinline__ void q_unit(float top, float scale, float &up, float &down) {
    int e = 13 - (static_cast<int>(__float_as_uint(top) >> 23) - 127);
    e = min(100, e);  // -114 at least
    up = __uint_as_float((static_cast<uint32_t>(e + 127) << 23) | (scale < 0.0f ? 0x80000000u : 0u));
    down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}
// Whether a scale of the warp's tokens is 7 or more, so that p times it may be no fp16 number. Bit 14 says 2 or more: the others
// are looked at only then.
template <int NB> __device__ __forceinline__ bool scales_large(const uint32_t (&dv)[4][NB]) {
    uint32_t any = 0;
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int b = 0; b < NB; ++b) any |= dv[h][b];
    if (!__any_sync(0xffffffffu, (any & 0x40004000u) != 0)) return false;
    uint32_t top = 0;
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int b = 0; b < NB; ++b) top = max(top, max(dv[h][b] & 0x7fffu, dv[h][b] >> 16 & 0x7fffu));
    return __any_sync(0xffffffffu, top >= 0x4700u);
}
// Which of a lane's tokens tok, tok + 1, tok + 8, ... of a unit are in low .. end - 1, a bit each.
__device__ __forceinline__ uint32_t seen_tokens(int tok, int low, int end) {
    uint32_t seen = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int a = tok + 8 * (i >> 1) + (i & 1);
        seen |= (a >= low && a < end ? 1u : 0u) << i;
    }
    return seen;
}
// x = p d_v of a unit's tokens (a lane's pairs; the lanes of a column are t = 0 .. 3) in two fp16 parts whose unit is 2^-e for
// the column's largest x: x = down * (hi + lo). V of what the column does not see may be no number, and x is 0 there.
__device__ __forceinline__ void split_x(uint64_t (&x)[4], uint32_t seen, uint32_t (&hi)[4], uint32_t (&lo)[4], float &down) {
    float top = 0.0f, up;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const float2 y = f2_parts(x[h]), v = make_float2((seen >> 2 * h & 1u) ? y.x : 0.0f, (seen >> (2 * h + 1) & 1u) ? y.y : 0.0f);
        x[h] = f2(v.x, v.y);
        top = fmaxf(fmaxf(top, fabsf(v.x)), fabsf(v.y));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    q_unit(top, 1.0f, up, down);
#pragma unroll
    for (int h = 0; h < 4; ++h) split_f2(f2_mul(x[h], f2(up, up)), hi[h], lo[h]);
}

// The copies of a stretch of units (pairs of tiles, a ring slot each): unit first_unit + k * step, k = 0, 1, ...; a warp's
// lanes look up the pages of 16 units at a time, lanes 2j and 2j + 1 copy unit j's tiles.
template <int NB> struct TileFeed {
    const uint8_t *src = nullptr;  // this lane's tile
    bool in = false;               // ... is one of the split's
    __device__ static int page_at(const AttnArgs &a, const int32_t *table, int tile) {
        const int slot = a.by_page_tiles.div(tile);
        return slot < a.c.max_pages ? table[slot] : 0;
    }
    // the same, now: a plain load may be put off to its use, behind the loads that it should run beside
    __device__ static int page_early(const AttnArgs &a, const int32_t *table, int tile) {
        const int slot = min(a.by_page_tiles.div(tile), a.c.max_pages - 1);
        int page;
        asm volatile("ld.global.b32 %0, [%1];" : "=r"(page) : "l"(table + slot));
        return page;
    }
    __device__ void look(const AttnArgs &a, const uint8_t *head, int page, int tile, int last, int *sh_bad) {
        in = tile < last;
        const bool wrong = in && (page < 0 || page >= a.c.n_pages);
        if (wrong) {  // seen by whoever waits for the copy that follows
            *sh_bad = 1;
            if (a.status) *a.status = 1;
        }
        if (wrong || !in) page = 0;
        __syncwarp();
        src = head + page * a.c.page_bytes +
              static_cast<int64_t>(a.by_page_tiles.mod(tile, a.by_page_tiles.div(tile))) * KvGeom<NB>::kTileBytes;
    }
    __device__ void start(const AttnArgs &a, const AttnSeg &s, int tile, int *sh_bad, int early_tile = -1, int early_page = 0) {
        const int32_t *table = a.c.table + static_cast<int64_t>(s.seq) * a.c.max_pages;
        const int page = tile >= s.last ? 0 : (tile == early_tile ? early_page : page_at(a, table, tile));
        look(a, a.c.pages + static_cast<int64_t>(s.kvh) * static_cast<int>(a.by_page_tiles.d) * KvGeom<NB>::kTileBytes, page, tile,
             s.last, sh_bad);
    }
    // unit j of the stretch into `slot`
    __device__ void copy(int j, int lane, uint8_t *slot, uint64_t *full, uint64_t policy) const {
        constexpr uint32_t kBytes = KvGeom<NB>::kTileBytes;
        const uint32_t both = __ballot_sync(0xffffffffu, in) >> (2 * j + 1) & 1u;
        if (lane == 2 * j) mbar_arrive_expect_tx(full, kBytes << both);
        __syncwarp();
        if (lane >> 1 == j && in) bulk_copy_g2s(slot + (lane & 1) * kBytes, src, kBytes, full, policy);
    }
};

// The CTA's end: the warps' sums (already in the unit of their common maximum) added up, and stored as the result or,
// where CTAs share the item, as a part; the CTA that comes last joins the parts, in their
// order: out = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s. `sum`: [warp][WCOLS][D]; m, l: [warp][WCOLS], l in the
// common unit too; TURNED: column c's quads lie exchanged by c & 7.
template <int D, int WCOLS, int WARPS, bool TURNED = false>
__device__ __forceinline__ void attn_store(const AttnArgs &a, const AttnSeg &seg, int cols, int wc, int n_wt, float *sum, const float *m,
                                           const float *l, bool bad, int *sh_last) {
    constexpr int kThreads = WARPS * 32, kQuads = D / 4, kAhead = WARPS > 12 ? 4 : kJoinAhead;  // as registers allow
    const int tid = threadIdx.x;
    const AttnRange &r = seg.r;
    const int ct = seg.ct, kvh = seg.kvh, n_splits = seg.parts;
    const int live = min(cols, r.n * a.group - ct * cols);  // columns that are query rows
    if (r.bad && tid == 0 && a.status) *a.status = 1;
    const auto row = [&](int col) {
        const int i = a.by_group.div(col);
        return a.out + (static_cast<int64_t>(r.q0 + i) * a.n_q_heads + kvh * a.group + (col - i * a.group)) * D;
    };
    for (int k = tid; k < live * kQuads; k += kThreads) {
        const int c = k / kQuads, e = 4 * (k % kQuads);
        const int w0 = c / WCOLS, wcol = c % WCOLS;
        float ls = 0.0f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < n_wt; ++w) {
            const int at = (w * wc + w0) * WCOLS + wcol;
            ls += l[at];
            const float4 x = *reinterpret_cast<const float4 *>(sum + at * D + (TURNED ? e ^ 4 * (c & 7) : e));
            acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
        }
        if (bad) ls = __int_as_float(0x7fffffff);
        if (n_splits == 1) {
            const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
            *reinterpret_cast<float4 *>(row(ct * cols + c) + e) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        } else {
            const int64_t at = static_cast<int64_t>(seg.mine) * cols + c;
            __stcg(reinterpret_cast<float4 *>(a.part + at * D + e), acc);
            if (e == 0) {
                float top = -INFINITY;
                for (int w = 0; w < n_wt; ++w) top = fmaxf(top, m[(w * wc + w0) * WCOLS + wcol]);
                __stcg(&a.part_ml[at], make_float2(top, ls));
            }
        }
    }
    if (n_splits == 1) return;
    __syncthreads();
    if (tid == 0) {
        // releases the CTA's partial sums (which the barrier orders before it), acquires the others'
        uint32_t before;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(a.count + seg.counter) : "memory");
        const bool is_last = before == static_cast<uint32_t>(n_splits) - 1u;
        if (is_last) a.count[seg.counter] = 0;
        *sh_last = is_last;
    }
    __syncthreads();
    if (!*sh_last) return;
    // a thread for four dimensions of a column, kAhead splits' loads in flight; where that leaves threads over, groups of
    // them share the splits
    const int quads = live * kQuads, groups = max(1, kThreads / quads);
    float4 *grp_sum = reinterpret_cast<float4 *>(sum);  // [group][quads], then their maxima and sums of p
    float2 *grp_ml = reinterpret_cast<float2 *>(grp_sum + kThreads);
    for (int k0 = 0; k0 < quads; k0 += kThreads) {
        const int grp = groups > 1 ? tid / quads : 0, k = k0 + tid - grp * quads;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float top = -INFINITY, ls = 0.0f;
        const int c = k / kQuads, e = 4 * (k % kQuads);
        if (k < quads && grp < groups) {
            for (int s0 = grp; s0 < n_splits; s0 += kAhead * groups) {
                float2 ml[kAhead];
                float4 x[kAhead];
                float to = top;
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const int s = s0 + i * groups;
                    const int64_t p = static_cast<int64_t>(seg.part(s)) * cols + c;
                    ml[i] = s < n_splits ? __ldcg(&a.part_ml[p]) : make_float2(-INFINITY, 0.0f);
                    x[i] = s < n_splits ? __ldcg(reinterpret_cast<const float4 *>(a.part + p * D + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int i = 0; i < kAhead; ++i) to = fmaxf(to, ml[i].x);
                const float keep = top == -INFINITY ? 0.0f : exp2_approx(top - to);
                top = to;
                ls *= keep;
                acc.x *= keep; acc.y *= keep; acc.z *= keep; acc.w *= keep;
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const float f = ml[i].x == -INFINITY ? 0.0f : exp2_approx(ml[i].x - top);
                    ls += f * ml[i].y;  // NaN where a split is bad, whatever its weight
                    acc.x += f * x[i].x; acc.y += f * x[i].y; acc.z += f * x[i].z; acc.w += f * x[i].w;
                }
            }
        }
        if (groups > 1) {  // one round
            if (grp < groups) {
                grp_sum[tid] = acc;
                grp_ml[tid] = make_float2(top, ls);
            }
            __syncthreads();
            if (grp != 0) return;
            float to = top;
            for (int q = 1; q < groups; ++q) to = fmaxf(to, grp_ml[q * quads + k].x);
            const float keep = top == -INFINITY ? 0.0f : exp2_approx(top - to);
            ls *= keep;
            acc.x *= keep; acc.y *= keep; acc.z *= keep; acc.w *= keep;
            for (int q = 1; q < groups; ++q) {
                const float2 ml = grp_ml[q * quads + k];
                const float f = ml.x == -INFINITY ? 0.0f : exp2_approx(ml.x - to);
                const float4 x = grp_sum[q * quads + k];
                ls += f * ml.y;
                acc.x += f * x.x; acc.y += f * x.y; acc.z += f * x.z; acc.w += f * x.w;
            }
        }
        if (k < quads) {
            const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
            *reinterpret_cast<float4 *>(row(ct * cols + c) + e) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        }
    }
}

// The narrow form: up to 4 columns, each as two neighbouring columns (upper and lower part) of the MMAs' 8.
//  * Scores: A = 16 tokens' codes, B = q's parts: C holds, per lane (g, t), column t's upper and lower sum for the
//    tokens g and g + 8, so a score is d_k * (c0 + c1) and nothing is computed twice (the wide form with 4 columns
//    spends twice the MMAs, scales and exponentials).
//  * p's parts go to the B fragment of the product with V (tokens x parts) by a transpose of 8 x 8 fp16 pairs
//    (movmatrix): the pairs (0, ph) and (ph, pl), whose rows are then 0 or ph, and ph or pl, so that one formula
//    x = fma(second, d_v, fma(first, d_v, -(first * d_v))) is xh on a row of ph and xl on a row of pl.
//  * The product's C holds column t's two parts side by side again: they are one sum of fp32 pairs.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
constexpr int kNarrowCols = 4;
template <int NB> __global__ void __launch_bounds__(kAttnThreads, attn_ctas_per_sm(NB, 1)) attn_narrow_kernel(AttnArgs a) {
    using G = KvGeom<NB>;
    constexpr int D = G::kDim, kWarps = kAttnWarps;
    constexpr int kSlotBytes = 2 * G::kTileBytes;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float sh_m[kWarps][kNarrowCols], sh_l[kWarps][kNarrowCols];
    __shared__ int sh_bad[2], sh_last, sh_scan[kWarps];
    __shared__ uint32_t sh_magic;
    __shared__ AttnSeg sh_seg[2];
    __shared__ AttnWalk sh_walk;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem) + 2 * warp;  // the warp's two slots
    uint8_t *ring = smem + kAttnBarBytes + 2 * warp * kSlotBytes;
    uint2 *q_sm = reinterpret_cast<uint2 *>(smem + kAttnBarBytes + 2 * kWarps * kSlotBytes) + lane;
    float *sum = reinterpret_cast<float *>(smem + kAttnBarBytes + 2 * kWarps * kSlotBytes + 2 * NB * 256);  // [warp][column][D]
    if (lane == 0) {
        mbar_init(&full[0], 1);
        mbar_init(&full[1], 1);
        fence_barrier_init();
    }
    if (tid == 0) {
        sh_bad[0] = sh_bad[1] = 0;
        sh_magic = kCodeMagic;
    }
    __syncthreads();
    block_op_wait();
    block_op_release();

    const int tile_off = 2 * (warp + (lane >> 1) * kWarps) + (lane & 1);
    int early_tile = -1, early_page = 0;
    const uint64_t policy = l2_evict_first_policy();
    TileFeed<NB> feed;
    int slot = 0;
    uint32_t phases = 0, pending = 0;  // by slot: the parity to wait for, copies not yet waited for
    bool dead = false;
    // the warp's first two units of a segment, on their way
    const auto begin = [&](const AttnSeg &s, int *bad) {
        feed.start(a, s, s.first + tile_off, bad, early_tile, early_page);
        early_tile = -1;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (s.first + 2 * (warp + j * kWarps) < s.last) {
                const int to = slot ^ j;
                fence_proxy_async_smem();
                feed.copy(j, lane, ring + to * kSlotBytes, &full[to], policy);
                pending |= 1u << to;
            }
    };
    const int g = lane >> 2, t = lane & 3;
    // q: column g / 2, this lane's dimensions 8t .. 8t+7 of every block; asked for before the tiles' copies, which it
    // would otherwise wait behind
    float v[NB][8];
    if (a.n_split > 0) {
        // without a window a sequence of the full length has its split's pages here: looked up beside the lengths
        if (a.window == 0) {
            early_tile = blockIdx.y * a.chunk + tile_off;
            const int seq = a.by_heads.div(a.by_ct.div(blockIdx.x));
            early_page = TileFeed<NB>::page_early(a, a.c.table + static_cast<int64_t>(seq) * a.c.max_pages, early_tile);
        }
        AttnSeg seg;
        if (!attn_grid_seg(a, kNarrowCols, seg)) return;
        load_q<NB>(a, seg.r, seg.kvh, g / 2, t, v);
        begin(seg, &sh_bad[0]);
        if (tid == kWalker) {
            sh_seg[0] = seg;
            sh_seg[1].some = false;
        }
        __syncthreads();
    } else {
        if (!AttnWalk::begin(a, kNarrowCols, sh_scan, &sh_walk)) return;
        if (tid == kWalker) sh_walk.next(a, kNarrowCols, sh_seg[0]);
        __syncthreads();
        load_q<NB>(a, sh_seg[0].r, sh_seg[0].kvh, g / 2, t, v);
        begin(sh_seg[0], &sh_bad[0]);
    }
    const uint32_t magic = lds32(smem_addr(&sh_magic));
    const uint32_t pick = (g & 1) ? 0x7632u : 0x5410u;  // the token's half of two words of scales

    for (int n_seg = 0;; ++n_seg) {
    const AttnSeg &seg = sh_seg[n_seg & 1], &ahead = sh_seg[~n_seg & 1];
    const AttnRange &r = seg.r;
    const int first = seg.first, last = seg.last;
    const int n_units = (last - first + 1) / 2;   // pairs of tiles
    // its B fragments, the upper (g even) or lower part
    uint32_t qf[NB][4];
    float qs;
    {
        float top = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(v[b][k]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float up, down;
        q_unit(top, a.scale_log2, up, down);
        qs = __shfl_sync(0xffffffffu, fmaxf(fabsf(a.scale_log2) * down, 1e-37f), 8 * t);  // column t's
#pragma unroll
        for (int k = 0; k < 2 * NB; ++k) {
            if (k % kWarps != warp) continue;
            const int b = k / 2, h = k % 2;
            uint32_t f[4];
            split_h2(v[b][2 * h] * up, v[b][2 * h + 4] * up, f[0], f[1]);
            split_h2(v[b][2 * h + 1] * up * 0.0625f, v[b][2 * h + 5] * up * 0.0625f, f[2], f[3]);
            q_sm[k * 32] = (g & 1) ? make_uint2(f[1], f[3]) : make_uint2(f[0], f[2]);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2 * NB; ++k) {
            const uint2 f = q_sm[k * 32];
            qf[k / 2][2 * (k % 2)] = f.x;
            qf[k / 2][2 * (k % 2) + 1] = f.y;
        }
    }
    if (tid == kWalker && a.n_split == 0) {
        sh_walk.share(sh_seg[n_seg & 1]);
        sh_walk.next(a, kNarrowCols, sh_seg[~n_seg & 1]);
    }
    __syncwarp();
    // what column t sees, of this split's tiles
    const int limit = min(r.len, last * kKvSlab);
    const int ti = a.by_group.div(t);
    const int end = ti < r.n ? min(limit, max(0, r.len - (r.n - 1 - ti))) : limit;
    const int low = ti < r.n && a.window > 0 ? max(0, r.len - (r.n - 1 - ti) - a.window) : 0;
    const int end_min = __reduce_min_sync(0xffffffffu, end), low_max = __reduce_max_sync(0xffffffffu, low);

    float m = -INFINITY, l = 0.0f;
    bool huge = false;
    uint64_t o[2 * NB];  // column t, dimensions 4g and 4g + 1, or 4g + 2 and 4g + 3, of the block
#pragma unroll
    for (int k = 0; k < 2 * NB; ++k) o[k] = 0;

    for (int u = warp, j_next = 2; u < n_units && !dead; u += kWarps) {
        if (!__all_sync(0xffffffffu, mbar_wait(&full[slot], phases >> slot & 1u))) {
            if (lane == 0) atomicOr(a.fault, 1u);
            dead = true;
            break;
        }
        phases ^= 1u << slot;
        pending &= ~(1u << slot);
        const uint32_t tile = smem_addr(ring) + slot * kSlotBytes;
        const int t0 = (first + 2 * u) * kKvSlab;
        // ------------------------------------------------ scores of column t: tokens 8h + g
        float sc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            uint32_t kw[2][NB], dk[2][NB];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                lds_words<NB, G::kVec>(tile + s * G::kTileBytes + (h * NB * 32 + lane * G::kVec) * 4, 128 * G::kVec, kw[h]);
                lds_words<NB, G::kVec>(tile + s * G::kTileBytes + G::kKScaleAt + (g / 2 + 4 * h) * NB * 4, 4 * G::kVec, dk[h]);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint32_t k0[4], k1[4];
                code_pairs(kw[0][b], magic, k0);
                code_pairs(kw[1][b], magic, k1);
                const uint32_t a0[4] = {k0[0], k1[0], k0[1], k1[1]}, a1[4] = {k0[2], k1[2], k0[3], k1[3]};
                float c[4];
                mma_first(c, a0, qf[b][0], qf[b][1]);
                mma_acc(c, a1, qf[b][2], qf[b][3]);
                const uint64_t d = f2_half2(__byte_perm(dk[0][b], dk[1][b], pick));  // tokens g, g + 8
                const float2 dd = f2_parts(d);
                sc[2 * s] = fmaf(dd.x, c[0] + c[1], sc[2 * s]);
                sc[2 * s + 1] = fmaf(dd.y, c[2] + c[3], sc[2 * s + 1]);
            }
        }
        uint32_t dv[4][NB];
#pragma unroll
        for (int h = 0; h < 4; ++h)
            lds_words<NB, G::kVec>(tile + (h >> 1) * G::kTileBytes + G::kVScaleAt + (t + 4 * (h & 1)) * NB * 4, 4 * G::kVec, dv[h]);
        if (t0 + 2 * kKvSlab > end_min || t0 < low_max) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int tok = t0 + 8 * h + g;
                if (tok < low || tok >= end) sc[h] = -INFINITY;
                // a token past the sequence's (or a stale half slot) may hold anything, NaN among it: its V
                // counts for nothing
                const int pair = t0 + 8 * h + 2 * t;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if (pair >= limit) dv[h][b] = 0;
                    else if (pair + 1 >= limit) dv[h][b] &= 0xffffu;
                }
            }
        }
        const bool large = scales_large(dv);
        // ------------------------------------------------ softmax
        float top = fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        top *= qs;
        if (__any_sync(0xffffffffu, top > m)) {
            const float to = fmaxf(m, top);
            const float keep = to > m ? exp2_approx(m - to) : 1.0f;  // 0 where nothing was seen before
            m = to;
            l *= keep;
#pragma unroll
            for (int k = 0; k < 2 * NB; ++k) o[k] = f2_mul(o[k], f2(keep, keep));
            huge = __any_sync(0xffffffffu, score_huge(m, kHugeScore));
        }
        float base = m == -INFINITY ? 0.0f : m - kAttnUnit, unit = qs;
        if (huge) {
#pragma unroll
            for (int h = 0; h < 4; ++h) sc[h] = __fadd_rn(__fmul_rn(sc[h], qs), m == -INFINITY ? 0.0f : -m);
            base = -kAttnUnit;
            unit = 1.0f;
        }
        uint32_t p0[4], p1[4];  // rows 0 or ph, and ph or pl, of tokens 8h + 2t, + 1
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const float p = exp2_approx(fmaf(sc[h], unit, -base));
            l += p;
            const uint32_t w = pack_h2(0.0f, p);
            p0[h] = transpose_8x8(w);
            p1[h] = transpose_8x8(pack_h2(p, p - f2_parts(f2_half2(w)).y));
        }
        // ------------------------------------------------ product with V
        uint32_t vw[4][NB];
#pragma unroll
        for (int h = 0; h < 4; ++h)
            lds_words<NB, G::kVec>(tile + (h >> 1) * G::kTileBytes + G::kVAt + ((h & 1) * NB * 32 + lane * G::kVec) * 4,
                                   128 * G::kVec, vw[h]);
        const auto product = [&](auto wide_range) {
            uint32_t seen = 0;  // by column g / 2
            if constexpr (decltype(wide_range)::value)
                seen = seen_tokens(t0 + 2 * t, __shfl_sync(0xffffffffu, low, g >> 1), __shfl_sync(0xffffffffu, end, g >> 1));
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                uint32_t f[2][2][4], x[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t vc[4];
                    code_pairs(vw[h][j], magic, vc);
                    f[h >> 1][0][2 * (h & 1)] = vc[0]; f[h >> 1][0][2 * (h & 1) + 1] = vc[1];
                    f[h >> 1][1][2 * (h & 1)] = vc[2]; f[h >> 1][1][2 * (h & 1) + 1] = vc[3];
                }
                float down = 1.0f;
                if constexpr (decltype(wide_range)::value) {
                    // the rows of pl have p itself; those of ph get x's upper part from them
                    uint64_t px[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) px[h] = f2_mul(f2_add(f2_half2(p0[h]), f2_half2(p1[h])), f2_half2(dv[h][j]));
                    uint32_t lo[4];
                    split_x(px, seen, x, lo, down);
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const uint32_t hi = __shfl_xor_sync(0xffffffffu, x[h], 4);
                        x[h] = (g & 1) ? lo[h] : hi;
                    }
                    down = __shfl_sync(0xffffffffu, down, 8 * t + 4);
                } else {
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        x[h] = h2_fma(p1[h], dv[h][j], h2_fma(p0[h], dv[h][j], h2_neg(h2_mul(p0[h], dv[h][j]))));
                }
                // summed over the unit by the tensor cores (they truncate), over the units in fp32
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float c[4];
                    mma_first(c, f[0][i], x[0], x[1]);
                    mma_acc(c, f[1][i], x[2], x[3]);
                    const uint64_t y = f2(c[0] + c[1], c[2] + c[3]);
                    if constexpr (decltype(wide_range)::value) o[2 * j + i] = f2_fma(y, f2(down, down), o[2 * j + i]);
                    else o[2 * j + i] = f2_add(o[2 * j + i], y);
                }
            }
        };
        if (large) product(std::true_type{});
        else product(std::false_type{});
        __syncwarp();
        if (u + 2 * kWarps < n_units) {  // the warp's unit after next takes the slot's place
            if (j_next == 16) {
                j_next = 0;
                feed.start(a, seg, first + 2 * (u - warp + 2 * kWarps) + tile_off, &sh_bad[n_seg & 1]);
            }
            fence_proxy_async_smem();
            feed.copy(j_next++, lane, ring + slot * kSlotBytes, &full[slot], policy);
            pending |= 1u << slot;
        }
        slot ^= 1;
    }
    // ------------------------------------------------ join the warps
    l += __shfl_xor_sync(0xffffffffu, l, 4);
    l += __shfl_xor_sync(0xffffffffu, l, 8);
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    if (g == 0) sh_m[warp][t] = m;
    __syncthreads();
    // the next segment's first tiles come while this one's sums are joined
    if (ahead.some && !dead) begin(ahead, &sh_bad[(n_seg + 1) & 1]);
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh_m[w][t]);
    const float f0 = top == -INFINITY ? 0.0f : exp2_approx(m - top), f1 = f0 * 0.0625f;
    if (g == 0) sh_l[warp][t] = dead ? __int_as_float(0x7fffffff) : l * f0;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const float2 x = f2_parts(o[2 * j]), y = f2_parts(o[2 * j + 1]);
        // the second of each pair is 16 times too large
        *reinterpret_cast<float4 *>(sum + (warp * kNarrowCols + t) * D + 4 * g + j * kQK) =
            make_float4(x.x * f0, x.y * f1, y.x * f0, y.y * f1);
    }
    __syncthreads();
    attn_store<D, kNarrowCols, kWarps>(a, seg, kNarrowCols, 1, kWarps, sum, &sh_m[0][0], &sh_l[0][0], r.bad || sh_bad[n_seg & 1], &sh_last);
    if (!ahead.some) break;
    load_q<NB>(a, ahead.r, ahead.kvh, g / 2, t, v);
    __syncthreads();  // the sums are read
    if (tid == 0) sh_bad[n_seg & 1] = 0;
    }
    // leave only when the warp's copies have landed (after a wait that gave up: as far as they will)
    for (int k = 0; k < 2; ++k)
        if (pending >> k & 1u) (void)mbar_wait(&full[k], phases >> k & 1u);
}

// The wide form: each warp 8 * NT columns. With a shared ring the warps split the columns (a.wc of them; the others the
// ring's slots), and warp 0 feeds it half a ring ahead of itself. The prompt form (all warps of a CTA split the columns, as
// evenly as the fewest column tiles allow): every unit's codes become fp16 fragments in shared memory once, an eighth by each
// warp, a unit ahead of their use (one barrier a unit; converting in every warp costs 144 of its 480 instructions a tile). Two
// warps a scheduler (the output's and the products' registers allow no more) wait for each other's products (8 cycles an
// m16n8k16, 22 one that needs the one before): with heads of 128 they kept the tensor cores 40% busy, and q's fragments in
// registers, a product's sums put off behind the next block's products or warps that drift apart gained nothing. Heads of up
// to 128 dimensions have a form of their own (zdmmv_attn_prompt.cuh).
template <int NB, int NT, int FORM>
__global__ void __launch_bounds__(kAttnWarps * 32, FORM != kOwn ? 1 : attn_ctas_per_sm(NB, NT)) attn_kernel(AttnArgs a) {
    constexpr bool SHARED = FORM != kOwn, PROMPT = FORM == kPrompt;
    using G = KvGeom<NB>;
    constexpr int kWarps = kAttnWarps, kSlots = attn_slots(NB, FORM);
    constexpr int D = G::kDim;
    constexpr int kSlotBytes = 2 * G::kTileBytes;
    constexpr bool kApart = attn_sums_apart(NB, NT, FORM);
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float sh_m[kWarps][NT * 8], sh_l[kWarps][NT * 8], sh_qs[kWarps][NT * 8];
    __shared__ int sh_bad[2], sh_last, sh_scan[kWarps];
    __shared__ uint32_t sh_magic;
    __shared__ AttnSeg sh_seg[2];
    __shared__ AttnWalk sh_walk;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem);
    uint64_t *empty = full + kSlots;
    uint8_t *ring = smem + kAttnBarBytes;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cols = 8 * NT * a.wc;  // columns of the CTA
    if (tid == 0) {
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], a.wc);
        }
        sh_bad[0] = sh_bad[1] = 0;
        sh_magic = kCodeMagic;
        fence_barrier_init();
    }
    __syncthreads();
    block_op_wait();
    block_op_release();

    const int tile_off = SHARED ? lane : 2 * (warp + (lane >> 1) * kWarps) + (lane & 1);
    int early_tile = -1, early_page = 0;
    if (SHARED || a.n_split > 0) {
        AttnSeg seg;
        if (a.window == 0) {
            early_tile = blockIdx.y * a.chunk + tile_off;
            const int seq = a.by_heads.div(a.by_ct.div(blockIdx.x));
            early_page = TileFeed<NB>::page_early(a, a.c.table + static_cast<int64_t>(seq) * a.c.max_pages, early_tile);
        }
        if (!attn_grid_seg(a, cols, seg)) return;
        if (tid == kWarps * 32 - 1) {
            sh_seg[0] = seg;
            sh_seg[1].some = false;
        }
    } else {
        if (!AttnWalk::begin(a, cols, sh_scan, &sh_walk)) return;
        if (tid == kWarps * 32 - 1) sh_walk.next(a, cols, sh_seg[0]);
    }
    __syncthreads();
    const uint64_t policy = l2_evict_first_policy();
    TileFeed<NB> feed;
    int slot = SHARED ? warp / a.wc : warp;
    uint32_t phases = 0, pending = 0;  // by slot: the parity to wait for, own copies not yet waited for
    bool dead = false;
    // the first units of a segment on their way: the warp's two, or all that the shared ring takes
    const auto begin = [&](const AttnSeg &s, int *bad) {
        if constexpr (SHARED) {
            if (warp != 0) return;
            feed.start(a, s, s.first + tile_off, bad, early_tile, early_page);
            for (int k = 0; k < kSlots && s.first + 2 * k < s.last; ++k) feed.copy(k, lane, ring + k * kSlotBytes, &full[k], policy);
        } else {
            feed.start(a, s, s.first + tile_off, bad, early_tile, early_page);
            early_tile = -1;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (s.first + 2 * (warp + k * kWarps) < s.last) {
                    const int to = slot ^ (k * kWarps);
                    fence_proxy_async_smem();
                    feed.copy(k, lane, ring + to * kSlotBytes, &full[to], policy);
                    pending |= 1u << to;
                }
        }
    };
    const int g = lane >> 2, t = lane & 3;
    const int wc = PROMPT ? warp : warp % a.wc, wt = PROMPT ? 0 : warp / a.wc, n_wt = PROMPT ? 1 : kWarps / a.wc;
    uint4 *q_sm = reinterpret_cast<uint4 *>(ring + kSlots * kSlotBytes) + wc * (NT * 2 * NB * 32) + lane;
    // the warps' sums [warp][column of the warp][D], behind q's fragments or over the ring
    float *sum = reinterpret_cast<float *>(kApart ? ring + kSlots * kSlotBytes + NT * 2 * NB * 512 : ring);
    const uint32_t magic = lds32(smem_addr(&sh_magic));
    const uint32_t q_at = smem_addr(q_sm);
    // PROMPT: the fragments of two units, [octet][block][lane] of K, then [tile][block][half][lane] of V
    constexpr uint32_t kFragV = 4 * NB * 512, kFragBytes = 8 * NB * 512;
    const uint32_t frag0 = smem_addr(ring) + kSlots * kSlotBytes + a.wc * (NT * 2 * NB * 512);
    const auto convert = [&](uint32_t tile, uint32_t to) {
        const auto word = [&](int s, int at, int plane, int b) {
            return lds32(tile + s * G::kTileBytes + at + (((plane * (NB / G::kVec) + b / G::kVec) * 32 + lane) * G::kVec + b % G::kVec) * 4);
        };
        for (int k = warp; k < 4 * NB; k += kWarps) {
            const int h = k / NB, b = k % NB;
            uint32_t c[4];
            code_pairs(word(h >> 1, 0, h & 1, b), magic, c);
            sts128(to + k * 512 + lane * 16, c[0], c[1], c[2], c[3]);
        }
        for (int k = warp; k < 2 * NB; k += kWarps) {
            const int s = k / NB, j = k % NB;
            uint32_t c[4], d[4];
            code_pairs(word(s, G::kVAt, 0, j), magic, c);
            code_pairs(word(s, G::kVAt, 1, j), magic, d);
            sts128(to + kFragV + 2 * k * 512 + lane * 16, c[0], c[1], d[0], d[1]);
            sts128(to + kFragV + (2 * k + 1) * 512 + lane * 16, c[2], c[3], d[2], d[3]);
        }
    };
    const auto wait_full = [&](int s) {  // PROMPT: a wait that gave up ends no loop, so that every barrier is met
        if (!dead && !__all_sync(0xffffffffu, mbar_wait(&full[s], phases >> s & 1u))) {
            if (lane == 0) atomicOr(a.fault, 1u);
            dead = true;
        }
        phases ^= 1u << s;
    };
    if (!SHARED) begin(sh_seg[0], &sh_bad[0]);

    for (int n_seg = 0;; ++n_seg) {
    const AttnSeg &seg = sh_seg[n_seg & 1], &ahead = sh_seg[~n_seg & 1];
    const AttnRange &r = seg.r;
    const int first = seg.first, last = seg.last;
    const int n_units = (last - first + 1) / 2;   // pairs of tiles, a ring slot each
    const int col0 = seg.ct * cols + wc * 8 * NT;  // the warp's first column
    const bool idle = PROMPT && (warp >= a.wc || col0 >= r.n * a.group);  // no columns: the warp converts, and that is all
    // q's fragments: column g of each group of 8, this lane's 8 dimensions 8t.. of every block
#pragma unroll 1
    for (int nt = wt; nt < NT && !idle; nt += n_wt) {
        float v[NB][8];
        load_q<NB>(a, r, seg.kvh, col0 + 8 * nt + g, t, v);
        float top = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(v[b][k]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float up, down;
        q_unit(top, a.scale_log2, up, down);
        if (t == 0) sh_qs[wc][8 * nt + g] = fmaxf(fabsf(a.scale_log2) * down, 1e-37f);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // k slots: the codes at bits 0 and 16 of the (shifted) word, then those at bits 4 and 20
                uint4 f;
                split_h2(v[b][2 * h] * up, v[b][2 * h + 4] * up, f.x, f.y);
                split_h2(v[b][2 * h + 1] * up * 0.0625f, v[b][2 * h + 5] * up * 0.0625f, f.z, f.w);
                q_sm[(nt * 2 * NB + 2 * b + h) * 32] = f;
            }
        }
    }
    if (SHARED) begin(seg, &sh_bad[0]);
    // what each column sees, of this split's tiles
    int end[NT], low[NT];
    const int limit = min(r.len, last * kKvSlab);
    int end_min = limit, low_max = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int i = a.by_group.div(col0 + 8 * nt + g);
        const bool valid = i < r.n;
        end[nt] = valid ? min(limit, max(0, r.len - (r.n - 1 - i))) : limit;
        low[nt] = valid && a.window > 0 ? max(0, r.len - (r.n - 1 - i) - a.window) : 0;
        end_min = min(end_min, end[nt]);
        low_max = max(low_max, low[nt]);
    }
    // units outside low_max .. end_min need masks (warp-uniform)
    end_min = __reduce_min_sync(0xffffffffu, end_min);
    low_max = __reduce_max_sync(0xffffffffu, low_max);
    __syncthreads();

    if (!SHARED && tid == kWarps * 32 - 1 && a.n_split == 0) {
        sh_walk.share(sh_seg[n_seg & 1]);
        sh_walk.next(a, cols, sh_seg[~n_seg & 1]);
    }
    __syncwarp();

    float m[NT], l[NT], qs[NT];
    bool huge = false;
    uint64_t o[NT][2 * NB][2];  // columns 2t, 2t+1: dimension pairs' first and second
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt] = -INFINITY;
        l[nt] = 0.0f;
        qs[nt] = sh_qs[wc][8 * nt + g];
#pragma unroll
        for (int k = 0; k < 2 * NB; ++k) o[nt][k][0] = o[nt][k][1] = 0;
    }

    if (PROMPT && n_units > 0) {
        wait_full(0);
        convert(smem_addr(ring), frag0);
        __syncthreads();
    }

    int fed = kSlots;  // SHARED: units that warp 0 has asked for
    for (int u = wt, j_next = 2; u < n_units && (PROMPT || !dead); u += n_wt) {
        if (PROMPT) {
            const int s = (u + 1) % kSlots;
            if (u + 1 < n_units) {
                wait_full(s);
                convert(smem_addr(ring) + s * kSlotBytes, frag0 + (~u & 1) * kFragBytes);
            }
        }
        const uint32_t frag = frag0 + (u & 1) * kFragBytes + lane * 16;
        if (!idle) {
        if (SHARED && !PROMPT && warp == 0) {
            for (; fed < n_units && fed <= u + kSlots / 2; ++fed) {
                const int s = fed % kSlots;
                // unit fed - kSlots, before u: every warp that needs it has it, so this ends
                if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], static_cast<uint32_t>(fed / kSlots - 1) & 1u))) {
                    if (lane == 0) atomicOr(a.fault, 1u);
                    dead = true;
                    break;
                }
                if (fed % 16 == 0) feed.start(a, seg, first + 2 * fed + tile_off, &sh_bad[0]);
                fence_proxy_async_smem();
                feed.copy(fed % 16, lane, ring + s * kSlotBytes, &full[s], policy);
            }
        }
        if constexpr (!PROMPT) {
            if (!__all_sync(0xffffffffu, mbar_wait(&full[slot], phases >> slot & 1u))) {
                if (lane == 0) atomicOr(a.fault, 1u);
                dead = true;
                break;
            }
            phases ^= 1u << slot;
            pending &= ~(1u << slot);
        }
        const uint32_t tile = smem_addr(ring) + slot * kSlotBytes;
        const int t0 = (first + 2 * u) * kKvSlab;
        // ------------------------------------------------ scores: column g, tokens 8h + 2t, 8h + 2t + 1
        uint64_t acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 4; ++h) acc[nt][h] = 0;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            uint32_t kw[2][NB], dk[2][NB];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (!PROMPT)
                    lds_words<NB, G::kVec>(tile + s * G::kTileBytes + (h * NB * 32 + lane * G::kVec) * 4, 128 * G::kVec, kw[h]);
                lds_words<NB, G::kVec>(tile + s * G::kTileBytes + G::kKScaleAt + (t + 4 * h) * NB * 4, 4 * G::kVec, dk[h]);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint32_t qa[NT][2][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint4 f = lds128(q_at + (nt * 2 * NB + 2 * b + k) * 512);
                        qa[nt][k][0] = f.x; qa[nt][k][1] = f.y; qa[nt][k][2] = f.z; qa[nt][k][3] = f.w;
                    }
                float c[2][NT][4];
                uint32_t kc[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (PROMPT) {
                        const uint4 f = lds128(frag + ((2 * s + h) * NB + b) * 512);
                        kc[h][0] = f.x; kc[h][1] = f.y; kc[h][2] = f.z; kc[h][3] = f.w;
                    } else {
                        code_pairs(kw[h][b], magic, kc[h]);
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_first(c[h][nt], qa[nt][0], kc[h][0], kc[h][1]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_acc(c[h][nt], qa[nt][1], kc[h][2], kc[h][3]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint64_t d = f2_half2(dk[h][b]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        acc[nt][2 * s + h] = f2_fma(d, f2_add(f2(c[h][nt][0], c[h][nt][1]), f2(c[h][nt][2], c[h][nt][3])), acc[nt][2 * s + h]);
                }
            }
        }
        uint32_t dv[4][NB];
#pragma unroll
        for (int h = 0; h < 4; ++h)
            lds_words<NB, G::kVec>(tile + (h >> 1) * G::kTileBytes + G::kVScaleAt + (t + 4 * (h & 1)) * NB * 4, 4 * G::kVec, dv[h]);
        float sc[NT][8];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const float2 v = f2_parts(acc[nt][h]);
                sc[nt][2 * h] = v.x;
                sc[nt][2 * h + 1] = v.y;
            }
        if (t0 + 2 * kKvSlab > end_min || t0 < low_max) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int tok = t0 + 2 * t + (i & 1) + 8 * (i >> 1);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    if (tok < low[nt] || tok >= end[nt]) sc[nt][i] = -INFINITY;
                // a token past the sequence's (or a stale half slot) may hold anything, NaN among it: its V
                // counts for nothing
                if (tok >= limit) {
#pragma unroll
                    for (int b = 0; b < NB; ++b) dv[i >> 1][b] &= (i & 1) ? 0x0000ffffu : 0xffff0000u;
                }
            }
        }
        const bool large = scales_large(dv);
        // ------------------------------------------------ softmax
        bool grow = false;
        float top[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float x = sc[nt][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) x = fmaxf(x, sc[nt][i]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            top[nt] = x * qs[nt];
            grow |= top[nt] > m[nt];
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float to = fmaxf(m[nt], top[nt]);
                const float keep = to > m[nt] ? exp2_approx(m[nt] - to) : 1.0f;  // 0 where nothing was seen before
                m[nt] = to;
                l[nt] *= keep;
                const uint64_t k01 = f2(__shfl_sync(0xffffffffu, keep, 8 * t), __shfl_sync(0xffffffffu, keep, 8 * t + 4));
#pragma unroll
                for (int j = 0; j < 2 * NB; ++j) {
                    o[nt][j][0] = f2_mul(o[nt][j][0], k01);
                    o[nt][j][1] = f2_mul(o[nt][j][1], k01);
                }
            }
            bool any = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) any |= score_huge(m[nt], kHugeScore);
            huge = __any_sync(0xffffffffu, any);
        }
        uint32_t ph[NT][4], pl[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float base = m[nt] == -INFINITY ? 0.0f : m[nt] - kAttnUnit, unit = qs[nt];
            if (huge) {
#pragma unroll
                for (int i = 0; i < 8; ++i) sc[nt][i] = __fadd_rn(__fmul_rn(sc[nt][i], unit), m[nt] == -INFINITY ? 0.0f : -m[nt]);
                base = -kAttnUnit;
                unit = 1.0f;
            }
            float e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = exp2_approx(fmaf(sc[nt][i], unit, -base));
            l[nt] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
#pragma unroll
            for (int h = 0; h < 4; ++h) split_f2(f2(e[2 * h], e[2 * h + 1]), ph[nt][h], pl[nt][h]);
        }
        // ------------------------------------------------ product with V
        uint32_t vw[4][NB];
        if constexpr (!PROMPT) {
#pragma unroll
            for (int h = 0; h < 4; ++h)
                lds_words<NB, G::kVec>(tile + (h >> 1) * G::kTileBytes + G::kVAt + ((h & 1) * NB * 32 + lane * G::kVec) * 4,
                                       128 * G::kVec, vw[h]);
        }
        const auto product = [&](auto wide_range) {
            uint32_t seen[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) seen[nt] = decltype(wide_range)::value ? seen_tokens(t0 + 2 * t, low[nt], end[nt]) : 0;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            uint32_t f[2][2][4];  // [tile][dimensions 4g, 4g+1 / 4g+2, 4g+3 of the block]
            if constexpr (PROMPT) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 x = lds128(frag + kFragV + (2 * ((k >> 1) * NB + j) + (k & 1)) * 512);
                    f[k >> 1][k & 1][0] = x.x; f[k >> 1][k & 1][1] = x.y; f[k >> 1][k & 1][2] = x.z; f[k >> 1][k & 1][3] = x.w;
                }
            } else {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t vc[4];
                    code_pairs(vw[h][j], magic, vc);
                    f[h >> 1][0][2 * (h & 1)] = vc[0]; f[h >> 1][0][2 * (h & 1) + 1] = vc[1];
                    f[h >> 1][1][2 * (h & 1)] = vc[2]; f[h >> 1][1][2 * (h & 1) + 1] = vc[3];
                }
            }
            uint32_t hi[NT][4], lo[NT][4];
            float down[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if constexpr (decltype(wide_range)::value) {
                    uint64_t px[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) px[h] = f2_mul(f2_add(f2_half2(ph[nt][h]), f2_half2(pl[nt][h])), f2_half2(dv[h][j]));
                    split_x(px, seen[nt], hi[nt], lo[nt], down[nt]);
                } else {
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        hi[nt][h] = h2_mul(ph[nt][h], dv[h][j]);
                        lo[nt][h] = h2_fma(pl[nt][h], dv[h][j], h2_fma(ph[nt][h], dv[h][j], h2_neg(hi[nt][h])));
                    }
                }
            }
            // summed over the unit by the tensor cores (they truncate), over the units in fp32
            float c[NT][2][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int s = 0; s < 2; ++s) mma_first(c[nt][s], f[0][s], lo[nt][0], lo[nt][1]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int s = 0; s < 2; ++s) mma_acc(c[nt][s], f[1][s], lo[nt][2], lo[nt][3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int s = 0; s < 2; ++s) mma_acc(c[nt][s], f[0][s], hi[nt][0], hi[nt][1]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int s = 0; s < 2; ++s) mma_acc(c[nt][s], f[1][s], hi[nt][2], hi[nt][3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint64_t unit = 0;
                if constexpr (decltype(wide_range)::value)
                    unit = f2(__shfl_sync(0xffffffffu, down[nt], 8 * t), __shfl_sync(0xffffffffu, down[nt], 8 * t + 4));
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint64_t &to = o[nt][2 * j + s][i];
                        const uint64_t y = f2(c[nt][s][2 * i], c[nt][s][2 * i + 1]);
                        if constexpr (decltype(wide_range)::value) to = f2_fma(y, unit, to);
                        else to = f2_add(to, y);
                    }
            }
        }
        };
        if (large) product(std::true_type{});
        else product(std::false_type{});
        }
        __syncwarp();
        if constexpr (PROMPT) {
            __syncthreads();  // the unit's slot and fragments are free, the next one's fragments are there
            if (warp == 0 && u + kSlots < n_units && !dead) {
                if ((u + kSlots) % 16 == 0) feed.start(a, seg, first + 2 * (u + kSlots) + tile_off, &sh_bad[0]);
                fence_proxy_async_smem();
                feed.copy((u + kSlots) % 16, lane, ring + slot * kSlotBytes, &full[slot], policy);
                fed = u + kSlots + 1;
            }
            if (++slot == kSlots) slot = 0;
        } else if constexpr (SHARED) {
            if (lane == 0) mbar_arrive(&empty[slot]);
            slot += n_wt;
            if (slot >= kSlots) slot -= kSlots;
        } else {
            if (u + 2 * kWarps < n_units) {  // the warp's unit after next takes the slot's place
                if (j_next == 16) {
                    j_next = 0;
                    feed.start(a, seg, first + 2 * (u - warp + 2 * kWarps) + tile_off, &sh_bad[n_seg & 1]);
                }
                fence_proxy_async_smem();
                feed.copy(j_next++, lane, ring + slot * kSlotBytes, &full[slot], policy);
                pending |= 1u << slot;
            }
            slot ^= kWarps;
        }
    }
    if (SHARED && dead && warp == 0) {
        // leave only when the copies have landed, as far as they will
        for (int k = max(0, min(fed, n_units) - kSlots); k < min(fed, n_units); ++k)
            (void)mbar_wait(&full[k % kSlots], static_cast<uint32_t>(k / kSlots) & 1u);
    }

    // ------------------------------------------------ join the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        l[nt] += __shfl_xor_sync(0xffffffffu, l[nt], 1);
        l[nt] += __shfl_xor_sync(0xffffffffu, l[nt], 2);
        if (t == 0) sh_m[warp][8 * nt + g] = m[nt];
    }
    __syncthreads();  // every warp is done with the ring
    // the next segment's first tiles come while this one's sums are joined, where these lie apart from the ring
    if (!SHARED && kApart && ahead.some && !dead) begin(ahead, &sh_bad[(n_seg + 1) & 1]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        // this warp's sums in the unit of the warps' common maximum: the lane's column g, columns 2t and 2t + 1 of o
        float top = -INFINITY;
        for (int w = 0; w < n_wt; ++w) top = fmaxf(top, sh_m[w * a.wc + wc][8 * nt + g]);
        const float fg = top == -INFINITY ? 0.0f : exp2_approx(m[nt] - top);
        if (t == 0) sh_l[warp][8 * nt + g] = dead ? __int_as_float(0x7fffffff) : l[nt] * fg;
        const float f[2] = {__shfl_sync(0xffffffffu, fg, 8 * t), __shfl_sync(0xffffffffu, fg, 8 * t + 4)};
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const float2 x0 = f2_parts(o[nt][2 * j][0]), x1 = f2_parts(o[nt][2 * j][1]);
            const float2 x2 = f2_parts(o[nt][2 * j + 1][0]), x3 = f2_parts(o[nt][2 * j + 1][1]);
            float *dst = sum + (warp * NT * 8 + 8 * nt + 2 * t) * D + 4 * g + j * kQK;
            const float s0 = f[0] * 0.0625f, s1 = f[1] * 0.0625f;  // the second of each pair is 16 times too large
            *reinterpret_cast<float4 *>(dst) = make_float4(x0.x * f[0], x1.x * s0, x2.x * f[0], x3.x * s0);
            *reinterpret_cast<float4 *>(dst + D) = make_float4(x0.y * f[1], x1.y * s1, x2.y * f[1], x3.y * s1);
        }
    }
    __syncthreads();
    attn_store<D, 8 * NT, kWarps>(a, seg, cols, a.wc, n_wt, sum, &sh_m[0][0], &sh_l[0][0], r.bad || sh_bad[n_seg & 1], &sh_last);
    if (!ahead.some) break;
    __syncthreads();  // the sums and q's fragments are read
    if (tid == 0) sh_bad[n_seg & 1] = 0;
    if (!kApart && !dead) begin(ahead, &sh_bad[(n_seg + 1) & 1]);
    }
    // leave only when the warp's copies have landed (after a wait that gave up: as far as they will)
    for (uint32_t left = pending; left != 0; left &= left - 1) {
        const int k = __ffs(left) - 1;
        (void)mbar_wait(&full[k], phases >> k & 1u);
    }
}

// ------------------------------------------------------------------ host side
struct AttnPlan {
    int nt, wc;           // column groups of 8 a warp, warps that split the columns
    bool tall;            // the form on tcgen05
    int n_ct, cols;       // column tiles, columns of a tile
    int64_t items;        // kv heads of sequences x column tiles
    int chunk, n_split;   // the grid's form: tiles of a split, most splits; else 0
    int ctas;             // ... CTAs of the grid
    int round;            // ... and what these are a multiple of
    int64_t parts;        // parts that the workspace holds
};

template <int NB> cudaError_t launch_attn(AttnArgs a, const AttnPlan &p, cudaStream_t st);
template <int NB> cudaError_t launch_attn_tall(const AttnArgs &a, const AttnPlan &p, cudaStream_t st);  // NB <= kTallBlocks
extern template cudaError_t launch_attn<2>(AttnArgs, const AttnPlan &, cudaStream_t);
extern template cudaError_t launch_attn<3>(AttnArgs, const AttnPlan &, cudaStream_t);
extern template cudaError_t launch_attn<4>(AttnArgs, const AttnPlan &, cudaStream_t);
extern template cudaError_t launch_attn<6>(AttnArgs, const AttnPlan &, cudaStream_t);
extern template cudaError_t launch_attn<8>(AttnArgs, const AttnPlan &, cudaStream_t);

#ifdef ZDMMV_ATTN_INSTANTIATE
template <auto KERNEL> cudaError_t launch_attn_kernel(const AttnPlan &p, size_t smem, const AttnArgs &a, cudaStream_t st) {
    const cudaError_t e = smem_limit_raised<KERNEL>();
    if (e != cudaSuccess) return e;
    const dim3 grid = p.n_split > 0 ? dim3(static_cast<unsigned>(p.items), p.n_split) : dim3(p.ctas);
    return launch_block_op(KERNEL, grid, dim3(kAttnThreads), kAttnBarBytes + smem, st, a);
}
template <int NB, int NT, int FORM> cudaError_t launch_attn_form(const AttnArgs &a, const AttnPlan &p, cudaStream_t st) {
    const size_t ring = attn_slots(NB, FORM) * 2 * KvGeom<NB>::kTileBytes + static_cast<size_t>(p.wc) * NT * 2 * NB * 512 +
                        (FORM == kPrompt ? 2 * 8 * NB * 512 : 0);
    const size_t sums = static_cast<size_t>(kAttnWarps) * NT * 8 * NB * kQK * 4;
    const size_t smem = attn_sums_apart(NB, NT, FORM) ? ring + sums : (ring > sums ? ring : sums);
    return launch_attn_kernel<&attn_kernel<NB, NT, FORM>>(p, smem, a, st);
}
template <int NB> cudaError_t launch_attn(AttnArgs a, const AttnPlan &p, cudaStream_t st) {
    if (p.cols == kNarrowCols) {
        constexpr size_t kRing = attn_slots(NB, kOwn) * 2 * KvGeom<NB>::kTileBytes, kQ = 2 * NB * 256;
        constexpr size_t kSums = kAttnWarps * kNarrowCols * NB * kQK * 4;
        return launch_attn_kernel<&attn_narrow_kernel<NB>>(p, kRing + kQ + kSums, a, st);
    }
    if constexpr (NB <= kTallBlocks) {
        if (p.tall) return launch_attn_tall<NB>(a, p, st);
    } else {
        if (p.wc > 4) return launch_attn_form<NB, attn_prompt_nt(NB), kPrompt>(a, p, st);
        if (p.wc > 1) return launch_attn_form<NB, 2, kShared>(a, p, st);
    }
    return p.nt == 1 ? launch_attn_form<NB, 1, kOwn>(a, p, st) : launch_attn_form<NB, 2, kOwn>(a, p, st);
}
#endif

}  // namespace zdmmv
