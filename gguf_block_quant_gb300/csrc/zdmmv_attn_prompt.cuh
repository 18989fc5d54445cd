// zdmmv_attn_prompt.cuh -- attention of more than 16 columns (prompts, drafted tokens of
// grouped heads) over the paged 4-bit cache, heads of up to 128 dimensions, on the
// fifth-generation tensor cores (zdmmv_attn.cuh has the formula, the columns and the
// join of parts).
//
// A CTA takes 128 columns of a kv head (the 128 rows of tcgen05.mma's D) and runs
// over its split's tokens in tiles of 128:
//   S = Q K^T, p = exp2(S - max) in registers, O = P V, out += O
//  * Operands are fp16, each in two parts that hold it to 22 bits (q, p) or exactly
//    (k = d (n - 8): 11 + 4 bits): three products hi hi + lo hi + hi lo, the fourth
//    being below 2^-22 of the first.
//  * Q and P are A operands in tensor memory, K and V B operands in shared memory
//    (128-byte swizzle; K by rows of its dimensions, V transposed by the hardware).
//    Tensor memory's 512 columns: Q 128, two tiles of S 256 (P takes S's place, 16
//    tokens' two parts over their 16 sums), O 128.
//  * O leaves tensor memory after every tile and is added up in fp32 registers: the
//    tensor cores truncate where they add, which a tile's additions do not show,
//    but those of thousands of tokens would.
//
//  * 8 d has to be an fp16 number: where a tile has a scale of 2^13 or more (values past 65000), V's operand takes that
//    block's dimensions in units of 16, K's all of the tile, whose scales then count to 2^-21. A unit for each token of K
//    (its sums put right before the softmax) cost every tile of any call 10% of its time.
//
// Warps 0-7 take the softmax and the sums: a thread has 64 of a tile's tokens of a row, whose maximum the row's two threads
// exchange, and half of the row's output. Warps 8-15 turn the cache's codes into operands, three of which fit shared memory,
// in the order S0 S1 O0 S2 O1 S3 ..., and warp 16 starts the products in that order, as soon as warp 19 says so, which also
// finds out what must be made in units of 16: each softmax has the time of two operands' products. (Starting blocks while the
// tensor cores are a product or two behind, and a thread that waits for all of it too leaves them idle for a third of the
// time.) Warps 17 and 18 copy the cache's tiles three operands ahead.
//
// Bound: 24 products of 64 cycles an operand, 3072 cycles a tile, 42 us for 256 tokens over 8192 (32 heads of 128, 152 SMs),
// which takes 82: 128 CTAs of 32 tiles of some 4000 cycles each, and 8 us of starts and ends. A tile's time goes by the
// conversion (1250 to 1500 cycles an operand, 8 warps that share the schedulers with the softmax) and by how soon the next
// tiles' bytes are there. Measured and not kept, each with what was there then: warp 8 starting the products between its
// conversions (230), one thread both waiting and starting (105), a thread for each kind of product (96), operands converted
// and waited for in halves (106 against 97), the tiles' copies by one warp (93), by cp.async (108), and by one lane (123).
#pragma once

#include "zdmmv_attn.cuh"

namespace zdmmv {

constexpr int kPromptThreads = 640, kPromptRows = 128, kPromptTokens = 128, kPromptSlots = 3, kPromptRaw = 3;
constexpr int kPromptSlabs = kPromptTokens / kKvSlab;
// Registers a thread: what the kernel is launched with (20 warps share 65536) is shared out again, 8 warps of softmax, 8 that
// convert, 4 that copy, look over and start the products.
constexpr int kRegsLaunch = 96, kRegsSoft = 160, kRegsFeed = 56, kRegsStart = 48;
static_assert(8 * kRegsSoft + 8 * kRegsFeed + 4 * kRegsStart <= 20 * kRegsLaunch, "more would wait for ever");
// tensor memory columns
constexpr uint32_t kTmCols = 512, kTmS = 128, kTmO = 384;
// barriers: Q is in tensor memory; by half (tile & 1): S is made, P is stored, O is made; O is read; by slot: the operand is
// converted, its products are done; by place of the cache's tiles: copied, looked over, converted; by slot:
// its products may start; all products are done
constexpr int kWaitQ = 0, kWaitS = 1, kWaitP = 3, kWaitO = 5, kWaitFree = 7, kWaitFull = 8, kWaitSlot = 11, kWaitCopy = 14,
              kWaitRaw = 17, kWaitRawFree = 20, kWaitGo = 23, kWaitEnd = 26, kPromptBars = 27;

template <int NB> struct PromptGeom {
    static constexpr int kChunks = (NB + 1) / 2;                          // of 64 dimensions
    static constexpr uint32_t kChunkBytes = kPromptTokens * 128;          // 64 dimensions of a tile
    static constexpr uint32_t kPartBytes = kChunks * kChunkBytes;         // upper or lower parts
    static constexpr uint32_t kSlotBytes = 2 * kPartBytes;
    static constexpr size_t kSmem = kPromptSlots * kSlotBytes + kPromptRaw * 8 * 9 * NB * kQK + 1024;  // aligned to 1024
    static_assert(kPromptRows * NB * kQK * 4 <= kPromptSlots * kSlotBytes, "the sums lie over the slots");
};

// ------------------------------------------------------------------ tensor memory
__device__ __forceinline__ void tm_alloc(uint32_t *to) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(to)), "n"(kTmCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tm_free(uint32_t at) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "n"(kTmCols));
}
__device__ __forceinline__ void tm_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 16 columns of the warp's 32 rows: word i of a lane is its row's column i. The words are there after tm_loaded().
__device__ __forceinline__ void tm_load(uint32_t at, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
}
// ... (each array's words depend on it, so that none is used before)
template <int N> __device__ __forceinline__ void tm_loaded(uint32_t (&r)[N][16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int k = 0; k < N; ++k)
        asm volatile("" : "+r"(r[k][0]), "+r"(r[k][1]), "+r"(r[k][2]), "+r"(r[k][3]), "+r"(r[k][4]), "+r"(r[k][5]), "+r"(r[k][6]),
                          "+r"(r[k][7]), "+r"(r[k][8]), "+r"(r[k][9]), "+r"(r[k][10]), "+r"(r[k][11]), "+r"(r[k][12]), "+r"(r[k][13]),
                          "+r"(r[k][14]), "+r"(r[k][15]));
}
__device__ __forceinline__ void tm_store(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(
            r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(at)
        : "memory");
}
__device__ __forceinline__ void tm_store4(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%4], {%0, %1, %2, %3};" ::"r"(x), "r"(y), "r"(z), "r"(w), "r"(at) : "memory");
}
// D (128 x N, tensor memory) = (or, if `more`, +=) A (128 x 16 fp16, tensor memory) B (16 x N fp16, shared memory)
template <uint32_t KIND> __device__ __forceinline__ void tm_mma(uint32_t d, uint32_t a, uint64_t b, bool more) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a),
        "l"(b), "r"(KIND), "r"(static_cast<uint32_t>(more))
        : "memory");
}
// D = the sum of STEPS products of 16, of A's parts (a step's lower one 8 columns on) and B's (the lower one LOWER on; step k
// is at(k) on). The two products with a lower part come first: their sums are small, so that D is truncated in its full size
// STEPS times only (2.2e-6 of the result against 64 bits for 8192 tokens with all three in turn).
template <uint32_t KIND, int STEPS, uint32_t LOWER, typename At>
__device__ __forceinline__ void tm_mma_parts(uint32_t d, uint32_t a, uint64_t b, At at) {
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        tm_mma<KIND>(d, a + 16 * k + 8, b + (at(k) >> 4), k > 0);
        tm_mma<KIND>(d, a + 16 * k, b + ((at(k) + LOWER) >> 4), true);
    }
#pragma unroll
    for (int k = 0; k < STEPS; ++k) tm_mma<KIND>(d, a + 16 * k, b + (at(k) >> 4), true);
}
__device__ __forceinline__ bool one_lane() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// an arrival on `bar` when the products started so far are done
__device__ __forceinline__ void tm_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// A B operand in rows of 128 bytes, swizzled by 128 bytes, 8 rows a group of 1024 bytes; for one that is transposed, `lead`
// is the distance of its chunks of 64 columns.
__device__ __forceinline__ uint64_t tm_operand(uint32_t at, uint32_t lead) {
    return static_cast<uint64_t>((at >> 4) & 0x3FFFu) | static_cast<uint64_t>(lead >> 4) << 16 | 64ull << 32 | 1ull << 46 | 2ull << 61;
}
// fp16 operands, fp32 sums, 128 rows, n columns; transposed: B's rows are the summed index
__host__ __device__ constexpr uint32_t tm_kind(int n, bool transposed) {
    return 1u << 4 | (transposed ? 1u << 16 : 0u) | static_cast<uint32_t>(n / 8) << 17 | (kPromptRows / 16) << 24;
}

// ------------------------------------------------------------------ the cache's operands
// Operand i of n tiles' 2 n: K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1). A warp of 8-15 has a cache tile (16 tokens) of each.
template <int NB> struct PromptFeed {
    using G = KvGeom<NB>;
    static constexpr uint32_t kRawBytes = G::kCodeBytes + G::kScaleBytes;  // a cache tile's K or V
    static_assert(kPromptRaw == kPromptSlots && kPromptRaw * 2 == 6, "operand i's place is its slot; its unit lives for two turns");

    __device__ static bool is_v(int i, int n) { return i == 2 * n - 1 || (i > 0 && !(i & 1)); }
    __device__ static int tile(int i, int n) { return i == 2 * n - 1 ? n - 1 : (i == 0 ? 0 : ((i & 1) ? (i + 1) / 2 : i / 2 - 1)); }
    // the token of an octet that this lane's words become a row of
    __device__ static int token(int lane, bool v) { return v ? 2 * (lane & 3) + (lane >> 2 & 1) : lane >> 2; }
    // 8 codes times d: the upper parts to `at`, the lower ones behind them. Order: dimensions 0 4 1 5 2 6 3 7.
    __device__ static void put(uint32_t w, uint32_t d, uint32_t magic, uint32_t at) {
        constexpr uint32_t kM1032 = 0xE408E408u, kM72 = 0xD480D480u, k16th = 0x2C002C00u;
        const uint32_t w8 = w >> 8;
        uint32_t n[4], lo[4];
        n[0] = h2_add((w & 0x000F000Fu) | magic, kM1032);
        n[1] = h2_fma((w & 0x00F000F0u) | magic, k16th, kM72);
        n[2] = h2_add((w8 & 0x000F000Fu) | magic, kM1032);
        n[3] = h2_fma((w8 & 0x00F000F0u) | magic, k16th, kM72);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t hi = h2_mul(n[k], d);
            lo[k] = h2_fma(n[k], d, h2_neg(hi));
            n[k] = hi;
        }
        sts128(at, n[0], n[1], n[2], n[3]);
        sts128(at + PromptGeom<NB>::kPartBytes, lo[0], lo[1], lo[2], lo[3]);
    }
    // Octet u of the cache tile at `raw` becomes rows row0 .. row0+7 of the operand at `slot`; rows from `live` on are no
    // tokens and become zeros, whatever the cache holds there.
    template <bool V> __device__ static void convert(uint32_t raw, int u, uint32_t slot, int row0, int live, uint32_t units, uint32_t magic, int lane) {
        const int tok = token(lane, V), row = row0 + tok, t8 = V ? lane >> 3 : lane & 3;
        const uint32_t pick = row >= live ? 0x4444u : ((tok & 1) ? 0x3232u : 0x1010u);
        uint32_t w[NB], d[NB];
        lds_words<NB, G::kVec>(raw + (u * NB * 32 + lane * G::kVec) * 4, 128 * G::kVec, w);
        lds_words<NB, G::kVec>(raw + G::kCodeBytes + (4 * u + (tok >> 1)) * NB * 4, 4 * G::kVec, d);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            d[b] = __byte_perm(d[b], 0, pick);
            if (V) {  // two tokens of 4 dimensions: the neighbour's for one token of 8
                const uint32_t o = __shfl_xor_sync(0xffffffffu, w[b], 4);
                w[b] = __byte_perm(w[b], o, (lane & 4) ? 0x3276 : 0x5410);
            }
        }
        if (units != 0)
#pragma unroll
            for (int b = 0; b < NB; ++b)
                if (units >> b & 1u) d[b] = h2_mul(d[b], 0x2C002C00u);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            // K: odd rows begin with the other block of a chunk, so that 8 lanes' stores meet 8 different banks
            const int o = (b ^ 1) < NB ? b ^ 1 : b;
            const bool other = !V && o != b && (row & 1);
            const uint32_t x = other ? w[o] : w[b], y = other ? d[o] : d[b];
            const int c = (((b & 1) ^ (other ? 1 : 0)) * 4 + t8) ^ (row & 7);
            put(x, y, magic, slot + (b >> 1) * PromptGeom<NB>::kChunkBytes + row * 128 + c * 16);
        }
    }
    // The blocks that are made in units of 16, a bit each: those with a scale of a live token of the 8 cache tiles at `raw` that
    // is 2^13 or more (its exponent's upper three bits are set), so that 8 d is no fp16 number; of K all or none, whose blocks
    // are one sum.
    __device__ static uint32_t units(uint32_t raw, int live, bool v, int lane) {
        uint32_t any = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w)
            for (int k = lane; k < 8 * NB; k += 32) {
                const uint32_t d = lds32(raw + w * kRawBytes + G::kCodeBytes + k * 4);
                const int tok = 16 * w + 2 * (k / NB);
                any |= d & d << 1 & d << 2 & ((tok < live ? 0x4000u : 0u) | (tok + 1 < live ? 0x40000000u : 0u));
            }
        if (!__any_sync(0xffffffffu, any != 0)) return 0;
        if (!v) return ~0u;
        uint32_t blocks = 0;
#pragma unroll 1
        for (int i = lane; i < 64 * NB; i += 32) {
            const int w = i / (8 * NB), k = i % (8 * NB), tok = 16 * w + 2 * (k / NB);
            const uint32_t d = lds32(raw + w * kRawBytes + G::kCodeBytes + k * 4);
            if (d & d << 1 & d << 2 & ((tok < live ? 0x4000u : 0u) | (tok + 1 < live ? 0x40000000u : 0u))) blocks |= 1u << k % NB;
        }
        return __reduce_or_sync(0xffffffffu, blocks);
    }
};

// A row once more, token by token, by a warp with a lane for a dimension of each block: what the row sees of the split, its sums
// to `sum` (column's quads exchanged as the kernel has them), its maximum and sum of p. Two kinds of rows need it, neither of
// ordinary calls: where V is an infinity or NaN the products are NaN for rows that do not see it (0 times NaN); and from scores
// of kHugeScoreTall on the fma of p's exponent does not do. (In the tiles' loops the one cost every call 2 to 10% of its time, the
// other 2.)
template <int NB>
__device__ __forceinline__ void attn_redo(const AttnArgs &a, const AttnSeg &seg, int col, int row, float *sum, float &row_m, float &row_l, int lane) {
    using G = KvGeom<NB>;
    const AttnRange &r = seg.r;
    const int i = a.by_group.div(col), seen = max(0, r.len - (r.n - 1 - i));
    const int end = min(min(r.len, seg.last * kKvSlab), seen);
    const int low = max(seg.first * kKvSlab, a.window > 0 ? seen - a.window : 0);
    const int32_t *table = a.c.table + static_cast<int64_t>(seg.seq) * a.c.max_pages;
    const uint8_t *head = a.c.pages + static_cast<int64_t>(seg.kvh) * static_cast<int>(a.by_page_tiles.d) * G::kTileBytes;
    const float *src = a.q + static_cast<int64_t>(r.q0 + i) * a.q_stride + static_cast<int64_t>(seg.kvh * a.group + col - i * a.group) * G::kDim + lane;
    float q[NB], o[NB], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        q[b] = src[b * kQK];
        o[b] = 0.0f;
    }
#pragma unroll 1
    for (int t = low; t < end; ++t) {
        const int slab = t / kKvSlab, tok = t % kKvSlab, slot = a.by_page_tiles.div(slab);
        const uint8_t *tile = head + table[slot] * a.c.page_bytes + static_cast<int64_t>(a.by_page_tiles.mod(slab, slot)) * G::kTileBytes;
        const __half *scales = reinterpret_cast<const __half *>(tile + G::kKScaleAt);  // then V's
        float s = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t code = reinterpret_cast<const uint32_t *>(tile)[G::k_word(tok, b, lane / 8)] >> 4 * (lane % 8) & 15u;
            s = fmaf(q[b], __half2float(scales[G::scale_half(tok, b)]) * (static_cast<float>(code) - 8.0f), s);
        }
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
        s *= a.scale_log2;
        const float to = fmaxf(m, s), keep = m == -INFINITY ? 0.0f : exp2_approx(m - to), p = exp2_approx(__fadd_rn(s, -to) + kAttnUnit);
        m = to;
        l = fmaf(l, keep, p);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t code = reinterpret_cast<const uint16_t *>(tile + G::kVAt)[G::v_half(tok, b, lane / 4)] >> 4 * (lane % 4) & 15u;
            const float v = __half2float(scales[G::kScaleBytes / 2 + G::scale_half(tok, b)]) * (static_cast<float>(code) - 8.0f);
            o[b] = fmaf(o[b], keep, p * v);
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) sum[row * G::kDim + 4 * ((8 * b + lane / 4) ^ (row & 7)) + lane % 4] = o[b];
    if (lane == 0) {
        row_m = m;
        row_l = l;
    }
}

template <int NB> __global__ void __launch_bounds__(kPromptThreads, 1) attn_prompt_kernel(AttnArgs a) {
    using G = KvGeom<NB>;
    using P = PromptGeom<NB>;
    constexpr int D = G::kDim;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bar[kPromptBars];
    __shared__ float sh_top[2][2][kPromptRows], sh_m[kPromptRows], sh_l[2][kPromptRows], sh_made_k[4];
    __shared__ int sh_bad, sh_last, sh_redo;
    __shared__ uint32_t sh_tm, sh_magic, sh_unit[6], sh_made_v[4];
    __shared__ AttnSeg sh_seg;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, half = warp >> 2;
    if (tid == 0) {
        for (int k = 0; k < kPromptBars; ++k) {
            const bool rows = k == kWaitQ || k == kWaitP || k == kWaitP + 1 || k == kWaitFree;  // warps 0-7
            const bool each = (k >= kWaitFull && k < kWaitSlot) || (k >= kWaitRawFree && k < kWaitGo);  // warps 8-15
            // the products and their unit
            const bool both = k == kWaitS || k == kWaitS + 1 || k == kWaitO || k == kWaitO + 1;
            mbar_init(&bar[k], rows ? 2 * kPromptRows : (each ? 8 : (both || (k >= kWaitCopy && k < kWaitRaw) ? 2 : 1)));
        }
        sh_bad = sh_redo = 0;
        sh_magic = kCodeMagic;
        fence_barrier_init();
    }
    block_op_wait();
    block_op_release();
    {
        AttnSeg seg;
        if (!attn_grid_seg(a, kPromptRows, seg)) return;
        if (tid == 0) sh_seg = seg;
    }
    if (warp == 16) tm_alloc(&sh_tm);
    tm_before_sync();
    __syncthreads();
    tm_after_sync();
    const AttnSeg &seg = sh_seg;
    const AttnRange &r = seg.r;
    const uint32_t tm = sh_tm;
    const uint32_t slots = (smem_addr(smem) + 1023u) & ~1023u;
    float *sum = reinterpret_cast<float *>(smem + (slots - smem_addr(smem)));
    uint8_t *raws = reinterpret_cast<uint8_t *>(sum) + kPromptSlots * P::kSlotBytes;  // [place][8] cache tiles' K or V
    const int first = seg.first, last = seg.last, limit = min(r.len, last * kKvSlab);
    const int n = (last - first + kPromptSlabs - 1) / kPromptSlabs;
    bool dead = false;  // a wait gave up: no more waits, but every barrier of threads is met; the result is NaN
    const auto wait = [&](int which, uint32_t parity) {
        if (!dead && !mbar_wait(&bar[which], parity)) {
            atomicOr(a.fault, 1u);
            dead = true;
        }
    };

    if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsStart));
        if (warp == 19) {  // finds the operands' unit, two ahead, and says when the products may start
            const auto scan = [&](int i) {
                const int s = i % kPromptRaw, tile = PromptFeed<NB>::tile(i, n);
                wait(kWaitCopy + s, i / kPromptRaw & 1);
                __syncwarp();
                const uint32_t units = PromptFeed<NB>::units(smem_addr(raws) + s * 8 * PromptFeed<NB>::kRawBytes,
                                                             limit - first * kKvSlab - tile * kPromptTokens, PromptFeed<NB>::is_v(i, n), lane);
                if (lane == 0) {
                    sh_unit[i % 6] = units;
                    mbar_arrive(&bar[kWaitRaw + s]);
                }
            };
            for (int i = 0; i < min(2, 2 * n); ++i) scan(i);
            wait(kWaitQ, 0);
#pragma unroll 1
            for (int i = 0; i < 2 * n; ++i) {
                const int s = i % kPromptSlots, tile = PromptFeed<NB>::tile(i, n), b = tile & 1;
                const bool v = PromptFeed<NB>::is_v(i, n);
                if (i + 2 < 2 * n) scan(i + 2);
                if (v) {
                    wait(kWaitP + b, tile >> 1 & 1);
                    if (tile > 0) wait(kWaitFree, (tile - 1) & 1);
                }
                wait(kWaitFull + s, i / kPromptSlots & 1);
                tm_after_sync();
                if (lane == 0 && !dead) {
                    if (v) sh_made_v[tile & 3] = sh_unit[i % 6];
                    else sh_made_k[tile & 3] = sh_unit[i % 6] ? 16.0f : 1.0f;
                    mbar_arrive(&bar[(v ? kWaitO : kWaitS) + b]);
                    tm_before_sync();
                    mbar_arrive(&bar[kWaitGo + s]);
                }
                __syncwarp();
            }
        }
        if (warp == 16) {  // starts them: by one lane, but with addresses that the compiler sees to be the warp's
            const int todo = __shfl_sync(0xffffffffu, 2 * n, 0);
            const uint32_t tm0 = __shfl_sync(0xffffffffu, tm, 0);
            int s = 0, phase = 0;
#pragma unroll 1
            for (int i = 0; i < todo; ++i) {
                const bool v = PromptFeed<NB>::is_v(i, todo / 2);
                const int b = PromptFeed<NB>::tile(i, todo / 2) & 1;
                const uint32_t half_at = tm0 + kTmS + b * kPromptTokens;
                const uint64_t operand = tm_operand(slots + s * P::kSlotBytes, P::kChunkBytes);
                wait(kWaitGo + s, phase);
                if (__any_sync(0xffffffffu, dead)) break;
                tm_after_sync();
                if (one_lane()) {
                    if (v)
                        tm_mma_parts<tm_kind(D, true), kPromptTokens / 16, P::kPartBytes>(tm0 + kTmO, half_at, operand,
                                                                                          [](int k) { return k * 2048u; });
                    else
                        tm_mma_parts<tm_kind(kPromptTokens, false), D / 16, P::kPartBytes>(
                            half_at, tm0, operand, [](int k) { return (k >> 2) * P::kChunkBytes + (k & 3) * 32u; });
                    tm_commit(&bar[(v ? kWaitO : kWaitS) + b]);
                    tm_commit(&bar[kWaitSlot + s]);
                }
                __syncwarp();
                if (++s == kPromptSlots) {
                    s = 0;
                    phase ^= 1;
                }
            }
            // the products that were started are done before their operands' and sums' memory is another's
            if (one_lane()) tm_commit(&bar[kWaitEnd]);
            if (!mbar_wait(&bar[kWaitEnd], 0)) {
                atomicOr(a.fault, 1u);
                dead = true;
            }
        }
        if (warp == 17 || warp == 18) {  // the cache's tiles, a lane each of half an operand's 8 (a lane's copy takes 90 cycles, one after another)
            const int32_t *table = a.c.table + static_cast<int64_t>(seg.seq) * a.c.max_pages;
            const uint8_t *head = a.c.pages + static_cast<int64_t>(seg.kvh) * static_cast<int>(a.by_page_tiles.d) * G::kTileBytes;
            const uint64_t policy = l2_evict_first_policy();
            int i = 0;
#pragma unroll 1
            for (; i < 2 * n; ++i) {
                const int s = i % kPromptRaw, mine = 4 * (warp - 17) + lane, slab = first + PromptFeed<NB>::tile(i, n) * kPromptSlabs + mine;
                const bool v = PromptFeed<NB>::is_v(i, n), in = lane < kPromptSlabs / 2 && slab < last;
                int page = in ? TileFeed<NB>::page_at(a, table, slab) : 0;
                if (in && (page < 0 || page >= a.c.n_pages)) {
                    sh_bad = 1;
                    if (a.status) *a.status = 1;
                    page = 0;
                }
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, in)) * PromptFeed<NB>::kRawBytes;
                if (i >= kPromptRaw) wait(kWaitRawFree + s, (i / kPromptRaw - 1) & 1);
                if (__any_sync(0xffffffffu, dead)) break;
                if (lane == 0) mbar_arrive_expect_tx(&bar[kWaitCopy + s], bytes);
                __syncwarp();
                if (in) {
                    const uint8_t *src = head + page * a.c.page_bytes +
                                         static_cast<int64_t>(a.by_page_tiles.mod(slab, a.by_page_tiles.div(slab))) * G::kTileBytes;
                    uint8_t *to = raws + (s * 8 + mine) * PromptFeed<NB>::kRawBytes;
                    bulk_copy_g2s(to, src + (v ? G::kVAt : 0), G::kCodeBytes, &bar[kWaitCopy + s], policy);
                    bulk_copy_g2s(to + G::kCodeBytes, src + (v ? G::kVScaleAt : G::kKScaleAt), G::kScaleBytes, &bar[kWaitCopy + s], policy);
                }
            }
            // leave only when the copies have landed (after a wait that gave up: as far as they will)
            for (int k = max(0, i - kPromptRaw); k < i; ++k) (void)mbar_wait(&bar[kWaitCopy + k % kPromptRaw], k / kPromptRaw & 1);
        }
        if (dead) sh_bad = 1;
        __syncwarp();
        __syncthreads();
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFeed));
        const int w = warp - 8;
        const uint32_t magic = lds32(smem_addr(&sh_magic));
        using F = PromptFeed<NB>;
#pragma unroll 1
        for (int i = 0; i < 2 * n; ++i) {
            const int s = i % kPromptSlots, tile = F::tile(i, n), live = limit - first * kKvSlab - tile * kPromptTokens;
            const uint32_t slot = slots + s * P::kSlotBytes, raw = smem_addr(raws) + (s * 8 + w) * F::kRawBytes;
            wait(kWaitRaw + s, i / kPromptRaw & 1);
            if (i == kPromptSlots - 1) wait(kWaitQ, 0);  // Q has left the slot
            if (i >= kPromptSlots) wait(kWaitSlot + s, (i / kPromptSlots - 1) & 1);
            __syncwarp();
            const uint32_t units = sh_unit[i % 6];
            if (F::is_v(i, n)) {
#pragma unroll
                for (int u = 0; u < 2; ++u) F::template convert<true>(raw, u, slot, 16 * w + 8 * u, live, units, magic, lane);
            } else {
#pragma unroll
                for (int u = 0; u < 2; ++u) F::template convert<false>(raw, u, slot, 16 * w + 8 * u, live, units, magic, lane);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar[kWaitFull + s]);
                mbar_arrive(&bar[kWaitRawFree + s]);
            }
        }
        if (dead) sh_bad = 1;
        __syncthreads();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
        const int row = tid & (kPromptRows - 1), col = seg.ct * kPromptRows + row;
        const uint32_t rows = tm + (static_cast<uint32_t>(warp & 3) << 21);  // the warp's 32 rows
        const int i = a.by_group.div(col);
        const bool valid = i < r.n;
        float qs;
        {  // Q: whole rows by a warp (a lane's own row at once costs 4096 cycles of cache lines), through the last slot
            constexpr int kQuads = D / 4;
            float4 x[D / 8];
            float4 *stage = reinterpret_cast<float4 *>(reinterpret_cast<uint8_t *>(sum) + (kPromptSlots - 1) * P::kSlotBytes);
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                const int at = 32 * k + lane, to = 16 * warp + at / kQuads, c = seg.ct * kPromptRows + to, token = a.by_group.div(c);
                x[k] = token < r.n ? *reinterpret_cast<const float4 *>(a.q + static_cast<int64_t>(r.q0 + token) * a.q_stride +
                                                                       static_cast<int64_t>(seg.kvh * a.group + c - token * a.group) * D +
                                                                       4 * (at % kQuads))
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                const int at = 32 * k + lane, to = 16 * warp + at / kQuads;
                stage[to * kQuads + (at % kQuads ^ (to & 7))] = x[k];
            }
            asm volatile("barrier.cta.sync 2, 256;" ::: "memory");
#pragma unroll
            for (int e = 0; e < D / 8; ++e) x[e] = stage[row * kQuads + ((half * (D / 8) + e) ^ (row & 7))];
            float top = 0.0f;
#pragma unroll
            for (int e = 0; e < D / 8; ++e)
                top = fmaxf(fmaxf(fmaxf(top, fabsf(x[e].x)), fmaxf(fabsf(x[e].y), fabsf(x[e].z))), fabsf(x[e].w));
            sh_top[1][half][row] = top;
            asm volatile("barrier.cta.sync 2, 256;" ::: "memory");
            top = fmaxf(top, sh_top[1][half ^ 1][row]);
            float up, down;
            q_unit(top, a.scale_log2, up, down);
            qs = fmaxf(fabsf(a.scale_log2) * down, 1e-37f);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {  // 8 dimensions
                uint32_t f[8];
                const float4 y = x[2 * k], z = x[2 * k + 1];
                split_h2(y.x * up, z.x * up, f[0], f[4]);
                split_h2(y.y * up, z.y * up, f[1], f[5]);
                split_h2(y.z * up, z.z * up, f[2], f[6]);
                split_h2(y.w * up, z.w * up, f[3], f[7]);
                const int e = half * (D / 16) + k;  // of the row's D / 8
                tm_store4(rows + 16 * (e >> 1) + 4 * (e & 1), f[0], f[1], f[2], f[3]);
                tm_store4(rows + 16 * (e >> 1) + 8 + 4 * (e & 1), f[4], f[5], f[6], f[7]);
            }
            tm_stored();
            tm_before_sync();
            mbar_arrive(&bar[kWaitQ]);
        }
        const int seen = max(0, r.len - (r.n - 1 - i));
        const int end = valid ? min(limit, seen) : limit, low = valid && a.window > 0 ? max(0, seen - a.window) : 0;
        float m = -INFINITY, keep = 0.0f;
        constexpr int kLoads = D / 32;  // of 16 of the thread's D / 2 dimensions
        uint64_t l2 = 0, acc[D / 4];    // acc[4 g + k]: dimensions 8 g + k and 8 g + 4 + k of its half
#pragma unroll
        for (int k = 0; k < D / 4; ++k) acc[k] = 0;
        const auto drain = [&](int tile) {  // the sums of a tile
            wait(kWaitO + (tile & 1), tile >> 1 & 1);
            __syncwarp();
            tm_after_sync();
            const uint32_t units = sh_made_v[tile & 3];
            uint32_t o[kLoads][16];
#pragma unroll
            for (int c = 0; c < kLoads; ++c) tm_load(rows + kTmO + half * (D / 2) + 16 * c, o[c]);
            tm_loaded(o);
            tm_before_sync();
            mbar_arrive(&bar[kWaitFree]);
            if (units != 0) {
#pragma unroll
                for (int c = 0; c < kLoads; ++c)
                    if (units >> ((half * (D / 2) + 16 * c) / kQK) & 1u)
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[c][k] = __float_as_uint(16.0f * __uint_as_float(o[c][k]));
            }
            const uint64_t keep2 = f2(keep, keep);
#pragma unroll
            for (int c = 0; c < kLoads; ++c)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    acc[8 * c + k] = f2_fma(acc[8 * c + k], keep2, f2(__uint_as_float(o[c][2 * k]), __uint_as_float(o[c][2 * k + 1])));
        };
#pragma unroll 1
        for (int tile = 0; tile < n; ++tile) {
            const uint32_t at = rows + kTmS + (tile & 1) * kPromptTokens + half * (kPromptTokens / 2);
            const int t0 = first * kKvSlab + tile * kPromptTokens + half * (kPromptTokens / 2);
            wait(kWaitS + (tile & 1), tile >> 1 & 1);
            __syncwarp();
            tm_after_sync();
            const float unit = qs * sh_made_k[tile & 3];
            uint32_t s[4][16];
#pragma unroll
            for (int c = 0; c < 4; ++c) tm_load(at + 16 * c, s[c]);
            tm_loaded(s);
            if (__any_sync(0xffffffffu, t0 < low || t0 + kPromptTokens / 2 > end)) {
#pragma unroll
                for (int k = 0; k < 64; ++k)
                    if (t0 + k < low || t0 + k >= end) s[k / 16][k % 16] = 0xff800000u;
            }
            float top = -INFINITY, top1 = -INFINITY;
#pragma unroll
            for (int k = 0; k < 64; k += 4) {
                top = fmaxf(fmaxf(top, __uint_as_float(s[k / 16][k % 16])), __uint_as_float(s[k / 16][k % 16 + 1]));
                top1 = fmaxf(fmaxf(top1, __uint_as_float(s[k / 16][k % 16 + 2])), __uint_as_float(s[k / 16][k % 16 + 3]));
            }
            top = fmaxf(top, top1) * unit;
            sh_top[tile & 1][half][row] = top;
            asm volatile("barrier.cta.sync 2, 256;" ::: "memory");
            const float to = fmaxf(m, fmaxf(top, sh_top[tile & 1][half ^ 1][row]));
            const float then = m == -INFINITY ? 0.0f : exp2_approx(m - to);
            m = to;
            const float shift = to == -INFINITY ? 0.0f : kAttnUnit - to;
            const uint64_t unit2 = f2(unit, unit), shift2 = f2(shift, shift);
            l2 = f2_mul(l2, f2(then, then));
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t f[16];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint64_t x = f2_fma(f2(__uint_as_float(s[c][2 * k]), __uint_as_float(s[c][2 * k + 1])), unit2, shift2);
                    const float2 v = f2_parts(x);
                    const uint64_t p = f2(exp2_approx(v.x), exp2_approx(v.y));
                    l2 = f2_add(l2, p);
                    split_f2(p, f[k], f[8 + k]);
                }
                tm_store(at + 16 * c, f);
            }
            tm_stored();
            tm_before_sync();
            mbar_arrive(&bar[kWaitP + (tile & 1)]);
            if (tile > 0) drain(tile - 1);
            keep = then;
        }
        if (n > 0) drain(n - 1);
        if (dead) sh_bad = 1;
        uint64_t no = 0;  // 0 times a sum that is no number
#pragma unroll
        for (int k = 0; k < D / 4; ++k) no = f2_fma(acc[k], 0, no);
        if (!(f2_parts(no).x + f2_parts(no).y == 0.0f) || score_huge(m, kHugeScoreTall)) sh_redo = 1;
        const float2 ls = f2_parts(l2);
        sh_l[half][row] = ls.x + ls.y;
        __syncthreads();  // the products are done; their operands' memory takes the sums
        if (half == 0) {
            sh_m[row] = m;
            sh_l[0][row] += sh_l[1][row];
        }
        float *mine = sum + row * D;
#pragma unroll
        for (int g = 0; g < D / 16; ++g) {
            float2 x[4];
            const int quad = half * (D / 8) + 2 * g;
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = f2_parts(acc[4 * g + k]);
            *reinterpret_cast<float4 *>(mine + 4 * (quad ^ (row & 7))) = make_float4(x[0].x, x[1].x, x[2].x, x[3].x);
            *reinterpret_cast<float4 *>(mine + 4 * ((quad + 1) ^ (row & 7))) = make_float4(x[0].y, x[1].y, x[2].y, x[3].y);
        }
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));
    }
    if (warp >= 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));  // waits for warps 0-7 to give theirs back, which wait for nothing
    tm_before_sync();
    __syncthreads();
    tm_after_sync();
    if (warp == 16) tm_free(tm);
    if (sh_redo && !sh_bad && !r.bad) {
        for (int row = warp; row < kPromptRows; row += kPromptThreads / 32) {
            const int col = seg.ct * kPromptRows + row;
            if (col >= r.n * a.group) break;
            bool no = false;
            for (int e = lane; e < D; e += 32) no |= !isfinite(sum[row * D + e]);
            if (score_huge(sh_m[row], kHugeScoreTall) || (__any_sync(0xffffffffu, no) && isfinite(sh_l[0][row])))
                attn_redo<NB>(a, seg, col, row, sum, sh_m[row], sh_l[0][row], lane);
        }
        __syncthreads();
    }
    attn_store<D, kPromptRows, kPromptThreads / 32, true>(a, seg, kPromptRows, 1, 1, sum, sh_m, &sh_l[0][0], r.bad || sh_bad, &sh_last);
}

template <int NB> cudaError_t launch_attn_tall(const AttnArgs &a, const AttnPlan &p, cudaStream_t st) {
    const cudaError_t e = smem_limit_raised<&attn_prompt_kernel<NB>>();
    if (e != cudaSuccess) return e;
    static const bool shares_fit = [] {  // the compiler may have launched it with fewer registers than are shared out
        cudaFuncAttributes f{};
        return cudaFuncGetAttributes(&f, attn_prompt_kernel<NB>) == cudaSuccess && f.numRegs == kRegsLaunch;
    }();
    if (!shares_fit) return cudaErrorLaunchOutOfResources;
    return launch_block_op(&attn_prompt_kernel<NB>, dim3(static_cast<unsigned>(p.items), p.n_split), dim3(kPromptThreads),
                           PromptGeom<NB>::kSmem, st, a);
}

}  // namespace zdmmv
