// zdmmv_kv_keep.cu -- what stays in the paged 4-bit cache: zdmmv_kv_evict_q4_0 (the tokens with the largest sums of attention
// weights, to other pages) and zdmmv_kv_accept_q4_0 (the accepted path of a drafted tree, in place).
#include <cooperative_groups.h>

#include <algorithm>

#include "zdmmv_kv.cuh"
#include "zdmmv_internal.h"

namespace zdmmv {
namespace {

namespace cg = cooperative_groups;

struct KeepArgs {
    KvView from, to;
    FastDiv by_heads, from_page_tiles, to_page_tiles, by_tiles;
    const int32_t *kv_len;
    const float *sums;
    int32_t *index;
    float *sums_out;
    int32_t *len_out, *status;
    int64_t sums_stride, sums_out_stride;
    int32_t max_kv_len, budget, sinks, recent;
    int32_t held;  // sums of a CTA that its shared memory holds, as keys
};

// Whether a sequence's length is none that a call takes.
__device__ __forceinline__ bool keep_bad(const KeepArgs &a, int n) {
    return n < 0 || n > a.max_kv_len || n > static_cast<int64_t>(a.from.max_pages) * a.from.page_tokens;
}

// A sum as a whole number that rises with it: -0 is 0, a NaN is below all.
__device__ __forceinline__ uint32_t sum_key(float x) {
    if (x != x) x = -INFINITY;
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

// ------------------------------------------------------------------ which tokens stay
// A cluster of CTAs for a kv head of a sequence (one CTA for up to 20480 tokens), each with an equal stretch of the tokens between the
// first and the latest ones, whose sums it reads once into shared memory. The smallest sum that stays is found digit by digit,
// 11 bits at a time from the top: every CTA counts its sums by digit, and adds up the cluster's counts. Then each CTA knows how
// many tokens stay before its own, and writes its own in their order: of sums equal to the smallest, the first ones.
// 32 kv heads of up to 65536 tokens: 16 to 19 us, of which the sums' loads take 3, each of the two or three counts 3 (its additions in
// shared memory, the cluster's barrier, the reading of four CTAs' counts), the rising places 3. Bound by these steps' latencies.
constexpr int kPickThreads = 1024, kPickWarps = kPickThreads / 32, kDigit = 2048, kPickCluster = 8;
// Tokens up to which a CTA more costs more than it saves, the cluster's barriers above all (8 kv heads, one, two, four and eight
// CTAs each: 16000 tokens 12.3 12.9 13.5 17.0 us with the move of 256, 32000 17.5 15.2 14.6 17.5, 131072 132 60 22.2 20.9).
constexpr int kPickEach = 20 * 1024;
constexpr int kPickMost = 0x7fff0000;  // tokens, and places of index: so that a cluster's step past the last one is a number too
constexpr int kPickHeld = 48 * 1024;   // most sums that a CTA holds; those beyond it are read again (65536 by one CTA 56 us, by two 20)

template <bool CLUSTER> __global__ void __launch_bounds__(kPickThreads) kv_pick_kernel(KeepArgs a) {
    extern __shared__ uint32_t held[];
    __shared__ __align__(16) uint32_t sh_count[3][kDigit];  // of this CTA's sums, by digit
    __shared__ uint32_t sh_scan[kPickWarps], sh_above[kPickWarps], sh_equal[kPickWarps];
    __shared__ uint32_t sh_found, sh_want, sh_have, sh_mine[2];
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = CLUSTER ? static_cast<int>(cluster.num_blocks()) : 1, rank = CLUSTER ? static_cast<int>(cluster.block_rank()) : 0;
    const auto sync_all = [&] {
        if constexpr (CLUSTER) cluster.sync();
        else __syncthreads();
    };
    const auto of_rank = [&](uint32_t *p, int q) { return CLUSTER ? cluster.map_shared_rank(p, q) : p; };
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    block_op_wait();
    block_op_release();
    const int item = blockIdx.x / ranks, seq = a.by_heads.div(item);
    const float *sums = a.sums + static_cast<int64_t>(item) * a.sums_stride;
    int32_t *index = a.index + static_cast<int64_t>(item) * a.budget;
    const int n = a.kv_len[seq];
    const bool bad = keep_bad(a, n);
    if (bad && rank == 0 && tid == 0 && a.status) *a.status = 1;
    const int me = rank * kPickThreads + tid, all = ranks * kPickThreads;
    if (bad || n <= a.budget) {  // the whole cluster takes this way
        for (int j = me; j < a.budget; j += all) index[j] = !bad && j < n ? j : -1;
        return;
    }
    for (int j = me; j < a.sinks; j += all) index[j] = j;
    for (int j = me; j < a.recent; j += all) index[a.budget - a.recent + j] = n - a.recent + j;
    const int between = n - a.sinks - a.recent;                 // more than are wanted of them
    uint32_t want = static_cast<uint32_t>(a.budget - a.sinks - a.recent);
    if (want == 0) return;
    const int each = (between + ranks - 1) / ranks, first = min(between, rank * each), mine = min(each, between - first);
    const float *src = sums + a.sinks + first;
    const int here = min(mine, a.held);
    constexpr int kAhead = 16;  // loads at a time in flight
    for (int i0 = tid; i0 < here; i0 += kAhead * kPickThreads) {
        float x[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) x[k] = i0 + k * kPickThreads < here ? src[i0 + k * kPickThreads] : 0.0f;
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i0 + k * kPickThreads < here) held[i0 + k * kPickThreads] = sum_key(x[k]);
    }
    for (int i = tid; i < 3 * kDigit; i += kPickThreads) (&sh_count[0][0])[i] = 0;
    __syncthreads();
    // for every sum of from .. to - 1, a lane's turn each, whole warps at a time: at(i, key, whether there is one)
    const auto each_key = [&](int from, int to, int step, auto at) {
        int i = from;
#pragma unroll 4
        for (; i - lane + 31 < min(to, here); i += step) at(i, held[i], true);
        for (; i - lane < to; i += step) at(i, i < to ? (i < here ? held[i] : sum_key(src[i])) : 0u, i < to);
    };

    uint32_t known = 0;  // the smallest sum's digits so far
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), above = shift + (pass == 2 ? 10 : 11);
        const uint32_t mask = pass == 2 ? 1023u : 2047u;
        each_key(tid, mine, kPickThreads, [&](int, uint32_t k, bool in) {
            if (in && (pass == 0 || k >> above == known >> above)) atomicAdd(&sh_count[pass][k >> shift & mask], 1u);
        });
        sync_all();
        // two digits a thread, the largest first; `want` of the cluster's sums with the known digits stay
        static_assert(kDigit == 2 * kPickThreads, "two digits a thread");
        uint32_t c0 = 0, c1 = 0;
        for (int q = 0; q < ranks; ++q) {
            const uint2 x = *reinterpret_cast<const uint2 *>(of_rank(&sh_count[pass][kDigit - 2 - 2 * tid], q));
            c0 += x.y;
            c1 += x.x;
        }
        const uint32_t sum = c0 + c1;
        uint32_t upto = sum;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, upto, k);
            if (lane >= k) upto += o;
        }
        if (lane == 31) sh_scan[warp] = upto;
        __syncthreads();
        uint32_t front = lane < warp ? sh_scan[lane] : 0;  // the warps before
        upto += __reduce_add_sync(0xffffffffu, front);
        const uint32_t over = upto - sum;  // sums of larger digits than this thread's
        if (over < want && want <= upto) {
            const bool second = want > over + c0;
            sh_found = static_cast<uint32_t>(kDigit - 1 - 2 * tid - (second ? 1 : 0));
            sh_want = want - over - (second ? c0 : 0);
            sh_have = second ? c1 : c0;
        }
        __syncthreads();
        known |= sh_found << shift;
        want = sh_want;
        if (want == sh_have) {  // all with these digits stay (mostly one after two counts): all above the number before
            --known;            // no sum's digits are all 0
            want = 0;
            break;
        }
    }
    // `want` of the sums equal to `known` stay, and all above it: a warp's stretch of the CTA's
    const int per_warp = (mine + 32 * kPickWarps - 1) / (32 * kPickWarps) * 32;
    const int from = min(mine, warp * per_warp), to = min(mine, from + per_warp);
    uint32_t more = 0, same = 0;
    each_key(from + lane, to, 32, [&](int, uint32_t k, bool in) {
        more += in && k > known;
        same += in && k == known;
    });
    more = __reduce_add_sync(0xffffffffu, more);
    same = __reduce_add_sync(0xffffffffu, same);
    if (lane == 0) {
        sh_above[warp] = more;
        sh_equal[warp] = same;
    }
    __syncthreads();
    static_assert(kPickWarps == 32, "a lane for each warp");
    if (warp == 0) {
        const uint32_t m = __reduce_add_sync(0xffffffffu, sh_above[lane]), e = __reduce_add_sync(0xffffffffu, sh_equal[lane]);
        if (lane == 0) {
            sh_mine[0] = m;
            sh_mine[1] = e;
        }
    }
    sync_all();
    more = same = 0;
    for (int q = 0; q < rank; ++q) {
        const uint32_t *o = of_rank(&sh_mine[0], q);
        more += o[0];
        same += o[1];
    }
    more += __reduce_add_sync(0xffffffffu, lane < warp ? sh_above[lane] : 0u);
    same += __reduce_add_sync(0xffffffffu, lane < warp ? sh_equal[lane] : 0u);
    const uint32_t before = (1u << lane) - 1u;
    each_key(from + lane, to, 32, [&](int i, uint32_t k, bool in) {
        const uint32_t ups = __ballot_sync(0xffffffffu, in && k > known), eqs = __ballot_sync(0xffffffffu, in && k == known);
        const uint32_t m = more + __popc(ups & before), s = same + __popc(eqs & before);
        if (in && (k > known || (k == known && s < want))) index[a.sinks + static_cast<int>(m + min(s, want))] = a.sinks + first + i;
        more += __popc(ups);
        same += __popc(eqs);
    });
    if constexpr (CLUSTER) cluster.sync();  // no CTA leaves while another may read its counts
}

// ------------------------------------------------------------------ their move
// A warp makes a tile of 16 tokens of one head: a lane brings the words of the new tile that it stores, from wherever their
// tokens lie. A token's K words are the same there and here; a V word holds two tokens' halves. The tokens' sums go along.
// Four sequences of up to 65536 tokens, 8 kv heads of 128, to 16000: 34 us, 163 MB read and 34 written of the 66 (the others
// stay in L2), 87% of the copy rate. The floor counts the kept tokens alone, 66 MB each way, but a V word holds two tokens'
// halves and a 32-byte sector eight tokens', so that a quarter of the tokens takes nearly all of V's sectors.
constexpr int kGatherWarps = 8;
template <int NB> __global__ void __launch_bounds__(kGatherWarps * 32) kv_gather_kernel(KeepArgs a, int64_t n_jobs) {
    using G = KvGeom<NB>;
    constexpr int V = G::kVec;
    struct __align__(4 * V) Words {
        uint32_t w[V];
    };
    const int lane = threadIdx.x & 31;
    const int64_t job = static_cast<int64_t>(blockIdx.x) * kGatherWarps + (threadIdx.x >> 5);
    block_op_wait();
    block_op_release();
    if (job >= n_jobs) return;
    const int item = a.by_tiles.div(static_cast<int>(job)), tile = a.by_tiles.mod(static_cast<int>(job), item);
    const int seq = a.by_heads.div(item), kvh = a.by_heads.mod(item, seq);
    const int t0 = tile * kKvSlab;
    // here, where one thread alone looks at a sequence's length any more: len_out may be kv_len
    if (a.len_out && tile == 0 && kvh == 0 && lane == 0) {
        const int n = a.kv_len[seq];
        a.len_out[seq] = keep_bad(a, n) ? -1 : min(n, a.budget);
    }
    // lanes 0 .. 15: where the tile's tokens are
    const uint8_t *src = nullptr;
    int r = 0;
    bool some = false, wrong = false;
    float sum = 0.0f;
    if (lane < kKvSlab && t0 + lane < a.budget) {
        const int t = a.index[static_cast<int64_t>(item) * a.budget + t0 + lane];
        some = t >= 0;
        if (a.sums_out && some) sum = a.sums[static_cast<int64_t>(item) * a.sums_stride + t];
        if (some) {
            const int slab = t / kKvSlab, slot = a.from_page_tiles.div(slab);
            const int page = a.from.table[static_cast<int64_t>(seq) * a.from.max_pages + slot];
            wrong = page < 0 || page >= a.from.n_pages;
            r = t % kKvSlab;
            if (!wrong)
                src = a.from.pages + page * a.from.page_bytes +
                      (static_cast<int64_t>(kvh) * static_cast<int>(a.from_page_tiles.d) + a.from_page_tiles.mod(slab, slot)) * G::kTileBytes;
        }
    }
    const bool put_sum = a.sums_out && lane < kKvSlab && t0 + lane < a.budget;
    float *sum_to = a.sums_out + static_cast<int64_t>(item) * a.sums_out_stride + t0 + lane;
    if (!__any_sync(0xffffffffu, some)) {
        if (put_sum) *sum_to = 0.0f;
        return;
    }
    const int slot = a.to_page_tiles.div(tile), page = a.to.table[static_cast<int64_t>(seq) * a.to.max_pages + slot];
    const bool lost = page < 0 || page >= a.to.n_pages;
    if ((wrong || (lost && lane == 0)) && a.status) *a.status = 1;
    if (lost) {
        if (put_sum) *sum_to = sum;
        return;
    }
    uint8_t *dst = a.to.pages + page * a.to.page_bytes +
                   (static_cast<int64_t>(kvh) * static_cast<int>(a.to_page_tiles.d) + a.to_page_tiles.mod(tile, slot)) * G::kTileBytes;
    const uint32_t nans = __ballot_sync(0xffffffffu, wrong);
    const auto tile_of = [&](int tok) {
        return reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), tok));
    };
    Words k[2][NB / V], v[2][NB / V][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int tok = 8 * h + (lane >> 2);
        const uint8_t *p = tile_of(tok);
        const int at = __shfl_sync(0xffffffffu, r, tok);
#pragma unroll
        for (int b = 0; b < NB / V; ++b) {
            k[h][b] = Words{};
            if (p) k[h][b] = *reinterpret_cast<const Words *>(p + G::k_word(at, b * V, lane & 3) * 4);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int two = 8 * h + 2 * (lane & 3) + i;
            const uint8_t *q = tile_of(two);
            const int to = __shfl_sync(0xffffffffu, r, two);
#pragma unroll
            for (int b = 0; b < NB / V; ++b) {
                v[h][b][i] = Words{};
                if (q) {
                    v[h][b][i] = *reinterpret_cast<const Words *>(q + G::kVAt + (G::v_half(to, b * V, lane >> 2) >> 1) * 4);
#pragma unroll
                    for (int x = 0; x < V; ++x) v[h][b][i].w[x] = (v[h][b][i].w[x] >> (16 * (to & 1)) & 0xffffu) << (16 * i);
                }
            }
        }
    }
    // scales: word (pair of tokens, block), K's then V's
    constexpr int kScaleWords = 16 * NB, kPer = (kScaleWords + 31) / 32;
    uint32_t d[kPer];
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
        const int word = 32 * c + lane, which = word / (8 * NB), pair = word % (8 * NB) / NB, b = word % NB;
        d[c] = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint8_t *p = tile_of(2 * pair + i);
            const int at = __shfl_sync(0xffffffffu, r, 2 * pair + i);
            uint32_t x = nans >> (2 * pair + i) & 1u ? 0x7fffu : 0u;
            if (p && word < kScaleWords) x = reinterpret_cast<const uint16_t *>(p + G::kKScaleAt + which * G::kScaleBytes)[G::scale_half(at, b)];
            d[c] |= x << (16 * i);
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < NB / V; ++b) {
            const int at = (h * (NB / V) + b) * 32 * V + lane * V;
            Words x;
#pragma unroll
            for (int w = 0; w < V; ++w) x.w[w] = v[h][b][0].w[w] | v[h][b][1].w[w];
            *reinterpret_cast<Words *>(dst + at * 4) = k[h][b];
            *reinterpret_cast<Words *>(dst + G::kVAt + at * 4) = x;
        }
#pragma unroll
    for (int c = 0; c < kPer; ++c)
        if (32 * c + lane < kScaleWords) reinterpret_cast<uint32_t *>(dst + G::kKScaleAt)[32 * c + lane] = d[c];
    if (put_sum) *sum_to = sum;
}

// ------------------------------------------------------------------ the accepted path
// A CTA for a kv head of a sequence. The path rises, so number j of it is j or more: 16 tokens at a time are read before they
// are written, and none that is still to be read is written over. 2.0 to 2.5 us for one path or 48: the latency of four loads
// one after another (path, page, codes, and the store).
struct AcceptArgs {
    KvView c;
    FastDiv by_heads, by_page;
    const int32_t *base, *path, *n_path;
    int32_t *len_out, *status;
    float *sums;
    int64_t sums_stride;
    int64_t room;  // tokens that the sums have room for, and that a place is a number of
    int32_t max_path;
};
constexpr int kAcceptWarps = 8, kAcceptThreads = kAcceptWarps * 32, kMostPath = 1024;
template <int NB> __global__ void __launch_bounds__(kAcceptThreads) kv_accept_kernel(AcceptArgs a) {
    using G = KvGeom<NB>;
    __shared__ int sh_path[kMostPath], sh_from[kMostPath], sh_to[kMostPath];  // the path, and the pages from and to which it moves
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    block_op_wait();
    block_op_release();
    const int seq = a.by_heads.div(blockIdx.x), kvh = a.by_heads.mod(blockIdx.x, seq);
    const int base = a.base[seq], n = a.n_path[seq];
    const int32_t *path = a.path + static_cast<int64_t>(seq) * a.max_path;
    const int64_t room = min(static_cast<int64_t>(a.c.max_pages) * a.c.page_tokens, a.room);
    bool bad = base < 0 || n < 0 || n > a.max_path;
    const int32_t *table = a.c.table + static_cast<int64_t>(seq) * a.c.max_pages;
    if (!bad) {
        for (int j = tid; j < n; j += kAcceptThreads) {
            const int p = path[j], prev = j > 0 ? path[j - 1] : -1;
            sh_path[j] = p;
            if (p <= prev || prev < -1 || static_cast<int64_t>(base) + p >= room) {
                bad = true;
                break;
            }
            const int from = a.by_page.div(base + p), to = a.by_page.div(base + j);
            sh_from[j] = table[from];
            sh_to[j] = table[to];
            if (p != j) bad |= sh_from[j] < 0 || sh_from[j] >= a.c.n_pages || sh_to[j] < 0 || sh_to[j] >= a.c.n_pages;
        }
    }
    bad = __syncthreads_or(bad);
    if (kvh == 0 && tid == 0) {
        if (a.len_out) a.len_out[seq] = bad ? -1 : base + n;
        if (bad && a.status) *a.status = 1;
    }
    if (bad) return;
    const int64_t head = static_cast<int64_t>(kvh) * (a.c.page_tokens / kKvSlab);
    const auto tile_of = [&](int page, int tok) {
        return a.c.pages + page * a.c.page_bytes + (head + tok / kKvSlab) * G::kTileBytes;
    };
    float *sums = a.sums ? a.sums + static_cast<int64_t>(blockIdx.x) * a.sums_stride + base : nullptr;
    constexpr int kAtOnce = 2 * kAcceptWarps;
    for (int j0 = 0; j0 < n; j0 += kAtOnce) {
        uint32_t k[2];
        uint16_t v[2][(8 * NB + 31) / 32], d[2];
        float sum[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = j0 + warp + i * kAcceptWarps;
            if (j >= n || sh_path[j] == j) continue;
            const int at = a.by_page.mod(base + sh_path[j], a.by_page.div(base + sh_path[j])), r = at % kKvSlab;
            const uint8_t *src = tile_of(sh_from[j], at);
            if (sums) sum[i] = sums[sh_path[j]];
            if (lane < 4 * NB) k[i] = reinterpret_cast<const uint32_t *>(src)[G::k_word(r, lane >> 2, lane & 3)];
#pragma unroll
            for (int c = 0; c < (8 * NB + 31) / 32; ++c)
                if (32 * c + lane < 8 * NB) v[i][c] = reinterpret_cast<const uint16_t *>(src + G::kVAt)[G::v_half(r, (32 * c + lane) >> 3, lane & 7)];
            if (lane < 2 * NB)
                d[i] = reinterpret_cast<const uint16_t *>(src + (lane < NB ? G::kKScaleAt : G::kVScaleAt))[G::scale_half(r, lane % NB)];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = j0 + warp + i * kAcceptWarps;
            if (j >= n || sh_path[j] == j) continue;
            const int at = a.by_page.mod(base + j, a.by_page.div(base + j)), r = at % kKvSlab;
            uint8_t *dst = tile_of(sh_to[j], at);
            if (sums && lane == 0) sums[j] = sum[i];
            if (lane < 4 * NB) reinterpret_cast<uint32_t *>(dst)[G::k_word(r, lane >> 2, lane & 3)] = k[i];
#pragma unroll
            for (int c = 0; c < (8 * NB + 31) / 32; ++c)
                if (32 * c + lane < 8 * NB) reinterpret_cast<uint16_t *>(dst + G::kVAt)[G::v_half(r, (32 * c + lane) >> 3, lane & 7)] = v[i][c];
            if (lane < 2 * NB)
                reinterpret_cast<uint16_t *>(dst + (lane < NB ? G::kKScaleAt : G::kVScaleAt))[G::scale_half(r, lane % NB)] = d[i];
        }
        __syncthreads();
    }
}

// Whether n ints at p and m at q share a byte (a null pointer has none).
bool ints_overlap(const int32_t *p, int64_t n, const int32_t *q, int64_t m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && a < b + 4 * static_cast<uintptr_t>(m) && b < a + 4 * static_cast<uintptr_t>(n);
}

template <int NB> cudaError_t launch_gather(const KeepArgs &a, int64_t jobs, cudaStream_t st) {
    return launch_block_op(kv_gather_kernel<NB>, dim3(static_cast<unsigned>((jobs + kGatherWarps - 1) / kGatherWarps)), dim3(kGatherWarps * 32),
                           0, st, a, jobs);
}
template <int NB> cudaError_t launch_accept(const AcceptArgs &a, cudaStream_t st) {
    return launch_block_op(kv_accept_kernel<NB>, dim3(static_cast<unsigned>(a.c.n_seq) * a.c.n_kv_heads), dim3(kAcceptThreads), 0, st, a);
}
cudaError_t launch_pick(KeepArgs a, int64_t items, cudaStream_t st) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // a CTA an SM, so clusters of no more than fill the device once, unless their sums would be read again (32 kv heads of 65536
    // tokens: eight CTAs each 33.6 us, four 18.0)
    int ranks = 1;
    while (ranks < kPickCluster && a.max_kv_len / ranks > kPickEach && (items * ranks * 2 <= sms || a.max_kv_len / ranks > kPickHeld)) ranks *= 2;
    a.held = std::min(a.max_kv_len / ranks + 1, kPickHeld);
    const size_t smem = static_cast<size_t>(a.held) * 4;
    if (ranks == 1) {
        e = smem_limit_raised<&kv_pick_kernel<false>>();
        if (e != cudaSuccess) return e;
        return launch_block_op(&kv_pick_kernel<false>, dim3(static_cast<unsigned>(items)), dim3(kPickThreads), smem, st, a);
    }
    e = smem_limit_raised<&kv_pick_kernel<true>>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(items * ranks));
    cfg.blockDim = dim3(kPickThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kv_pick_kernel<true>, a);
}

}  // namespace
}  // namespace zdmmv

using namespace zdmmv;

extern "C" {

zdmmv_status zdmmv_kv_evict_q4_0(const zdmmv_kv_cache *from, const zdmmv_kv_cache *to, const zdmmv_kv_evict_args *args,
                                 zdmmv_stream_t stream) {
    if (!args) return ZDMMV_ERR_NULL;
    KeepArgs a{};
    zdmmv_status st = kv_check(from, &a.from);
    if (st == ZDMMV_OK) st = kv_check(to, &a.to);
    if (st != ZDMMV_OK) return st;
    const zdmmv_kv_evict_args &g = *args;
    const int64_t items = static_cast<int64_t>(a.from.n_seq) * a.from.n_kv_heads;
    const int64_t tiles = (static_cast<int64_t>(g.budget) + kKvSlab - 1) / kKvSlab, jobs = items * tiles;
    if (from->n_seq != to->n_seq || from->n_kv_heads != to->n_kv_heads || from->head_dim != to->head_dim || g.max_kv_len < 0 ||
        g.max_kv_len > kPickMost || g.budget < 1 || g.budget > kPickMost || g.sinks < 0 || g.recent < 0 || static_cast<int64_t>(g.sinks) + g.recent > g.budget ||
        g.budget > static_cast<int64_t>(a.to.max_pages) * a.to.page_tokens || jobs > 0x7fffff00 || items * kPickCluster > 0x7fffff00)
        return ZDMMV_ERR_SHAPE;
    if (!g.kv_len || !g.sums || !g.index) return ZDMMV_ERR_NULL;
    if (g.sums_stride < g.max_kv_len || (g.sums_out && (g.sums_out_stride < g.budget || g.sums_out == g.sums))) return ZDMMV_ERR_SHAPE;
    if (kv_misaligned(g.kv_len, 4) || kv_misaligned(g.sums, 4) || kv_misaligned(g.index, 4) || kv_misaligned(g.sums_out, 4) ||
        kv_misaligned(g.len_out, 4) || kv_misaligned(g.status_dev, 4))
        return ZDMMV_ERR_ALIGN;
    if (from->pages == to->pages && from->page_table == to->page_table) return ZDMMV_ERR_SHAPE;
    if (g.len_out != g.kv_len && ints_overlap(g.len_out, from->n_seq, g.kv_len, from->n_seq)) return ZDMMV_ERR_SHAPE;
    a.by_heads = FastDiv::of(from->n_kv_heads);
    a.from_page_tiles = FastDiv::of(from->page_tokens / kKvSlab);
    a.to_page_tiles = FastDiv::of(to->page_tokens / kKvSlab);
    a.by_tiles = FastDiv::of(static_cast<int32_t>(tiles));
    a.kv_len = g.kv_len; a.sums = g.sums; a.index = g.index; a.sums_out = g.sums_out; a.len_out = g.len_out; a.status = g.status_dev;
    a.sums_stride = g.sums_stride; a.sums_out_stride = g.sums_out_stride;
    a.max_kv_len = g.max_kv_len; a.budget = g.budget; a.sinks = g.sinks; a.recent = g.recent;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch_pick(a, items, s);
    if (e != cudaSuccess) return ZDMMV_ERR_CUDA;
    e = cudaErrorInvalidValue;
    switch (kv_blocks(from->head_dim)) {
    case 2: e = launch_gather<2>(a, jobs, s); break;
    case 3: e = launch_gather<3>(a, jobs, s); break;
    case 4: e = launch_gather<4>(a, jobs, s); break;
    case 6: e = launch_gather<6>(a, jobs, s); break;
    case 8: e = launch_gather<8>(a, jobs, s); break;
    }
    return e == cudaSuccess ? ZDMMV_OK : ZDMMV_ERR_CUDA;
}

zdmmv_status zdmmv_kv_accept_q4_0(const zdmmv_kv_cache *cache, const zdmmv_kv_accept_args *args, zdmmv_stream_t stream) {
    if (!args) return ZDMMV_ERR_NULL;
    AcceptArgs a{};
    const zdmmv_status st = kv_check(cache, &a.c);
    if (st != ZDMMV_OK) return st;
    const zdmmv_kv_accept_args &g = *args;
    if (g.max_path < 1 || g.max_path > kMostPath || static_cast<int64_t>(a.c.n_seq) * a.c.n_kv_heads > 0x7fffff00) return ZDMMV_ERR_SHAPE;
    if (!g.base || !g.path || !g.n_path) return ZDMMV_ERR_NULL;
    if (g.sums && (g.sums_stride < g.max_path || g.sums_len < g.max_path || g.sums_stride < g.sums_len)) return ZDMMV_ERR_SHAPE;
    if (kv_misaligned(g.base, 4) || kv_misaligned(g.path, 4) || kv_misaligned(g.n_path, 4) || kv_misaligned(g.len_out, 4) ||
        kv_misaligned(g.status_dev, 4) || kv_misaligned(g.sums, 4))
        return ZDMMV_ERR_ALIGN;
    // a sequence's heads have a CTA each, which all read what the first one's would write over
    if (ints_overlap(g.len_out, a.c.n_seq, g.base, a.c.n_seq) || ints_overlap(g.len_out, a.c.n_seq, g.n_path, a.c.n_seq) ||
        ints_overlap(g.len_out, a.c.n_seq, g.path, static_cast<int64_t>(a.c.n_seq) * g.max_path))
        return ZDMMV_ERR_SHAPE;
    a.by_heads = FastDiv::of(cache->n_kv_heads);
    a.by_page = FastDiv::of(cache->page_tokens);
    a.base = g.base; a.path = g.path; a.n_path = g.n_path; a.len_out = g.len_out; a.status = g.status_dev;
    a.max_path = g.max_path;
    a.sums = g.sums; a.sums_stride = g.sums_stride;
    a.room = g.sums ? std::min<int64_t>(0x7fffff00, g.sums_len) : 0x7fffff00;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
    switch (kv_blocks(cache->head_dim)) {
    case 2: e = launch_accept<2>(a, s); break;
    case 3: e = launch_accept<3>(a, s); break;
    case 4: e = launch_accept<4>(a, s); break;
    case 6: e = launch_accept<6>(a, s); break;
    case 8: e = launch_accept<8>(a, s); break;
    }
    return e == cudaSuccess ? ZDMMV_OK : ZDMMV_ERR_CUDA;
}

}  // extern "C"
