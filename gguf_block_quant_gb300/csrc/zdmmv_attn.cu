// zdmmv_attn.cu -- zdmmv_attn_q4_0: argument checks and the plan of the launch
// (the kernels: zdmmv_attn.cuh).
#include <algorithm>
#include <cmath>

#include "zdmmv_attn.cuh"
#include "zdmmv_internal.h"

namespace zdmmv {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Up to four columns a kv head of a sequence take the narrow form, up to 16 the wide one, more the form on tcgen05 or (heads
// past 128 dimensions) a shared ring. The grid is (items) x (splits of their tokens): as many as run at once; up to four times that for several sequences, whose lengths may
// differ, while a split has kRaggedChunk tiles; whole waves of
// CTAs for more than 16 columns. Long sequences' decoding, from kWalkSteps steps
// a CTA on, goes by the lengths instead (AttnWalk): 64 of up to 16384 tokens 109 us with the grid and 96 so, 64 of 4096 71
// and 68, but 64 of 1000 22.4 and 24.6.
constexpr int kWalkSteps = 12;
constexpr int kRaggedChunk = 128;
constexpr int kEnds = 8;
constexpr int kTallEnds = 32, kTallJoin = 1;  // ... of the form on tcgen05: its start, and the join's loads of four parts for 2560 values
constexpr int kCounters = ZDMMV_ATTN_COUNTER_BYTES / 4;

bool attn_plan(const KvView &c, int head_dim, int n_q_heads, int max_q_len, int64_t max_tokens, AttnPlan *out) {
    static const int sms = [] {
        int dev = 0, n = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return 152;
        return n;
    }();
    AttnPlan p{};
    const int64_t columns = static_cast<int64_t>(max_q_len) * (n_q_heads / c.n_kv_heads);
    const int nb = kv_blocks(head_dim);
    p.wc = columns <= 16 ? 1 : (columns <= 32 ? 2 : (columns <= 64 ? 4 : 8));
    p.nt = p.wc > 4 ? attn_prompt_nt(nb) : (columns <= 8 ? 1 : 2);
    p.tall = columns > kTallColumns && nb <= kTallBlocks;
    if (p.tall) {  // 128 columns
        p.wc = 8;
        p.nt = 2;
    } else if (p.wc > 4) {
        // the fewest column tiles, the columns evenly over them
        const int64_t tiles_of = ceil_div(columns, 8 * p.nt * p.wc);
        p.wc = static_cast<int>(ceil_div(ceil_div(columns, tiles_of), 8 * p.nt));
    }
    p.cols = columns <= kNarrowCols ? kNarrowCols : 8 * p.nt * p.wc;
    const int64_t n_ct = ceil_div(columns, p.cols);
    p.items = static_cast<int64_t>(c.n_seq) * c.n_kv_heads * n_ct;
    const int64_t tiles = std::max<int64_t>(1, ceil_div(max_tokens, kKvSlab));
    const int64_t steps = p.items * ceil_div(tiles, kStepTiles);
    if (steps > 0x7fffffff || columns > 0x7fffff00) return false;
    p.n_ct = static_cast<int>(n_ct);
    p.round = p.tall ? 8 : 2;  // whole tiles of 128 tokens, whole ring slots
    const int64_t slots = static_cast<int64_t>(sms) * (p.wc > 1 ? 1 : attn_ctas_per_sm(nb, p.nt));
    if (p.wc == 1 && c.n_seq > 1 && steps > kWalkSteps * slots) {
        p.ctas = static_cast<int>(std::min<int64_t>(slots, kCounters));
        p.parts = steps > p.items ? 2 * p.ctas : 0;  // an item of one step is never shared
    } else {
        int64_t splits = p.items > kCounters ? 1 : std::max<int64_t>(1, slots / p.items);
        if (p.wc == 1 && c.n_seq > 1 && p.items <= kCounters)
            splits = std::max(splits, std::min(ceil_div(4 * slots, p.items), ceil_div(tiles, kRaggedChunk)));
        int64_t most = std::min(splits, ceil_div(tiles, kMinChunk));
        p.parts = most;
        if (p.wc > 1 && p.items <= kCounters) {
            // whole waves of CTAs: the split whose waves cost least, a CTA's start and end as much as kEnds tiles
            p.parts = std::min(4 * splits, ceil_div(tiles, kMinChunk));
            const int64_t cols = std::min<int64_t>(columns, p.cols);
            const auto cost = [&](int64_t n) {
                const int64_t ends = p.tall ? kTallEnds + kTallJoin * ceil_div(cols * head_dim, 2560) * ceil_div(n, 4) : kEnds;
                return ceil_div(p.items * n, slots) * (ceil_div(tiles, n) + ends);
            };
            for (int64_t n = most / 2; p.tall && n > 1; n /= 2)
                if (cost(n) < cost(most)) most = n;
            for (int waves = 1; waves <= 4; ++waves) {
                const int64_t n = std::min(std::max<int64_t>(1, waves * slots / p.items), p.parts);
                if (cost(n) < cost(most)) most = n;
            }
        }
        p.chunk = static_cast<int>(std::max<int64_t>(kMinChunk, ceil_div(ceil_div(tiles, most), p.round) * p.round));
        p.n_split = static_cast<int>(most);
        p.parts = p.parts > 1 ? p.items * p.parts : 0;
    }
    *out = p;
    return true;
}

size_t attn_workspace(const AttnPlan &p, int head_dim) {
    if (p.parts == 0) return 0;
    return ZDMMV_ATTN_COUNTER_BYTES + static_cast<size_t>(p.parts) * p.cols * (head_dim + 2) * 4;
}

}  // namespace
}  // namespace zdmmv

using namespace zdmmv;

extern "C" {

size_t zdmmv_attn_q4_0_workspace_bytes(const zdmmv_kv_cache *cache, int n_q_heads, int max_q_len, int max_kv_len) {
    KvView c{};
    AttnPlan p{};
    if (kv_check(cache, &c) != ZDMMV_OK || n_q_heads < 1 || n_q_heads > 65535 || n_q_heads % c.n_kv_heads ||
        max_q_len < 1 || max_kv_len < 0 || !attn_plan(c, cache->head_dim, n_q_heads, max_q_len, max_kv_len, &p))
        return 0;
    return attn_workspace(p, cache->head_dim);
}

zdmmv_status zdmmv_attn_q4_0(const zdmmv_kv_cache *cache, const zdmmv_attn_args *args, zdmmv_stream_t stream) {
    if (!args) return ZDMMV_ERR_NULL;
    AttnArgs a{};
    const zdmmv_status st = kv_check(cache, &a.c);
    if (st != ZDMMV_OK) return st;
    const zdmmv_attn_args &g = *args;
    AttnPlan p{}, whole{};
    if (g.n_tok < 0 || g.n_q_heads < 1 || g.n_q_heads > 65535 || g.n_q_heads % cache->n_kv_heads || g.max_q_len < 1 ||
        g.max_kv_len < 0 || g.window < 0 || !std::isfinite(g.scale))
        return ZDMMV_ERR_SHAPE;
    // with a window, no column tile sees more than the window and its own new tokens
    const int64_t seen = g.window > 0 ? std::min<int64_t>(g.max_kv_len, static_cast<int64_t>(g.window) + g.max_q_len + kKvSlab)
                                      : g.max_kv_len;
    if (!attn_plan(a.c, cache->head_dim, g.n_q_heads, g.max_q_len, g.max_kv_len, &whole) ||
        !attn_plan(a.c, cache->head_dim, g.n_q_heads, g.max_q_len, seen, &p))
        return ZDMMV_ERR_SHAPE;
    if (g.n_tok == 0) return ZDMMV_OK;
    if (!g.q || !g.q_start || !g.kv_len || !g.out) return ZDMMV_ERR_NULL;
    if (g.q_stride < static_cast<int64_t>(g.n_q_heads) * cache->head_dim) return ZDMMV_ERR_SHAPE;
    if (kv_misaligned(g.q, 16) || kv_misaligned(g.out, 16) || kv_misaligned(g.workspace, 16) ||
        kv_misaligned(g.q_start, 4) || kv_misaligned(g.kv_len, 4) || kv_misaligned(g.status_dev, 4) || g.q_stride % 4)
        return ZDMMV_ERR_ALIGN;
    const size_t need = attn_workspace(whole, cache->head_dim);
    if (need && !g.workspace) return ZDMMV_ERR_NULL;
    if (g.workspace_bytes < need) return ZDMMV_ERR_SIZE;
    a.q = g.q; a.q_start = g.q_start; a.kv_len = g.kv_len; a.out = g.out; a.status = g.status_dev;
    a.fault = current_fault_word();
    if (!a.fault) return ZDMMV_ERR_CUDA;
    a.q_stride = g.q_stride;
    a.n_tok = g.n_tok; a.n_q_heads = g.n_q_heads; a.group = g.n_q_heads / cache->n_kv_heads;
    a.max_q_len = g.max_q_len; a.max_kv_len = g.max_kv_len; a.window = g.window;
    a.scale_log2 = g.scale * 1.44269504088896340736f;
    a.by_ct = FastDiv::of(p.n_ct);
    a.by_heads = FastDiv::of(cache->n_kv_heads);
    a.by_group = FastDiv::of(a.group);
    a.by_page_tiles = FastDiv::of(cache->page_tokens / kKvSlab);
    a.by_split = FastDiv::of(std::max(1, p.n_split));
    a.n_ct = p.n_ct; a.n_split = p.n_split; a.chunk = p.chunk; a.round = p.round; a.wc = p.wc;
    a.count = static_cast<uint32_t *>(g.workspace);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(g.workspace) + ZDMMV_ATTN_COUNTER_BYTES);
    a.part_ml = reinterpret_cast<float2 *>(a.part + p.parts * p.cols * cache->head_dim);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
    switch (kv_blocks(cache->head_dim)) {
    case 2: e = launch_attn<2>(a, p, s); break;
    case 3: e = launch_attn<3>(a, p, s); break;
    case 4: e = launch_attn<4>(a, p, s); break;
    case 6: e = launch_attn<6>(a, p, s); break;
    case 8: e = launch_attn<8>(a, p, s); break;
    }
    return e == cudaSuccess ? ZDMMV_OK : ZDMMV_ERR_CUDA;
}

}  // extern "C"
