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
// past 128 dimensions) a shared ring. The grid is (items) x (splits of their tokens): as many as run at once; up to four
// times that for several sequences, whose lengths may differ, while a split has kRaggedChunk tiles; whole waves of CTAs for
// more than 16 columns. Long sequences' decoding, from kWalkSteps steps a CTA on, goes by the lengths instead (AttnWalk): 64
// of up to 16384 tokens 109 us with the grid and 96 so, 64 of 4096 71 and 68, but 64 of 1000 22.4 and 24.6.
// The plan is made for what a window leaves to see of the longest sequence, and the workspace is checked for that plan.
constexpr int kWalkSteps = 12;
constexpr int kRaggedChunk = 128;
constexpr int kEnds = 8;
constexpr int kPromptCols = 128;  // of a CTA of the form on tcgen05
constexpr int kTallEnds = 32, kTallJoin = 1;  // ... of the form on tcgen05: its start, and the join's loads of four parts for 2560 values
constexpr int kMostTokens = 0x7fffff00;  // so that a tile's end past the last token is a number too
constexpr int kCounters = ZDMMV_ATTN_COUNTER_BYTES / 4;

int device_sms() {
    static const int sms = [] {
        int dev = 0, n = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return 152;
        return n;
    }();
    return sms;
}

// How the columns of a kv head of a sequence lie over CTAs: the kernel's form, the columns of a CTA, its column tiles, and
// the CTAs that the device runs at once.
struct AttnLayout {
    int nt, wc, cols;
    bool tall;
    int64_t n_ct, slots;
};
AttnLayout attn_layout(int64_t columns, int head_dim) {
    AttnLayout f{};
    const int nb = kv_blocks(head_dim);
    f.wc = columns <= 16 ? 1 : (columns <= 32 ? 2 : (columns <= 64 ? 4 : 8));
    f.nt = f.wc > 4 ? attn_prompt_nt(nb) : (columns <= 8 ? 1 : 2);
    f.tall = columns > kTallColumns && nb <= kTallBlocks;
    if (f.tall) {  // kPromptCols
        f.wc = 8;
        f.nt = 2;
    } else if (f.wc > 4) {
        // the fewest column tiles, the columns evenly over them
        const int64_t tiles_of = ceil_div(columns, 8 * f.nt * f.wc);
        f.wc = static_cast<int>(ceil_div(ceil_div(columns, tiles_of), 8 * f.nt));
    }
    f.cols = columns <= kNarrowCols ? kNarrowCols : 8 * f.nt * f.wc;
    f.n_ct = ceil_div(columns, f.cols);
    f.slots = static_cast<int64_t>(device_sms()) * (f.wc > 1 ? 1 : attn_ctas_per_sm(nb, f.nt));
    return f;
}

int64_t attn_tiles(int64_t tokens) { return std::max<int64_t>(1, ceil_div(tokens, kKvSlab)); }

// Whether `items` of `tiles` tiles each are walked by equal stretches, and the parts that this takes (an item of one step is
// never shared).
bool attn_walks(const AttnLayout &f, int n_seq, int64_t items, int64_t tiles) {
    return f.wc == 1 && n_seq > 1 && items * ceil_div(tiles, kStepTiles) > kWalkSteps * f.slots;
}
int64_t attn_walk_ctas(const AttnLayout &f) { return std::min<int64_t>(f.slots, kCounters); }
int64_t attn_walk_parts(const AttnLayout &f, int64_t tiles) { return tiles > kStepTiles ? 2 * attn_walk_ctas(f) : 0; }

// The grid's splits of an item: the number taken, or the most that is taken for this many tiles or fewer. Both rise with the
// tiles.
int64_t attn_own_splits(const AttnLayout &f, int n_seq, int64_t items, int64_t tiles) {
    if (items > kCounters) return 1;
    int64_t splits = std::max<int64_t>(1, f.slots / items);
    if (n_seq > 1) splits = std::max(splits, std::min(ceil_div(4 * f.slots, items), ceil_div(tiles, kRaggedChunk)));
    return std::min(splits, ceil_div(tiles, kMinChunk));
}
int64_t attn_most_shared_splits(const AttnLayout &f, int64_t items, int64_t tiles) {
    if (items > kCounters) return 1;
    return std::min(std::max<int64_t>(1, 4 * f.slots / items), ceil_div(tiles, kMinChunk));
}
// Whole waves of CTAs: the split whose waves cost least, a CTA's start and end as much as kEnds tiles.
int64_t attn_shared_splits(const AttnLayout &f, int64_t items, int64_t tiles, int64_t columns, int head_dim) {
    if (items > kCounters) return 1;
    const int64_t splits = std::max<int64_t>(1, f.slots / items), most = std::min(4 * splits, ceil_div(tiles, kMinChunk));
    const int64_t cols = std::min<int64_t>(columns, f.cols);
    const auto cost = [&](int64_t n) {
        const int64_t ends = f.tall ? kTallEnds + kTallJoin * ceil_div(cols * head_dim, 2560) * ceil_div(n, 4) : kEnds;
        return ceil_div(items * n, f.slots) * (ceil_div(tiles, n) + ends);
    };
    int64_t best = std::min(splits, ceil_div(tiles, kMinChunk));
    for (int64_t n = best / 2; f.tall && n > 1; n /= 2)
        if (cost(n) < cost(best)) best = n;
    for (int waves = 1; waves <= 4; ++waves) {
        const int64_t n = std::min(std::max<int64_t>(1, waves * f.slots / items), most);
        if (cost(n) < cost(best)) best = n;
    }
    return best;
}

bool attn_plan(const KvView &c, int head_dim, int n_q_heads, int max_q_len, int64_t max_tokens, AttnPlan *out) {
    AttnPlan p{};
    const int64_t columns = static_cast<int64_t>(max_q_len) * (n_q_heads / c.n_kv_heads);
    if (columns > 0x7fffff00) return false;
    const AttnLayout f = attn_layout(columns, head_dim);
    p.nt = f.nt;
    p.wc = f.wc;
    p.cols = f.cols;
    p.tall = f.tall;
    p.items = static_cast<int64_t>(c.n_seq) * c.n_kv_heads * f.n_ct;
    const int64_t tiles = attn_tiles(max_tokens);
    if (p.items * ceil_div(tiles, kStepTiles) > 0x7fffffff) return false;
    p.n_ct = static_cast<int>(f.n_ct);
    p.round = p.tall ? 8 : 2;  // whole tiles of 128 tokens, whole ring slots
    if (attn_walks(f, c.n_seq, p.items, tiles)) {
        p.ctas = static_cast<int>(attn_walk_ctas(f));
        p.parts = attn_walk_parts(f, tiles);
    } else {
        const int64_t splits = f.wc == 1 ? attn_own_splits(f, c.n_seq, p.items, tiles)
                                         : attn_shared_splits(f, p.items, tiles, columns, head_dim);
        p.chunk = static_cast<int>(std::max<int64_t>(kMinChunk, ceil_div(ceil_div(tiles, splits), p.round) * p.round));
        p.n_split = static_cast<int>(splits);
        p.parts = splits > 1 ? p.items * splits : 0;
    }
    *out = p;
    return true;
}

size_t attn_parts_bytes(int64_t parts, int64_t cols, int head_dim) {
    return parts == 0 ? 0 : ZDMMV_ATTN_COUNTER_BYTES + static_cast<size_t>(parts * cols) * (head_dim + 2) * 4;
}

// What any call with this layout and up to `tokens` tokens (all of a sequence, or what a window leaves of it) needs. The need
// does not rise with the length by itself: 384 items are cut into 768 parts of the grid at 2100 tokens, and walked in 608 at
// 16384. Each way's does, so the most is the longest grid's or the walk's.
size_t attn_layout_bytes(const AttnLayout &f, const KvView &c, int head_dim, int64_t tokens) {
    const int64_t items = static_cast<int64_t>(c.n_seq) * c.n_kv_heads * f.n_ct;
    int64_t tiles = attn_tiles(tokens), parts = 0;
    if (attn_walks(f, c.n_seq, items, tiles)) {
        parts = attn_walk_parts(f, tiles);
        tiles = kWalkSteps * f.slots / items * kStepTiles;  // the longest that are not walked
    }
    const int64_t splits = tiles == 0 ? 1 : (f.wc == 1 ? attn_own_splits(f, c.n_seq, items, tiles) : attn_most_shared_splits(f, items, tiles));
    if (splits > 1) parts = std::max(parts, items * splits);
    return attn_parts_bytes(parts, f.cols, head_dim);
}

// ... and with `columns` or fewer, which may take any other form. Those of up to 16 columns have one column tile and are taken
// one by one; of the others, CTAs of `top` columns or fewer, at most four times as many as run at once, and no more than there
// are steps.
size_t attn_bounds_bytes(const KvView &c, int head_dim, int group, int64_t columns, int64_t tokens) {
    size_t most = 0;
    for (int64_t form = kNarrowCols, below = 0; form <= 16; below = form, form *= 2) {
        const int64_t last = std::min(columns, form) / group * group;  // the most columns that take it
        if (last > below) most = std::max(most, attn_layout_bytes(attn_layout(last, head_dim), c, head_dim, tokens));
    }
    const int64_t heads = static_cast<int64_t>(c.n_seq) * c.n_kv_heads, steps = ceil_div(attn_tiles(tokens), kMinChunk);
    const AttnLayout f = attn_layout(columns, head_dim);
    if (f.wc == 1 || heads > kCounters || steps == 1 || 4 * f.slots / heads < 2) return most;
    columns = std::min<int64_t>(columns, 0x7fffff00);  // more are refused
    const int64_t top = f.tall ? kPromptCols : (columns <= 32 ? 32 : (columns <= 64 ? 64 : 64 * attn_prompt_nt(kv_blocks(head_dim))));
    return std::max(most, attn_parts_bytes(std::min(4 * f.slots, heads * ceil_div(columns, top) * steps), top, head_dim));
}

}  // namespace
}  // namespace zdmmv

using namespace zdmmv;

extern "C" {

size_t zdmmv_attn_q4_0_workspace_bytes(const zdmmv_kv_cache *cache, int n_q_heads, int max_q_len, int max_kv_len) {
    KvView c{};
    if (kv_check(cache, &c) != ZDMMV_OK || n_q_heads < 1 || n_q_heads > 65535 || n_q_heads % c.n_kv_heads || max_q_len < 1 ||
        max_kv_len < 0)
        return 0;
    const int group = n_q_heads / c.n_kv_heads;
    return attn_bounds_bytes(c, cache->head_dim, group, static_cast<int64_t>(max_q_len) * group, max_kv_len);
}

zdmmv_status zdmmv_attn_q4_0(const zdmmv_kv_cache *cache, const zdmmv_attn_args *args, zdmmv_stream_t stream) {
    if (!args) return ZDMMV_ERR_NULL;
    AttnArgs a{};
    const zdmmv_status st = kv_check(cache, &a.c);
    if (st != ZDMMV_OK) return st;
    const zdmmv_attn_args &g = *args;
    AttnPlan p{};
    if (g.n_tok < 0 || g.n_q_heads < 1 || g.n_q_heads > 65535 || g.n_q_heads % cache->n_kv_heads || g.max_q_len < 1 ||
        g.max_kv_len < 0 || g.window < 0 || !std::isfinite(g.scale))
        return ZDMMV_ERR_SHAPE;
    // with a window, no column tile sees more than the window and its own new tokens
    const int64_t seen = g.window > 0 ? std::min<int64_t>(g.max_kv_len, static_cast<int64_t>(g.window) + g.max_q_len + kKvSlab)
                                      : g.max_kv_len;
    if (!attn_plan(a.c, cache->head_dim, g.n_q_heads, g.max_q_len, seen, &p)) return ZDMMV_ERR_SHAPE;
    if (g.n_tok == 0) return ZDMMV_OK;
    if (!g.q || !g.q_start || !g.kv_len || !g.out) return ZDMMV_ERR_NULL;
    if (g.q_stride < static_cast<int64_t>(g.n_q_heads) * cache->head_dim) return ZDMMV_ERR_SHAPE;
    if (kv_misaligned(g.q, 16) || kv_misaligned(g.out, 16) || kv_misaligned(g.workspace, 16) ||
        kv_misaligned(g.q_start, 4) || kv_misaligned(g.kv_len, 4) || kv_misaligned(g.status_dev, 4) || g.q_stride % 4)
        return ZDMMV_ERR_ALIGN;
    const size_t need = attn_parts_bytes(p.parts, p.cols, cache->head_dim);  // of the plan that is launched
    if (need && !g.workspace) return ZDMMV_ERR_NULL;
    if (g.workspace_bytes < need) return ZDMMV_ERR_SIZE;
    a.q = g.q; a.q_start = g.q_start; a.kv_len = g.kv_len; a.out = g.out; a.status = g.status_dev;
    a.fault = current_fault_word();
    if (!a.fault) return ZDMMV_ERR_CUDA;
    a.q_stride = g.q_stride;
    a.n_tok = g.n_tok; a.n_q_heads = g.n_q_heads; a.group = g.n_q_heads / cache->n_kv_heads;
    a.max_q_len = g.max_q_len; a.max_kv_len = std::min(g.max_kv_len, kMostTokens); a.window = g.window;
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
