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
    FastDiv by_groups, by_page;
    const float *k, *v, *q;
    const int32_t *seq, *pos;
    const float *rope;
    float *q_out;
    __half *k_val, *v_val;
    int32_t *status;
    uint32_t *fault;
    int32_t head_bytes;  // of a page's head
    int64_t k_stride, v_stride, q_stride, rope_rows;
    int32_t n_tok, n_q_heads, rot_dim, halves;
};

// The rotation of four neighbouring dimensions e0 .. e0+3 of a head: their cosines and sines, the sines of a pair's first
// dimension negated (its result is x cos - partner sin). Every product and sum is rounded by itself (no fused
// multiply-add), so that the result is the same wherever it is computed.
struct Turn {
    float c[4], s[4];
};

// FAST: four neighbouring dimensions are all rotated or none, and their partners and angles are neighbours too (pairs:
// rot_dim a multiple of 4; halves: rot_dim a multiple of 8), so everything is 128-bit loads.
template <bool FAST> __device__ __forceinline__ Turn load_turn(const AppendArgs &a, int pos, int e0) {
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
// Four dimensions of a head at `src` (global or shared memory) and, where the head is turned, their partners.
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
template <bool FAST>
__device__ __forceinline__ void turn_head(const AppendArgs &a, int e0, const Turn &t, const float (&o)[4], float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (FAST || e0 + i < a.rot_dim) x[i] = __fadd_rn(__fmul_rn(x[i], t.c[i]), __fmul_rn(o[i], t.s[i]));
}
// The head's row in the call's inputs: heads 0 .. of q, then those of k, then those of v.
__device__ __forceinline__ const float *head_row(const AppendArgs &a, int tok, int head, int dim) {
    const int kvh = head - a.n_q_heads;
    if (kvh < 0) return a.q + tok * a.q_stride + static_cast<int64_t>(head) * dim;
    if (kvh < a.c.n_kv_heads) return a.k + tok * a.k_stride + static_cast<int64_t>(kvh) * dim;
    return a.v + tok * a.v_stride + static_cast<int64_t>(kvh - a.c.n_kv_heads) * dim;
}

// Where a token goes in the cache.
struct Place {
    int page, in;   // page (0 where none is written), token of the page
    bool ok, bad;   // written to the cache; outside what the cache and the rotation table have
};
// The page's look-up is the one load: place_check looks at what it brought.
__device__ __forceinline__ Place place_of(const AppendArgs &a, int pos, int seq) {
    Place w;
    const bool pad = pos < 0;
    const int slot = pad ? 0 : a.by_page.div(pos);
    w.in = pad ? 0 : a.by_page.mod(pos, slot);
    w.bad = !pad && (seq < 0 || seq >= a.c.n_seq || slot >= a.c.max_pages || (a.rot_dim > 0 && pos >= a.rope_rows));
    w.ok = !pad && !w.bad;
    w.page = w.ok ? a.c.table[static_cast<int64_t>(seq) * a.c.max_pages + slot] : 0;
    return w;
}
__device__ __forceinline__ void place_check(const AppendArgs &a, Place &w, int lane) {
    if (w.page < 0 || w.page >= a.c.n_pages) w.bad = true;
    if (!w.bad) return;
    w.ok = false;
    w.page = 0;
    if (lane == 0 && a.status) *a.status = 1;
}
__device__ __forceinline__ float place_fill(const Place &w) { return w.bad ? __int_as_float(0x7fffffff) : 0.0f; }

// Where a token's results go, found once a token: its rows of q_out, k_val and v_val, and of the cache its tile of head 0
// (nullptr where it is not written) with its places in it.
struct Rows {
    float *q;
    __half *k, *v;
    uint8_t *tile;
    int r;  // token of the tile
};
template <int NB> __device__ __forceinline__ Rows rows_of(const AppendArgs &a, const Place &w, int tok) {
    using G = KvGeom<NB>;
    const int64_t kv = static_cast<int64_t>(tok) * a.c.n_kv_heads * G::kDim;
    Rows y;
    y.q = a.q_out + static_cast<int64_t>(tok) * a.n_q_heads * G::kDim;
    y.k = a.k_val ? a.k_val + kv : nullptr;
    y.v = a.v_val ? a.v_val + kv : nullptr;
    y.tile = w.ok ? a.c.pages + w.page * a.c.page_bytes + static_cast<int64_t>(w.in / kKvSlab) * G::kTileBytes : nullptr;
    y.r = w.in % kKvSlab;
    return y;
}

// Four dimensions e0 .. e0+3 of a (rotated) head: q's are stored; k's and v's are quantized and stored in the cache and as
// values. The whole warp calls it: a block's 8 lanes exchange its maximum.
template <int NB>
__device__ __forceinline__ void put_head(const AppendArgs &a, const Rows &to, int head, int e0, int lane, const float (&x)[4]) {
    using G = KvGeom<NB>;
    const bool inside = e0 < G::kDim;
    const int kvh = head - a.n_q_heads;
    if (kvh < 0) {
        if (inside)
            *reinterpret_cast<float4 *>(to.q + head * G::kDim + e0) = make_float4(x[0], x[1], x[2], x[3]);
        return;
    }
    const bool is_k = kvh < a.c.n_kv_heads;
    const int h = is_k ? kvh : kvh - a.c.n_kv_heads;
    // the first value of the largest magnitude, over the block's 8 lanes
    float big = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
    for (int s = 1; s < 8; s <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, s));
    float m = x[3];
#pragma unroll
    for (int i = 2; i >= 0; --i)
        if (fabsf(x[i]) == big) m = x[i];
    const uint32_t has = __ballot_sync(0xffffffffu, fabsf(m) == big) >> (lane & 24) & 0xffu;
    m = __shfl_sync(0xffffffffu, m, (lane & 24) + (has ? __ffs(has) - 1 : 0));
    const float d = m * -0.125f;  // exactly m / -8
    const float id = d != 0.0f ? __frcp_rn(d) : 0.0f;
    const __half dh = __float2half_rn(d);
    uint32_t code[4], packed = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = static_cast<int>(__fadd_rn(__fmul_rn(x[i], id), 8.5f));
        code[i] = c < 0 ? 0 : (c > 15 ? 15 : c);
        packed |= code[i] << (4 * i);
    }
    const uint32_t upper = __shfl_down_sync(0xffffffffu, packed, 1);
    if (!inside) return;
    const int b = e0 / kQK, g = (e0 % kQK) / 4, r = to.r;
    if (to.tile) {
        uint8_t *tile = to.tile + static_cast<int64_t>(h) * a.head_bytes;
        __half *scales = reinterpret_cast<__half *>(tile + (is_k ? G::kKScaleAt : G::kVScaleAt));
        if (g == 0) scales[G::scale_half(r, b)] = dh;
        if (is_k) {
            if ((g & 1) == 0) reinterpret_cast<uint32_t *>(tile)[G::k_word(r, b, g / 2)] = packed | (upper << 16);
        } else {
            reinterpret_cast<uint16_t *>(tile + G::kVAt)[G::v_half(r, b, g)] = static_cast<uint16_t>(packed);
        }
    }
    __half *val = is_k ? to.k : to.v;
    if (!val) return;
    const float df = __half2float(dh);
    __half2 y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        y[i] = __floats2half2_rn(df * (static_cast<float>(code[2 * i]) - 8.0f), df * (static_cast<float>(code[2 * i + 1]) - 8.0f));
    *reinterpret_cast<uint2 *>(val + h * G::kDim + e0) = *reinterpret_cast<uint2 *>(y);
}

// Few tokens: one warp per token and head. Lane l holds the four dimensions 4l .. 4l+3 of each pass of 128 and loads all
// of a head before it stores any (so q_out may be q); the look-up of the token's place runs beside the loads. Bound by
// the latency of its three dependent loads (2.2 us for 48 tokens of 48 heads of 128).
constexpr int kAppendWarps = 4;
template <int NB, bool FAST> __global__ void __launch_bounds__(kAppendWarps * 32) kv_append_kernel(AppendArgs a) {
    using G = KvGeom<NB>;
    constexpr int kPass = (G::kDim + 127) / 128;
    const int lane = threadIdx.x & 31;
    const int job = static_cast<int>(blockIdx.x) * kAppendWarps + static_cast<int>(threadIdx.x >> 5);
    const int tok = a.by_groups.div(job), head = a.by_groups.mod(job, tok);
    block_op_wait();
    block_op_release();
    if (tok >= a.n_tok) return;
    const bool turned = head < a.n_q_heads + a.c.n_kv_heads;
    const int pos = a.pos[tok], seq = a.seq[tok];
    float v[kPass][4], o[kPass][4];
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
        const int e0 = p * 128 + 4 * lane;
        v[p][0] = v[p][1] = v[p][2] = v[p][3] = 0.0f;
        if (e0 < G::kDim) load_head<FAST>(a, head_row(a, tok, head, G::kDim), e0, turned && e0 < a.rot_dim, v[p], o[p]);
    }
    Place w = place_of(a, pos, seq);
    Turn turn[kPass];
#pragma unroll
    for (int p = 0; p < kPass; ++p)
        if (w.ok && turned && p * 128 + 4 * lane < a.rot_dim) turn[p] = load_turn<FAST>(a, pos, p * 128 + 4 * lane);
    place_check(a, w, lane);
    const Rows to = rows_of<NB>(a, w, tok);
    __syncwarp();
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
        const int e0 = p * 128 + 4 * lane;
        if (!w.ok) v[p][0] = v[p][1] = v[p][2] = v[p][3] = place_fill(w);
        else if (turned && e0 < a.rot_dim) turn_head<FAST>(a, e0, turn[p], o[p], v[p]);
        put_head<NB>(a, to, head, e0, lane, v[p]);
    }
}

// Prompts: bound by memory. Each warp takes a stretch of consecutive (token, group of kStreamHeads heads) pairs and keeps
// the next kStreamSlots of them on their way into its own ring in shared memory (a bulk copy a head), so that the loads
// wait neither for the token's look-up nor for the quantization; a token's place, cosines and sines are read once and
// kept for all its heads. 4093 tokens of 48 heads of 128: one warp a head without the ring 49 us at best (48 warps an
// SM, each with its loads in flight for half of its life), with it 37.0 us (76% of the copy rate), then bound by issue (67%
// active, 135 instructions a head; 41 us with 154 before the token's row addresses were found once).
constexpr int kStreamWarps = 8, kStreamHeads = 4, kStreamSlots = 3;
template <int NB, bool FAST> __global__ void __launch_bounds__(kStreamWarps * 32, NB <= 4 ? 3 : 2) kv_append_stream_kernel(AppendArgs a, int n_jobs) {
    using G = KvGeom<NB>;
    constexpr int kPass = (G::kDim + 127) / 128, kHeadBytes = G::kDim * 4, kSlotBytes = kStreamHeads * kHeadBytes;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem) + warp * kStreamSlots;
    uint8_t *ring = smem + 256 + warp * (kStreamSlots * kSlotBytes);
    if (lane == 0) {
        for (int s = 0; s < kStreamSlots; ++s) mbar_init(&full[s], 1);
        fence_barrier_init();
    }
    __syncwarp();
    block_op_wait();
    block_op_release();
    const int heads = a.n_q_heads + 2 * a.c.n_kv_heads;
    const int64_t n_warps = static_cast<int64_t>(gridDim.x) * kStreamWarps, me = static_cast<int64_t>(blockIdx.x) * kStreamWarps + warp;
    const int first = static_cast<int>(n_jobs * me / n_warps), last = static_cast<int>(n_jobs * (me + 1) / n_warps);
    const uint64_t policy = l2_evict_first_policy();
    const auto copy = [&](int job, int s) {
        const int tok = a.by_groups.div(job), h0 = a.by_groups.mod(job, tok) * kStreamHeads;
        const int n = min(kStreamHeads, heads - h0);
        if (lane == 0) mbar_arrive_expect_tx(&full[s], n * kHeadBytes);
        __syncwarp();
        if (lane < n)
            bulk_copy_g2s(ring + s * kSlotBytes + lane * kHeadBytes, head_row(a, tok, h0 + lane, G::kDim), kHeadBytes, &full[s], policy);
    };
    for (int s = 0; s < kStreamSlots; ++s)
        if (first + s < last) copy(first + s, s);
    int at = -1, s = 0;
    uint32_t phase = 0;
    Place w{};
    Rows to{};
    Turn turn[kPass];
    int lost = -1;  // the job whose wait gave up: the rows from it on are NaN
    int tok = a.by_groups.div(first), h0 = a.by_groups.mod(first, tok) * kStreamHeads;
    for (int job = first; job < last; ++job, h0 += kStreamHeads) {
        if (h0 >= heads) {
            h0 = 0;
            ++tok;
        }
        if (tok != at) {
            at = tok;
            const int pos = a.pos[tok];
            w = place_of(a, pos, a.seq[tok]);
#pragma unroll
            for (int p = 0; p < kPass; ++p)
                if (w.ok && p * 128 + 4 * lane < a.rot_dim) turn[p] = load_turn<FAST>(a, pos, p * 128 + 4 * lane);
            place_check(a, w, lane);
            to = rows_of<NB>(a, w, tok);
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&full[s], phase))) {
            if (lane == 0) atomicOr(a.fault, 1u);
            lost = job;
            break;
        }
        const float *rows = reinterpret_cast<const float *>(ring + s * kSlotBytes);
#pragma unroll
        for (int u = 0; u < kStreamHeads; ++u) {
            const int head = h0 + u;
            if (head >= heads) break;
            const bool turned = head < a.n_q_heads + a.c.n_kv_heads;
#pragma unroll
            for (int p = 0; p < kPass; ++p) {
                const int e0 = p * 128 + 4 * lane;
                float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, o[4];
                if (!w.ok) {
                    v[0] = v[1] = v[2] = v[3] = place_fill(w);
                } else if (e0 < G::kDim) {
                    const bool turn_it = turned && e0 < a.rot_dim;
                    load_head<FAST>(a, rows + u * G::kDim, e0, turn_it, v, o);
                    if (turn_it) turn_head<FAST>(a, e0, turn[p], o, v);
                }
                put_head<NB>(a, to, head, e0, lane, v);
            }
        }
        __syncwarp();
        if (job + kStreamSlots < last) {
            fence_proxy_async_smem();
            copy(job + kStreamSlots, s);
        }
        if (++s == kStreamSlots) {
            s = 0;
            phase ^= 1;
        }
    }
    if (lost < 0) return;
    // leave only when the copies have landed, as far as they will
    for (int k = lost; k < min(lost + kStreamSlots, last); ++k) (void)mbar_wait(&full[(k - first) % kStreamSlots], (k - first) / kStreamSlots & 1);
    const float nan = __int_as_float(0x7fffffff), row[4] = {nan, nan, nan, nan};
    for (int job = lost; job < last; ++job) {
        const int t = a.by_groups.div(job), from = a.by_groups.mod(job, t) * kStreamHeads;
        Place where = place_of(a, a.pos[t], a.seq[t]);
        place_check(a, where, lane);
        const Rows dst = rows_of<NB>(a, where, t);
        for (int head = from; head < min(from + kStreamHeads, heads); ++head)
            for (int p = 0; p < kPass; ++p) put_head<NB>(a, dst, head, p * 128 + 4 * lane, lane, row);
    }
}

template <int NB, bool FAST> cudaError_t launch_append_as(AppendArgs a, cudaStream_t st) {
    const int heads = a.n_q_heads + 2 * a.c.n_kv_heads;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // the stream kernel from as many (token, head) pairs as the device holds warps
    const int64_t pairs = static_cast<int64_t>(a.n_tok) * heads;
    if (pairs <= static_cast<int64_t>(sms) * 64) {
        a.by_groups = FastDiv::of(heads);
        return launch_block_op(kv_append_kernel<NB, FAST>, dim3(static_cast<unsigned>((pairs + kAppendWarps - 1) / kAppendWarps)),
                               dim3(kAppendWarps * 32), 0, st, a);
    }
    const int groups = (heads + kStreamHeads - 1) / kStreamHeads;
    a.by_groups = FastDiv::of(groups);
    const int n_jobs = a.n_tok * groups;
    constexpr size_t kSmem = 256 + static_cast<size_t>(kStreamWarps) * kStreamSlots * kStreamHeads * NB * kQK * 4;
    constexpr int kCtas = kSmem <= 55 * 1024 ? 3 : 2;  // per SM: as many as fit
    e = smem_limit_raised<&kv_append_stream_kernel<NB, FAST>>();
    if (e != cudaSuccess) return e;
    return launch_block_op(kv_append_stream_kernel<NB, FAST>, dim3(sms * kCtas), dim3(kStreamWarps * 32), kSmem, st, a, n_jobs);
}
template <int NB> cudaError_t launch_append(const AppendArgs &a, cudaStream_t st) {
    return a.rot_dim % (a.halves ? 8 : 4) == 0 ? launch_append_as<NB, true>(a, st) : launch_append_as<NB, false>(a, st);
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
        (g.rot_dim > 0 && g.rope_rows < 1) || static_cast<int64_t>(g.n_tok) * (g.n_q_heads + 2 * cache->n_kv_heads) > 0x7fffff00 || g.n_q_heads < 0 || g.n_q_heads > 65535 || (g.q != nullptr) != (g.n_q_heads > 0))
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
    a.by_page = FastDiv::of(cache->page_tokens);
    a.head_bytes = cache->page_tokens / kKvSlab * 18 * cache->head_dim;
    a.k = g.k; a.v = g.v; a.q = g.q;
    a.seq = g.seq; a.pos = g.pos; a.rope = g.rope;
    a.q_out = g.q_out;
    a.k_val = static_cast<__half *>(g.k_val);
    a.v_val = static_cast<__half *>(g.v_val);
    a.status = g.status_dev;
    a.fault = current_fault_word();
    if (!a.fault) return ZDMMV_ERR_CUDA;
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
