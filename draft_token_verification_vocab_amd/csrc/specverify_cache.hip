// specverify_cache.hip -- host side of the paged-cache calls declared in
// include/specverify.h: tree attention, appending, accepting and keeping a
// path, and the pages' sharing.  Argument validation, workspace layout, kernel
// selection and launches on the caller's stream.  No allocation, no
// synchronisation.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "specverify.h"
#include "sv_cache.hpp"
#include "sv_common.hpp"
#include "sv_host.hpp"
#include "sv_launch.hpp"
#include "sv_layout.hpp"
#include "sv_tree.hpp"

namespace {

using namespace sv;

constexpr int kUnits = 256;            // compute units
constexpr int kMaxSlices = 2 * kUnits; // runs of tiles
constexpr int kMaxChainNodes = 65536;
constexpr int kMaxHeads = 65535;
constexpr int kMaxRoom = 1 << 30;      // positions that a table row can hold

int page_shift(int32_t page_size) {
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

bool page_size_ok(int32_t s) { return s >= 8 && s <= 1024 && (s & (s - 1)) == 0; }

// A table row's shape, for the calls that take no pools.
spec_status check_table(int32_t table_width, int32_t page_size, int32_t num_pages) {
    if (table_width < 1 || num_pages < 1 || page_size < 1) return SPEC_ERR_ARG;
    if (!page_size_ok(page_size)) return SPEC_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(table_width) * page_size > kMaxRoom) return SPEC_ERR_UNSUPPORTED;
    return SPEC_OK;
}

// A stride of n elements of e bytes: looked at before it is multiplied, which may wrap.
bool stride_ok(int64_t n, int e) { return n >= 0 && n % (16 / e) == 0; }

// Addresses [from, to); an empty range meets nothing.
struct Range {
    const char *from, *to;
    bool meets(const Range &o) const {
        return from < o.to && o.from < to && from < to && o.from < o.to;
    }
};
Range range(const void *p, int64_t bytes) {
    const char *c = static_cast<const char *>(p);
    return Range{c, c + bytes};
}

Range ints(const int32_t *p, int64_t n) { return range(p, p ? n * 4 : 0); }

// Whether something that is written meets something that is read, or another that is
// written.
template <int W, int R>
bool writes_meet(const Range (&to)[W], const Range (&in)[R]) {
    for (int i = 0; i < W; ++i) {
        for (int j = 0; j < i; ++j)
            if (to[i].meets(to[j])) return true;
        for (const Range &r : in)
            if (to[i].meets(r)) return true;
    }
    return false;
}

// Strides, and counts times them, that keep the address arithmetic far from 2^63.
constexpr int64_t kMaxStride = int64_t{1} << 40, kMaxSpan = int64_t{1} << 56;
bool span_ok(int64_t n, int64_t stride) { return stride < 1 || n <= kMaxSpan / stride; }

spec_status check_cache(const spec_cache *c) {
    if (!c || c->batch < 0 || c->reserved != 0) return SPEC_ERR_ARG;
    if (c->dtype != SPEC_DTYPE_F32 && c->dtype != SPEC_DTYPE_BF16 && c->dtype != SPEC_DTYPE_F16)
        return SPEC_ERR_ARG;
    if (c->kv_heads < 1 || c->dim < 8 || c->dim % 8 != 0) return SPEC_ERR_ARG;
    const spec_status s = check_table(c->table_width, c->page_size, c->num_pages);
    if (s != SPEC_OK) return s;
    const int e = elem_size(c->dtype);
    if (c->page_stride > kMaxStride || c->head_stride > kMaxStride ||
        c->slot_stride > kMaxStride || !span_ok(c->num_pages, c->page_stride))
        return SPEC_ERR_UNSUPPORTED;
    if (!stride_ok(c->page_stride, e) || !stride_ok(c->head_stride, e) ||
        !stride_ok(c->slot_stride, e) || c->slot_stride < c->dim)
        return SPEC_ERR_ARG;
    if (c->dim > 256 || c->kv_heads > kMaxHeads) return SPEC_ERR_UNSUPPORTED;
    return SPEC_OK;
}

// The bytes from a pool's base to its last element's end.
int64_t pool_bytes(const spec_cache_pools *p) {
    return (p->num_pages - 1) * p->page_stride + (p->heads - 1) * p->head_stride +
           (p->page_size - 1) * p->slot_stride + p->slot_bytes;
}
int64_t pool_bytes(const spec_cache *c) {
    return ((c->num_pages - 1) * c->page_stride + (c->kv_heads - 1) * c->head_stride +
            (c->page_size - 1) * c->slot_stride + c->dim) *
           elem_size(c->dtype);
}

// Whether every element of a pool that is written to has a place of its own: one that
// pages, heads or slots share has two writers.
bool elements_apart(const spec_cache *c, PoolLayout *p) {
    const int64_t e = elem_size(c->dtype);
    return lay_out({c->num_pages, c->kv_heads, c->page_size},
                   {c->page_stride * e, c->head_stride * e, c->slot_stride * e}, c->dim * e, p);
}
bool elements_apart(const spec_cache_pools *c, PoolLayout *p) {
    return lay_out({c->num_pages, c->heads, c->page_size},
                   {c->page_stride, c->head_stride, c->slot_stride}, c->slot_bytes, p);
}

bool pools_ok(const spec_cache *c) {
    return c->keys && c->values && aligned16(c->keys) && aligned16(c->values) && c->table &&
           c->lengths;
}

// ---------------------------------------------------------------------------
// Tree attention
// ---------------------------------------------------------------------------
// Slots of 16-bit types: eight of them have offsets below 2^32 bytes.
constexpr int64_t kMaxWideSlot = int64_t{1} << 28;
// Tiles of the longest sequence that is not cut, and so needs no second launch: one
// of float32 (one sequence of two tiles 19.0 us whole, 17.5 cut), four of 16-bit
// types, where five nodes of 64 sequences take 24.2 us whole and 26.7 cut, of one
// sequence 13.1 and 14.0 (11.4 in a graph); of eight tiles one takes 21.3 and 13.8.
constexpr int kTreeWhole = 4;

struct TreePlan {
    int dp;      // dimensions, rounded up to what a kernel takes
    bool wide;   // rows shared out to the waves, else keys
    int rt;      // 16-row tiles to a wave
    int rows;    // of a workgroup
    int waves;   // workgroups to a compute unit
    int mtiles;
    bool whole;  // a slice is a sequence
    int slices;
    size_t first, part, part_ml, total;  // workspace
};

spec_status check_tree(const spec_cache *c, int32_t nodes, int32_t heads, bool tree) {
    spec_status s = check_cache(c);
    if (s != SPEC_OK) return s;
    if (nodes < 1 || heads < 1 || heads % c->kv_heads != 0) return SPEC_ERR_ARG;
    if (nodes > (tree ? kMaxTreeNodes : kMaxChainNodes) || heads > kMaxHeads)
        return SPEC_ERR_UNSUPPORTED;
    if (c->dtype != SPEC_DTYPE_F32 && c->slot_stride > kMaxWideSlot) return SPEC_ERR_UNSUPPORTED;
    const int64_t tiles =
        (static_cast<int64_t>(c->table_width) * c->page_size + kTreeTile - 1) / kTreeTile;
    // counted in 32 bits, and rounded up to whole runs
    if (c->batch > (INT32_MAX - kMaxSlices) / tiles) return SPEC_ERR_UNSUPPORTED;
    const int64_t rows = static_cast<int64_t>(c->batch) * nodes;
    if (rows > 0 && rows > (int64_t{1} << 40) / heads) return SPEC_ERR_UNSUPPORTED;
    const int64_t joins = (static_cast<int64_t>(nodes) * heads / kTreeWaves + 1) * c->batch;
    if (!grid_fits(joins, kTreeBlock)) return SPEC_ERR_UNSUPPORTED;
    return SPEC_OK;
}

TreePlan plan_tree(const spec_cache *c, int32_t nodes, int32_t heads) {
    TreePlan p;
    p.dp = c->dim <= 64 ? 64 : (c->dim <= 128 ? 128 : 256);
    const int64_t rows = static_cast<int64_t>(nodes) * (heads / c->kv_heads);
    const int64_t tiles16 = (rows + 15) / 16;
    const int64_t longest =
        (static_cast<int64_t>(c->table_width) * c->page_size + kTreeTile - 1) / kTreeTile;
    // 16-bit types' keys and values go through shared memory, float32's straight into
    // registers: of 16 bits those were never sooner by more than 2 us (one sequence of
    // 512 positions, 10.8 us against 12.7) and up to 2.3 times slower (rows of 64)
    p.wide = c->dtype != SPEC_DTYPE_F32;
    if (p.wide) {
        p.rt = tiles16 > 4 ? 2 : 1;
        p.rows = 64 * p.rt;
        p.waves = p.dp == 256 ? 1 : 2;
    } else {
        const int most = p.dp == 256 ? 1 : 2;
        const int64_t splits = (tiles16 + most - 1) / most;
        p.rt = static_cast<int>((tiles16 + splits - 1) / splits);
        p.rows = 16 * p.rt;
        p.waves = tree_waves(p.dp);
    }
    p.mtiles = static_cast<int>((rows + p.rows - 1) / p.rows);
    const int64_t units = static_cast<int64_t>(p.mtiles) * c->kv_heads;
    const int64_t tiles = c->batch * longest;
    // short sequences are not cut: no second launch
    p.whole = longest <= (p.wide ? kTreeWhole : 1);
    int64_t slices = (p.waves * kUnits + units - 1) / units;
    if (slices > tiles) slices = tiles;
    p.slices = p.whole ? c->batch : static_cast<int>(slices < 1 ? 1 : slices);
    const int64_t parts = p.whole ? 0 : 2 * units * p.slices * p.rows;
    p.first = 0;
    p.part = align_up((static_cast<size_t>(c->batch) + 1) * sizeof(int32_t));
    p.part_ml = p.part + align_up(static_cast<size_t>(parts) * c->dim * sizeof(float));
    p.total = p.whole ? 0 : p.part_ml + align_up(static_cast<size_t>(parts) * 4 * sizeof(float));
    return p;
}

template <typename T, int DP, bool FULL>
void launch_tree_rt(const TreeArgs &a, const TreePlan &p, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>(p.slices * a.KV * p.mtiles)), block(kTreeBlock);
    if constexpr (sizeof(T) == 2) {
        if (p.mtiles > 1)
            tree_wide_kernel<T, DP, 2, FULL, false><<<grid, block, 0, st>>>(a);
        else if (p.rt == 2)
            tree_wide_kernel<T, DP, 2, FULL, true><<<grid, block, 0, st>>>(a);
        else
            tree_wide_kernel<T, DP, 1, FULL, true><<<grid, block, 0, st>>>(a);
    } else {
        if constexpr (DP <= 128) {
            if (p.rt == 2) {
                tree_attention_kernel<DP, 2, FULL><<<grid, block, 0, st>>>(a);
                return;
            }
        }
        tree_attention_kernel<DP, 1, FULL><<<grid, block, 0, st>>>(a);
    }
}

template <typename T, int DP>
void launch_tree_dim(const TreeArgs &a, const TreePlan &p, hipStream_t st) {
    if (a.D == DP && a.slot_stride == DP)
        launch_tree_rt<T, DP, true>(a, p, st);
    else
        launch_tree_rt<T, DP, false>(a, p, st);
}

template <typename T>
void launch_tree(const TreeArgs &a, const TreePlan &p, hipStream_t st) {
    if (p.dp == 64)
        launch_tree_dim<T, 64>(a, p, st);
    else if (p.dp == 128)
        launch_tree_dim<T, 128>(a, p, st);
    else
        launch_tree_dim<T, 256>(a, p, st);
}

// Four rows to a wave where there are rows for every wave that the chip holds: 16
// trees of 64 nodes and 64 heads 309 us against 317, 64 chains of nine (18432 rows)
// 211.9 against 213.0; with four, 64 single tokens' 2048 rows take 97.0 against 94.2,
// two caches' 1152 rows 193.7 against 175.5.
constexpr int64_t kJoinRows = 8192;

template <typename T, int L>
void launch_join_rows(const TreeArgs &a, const TreePlan &p, hipStream_t st) {
    const int rows = a.T * a.H;
    const bool four = static_cast<int64_t>(a.B) * rows >= kJoinRows && rows % 4 == 0;
    const int per = kTreeWaves * (four ? 4 : 1), blocks = (rows + per - 1) / per;
    const dim3 grid(static_cast<unsigned>(blocks * a.B)), block(kTreeBlock);
    if (four)
        tree_join_kernel<T, L, 4><<<grid, block, 0, st>>>(a, p.rows, blocks);
    else
        tree_join_kernel<T, L, 1><<<grid, block, 0, st>>>(a, p.rows, blocks);
}

template <typename T>
void launch_join(const TreeArgs &a, const TreePlan &p, hipStream_t st) {
    if (p.dp == 64)
        launch_join_rows<T, 16>(a, p, st);
    else if (p.dp == 128)
        launch_join_rows<T, 32>(a, p, st);
    else
        launch_join_rows<T, 64>(a, p, st);
}

// ---------------------------------------------------------------------------
// Pools
// ---------------------------------------------------------------------------
// twice: whether a pool that is given twice counts as sharing its memory.
spec_status check_pools(const spec_cache_pools *p, bool twice) {
    if (!p || p->num_pools < 0 || p->num_pages < 1 || p->page_size < 1 || p->heads < 1 ||
        p->slot_bytes < 1)
        return SPEC_ERR_ARG;
    if (p->page_stride > kMaxStride || p->head_stride > kMaxStride ||
        p->slot_stride > kMaxStride || !span_ok(p->num_pages, p->page_stride))
        return SPEC_ERR_UNSUPPORTED;
    if (!stride_ok(p->page_stride, 1) || !stride_ok(p->head_stride, 1) ||
        !stride_ok(p->slot_stride, 1) || p->slot_bytes % 16 != 0 ||
        p->slot_stride < p->slot_bytes)
        return SPEC_ERR_ARG;
    if (!page_size_ok(p->page_size) || p->heads > kMaxHeads || p->slot_bytes > 65536)
        return SPEC_ERR_UNSUPPORTED;
    PoolLayout layout;
    if (!elements_apart(p, &layout)) return SPEC_ERR_ARG;
    if (p->num_pools > 0 && !p->bases) return SPEC_ERR_ARG;
    for (int i = 0; i < p->num_pools; ++i)
        if (!p->bases[i] || !aligned16(p->bases[i])) return SPEC_ERR_ARG;
    return any_pools_meet(layout, p->bases, p->num_pools, twice) ? SPEC_ERR_ARG : SPEC_OK;
}

// Pools [first, first + count) as a kernel takes them.
PoolArgs pool_args(const spec_cache_pools *p, int first, int count) {
    PoolArgs a{};
    for (int i = 0; i < count; ++i) a.base[i] = static_cast<char *>(p->bases[first + i]);
    a.page_stride = p->page_stride;
    a.head_stride = p->head_stride;
    a.slot_stride = p->slot_stride;
    a.count = count;
    a.heads = p->heads;
    a.units = static_cast<int32_t>(p->slot_bytes / 16);
    a.pages = p->num_pages;
    a.shift = page_shift(p->page_size);
    return a;
}

struct ReservePlan {
    int chunks;
    size_t words, before, counts, total;
};

ReservePlan plan_reserve(int32_t num_pages) {
    ReservePlan p;
    p.chunks = (num_pages + kPageChunk - 1) / kPageChunk;
    const size_t n = static_cast<size_t>(p.chunks) * kChunkWords;
    p.words = 0;
    p.before = align_up(n * sizeof(uint64_t));
    p.counts = p.before + align_up(n * sizeof(int32_t));
    p.total = p.counts + align_up(p.chunks * sizeof(int32_t));
    return p;
}

}  // namespace

extern "C" {

size_t spec_tree_attention_workspace_bytes(const spec_cache *cache, int32_t nodes,
                                           int32_t heads) {
    if (check_tree(cache, nodes, heads, false) != SPEC_OK || cache->batch == 0) return 0;
    return plan_tree(cache, nodes, heads).total;
}

spec_status spec_tree_attention(const spec_cache *cache, const void *q, int64_t q_batch_stride,
                                int64_t q_node_stride, int64_t q_head_stride, int32_t nodes,
                                int32_t heads, const int32_t *parents, const int32_t *num_nodes,
                                float scale, void *out, float *lse, void *workspace,
                                size_t workspace_bytes, void *stream) {
    const spec_status s = check_tree(cache, nodes, heads, parents != nullptr);
    if (s != SPEC_OK) return s;
    if (!(scale > 0.0f) || !std::isfinite(scale * kLog2e)) return SPEC_ERR_ARG;
    const int e = elem_size(cache->dtype);
    if (q_batch_stride > kMaxStride || q_node_stride > kMaxStride ||
        q_head_stride > kMaxStride || !span_ok(cache->batch, q_batch_stride))
        return SPEC_ERR_UNSUPPORTED;
    if (!stride_ok(q_batch_stride, e) || !stride_ok(q_node_stride, e) ||
        !stride_ok(q_head_stride, e))
        return SPEC_ERR_ARG;
    if (cache->batch == 0) return SPEC_OK;
    if (!pools_ok(cache) || !q || !aligned16(q) || !out || !aligned16(out)) return SPEC_ERR_ARG;
    const int64_t rows = static_cast<int64_t>(cache->batch) * nodes * heads;
    const TreePlan p = plan_tree(cache, nodes, heads);
    if (!grid_fits(static_cast<int64_t>(p.slices) * cache->kv_heads * p.mtiles, kTreeBlock))
        return SPEC_ERR_UNSUPPORTED;
    if (p.total > 0 && (!workspace || workspace_bytes < p.total)) return SPEC_ERR_WORKSPACE;
    if (!aligned16(workspace)) return SPEC_ERR_ARG;
    const int64_t batch = cache->batch;
    const Range to[] = {range(out, rows * cache->dim * e), range(lse, lse ? rows * 4 : 0),
                        range(workspace, static_cast<int64_t>(p.total))};
    const Range in[] = {
        range(cache->keys, pool_bytes(cache)), range(cache->values, pool_bytes(cache)),
        range(q, ((batch - 1) * q_batch_stride + (nodes - 1) * q_node_stride +
                  (heads - 1) * q_head_stride + cache->dim) *
                     e),
        ints(cache->table, batch * cache->table_width), ints(cache->lengths, batch),
        ints(parents, batch * nodes), ints(num_nodes, batch)};
    if (writes_meet(to, in)) return SPEC_ERR_ARG;
    char *w = static_cast<char *>(workspace);
    TreeArgs a{};
    a.keys = cache->keys;
    a.values = cache->values;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.table = cache->table;
    a.lengths = cache->lengths;
    a.nodes = num_nodes;
    a.parents = parents;
    if (!p.whole) {
        a.first = reinterpret_cast<int32_t *>(w + p.first);
        a.part = reinterpret_cast<float *>(w + p.part);
        a.part_ml = reinterpret_cast<float *>(w + p.part_ml);
    }
    a.page_stride = cache->page_stride;
    a.head_stride = cache->head_stride;
    a.slot_stride = cache->slot_stride;
    a.q_batch = q_batch_stride;
    a.q_node = q_node_stride;
    a.q_head = q_head_stride;
    a.B = cache->batch;
    a.T = nodes;
    a.H = heads;
    a.KV = cache->kv_heads;
    a.G = heads / cache->kv_heads;
    a.D = cache->dim;
    a.P = cache->table_width;
    a.pages = cache->num_pages;
    a.shift = page_shift(cache->page_size);
    a.slices = p.slices;
    a.whole = p.whole;
    a.mtiles = p.mtiles;
    a.scale2 = scale * kLog2e;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (cache->dtype == SPEC_DTYPE_BF16)
        launch_tree<__bf16>(a, p, st);
    else if (cache->dtype == SPEC_DTYPE_F16)
        launch_tree<_Float16>(a, p, st);
    else
        launch_tree<float>(a, p, st);
    const spec_status r = launch_status();
    if (r != SPEC_OK || p.whole) return r;
    if (cache->dtype == SPEC_DTYPE_BF16)
        launch_join<__bf16>(a, p, st);
    else if (cache->dtype == SPEC_DTYPE_F16)
        launch_join<_Float16>(a, p, st);
    else
        launch_join<float>(a, p, st);
    return launch_status();
}

spec_status spec_cache_append(const spec_cache *cache, const void *k, const void *v,
                              int64_t batch_stride, int64_t node_stride, int64_t head_stride,
                              int32_t nodes, const int32_t *num_nodes, void *stream) {
    const spec_status s = check_cache(cache);
    if (s != SPEC_OK) return s;
    const int e = elem_size(cache->dtype);
    if (nodes < 0) return SPEC_ERR_ARG;
    if (batch_stride > kMaxStride || node_stride > kMaxStride || head_stride > kMaxStride ||
        nodes > kMaxRoom || !span_ok(cache->batch, batch_stride) || !span_ok(nodes, node_stride))
        return SPEC_ERR_UNSUPPORTED;
    if (!stride_ok(batch_stride, e) || !stride_ok(node_stride, e) || !stride_ok(head_stride, e))
        return SPEC_ERR_ARG;
    if (cache->batch == 0 || nodes == 0) return SPEC_OK;
    if (!pools_ok(cache) || !k || !v || !aligned16(k) || !aligned16(v)) return SPEC_ERR_ARG;
    // two writers to an element
    PoolLayout layout;
    void *const both[] = {cache->keys, cache->values};
    if (!elements_apart(cache, &layout) || any_pools_meet(layout, both, 2, true))
        return SPEC_ERR_ARG;
    const int64_t span = ((cache->batch - 1) * batch_stride + (nodes - 1) * node_stride +
                          (cache->kv_heads - 1) * head_stride + cache->dim) *
                         e;
    const Range pools[] = {range(cache->keys, pool_bytes(cache)),
                           range(cache->values, pool_bytes(cache))};
    const int64_t batch = cache->batch;
    const Range in[] = {range(k, span), range(v, span),
                        ints(cache->table, batch * cache->table_width),
                        ints(cache->lengths, batch), ints(num_nodes, batch)};
    for (const Range &r : in)
        if (pools[0].meets(r) || pools[1].meets(r)) return SPEC_ERR_ARG;
    AppendArgs a{};
    a.k = static_cast<const char *>(k);
    a.v = static_cast<const char *>(v);
    a.keys = static_cast<char *>(cache->keys);
    a.values = static_cast<char *>(cache->values);
    a.table = cache->table;
    a.lengths = cache->lengths;
    a.nodes = num_nodes;
    a.batch_stride = batch_stride * e;
    a.node_stride = node_stride * e;
    a.k_head_stride = head_stride * e;
    a.page_stride = cache->page_stride * e;
    a.head_stride = cache->head_stride * e;
    a.slot_stride = cache->slot_stride * e;
    a.T = nodes;
    a.P = cache->table_width;
    a.heads = cache->kv_heads;
    a.units = cache->dim * e / 16;
    a.pages = cache->num_pages;
    a.shift = page_shift(cache->page_size);
    const int64_t blocks =
        (static_cast<int64_t>(nodes) * a.heads * a.units + kCacheBlock - 1) / kCacheBlock;
    if (blocks > INT32_MAX / cache->batch || !grid_fits(blocks * cache->batch, kCacheBlock))
        return SPEC_ERR_UNSUPPORTED;
    a.blocks = static_cast<int32_t>(blocks);
    cache_append_kernel<<<dim3(static_cast<unsigned>(blocks * cache->batch)), dim3(kCacheBlock),
                          0, static_cast<hipStream_t>(stream)>>>(a);
    return launch_status();
}

spec_status spec_tree_accept(const int32_t *parents, const int32_t *tokens,
                             const int32_t *chosen, const int32_t *num_nodes, int32_t batch,
                             int32_t nodes, int32_t *path, int32_t *count, int32_t *emitted,
                             void *stream) {
    if (batch < 0 || nodes < 1) return SPEC_ERR_ARG;
    if (nodes > kMaxAcceptNodes) return SPEC_ERR_UNSUPPORTED;
    if (batch == 0) return SPEC_OK;
    if (!parents || !tokens || !chosen || !path || !count || !emitted) return SPEC_ERR_ARG;
    // a sequence's row is read before it is written, so an output may be an input
    const int64_t row = int64_t{batch} * nodes;
    const Range to[] = {ints(path, row), ints(emitted, row), ints(count, batch)};
    const Range in[] = {ints(parents, row), ints(tokens, row), ints(chosen, row),
                        ints(num_nodes, batch)};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < i; ++j)
            if (to[i].meets(to[j])) return SPEC_ERR_ARG;
        for (const Range &r : in)
            if (to[i].meets(r) && !(to[i].from == r.from && to[i].to == r.to)) return SPEC_ERR_ARG;
    }
    AcceptArgs a{};
    a.parents = parents;
    a.tokens = tokens;
    a.chosen = chosen;
    a.nodes = num_nodes;
    a.path = path;
    a.count = count;
    a.emitted = emitted;
    a.B = batch;
    a.T = nodes;
    constexpr int per = kCacheBlock / kWave;
    const int64_t blocks = (static_cast<int64_t>(batch) + per - 1) / per;
    if (!grid_fits(blocks, kCacheBlock)) return SPEC_ERR_UNSUPPORTED;
    tree_accept_kernel<<<dim3(static_cast<unsigned>(blocks)), dim3(kCacheBlock), 0,
                         static_cast<hipStream_t>(stream)>>>(a);
    return launch_status();
}

spec_status spec_cache_keep(const spec_cache_pools *pools, const int32_t *table,
                            int32_t table_width, const int32_t *lengths, const int32_t *path,
                            const int32_t *count, int32_t batch, int32_t nodes,
                            int32_t *new_lengths, void *stream) {
    spec_status s = check_pools(pools, true);
    if (s != SPEC_OK) return s;
    if ((s = check_table(table_width, pools->page_size, pools->num_pages)) != SPEC_OK) return s;
    if (batch < 0 || nodes < 1) return SPEC_ERR_ARG;
    if (nodes > kMaxKeepNodes) return SPEC_ERR_UNSUPPORTED;
    if (batch == 0) return SPEC_OK;
    if (!table || !lengths || !path || !count || !new_lengths) return SPEC_ERR_ARG;
    const Range to[] = {ints(new_lengths, batch)};
    const Range in[] = {ints(lengths, batch), ints(count, batch),
                        ints(path, int64_t{batch} * nodes),
                        ints(table, int64_t{batch} * table_width)};
    if (writes_meet(to, in)) return SPEC_ERR_ARG;
    for (int i = 0; i < pools->num_pools; ++i) {
        const Range pool = range(pools->bases[i], pool_bytes(pools));
        for (const Range &r : in)
            if (pool.meets(r)) return SPEC_ERR_ARG;
        if (pool.meets(to[0])) return SPEC_ERR_ARG;
    }
    KeepArgs a{};
    a.table = table;
    a.lengths = lengths;
    a.path = path;
    a.count = count;
    a.T = nodes;
    a.P = table_width;
    const int64_t column = static_cast<int64_t>(pools->heads) * (pools->slot_bytes / 16);
    // no pools: the lengths alone
    const int step = pools->num_pools ? keep_pools_per_launch(column, batch, pools->num_pools) : 1;
    if (step == 0 || !grid_fits(batch, kCacheBlock)) return SPEC_ERR_UNSUPPORTED;
    for (int first = 0; first == 0 || first < pools->num_pools; first += step) {
        const int n = pools->num_pools - first < step ? pools->num_pools - first : step;
        a.pool = pool_args(pools, first, n);
        a.new_lengths = first == 0 ? new_lengths : nullptr;
        a.blocks = static_cast<int32_t>(keep_blocks(column, n));
        cache_keep_kernel<<<dim3(static_cast<unsigned>(a.blocks * batch)), dim3(kCacheBlock), 0,
                            static_cast<hipStream_t>(stream)>>>(a);
        if ((s = launch_status()) != SPEC_OK) return s;
    }
    return SPEC_OK;
}

spec_status spec_pages_fork(const int32_t *table, const int32_t *lengths, const int32_t *parents,
                            int32_t batch, int32_t num_beams, int32_t num_out,
                            int32_t table_width, int32_t page_size, int32_t num_pages,
                            int32_t *refs, int32_t *out_table, int32_t *out_lengths,
                            void *stream) {
    const spec_status s = check_table(table_width, page_size, num_pages);
    if (s != SPEC_OK) return s;
    if (batch < 0 || num_beams < 1 || num_out < 1) return SPEC_ERR_ARG;
    if (batch == 0) return SPEC_OK;
    if (!table || !lengths || !parents || !refs || !out_table || !out_lengths) return SPEC_ERR_ARG;
    const int64_t rows = static_cast<int64_t>(batch) * num_out;
    const int64_t from = static_cast<int64_t>(batch) * num_beams;
    if (!grid_fits(rows, kCacheBlock) || from > INT32_MAX) return SPEC_ERR_UNSUPPORTED;
    const Range to[] = {ints(out_table, rows * table_width), ints(out_lengths, rows),
                        ints(refs, num_pages)};
    const Range in[] = {ints(table, from * table_width), ints(lengths, from), ints(parents, rows)};
    if (writes_meet(to, in)) return SPEC_ERR_ARG;
    ForkArgs a{};
    a.table = table;
    a.lengths = lengths;
    a.parents = parents;
    a.refs = refs;
    a.out = out_table;
    a.out_lengths = out_lengths;
    a.W = num_beams;
    a.n = num_out;
    a.P = table_width;
    a.shift = page_shift(page_size);
    a.pages = num_pages;
    pages_fork_kernel<<<dim3(static_cast<unsigned>(rows)), dim3(kCacheBlock), 0,
                        static_cast<hipStream_t>(stream)>>>(a);
    return launch_status();
}

spec_status spec_pages_release(int32_t *table, const int32_t *lengths, int32_t rows,
                               int32_t table_width, int32_t page_size, int32_t num_pages,
                               int32_t *refs, void *stream) {
    const spec_status s = check_table(table_width, page_size, num_pages);
    if (s != SPEC_OK) return s;
    if (rows < 0) return SPEC_ERR_ARG;
    if (rows == 0) return SPEC_OK;
    if (!table || !refs) return SPEC_ERR_ARG;
    if (!grid_fits(rows, kCacheBlock)) return SPEC_ERR_UNSUPPORTED;
    const Range to[] = {ints(table, int64_t{rows} * table_width), ints(refs, num_pages)};
    const Range in[] = {ints(lengths, rows)};
    if (writes_meet(to, in)) return SPEC_ERR_ARG;
    ReleaseArgs a{};
    a.table = table;
    a.refs = refs;
    a.lengths = lengths;
    a.P = table_width;
    a.shift = page_shift(page_size);
    a.pages = num_pages;
    pages_release_kernel<<<dim3(static_cast<unsigned>(rows)), dim3(kCacheBlock), 0,
                           static_cast<hipStream_t>(stream)>>>(a);
    return launch_status();
}

size_t spec_pages_reserve_workspace_bytes(int32_t rows, int32_t num_pages) {
    if (rows < 1 || num_pages < 1 || rows > kMaxReserveRows || num_pages > kMaxReservePages)
        return 0;
    return plan_reserve(num_pages).total;
}

spec_status spec_pages_reserve(int32_t *table, const int32_t *lengths,
                               const int32_t *new_positions, int32_t rows, int32_t table_width,
                               int32_t page_size, int32_t num_pages, int32_t *refs,
                               int32_t *copies, int32_t *missing, void *workspace,
                               size_t workspace_bytes, void *stream) {
    const spec_status s = check_table(table_width, page_size, num_pages);
    if (s != SPEC_OK) return s;
    if (rows < 0) return SPEC_ERR_ARG;
    if (rows > kMaxReserveRows || num_pages > kMaxReservePages) return SPEC_ERR_UNSUPPORTED;
    if (rows == 0) return SPEC_OK;
    if (!table || !lengths || !new_positions || !refs || !copies || !missing) return SPEC_ERR_ARG;
    const ReservePlan p = plan_reserve(num_pages);
    if (!workspace || workspace_bytes < p.total) return SPEC_ERR_WORKSPACE;
    if (!aligned16(workspace)) return SPEC_ERR_ARG;
    const Range to[] = {ints(table, int64_t{rows} * table_width), ints(refs, num_pages),
                        ints(copies, int64_t{rows} * 3), ints(missing, 1),
                        range(workspace, static_cast<int64_t>(p.total))};
    const Range in[] = {ints(lengths, rows), ints(new_positions, rows)};
    if (writes_meet(to, in)) return SPEC_ERR_ARG;
    char *w = static_cast<char *>(workspace);
    ReserveArgs a{};
    a.table = table;
    a.refs = refs;
    a.copies = copies;
    a.missing = missing;
    a.lengths = lengths;
    a.news = new_positions;
    a.words = reinterpret_cast<unsigned long long *>(w + p.words);
    a.before = reinterpret_cast<int32_t *>(w + p.before);
    a.counts = reinterpret_cast<int32_t *>(w + p.counts);
    a.rows = rows;
    a.P = table_width;
    a.shift = page_shift(page_size);
    a.pages = num_pages;
    a.chunks = p.chunks;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (a.chunks > kReserveAlone) {
        constexpr int per = kCacheBlock / kWave;
        pages_free_kernel<<<dim3(static_cast<unsigned>((a.chunks + per - 1) / per)),
                            dim3(kCacheBlock), 0, st>>>(a);
        const spec_status r = launch_status();
        if (r != SPEC_OK) return r;
    }
    pages_reserve_kernel<<<dim3(1), dim3(kReserveBlock), 0, st>>>(a);
    return launch_status();
}

spec_status spec_pages_copy(const spec_cache_pools *pools, const int32_t *copies, int32_t rows,
                            void *stream) {
    spec_status s = check_pools(pools, false);
    if (s != SPEC_OK) return s;
    if (rows < 0) return SPEC_ERR_ARG;
    if (rows == 0 || pools->num_pools == 0) return SPEC_OK;
    if (!copies) return SPEC_ERR_ARG;
    for (int i = 0; i < pools->num_pools; ++i)
        if (range(pools->bases[i], pool_bytes(pools)).meets(ints(copies, int64_t{rows} * 3)))
            return SPEC_ERR_ARG;
    CopyArgs a{};
    a.copies = copies;
    const int step = copy_pools_per_launch(rows, pools->heads, pools->num_pools);
    if (step == 0) return SPEC_ERR_UNSUPPORTED;
    for (int first = 0; first < pools->num_pools; first += step) {
        const int n = pools->num_pools - first < step ? pools->num_pools - first : step;
        a.pool = pool_args(pools, first, n);
        pages_copy_kernel<<<dim3(static_cast<unsigned>(rows * pools->heads * n)),
                            dim3(kCacheBlock), 0, static_cast<hipStream_t>(stream)>>>(a);
        if ((s = launch_status()) != SPEC_OK) return s;
    }
    return SPEC_OK;
}

}  // extern "C"
