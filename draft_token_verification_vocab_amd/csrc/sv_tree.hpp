// sv_tree.hpp -- attention of a chain or a tree of new tokens over a paged
// cache.
//
// For each sequence and key head the G query heads that share it and the T new
// tokens (nodes) make M = T*G query rows over the same n keys:
//   out = sum_p e^(s_p - lse) v_p,   s_p = scale q.k_p,   lse = ln sum_p e^s_p
// over the cached positions p < L, which every row sees, and the row's own node
// and its ancestors among the n - L nodes behind them.
//
// One pass over the keys with a running maximum and sum per row:
//   S^T = K Q^T   a lane's operand is 8 consecutive elements of a key's row.  The
//                 instruction's 16 rows are given keys in the order that leaves
//                 lane group g (of four) with the scores of keys 8g..8g+7, all of
//                 one query row.
//   O^T = V^T P^T those 8 weights are the lane's operand as they stand; the
//                 other one is 8 keys' values of one dimension.
// A query row is a column throughout, so its maximum, sum and rescaling stay in
// its lanes.  Products are added in 32 bits.  For 16-bit types the weights are
// rounded to the type before the second product, as its matrix instructions take
// them: a relative 2^-9 (bfloat16) or 2^-12 (float16) of each, with independent signs;
// float16 weights below 2^-23 of the row's largest keep an absolute 2^-34 of it instead
// (see kLift).  lse comes from their sum before that rounding, in 32 bits.
//
// Two kernels: tree_wide_kernel for 16-bit types, where rows are shared out to the
// waves and keys come through shared memory, and tree_attention_kernel for
// float32, where keys are shared out to the waves and come straight into
// registers (a tile of float32 keys and values takes twice the shared memory, for
// products of a 16th of the rate).
//
// The keys of all sequences are cut into tiles of 128 and the tiles dealt out
// evenly to as many workgroups as the chip holds, rounded up: a workgroup takes a
// run of tiles, which may end inside a sequence and hold several short ones, so
// ragged batches load every workgroup alike.  More, smaller runs were slower (1.5, 2 and 3
// times as many).  A sequence whose tiles are in several workgroups is joined by a
// second launch.  Where every sequence is short, a workgroup takes a whole one
// and there is none.
//
// Measured (kernel + join, medians of traces of 60 calls): 64 single tokens over up to
// 4000 positions, 552 MB, 90.4 + 4.8 us (6.1 TB/s); 64 chains of nine over up to 8000,
// 1.19 GB, 203 + 12 (5.9 TB/s); two caches of 131072, 1.03 GB, 173 + 10.8 (5.9 TB/s):
// memory.  16 trees of 64 nodes, 64 heads, over up to 12000 positions, 225 GFLOP, 321 +
// 28 (702 TFLOP/s in the main kernel; the fastest call 290 + 25, and 309 to 322 for both
// without a trace): the exponentials' and conversions' issue beside the products, and
// shared memory, of which each wave reads a whole tile for 32 rows: four waves' 128 KB
// to 64 keys take as many cycles at 128 bytes as their products at the full rate.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "sv_common.hpp"

namespace sv {

constexpr int kTreeBlock = 256;
constexpr int kTreeWaves = kTreeBlock / kWave;
constexpr int kTreeKeys = 32;                        // a wave's keys at a time
constexpr int kTreeTile = kTreeKeys * kTreeWaves;    // the unit that is dealt out
constexpr int kMaxTreeNodes = 128;                   // of a tree; chains may be longer

typedef unsigned int v2u32 __attribute__((ext_vector_type(2)));
typedef float v4f32 __attribute__((ext_vector_type(4)));
typedef float v8f32 __attribute__((ext_vector_type(8)));
typedef __bf16 v8bf16 __attribute__((ext_vector_type(8)));
typedef _Float16 v8f16 __attribute__((ext_vector_type(8)));

struct TreeArgs {
    const void *keys;
    const void *values;
    const void *q;
    void *out;               // [B][T][H][D]
    float *lse;              // [B][T][H] or null
    const int32_t *table;    // [B][P]
    const int32_t *lengths;  // [B]
    const int32_t *nodes;    // [B] or null (= T)
    const int32_t *parents;  // [B][T] or null (a chain)
    float *part;             // [workgroup][2][rows][D]: unfinished sums
    float *part_ml;          // [workgroup][2][rows][4]: reference, sum, divisor of the output
    int32_t *first;          // [B + 1]: sequences' first tiles, then the tiles per slice
    int64_t page_stride, head_stride, slot_stride;  // elements
    int64_t q_batch, q_node, q_head;                // elements
    int32_t B, T, H, KV, G, D, P;
    int32_t pages, shift;    // page size 2^shift
    int32_t slices, mtiles, whole;
    float scale2;            // scale * log2(e)
};

// Types of keys and values.  Frag: a matrix operand's 8 elements along the
// summed dimension; load8: 8 consecutive elements; kTop: the power of two that
// weights may reach where the type's exponents are too few below 1 (else 0).
template <typename T>
struct TreeElem;

template <typename V8>
struct TreeElem16 {
    using Frag = V8;
    struct Raw {
        v4u32 w;
    };
    __device__ static __forceinline__ Frag frag(const Raw &r) {
        return __builtin_bit_cast(V8, r.w);
    }
    __device__ static __forceinline__ Frag from(const float *x) {
        v8f32 v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = x[j];
        return __builtin_convertvector(v, V8);
    }
    __device__ static __forceinline__ Frag ones() {
        const float x[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
        return from(x);
    }
};

template <>
struct TreeElem<__bf16> : TreeElem16<v8bf16> {
    __device__ static __forceinline__ v4f32 mma(Frag a, Frag b, v4f32 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static constexpr uint32_t kExponent = 0x7F80u;
    static constexpr float kTop = 0.0f;
};

template <>
struct TreeElem<_Float16> : TreeElem16<v8f16> {
    __device__ static __forceinline__ v4f32 mma(Frag a, Frag b, v4f32 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static constexpr uint32_t kExponent = 0x7C00u;
    static constexpr float kTop = 15.0f;
};

template <>
struct TreeElem<float> {
    using Frag = v8f32;
    struct Raw {
        v8f32 w;
    };
    __device__ static __forceinline__ Frag frag(const Raw &r) { return r.w; }
    __device__ static __forceinline__ Frag from(const float *x) {
        v8f32 v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = x[j];
        return v;
    }
    // The sum's order is free, so element j of every lane group makes one
    // instruction of four terms.
    __device__ static __forceinline__ v4f32 mma(const Frag &a, const Frag &b, v4f32 c) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
        return c;
    }
};

template <typename T>
__device__ __forceinline__ typename TreeElem<T>::Raw tree_load8(const T *p) {
    return *reinterpret_cast<const typename TreeElem<T>::Raw *>(p);
}
// float32 keys and values are read once, so past the caches' usual order.
__device__ __forceinline__ v8f32 tree_stream8(const float *p) {
    return __builtin_nontemporal_load(reinterpret_cast<const v8f32 *>(p));
}

template <int C>
__device__ __forceinline__ void tree_load_row(const float *p, uint32_t *w) {
#pragma unroll
    for (int i = 0; i < C / 4; ++i) {
        const v4u32 v = __builtin_nontemporal_load(reinterpret_cast<const v4u32 *>(p) + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[4 * i + k] = v[k];
    }
}

// Element t of 8 keys' rows as an operand.
template <int C>
__device__ __forceinline__ v8f32 tree_column(const uint32_t (&w)[8][C], int t) {
    v8f32 v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j][t]);
    return v;
}

// A word with its infinities and NaNs taken out.
template <typename T>
__device__ __forceinline__ uint32_t tree_finite(uint32_t w) {
    if constexpr (sizeof(T) == 4) {
        return (w & 0x7F800000u) == 0x7F800000u ? 0u : w;
    } else {
        constexpr uint32_t e = TreeElem<T>::kExponent;
        if ((w & e) == e) w &= 0xFFFF0000u;
        return ((w >> 16) & e) == e ? w & 0xFFFFu : w;
    }
}

// A barrier over shared memory alone: stores to memory need not have arrived.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

__device__ __forceinline__ float across_groups_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16, kWave));
    return fmaxf(v, __shfl_xor(v, 32, kWave));
}
__device__ __forceinline__ float across_groups_sum(float v) {
    v += __shfl_xor(v, 16, kWave);
    return v + __shfl_xor(v, 32, kWave);
}

// A sequence's keys and nodes as far as its table row reaches.
struct TreeSpan {
    int cached;  // L
    int live;    // nodes in use
    int keys;    // positions that are read: L + live, within the table
};
__device__ __forceinline__ TreeSpan tree_span(const TreeArgs &a, int b) {
    const int room = a.P << a.shift;
    TreeSpan s;
    s.live = a.nodes ? clamp_len(a.nodes[b], a.T) : a.T;
    s.cached = clamp_len(a.lengths[b], room);
    s.keys = s.live == 0 ? 0 : (s.cached > room - s.live ? room : s.cached + s.live);
    return s;
}
__device__ __forceinline__ int tree_tiles(int keys) {
    return keys <= kTreeTile ? 1 : (keys + kTreeTile - 1) / kTreeTile;
}

// Whether a row sees a node: its own or an ancestor.
__device__ __forceinline__ bool tree_sees(const uint64_t (*mask)[2], bool chain, int row_node,
                                          int node) {
    if (chain) return node <= row_node;
    return (mask[row_node][node >> 6] >> (node & 63)) & 1;
}

// Which of the 8 positions from node `at` on (below 0: cached ones) a row sees, a
// bit for each; nothing where its node is -1.
__device__ __forceinline__ uint32_t tree_sees8(const uint64_t (*mask)[2], bool chain,
                                               int row_node, int at) {
    if (row_node < 0) return 0;
    // bits 0..7 of a window that begins at node `at`
    if (chain) {
        const int n = row_node + 1 - at;  // positions up to the row's own node
        return n >= 8 ? 0xFFu : (n <= 0 ? 0u : (1u << n) - 1);
    }
    if (at <= -8) return 0xFFu;
    const uint64_t lo = mask[row_node][0], hi = mask[row_node][1];
    if (at < 0) return (static_cast<uint32_t>(lo << -at) | ((1u << -at) - 1)) & 0xFFu;
    if (at >= 128) return 0;
    const uint64_t w = at >= 64 ? hi >> (at - 64) : (lo >> at) | (at ? hi << (64 - at) : 0);
    return static_cast<uint32_t>(w) & 0xFFu;
}

// Where values of nodes hold an infinity or a NaN: positions [from, to), as tiles.
struct TreeOdd {
    int from, to;
    __device__ __forceinline__ void clear() {
        from = 0x7FFFFFFF;
        to = 0;
    }
    __device__ __forceinline__ void add(int at, int n) {
        atomicMin(&from, at);
        atomicMax(&to, at + n);
    }
};

// Queries and joined sums are not needed at the same time.
template <int DP, int R>
struct TreeShared {
    static constexpr int kPitch = DP + 4;  // 16 rows' starts on different banks
    // row tiles that are joined at a time, by what shared memory holds beside
    // another workgroup's
    static constexpr int kJoin = R == 2 && DP <= 128 ? 2 : 1;
    union {
        float merge[kJoin][kTreeWaves][16][kPitch];
        v8f32 q[R][DP / 32][kWave];
    };
    float ml[kTreeWaves][16 * R][2];
    int node[16 * R];  // a row's node
    TreeOdd odd;
    uint64_t mask[kMaxTreeNodes][2];
    int up[kMaxTreeNodes];
};

// The thread's index as a value the compiler knows nothing about, so that what
// a segment's beginning and end derive from it is not kept in registers
// throughout the loop between them.
__device__ __forceinline__ int fresh_tid() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

__device__ __forceinline__ int tree_scan(int v, int lane) {
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int u = __shfl_up(v, o, kWave);
        if (lane >= o) v += u;
    }
    return v;
}

struct TreePlace {
    int start, end;  // this slice's tiles
    int b, first;    // the sequence that holds start, and its first tile
    TreeSpan span;   // of that sequence
};

// Finds a slice's place, in every wave for itself: a lane adds up an equal share
// of the sequences, a scan over the lanes finds the share that holds the
// slice's first tile, and a second one, over that share, the sequence.
// Workgroup 0 leaves the sequences' first tiles for the second launch.  Where
// sequences are not cut (whole), a slice is a sequence.
__device__ __forceinline__ TreePlace tree_plan(const TreeArgs &a, int slice, int lane,
                                               bool leave) {
    if (a.whole) {
        TreePlace p{};
        p.b = slice;
        p.span = tree_span(a, slice);
        p.end = tree_tiles(p.span.keys);
        return p;
    }
    const int share = (a.B + kWave - 1) / kWave;
    int mine = 0;
    for (int k = 0; k < share; ++k) {
        const int i = lane * share + k;
        if (i < a.B) mine += tree_tiles(tree_span(a, i).keys);
    }
    const int upto = tree_scan(mine, lane);
    const int total = __builtin_amdgcn_readlane(upto, kWave - 1);
    const int per = (total + a.slices - 1) / a.slices;
    if (leave) {
        int before = upto - mine;
        for (int k = 0; k < share; ++k) {
            const int i = lane * share + k;
            if (i >= a.B) break;
            a.first[i] = before;
            before += tree_tiles(tree_span(a, i).keys);
        }
        if (lane == 0) a.first[a.B] = per;
    }
    TreePlace p{};
    p.start = slice * per;
    p.end = p.start + per < total ? p.start + per : total;
    if (p.start >= total) return p;
    uint64_t found = __ballot(p.start < upto);
    const int at = __builtin_amdgcn_readfirstlane(__ffsll(static_cast<long long>(found)) - 1);
    int before = __builtin_amdgcn_readlane(upto - mine, at);
    for (int i0 = at * share;; i0 += kWave) {
        const int i = i0 + lane;
        const bool in = i < at * share + share && i < a.B;
        const TreeSpan span = in ? tree_span(a, i) : TreeSpan{0, 0, 0};
        const int upto_i = before + tree_scan(in ? tree_tiles(span.keys) : 0, lane);
        found = __ballot(p.start < upto_i);
        if (found) {
            const int k =
                __builtin_amdgcn_readfirstlane(__ffsll(static_cast<long long>(found)) - 1);
            p.b = i0 + k;
            p.span.cached = __builtin_amdgcn_readlane(span.cached, k);
            p.span.live = __builtin_amdgcn_readlane(span.live, k);
            p.span.keys = __builtin_amdgcn_readlane(span.keys, k);
            p.first = __builtin_amdgcn_readlane(upto_i, k) - tree_tiles(p.span.keys);
            return p;
        }
        before = __builtin_amdgcn_readlane(upto_i, kWave - 1);
    }
}

// Ancestor masks of a tree's nodes, the node itself included, by doubling the
// distance of the jump: 7 rounds for 128 nodes.  A parent that does not precede
// its node makes it a root.
template <typename Shared>
__device__ __forceinline__ void tree_masks(const TreeArgs &a, Shared &sh, int b, int live) {
    const int i = fresh_tid();
    if (i < kMaxTreeNodes) {
        int up = i < live ? a.parents[static_cast<int64_t>(b) * a.T + i] : -1;
        if (up < 0 || up >= i) up = -1;
        sh.up[i] = up;
        sh.mask[i][0] = i < 64 ? 1ull << i : 0;
        sh.mask[i][1] = i < 64 ? 0 : 1ull << (i - 64);
    }
    lds_barrier();
    for (int round = 1; round < live; round <<= 1) {
        uint64_t m0 = 0, m1 = 0;
        int up = -1;
        if (i < live && sh.up[i] >= 0) {
            up = sh.up[sh.up[i]];
            m0 = sh.mask[sh.up[i]][0];
            m1 = sh.mask[sh.up[i]][1];
        }
        lds_barrier();
        if (i < live) {
            sh.up[i] = up;
            sh.mask[i][0] |= m0;
            sh.mask[i][1] |= m1;
        }
        lds_barrier();
    }
}

// Adds the infinities and NaNs among the values of nodes, between positions
// `from` and `to`, to the rows that see them: a weight above 0 times one is that
// again.  The workgroup's rows row0 .. row0 + rows - 1 have been written, to out
// (whole) or to its part.  A thread takes a dimension and a run of rows.  Of a chain
// it walks along the positions once, as a row sees all up to its own: a running sum
// goes to each row in turn.  Of a tree it keeps which nodes hold what, in bits, and
// meets them with what a row sees.
template <typename T>
__device__ __forceinline__ void tree_add_odd(const TreeArgs &a, const uint64_t (*mask)[2],
                                             const TreeOdd &odd, const TreeSpan &span, int b,
                                             int h, int from, int to, bool whole, int64_t slot,
                                             int row0, int rows) {
    __threadfence_block();
    __syncthreads();
    const int threads = kTreeBlock / a.D, d = threadIdx.x % a.D, k = threadIdx.x / a.D;
    if (k >= threads) return;
    int in = rows * k / threads, end = rows * (k + 1) / threads;
    if (end > span.live * a.G - row0) end = span.live * a.G - row0;  // rows in use
    if (from < span.cached) from = span.cached;
    if (from < odd.from) from = odd.from;
    if (to > odd.to) to = odd.to;
    // rows of nodes before the first of them
    const int64_t before = static_cast<int64_t>(from - span.cached) * a.G - row0;
    if (in < before) in = before < end ? static_cast<int>(before) : end;
    if (in >= end) return;
    const int last = (row0 + end - 1) / a.G;
    if (to > span.cached + last + 1) to = span.cached + last + 1;

    auto add = [&](int i, float sum) {
        const int row = row0 + i;
        if (whole) {
            T *out = static_cast<T *>(a.out) + ((static_cast<int64_t>(b) * a.T + row / a.G) * a.H +
                                                h * a.G + row % a.G) *
                                                   a.D + d;
            *out = static_cast<T>(static_cast<float>(*out) + sum);
        } else {
            a.part[(slot * rows + i) * a.D + d] += sum;
        }
    };
    const bool chain = a.parents == nullptr;
    const int32_t *table = a.table + static_cast<int64_t>(b) * a.P;
    float sum = 0.0f;
    int node = (row0 + in) / a.G;
    uint64_t up[2] = {0, 0}, down[2] = {0, 0};  // nodes of +inf or NaN, of -inf or NaN
    for (int p0 = from & ~7; p0 < to && in < end && !(sum != sum); p0 += 8) {
        const int page = table[p0 >> a.shift];
        const bool held = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pages);
        const T *at = static_cast<const T *>(a.values) + (held ? page : 0) * a.page_stride +
                      h * a.head_stride + (p0 & ((1 << a.shift) - 1)) * a.slot_stride + d;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = static_cast<float>(at[j * a.slot_stride]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int n = p0 + j - span.cached;
            if (p0 + j < from || p0 + j >= to) continue;
            if (held && !(__builtin_fabsf(v[j]) < __builtin_inff())) {
                sum += v[j];
                if (!chain) {
                    const uint64_t bit = 1ull << (n & 63);
                    if (!(v[j] < 0.0f)) up[n >> 6] |= bit;
                    if (!(v[j] > 0.0f)) down[n >> 6] |= bit;
                }
            }
            if (!chain) continue;
            for (; in < end && node <= n; ++in, node = (row0 + in) / a.G)
                if (!(sum == 0.0f)) add(in, sum);
        }
        if (!chain) sum = 0.0f;
    }
    for (; in < end; ++in) {
        if (!chain) {
            node = (row0 + in) / a.G;
            sum = 0.0f;
            if ((mask[node][0] & up[0]) | (mask[node][1] & up[1])) sum += __builtin_inff();
            if ((mask[node][0] & down[0]) | (mask[node][1] & down[1])) sum -= __builtin_inff();
        }
        if (!(sum == 0.0f)) add(in, sum);
    }
}

// Waves that a compute unit's SIMD holds, by the registers that R row tiles need
// (an accumulator takes DP/4 of them, a block's keys and values DP).
constexpr int tree_waves(int dp) { return dp == 64 ? 2 : 1; }

// float32: the workgroup's four waves take 32 keys at a time in turn, each for all of
// its 16 R rows, straight from memory into the matrix instructions' registers, and
// join through shared memory at the end.  Two row tiles to a wave halve what is
// loaded for a row; at 256 dimensions their registers would leave nothing for loads
// in flight (64 nodes, 774 us against 735 with one).  13 nodes of five sequences of
// up to 1500 positions, 80 dimensions: 16.6 us (and 4.0 joined), a chain of dependent
// reads, products (80 dimensions computed as 128, 39 rows as 64) and the waves' join.
// 16 trees of 64 nodes, 32 heads on 8, over 2000 to 4000 positions reach 71, 85 and 37
// TFLOP/s at 64, 128 and 256 dimensions of the 137 of a large product: with one wave to
// a SIMD (two at 64) nothing else fills the time of exponentials and late loads, and at
// 256 a block of keys and values feeds 16 rows alone.
// FULL: a slot has DP elements and the next one follows it, so that the
// loads of a block share their addresses; otherwise fewer than DP or further apart.
template <int DP, int R, bool FULL>
__global__ __launch_bounds__(kTreeBlock, tree_waves(DP)) void tree_attention_kernel(TreeArgs a) {
    using T = float;
    using E = TreeElem<T>;
    using Frag = typename E::Frag;
    using Raw = typename E::Raw;
    constexpr int kSteps = DP / 32;             // matrix instructions along a key's row
    constexpr int kCols = DP / 16;              // along the output's dimensions
    constexpr int kChunk = kCols < 8 ? kCols : 8;   // elements of a value load
    constexpr int kChunks = kCols / kChunk;
    using Shared = TreeShared<DP, R>;
    __shared__ Shared sh;

    const int units = a.slices * a.KV;
    const int mt = blockIdx.x / units;
    const int slice = (blockIdx.x % units) / a.KV;
    const int h = blockIdx.x % a.KV;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int i16 = lane & 15, g = lane >> 4;
    const bool chain = a.parents == nullptr;

    TreePlace place = tree_plan(a, slice, lane, blockIdx.x == 0 && wave == 0);
    int tile = place.start, b = place.b, first = place.first;
    const int end = place.end;
    TreeSpan span = place.span;

    // this lane's place in a key's row and in a value's; past the row's end
    // (D < DP) it reads its start, and a key's elements there become 0 (the
    // queries' are 0 too); the values' dimensions there are never written
    const int slot_mask = (1 << a.shift) - 1;
    const int64_t slot_stride = FULL ? DP : a.slot_stride;
    const T *keys = static_cast<const T *>(a.keys) + h * a.head_stride;
    const T *values = static_cast<const T *>(a.values) + h * a.head_stride;
    int dk[kSteps], dv[kChunks];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) dk[s] = FULL || 32 * s + 8 * g < a.D ? 32 * s + 8 * g : 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        dv[c] = c * 16 * kChunk + i16 * kChunk;
        if (!FULL && dv[c] >= a.D) dv[c] = 0;
    }

    while (tile < end) {
        const int nt = tree_tiles(span.keys);
        const int from = tile - first;
        const int to = nt < from + end - tile ? nt : from + end - tile;
        const bool whole = from == 0 && to == nt;
        const bool dead = mt * 16 * R >= span.live * a.G;  // no row in use
        const int32_t *table = a.table + static_cast<int64_t>(b) * a.P;

        // no row sees past its own node, so this workgroup's last one bounds the keys
        const int last = ((mt + 1) * 16 * R - 1) / a.G;
        int keys_end = to * kTreeTile < span.keys ? to * kTreeTile : span.keys;
        if (last < span.live && keys_end > span.cached + last + 1)
            keys_end = span.cached + last + 1;
        if (dead) keys_end = 0;

        // the queries: a row's operand in the lanes that take it
        constexpr int kQueries = (R * kSteps * kWave + kTreeBlock - 1) / kTreeBlock;
        Raw queries[kQueries];
        const int qt = fresh_tid();
#pragma unroll
        for (int k = 0; k < kQueries; ++k) {
            const int e = k * kTreeBlock + qt;
            const int s = e / kWave % kSteps, r = e / kWave / kSteps;
            const int row = (mt * R + r) * 16 + (qt & 15);
            const int node = row / a.G, d = 32 * s + 8 * (qt >> 4 & 3);
            queries[k] = Raw{};
            if (r < R && node < a.T && d < a.D)
                queries[k] = tree_load8<T>(static_cast<const T *>(a.q) + b * a.q_batch +
                                           node * a.q_node + (h * a.G + row % a.G) * a.q_head + d);
        }
        const int mine = (mt * 16 * R + qt) / a.G;  // the node of row qt

        // the pages of the keys that this lane loads at p0: keys 8(i16/4).. of the
        // first product, keys 8g.. of the second
        // (an entry behind the sequence's end may be anything, and its page, if it is
        // one, is read and not used)
        auto entry_of = [&](int p) {
            const int e = p >> a.shift;
            return table[e < a.P ? e : a.P - 1];
        };
        auto is_page = [&](int e) {
            return static_cast<uint32_t>(e) < static_cast<uint32_t>(a.pages);
        };
        Frag kf[2][kSteps];
        uint32_t vw[kChunks][8][kChunk];
        auto load_keys = [&](int p0, int page) {
            if (!is_page(page)) page = 0;
            const T *kp = keys + page * a.page_stride +
                          (((p0 + 8 * (i16 >> 2)) & slot_mask) + (i16 & 3)) * slot_stride;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
                    kf[c][s] = tree_stream8(kp + 4 * c * slot_stride + dk[s]);
        };
        auto load_values = [&](int p0, int page) {
            if (!is_page(page)) page = 0;
            const T *vp = values + page * a.page_stride +
                          ((p0 + 8 * g) & slot_mask) * slot_stride;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    tree_load_row<kChunk>(vp + j * slot_stride + dv[c], vw[c][j]);
        };
        int p0 = from * kTreeTile + wave * kTreeKeys;
        int page_k = -1, page_v = -1, next_k = -1, next_v = -1;
        if (p0 < keys_end) {
            page_k = entry_of(p0 + 8 * (i16 >> 2));
            page_v = entry_of(p0 + 8 * g);
            next_k = entry_of(p0 + kTreeTile + 8 * (i16 >> 2));
            next_v = entry_of(p0 + kTreeTile + 8 * g);
            load_keys(p0, page_k);
            load_values(p0, page_v);
        }

        lds_barrier();
        if (!dead && keys_end > span.cached && !chain) tree_masks(a, sh, b, span.live);
#pragma unroll
        for (int k = 0; k < kQueries; ++k)
            if (k * kTreeBlock + qt < R * kSteps * kWave)
                (&sh.q[0][0][0])[k * kTreeBlock + qt] = queries[k].w;
        if (qt < 16 * R) sh.node[qt] = mine;
        if (qt == 0) sh.odd.clear();
        lds_barrier();

        float m[R], l[R];  // a row's maximum, scaled to powers of two, and the lane's sum
        v4f32 o[R][kCols];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -__builtin_inff();
            l[r] = 0.0f;
#pragma unroll
            for (int t = 0; t < kCols; ++t) o[r][t] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};
        }

        v4f32 z[R][2];
        auto score = [&]() {
            asm volatile("" ::: "memory");  // the queries are read again, not kept
            if (!FULL) {
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
                    if (32 * s + 8 * g >= a.D) kf[0][s] = kf[1][s] = E::frag(Raw{});
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                z[r][0] = z[r][1] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    const Frag qf = sh.q[r][s][lane];
                    z[r][0] = E::mma(kf[0][s], qf, z[r][0]);
                    z[r][1] = E::mma(kf[1][s], qf, z[r][1]);
                }
            }
        };
        auto add_values = [&]() {
            // a maximum that has been passed moves
            float top[R];
            bool behind = false;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float t = z[r][0][0];
#pragma unroll
                for (int j = 1; j < 8; ++j) t = fmaxf(t, z[r][j / 4][j % 4]);
                top[r] = t * a.scale2;
                behind |= top[r] > m[r];
            }
            if (__builtin_expect(__any(behind), 0)) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float to = fmaxf(m[r], across_groups_max(top[r]));
                    // a row that has seen nothing keeps -inf
                    const float f = to == -__builtin_inff() ? 1.0f : hw_exp2(m[r] - to);
                    l[r] *= f;
#pragma unroll
                    for (int t = 0; t < kCols; ++t) o[r][t] *= f;
                    m[r] = to;
                }
            }
            Frag pf[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float shift = m[r] == -__builtin_inff() ? 0.0f : m[r];
                float w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    w[j] = hw_exp2(__builtin_fmaf(z[r][j / 4][j % 4], a.scale2, -shift));
                    l[r] += w[j];
                }
                pf[r] = E::from(w);
            }
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
#pragma unroll
                for (int t = 0; t < kChunk; ++t) {
                    const Frag vf = tree_column<kChunk>(vw[c], t);
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        o[r][c * kChunk + t] = E::mma(vf, pf[r], o[r][c * kChunk + t]);
                }
        };

        // Blocks in turn.  A block's keys are loaded while the block before is
        // weighed and added, its values while it is scored itself: each set of
        // registers is filled again as soon as its products are done.  page_v is
        // the block's own entry, next_k and next_v the next one's.
        // The loop runs while every row sees every key (only cached positions, all
        // of them held) and a block follows, so that its loads are always in
        // flight; the second one takes the rest: the last block, the nodes, and
        // everything behind a page that is missing.
        while (p0 + kTreeTile < keys_end && p0 + kTreeKeys <= span.cached &&
               __all(is_page(page_v))) {
            score();
            load_keys(p0 + kTreeTile, next_k);
            add_values();
            p0 += kTreeTile;
            page_v = next_v;
            load_values(p0, page_v);
            next_k = entry_of(p0 + kTreeTile + 8 * (i16 >> 2));
            next_v = entry_of(p0 + kTreeTile + 8 * g);
        }
        while (p0 < keys_end) {
            const int pv = p0 + 8 * g;
            const bool held = is_page(page_v) && pv < span.keys;
            score();
            // a node's infinities and NaNs, which some rows do not see, are taken
            // out here and added to the rows that do at the end
            uint32_t odd = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t there = held && pv + j < span.keys ? ~0u : 0u;
                const uint32_t node = pv + j >= span.cached ? ~0u : 0u;
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
#pragma unroll
                    for (int k = 0; k < kChunk; ++k) {
                        const uint32_t w = vw[c][j][k] & there;
                        const uint32_t out = (w ^ tree_finite<T>(w)) & node;
                        odd |= out;
                        vw[c][j][k] = w ^ out;
                    }
            }
            if (odd) sh.odd.add(p0, kTreeKeys);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int node = sh.node[16 * r + i16];
                const uint32_t see =
                    tree_sees8(sh.mask, chain, node < span.live ? node : -1, pv - span.cached) &
                    (held ? 0xFFu >> clamp_len(pv + 8 - span.keys, 8) : 0u);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (!(see >> j & 1)) z[r][j / 4][j % 4] = -__builtin_inff();
            }
            add_values();
            p0 += kTreeTile;
            if (p0 < keys_end) {
                load_keys(p0, next_k);
                page_v = next_v;
                load_values(p0, page_v);
                next_k = entry_of(p0 + kTreeTile + 8 * (i16 >> 2));
                next_v = entry_of(p0 + kTreeTile + 8 * g);
            }
        }

        // join the four waves and leave the rows, or their part
        const int jt = fresh_tid(), ji = jt & 15, jg = jt >> 4 & 3;
        lds_barrier();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            l[r] = across_groups_sum(l[r]);
            if (jg == 0) {
                sh.ml[wave][16 * r + ji][0] = m[r];
                sh.ml[wave][16 * r + ji][1] = l[r];
            }
        }
        lds_barrier();
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (from == 0 ? 1 : 0);
        constexpr int kJoin = Shared::kJoin, kPerRow = kTreeBlock / 16;  // threads to a row
#pragma unroll
        for (int r0 = 0; r0 < R; r0 += kJoin) {
#pragma unroll
            for (int rj = 0; rj < kJoin; ++rj) {
                const int r = r0 + rj;
                float top = -__builtin_inff();
#pragma unroll
                for (int w = 0; w < kTreeWaves; ++w) top = fmaxf(top, sh.ml[w][16 * r + ji][0]);
                const float ref = top == -__builtin_inff() ? 0.0f : top;
                const float f = hw_exp2(m[r] - ref);
                // lane: query row ji, dimensions kChunk*(4 jg + e) + t of each chunk
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int t4 = 0; t4 < kChunk / 4; ++t4) {
                            v4f32 v;
#pragma unroll
                            for (int t = 0; t < 4; ++t)
                                v[t] = o[r][c * kChunk + 4 * t4 + t][e] * f;
                            *reinterpret_cast<v4f32 *>(
                                &sh.merge[rj][wave][ji][c * 16 * kChunk + kChunk * (4 * jg + e) +
                                                        4 * t4]) = v;
                        }
            }
            lds_barrier();
#pragma unroll
            for (int rj = 0; rj < kJoin; ++rj) {
                const int r = r0 + rj, qr = jt / kPerRow, in = jt % kPerRow;
                const int row = (mt * R + r) * 16 + qr;
                const int nd = sh.node[16 * r + qr];
                float rtop = -__builtin_inff(), sum = 0.0f;
#pragma unroll
                for (int w = 0; w < kTreeWaves; ++w) rtop = fmaxf(rtop, sh.ml[w][16 * r + qr][0]);
                const float rref = rtop == -__builtin_inff() ? 0.0f : rtop;
#pragma unroll
                for (int w = 0; w < kTreeWaves; ++w)
                    sum += sh.ml[w][16 * r + qr][1] * hw_exp2(sh.ml[w][16 * r + qr][0] - rref);
                const bool on = nd < span.live, some = on && !(sum == 0.0f);
                if (nd >= a.T || !(whole || on)) continue;
                const float inv = 1.0f / sum;
                const int64_t orow =
                    (static_cast<int64_t>(b) * a.T + nd) * a.H + h * a.G + row - nd * a.G;
                for (int d = in * 4; d < a.D; d += kPerRow * 4) {
                    v4f32 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int w = 0; w < kTreeWaves; ++w)
                        v += *reinterpret_cast<const v4f32 *>(&sh.merge[rj][w][qr][d]);
                    if (whole) {
                        T *out = static_cast<T *>(a.out) + orow * a.D + d;
#pragma unroll
                        for (int t = 0; t < 4; ++t)
                            out[t] = static_cast<T>(some ? v[t] * inv : 0.0f);
                    } else {
                        float *part = a.part + (slot * (16 * R) + 16 * r + qr) * a.D + d;
                        *reinterpret_cast<v4f32 *>(part) = v;
                    }
                }
                if (in == 0) {
                    if (whole) {
                        if (a.lse)
                            a.lse[orow] = some ? static_cast<float>(kLn2) * (rref + hw_log2(sum))
                                               : -__builtin_inff();
                    } else {
                        *reinterpret_cast<v4f32 *>(a.part_ml +
                                                   (slot * (16 * R) + 16 * r + qr) * 4) =
                            v4f32{rtop, sum, sum, 0.0f};
                    }
                }
            }
            if (r0 + kJoin < R) lds_barrier();
        }
        if (__builtin_expect(sh.odd.to > 0, 0))
            tree_add_odd<T>(a, sh.mask, sh.odd, span, b, h, from * kTreeTile, keys_end, whole, slot,
                            mt * 16 * R, 16 * R);
        tile += to - from;
        first += nt;
        ++b;
        if (tile < end) span = tree_span(a, b);
    }
}

// ---------------------------------------------------------------------------
// 16-bit types: each of the workgroup's four waves takes R row tiles of its own (one
// where that holds all rows, else two), and all read the same keys and values from
// shared memory, so that a key's bytes cross the vector registers' load path once for
// 64 R rows; with few rows, waves without any load as much as the others.
//
// A tile of keys is in shared memory while the next one is on its way there,
// past the registers.  Rows lie 16-byte chunk by chunk, chunk c of key k at c xor a
// function of k, so that what is read at once lies on different banks: of the
// keys, a chunk of 16 rows; of the values, two chunks of eight rows, by a
// transposing read that gives a lane four keys' elements of its dimension.  Keys and
// values are permuted differently; in the keys' order the values' reads met banks
// twice (half of shared memory's cycles, wide trees 327 us against 316).
//
// The weights' reference moves only when a score passes it by 2^6: they stay
// below 2^6 and sums of 2^30 of them far from a float's end.  float16 has normal
// numbers down to 2^-14 alone but up to 65504, so there the reference lies 2^9 (2^15
// without slack) below the largest score and weights reach 2^15: a key that takes
// nearly all of a row's weight and holds nothing leaves the others nine bits more.
// As the largest weight is then not exactly 1, the output is divided by the sum of
// the rounded weights, one more matrix product with a row of ones; lse takes the sum
// of the unrounded ones.
// ---------------------------------------------------------------------------
constexpr float kTreeSlack = 6.0f;
// What may be moved past a scheduling barrier: ordinary arithmetic, which then
// fills the time of the matrix products around it.
constexpr int kTreeArith = 0x406;

// 16 bytes a lane, at bytes behind p, to the wave's 1024 bytes of shared memory at
// lds, lane by lane; lanes that are off leave their places.  The load has no
// destination register and the compiler does not know of it, so that reading
// another stage does not wait for it; tree_loads_done() does.  Its base in shared
// memory is m0, which a load may take one wait state after a scalar write at the
// earliest; the compiler keeps no wait states within an asm block, so the s_nop does.
// m0 is reserved and cannot be listed as overwritten: nothing else in the kernel uses
// it (shared memory needs none on this architecture; tests/test_isa_hazards.py looks).
template <bool ONCE>
__device__ __forceinline__ void tree_load_lds(const void *p, uint32_t at, uint32_t lds) {
    // past the caches' usual order, the pass: 64 single tokens over up to 4000 positions
    // 94.2 us against 108.4, two caches of 131072 175.5 against 195.0
    if (ONCE)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt"
                     :
                     : "s"(lds), "v"(at), "s"(p)
                     : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                     :
                     : "s"(lds), "v"(at), "s"(p)
                     : "memory");
}
__device__ __forceinline__ void tree_loads_done() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <int DP>
constexpr int tree_wide_keys() {
    return DP <= 128 ? 64 : 32;
}

template <int DP>
__device__ __forceinline__ int tree_swizzle_k(int key) {
    return DP >= 128 ? (key & 3) | (key >> 1 & 12) : (key >> 1 & 1) | (key >> 2 & 6);
}
template <int DP>
__device__ __forceinline__ int tree_swizzle_v(int key) {
    return DP >= 128 ? (key << 1 & 6) | (key & 8) | (key >> 4 & 1)
                     : (key & 2) | (key >> 1 & 4) | (key >> 4 & 1);
}

typedef short v4i16 __attribute__((ext_vector_type(4)));

template <int N>
struct Tiles {
    static constexpr int value = N;
};

template <int DP>
struct TreeWideShared {
    v4u32 tile[2][2][tree_wide_keys<DP>() * DP / 8];  // [stage][keys, values]
    uint64_t mask[kMaxTreeNodes][2];
    int up[kMaxTreeNodes];
    TreeOdd odd;
};

// ONCE: no other workgroup reads the same keys.
template <typename T, int DP, int R, bool FULL, bool ONCE>
__global__ __launch_bounds__(kTreeBlock, (DP <= 128 ? 2 : 1)) void tree_wide_kernel(TreeArgs a) {
    using E = TreeElem<T>;
    using Frag = typename E::Frag;
    using Raw = typename E::Raw;
    constexpr int kKeys = tree_wide_keys<DP>();
    constexpr int kSteps = DP / 32, kCols = DP / 16, kRow = DP / 8;
    constexpr int kLoads = kKeys * kRow / kTreeBlock;  // chunks per thread and matrix
    constexpr int kTile = 64 * R;                      // rows of a workgroup
    // with few rows following every maximum costs next to nothing (64 single tokens
    // over up to 4000 positions 94.2 us, 93.8 with slack)
    constexpr float kSlack = R == 1 ? 0.0f : kTreeSlack;
    // how far the reference lies below the largest score at the time
    constexpr float kLift = E::kTop > 0.0f ? E::kTop - kSlack : 0.0f;
    static_assert(kTreeTile % kKeys == 0, "tiles are dealt out in whole ones");
    __shared__ TreeWideShared<DP> sh;

    const int units = a.slices * a.KV;
    const int mt = blockIdx.x / units;
    const int slice = (blockIdx.x % units) / a.KV;
    const int h = blockIdx.x % a.KV;
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int i16 = lane & 15, g = lane >> 4;
    const bool chain = a.parents == nullptr;

    TreePlace place = tree_plan(a, slice, lane, blockIdx.x == 0 && wave == 0);
    int tile = place.start, b = place.b, first = place.first;
    const int end = place.end;
    TreeSpan span = place.span;

    const int slot_mask = (1 << a.shift) - 1;
    const int64_t slot_stride = FULL ? DP : a.slot_stride;
    const T *keys = static_cast<const T *>(a.keys) + h * a.head_stride;
    const T *values = static_cast<const T *>(a.values) + h * a.head_stride;
    if (!FULL) {
        // chunks past a row's end are never loaded
        for (int e = tid; e < 4 * kKeys * kRow; e += kTreeBlock)
            (&sh.tile[0][0][0])[e] = v4u32{0, 0, 0, 0};
    }
    // this lane's chunks of a tile: the first one's key, and its place in a row
    const int key0 = tid / kRow;
    constexpr int kKeyStep = kTreeBlock / kRow, kWaveKeys = kWave / kRow;
    static_assert(kWaveKeys <= 8, "a wave's load stays in a page");
    // key0 lies below a load's step, so the swizzles of the two xor
    int chunk_k[kLoads], chunk_v[kLoads];
    uint32_t k_at[kLoads], v_at[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
        const int64_t row = lane / kRow * slot_stride;
        chunk_k[k] = (tid % kRow) ^ tree_swizzle_k<DP>(key0) ^ tree_swizzle_k<DP>(k * kKeyStep);
        chunk_v[k] = (tid % kRow) ^ tree_swizzle_v<DP>(key0) ^ tree_swizzle_v<DP>(k * kKeyStep);
        k_at[k] = static_cast<uint32_t>((row + 8 * chunk_k[k]) * sizeof(T));
        v_at[k] = static_cast<uint32_t>((row + 8 * chunk_v[k]) * sizeof(T));
    }
    // and its operands' addresses: chunk 4s + g of key i16's in the instruction's
    // order, and four dimensions of key 8g + i16/4
    constexpr uint32_t kStageBytes = kKeys * kRow * 16;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(
        reinterpret_cast<size_t>((__attribute__((address_space(3))) v4u32 *)&sh.tile[0][0][0]) +
        wave * kWave * 16));
    const int fk = tree_swizzle_k<DP>(8 * (i16 >> 2) + (i16 & 3));
    const int fv = tree_swizzle_v<DP>(8 * g + (i16 >> 2));

    while (tile < end) {
        const int nt = tree_tiles(span.keys);
        const int from = tile - first;
        const int to = nt < from + end - tile ? nt : from + end - tile;
        const bool whole = from == 0 && to == nt;
        const bool dead = mt * kTile >= span.live * a.G;  // no row in use
        const int32_t *table = a.table + static_cast<int64_t>(b) * a.P;
        const int last = ((mt + 1) * kTile - 1) / a.G;
        int keys_end = to * kTreeTile < span.keys ? to * kTreeTile : span.keys;
        if (last < span.live && keys_end > span.cached + last + 1)
            keys_end = span.cached + last + 1;
        if (dead) keys_end = 0;
        const int begin = from * kTreeTile;

        lds_barrier();
        if (tid == 0) sh.odd.clear();
        if (keys_end > span.cached && !chain) tree_masks(a, sh, b, span.live);

        // wave w's tile r is the workgroup's tile 4 r + w
        Frag qf[R][kSteps];
        int node[R];
        const int qt = fresh_tid();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = mt * kTile + (4 * r + wave) * 16 + (qt & 15);
            node[r] = row / a.G;
            if (node[r] >= span.live) node[r] = -1;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                Raw raw{};
                const int d = 32 * s + 8 * (qt >> 4 & 3);
                if (node[r] >= 0 && (FULL || d < a.D))
                    raw = tree_load8<T>(static_cast<const T *>(a.q) + b * a.q_batch +
                                        node[r] * a.q_node + (h * a.G + row % a.G) * a.q_head + d);
                qf[r][s] = E::frag(raw);
            }
        }
        float m[R], l[R];
        v4f32 n[R], o[R][kCols];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -__builtin_inff();
            l[r] = 0.0f;
            n[r] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int t = 0; t < kCols; ++t) o[r][t] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};
        }

        // lane k holds the table entry of key k of a tile
        auto entry_of = [&](int p0) {
            const int p = p0 + (lane & (kKeys - 1));
            return table[(p < span.keys ? p : span.keys - 1) >> a.shift];
        };
        auto held_of = [&](int p0, int entry) {
            return __ballot(p0 + (lane & (kKeys - 1)) < span.keys &&
                            static_cast<uint32_t>(entry) < static_cast<uint32_t>(a.pages));
        };
        // a tile's keys and values on their way to a stage.  The keys of one of a
        // wave's loads are consecutive, at most 8 and aligned, so they share a page,
        // and their addresses are a scalar and an offset that stays.
        auto load = [&](int stage, int p0, int entry) {
            const uint32_t to_k = lds0 + stage * 2 * kStageBytes, to_v = to_k + kStageBytes;
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int key = k * kKeyStep + wave * kWaveKeys;
                int page = __builtin_amdgcn_readlane(entry, key);
                if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.pages)) page = 0;
                const int64_t at =
                    page * a.page_stride + ((p0 + key) & slot_mask) * slot_stride;
                if (FULL || 8 * chunk_k[k] < a.D)
                    tree_load_lds<ONCE>(keys + at, k_at[k], to_k + k * kTreeBlock * 16);
                if (FULL || 8 * chunk_v[k] < a.D)
                    tree_load_lds<ONCE>(values + at, v_at[k], to_v + k * kTreeBlock * 16);
            }
        };
        // Values of positions that are not there become 0, and of nodes lose their
        // infinities and NaNs: each thread looks through the chunks it loaded.
        auto clean = [&](int stage, int p0, uint64_t held) {
            uint32_t odd = 0;
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int key = key0 + k * kKeyStep;
                const uint32_t there = held >> key & 1 ? ~0u : 0u;
                const uint32_t nodes = p0 + key >= span.cached ? ~0u : 0u;
                v4u32 v = sh.tile[stage][1][k * kTreeBlock + tid];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w = v[i] & there;
                    const uint32_t out = (w ^ tree_finite<T>(w)) & nodes;
                    odd |= out;
                    v[i] = w ^ out;
                }
                sh.tile[stage][1][k * kTreeBlock + tid] = v;
            }
            if (odd) sh.odd.add(p0, kKeys);
        };
        constexpr int kBlocks = kKeys / kTreeKeys;
        // a wave whose rows are not in use only loads, and one that has only its
        // first tile's works on that alone
        const bool mine = mt * kTile + 16 * wave < span.live * a.G;
        const bool all = mt * kTile + 16 * (4 * (R - 1) + wave) < span.live * a.G;
        v4f32 z[kBlocks][R][2];
        auto score = [&](auto tiles, int stage) {
            constexpr int N = decltype(tiles)::value;
            const v4u32 *kt = sh.tile[stage][0];
            // operands are read kAhead products before they are needed; the
            // barriers keep reads and products in this order
            constexpr int kAll = kBlocks * kSteps * 2, kAhead = 4;
            Raw kf[kAhead];
            auto operand = [&](int i) {
                const int c = i % 2, s = i / 2 % kSteps, kb = i / 2 / kSteps;
                const int key = 32 * kb + 8 * (i16 >> 2) + 4 * c + (i16 & 3);
                kf[i % kAhead].w = kt[key * kRow + ((4 * s + g) ^ fk)];
            };
#pragma unroll
            for (int i = 0; i < kAhead; ++i) operand(i);
#pragma unroll
            for (int i = 0; i < kAll; ++i) {
                const int c = i % 2, s = i / 2 % kSteps, kb = i / 2 / kSteps;
                __builtin_amdgcn_sched_barrier(kTreeArith);
#pragma unroll
                for (int r = 0; r < N; ++r)
                    z[kb][r][c] =
                        E::mma(E::frag(kf[i % kAhead]), qf[r][s],
                               s == 0 ? v4f32{0.0f, 0.0f, 0.0f, 0.0f} : z[kb][r][c]);
                __builtin_amdgcn_sched_barrier(kTreeArith);
                if (i + kAhead < kAll) operand(i + kAhead);
            }
        };
        auto add_values = [&](auto tiles, int stage) {
            constexpr int N = decltype(tiles)::value;
            const char *vt = reinterpret_cast<const char *>(sh.tile[stage][1]);
            float top[N];
            bool behind = false;
#pragma unroll
            for (int r = 0; r < N; ++r) {
                float t = z[0][r][0][0];
#pragma unroll
                for (int j = 1; j < 8 * kBlocks; ++j)
                    t = fmaxf(t, z[j / 8][r][j / 4 % 2][j % 4]);
                top[r] = t * a.scale2;
                behind |= top[r] > m[r] + (kSlack + kLift);
            }
            if (__builtin_expect(__any(behind), 0)) {
#pragma unroll
                for (int r = 0; r < N; ++r) {
                    const float up = fmaxf(m[r], across_groups_max(top[r]) - kLift);
                    const float f = up == -__builtin_inff() ? 1.0f : hw_exp2(m[r] - up);
                    l[r] *= f;
                    n[r] *= f;
#pragma unroll
                    for (int t = 0; t < kCols; ++t) o[r][t] *= f;
                    m[r] = up;
                }
            }
            // the values' operands, read kAhead products before they are needed
            constexpr int kAll = kBlocks * kCols, kAhead = 4;
            Frag vf[kAhead];
            auto operand = [&](int i) {
                v4i16 half[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int key = 32 * (i / kCols) + 8 * g + 4 * u + (i16 >> 2);
                    const int c = (2 * (i % kCols) + (i16 >> 1 & 1)) ^ fv;
                    half[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (__attribute__((address_space(3))) v4i16 *)(vt + (key * kRow + c) * 16 +
                                                                   (i16 & 1) * 8));
                }
                vf[i % kAhead] = __builtin_bit_cast(
                    Frag, __builtin_shufflevector(half[0], half[1], 0, 1, 2, 3, 4, 5, 6, 7));
            };
#pragma unroll
            for (int i = 0; i < kAhead; ++i) operand(i);
            float shift[N], w[kBlocks][N][8];
#pragma unroll
            for (int r = 0; r < N; ++r) shift[r] = m[r] == -__builtin_inff() ? 0.0f : m[r];
            auto weigh = [&](int kb, int j) {
#pragma unroll
                for (int r = 0; r < N; ++r) {
                    w[kb][r][j] =
                        hw_exp2(__builtin_fmaf(z[kb][r][j / 4][j % 4], a.scale2, -shift[r]));
                    l[r] += w[kb][r][j];
                }
            };
#pragma unroll
            for (int j = 0; j < 8; ++j) weigh(0, j);
            Frag pf[N];
#pragma unroll
            for (int i = 0; i < kAll; ++i) {
                const int kb = i / kCols, t = i % kCols;
                if (t == 0) {
#pragma unroll
                    for (int r = 0; r < N; ++r) {
                        pf[r] = E::from(w[kb][r]);
                        n[r] = E::mma(E::ones(), pf[r], n[r]);
                    }
                }
#pragma unroll
                for (int r = 0; r < N; ++r) o[r][t] = E::mma(vf[i % kAhead], pf[r], o[r][t]);
                __builtin_amdgcn_sched_barrier(kTreeArith);
                if (i + kAhead < kAll) operand(i + kAhead);
                // the next block's weights between this one's products
                if (kb + 1 < kBlocks) {
#pragma unroll
                    for (int j = t * 8 / kCols; j < (t + 1) * 8 / kCols; ++j) weigh(kb + 1, j);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };

        // entry and held: the tile's own; entry_next: the following one's
        int entry = 0, entry_next = 0, p0 = begin, stage = 0;
        uint64_t held = 0;
        lds_barrier();  // the stages are free
        if (p0 < keys_end) {
            entry = entry_of(p0);
            entry_next = entry_of(p0 + kKeys);
            held = held_of(p0, entry);
            load(0, p0, entry);
            tree_loads_done();
        }
        lds_barrier();
        // while every row sees every key and a tile follows, which is on its way
        // meanwhile; then the rest: the last tile, the nodes, and everything behind
        // a page that is missing
        auto plain = [&](auto tiles) {
            while (p0 + kKeys < keys_end && p0 + kKeys <= span.cached && ~held == 0) {
                load(stage ^ 1, p0 + kKeys, entry_next);
                held = held_of(p0 + kKeys, entry_next);
                entry_next = entry_of(p0 + 2 * kKeys);
                if (mine) {
                    score(tiles, stage);
                    // the compute unit's other workgroup scores meanwhile: wide trees
                    // 350 -> 327 us, two caches of 131072 184.7 -> 176.7
                    __builtin_amdgcn_s_setprio(1);
                    add_values(tiles, stage);
                    __builtin_amdgcn_s_setprio(0);
                }
                p0 += kKeys;
                stage ^= 1;
                tree_loads_done();
                lds_barrier();
            }
        };
        // a wave with one row tile in use runs a loop of its own (wide trees 321 ->
        // 314 us); a branch within one loop spills registers (351 to 403)
        if (all)
            plain(Tiles<R>{});
        else
            plain(Tiles<1>{});
        while (p0 < keys_end) {
            clean(stage, p0, held);
            lds_barrier();
            if (mine) score(Tiles<R>{}, stage);
#pragma unroll
            for (int kb = 0; kb < kBlocks; ++kb) {
                const uint32_t there = static_cast<uint32_t>(held >> (32 * kb + 8 * g)) & 0xFFu;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const uint32_t see =
                        tree_sees8(sh.mask, chain, node[r], p0 + 32 * kb + 8 * g - span.cached) &
                        there;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (!(see >> j & 1)) z[kb][r][j / 4][j % 4] = -__builtin_inff();
                }
            }
            if (mine) add_values(Tiles<R>{}, stage);
            p0 += kKeys;
            if (p0 < keys_end) {
                stage ^= 1;  // free since the last barrier
                load(stage, p0, entry_next);
                held = held_of(p0, entry_next);
                entry_next = entry_of(p0 + kKeys);
                tree_loads_done();
            }
            lds_barrier();
        }

        // leave the rows, or their part
        const int jt = fresh_tid(), ji = jt & 15, jg = jt >> 4 & 3;
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (from == 0 ? 1 : 0);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int in = (4 * r + wave) * 16 + ji, row = mt * kTile + in;
            const int nd = row / a.G;
            const float sum = across_groups_sum(l[r]);
            const bool on = node[r] >= 0, some = on && !(sum == 0.0f);
            if (nd >= a.T || !(whole || on)) continue;
            const int64_t orow = (static_cast<int64_t>(b) * a.T + nd) * a.H + h * a.G + row % a.G;
            const float inv = 1.0f / n[r][0];
#pragma unroll
            for (int t = 0; t < kCols; ++t) {
                const int d = 16 * t + 4 * jg;
                if (!FULL && d >= a.D) continue;
                const v4f32 v = o[r][t];
                if (whole) {
                    T x[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = static_cast<T>(some ? v[k] * inv : 0.0f);
                    *reinterpret_cast<v2u32 *>(static_cast<T *>(a.out) + orow * a.D + d) =
                        __builtin_bit_cast(v2u32, x);
                } else {
                    *reinterpret_cast<v4f32 *>(a.part + (slot * kTile + in) * a.D + d) = v;
                }
            }
            if (jg == 0) {
                if (!whole)
                    *reinterpret_cast<v4f32 *>(a.part_ml + (slot * kTile + in) * 4) =
                        v4f32{m[r], sum, n[r][0], 0.0f};
                else if (a.lse)
                    a.lse[orow] = some ? static_cast<float>(kLn2) * (m[r] + hw_log2(sum))
                                       : -__builtin_inff();
            }
        }
        if (__builtin_expect(sh.odd.to > 0, 0))
            tree_add_odd<T>(a, sh.mask, sh.odd, span, b, h, begin, keys_end, whole, slot,
                            mt * kTile, kTile);
        tile += to - from;
        first += nt;
        ++b;
        if (tile < end) span = tree_span(a, b);
    }
}

// A part times its factor.  A factor that is 0 only in 32 bits leaves infinities and
// NaNs what they are, as a node's weight within a part does.
__device__ __forceinline__ v4f32 tree_scaled(v4f32 p, float f) {
    v4f32 v = p * f;
    if (f == 0.0f) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            v[t] = __builtin_fabsf(p[t]) < __builtin_inff() ? 0.0f : p[t];
    }
    return v;
}

// Joins the parts of the rows of sequences that were cut.  A wave takes NR rows of
// a sequence; its lanes take the parts' references and sums, then 64 / L parts at
// a time, L lanes to a part's dimensions.  Everything that depends on nothing read
// before is asked for at once: the launch is bound by how often it waits.
template <typename T, int L, int NR>
__global__ __launch_bounds__(kTreeBlock) void tree_join_kernel(TreeArgs a, int rows16,
                                                               int blocks) {
    constexpr int kAt = kWave / L, kAhead = NR == 1 ? 8 : 2;  // parts at a time, and ahead
    const int b = blockIdx.x / blocks;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int per = a.first[a.B], first = a.first[b];
    const TreeSpan span = tree_span(a, b);
    const int w0 = first / per, w1 = (first + tree_tiles(span.keys) - 1) / per;
    const int n = w1 - w0 + 1;
    if (n == 1) return;
    const int of = a.T * a.H;  // rows of the sequence
    const int row0 = ((blockIdx.x % blocks) * kTreeWaves + wave) * NR;
    if (row0 >= of) return;
    const int d = lane % L * 4;
    const int64_t step = static_cast<int64_t>(a.KV) * 2 * rows16;  // to the next slice's part
    int64_t at0[NR];
    bool on[NR];
    v4f32 ml[NR], p[NR][kAhead];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int nd = (row0 + r) / a.H, head = (row0 + r) % a.H;
        on[r] = nd < span.live;
        const int h = head / a.G, row = nd * a.G + head - h * a.G;
        // a slice's part 1 where the sequence begins in it, else 0
        at0[r] = ((static_cast<int64_t>(row / rows16) * a.slices + w0) * a.KV + h) * 2 * rows16 +
                 row % rows16;
        ml[r] = v4f32{-__builtin_inff(), 0.0f, 0.0f, 0.0f};
        if (on[r] && lane < n)
            ml[r] = *reinterpret_cast<const v4f32 *>(
                a.part_ml + (at0[r] + lane * step + (lane ? 0 : rows16)) * 4);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int k = u * kAt + lane / L;
            p[r][u] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};
            if (on[r] && k < n && d < a.D)
                p[r][u] = *reinterpret_cast<const v4f32 *>(
                    a.part + (at0[r] + k * step + (k ? 0 : rows16)) * a.D + d);
        }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        if (row0 + r >= of) break;
        const int64_t row_at = static_cast<int64_t>(b) * of + row0 + r;
        T *out = static_cast<T *>(a.out) + row_at * a.D;
        auto ml_of = [&](int k) {
            return k < n ? *reinterpret_cast<const v4f32 *>(
                               a.part_ml + (at0[r] + k * step + (k ? 0 : rows16)) * 4)
                         : v4f32{-__builtin_inff(), 0.0f, 0.0f, 0.0f};
        };
        float top = ml[r][0];
        if (on[r])
            for (int k = kWave; k < n; k += kWave) top = fmaxf(top, ml_of(k + lane)[0]);
        // the first n lanes hold something
        for (int o = 1; o < n && o < kWave; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, kWave));
        top = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(top)));
        const float ref = top == -__builtin_inff() ? 0.0f : top;
        float f = hw_exp2(ml[r][0] - ref);
        float sum = f * ml[r][1], norm = f * ml[r][2];
        v4f32 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            v += p[r][u] * __shfl(f, (u * kAt + lane / L) & (kWave - 1), kWave);
        if (on[r])
            for (int k0 = kAhead * kAt; k0 < n; k0 += kAt) {
                if (k0 % kWave == 0) {
                    const v4f32 more = ml_of(k0 + lane);
                    f = hw_exp2(more[0] - ref);
                    sum += f * more[1];
                    norm += f * more[2];
                }
                const int k = k0 + lane / L;
                const float fk = __shfl(f, k & (kWave - 1), kWave);
                if (k < n && d < a.D)
                    v += *reinterpret_cast<const v4f32 *>(a.part + (at0[r] + k * step) * a.D + d) *
                         fk;
            }
        // a NaN may be an infinite part times a factor that is 0: once more, with care
        const float all = v[0] + v[1] + v[2] + v[3];
        if (__builtin_expect(__any(all != all), 0)) {
            v = v4f32{0.0f, 0.0f, 0.0f, 0.0f};
            for (int k0 = 0; k0 < n; k0 += kAt) {
                if (k0 % kWave == 0) f = hw_exp2(ml_of(k0 + lane)[0] - ref);
                const int k = k0 + lane / L;
                const float fk = __shfl(f, k & (kWave - 1), kWave);
                if (k < n && d < a.D)
                    v += tree_scaled(*reinterpret_cast<const v4f32 *>(
                                         a.part + (at0[r] + k * step + (k ? 0 : rows16)) * a.D + d),
                                     fk);
            }
        }
        for (int o = 1; o < n && o < kWave; o <<= 1) {
            sum += __shfl_xor(sum, o, kWave);
            norm += __shfl_xor(norm, o, kWave);
        }
        sum = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(sum)));
        norm = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(norm)));
#pragma unroll
        for (int o = L; o < kWave; o <<= 1)
#pragma unroll
            for (int t = 0; t < 4; ++t) v[t] += __shfl_xor(v[t], o, kWave);
        const bool some = on[r] && !(sum == 0.0f);
        if (lane < L && d < a.D) {
#pragma unroll
            for (int t = 0; t < 4; ++t) out[d + t] = static_cast<T>(some ? v[t] / norm : 0.0f);
        }
        if (lane == 0 && a.lse)
            a.lse[row_at] = some ? static_cast<float>(kLn2) * (ref + hw_log2(sum))
                                 : -__builtin_inff();
    }
}

}  // namespace sv
