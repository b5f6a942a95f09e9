// sv_tree.hpp -- attention of a chain or a tree of new tokens over a paged
// cache.
//
// For each sequence and key head the G query heads that share it and the T new
// tokens (nodes) make M = T*G query rows over the same n keys:
//   out = sum_p e^(s_p - lse) v_p,   s_p = scale q.k_p,   lse = ln sum_p e^s_p
// over the cached positions p < L, which every row sees, and the row's own node
// and its ancestors among the n - L nodes behind them.
//
// One pass over the keys with a running maximum and sum per row.  A wave takes
// 32 keys at a time straight from memory into the matrix instructions'
// registers, without shared memory:
//   S^T = K Q^T   a lane's operand is 8 consecutive elements of a key's row, a
//                 16-byte load.  The instruction's 16 rows are given keys in
//                 the order that leaves lane group g (of four) with the scores
//                 of keys 8g..8g+7, all of one query row.
//   O^T = V^T P^T those 8 weights are the lane's operand as they stand; the
//                 other one is 8 keys' values of one dimension, which the lane
//                 picks from its own 8 loads (a load: 8 consecutive dimensions
//                 of one key), for 16-bit types two at a time by a byte
//                 permutation.
// A query row is a column throughout, so its maximum, sum and rescaling stay in
// its lanes.  Products are added in 32 bits.  The weights are rounded to the
// values' type before the second product, as the matrix instructions of 16-bit
// types take them (a relative 2^-9 or 2^-12 of each, with independent signs);
// their sum is taken before that rounding, in 32 bits, so that lse is good to
// 32 bits.
//
// The keys of all sequences are cut into tiles and the tiles dealt out evenly:
// a workgroup takes a run of tiles, which may end inside a sequence and hold
// several short ones, so ragged batches load every workgroup alike.  A
// sequence whose tiles are in several workgroups is joined by a second launch.
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
    float *part_ml;          // [workgroup][2][rows][2]: their maximum and sum
    int32_t *first;          // [B + 1]: sequences' first tiles, then the tiles per slice
    int64_t page_stride, head_stride, slot_stride;  // elements
    int64_t q_batch, q_node, q_head;                // elements
    int32_t B, T, H, KV, G, D, P;
    int32_t pages, shift;    // page size 2^shift
    int32_t slices, mtiles;
    float scale2;            // scale * log2(e)
};

// Types of keys and values.  Frag: a matrix operand's 8 elements along the
// summed dimension; load8: 8 consecutive elements.
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
};

template <>
struct TreeElem<__bf16> : TreeElem16<v8bf16> {
    __device__ static __forceinline__ v4f32 mma(Frag a, Frag b, v4f32 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static constexpr uint32_t kExponent = 0x7F80u;
};

template <>
struct TreeElem<_Float16> : TreeElem16<v8f16> {
    __device__ static __forceinline__ v4f32 mma(Frag a, Frag b, v4f32 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static constexpr uint32_t kExponent = 0x7C00u;
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

// Words of 32 bits that C elements take.
template <typename T, int C>
constexpr int tree_words() {
    return C * static_cast<int>(sizeof(T)) / 4;
}

template <typename T, int C>
__device__ __forceinline__ void tree_load_row(const T *p, uint32_t *w) {
    constexpr int n = tree_words<T, C>();
    if constexpr (n == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < n / 4; ++i) {
            const v4u32 v = reinterpret_cast<const v4u32 *>(p)[i];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[4 * i + k] = v[k];
        }
    }
}

// Element t of 8 keys' rows as an operand.
template <typename T, int C>
__device__ __forceinline__ typename TreeElem<T>::Frag tree_column(
    const uint32_t (&w)[8][tree_words<T, C>()], int t) {
    if constexpr (sizeof(T) == 4) {
        v8f32 v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j][t]);
        return v;
    } else {
        v4u32 v;
        const uint32_t pick = t % 2 ? 0x07060302u : 0x05040100u;
#pragma unroll
        for (int m = 0; m < 4; ++m)
            v[m] = __builtin_amdgcn_perm(w[2 * m + 1][t / 2], w[2 * m][t / 2], pick);
        return __builtin_bit_cast(typename TreeElem<T>::Frag, v);
    }
}

// Whether a word holds an infinity or a NaN.
template <typename T>
__device__ __forceinline__ bool tree_nonfinite(uint32_t w) {
    if constexpr (sizeof(T) == 4) {
        return (w & 0x7F800000u) == 0x7F800000u;
    } else {
        constexpr uint32_t e = TreeElem<T>::kExponent;
        return (w & e) == e || ((w >> 16) & e) == e;
    }
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

template <typename T, int DP, int R>
struct TreeShared {
    static constexpr int kPitch = DP + 4;  // 16 rows' starts on different banks
    float merge[kTreeWaves][16][kPitch];
    float ml[kTreeWaves][16 * R][2];
    uint64_t mask[kMaxTreeNodes][2];
    int up[kMaxTreeNodes];
    int scan[kTreeWaves];
    int plan[4];
};

// Finds this slice's tiles: [start, end), the sequence that holds start and
// that sequence's first tile.  Workgroup 0 leaves the sequences' first tiles
// for the second launch.
template <typename Shared>
__device__ __forceinline__ void tree_plan(const TreeArgs &a, Shared &sh, int slice, bool leave,
                                          int &start, int &end, int &b, int &first) {
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    int total = 0;
    for (int pass = 0; pass < 2; ++pass) {
        // pass 0 adds the tiles up, pass 1 finds the place
        int per = 0;
        if (pass == 1) {
            per = (total + a.slices - 1) / a.slices;
            start = slice * per;
            end = start + per < total ? start + per : total;
            if (tid == 0) sh.plan[0] = a.B;
            if (leave && tid == 0) a.first[a.B] = per;
        }
        int base = 0;
        for (int b0 = 0; b0 < a.B; b0 += kTreeBlock) {
            const int i = b0 + tid;
            const int mine = i < a.B ? tree_tiles(tree_span(a, i).keys) : 0;
            int upto = mine;
#pragma unroll
            for (int o = 1; o < kWave; o <<= 1) {
                const int v = __shfl_up(upto, o, kWave);
                if (lane >= o) upto += v;
            }
            __syncthreads();
            if (lane == kWave - 1) sh.scan[wave] = upto;
            __syncthreads();
            int before = base;
            for (int w = 0; w < wave; ++w) before += sh.scan[w];
            before += upto - mine;
            if (pass == 1 && i < a.B) {
                if (leave) a.first[i] = before;
                if (start >= before && start < before + mine) {
                    sh.plan[0] = i;
                    sh.plan[1] = before;
                }
            }
            for (int w = 0; w < kTreeWaves; ++w) base += sh.scan[w];
        }
        total = base;
    }
    __syncthreads();
    b = sh.plan[0];
    first = sh.plan[1];
}

// Ancestor masks of a tree's nodes, the node itself included, by doubling the
// distance of the jump: 7 rounds for 128 nodes.  A parent that does not precede
// its node makes it a root.
template <typename Shared>
__device__ __forceinline__ void tree_masks(const TreeArgs &a, Shared &sh, int b, int live) {
    const int i = threadIdx.x;
    if (i < kMaxTreeNodes) {
        int up = i < live ? a.parents[static_cast<int64_t>(b) * a.T + i] : -1;
        if (up < 0 || up >= i) up = -1;
        sh.up[i] = up;
        sh.mask[i][0] = i < 64 ? 1ull << i : 0;
        sh.mask[i][1] = i < 64 ? 0 : 1ull << (i - 64);
    }
    __syncthreads();
    for (int round = 1; round < live; round <<= 1) {
        uint64_t m0 = 0, m1 = 0;
        int up = -1;
        if (i < live && sh.up[i] >= 0) {
            up = sh.up[sh.up[i]];
            m0 = sh.mask[sh.up[i]][0];
            m1 = sh.mask[sh.up[i]][1];
        }
        __syncthreads();
        if (i < live) {
            sh.up[i] = up;
            sh.mask[i][0] |= m0;
            sh.mask[i][1] |= m1;
        }
        __syncthreads();
    }
}

template <typename T, int DP, int R>
__global__ __launch_bounds__(kTreeBlock) void tree_attention_kernel(TreeArgs a) {
    using E = TreeElem<T>;
    using Frag = typename E::Frag;
    constexpr int kSteps = DP / 32;             // matrix instructions along a key's row
    constexpr int kCols = DP / 16;              // along the output's dimensions
    constexpr int kChunk = kCols < 8 ? kCols : 8;   // elements of a value load
    constexpr int kChunks = kCols / kChunk;
    constexpr int kWords = tree_words<T, kChunk>();
    using Shared = TreeShared<T, DP, R>;
    __shared__ Shared sh;

    const int units = a.slices * a.KV;
    const int mt = blockIdx.x / units;
    const int slice = (blockIdx.x % units) / a.KV;
    const int h = blockIdx.x % a.KV;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int i16 = lane & 15, g = lane >> 4;
    const bool chain = a.parents == nullptr;

    int tile, end, b, first;
    tree_plan(a, sh, slice, blockIdx.x == 0, tile, end, b, first);

    const T *keys = static_cast<const T *>(a.keys) + h * a.head_stride;
    const T *values = static_cast<const T *>(a.values) + h * a.head_stride;
    const int slot_mask = (1 << a.shift) - 1;

    while (tile < end) {
        const TreeSpan span = tree_span(a, b);
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
        const bool nodes_here = !dead && keys_end > span.cached;
        if (nodes_here && !chain) tree_masks(a, sh, b, span.live);

        Frag qf[R][kSteps];
        int node[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = (mt * R + r) * 16 + i16;
            node[r] = row / a.G;
            const bool on = node[r] < span.live;
            const T *q = static_cast<const T *>(a.q) + b * a.q_batch + node[r] * a.q_node +
                         (h * a.G + row % a.G) * a.q_head;
            if (!on) node[r] = -1;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                typename E::Raw raw{};
                const int d = 32 * s + 8 * g;
                if (on && d < a.D) raw = tree_load8<T>(q + d);
                qf[r][s] = E::frag(raw);
            }
        }

        float m[R], l[R];
        v4f32 o[R][kCols];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -__builtin_inff();
            l[r] = 0.0f;
#pragma unroll
            for (int t = 0; t < kCols; ++t) o[r][t] = v4f32{0.0f, 0.0f, 0.0f, 0.0f};
        }

        for (int p0 = from * kTreeTile + wave * kTreeKeys; p0 < keys_end; p0 += kTreeTile) {
            // the pages of the keys that this lane loads: keys 8(i16/4).. of
            // the first product, keys 8g.. of the second
            const int pk = p0 + 8 * (i16 >> 2), pv = p0 + 8 * g;
            int page_k = pk < span.keys ? table[pk >> a.shift] : -1;
            int page_v = pv < span.keys ? table[pv >> a.shift] : -1;
            const bool held = static_cast<uint32_t>(page_v) < static_cast<uint32_t>(a.pages);
            if (static_cast<uint32_t>(page_k) >= static_cast<uint32_t>(a.pages)) page_k = 0;
            if (!held) page_v = 0;
            const T *kp = keys + page_k * a.page_stride +
                          ((pk & slot_mask) + (i16 & 3)) * a.slot_stride;
            const T *vp = values + page_v * a.page_stride + (pv & slot_mask) * a.slot_stride;

            Frag kf[2][kSteps];
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    typename E::Raw raw{};
                    const int d = 32 * s + 8 * g;
                    if (d < a.D) raw = tree_load8<T>(kp + 4 * c * a.slot_stride + d);
                    kf[c][s] = E::frag(raw);
                }
            uint32_t vw[kChunks][8][kWords];
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int d = c * 16 * kChunk + i16 * kChunk;
#pragma unroll
                    for (int k = 0; k < kWords; ++k) vw[c][j][k] = 0;
                    if (d < a.D) tree_load_row<T, kChunk>(vp + j * a.slot_stride + d, vw[c][j]);
                }

            // every row sees every key: only cached positions, all of them held
            const bool plain = __all(held && p0 + kTreeKeys <= span.cached);
            bool apart = false;  // a node's infinity or NaN, which some rows may not see
            if (!plain) {
                bool odd = false;
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const bool there = held && pv + j < span.keys;
#pragma unroll
                        for (int k = 0; k < kWords; ++k) {
                            if (!there) vw[c][j][k] = 0;
                            odd |= pv + j >= span.cached && tree_nonfinite<T>(vw[c][j][k]);
                        }
                    }
                apart = __any(odd);
            }

#pragma unroll
            for (int r = 0; r < R; ++r) {
                v4f32 s0 = {0.0f, 0.0f, 0.0f, 0.0f}, s1 = s0;
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    s0 = E::mma(kf[0][s], qf[r][s], s0);
                    s1 = E::mma(kf[1][s], qf[r][s], s1);
                }
                float z[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]};
                if (!plain) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int at = pv + j - span.cached;
                        bool see = held && pv + j < span.keys && node[r] >= 0;
                        if (see && at >= 0) see = tree_sees(sh.mask, chain, node[r], at);
                        if (!see) z[j] = -__builtin_inff();
                    }
                }
                float top = z[0];
#pragma unroll
                for (int j = 1; j < 8; ++j) top = fmaxf(top, z[j]);
                top = fmaxf(m[r], across_groups_max(top));
                const float ref = top == -__builtin_inff() ? 0.0f : top;
                const float shift2 = ref * a.scale2;
                if (__any(top > m[r])) {
                    const float f = hw_exp2(m[r] * a.scale2 - shift2);
                    l[r] *= f;
#pragma unroll
                    for (int t = 0; t < kCols; ++t) o[r][t] *= f;
                    m[r] = top;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    z[j] = hw_exp2(__builtin_fmaf(z[j], a.scale2, -shift2));
                    l[r] += z[j];
                }
                const Frag pf = E::from(z);
                if (!apart) {
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
#pragma unroll
                        for (int t = 0; t < kChunk; ++t)
                            o[r][c * kChunk + t] = E::mma(tree_column<T, kChunk>(vw[c], t), pf,
                                                          o[r][c * kChunk + t]);
                } else {
                    // key by key, added only where the row sees it
                    for (int key = 0; key < kTreeKeys; ++key) {
                        const int at = p0 + key - span.cached;
                        const bool see = p0 + key < span.keys && node[r] >= 0 &&
                                         (at < 0 || tree_sees(sh.mask, chain, node[r], at));
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) {
                            uint32_t one[8][kWords];
#pragma unroll
                            for (int j = 0; j < 8; ++j)
#pragma unroll
                                for (int k = 0; k < kWords; ++k)
                                    one[j][k] = 8 * g + j == key ? vw[c][j][k] : 0u;
#pragma unroll
                            for (int t = 0; t < kChunk; ++t) {
                                const v4f32 add = E::mma(tree_column<T, kChunk>(one, t), pf,
                                                         v4f32{0.0f, 0.0f, 0.0f, 0.0f});
                                if (see) o[r][c * kChunk + t] += add;
                            }
                        }
                    }
                }
            }
        }

        // join the four waves and leave the rows, or their part
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            l[r] = across_groups_sum(l[r]);
            if (g == 0) {
                sh.ml[wave][16 * r + i16][0] = m[r];
                sh.ml[wave][16 * r + i16][1] = l[r];
            }
        }
        __syncthreads();
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (from == 0 ? 1 : 0);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float top = -__builtin_inff();
#pragma unroll
            for (int w = 0; w < kTreeWaves; ++w) top = fmaxf(top, sh.ml[w][16 * r + i16][0]);
            const float ref = top == -__builtin_inff() ? 0.0f : top;
            const float f = hw_exp2(m[r] * a.scale2 - ref * a.scale2);
            // lane: query row i16, dimensions kChunk*(4g + e) + t of each chunk
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int t4 = 0; t4 < kChunk / 4; ++t4) {
                        v4f32 v;
#pragma unroll
                        for (int t = 0; t < 4; ++t) v[t] = o[r][c * kChunk + 4 * t4 + t][e] * f;
                        *reinterpret_cast<v4f32 *>(
                            &sh.merge[wave][i16][c * 16 * kChunk + kChunk * (4 * g + e) +
                                                 4 * t4]) = v;
                    }
            __syncthreads();
            const int qr = tid >> 4;  // 16 threads to a row
            const int row = (mt * R + r) * 16 + qr;
            const int nd = row / a.G;
            float rtop = -__builtin_inff(), sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kTreeWaves; ++w) rtop = fmaxf(rtop, sh.ml[w][16 * r + qr][0]);
            const float rref = rtop == -__builtin_inff() ? 0.0f : rtop;
#pragma unroll
            for (int w = 0; w < kTreeWaves; ++w)
                sum += sh.ml[w][16 * r + qr][1] *
                       hw_exp2(sh.ml[w][16 * r + qr][0] * a.scale2 - rref * a.scale2);
            const bool on = nd < span.live;
            if (nd < a.T && (whole || on)) {
                const float inv = whole ? (on && !(sum == 0.0f) ? 1.0f / sum : 0.0f) : 1.0f;
                const int64_t orow = (static_cast<int64_t>(b) * a.T + nd) * a.H + h * a.G +
                                     row % a.G;
                for (int d = (tid & 15) * 4; d < a.D; d += 64) {
                    v4f32 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int w = 0; w < kTreeWaves; ++w)
                        v += *reinterpret_cast<const v4f32 *>(&sh.merge[w][qr][d]);
                    if (whole) {
                        T *out = static_cast<T *>(a.out) + orow * a.D + d;
#pragma unroll
                        for (int t = 0; t < 4; ++t)
                            out[t] = static_cast<T>(on && !(sum == 0.0f) ? v[t] * inv : 0.0f);
                    } else {
                        float *part = a.part + (slot * (16 * R) + 16 * r + qr) * a.D + d;
                        *reinterpret_cast<v4f32 *>(part) = v;
                    }
                }
                if ((tid & 15) == 0) {
                    if (whole) {
                        if (a.lse)
                            a.lse[orow] = on && !(sum == 0.0f)
                                              ? static_cast<float>(kLn2) *
                                                    (rref * a.scale2 + hw_log2(sum))
                                              : -__builtin_inff();
                    } else {
                        float *ml = a.part_ml + (slot * (16 * R) + 16 * r + qr) * 2;
                        ml[0] = rtop;
                        ml[1] = sum;
                    }
                }
            }
            __syncthreads();
        }
        tile += to - from;
        first += nt;
        ++b;
    }
}

// Joins the parts of a row whose sequence was cut: a wave per row.
template <typename T>
__global__ __launch_bounds__(kTreeBlock) void tree_join_kernel(TreeArgs a, int rows16) {
    const int64_t row_at = static_cast<int64_t>(blockIdx.x) * kTreeWaves + threadIdx.x / kWave;
    const int lane = threadIdx.x & (kWave - 1);
    if (row_at >= static_cast<int64_t>(a.B) * a.T * a.H) return;
    const int head = static_cast<int>(row_at % a.H);
    const int nd = static_cast<int>(row_at / a.H % a.T);
    const int b = static_cast<int>(row_at / a.H / a.T);
    const TreeSpan span = tree_span(a, b);
    const int per = a.first[a.B], first = a.first[b];
    const int w0 = first / per, w1 = (first + tree_tiles(span.keys) - 1) / per;
    if (w0 == w1) return;
    T *out = static_cast<T *>(a.out) + row_at * a.D;
    const int h = head / a.G;
    const int row = nd * a.G + head % a.G;
    const int mt = row / rows16, in = row % rows16;
    float top = -__builtin_inff(), sum = 0.0f;
    const bool on = nd < span.live;
    auto at = [&](int w) {
        const int64_t wg = (static_cast<int64_t>(mt) * a.slices + w) * a.KV + h;
        return (2 * wg + (w == w0 ? 1 : 0)) * rows16 + in;
    };
    if (on)
        for (int w = w0; w <= w1; ++w) top = fmaxf(top, a.part_ml[at(w) * 2]);
    const float ref = top == -__builtin_inff() ? 0.0f : top;
    v4f32 v = {0.0f, 0.0f, 0.0f, 0.0f};
    const int d = lane * 4;
    if (on)
        for (int w = w0; w <= w1; ++w) {
            const float f = hw_exp2(a.part_ml[at(w) * 2] * a.scale2 - ref * a.scale2);
            sum += f * a.part_ml[at(w) * 2 + 1];
            if (d < a.D) v += *reinterpret_cast<const v4f32 *>(a.part + at(w) * a.D + d) * f;
        }
    const bool some = on && !(sum == 0.0f);
    if (d < a.D) {
#pragma unroll
        for (int t = 0; t < 4; ++t) out[d + t] = static_cast<T>(some ? v[t] / sum : 0.0f);
    }
    if (lane == 0 && a.lse)
        a.lse[row_at] = some ? static_cast<float>(kLn2) * (ref * a.scale2 + hw_log2(sum))
                             : -__builtin_inff();
}

}  // namespace sv
