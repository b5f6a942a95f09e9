// sv_cache.hpp -- the upkeep of a paged cache: appending new tokens' keys and
// values, accepting a path of a drafted tree and moving its positions together,
// and sharing, reserving, releasing and copying pages.
//
// All of it moves bytes or counts; none of it computes numbers, and every
// result is a pure function of the inputs: integer atomics only add, subtract
// or take minima, and what they decide is read after a barrier.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "sv_common.hpp"
#include "sv_launch.hpp"

namespace sv {

constexpr int kMaxKeepNodes = 1024;  // entries of a path
constexpr int kMaxAcceptNodes = 128;

// ---------------------------------------------------------------------------
// Appending: a thread per 16 bytes of a node's head, keys and values together, so
// that both matrices' loads are in flight at once and the page is looked up once.
// Five nodes of a sequence 2.1 us (a launch), eight pieces of a prompt of 301 to
// 512 nodes 5.7 us, 27 MB read and written (4.6 TB/s): memory.
// ---------------------------------------------------------------------------
struct AppendArgs {
    const char *k, *v;
    char *keys, *values;
    const int32_t *table, *lengths, *nodes;
    int64_t batch_stride, node_stride, k_head_stride;       // bytes, of k and v
    int64_t page_stride, head_stride, slot_stride;          // bytes, of the pools
    int32_t T, P, heads, units, pages, shift;
    int32_t blocks;  // workgroups per sequence
};

__global__ __launch_bounds__(kCacheBlock) void cache_append_kernel(AppendArgs a) {
    const int b = blockIdx.x / a.blocks;
    const int live = a.nodes ? clamp_len(a.nodes[b], a.T) : a.T;
    const int64_t i = static_cast<int64_t>(blockIdx.x % a.blocks) * kCacheBlock + threadIdx.x;
    const int unit = static_cast<int>(i % a.units);
    const int h = static_cast<int>(i / a.units % a.heads);
    const int64_t j = i / a.units / a.heads;
    if (j >= live) return;
    const int room = a.P << a.shift;
    const int64_t at = clamp_len(a.lengths[b], room) + j;
    if (at >= room) return;
    const int page = a.table[static_cast<int64_t>(b) * a.P + (at >> a.shift)];
    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.pages)) return;
    const int64_t from = b * a.batch_stride + j * a.node_stride + h * a.k_head_stride + unit * 16;
    const int64_t to = page * a.page_stride + h * a.head_stride +
                       (at & ((1 << a.shift) - 1)) * a.slot_stride + unit * 16;
    const v4u32 x = *reinterpret_cast<const v4u32 *>(a.k + from);
    const v4u32 y = *reinterpret_cast<const v4u32 *>(a.v + from);
    *reinterpret_cast<v4u32 *>(a.keys + to) = x;
    *reinterpret_cast<v4u32 *>(a.values + to) = y;
}

// ---------------------------------------------------------------------------
// Accepting a path: a wave per sequence, two nodes to a lane.  A step compares
// every node's parent and token at once and takes the lowest that fits, so a
// sequence costs its accepted length, not its nodes.  Eight nodes 1.5 us, 256 trees
// of 64 nodes 3.2 us: a step's latency (a ballot and two lane reads).
// ---------------------------------------------------------------------------
struct AcceptArgs {
    const int32_t *parents, *tokens, *chosen, *nodes;
    int32_t *path, *count, *emitted;
    int32_t B, T;
};

__global__ __launch_bounds__(kCacheBlock) void tree_accept_kernel(AcceptArgs a) {
    const int b = blockIdx.x * (kCacheBlock / kWave) + threadIdx.x / kWave;
    const int lane = threadIdx.x & (kWave - 1);
    if (b >= a.B) return;
    const int live = a.nodes ? clamp_len(a.nodes[b], a.T) : a.T;
    const int64_t row = static_cast<int64_t>(b) * a.T;
    int parent[2], token[2], choice[2], path[2] = {-1, -1}, said[2] = {-1, -1};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int j = lane + 64 * k;
        const bool on = j < live;
        parent[k] = on ? a.parents[row + j] : -1;
        token[k] = on ? a.tokens[row + j] : 0;
        choice[k] = on ? a.chosen[row + j] : 0;
        if (parent[k] >= j) parent[k] = -1;  // does not precede its node
    }
    int count = 0;
    for (int node = live > 0 ? 0 : -1; node >= 0;) {
        const int want = __builtin_amdgcn_readlane(node < 64 ? choice[0] : choice[1], node & 63);
        const uint64_t lo = __ballot(parent[0] == node && token[0] == want);
        const uint64_t hi = __ballot(parent[1] == node && token[1] == want);
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (lane + 64 * k == count) {
                path[k] = node;
                said[k] = want;
            }
        ++count;
        node = lo ? __ffsll(static_cast<long long>(lo)) - 1
                  : (hi ? 63 + __ffsll(static_cast<long long>(hi)) : -1);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int j = lane + 64 * k;
        if (j < a.T) {
            a.path[row + j] = path[k];
            a.emitted[row + j] = said[k];
        }
    }
    if (lane == 0) a.count[b] = count;
}

// ---------------------------------------------------------------------------
// Moving accepted positions together, in place.  The path ascends, so position
// i is never the source of a later move than its own: a thread that owns 16
// bytes of a head's slots moves them in order, four loads before their stores,
// and no other thread touches them.  Four pools of a sequence 2.2 us, eight pools of
// 256 trees of 64 nodes 6.8 us: four reads that wait for each other (path, lengths
// and table, the slots' own) and then memory.
// ---------------------------------------------------------------------------
struct PoolArgs {
    char *base[kMaxPools];
    int64_t page_stride, head_stride, slot_stride;
    int32_t count, heads, units, pages, shift;
};

struct KeepArgs {
    PoolArgs pool;
    const int32_t *table, *lengths, *path, *count;
    int32_t *new_lengths;  // null but in the first launch
    int32_t T, P, blocks;  // blocks: workgroups per sequence
};

__global__ __launch_bounds__(kCacheBlock) void cache_keep_kernel(KeepArgs a) {
    __shared__ int64_t sh_from[kMaxKeepNodes], sh_to[kMaxKeepNodes];
    __shared__ int sh_end, sh_any;
    const int b = blockIdx.x / a.blocks, part = blockIdx.x % a.blocks;
    const int tid = threadIdx.x;
    const int n = clamp_len(a.count[b], a.T);
    const int32_t *path = a.path + static_cast<int64_t>(b) * a.T;
    if (tid == 0) {
        sh_end = n;
        sh_any = kMaxKeepNodes;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kCacheBlock) {
        const int p = path[i];
        if (p >= a.T || p <= (i ? path[i - 1] : -1)) atomicMin(&sh_end, i);
    }
    __syncthreads();
    const int end = sh_end;
    const int room = a.P << a.pool.shift;
    const int length = clamp_len(a.lengths[b], room);
    if (part == 0 && tid == 0 && a.new_lengths)
        a.new_lengths[b] = length > room - end ? room : length + end;
    const int32_t *table = a.table + static_cast<int64_t>(b) * a.P;
    const int slot_mask = (1 << a.pool.shift) - 1;
    for (int i = tid; i < end; i += kCacheBlock) {
        const int64_t from = static_cast<int64_t>(length) + path[i], to = length + i;
        int64_t x = -1, y = -1;
        if (from != to && from < room) {
            const int pf = table[from >> a.pool.shift], pt = table[to >> a.pool.shift];
            if (static_cast<uint32_t>(pf) < static_cast<uint32_t>(a.pool.pages) &&
                static_cast<uint32_t>(pt) < static_cast<uint32_t>(a.pool.pages)) {
                x = pf * a.pool.page_stride + (from & slot_mask) * a.pool.slot_stride;
                y = pt * a.pool.page_stride + (to & slot_mask) * a.pool.slot_stride;
                atomicMin(&sh_any, i);
            }
        }
        sh_from[i] = x;
        sh_to[i] = y;
    }
    __syncthreads();
    const int columns = a.pool.count * a.pool.heads * a.pool.units;
    const int c = part * kCacheBlock + tid;
    if (c >= columns) return;
    const int unit = c % a.pool.units, h = c / a.pool.units % a.pool.heads;
    char *base = a.pool.base[c / a.pool.units / a.pool.heads] + h * a.pool.head_stride + unit * 16;
    for (int i = sh_any; i < end; i += 4) {
        v4u32 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < end && sh_from[i + k] >= 0)
                v[k] = *reinterpret_cast<const v4u32 *>(base + sh_from[i + k]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < end && sh_from[i + k] >= 0)
                *reinterpret_cast<v4u32 *>(base + sh_to[i + k]) = v[k];
    }
}

// ---------------------------------------------------------------------------
// Copying pages: a workgroup per row, pool and head, whose slots lie together.  Four
// branches 3.0 us, 512 in eight pools, 134 MB read and written, 23.7 us (5.7 TB/s):
// memory.
// ---------------------------------------------------------------------------
struct CopyArgs {
    PoolArgs pool;
    const int32_t *copies;  // [rows][3]
};

__global__ __launch_bounds__(kCacheBlock) void pages_copy_kernel(CopyArgs a) {
    const int parts = a.pool.count * a.pool.heads;
    const int row = blockIdx.x / parts, part = blockIdx.x % parts;
    const int32_t *c = a.copies + static_cast<int64_t>(row) * 3;
    const int from = c[0], to = c[1];
    const int slots = clamp_len(c[2], 1 << a.pool.shift);
    if (static_cast<uint32_t>(from) >= static_cast<uint32_t>(a.pool.pages) ||
        static_cast<uint32_t>(to) >= static_cast<uint32_t>(a.pool.pages) || from == to)
        return;
    char *base = a.pool.base[part / a.pool.heads] + part % a.pool.heads * a.pool.head_stride;
    const char *src = base + from * a.pool.page_stride;
    char *dst = base + to * a.pool.page_stride;
    for (int i = threadIdx.x; i < slots * a.pool.units; i += kCacheBlock) {
        const int64_t at = i / a.pool.units * a.pool.slot_stride + i % a.pool.units * 16;
        *reinterpret_cast<v4u32 *>(dst + at) = *reinterpret_cast<const v4u32 *>(src + at);
    }
}

// ---------------------------------------------------------------------------
// Sharing and releasing: a workgroup per table row, a thread per entry.  Four rows 2.1
// us, 512 rows 3.6 to 4.2: the counts' atomics, which eight branches of a sequence
// send to the same places.
// ---------------------------------------------------------------------------
struct ForkArgs {
    const int32_t *table, *lengths, *parents;
    int32_t *refs, *out, *out_lengths;
    int32_t W, n, P, shift, pages;
};

__global__ __launch_bounds__(kCacheBlock) void pages_fork_kernel(ForkArgs a) {
    const int b = blockIdx.x / a.n;
    const int w = a.parents[blockIdx.x];
    const bool there = w >= 0 && w < a.W;
    const int64_t from = static_cast<int64_t>(b) * a.W + (there ? w : 0);
    const int length = there ? a.lengths[from] : 0;
    const int held = (clamp_len(length, a.P << a.shift) + (1 << a.shift) - 1) >> a.shift;
    if (threadIdx.x == 0) a.out_lengths[blockIdx.x] = length;
    for (int i = threadIdx.x; i < a.P; i += kCacheBlock) {
        int page = i < held ? a.table[from * a.P + i] : -1;
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.pages))
            page = -1;
        else
            atomicAdd(&a.refs[page], 1);
        a.out[static_cast<int64_t>(blockIdx.x) * a.P + i] = page;
    }
}

struct ReleaseArgs {
    int32_t *table, *refs;
    const int32_t *lengths;  // or null (= 0)
    int32_t P, shift, pages;
};

__global__ __launch_bounds__(kCacheBlock) void pages_release_kernel(ReleaseArgs a) {
    const int length = a.lengths ? clamp_len(a.lengths[blockIdx.x], a.P << a.shift) : 0;
    const int held = (length + (1 << a.shift) - 1) >> a.shift;
    int32_t *row = a.table + static_cast<int64_t>(blockIdx.x) * a.P;
    for (int i = held + threadIdx.x; i < a.P; i += kCacheBlock) {
        const int page = row[i];
        if (static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pages)) {
            // a count that has run out is put back; as many of the subtractions
            // succeed as there were references, in any order
            if (atomicSub(&a.refs[page], 1) <= 0) atomicAdd(&a.refs[page], 1);
        }
        row[i] = -1;
    }
}

// ---------------------------------------------------------------------------
// Reserving.  One workgroup finds what the rows need and hands out free pages in
// order; which pages are free, 64 to a word, with the words' running counts in
// every chunk of 1024, it looks up itself in a small pool and a launch before it
// does in a larger one.
//
// A row's entries that are about to be written belong to a group of lanes, as
// many as the widest row needs.  Shared pages among them are settled in the
// pages' own counts: every entry takes its reference off; a page that has none
// left then has all its holders here, and the lowest row among them, found by a
// minimum over row - 2^30, keeps it, with the first entry that lists the page where
// the row does so more than once.
//
// Where the rows fit the workgroup, an entry to a thread (a step of decoding),
// entries stay in registers (four rows in 4096 pages 6.9 us, 512 rows in 40000 pages
// 3.9 us for the first launch and 11.5: barriers and atomics that wait for each
// other in one workgroup; through the table the same 512 rows took 23); otherwise
// shared ones are marked in the table (kSharedMark + page) until they are settled.
// ---------------------------------------------------------------------------
constexpr int kReserveBlock = 1024;
constexpr int kPageChunk = 1024;                   // pages to a count
constexpr int kChunkWords = kPageChunk / kWave;
constexpr int kMaxReservePages = 1 << 22;
constexpr int kMaxReserveRows = 65536;
constexpr int kKeeper = 1 << 30;
constexpr int kSharedMark = -2147483647 - 1;
// Chunks that the workgroup looks through by itself.  In a graph 4 take 6.2 us and 7.2
// with a launch before it, 16 take 7.3 and 7.4, 32 take 10.5 and 7.5; called one by
// one, the launch costs the host 3.5 us more.
constexpr int kReserveAlone = 16;

struct ReserveArgs {
    int32_t *table, *refs, *copies, *missing;
    const int32_t *lengths, *news;
    unsigned long long *words;  // [chunks][16]
    int32_t *before;            // [chunks][16]: free pages of the chunk before a word
    int32_t *counts;            // [chunks]
    int32_t rows, P, shift, pages, chunks;
};

// One wave: a chunk's words and counts.
__device__ __forceinline__ void chunk_words(const ReserveArgs &a, int c, int lane) {
    int v[kChunkWords];
#pragma unroll
    for (int k = 0; k < kChunkWords; ++k) {
        const int at = c * kPageChunk + k * kWave + lane;
        v[k] = a.refs[at < a.pages ? at : a.pages - 1];
        if (at >= a.pages) v[k] = 1;
    }
    int free = 0;
#pragma unroll
    for (int k = 0; k < kChunkWords; ++k) {
        const uint64_t w = __ballot(v[k] <= 0);
        if (lane == 0) {
            a.words[c * kChunkWords + k] = w;
            a.before[c * kChunkWords + k] = free;
        }
        free += __popcll(w);
    }
    if (lane == 0) a.counts[c] = free;
}

__global__ __launch_bounds__(kCacheBlock) void pages_free_kernel(ReserveArgs a) {
    const int c = blockIdx.x * (kCacheBlock / kWave) + threadIdx.x / kWave;
    if (c < a.chunks) chunk_words(a, c, threadIdx.x & (kWave - 1));
}

// Inclusive scan of v over the workgroup; the total goes to every thread.
__device__ __forceinline__ int reserve_scan(int v, int *sh, int &total) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int u = __shfl_up(v, o, kWave);
        if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == kWave - 1) sh[wave] = v;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kReserveBlock / kWave; ++w) {
        if (w < wave) v += sh[w];
        total += sh[w];
    }
    return v;
}

// The free page of this rank: the chunk is the last one with no more before it,
// likewise the word.
__device__ __forceinline__ int free_page(const ReserveArgs &a, const int *before, int rank) {
    int c = 0;
    for (int step = kMaxReservePages / kPageChunk; step; step >>= 1)
        if (c + step < a.chunks && before[c + step] <= rank) c += step;
    rank -= before[c];
    int w = -1, base = 0;
#pragma unroll
    for (int k = 0; k < kChunkWords; ++k) {
        const int b = a.before[c * kChunkWords + k];
        if (b <= rank) {
            ++w;
            base = b;
        }
    }
    uint64_t bits = a.words[c * kChunkWords + w];
    for (rank -= base; rank > 0; --rank) bits &= bits - 1;
    return c * kPageChunk + w * kWave + __ffsll(static_cast<long long>(bits)) - 1;
}

__global__ __launch_bounds__(kReserveBlock) void pages_reserve_kernel(ReserveArgs a) {
    __shared__ int sh_before[kMaxReservePages / kPageChunk];
    __shared__ int sh_scan[kReserveBlock / kWave];
    __shared__ int sh_widest, sh_over, sh_twice;
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    if (tid == 0) {
        sh_widest = 1;
        sh_over = 0;
        sh_twice = 0;
    }
    const int room = a.P << a.shift, page_size = 1 << a.shift;
    // the table entries [lo, hi) that row r is about to write (hi -1: too many)
    auto range = [&](int r, int &lo, int &hi, int &length) {
        lo = hi = length = 0;
        if (r >= a.rows) return;
        const int given = a.lengths[r], more = a.news[r] > 0 ? a.news[r] : 0;
        length = clamp_len(given, room);
        lo = length >> a.shift;
        if (more > room - length || (more > 0 && given > room))
            hi = -1;
        else
            hi = more == 0 ? lo : (length + more + page_size - 1) >> a.shift;
    };
    __syncthreads();
    for (int r = tid; r < a.rows; r += kReserveBlock) {
        int lo, hi, length;
        range(r, lo, hi, length);
        if (hi < 0)
            atomicMax(&sh_over, 1);
        else
            atomicMax(&sh_widest, hi - lo);
    }
    if (a.chunks <= kReserveAlone) {
        for (int c = tid / kWave; c < a.chunks; c += kReserveBlock / kWave) chunk_words(a, c, lane);
        __threadfence_block();
    }
    __syncthreads();
    // free pages before each chunk
    int free = 0;
    for (int c0 = 0; c0 < a.chunks; c0 += kReserveBlock) {
        const int c = c0 + tid, mine = c < a.chunks ? a.counts[c] : 0;
        int total;
        const int upto = reserve_scan(mine, sh_scan, total);
        if (c < a.chunks) sh_before[c] = free + upto - mine;
        free += total;
    }
    const bool over = sh_over != 0;
    // lanes to a row: a power of two that holds the widest range, up to a wave
    int group = 1;
    while (group < kWave && group < sh_widest) group <<= 1;
    const int in = tid & (group - 1), batch = kReserveBlock / group;
    auto copy_of = [&](int r, int from, int to, int n) {
        int32_t *c = a.copies + 3 * static_cast<int64_t>(r);
        c[0] = from;
        c[1] = to;
        c[2] = n;
    };
    auto is_page = [&](int e) { return static_cast<uint32_t>(e) < static_cast<uint32_t>(a.pages); };
    auto is_mark = [&](int e) { return e < kSharedMark + a.pages; };

    if (a.rows <= batch && sh_widest <= group) {
        const int r = tid / group;
        int lo, hi, length;
        range(r, lo, hi, length);
        int32_t *at = a.table + static_cast<int64_t>(r) * a.P + lo + in;
        const bool mine = !over && lo + in < hi;
        const int e = mine ? *at : -1;
        const bool held = mine && is_page(e);
        const bool shared = held && a.refs[held ? e : 0] > 1;
        bool stays = false;
        if (__syncthreads_or(shared)) {
            if (shared) atomicSub(&a.refs[e], 1);
            __syncthreads();
            // threads are in the entries' order
            if (shared && atomicAdd(&a.refs[e], 0) <= 0) atomicMin(&a.refs[e], tid - kKeeper);
            __syncthreads();
            if (shared) stays = atomicAdd(&a.refs[e], 0) + kKeeper == tid;
        }
        const bool fresh = mine && (!held || (shared && !stays));
        int total;
        const int upto = reserve_scan(fresh, sh_scan, total);
        const int missing = over ? -1 : (total > free ? total - free : 0);
        if (tid == 0) a.missing[0] = missing;
        int page = -1;
        if (missing != 0) {
            // nothing is taken: the references go back
            if (stays) atomicExch(&a.refs[e], 0);
            __syncthreads();
            if (shared) atomicAdd(&a.refs[e], 1);
        } else {
            if (stays) atomicExch(&a.refs[e], 1);
            if (fresh) {
                page = free_page(a, sh_before, upto - 1);
                *at = page;
                a.refs[page] = 1;
            }
        }
        if (r < a.rows && in == 0) {
            const int n = length & (page_size - 1);
            const bool moved = page >= 0 && held && n > 0;
            copy_of(r, moved ? e : -1, moved ? page : -1, moved ? n : 0);
        }
        return;
    }

    const uint64_t below = (group == kWave ? ~0ull : ((1ull << group) - 1))
                           << (lane & ~(group - 1));
    // what a page's count says once row r is to keep it, and once an entry of it does
    auto keeper = [](int r) { return r - kKeeper; };
    auto claimed = [](int r) { return r - kKeeper - kMaxReserveRows; };
    // whether the marked entry i of row r, which begins at lo, keeps its page (after
    // phase 3)
    auto keeps = [&](const int32_t *row, int lo, int i, int r) {
        const int e = row[i];
        if (atomicAdd(&a.refs[e - kSharedMark], 0) != claimed(r)) return false;
        if (sh_twice)
            for (int j = lo; j < i; ++j)
                if (row[j] == e) return false;
        return true;
    };
    int need = 0;
    // phase 0 marks shared entries, 1 takes their references off, 2 finds who
    // keeps, 3 counts what is needed
    for (int phase = 0; phase < 4 && !over; ++phase) {
        for (int r0 = 0; r0 < a.rows; r0 += batch) {
            const int r = r0 + tid / group;
            int lo, hi, length;
            range(r, lo, hi, length);
            int32_t *row = a.table + static_cast<int64_t>(r) * a.P;
            for (int i = lo + in; i < hi; i += group) {
                const int e = row[i];
                if (phase == 0) {
                    if (is_page(e)) {
                        if (a.refs[e] > 1) row[i] = kSharedMark + e;
                    } else if (is_mark(e)) {
                        row[i] = -1;  // lists nothing, and must not be taken for a mark
                    }
                } else if (is_mark(e)) {
                    int *ref = &a.refs[e - kSharedMark];
                    if (phase == 1) atomicSub(ref, 1);
                    if (phase == 2 && atomicAdd(ref, 0) <= 0) atomicMin(ref, keeper(r));
                    if (phase == 3) {
                        const int v = atomicCAS(ref, keeper(r), claimed(r));
                        if (v == claimed(r)) sh_twice = 1;  // the row lists it again
                        need += v != keeper(r);
                    }
                } else if (phase == 3) {
                    need += !is_page(e);
                }
            }
        }
        __threadfence_block();
        __syncthreads();
    }
    int total;
    reserve_scan(need, sh_scan, total);
    const int missing = over ? -1 : (total > free ? total - free : 0);
    if (tid == 0) a.missing[0] = missing;
    if (missing != 0) {
        // nothing is taken: the references and marks go back
        for (int phase = 0; phase < 2; ++phase) {
            for (int r0 = 0; r0 < a.rows; r0 += batch) {
                const int r = r0 + tid / group;
                if (r < a.rows && in == 0 && phase == 0) copy_of(r, -1, -1, 0);
                int lo, hi, length;
                range(r, lo, hi, length);
                int32_t *row = a.table + static_cast<int64_t>(r) * a.P;
                for (int i = lo + in; i < hi && !over; i += group) {
                    const int e = row[i];
                    if (!is_mark(e)) continue;
                    int *ref = &a.refs[e - kSharedMark];
                    if (phase == 0) {
                        if (atomicAdd(ref, 0) == claimed(r)) atomicExch(ref, 0);
                    } else {
                        atomicAdd(ref, 1);
                        row[i] = e - kSharedMark;
                    }
                }
            }
            __threadfence_block();
            __syncthreads();
        }
        return;
    }
    int taken = 0;  // pages handed out to earlier rows
    for (int r0 = 0; r0 < a.rows; r0 += batch) {
        const int r = r0 + tid / group;
        int lo, hi, length;
        range(r, lo, hi, length);
        int32_t *row = a.table + static_cast<int64_t>(r) * a.P;
        auto fresh = [&](int i, int &e) {
            e = i < hi ? row[i] : 0;
            if (is_mark(e)) return !keeps(row, lo, i, r);
            return !is_page(e);
        };
        int mine = 0, e;
        for (int i = lo + in; i < hi; i += group) mine += fresh(i, e);
        int all;
        const int upto = reserve_scan(mine, sh_scan, all);
        // the row's first: what all threads before its group's first need
        const int before = taken + __shfl(upto - mine, lane & ~(group - 1), kWave);
        int copy_from = -1, copy_to = -1, copy_n = 0, done = 0;
        for (int i0 = lo; __any(i0 < hi); i0 += group) {
            const int i = i0 + in;
            const bool f = fresh(i, e);
            const uint64_t who = __ballot(f) & below;
            if (f) {
                const int page =
                    free_page(a, sh_before, before + done + __popcll(who & ((1ull << lane) - 1)));
                row[i] = page;
                a.refs[page] = 1;
                if (is_mark(e) && i == lo && (length & (page_size - 1))) {
                    copy_from = e - kSharedMark;
                    copy_to = page;
                    copy_n = length & (page_size - 1);
                }
            }
            done += __popcll(who);
        }
        if (r < a.rows && in == 0) copy_of(r, copy_from, copy_to, copy_n);
        taken += all;
    }
    __threadfence_block();
    __syncthreads();
    // what keeps its page is its only holder now
    for (int r0 = 0; r0 < a.rows; r0 += batch) {
        const int r = r0 + tid / group;
        int lo, hi, length;
        range(r, lo, hi, length);
        int32_t *row = a.table + static_cast<int64_t>(r) * a.P;
        for (int i = lo + in; i < hi; i += group) {
            const int e = row[i];
            if (is_mark(e)) {
                row[i] = e - kSharedMark;
                atomicExch(&a.refs[e - kSharedMark], 1);
            }
        }
    }
}

}  // namespace sv
