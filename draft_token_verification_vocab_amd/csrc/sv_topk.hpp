// sv_topk.hpp -- the k largest logits of each row, in decreasing order with
// equal values by lowest id, and the row's log-normaliser, in one pass.
//
// A logit and its id make one 64-bit key: the ordered bits of the value above
// the complement of the id, so that "larger key" is "earlier in the list" and
// no two keys are equal.
//
// One workgroup streams a row (beam selection with few rows: a segment of it).  A thread keeps, beside
// the online softmax, its chunk (16 logits) with the largest maximum in LDS,
// which chunk comes second, and the second and third largest maximum.  The
// k-th largest of the threads' maxima is then a lower bound tau of the k-th
// largest logit: k threads hold a logit that large.  The logits at or above
// tau lie in about k best chunks, the few second chunks that reach tau (read
// again), and all chunks of the very few threads with a third one; they are
// collected and placed by counting.  A row whose collection overflows (many
// equal logits) is settled by further passes (collect_ties).
//
// Bound: vector issue and memory alike (9.1 instructions per logit, one of them
// the quarter-rate exp2: 79 % busy).  2304 rows of 128256 bfloat16 logits, k = 64:
// 96 us, 6.2 TB/s; without the normaliser 90; the load-only pass over the same
// rows takes 84.  Cut short after the stream the launch takes 89 to 90.  Two
// register buffers in turn took the whole from 108 to 96 us (the stream alone
// took 90 before, too).  Saving the second chunks in LDS too gained nothing (115
// us against 112 then).
// Few rows wait for one compute unit each: 256 KB take it 10 us.
#pragma once

#include "sv_stream.hpp"

namespace sv {

constexpr int kTopkMax = 128;        // longest list
constexpr int kTopkCollect = 1024;   // logits one workgroup can collect
constexpr int kTopkChunks = 1024;    // chunks it can note
constexpr int kRankKeys = 256;       // collected keys placed by counting

struct TopkArgs {
    const void *base;
    int64_t stride;          // elements between consecutive rows
    int32_t V;
    int32_t k;
    int32_t segs;            // segments (workgroups) per row, 1 without a list
    int32_t seg_vecs;        // 16-byte vectors per segment
    float c;                 // log2(e) / T
    float pad_;
    double inv_t;            // 1 / T
    // the caller's outputs (lse nullable)
    float *values;           // [rows][k]
    int32_t *ids;            // [rows][k]
    float *lse;              // [rows]
    // or lists for the beam merge: keys in decreasing order, 0 after the last
    unsigned long long *list;  // [rows][segs][k]
    double *seg_lse;           // [rows][segs] ln sum e^((l - max)/T), -inf when all is masked
    // rows that take no part (beam selection), both nullable
    const uint8_t *ended;    // [rows]
    const float *scores;     // [rows]: -inf takes no part
};

__device__ __forceinline__ uint64_t topk_key(float x, int id) {
    return (static_cast<uint64_t>(ordered_bits(x + 0.0f)) << 32) |
           static_cast<uint32_t>(~static_cast<uint32_t>(id));
}
__device__ __forceinline__ float key_value(uint64_t key) {
    return from_ordered_bits(static_cast<uint32_t>(key >> 32));
}
__device__ __forceinline__ int key_id(uint64_t key) {
    return static_cast<int>(~static_cast<uint32_t>(key));
}

// Sorts n2 (a power of two) keys in LDS in decreasing order.
template <int BLOCK>
__device__ void sort_keys(unsigned long long *key, int n2, int tid) {
    for (int size = 2; size <= n2; size *= 2) {
        for (int step = size / 2; step > 0; step /= 2) {
            __syncthreads();
            for (int p = tid; p < n2 / 2; p += BLOCK) {
                const int i = 2 * p - (p & (step - 1));
                const int j = i + step;
                const unsigned long long a = key[i], b = key[j];
                const bool up = (i & size) == 0;  // this run decreases
                if (up ? a < b : a > b) {
                    key[i] = b;
                    key[j] = a;
                }
            }
        }
    }
    __syncthreads();
}

// Collects exactly the segment's k first keys where more logits than can be
// collected reach the bound `lo` (at least k do; `hi` is the maximum; both as
// ordered bits): equal values, mostly.  Passes over the segment narrow [lo, hi]
// to the k-th largest value, 256 bins at a time (none when it is the maximum
// itself, as in a constant or clamped row); a last pass takes the values above
// it, and of those equal to it the first ids, counted tile by tile in id order.
// 2304 rows of 128256 bfloat16 logits, short bursts: 138 us when all are
// constant, 155 when clamped, 92 to 100 when none is (3700 with a radix
// selection over whole keys instead).
template <typename T, int BLOCK>
__device__ __attribute__((noinline)) int collect_ties(const T *row, int vbeg, int vend, int V,
                                                      int k, uint32_t lo, uint32_t hi,
                                                      unsigned long long *keys, int *hist,
                                                      int tid) {
    using E = Elem<T>;
    constexpr int EPV = E::kPerVec;
    constexpr int NW = BLOCK / kWave;
    __shared__ uint32_t sh_lo, sh_hi;
    __shared__ int sh_above, sh_n, sh_wave[NW];
    const int lane = tid & (kWave - 1), wv = tid / kWave;
    auto load = [&](int vi, uint32_t (&key)[EPV]) {  // ordered bits, 0 past the end
        float x[EPV];
        E::unpack(vi < vend ? ((vi + 1) * EPV <= V ? reinterpret_cast<const uint4 *>(row)[vi]
                                                   : E::partial(row, vi, V))
                            : make_uint4(E::pad_word(), E::pad_word(), E::pad_word(),
                                         E::pad_word()),
                  x);
#pragma unroll
        for (int e = 0; e < EPV; ++e) key[e] = x[e] > kMasked ? ordered_bits(x[e] + 0.0f) : 0u;
    };
    int above = 0;  // logits above hi
    while (lo < hi) {
        const int width = 32 - __clz(static_cast<int>(hi - lo));
        const int shift = width > 8 ? width - 8 : 0;
        for (int i = tid; i < 256; i += BLOCK) hist[i] = 0;
        __syncthreads();
        for (int vi = vbeg + tid; vi < vend; vi += BLOCK) {
            uint32_t key[EPV];
            load(vi, key);
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                if (key[e] < lo || key[e] > hi) continue;
                // lanes that share the first lane's bin count once together
                const int bin = static_cast<int>((key[e] - lo) >> shift);
                const int lead = __builtin_amdgcn_readfirstlane(bin);
                const uint64_t same = __ballot(bin == lead);
                if (bin != lead)
                    atomicAdd(&hist[bin], 1);
                else if (lane == __ffsll(static_cast<long long>(same)) - 1)
                    atomicAdd(&hist[lead], __popcll(same));
            }
        }
        __syncthreads();
        if (tid == 0) {
            int bin = static_cast<int>((hi - lo) >> shift), n = above;
            while (bin > 0 && n + hist[bin] < k) n += hist[bin--];
            const uint32_t from = lo + (static_cast<uint32_t>(bin) << shift);
            const uint32_t to = from + ((1u << shift) - 1u);
            sh_above = n;
            sh_lo = from;
            sh_hi = to < hi ? to : hi;
        }
        __syncthreads();
        above = sh_above;
        lo = sh_lo;
        hi = sh_hi;
        __syncthreads();  // read before the next pass writes them
    }
    // keys above lo, and the first `left` equal to it
    int left = k - above;
    if (tid == 0) sh_n = 0;
    __syncthreads();
    for (int tile = vbeg; tile < vend; tile += BLOCK) {
        const int vi = tile + tid;
        uint32_t key[EPV];
        load(vi, key);
        int equal = 0;
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
            equal += key[e] == lo;
            if (key[e] > lo)
                keys[atomicAdd(&sh_n, 1)] = (static_cast<uint64_t>(key[e]) << 32) |
                                            static_cast<uint32_t>(~(vi * EPV + e));
        }
        if (left <= 0) {  // the same for every thread
            if (above == 0) break;
            continue;
        }
        int upto = equal;         // within the wave, this lane included
#pragma unroll
        for (int o = 1; o < kWave; o *= 2) {
            const int below = __shfl_up(upto, o, kWave);
            if (lane >= o) upto += below;
        }
        if (lane == kWave - 1) sh_wave[wv] = upto;
        __syncthreads();
        int before = upto - equal, total = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            before += w < wv ? sh_wave[w] : 0;
            total += sh_wave[w];
        }
        if (equal != 0 && before < left) {
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                if (key[e] != lo || before >= left) continue;
                ++before;
                keys[atomicAdd(&sh_n, 1)] = (static_cast<uint64_t>(key[e]) << 32) |
                                            static_cast<uint32_t>(~(vi * EPV + e));
            }
        }
        left -= total;
        __syncthreads();  // sh_wave is free
    }
    __syncthreads();
    return sh_n;
}

// LSE: with the log-normaliser (else a third of the arithmetic is left out).
template <typename T, int BLOCK, int UNROLL, bool LSE>
__global__ __launch_bounds__(BLOCK) void topk_rows_kernel(TopkArgs a) {
    using E = Elem<T>;
    constexpr int EPV = E::kPerVec;
    constexpr int N = UNROLL * EPV;
    constexpr int NW = BLOCK / kWave;
    constexpr int kChunk = UNROLL * BLOCK;
    __shared__ uint4 sh_saved[UNROLL][BLOCK];  // the threads' best chunks
    __shared__ unsigned long long sh_key[kTopkCollect];
    __shared__ uint32_t sh_m[BLOCK];
    __shared__ int sh_item[kTopkChunks];
    __shared__ uint32_t sh_wm[NW], sh_wl[NW];
    __shared__ double sh_s[NW];
    __shared__ uint32_t sh_tau;
    __shared__ int sh_n, sh_items;
    static_assert(BLOCK <= 1024, "a noted chunk is its index and its thread");

    const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = tid / kWave;
    const int64_t row = blockIdx.x / a.segs;
    const int seg = static_cast<int>(blockIdx.x - row * a.segs);
    if (a.ended && a.ended[row]) return;
    if (a.scores && !(a.scores[row] > -__builtin_inff())) return;
    const T *rp = static_cast<const T *>(a.base) + row * a.stride;
    const int V = a.V, k = a.k;
    const float c = a.c;
    const int nvec = (V + EPV - 1) / EPV;
    const int vbeg = seg * a.seg_vecs;
    const int vend = vbeg + a.seg_vecs < nvec ? vbeg + a.seg_vecs : nvec;

    OnlineSum acc(c);
    int best = 0, second = 0;             // the chunks with the thread's largest maxima
    float m2 = kMasked, m3 = kMasked;     // the second and third largest chunk maximum
    stream_vectors<T, BLOCK, UNROLL>(rp, vbeg, vend, V, tid,
                                     [&](const uint4 (&buf)[UNROLL], int it) {
        float x[N];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) E::unpack(buf[u], x + u * EPV);
        const float cm = chunk_max(x);
        // acc.m >= m2 >= m3: the new second and third largest are medians
        m3 = __builtin_amdgcn_fmed3f(m3, cm, m2);
        second = cm > acc.m ? best : (cm > m2 ? it : second);
        m2 = __builtin_amdgcn_fmed3f(m2, cm, acc.m);
        if (cm > acc.m) {
            best = it;
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) sh_saved[u][tid] = buf[u];
        }
        if (LSE)
            acc.add(x, cm, c);
        else
            acc.m = cm > acc.m ? cm : acc.m;
    });

    // Segment maximum, smallest visible thread maximum, and the normaliser.
    const uint32_t masked = ordered_bits(kMasked);
    const uint32_t om = ordered_bits(acc.m + 0.0f);
    sh_m[tid] = om;
    const uint32_t wm = wave_max_u32(om);
    const uint32_t wl = wave_max_u32(om > masked ? ~om : 0u);
    if (lane == 0) {
        sh_wm[wv] = wm;
        sh_wl[wv] = wl;
    }
    if (tid == 0) sh_n = sh_items = 0;
    __syncthreads();
    uint32_t bm = sh_wm[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) bm = sh_wm[w] > bm ? sh_wm[w] : bm;
    const float M = from_ordered_bits(bm);
    if (LSE) {
        const double ws = wave_sum_f64(acc.at(M, c));
        if (lane == 0) sh_s[wv] = ws;
    }

    // tau: a value that at least k threads' maxima reach (all visible logits
    // when fewer than k threads hold one).  The first wave builds it bit by
    // bit below the bits that all visible maxima share, and stops as soon as
    // few more than k threads reach it.
    if (wv == 0) {
        uint32_t key[NW], bl = 0;
        int seen = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            key[w] = sh_m[w * kWave + lane];
            bl = sh_wl[w] > bl ? sh_wl[w] : bl;
            seen += __popcll(__ballot(key[w] > masked));
        }
        uint32_t tau = 0;
        if (seen >= k) {
            const int enough = k + k / 4 + 4;
            const uint32_t differ = bm ^ ~bl;
            int bit = 31 - __clz(static_cast<int>(differ));
            tau = differ == 0 ? bm : bm & ~((2u << bit) - 1u);
            for (; bit >= 0; --bit) {
                const uint32_t trial = tau | (1u << bit);
                int n = 0;
#pragma unroll
                for (int w = 0; w < NW; ++w) n += __popcll(__ballot(key[w] >= trial));
                if (n >= k) {
                    tau = trial;
                    if (n <= enough) break;
                }
            }
        }
        if (lane == 0) sh_tau = tau > masked ? tau : masked + 1u;
    }
    __syncthreads();
    const uint32_t tau = sh_tau;

    // Collect the logits at or above tau: those of a thread's best chunk from
    // LDS, and of its second chunk, or all its chunks when a third reaches
    // tau, from the row again, noted first and then read together, a vector
    // per thread (one memory latency, whatever the chunks' owners).
    const float least = from_ordered_bits(tau);  // above kMasked
    if (om >= tau) {
        uint32_t hit = 0;
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            float x[EPV];
            E::unpack(sh_saved[u][tid], x);
#pragma unroll
            for (int e = 0; e < EPV; ++e) hit |= x[e] >= least ? 1u << (u * EPV + e) : 0u;
        }
        int o = atomicAdd(&sh_n, __popc(hit));
        for (; hit && o < kTopkCollect; hit &= hit - 1, ++o) {  // one or two, mostly
            const int q = __ffs(static_cast<int>(hit)) - 1, u = q / EPV, e = q % EPV;
            const float x = E::at(reinterpret_cast<const T *>(&sh_saved[u][tid]), e);
            sh_key[o] = topk_key(x, (vbeg + best * kChunk + u * BLOCK + tid) * EPV + e);
        }
        if (m2 >= least) {
            const bool two = !(m3 >= least);
            const int from = two ? second : 0;
            const int to = two ? second : (vend - vbeg - 1 - tid) / kChunk;
            int o = atomicAdd(&sh_items, to - from + 1);
            for (int it = from; it <= to; ++it, ++o)
                if (o < kTopkChunks) sh_item[o] = it == best ? -1 : it * 1024 + tid;
        }
    }
    __syncthreads();
    const int items = sh_items;
    if (items > 0) {  // the same for every thread
        for (int j = tid; j < items * UNROLL && items <= kTopkChunks; j += BLOCK) {
            const int item = sh_item[j / UNROLL];
            const int vi = vbeg + (item >> 10) * kChunk + (j % UNROLL) * BLOCK + (item & 1023);
            if (item < 0 || vi >= vend) continue;
            const uint4 v = (vi + 1) * EPV <= V ? reinterpret_cast<const uint4 *>(rp)[vi]
                                                : E::partial(rp, vi, V);
            float x[EPV];
            E::unpack(v, x);
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                if (!(x[e] >= least)) continue;
                const int o = atomicAdd(&sh_n, 1);
                if (o < kTopkCollect) sh_key[o] = topk_key(x[e], vi * EPV + e);
            }
        }
        __syncthreads();
    }
    int n = items <= kTopkChunks ? sh_n : kTopkCollect + 1;
    if (n > kTopkCollect)  // too many logits reach tau
        n = collect_ties<T, BLOCK>(rp, vbeg, vend, V, k, tau, bm, sh_key, sh_item, tid);

    // Places: up to kRankKeys keys are counted against all others, a thread
    // each; more are sorted first.
    unsigned long long *list = a.list ? a.list + static_cast<int64_t>(blockIdx.x) * k : nullptr;
    auto put = [&](int rank, uint64_t key) {
        if (list) {
            list[rank] = key;
        } else {
            a.values[row * k + rank] = key ? key_value(key) : -__builtin_inff();
            a.ids[row * k + rank] = key ? key_id(key) : -1;
        }
    };
    if (n <= kRankKeys) {
        // as many lanes per key as the workgroup has, each against its share
        int share = 1;
        while (share < 16 && n * share * 2 <= BLOCK) share *= 2;
        const int at = tid / share;
        const uint64_t mine = at < n ? sh_key[at] : 0;
        int rank = 0;
#pragma unroll 4
        for (int j = tid & (share - 1); j < n; j += share) rank += sh_key[j] > mine;
        for (int o = 1; o < share; o *= 2) rank += __shfl_xor(rank, o, kWave);
        if (at < n && (tid & (share - 1)) == 0 && rank < k) put(rank, mine);
    } else {
        int n2 = 2 * kRankKeys;
        while (n2 < n) n2 *= 2;
        for (int i = n + tid; i < n2; i += BLOCK) sh_key[i] = 0;
        sort_keys<BLOCK>(sh_key, n2, tid);
        for (int i = tid; i < k && i < n; i += BLOCK) put(i, sh_key[i]);
    }
    for (int i = n + tid; i < k; i += BLOCK) put(i, 0);

    if (LSE && tid == BLOCK - 1) {
        double r = 0.0;
#pragma unroll
        for (int w = 0; w < NW; ++w) r += sh_s[w];
        const double l = bm > masked ? log_f64(r) - OnlineSum::above_max(M, c) * kLn2
                                     : -__builtin_inf();
        if (a.list)
            a.seg_lse[blockIdx.x] = l;
        else
            a.lse[row] = static_cast<float>(static_cast<double>(M) * a.inv_t + l);
    }
}

}  // namespace sv
