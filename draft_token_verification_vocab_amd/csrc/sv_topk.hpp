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
// collected and placed by counting.  A row whose collection overflows (many equal logits) is settled by a radix
// selection over the keys instead, which reads the row once per key byte.
//
// Bound: vector issue and memory alike (8.7 instructions per logit, one of them
// the quarter-rate exp2: 77 % busy).  2304 rows of 128256 bfloat16 logits, k = 64:
// 96 us, 6.2 TB/s; without the normaliser 90; the load-only pass over the same
// rows takes 84.  Cutting the launch short showed 90 of 108 us in the stream;
// keeping two register buffers in turn there gave 12 of them back.  Saving the
// second chunks in LDS too gained nothing (115 us against 112 then).
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

// The exact k-th largest key of a segment's visible logits (0 when there are
// at most k) by radix selection, eight key bits a pass over the segment.
template <typename T, int BLOCK>
__device__ __attribute__((noinline)) uint64_t radix_kth(const T *row, int ebeg, int eend, int k,
                                                        unsigned int *hist, int tid) {
    __shared__ uint64_t sh_prefix;
    __shared__ int sh_left;
    uint64_t prefix = 0, mask = 0;
    int left = k;
    for (int shift = 56; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += BLOCK) hist[i] = 0;
        __syncthreads();
        for (int i = ebeg + tid; i < eend; i += BLOCK) {
            const float x = Elem<T>::at(row, i);
            const uint64_t key = topk_key(x, i);
            if (x > kMasked && (key & mask) == prefix) {
                const int bin = static_cast<int>((key >> shift) & 255u);
                // lanes that share the first lane's bin count once together
                const int lead = __builtin_amdgcn_readfirstlane(bin);
                const uint64_t same = __ballot(bin == lead);
                if (bin != lead)
                    atomicAdd(&hist[bin], 1u);
                else if ((threadIdx.x & (kWave - 1)) ==
                         static_cast<unsigned>(__ffsll(static_cast<long long>(same)) - 1))
                    atomicAdd(&hist[lead], static_cast<unsigned>(__popcll(same)));
            }
        }
        __syncthreads();
        if (tid == 0) {
            int bin = 255, n = left;
            while (bin >= 0 && static_cast<int>(hist[bin]) < n) n -= static_cast<int>(hist[bin--]);
            sh_left = bin < 0 ? 0 : n;
            sh_prefix = bin < 0 ? 0 : prefix | (static_cast<uint64_t>(bin) << shift);
        }
        __syncthreads();
        left = sh_left;
        prefix = sh_prefix;
        mask |= 0xFFull << shift;
        __syncthreads();  // read before the next pass writes them
        if (left == 0) return 0;  // fewer than k: every visible logit is listed
    }
    return prefix;
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
    if (n > kTopkCollect) {
        // Too many logits reach tau: the k-th key itself, then exactly the
        // keys at or above it.
        const int ebeg = vbeg * EPV, eend = vend * EPV < V ? vend * EPV : V;
        const uint64_t kth = radix_kth<T, BLOCK>(rp, ebeg, eend, k,
                                                 reinterpret_cast<unsigned int *>(sh_key), tid);
        if (tid == 0) sh_n = 0;
        __syncthreads();
        for (int i = ebeg + tid; i < eend; i += BLOCK) {
            const float x = E::at(rp, i);
            const uint64_t key = topk_key(x, i);
            if (x > kMasked && key >= kth) {
                const int o = atomicAdd(&sh_n, 1);
                if (o < kTopkCollect) sh_key[o] = key;
            }
        }
        __syncthreads();
        n = sh_n;
    }

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
