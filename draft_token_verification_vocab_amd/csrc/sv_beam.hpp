// sv_beam.hpp -- one step of beam search: the best continuations of a
// sequence's beams over beams and vocabulary, and the reordering of the beams'
// states by the chosen parents.
//
// A continuation of beam w by token x has the score
//   score_w + l_wx / T - ln sum_x' e^(l_wx' / T).
// Within a beam the order is that of the logits, so its best num_out logits
// (a listing, sv_topk.hpp) hold every continuation that can be chosen.  The
// merge then compares continuations of different beams, in double.
//
// The listing's log-normalisers come from float sums.  Where two continuations
// of different beams that compete for a place lie closer than those sums'
// error bound, the merge computes the normalisers of the beams concerned again in
// double and places the continuations anew, so the choice is that of the exact
// scores.
#pragma once

#include "sv_topk.hpp"

namespace sv {

constexpr int kMaxBeams = 32;
constexpr int kMaxBeamOut = 64;

// Keys one merge takes: beams x segments x num_out.
constexpr int kMaxBeamKeys = 512;

struct BeamArgs {
    const void *base;                // logits, [B][W] rows
    const float *scores;             // [B][W]
    const uint8_t *ended;            // [B][W] or null
    const unsigned long long *list;  // [B][W][segs][n]
    const double *seg_lse;           // [B][W][segs], relative to the segment's maximum
    float *out_scores;               // [B][n]
    int32_t *parents;                // [B][n]
    int32_t *tokens;                 // [B][n]
    uint8_t *ended_out;              // [B][n] or null
    int64_t stride;
    int32_t V;
    int32_t W;
    int32_t n;
    int32_t segs;
    int32_t eos;
    int32_t pad_;
    double inv_t;
    double near;  // scores of two beams closer than this are compared exactly
};

// ln sum e^((l - M)/T) of a row in double, M its largest visible logit.  A
// term's exponent is i + k/64 + f/64 with |f| <= 1/2: 2^(k/64) from a table of
// 64 doubles times the Taylor series of 2^(f/64) to the fifth degree, whose next
// term is below 2^-54 (with 32 doubles it would be 2^-48.7, always to one side,
// in the same time).  Masked logits count 2^-1000 beside the maximum's 1.  Bound
// by issue of double-precision instructions: 25 us for 152064 bfloat16 logits, 27
// in float32 (31 and 33 with the series of twelve terms that needs no table; the
// next vector's load ahead of the sums gained nothing).
template <typename T, int BLOCK>
__device__ __attribute__((noinline)) double exact_normaliser(const T *row, int V, float M,
                                                            double inv_t, double *sh, int tid) {
    using E = Elem<T>;
    constexpr int EPV = E::kPerVec;
    __shared__ double sh_pow[64];
    const int nvec = (V + EPV - 1) / EPV;
    const double c64 = inv_t * kLog2eD * 64.0;
    const double deepest = -64000.0 / c64;  // below: 2^-1000, as good as 0
    const double top = static_cast<double>(M);
    constexpr double kRound = 0x1.8p52;  // leaves the integer in the low word
    constexpr double u = kLn2 / 64.0;
    constexpr double c2 = u * u / 2.0, c3 = c2 * u / 3.0, c4 = c3 * u / 4.0, c5 = c4 * u / 5.0;
    __syncthreads();  // the table of the row before is read no more
    if (tid < 64) sh_pow[tid] = exp2_f64(tid / 64.0);
    __syncthreads();
    double s = 0.0;
    for (int i = tid; i < nvec; i += BLOCK) {
        const uint4 v = (i + 1) * EPV <= V ? reinterpret_cast<const uint4 *>(row)[i]
                                           : E::partial(row, i, V);
        float x[EPV];
        E::unpack(v, x);
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
            const float l = x[e] > kMasked ? x[e] : -__builtin_inff();
            const double d = fmax(static_cast<double>(l) - top, deepest);
            const double y = fma(d, c64, kRound);
            const double f = fma(d, c64, kRound - y);
            const int n = __double2loint(y);
            double p = fma(c5, f, c4);
            p = fma(p, f, c3);
            p = fma(p, f, c2);
            p = fma(p, f, u);
            p = fma(p, f, 1.0) * sh_pow[n & 63];
            s += __hiloint2double(__double2hiint(p) + ((n & ~63) << 14), __double2loint(p));
        }
    }
    s = wave_sum_f64(s);
    __syncthreads();  // sh is free
    if ((tid & (kWave - 1)) == 0) sh[tid / kWave] = s;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < BLOCK / kWave; ++w) t += sh[w];
    return log_f64(t);
}

// One workgroup per sequence.  The segments' lists of a beam are joined first
// (whole keys, counted); then every continuation's place among the other
// beams' sorted scores is found by bisection, by as many lanes as there are
// for each.  Bound by latency: 3.8 us for one sequence of four beams, 5.1 for
// 128 of eight with 16 out (counting every continuation against all others took
// 7.6 there and 19 with eight segments a row: comparisons of doubles are slow).
// Two beams that nearly tie are read again, 25 us for each row of 152064 in
// double: 9 of 200 inputs of 128 sequences with eight beams had such a pair, 1 of
// 200 of 64 with four.
template <typename T, int BLOCK>
__global__ __launch_bounds__(BLOCK) void beam_merge_kernel(BeamArgs a) {
    static_assert(BLOCK >= kMaxBeamKeys, "a thread per key");
    __shared__ unsigned long long sh_in[kMaxBeamKeys];   // [W][segs][n]
    __shared__ unsigned long long sh_key[kMaxBeamKeys];  // [W][n], 0 after the last
    __shared__ double sh_score[kMaxBeamKeys];            // [W][n], -inf after the last
    // ln sum e^((l - M)/T) of each beam, M its largest logit (its first key's)
    __shared__ double sh_lse[kMaxBeams], sh_red[BLOCK / kWave];
    __shared__ float sh_prior[kMaxBeams];                // -inf: takes no part
    __shared__ int sh_ended[kMaxBeams];
    __shared__ int sh_pick[kMaxBeamOut];
    __shared__ unsigned int sh_again;  // beams whose normaliser is needed in double
    __shared__ int sh_count;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = tid / kWave;
    const int b = blockIdx.x, W = a.W, n = a.n, segs = a.segs;
    const int per = segs * n, total = W * n;
    const double inf = __builtin_inf();

    // The lists of beams that take no part, or have ended, were not written.
    if (tid < W * per) {
        const unsigned long long k = a.list[static_cast<int64_t>(b) * W * per + tid];
        (segs == 1 ? sh_key : sh_in)[tid] = k;
    }
    if (tid < W) {
        const float s = a.scores[static_cast<int64_t>(b) * W + tid];
        sh_prior[tid] = s > -__builtin_inff() ? s : -__builtin_inff();
        sh_ended[tid] = a.ended ? a.ended[static_cast<int64_t>(b) * W + tid] != 0 : 0;
    }
    if (segs == 1 && tid < W) sh_lse[tid] = a.seg_lse[static_cast<int64_t>(b) * W + tid];
    if (tid == 0) sh_again = 0;
    if (segs > 1) {
        if (tid < total) sh_key[tid] = 0;
        __syncthreads();
        for (int q = wv; q < W; q += BLOCK / kWave) {
            const bool there = lane < segs && sh_in[(q * segs + lane) * n] != 0;
            const float m = there ? key_value(sh_in[(q * segs + lane) * n]) : -__builtin_inff();
            const float M = wave_max_f32(m);
            const double e =
                there ? exp_f64((static_cast<double>(m) - static_cast<double>(M)) * a.inv_t +
                            a.seg_lse[(static_cast<int64_t>(b) * W + q) * segs + lane])
                      : 0.0;
            const double t = wave_sum_f64(e);
            if (lane == 0) sh_lse[q] = log_f64(t);
        }
        int share = 1;
        while (share < kWave && W * per * share * 2 <= BLOCK) share *= 2;
        const int at = tid / share, w = at / per;
        const unsigned long long mine = at < W * per ? sh_in[at] : 0;
        int rank = 0;
        if (mine)
#pragma unroll 4
            for (int j = tid & (share - 1); j < per; j += share)
                rank += sh_in[w * per + j] > mine;
        for (int o = 1; o < share; o *= 2) rank += __shfl_xor(rank, o, kWave);
        if (mine && (tid & (share - 1)) == 0 && rank < n) sh_key[w * n + rank] = mine;
    }
    __syncthreads();

    // Scores of the continuations, sorted within each beam.  A beam that has
    // ended continues once, as it is.
    auto score = [&]() {
        if (tid >= total) return;
        const int w = tid / n;
        const double s = static_cast<double>(sh_prior[w]);
        const unsigned long long key = sh_key[tid];
        double x = -inf;
        if (s > -inf) {
            if (sh_ended[w])
                x = tid == w * n ? s : -inf;
            else if (key)
                x = s + ((static_cast<double>(key_value(key)) -
                          static_cast<double>(key_value(sh_key[w * n]))) *
                             a.inv_t -
                         sh_lse[w]);
        }
        sh_score[tid] = x;
    };

    // Places among all continuations.  near > 0 also finds those within it of
    // a continuation of another beam; returns whether this lane's is one.
    int share = 1;
    while (share < kWave && share < W && total * share * 2 <= BLOCK) share *= 2;
    auto place = [&](double near) {
        const int at = tid / share;
        if (tid == 0) sh_count = 0;
        __syncthreads();
        const double x = at < total ? sh_score[at] : -inf;
        const int own = at / n;
        int rank = 0, close = 0;
        if (x > -inf) {
            for (int q = tid & (share - 1); q < W; q += share) {
                if (q == own) {
                    rank += at - own * n;
                    continue;
                }
                const double *o = sh_score + q * n;
                int lo = 0, hi = n;  // scores above x + near
                while (lo < hi) {
                    const int mid = (lo + hi) / 2;
                    if (o[mid] > x + near)
                        lo = mid + 1;
                    else
                        hi = mid;
                }
                rank += lo;
                for (; lo < n && o[lo] >= x - near && o[lo] > -inf; ++lo) {
                    close = 1;
                    rank += o[lo] > x || (o[lo] == x && q < own);
                }
            }
        }
        for (int o = 1; o < share; o *= 2) {
            rank += __shfl_xor(rank, o, kWave);
            close |= __shfl_xor(close, o, kWave);
        }
        const bool there = x > -inf && (tid & (share - 1)) == 0;
        if (there && rank < n) sh_pick[rank] = at;
        const uint64_t votes = __ballot(there);
        if (lane == 0 && votes) atomicAdd(&sh_count, __popcll(votes));
        __syncthreads();
        return close != 0 && there;
    };

    score();
    if (place(a.near)) {
        // a near continuation matters when it is chosen or could be
        const int at = tid / share;
        const double worst = sh_count >= n ? sh_score[sh_pick[n - 1]] : -inf;
        if (sh_score[at] >= worst - a.near && !sh_ended[at / n]) atomicOr(&sh_again, 1u << (at / n));
    }
    __syncthreads();
    unsigned int again = sh_again;
    if (again) {
        while (again) {
            const int q = __ffs(static_cast<int>(again)) - 1;
            again &= again - 1;
            const T *row = static_cast<const T *>(a.base) +
                           (static_cast<int64_t>(b) * W + q) * a.stride;
            const double l = exact_normaliser<T, BLOCK>(row, a.V, key_value(sh_key[q * n]),
                                                        a.inv_t, sh_red, tid);
            if (tid == 0) sh_lse[q] = l;
        }
        __syncthreads();
        score();
        place(0.0);
    }

    const int count = sh_count;
    if (tid < n) {
        const int64_t o = static_cast<int64_t>(b) * n + tid;
        float s = -__builtin_inff();
        int parent = -1, token = -1, over = 0;
        if (tid < count) {
            const int at = sh_pick[tid];
            parent = at / n;
            over = sh_ended[parent];
            token = over ? a.eos : key_id(sh_key[at]);
            over |= token == a.eos;
            s = static_cast<float>(sh_score[at]);
        }
        a.out_scores[o] = s;
        a.parents[o] = parent;
        a.tokens[o] = token;
        if (a.ended_out) a.ended_out[o] = static_cast<uint8_t>(over);
    }
}

// ---------------------------------------------------------------------------
// Reordering of states: dst[b][i] = src[b][parents[b][i]], the used positions
// of every segment.  A thread takes one unit (16, 4 or 1 bytes, for all states of
// a launch) of a sequence: it
// reads each parent that has children once and writes the children's rows.  In
// place it reads all the parents before it writes, and no other thread touches
// that unit, so nothing is overwritten that is still needed.  Bound by memory:
// 32 sequences of eight beams (five parents live) and 2.1 GB moved, 386 to 402 us,
// 5.3 to 5.5 TB/s, where a copy reaches 5.2; reading a parent once per child and
// without the non-temporal hint took 604 to 626.
// ---------------------------------------------------------------------------
constexpr int kMaxReorder = 32;  // states per launch

struct ReorderState {
    const char *src;
    char *dst;
    int64_t pos_bytes;   // bytes per position
    int32_t segments;    // per beam
    int32_t positions;   // allocated per segment
    int32_t chunks;      // workgroups per segment
    uint32_t first;      // first workgroup of this state
};

struct ReorderArgs {
    ReorderState st[kMaxReorder];
    const int32_t *parents;   // [B][n]
    const int32_t *lengths;   // [B] or null (= positions)
    int32_t count;
    int32_t W;
    int32_t n;
    int32_t pad_;
};

template <int BYTES>
struct ReorderUnit;
template <>
struct ReorderUnit<16> {
    using type = v4u32;
};
template <>
struct ReorderUnit<4> {
    using type = uint32_t;
};
template <>
struct ReorderUnit<1> {
    using type = uint8_t;
};

template <typename U>
__device__ __forceinline__ U load_unit(const char *p, int64_t i) {
    return __builtin_nontemporal_load(reinterpret_cast<const U *>(p) + i);
}

// GROUP parents are in flight at once; in place that is all of them (W <= GROUP).
template <int BYTES, int GROUP, int BLOCK>
__global__ __launch_bounds__(BLOCK) void beam_reorder_kernel(ReorderArgs a) {
    using U = typename ReorderUnit<BYTES>::type;
    int t = 0;
    while (t + 1 < a.count && blockIdx.x >= a.st[t + 1].first) ++t;
    const ReorderState &s = a.st[t];
    uint32_t at = blockIdx.x - s.first;
    const int chunk = static_cast<int>(at % s.chunks);
    at /= s.chunks;
    const int seg = static_cast<int>(at % s.segments);
    const int b = static_cast<int>(at / s.segments);
    const int used = a.lengths ? clamp_len(a.lengths[b], s.positions) : s.positions;
    const int64_t units = used * s.pos_bytes / BYTES;
    const int64_t i = static_cast<int64_t>(chunk) * BLOCK + threadIdx.x;
    if (i - threadIdx.x >= units) return;
    const int64_t seg_bytes = s.positions * s.pos_bytes;
    const int64_t beam_bytes = seg_bytes * s.segments;
    const char *src = s.src + static_cast<int64_t>(b) * a.W * beam_bytes + seg * seg_bytes;
    char *dst = s.dst + static_cast<int64_t>(b) * a.n * beam_bytes + seg * seg_bytes;

    // kids[w]: the rows that take parent w; in place a row that keeps its own
    // beam is not moved.
    const int lane = threadIdx.x & (kWave - 1);
    int mine = lane < a.n ? a.parents[static_cast<int64_t>(b) * a.n + lane] : -1;
    if (s.src == s.dst && mine == lane) mine = -1;
    for (int g = 0; g < a.W; g += GROUP) {
        uint64_t kids[GROUP];
#pragma unroll
        for (int k = 0; k < GROUP; ++k) kids[k] = g + k < a.W ? __ballot(mine == g + k) : 0;
        if (i >= units) continue;
        U v[GROUP];
#pragma unroll
        for (int k = 0; k < GROUP; ++k) {
            v[k] = U{};
            if (kids[k]) v[k] = load_unit<U>(src + (g + k) * beam_bytes, i);
        }
#pragma unroll
        for (int k = 0; k < GROUP; ++k) {
            for (uint64_t m = kids[k]; m; m &= m - 1) {
                const int child = __ffsll(static_cast<long long>(m)) - 1;
                __builtin_nontemporal_store(v[k],
                                            reinterpret_cast<U *>(dst + child * beam_bytes) + i);
            }
        }
    }
}

}  // namespace sv
