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
// error, the merge computes the normalisers of the beams concerned again in
// double and places the continuations anew, so the choice is that of the exact
// scores.
#pragma once

#include "sv_topk.hpp"

namespace sv {

constexpr int kMaxBeams = 32;
constexpr int kMaxBeamOut = 64;

// Bound on the error of the difference of two beams' log-normalisers.  Each
// is off by at most (V <= 2^20, mean exponent |d| <= 20): four half steps of
// |d| ln 2 (difference, log2(e), its division by T, product), one step of exp2
// and half a step for each of at most 60 additions a term goes through:
// (4 * 20 * 0.7 + 2 + 60) * 2^-24 = 7.1e-6.
constexpr double kNearBeam = 1.5e-5;

struct BeamArgs {
    const void *base;                // logits, [B][W] rows
    const float *scores;             // [B][W]
    const uint8_t *ended;            // [B][W] or null
    const unsigned long long *list;  // [B][W][segs][n]
    const double *seg_lse;           // [B][W][segs]
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
};

// ln sum e^(l/T) of a row in double, given its largest visible logit M.
template <typename T, int BLOCK>
__device__ __attribute__((noinline)) double exact_normaliser(const T *row, int V, float M,
                                                            double inv_t, double *sh, int tid) {
    double s = 0.0;
    for (int i = tid; i < V; i += BLOCK) {
        const float x = Elem<T>::at(row, i);
        if (x > kMasked) s += exp((static_cast<double>(x) - static_cast<double>(M)) * inv_t);
    }
    s = wave_sum_f64(s);
    __syncthreads();  // sh is free
    if ((tid & (kWave - 1)) == 0) sh[tid / kWave] = s;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < BLOCK / kWave; ++w) t += sh[w];
    return static_cast<double>(M) * inv_t + log(t);
}

// One workgroup per sequence.
template <typename T, int BLOCK>
__global__ __launch_bounds__(BLOCK) void beam_merge_kernel(BeamArgs a) {
    extern __shared__ __align__(16) unsigned char dyn[];
    double *key = reinterpret_cast<double *>(dyn);  // [W][segs][n], -inf: no continuation
    __shared__ double sh_lse[kMaxBeams], sh_red[BLOCK / kWave];
    __shared__ int sh_pick[kMaxBeamOut];
    __shared__ unsigned int sh_near[(4096 + 31) / 32];
    __shared__ unsigned int sh_again;  // beams whose normaliser is needed in double
    __shared__ int sh_count;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = tid / kWave;
    const int b = blockIdx.x, W = a.W, n = a.n, segs = a.segs;
    const int per = segs * n, total = W * per;
    const unsigned long long *list = a.list + static_cast<int64_t>(b) * total;
    const double inf = __builtin_inf();

    if (tid == 0) {
        sh_again = 0;
        sh_count = 0;
    }
    for (int i = tid; i < (total + 31) / 32; i += BLOCK) sh_near[i] = 0;
    for (int w = wv; w < W; w += BLOCK / kWave) {
        const double x = lane < segs ? a.seg_lse[(static_cast<int64_t>(b) * W + w) * segs + lane]
                                     : -inf;
        const double l = wave_log_sum(x, lane, segs);
        if (lane == 0) sh_lse[w] = l;
    }
    __syncthreads();

    // Scores of the continuations.  A beam that has ended continues once, as
    // it is; a beam of score -inf (or NaN) has none.
    auto score_all = [&]() {
        for (int i = tid; i < total; i += BLOCK) {
            const int w = i / per;
            const int64_t bw = static_cast<int64_t>(b) * W + w;
            const float s = a.scores[bw];
            double x = -inf;
            if (s > -__builtin_inff()) {
                if (a.ended && a.ended[bw])
                    x = i == w * per ? static_cast<double>(s) : -inf;
                else if (const unsigned long long k = list[i])
                    x = static_cast<double>(s) +
                        (static_cast<double>(key_value(k)) * a.inv_t - sh_lse[w]);
            }
            key[i] = x;
        }
    };

    // Places by bisection in every other list.  tol > 0 also notes the
    // continuations within tol of one of another beam.
    auto place_all = [&](double tol) {
        for (int i = tid; i < total; i += BLOCK) {
            const double x = key[i];
            if (!(x > -inf)) continue;
            const int own = i / n, w = i / per;
            int rank = i - own * n;
            bool near = false;
            for (int l = 0; l < W * segs; ++l) {
                if (l == own) continue;
                const double *o = key + l * n;
                const bool other = l / segs != w;
                const double slack = other ? tol : 0.0;
                int lo = 0, hi = n;  // entries above x + slack
                while (lo < hi) {
                    const int mid = (lo + hi) / 2;
                    if (o[mid] > x + slack)
                        lo = mid + 1;
                    else
                        hi = mid;
                }
                rank += lo;
                for (; lo < n && o[lo] >= x - slack && o[lo] > -inf; ++lo) {
                    near = near || (other && tol > 0.0);
                    rank += o[lo] > x || (o[lo] == x && l < own);
                }
            }
            if (near) atomicOr(&sh_near[i >> 5], 1u << (i & 31));
            atomicAdd(&sh_count, 1);
            if (rank < n) sh_pick[rank] = i;
        }
    };

    score_all();
    __syncthreads();
    place_all(kNearBeam);
    __syncthreads();
    // A near continuation matters when it is chosen or could be.
    const double worst = sh_count >= n ? key[sh_pick[n - 1]] : -inf;
    for (int i = tid; i < total; i += BLOCK) {
        if (!((sh_near[i >> 5] >> (i & 31)) & 1u) || key[i] < worst - kNearBeam) continue;
        const int w = i / per;
        if (!(a.ended && a.ended[static_cast<int64_t>(b) * W + w])) atomicOr(&sh_again, 1u << w);
    }
    __syncthreads();
    unsigned int again = sh_again;
    if (again) {
        while (again) {
            const int w = __ffs(static_cast<int>(again)) - 1;
            again &= again - 1;
            const int64_t bw = static_cast<int64_t>(b) * W + w;
            float M = -__builtin_inff();
            for (int s = 0; s < segs; ++s) {
                const unsigned long long k = list[w * per + s * n];
                if (k) M = fmaxf(M, key_value(k));
            }
            const double l = exact_normaliser<T, BLOCK>(
                static_cast<const T *>(a.base) + bw * a.stride, a.V, M, a.inv_t, sh_red, tid);
            if (tid == 0) sh_lse[w] = l;
        }
        if (tid == 0) sh_count = 0;
        __syncthreads();
        score_all();
        __syncthreads();
        place_all(0.0);
        __syncthreads();
    }

    const int count = sh_count;
    for (int i = tid; i < n; i += BLOCK) {
        const int64_t o = static_cast<int64_t>(b) * n + i;
        if (i >= count) {
            a.out_scores[o] = -__builtin_inff();
            a.parents[o] = -1;
            a.tokens[o] = -1;
            if (a.ended_out) a.ended_out[o] = 0;
            continue;
        }
        const int at = sh_pick[i], w = at / per;
        const bool over = a.ended && a.ended[static_cast<int64_t>(b) * W + w];
        const int token = over ? a.eos : key_id(list[at]);
        a.out_scores[o] = static_cast<float>(key[at]);
        a.parents[o] = w;
        a.tokens[o] = token;
        if (a.ended_out) a.ended_out[o] = over || token == a.eos;
    }
}

// ---------------------------------------------------------------------------
// Reordering of states: dst[b][i] = src[b][parents[b][i]], the used positions
// of every segment.  A thread takes one unit (16, 4 or 1 bytes) of a sequence,
// reads it from all the parents and only then writes the rows, so a state may
// be reordered in place: no other thread touches that unit.
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

// GROUP rows are in flight at once; in place that is all of them (n <= GROUP).
template <int BYTES, int GROUP, int BLOCK, int UNROLL>
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
    const int64_t seg_bytes = s.positions * s.pos_bytes;
    const int64_t beam_bytes = seg_bytes * s.segments;
    const char *src = s.src + static_cast<int64_t>(b) * a.W * beam_bytes + seg * seg_bytes;
    char *dst = s.dst + static_cast<int64_t>(b) * a.n * beam_bytes + seg * seg_bytes;
    const bool in_place = s.src == s.dst;
    const int32_t *par = a.parents + static_cast<int64_t>(b) * a.n;
    int64_t i = static_cast<int64_t>(chunk) * (BLOCK * UNROLL) + threadIdx.x;
    for (int u = 0; u < UNROLL; ++u, i += BLOCK) {
        if (i >= units) return;
        for (int g = 0; g < a.n; g += GROUP) {
            U v[GROUP];
#pragma unroll
            for (int k = 0; k < GROUP; ++k) {
                const int p = g + k < a.n ? par[g + k] : -1;
                v[k] = U{};
                if (p >= 0 && p < a.W && !(in_place && p == g + k))
                    v[k] = reinterpret_cast<const U *>(src + p * beam_bytes)[i];
            }
#pragma unroll
            for (int k = 0; k < GROUP; ++k) {
                const int p = g + k < a.n ? par[g + k] : -1;
                if (p >= 0 && p < a.W && !(in_place && p == g + k))
                    reinterpret_cast<U *>(dst + (g + k) * beam_bytes)[i] = v[k];
            }
        }
    }
}

}  // namespace sv
