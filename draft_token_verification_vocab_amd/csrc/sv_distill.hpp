// sv_distill.hpp -- distillation of a draft (student) model from a teacher's
// listed top logits: the loss per row and its gradient.
//
// With z = s/T, q = softmax(z) over the whole vocabulary, and the list's
// masses p_i = e^(t_i/T - L) (L the teacher's log-normaliser, or the list's
// own), P = sum p_i, r = max(0, 1 - P) the teacher's mass outside the list
// (0 with the list's own normaliser) and rho = sum of q outside the list:
//   loss      = sum_i p_i (ln p_i - ln q_i) + r (ln r - ln rho)
//   dloss/ds_j = (1/T) (q_j (P + r) - sum of p_i listed at j)   j in the list
//              = (1/T) q_j (P + r - r / rho)                   j outside it
// rho is summed over the entries outside the list themselves, with a maximum
// of their own: formed as one minus the list's share it would vanish in
// rounding, or the entries underflow, as soon as the student is sure.  So the
// stream leaves the listed entries out, and the list (at most 128 entries) is
// settled in double by one wave.
//
// Outside the list the gradient is one factor per row times 2^((s_j - M) c),
// M the largest logit outside the list; that factor's difference is taken in
// double.
#pragma once

#include "sv_stream.hpp"
#include "sv_topk.hpp"

namespace sv {

constexpr int kDistillMax = kTopkMax;         // longest list
constexpr int kListMapVocab = 1 << 18;        // ids the list's bitmap in LDS covers

// What the gradient needs of a row's forward pass.  Normalisers are kept
// relative to a logit, so that they lose nothing however large l/T is.
struct DistillRow {
    double lse;    // student: ln sum e^((s - top)/T)
    double norm;   // teacher: ln p_i = (t_i - t_top)/T - norm
    double mass;   // P + r, or -1 for a row that is left out
    double coef;   // (P + r) e^((m - top)/T - lse) - r / sum_{outside} 2^((s - m) c)
    float top;     // the largest of the student's logits
    float t_top;   // the largest listed logit (0 with the teacher's normaliser)
    float m;       // M, the largest logit outside the list
    int32_t pad_;
};
static_assert(sizeof(DistillRow) == 48, "spec_distill_state_bytes");

// ln q and ln p of a logit, in double.
__device__ __forceinline__ double log_q(const DistillRow &r, float s, double inv_t) {
    return (static_cast<double>(s) - static_cast<double>(r.top)) * inv_t - r.lse;
}
__device__ __forceinline__ double log_p(const DistillRow &r, float t, double inv_t) {
    return (static_cast<double>(t) - static_cast<double>(r.t_top)) * inv_t - r.norm;
}

struct DistillArgs {
    const void *student;
    const int32_t *ids;       // [rows][k]
    const float *logits;      // [rows][k]
    const float *lse;         // [rows] or null: the list's own normaliser
    const uint8_t *keep;      // [rows] or null
    const float *grad_loss;   // [rows] or null (= 1)
    float *loss;              // [rows]
    DistillRow *state;        // [rows] or null
    void *grad;               // rows of row_stride, or null
    int64_t stride;
    int32_t V;
    int32_t k;
    float c;                  // log2(e) / T
    int32_t seg_vecs;         // gradient pass: vectors per workgroup
    double inv_t;
};

// Four bytes of two bfloat16, rounded to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    const bf2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
    uint32_t r;
    __builtin_memcpy(&r, &v, 4);
    return r;
}

template <typename T>
struct GradOut;
template <>
struct GradOut<uint16_t> {
    __device__ static uint4 pack(const float *x) {
        return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                          pack_bf16(x[6], x[7]));
    }
    __device__ static uint16_t one(float x) { return static_cast<uint16_t>(pack_bf16(x, 0.f)); }
};
template <>
struct GradOut<float> {
    __device__ static uint4 pack(const float *x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
    __device__ static float one(float x) { return x; }
};

__device__ __forceinline__ void store_stream(uint4 *p, const uint4 &v) {
    const v4u32 r = {v.x, v.y, v.z, v.w};
    __builtin_nontemporal_store(r, reinterpret_cast<v4u32 *>(p));
}

// Gradients of a vector outside the list: G * 2^((x - M) c), 0 where masked.
template <typename T>
__device__ __forceinline__ uint4 outside_grad(const uint4 &v, float M, float c, float G) {
    constexpr int EPV = Elem<T>::kPerVec;
    float x[EPV];
    Elem<T>::unpack(v, x);
#pragma unroll
    for (int e = 0; e < EPV; ++e)
        x[e] = G * hw_exp2((fmaxf(x[e], 2.0f * kMasked) - M) * c);  // a NaN becomes masked
    return GradOut<T>::pack(x);
}

// The list of a row in LDS.
struct ListShared {
    int id[kDistillMax];       // -1: not a listed entry
    float s[kDistillMax];      // the student's logit there (-inf when masked)
    float t[kDistillMax];      // the teacher's
    double p[kDistillMax];     // masses
    float g[kDistillMax];      // gradients (the first of equal ids)
    int first[kDistillMax];    // nonzero: the first entry with this id
    int dup;                   // some id is listed twice
};

// One entry of a row's list on its way to LDS, in steps, so that its loads lie
// among the row's without a wait of their own.
struct ListEntry {
    int id = -1;     // -1: not a listed entry
    float t = 0.f;
    __device__ __forceinline__ void fetch(const DistillArgs &a, int64_t row, int i) {
        id = a.ids[row * a.k + i];
        t = a.logits[row * a.k + i];
    }
    __device__ __forceinline__ void put(const DistillArgs &a, ListShared &l, int i) {
        if (!(id >= 0 && id < a.V && t > kMasked)) id = -1;
        l.id[i] = id;
        l.t[i] = t;
        l.first[i] = id >= 0;
    }
    // The student's logit there, to be put in l.s by the same thread.
    template <typename T>
    __device__ __forceinline__ float gather(const T *rp) const {
        return id >= 0 ? Elem<T>::at(rp, id) : 0.f;
    }
    __device__ __forceinline__ static float seen(float s) {
        return s > kMasked ? s : -__builtin_inff();
    }
};

// first[] when some id is listed twice; call by threads i < k.
__device__ __forceinline__ void mark_first(int i, ListShared &l) {
    for (int j = 0; j < i; ++j)
        if (l.id[j] == l.id[i]) l.first[i] = 0;
}

// Gradient at the listed id i (the first of equal ids): its own share less the
// teacher's masses listed there.
__device__ __forceinline__ float listed_grad(int i, int k, const ListShared &l,
                                             const DistillRow &r, double inv_t, double g) {
    double p = l.p[i];
    if (l.dup)
        for (int j = i + 1; j < k; ++j)
            if (l.id[j] == l.id[i]) p += l.p[j];
    return static_cast<float>((exp_f64(log_q(r, l.s[i], inv_t)) * r.mass - p) * inv_t * g);
}

// One wave: the row's loss and gradient state from the list and the sum S of
// 2^((s - M) c) outside it (M <= kMasked: nothing visible there).
__device__ __forceinline__ DistillRow settle_row(const DistillArgs &a, int64_t row, int lane,
                                                 ListShared &l, float M, double S, float *loss) {
    const float inf = __builtin_inff();
    const double it = a.inv_t;
    const bool outside = M > kMasked;
    float t[2], s[2];
    bool first[2];
    float tm = -inf, sm = outside ? M : -inf;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = lane + h * kWave;
        const bool in = i < a.k && l.id[i] >= 0;
        t[h] = in ? l.t[i] : -inf;
        s[h] = in ? l.s[i] : -inf;
        first[h] = in && l.first[i];
        tm = fmaxf(tm, t[h]);
        sm = fmaxf(sm, s[h]);
    }
    tm = wave_max_f32(tm);
    sm = wave_max_f32(sm);
    DistillRow r{};
    r.mass = -1.0;
    r.m = M;
    *loss = 0.f;
    if (!(tm > -inf) || !(sm > -inf)) return r;  // nothing listed, or nothing visible
    r.top = sm;
    r.t_top = a.lse ? 0.f : tm;
    double zs = 0.0, ts = 0.0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (first[h]) zs += exp_f64(log_q(r, s[h], it));
        ts += exp_f64((static_cast<double>(t[h]) - static_cast<double>(tm)) * it);
    }
    // log_q and log_p of the row so far are without their normalisers (0)
    const double rest = outside ? log_q(r, M, it) + log_f64(S) : -static_cast<double>(inf);
    const double total = wave_sum_f64(zs) + (outside ? exp_f64(rest) : 0.0);
    r.lse = log_f64(total);
    r.norm = a.lse ? static_cast<double>(a.lse[row]) : log_f64(wave_sum_f64(ts));
    double ps = 0.0, ls = 0.0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const double lp = log_p(r, t[h], it), p = exp_f64(lp);
        if (lane + h * kWave < a.k) l.p[lane + h * kWave] = p;
        ps += p;
        if (p > 0.0) ls += p * (lp - log_q(r, s[h], it));
    }
    const double P = wave_sum_f64(ps);
    const double left = a.lse && outside ? fmax(0.0, 1.0 - P) : 0.0;
    double total_loss = wave_sum_f64(ls);
    if (left > 0.0) total_loss += left * (log_f64(left) - (rest - r.lse));
    *loss = static_cast<float>(total_loss);
    r.mass = P + left;
    r.coef = outside ? (r.mass * exp_f64(rest - r.lse) - left) / S : 0.0;
    return r;
}

// What a workgroup holds of its row besides the list.  The bitmap of listed ids
// (one bit per id, V <= kListMapVocab) is dynamic.
template <int BLOCK>
struct DistillShared {
    ListShared list;
    unsigned long long chunks[BLOCK];  // chunks (mod 64) of a thread with a listed entry
    uint32_t wm[BLOCK / kWave];
    double s[BLOCK / kWave];
    DistillRow row;
};

// Puts a row's list (entry tid of it in the threads below k) in LDS, with the
// bitmap and each thread's chunks (of UNROLL vectors a thread) that hold a
// listed entry.  Returns the thread's.  The student's logits there (l.s) follow.
template <typename T, int BLOCK, int UNROLL>
__device__ __forceinline__ unsigned long long prepare_list(const DistillArgs &a,
                                                           ListEntry &entry, int tid,
                                                           DistillShared<BLOCK> &sh,
                                                           uint32_t *map) {
    constexpr int EPV = Elem<T>::kPerVec;
    constexpr int kChunk = UNROLL * BLOCK;
    ListShared &list = sh.list;
    const bool mapped = a.V <= kListMapVocab;
    sh.chunks[tid] = 0;
    if (mapped)
        for (int i = tid; i < (a.V + 31) / 32; i += BLOCK) map[i] = 0;
    if (tid == 0) list.dup = 0;
    if (tid < a.k) entry.put(a, list, tid);
    __syncthreads();
    if (tid < a.k && list.id[tid] >= 0) {
        const int id = list.id[tid];
        const int w = id / EPV, it = w / kChunk, owner = (w % kChunk) % BLOCK;
        atomicOr(&sh.chunks[owner], 1ull << (it & 63));
        bool again = false;
        if (mapped)
            again = (atomicOr(&map[id >> 5], 1u << (id & 31)) >> (id & 31)) & 1u;
        else
            for (int j = 0; j < tid; ++j) again = again || list.id[j] == id;
        if (again) list.dup = 1;
    }
    __syncthreads();
    if (list.dup && tid < a.k && list.id[tid] >= 0) mark_first(tid, list);
    return sh.chunks[tid];
}

// Masks the listed entries among a vector's.
template <typename T>
__device__ __forceinline__ void leave_out_listed(const DistillArgs &a, const ListShared &list,
                                                 const uint32_t *map, int vi, int nvec,
                                                 float *x) {
    constexpr int EPV = Elem<T>::kPerVec;
    uint32_t bits = 0;
    if (a.V <= kListMapVocab) {
        if (vi < nvec) bits = map[vi * EPV >> 5] >> (vi * EPV & 31);
    } else {
        for (int j = 0; j < a.k; ++j) {
            const int e = list.id[j] - vi * EPV;
            if (e >= 0 && e < EPV) bits |= 1u << e;
        }
    }
#pragma unroll
    for (int e = 0; e < EPV; ++e)
        if ((bits >> e) & 1u) x[e] = 2.0f * kMasked;
}

// The row's results from the threads' sums, in sh.row; ends with a barrier.
template <int BLOCK>
__device__ __forceinline__ void finish_row(const DistillArgs &a, int64_t row,
                                           const OnlineSum &acc, int tid,
                                           DistillShared<BLOCK> &sh) {
    constexpr int NW = BLOCK / kWave;
    const int lane = tid & (kWave - 1), wv = tid / kWave;
    const uint32_t wm = wave_max_u32(ordered_bits(acc.m + 0.0f));
    if (lane == 0) sh.wm[wv] = wm;
    __syncthreads();
    uint32_t bm = sh.wm[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) bm = sh.wm[w] > bm ? sh.wm[w] : bm;
    const float M = from_ordered_bits(bm);
    const double ws = wave_sum_f64(acc.at(M, a.c));
    if (lane == 0) sh.s[wv] = ws;
    __syncthreads();
    if (wv == 0) {
        double S = 0.0;
#pragma unroll
        for (int w = 0; w < NW; ++w) S += sh.s[w];
        float loss;
        const DistillRow r =
            settle_row(a, row, lane, sh.list, M,
                       S * exp2_f64(-OnlineSum::above_max(M, a.c)), &loss);
        if (lane == 0) {
            sh.row = r;
            a.loss[row] = loss;
            if (a.state) a.state[row] = r;
        }
    }
    __syncthreads();
}

// A row that is left out, or whose loss has no gradient.
__device__ __forceinline__ void skip_row(const DistillArgs &a, int64_t row) {
    DistillRow r{};
    r.mass = -1.0;
    a.loss[row] = 0.f;
    if (a.state) a.state[row] = r;
}

template <int BLOCK>
__device__ __forceinline__ void zero_vectors(uint4 *out, int from, int to, int tid) {
    for (int i = from + tid; i < to; i += BLOCK) store_stream(out + i, make_uint4(0, 0, 0, 0));
}

// The gradients of the listed entries, over what the stream wrote there, once
// that is written.
template <typename T>
__device__ __forceinline__ void patch_listed(const DistillArgs &a, const DistillRow &r, double g,
                                             int tid, const ListShared &list, T *gp) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid < a.k && list.id[tid] >= 0 && list.first[tid])
        gp[list.id[tid]] = GradOut<T>::one(listed_grad(tid, a.k, list, r, a.inv_t, g));
}

// The loss, a workgroup per row.  KEEP: the row is read again soon.  Bound by
// memory: 2560 rows of 152064 bfloat16 logits 117 us (6.6 TB/s, the load-only
// pass 112); with the list prepared before the first loads instead of behind
// them it took 121 to 125.
template <typename T, int BLOCK, int UNROLL, bool KEEP>
__global__ __launch_bounds__(BLOCK) void distill_rows_kernel(DistillArgs a) {
    using E = Elem<T>;
    constexpr int EPV = E::kPerVec;
    constexpr int N = UNROLL * EPV;
    extern __shared__ __align__(16) unsigned char dyn[];
    uint32_t *map = reinterpret_cast<uint32_t *>(dyn);
    __shared__ DistillShared<BLOCK> sh;

    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const T *rp = static_cast<const T *>(a.student) + row * a.stride;
    const int V = a.V;
    const int nvec = (V + EPV - 1) / EPV;
    if (a.keep && !a.keep[row]) {
        if (tid == 0) skip_row(a, row);
        return;
    }
    ListEntry entry;
    if (tid < a.k) entry.fetch(a, row, tid);
    unsigned long long mine = 0;
    float at_id = 0.f;
    OnlineSum acc(a.c);
    stream_vectors<T, BLOCK, UNROLL, KEEP>(
        rp, 0, nvec, V, tid,
        [&](const uint4 (&buf)[UNROLL], int it) {
            float x[N];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) E::unpack(buf[u], x + u * EPV);
            if ((mine >> (it & 63)) & 1ull) {
#pragma unroll
                for (int u = 0; u < UNROLL; ++u)
                    leave_out_listed<T>(a, sh.list, map, (it * UNROLL + u) * BLOCK + tid, nvec,
                                        x + u * EPV);
            }
            acc.add(x, chunk_max(x), a.c);
        },
        [&]() {
            mine = prepare_list<T, BLOCK, UNROLL>(a, entry, tid, sh, map);
            at_id = entry.gather(rp);
        });
    if (tid < a.k) sh.list.s[tid] = ListEntry::seen(at_id);
    finish_row<BLOCK>(a, row, acc, tid, sh);
}

// Loss and gradient of a row whose first BLOCK*NV vectors are read once: a
// thread holds its NV of them in registers from the read to the gradient.
// What lies beyond is read twice, the first time without the non-temporal
// hint, so that the second read comes from the last-level cache.
//
// The bound is memory: with all of the row read twice, 2048 rows of 128256
// bfloat16 logits took 245 us, the fabric's rate for their 1.6 GB.  512 threads
// at 128 registers (two workgroups per compute unit, which cover each other's
// waits) hold 12 vectors each, 38 % of such a row: 202 to 207 us, what a copy
// of the same bytes takes (8 vectors: 214, 16: 211).  In float32 they hold 8
// (2048 rows of 32000: 98 us; 12 spill: 123).  A whole row in one workgroup of
// 1024 threads, alone on its compute unit, took 257 us.  Rows of up to 4096
// vectors take 256 threads with 8 (2048 rows of 4000 bfloat16 logits: 21 us
// against 36 with 512 threads).
template <typename T, int BLOCK, int NV>
__global__ __launch_bounds__(BLOCK, 4) void distill_held_kernel(DistillArgs a) {
    using E = Elem<T>;
    constexpr int EPV = E::kPerVec;
    constexpr int UNROLL = 16 / EPV;  // 16 logits a chunk, as in the stream
    constexpr int N = UNROLL * EPV;
    constexpr int kHeld = BLOCK * NV;
    static_assert(NV % UNROLL == 0, "whole chunks");
    extern __shared__ __align__(16) unsigned char dyn[];
    uint32_t *map = reinterpret_cast<uint32_t *>(dyn);
    __shared__ DistillShared<BLOCK> sh;

    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const T *rp = static_cast<const T *>(a.student) + row * a.stride;
    T *gp = static_cast<T *>(a.grad) + row * a.stride;
    const int V = a.V;
    const int nfull = V / EPV, nvec = (V + EPV - 1) / EPV;
    const int out_vecs = static_cast<int>(a.stride / EPV);
    uint4 *out = reinterpret_cast<uint4 *>(gp);
    if (a.keep && !a.keep[row]) {
        if (tid == 0) skip_row(a, row);
        zero_vectors<BLOCK>(out, 0, out_vecs, tid);
        return;
    }
    ListEntry entry;
    if (tid < a.k) entry.fetch(a, row, tid);
    // Vector u*BLOCK + tid; past the full ones the last full one stands in
    // until the ragged vector or padding takes its place below.
    const buf_rsrc rs = make_rsrc(rp, static_cast<uint32_t>(nfull) * 16u);
    uint4 v[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        if (u * BLOCK < nfull) {
            const int vi = u * BLOCK + tid;
            v[u] = load_row_buf<false>(rs, static_cast<uint32_t>(vi < nfull ? vi : nfull - 1) * 16u,
                                       0u);
        }
    }
    const unsigned long long mine = prepare_list<T, BLOCK, UNROLL>(a, entry, tid, sh, map);
    const float at_id = entry.gather(rp);
    const uint32_t pad = E::pad_word();
    OnlineSum acc(a.c);
#pragma unroll
    for (int it = 0; it < NV / UNROLL; ++it) {
        if (it * UNROLL * BLOCK >= nvec) break;
        float x[N];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int w = it * UNROLL + u, vi = w * BLOCK + tid;
            if ((w + 1) * BLOCK > nfull) {  // the same for every thread
                if (vi >= nvec || w * BLOCK >= nvec)
                    v[w] = make_uint4(pad, pad, pad, pad);
                else if (vi >= nfull)
                    v[w] = E::partial(rp, nfull, V);
            }
            E::unpack(v[w], x + u * EPV);
            if ((mine >> it) & 1ull) leave_out_listed<T>(a, sh.list, map, vi, nvec, x + u * EPV);
        }
        acc.add(x, chunk_max(x), a.c);
    }
    if (nvec > kHeld) {
        stream_vectors<T, BLOCK, UNROLL, true>(rp, kHeld, nvec, V, tid,
                                               [&](const uint4 (&buf)[UNROLL], int it) {
            it += NV / UNROLL;
            float x[N];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) E::unpack(buf[u], x + u * EPV);
            if ((mine >> (it & 63)) & 1ull) {
#pragma unroll
                for (int u = 0; u < UNROLL; ++u)
                    leave_out_listed<T>(a, sh.list, map, (it * UNROLL + u) * BLOCK + tid, nvec,
                                        x + u * EPV);
            }
            acc.add(x, chunk_max(x), a.c);
        });
    }
    if (tid < a.k) sh.list.s[tid] = ListEntry::seen(at_id);
    finish_row<BLOCK>(a, row, acc, tid, sh);
    const DistillRow r = sh.row;
    if (r.mass < 0.0) {
        zero_vectors<BLOCK>(out, 0, out_vecs, tid);
        return;
    }
    const double g = a.grad_loss ? static_cast<double>(a.grad_loss[row]) : 1.0;
    const float G = static_cast<float>(r.coef * a.inv_t * g);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int vi = u * BLOCK + tid;
        if (vi < nvec) store_stream(out + vi, outside_grad<T>(v[u], r.m, a.c, G));
    }
    if (nvec > kHeld) {
        stream_vectors<T, BLOCK, UNROLL>(rp, kHeld, nvec, V, tid,
                                         [&](const uint4 (&buf)[UNROLL], int it) {
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int vi = kHeld + (it * UNROLL + u) * BLOCK + tid;
                if (vi < nvec) store_stream(out + vi, outside_grad<T>(buf[u], r.m, a.c, G));
            }
        });
    }
    zero_vectors<BLOCK>(out, nvec, out_vecs, tid);
    patch_listed<T>(a, r, g, tid, sh.list, gp);
}

// The gradient alone, from the forward pass's state: every workgroup writes
// seg_vecs vectors of a row.  Bound by memory: 999 rows of 32000 floats (800
// kept) 38 us, 102 MB read, most of it from the last-level cache, and 128 MB
// written (6.1 TB/s).
template <typename T, int BLOCK, int UNROLL>
__global__ __launch_bounds__(BLOCK) void distill_grad_kernel(DistillArgs a, int32_t segs) {
    constexpr int EPV = Elem<T>::kPerVec;
    __shared__ ListShared list;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / segs;
    const int seg = static_cast<int>(blockIdx.x - row * segs);
    const T *rp = static_cast<const T *>(a.student) + row * a.stride;
    T *gp = static_cast<T *>(a.grad) + row * a.stride;
    const int V = a.V;
    const int nvec = (V + EPV - 1) / EPV;
    const int out_vecs = static_cast<int>(a.stride / EPV);
    const int vbeg = seg * a.seg_vecs;
    const int vend = vbeg + a.seg_vecs < out_vecs ? vbeg + a.seg_vecs : out_vecs;
    uint4 *out = reinterpret_cast<uint4 *>(gp);
    const DistillRow r = a.state[row];
    if (r.mass < 0.0) {
        zero_vectors<BLOCK>(out, vbeg, vend, tid);
        return;
    }
    if (tid == 0) list.dup = 0;
    if (tid < a.k) {
        ListEntry entry;
        entry.fetch(a, row, tid);
        entry.put(a, list, tid);
        list.s[tid] = ListEntry::seen(entry.gather(rp));
        list.p[tid] = list.id[tid] >= 0
                          ? exp_f64(log_p(r, list.t[tid], a.inv_t))
                          : 0.0;
    }
    __syncthreads();
    if (tid < a.k && list.id[tid] >= 0) {
        for (int j = 0; j < tid; ++j)
            if (list.id[j] == list.id[tid]) {
                list.first[tid] = 0;
                list.dup = 1;
            }
    }
    __syncthreads();
    const double g = a.grad_loss ? static_cast<double>(a.grad_loss[row]) : 1.0;
    const float G = static_cast<float>(r.coef * a.inv_t * g);
    const int vlast = vend < nvec ? vend : nvec;
    if (vbeg < vlast)
        stream_vectors<T, BLOCK, UNROLL>(rp, vbeg, vlast, V, tid,
                                         [&](const uint4 (&buf)[UNROLL], int it) {
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int vi = vbeg + (it * UNROLL + u) * BLOCK + tid;
                if (vi < vlast) store_stream(out + vi, outside_grad<T>(buf[u], r.m, a.c, G));
            }
        });
    zero_vectors<BLOCK>(out, vbeg > nvec ? vbeg : nvec, vend, tid);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid < a.k && list.id[tid] >= 0 && list.first[tid]) {
        const int w = list.id[tid] / EPV;
        if (w >= vbeg && w < vend)
            gp[list.id[tid]] =
                GradOut<T>::one(listed_grad(tid, a.k, list, r, a.inv_t, g));
    }
}

}  // namespace sv
