// sv_stream.hpp -- the walk over one logits row (or a segment of it) that the
// draft-model kernels share: a workgroup reads the row's 16-byte vectors in
// chunks of UNROLL vectors a thread, one chunk ahead of the arithmetic, and
// hands every chunk to a functor.
#pragma once

#include "sv_common.hpp"

namespace sv {

// Logits at or below this are masked: probability zero, never listed.  The
// value that replaces them where arithmetic must stay finite lies below it
// and survives a rounding to bfloat16 (it is Elem<>::pad_word).
constexpr float kMasked = kNoMax;

// A 16-byte buffer load with (KEEP = false) or without the non-temporal hint.
template <bool KEEP>
__device__ __forceinline__ uint4 load_row_buf(buf_rsrc r, uint32_t voff, uint32_t soff) {
    const v4u32 v = __builtin_amdgcn_raw_buffer_load_b128(
        r, static_cast<int>(voff), static_cast<int>(soff), KEEP ? 0 : kCachePolicyNT);
    return make_uint4(v.x, v.y, v.z, v.w);
}

// consume(buf, it): buf holds the thread's vectors of chunk `it`, vector u at
// index it*UNROLL*BLOCK + u*BLOCK + tid of the segment [vbeg, vend); vectors
// past the segment and entries past V are padding.  Threads without a vector
// in the last chunk are not called for it.
//
// The loads are the row pass's: buffer-addressed non-temporal 16-byte loads
// over the segment's full vectors, the next chunk issued before this chunk's
// arithmetic, a ragged last vector read element by element.  KEEP: without the
// non-temporal hint, for rows that are read again soon (the hint keeps them
// out of the caches).  first(): called once, after the first chunk's loads are
// issued and before any is consumed.
struct NoPrologue {
    __device__ __forceinline__ void operator()() const {}
};
template <typename T, int BLOCK, int UNROLL, bool KEEP = false, typename F,
          typename P = NoPrologue>
__device__ __forceinline__ void stream_vectors(const T *row, int vbeg, int vend, int V, int tid,
                                               F &&consume, P &&first = P{}) {
    using E = Elem<T>;
    constexpr int kChunk = UNROLL * BLOCK;
    const int nfull = V / E::kPerVec;
    const int nv = vend - vbeg;                            // vectors of the segment
    const int nf = (vend < nfull ? vend : nfull) - vbeg;   // full ones among them
    const int nit = nf / kChunk;
    const buf_rsrc rs = make_rsrc(reinterpret_cast<const uint4 *>(row) + vbeg,
                                  static_cast<uint32_t>(nf) * 16u);
    const uint32_t pad = E::pad_word();
    auto load_chunk = [&](uint4 (&buf)[UNROLL], int it) {
        const uint32_t soff = static_cast<uint32_t>(it) * (kChunk * 16u);
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
            buf[u] = load_row_buf<KEEP>(rs, static_cast<uint32_t>(tid + u * BLOCK) * 16u, soff);
    };
    // The last, partly filled chunk (index nit).
    const int v = nit * kChunk + tid;
    const bool tail = v < nv;
    auto load_tail = [&](uint4 (&buf)[UNROLL]) {
        if (!tail) return;
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int vi = v + u * BLOCK;
            buf[u] = make_uint4(pad, pad, pad, pad);
            if (vi < nf)
                buf[u] = load_row_buf<KEEP>(rs, static_cast<uint32_t>(vi) * 16u, 0u);
            else if (vi < nv)
                buf[u] = E::partial(row, nfull, V);
        }
    };
    // Two register buffers take turns: the loads of a chunk are in flight
    // while the wait for the one before it runs (a single prefetch buffer that
    // is copied over makes each wave drain its loads once a chunk).
    uint4 a[UNROLL], b[UNROLL];
    if (nit > 0) load_chunk(a, 0);
    first();
    int it = 0;
    for (; it + 3 <= nit; it += 2) {
        load_chunk(b, it + 1);
        consume(a, it);
        load_chunk(a, it + 2);
        consume(b, it + 1);
    }
    if (it + 2 == nit) {
        load_chunk(b, it + 1);
        consume(a, it);
        load_tail(a);
        consume(b, it + 1);
        if (tail) consume(a, nit);
    } else {
        load_tail(b);
        if (nit > 0) consume(a, it);
        if (tail) consume(b, nit);
    }
}

// Double-precision exponential and logarithm of the kernels' finishes.  They
// stand on every row's way to its result, in one wave; with the library's, which
// branch for every range, a listing of 2304 rows took 97.3 us instead of 96.2,
// loss and gradient of 2048 rows 214 instead of 208.
// 2^d: the Taylor series of e^(f ln 2) for the fraction f in [-1/2, 1/2], cut
// where the next term is below 2^-52.
__device__ __forceinline__ double exp2_f64(double d) {
    d = d < -1100.0 ? -1100.0 : d;  // -inf too: 0
    const double n = __builtin_rint(d);
    const double f = (d - n) * kLn2;
    double p = 1.0 / 479001600.0;  // 1 / 12!
    p = fma(p, f, 1.0 / 39916800.0);
    p = fma(p, f, 1.0 / 3628800.0);
    p = fma(p, f, 1.0 / 362880.0);
    p = fma(p, f, 1.0 / 40320.0);
    p = fma(p, f, 1.0 / 5040.0);
    p = fma(p, f, 1.0 / 720.0);
    p = fma(p, f, 1.0 / 120.0);
    p = fma(p, f, 1.0 / 24.0);
    p = fma(p, f, 1.0 / 6.0);
    p = fma(p, f, 0.5);
    p = fma(p, f, 1.0);
    p = fma(p, f, 1.0);
    return ldexp(p, static_cast<int>(n));
}
__device__ __forceinline__ double exp_f64(double x) { return exp2_f64(x * kLog2eD); }
// ln x of a normal float's size: the hardware's log2 L, off by some 1e-6, and
// the rest of ln x = L ln 2 + ln(x 2^-L) as a two-term series.
__device__ __forceinline__ double log_f64(double x) {
    const double L = static_cast<double>(hw_log2(static_cast<float>(x)));
    const double d = fma(x, exp2_f64(-L), -1.0);
    return fma(L, kLn2, d - 0.5 * d * d);
}

// One thread's running maximum m and sum of 2^(x*c - n) over the chunks it is
// given (an online softmax in base 2).  The reference n is m*c rounded up to
// an integer: a term's exponent is then one fused product, rounded once, and a
// rescaling to another reference is an exact power of two.  A chunk's terms are
// added in float, the chunks in double: that costs nothing measurable (97.1 us
// and 97.5 for 2304 rows) and halves the error that beam selection has to allow
// for.
//
// Beyond |m*c| = 2^30 neighbouring floats differ by 128 or more in the
// exponent, so only logits equal to the maximum count; there the rounding of
// m*c itself would be large, and a power of two takes the place of c that
// keeps those apart and makes m's own term exactly 1.
struct OnlineSum {
    float m = kMasked;
    float n = -kMasked;  // until a visible logit comes every term is 2^-huge = 0
    float slope;
    double s = 0.0;
    static constexpr float kFar = 0x1p30f;
    __device__ __forceinline__ explicit OnlineSum(float c) : slope(c) {}

    // x: the chunk's N logits, cm their maximum.  NaN entries count as masked.
    template <int N>
    __device__ __forceinline__ void add(const float (&x)[N], float cm, float c) {
        if (cm > m) {
            const float mc = mul_rn(cm, c);
            float to = ceilf(mc), k = c;
            if (slope != c) s = 0.0;
            if (fabsf(mc) >= kFar) {
                // 2^(31 - exponent of cm)
                k = __uint_as_float((285u - (__float_as_uint(cm) >> 23 & 255u)) << 23);
                to = cm * k;
                s = 0.0;
            }
            s = ldexp(s, static_cast<int>(n - to));
            m = cm;
            n = to;
            slope = k;
        }
        float s4[4];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float e = hw_exp2(fmaf(x[k], slope, -n));
            s4[k & 3] = k < 4 ? e : s4[k & 3] + e;
        }
        float cs = (s4[0] + s4[1]) + (s4[2] + s4[3]);
        if (!(cs == cs)) {  // a NaN entry: the chunk again without it, added alike
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float e = x[k] > kMasked ? hw_exp2(fmaf(x[k], slope, -n)) : 0.f;
                s4[k & 3] = k < 4 ? e : s4[k & 3] + e;
            }
            cs = (s4[0] + s4[1]) + (s4[2] + s4[3]);
        }
        s += static_cast<double>(cs);
    }
    // The reference that a maximum M has.
    __device__ __forceinline__ static float reference(float M, float c) {
        return ceilf(mul_rn(M, c));
    }
    // The thread's sum relative to the reference of a maximum M >= m.
    __device__ __forceinline__ double at(float M, float c) const {
        if (m == M) return s;
        return slope != c ? 0.0 : ldexp(s, static_cast<int>(n - reference(M, c)));
    }
    // The sum of the threads' at(M) is 2^above_max times the sum of
    // 2^((x - M)*c).
    __device__ __forceinline__ static double above_max(float M, float c) {
        if (fabsf(mul_rn(M, c)) >= kFar) return 0.0;
        return static_cast<double>(M) * static_cast<double>(c) -
               static_cast<double>(reference(M, c));
    }
};

// Largest float over the wave.
__device__ __forceinline__ float wave_max_f32(float x) {
    return from_ordered_bits(wave_max_u32(ordered_bits(x)));
}

// Largest of a chunk's logits in a chain of three-input maxima (NaN entries
// are passed over; a chunk of nothing else gives NaN, which no comparison takes).
template <int N>
__device__ __forceinline__ float chunk_max(const float (&x)[N]) {
    float cm = max3f(x[0], x[1], x[2]);
#pragma unroll
    for (int k = 3; k + 1 < N; k += 2) cm = max3f(cm, x[k], x[k + 1]);
    if (N % 2 == 0) cm = max3f(cm, x[N - 1], x[N - 1]);
    return cm;
}

}  // namespace sv
