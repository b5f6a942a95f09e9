// specverify_draft.hip -- host side of the draft-model calls declared in
// include/specverify.h: listing rows' top logits, distillation from such
// lists, beam selection and the reordering of beam states.  Argument validation,
// workspace layout, kernel selection and launches on the caller's stream.  No
// allocation, no synchronisation.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "specverify.h"
#include "sv_beam.hpp"
#include "sv_common.hpp"
#include "sv_distill.hpp"
#include "sv_host.hpp"
#include "sv_topk.hpp"

namespace {

using namespace sv;

// A grid's threads must stay below 2^32.
bool grid_fits(int64_t blocks, int block) {
    return blocks <= (int64_t{1} << 32) / block - 1 && blocks <= INT32_MAX;
}

// Workgroup shapes, a workgroup per row.  Long rows take the row pass's shapes.
// Rows of up to 128 KB take 256 threads: a row's fixed work (barriers, the
// list's selection or the loss) weighs more there, and more of the smaller
// workgroups share a compute unit.  2500 rows, us at 256 threads against the
// long rows' shape, top 16 (loss): 4000 bfloat16 logits 14 (14) against 39
// (30), 32000 31 (32) against 46 (42), 50264 44 (46) against 51 (51), 128256
// 101 (104) against 99 (100); 32000 float32 51 (52) against 56 (64), 50264 81
// (84) against 79 (81).  With at most a row per compute unit there is nothing to
// share it with, and rows above 32 KB take the long shape: 32 rows of 50264
// bfloat16 logits 9.1 (8.1) against 10.3 (10.6) at 256 threads, of 32000 float32
// 8.3 (8.0) against 9.2 (9.9); of 4000 bfloat16 6.1 (5.6) at 256 against 7.6
// (5.7).  Beam rows that are cut into segments take 256 too.
template <typename T>
struct LongShape;
template <>
struct LongShape<uint16_t> {
    static constexpr int block = 768, unroll = 2;
};
template <>
struct LongShape<float> {
    static constexpr int block = 512, unroll = 4;
};
constexpr int kShortBlock = 256;
constexpr int kUnits = 256;  // compute units

template <typename T>
int row_vecs(int32_t V) {
    constexpr int per = 16 / sizeof(T);
    return (V + per - 1) / per;
}

template <typename T>
bool long_shape(int64_t rows, int32_t V) {
    return row_vecs<T>(V) > (rows <= kUnits ? 2048 : 8192);
}

template <typename T, bool LSE>
void launch_topk_t(const TopkArgs &a, int64_t rows, hipStream_t st) {
    using S = LongShape<T>;
    const dim3 grid(static_cast<unsigned>(rows * a.segs));
    if (a.segs == 1 && long_shape<T>(rows, a.V))
        topk_rows_kernel<T, S::block, S::unroll, LSE><<<grid, dim3(S::block), 0, st>>>(a);
    else
        topk_rows_kernel<T, kShortBlock, S::unroll, LSE><<<grid, dim3(kShortBlock), 0, st>>>(a);
}

void launch_topk(const TopkArgs &a, int64_t rows, int32_t dtype, hipStream_t st) {
    const bool lse = a.list || a.lse;
    if (dtype == SPEC_DTYPE_BF16)
        lse ? launch_topk_t<uint16_t, true>(a, rows, st) : launch_topk_t<uint16_t, false>(a, rows, st);
    else
        lse ? launch_topk_t<float, true>(a, rows, st) : launch_topk_t<float, false>(a, rows, st);
}

TopkArgs topk_args(const void *logits, int64_t row_stride, int32_t V, int32_t dtype,
                   float temperature, int32_t k) {
    TopkArgs a{};
    a.base = logits;
    a.stride = row_stride;
    a.V = V;
    a.k = k;
    a.segs = 1;
    a.seg_vecs = dtype == SPEC_DTYPE_BF16 ? row_vecs<uint16_t>(V) : row_vecs<float>(V);
    a.c = log2e_over(temperature);
    a.inv_t = 1.0 / static_cast<double>(temperature);
    return a;
}

constexpr int32_t kMaxListVocab = 1 << 20;

// Distillation: a workgroup per row (the row pass's shapes); the gradient on
// its own is cut into segments of kGradVecs vectors.
constexpr int kGradBlock = 256;
constexpr int kGradVecs = 4096;
constexpr int kGradUnroll = 4;

spec_status check_distill(const void *student, const int32_t *ids, const float *logits,
                          const spec_distill_params *p) {
    if (!p) return SPEC_ERR_ARG;
    const spec_status s = check_logits_shape(p->vocab, p->row_stride, p->dtype, p->temperature);
    if (s != SPEC_OK) return s;
    if (p->rows < 0 || p->k < 1 || p->reserved != 0) return SPEC_ERR_ARG;
    if (p->k > kDistillMax || p->vocab > kMaxListVocab) return SPEC_ERR_UNSUPPORTED;
    if (p->rows == 0) return SPEC_OK;
    if (!student || !aligned16(student) || !ids || !logits) return SPEC_ERR_ARG;
    if (p->row_stride > INT32_MAX || p->row_stride * elem_size(p->dtype) > INT32_MAX ||
        !grid_fits(p->rows, 1024))
        return SPEC_ERR_UNSUPPORTED;
    return SPEC_OK;
}

// The gradient replaces the logits exactly, or shares no memory with them.
bool overlaps_partly(const void *student, const void *grad, const spec_distill_params *p) {
    const int64_t bytes = p->rows * p->row_stride * elem_size(p->dtype);
    const char *s = static_cast<const char *>(student), *g = static_cast<const char *>(grad);
    return s != g && s < g + bytes && g < s + bytes;
}

DistillArgs distill_args(const void *student, const int32_t *ids, const float *logits,
                         const spec_distill_params *p) {
    DistillArgs a{};
    a.student = student;
    a.ids = ids;
    a.logits = logits;
    a.stride = p->row_stride;
    a.V = p->vocab;
    a.k = p->k;
    a.c = log2e_over(p->temperature);
    a.inv_t = 1.0 / static_cast<double>(p->temperature);
    return a;
}

// Rows that are read again at once stay in the 256 MB last-level cache when
// the student's logits fit it.
constexpr int64_t kCacheBytes = int64_t{192} << 20;

size_t map_bytes(const DistillArgs &a) {
    return a.V <= kListMapVocab ? 4 * static_cast<size_t>((a.V + 31) / 32) : 0;
}

template <typename T>
void launch_loss_t(const DistillArgs &a, int64_t rows, hipStream_t st) {
    using S = LongShape<T>;
    const dim3 grid(static_cast<unsigned>(rows));
    const bool again = a.state && rows * a.V * static_cast<int64_t>(sizeof(T)) <= kCacheBytes;
    if (long_shape<T>(rows, a.V)) {
        if (again)
            distill_rows_kernel<T, S::block, S::unroll, true>
                <<<grid, dim3(S::block), map_bytes(a), st>>>(a);
        else
            distill_rows_kernel<T, S::block, S::unroll, false>
                <<<grid, dim3(S::block), map_bytes(a), st>>>(a);
    } else {
        if (again)
            distill_rows_kernel<T, kShortBlock, S::unroll, true>
                <<<grid, dim3(kShortBlock), map_bytes(a), st>>>(a);
        else
            distill_rows_kernel<T, kShortBlock, S::unroll, false>
                <<<grid, dim3(kShortBlock), map_bytes(a), st>>>(a);
    }
}

// With at most a row per compute unit, 1024 threads share the one row (us against
// the shapes below: one row of 32000 bfloat16 logits 9.1 to 12.2, 250 rows of
// 128256 29.4 to 31.2, 32 rows of 32000 float32 10.3 to 11.9).
template <typename T>
void launch_step_t(const DistillArgs &a, int64_t rows, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>(rows));
    const int nvec = row_vecs<T>(a.V);
    if (rows <= kUnits && nvec > 2048)
        distill_held_kernel<T, 1024, 8><<<grid, dim3(1024), map_bytes(a), st>>>(a);
    else if (nvec <= 4096)
        distill_held_kernel<T, 256, 8><<<grid, dim3(256), map_bytes(a), st>>>(a);
    else
        distill_held_kernel<T, 512, sizeof(T) == 2 ? 12 : 8><<<grid, dim3(512), map_bytes(a), st>>>(a);
}

// Beam selection.
constexpr int kBeamMergeBlock = 1024;

// How a beam selection's rows are cut into workgroups, and its workspace.  A
// row's listing keeps a compute unit's vector units busy (256 KB take 10 us
// there), so a few long rows are cut into segments, as far as the merge can
// take their lists: one sequence of four beams of 128256 bfloat16 logits 13.2 us
// against 16.4, eight of eight beams 14.6 against 17.6.  Rows of 128 KB lose by
// it (10.8 against 10.4), and so do 240 rows (21.5 against 19.0).
constexpr int kSplitRows = 64;       // most rows that are cut
constexpr int kSplitVecs = 12288;    // 16-byte vectors of the shortest that are
constexpr int kSplitBlocks = 1024;   // workgroups to aim for
constexpr int kMaxSegs = 64;         // one lane per segment in the merge
struct BeamPlan {
    int segs, seg_vecs;
    size_t list, seg_lse, total;  // workspace offsets
};

template <typename T>
BeamPlan plan_beam_t(int64_t rows, int32_t V, int32_t beams, int32_t n) {
    constexpr int split_chunk = kShortBlock * LongShape<T>::unroll;
    const int nvec = row_vecs<T>(V);
    BeamPlan p{1, nvec, 0, 0, 0};
    if (rows <= kSplitRows && nvec >= kSplitVecs) {
        int64_t want = (kSplitBlocks + rows - 1) / rows;
        const int by_len = (nvec + split_chunk - 1) / split_chunk;
        const int fit = kMaxBeamKeys / (beams * n);
        if (want > by_len) want = by_len;
        if (want > fit) want = fit;
        if (want > kMaxSegs) want = kMaxSegs;
        if (want > 1) {
            const int chunks = (by_len + static_cast<int>(want) - 1) / static_cast<int>(want);
            p.seg_vecs = chunks * split_chunk;
            p.segs = (nvec + p.seg_vecs - 1) / p.seg_vecs;
        }
    }
    const size_t lists = static_cast<size_t>(rows) * p.segs;
    p.seg_lse = align_up(8 * lists * static_cast<size_t>(n));
    p.total = align_up(p.seg_lse + 8 * lists);
    return p;
}

BeamPlan plan_beam(int64_t rows, int32_t V, int32_t dtype, int32_t beams, int32_t n) {
    return dtype == SPEC_DTYPE_BF16 ? plan_beam_t<uint16_t>(rows, V, beams, n)
                                    : plan_beam_t<float>(rows, V, beams, n);
}

// Bound on how far the listing's float sums can move the difference of two
// beams' log-normalisers.  A term's exponent d = l log2(e)/T - n is off by half
// a step (2^-24 of |d|) and by the constant's own error; the terms' mean |d|
// is at most log2 V + 1.  exp2 is off by one step, and the five float additions
// that a term goes through in its chunk by half a step each; beyond the chunk
// the sums are double.
double near_bound(int32_t V, float temperature) {
    const double h = 0x1p-24;
    const double exact = kLog2eD / static_cast<double>(temperature);
    const double constant = std::fabs(static_cast<double>(log2e_over(temperature)) / exact - 1.0);
    const double one = kLn2 * (std::log2(static_cast<double>(V)) + 1.0) * (h + constant) + 7 * h;
    return 2.0 * one * 1.0001;  // the products of the errors
}

spec_status check_beam(int32_t batch, int32_t beams, int32_t vocab, int32_t dtype,
                       int32_t num_out) {
    if (batch < 0 || beams < 1 || num_out < 1 || vocab < 2) return SPEC_ERR_ARG;
    if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16) return SPEC_ERR_ARG;
    if (beams > kMaxBeams || num_out > kMaxBeamOut || beams * num_out > kMaxBeamKeys ||
        vocab > kMaxListVocab)
        return SPEC_ERR_UNSUPPORTED;
    return SPEC_OK;
}

struct Span {
    const char *from, *to;
    bool meets(const Span &o) const { return from < o.to && o.from < to; }
};

// Reordering: a unit per thread.  More units a thread only queue up behind
// each other (2.1 GB of caches, eight beams: 386 us, with two a thread 415, with
// four 428, with eight 439).
constexpr int kReorderBlock = 256;

template <int BYTES>
void launch_reorder(const ReorderArgs &a, int group, uint32_t blocks, hipStream_t st) {
    const dim3 grid(blocks), block(kReorderBlock);
    if (group == 8)
        beam_reorder_kernel<BYTES, 8, kReorderBlock><<<grid, block, 0, st>>>(a);
    else if (group == 16)
        beam_reorder_kernel<BYTES, 16, kReorderBlock><<<grid, block, 0, st>>>(a);
    else
        beam_reorder_kernel<BYTES, 32, kReorderBlock><<<grid, block, 0, st>>>(a);
}

// Bytes that a thread takes of each beam: the widest access that the bits of
// the addresses and of the positions' sizes allow.
int reorder_unit(uint64_t bits) { return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 1; }

uint64_t reorder_bits(const spec_beam_state &s) {
    return reinterpret_cast<uintptr_t>(s.src) | reinterpret_cast<uintptr_t>(s.dst) |
           static_cast<uint64_t>(s.position_bytes);
}

// Workgroups per segment of a state, and for the state.
int64_t reorder_chunks(const spec_beam_state &s, int unit) {
    const int64_t chunk = static_cast<int64_t>(unit) * kReorderBlock;
    return (s.position_bytes * s.positions + chunk - 1) / chunk;
}
int64_t reorder_blocks(const spec_beam_state &s, int unit, int32_t batch) {
    return reorder_chunks(s, unit) * s.segments * batch;
}

void launch_reorder(const ReorderArgs &a, int unit, int group, int64_t blocks, hipStream_t st) {
    if (unit == 16)
        launch_reorder<16>(a, group, static_cast<uint32_t>(blocks), st);
    else if (unit == 4)
        launch_reorder<4>(a, group, static_cast<uint32_t>(blocks), st);
    else
        launch_reorder<1>(a, group, static_cast<uint32_t>(blocks), st);
}

// States of different units go in a launch per unit, so that an odd one among
// them leaves the others' accesses wide, or all in one launch in the unit that
// they share.  Each further launch costs the host 2.8 us, so little work stays
// together (us, four beams, 16-byte caches and a history in 4-byte units, 4096
// workgroups in the shared unit: 17.5 apart, 14.7 together; 16384: 24 and 38;
// 65536: 81 and 140; with flags in single bytes 262144: 84 and 490).  With more
// than 12 beams 4-byte units keep as many bytes in flight as memory takes (65536
// workgroups, in place: 12 beams 229 and 243, 14 beams 282 and 265, 32 beams
// 648 and 598).
constexpr int64_t kOneUnitWork = 49152;  // workgroups times beams
bool reorder_together(int64_t blocks, int common, int32_t beams) {
    return blocks * beams <= kOneUnitWork || (common == 4 && beams > 12);
}

}  // namespace

extern "C" {

spec_status spec_row_topk(const void *logits, int64_t rows, int32_t vocab, int64_t row_stride,
                          int32_t dtype, float temperature, int32_t k, float *values,
                          int32_t *ids, float *lse, void *stream) {
    const spec_status s = check_logits_shape(vocab, row_stride, dtype, temperature);
    if (s != SPEC_OK) return s;
    if (rows < 0 || k < 1) return SPEC_ERR_ARG;
    if (k > kTopkMax || vocab > kMaxListVocab || !grid_fits(rows, 1024))
        return SPEC_ERR_UNSUPPORTED;
    if (rows == 0) return SPEC_OK;
    if (!logits || !aligned16(logits) || !values || !ids) return SPEC_ERR_ARG;
    TopkArgs a = topk_args(logits, row_stride, vocab, dtype, temperature, k);
    a.values = values;
    a.ids = ids;
    a.lse = lse;
    launch_topk(a, rows, dtype, static_cast<hipStream_t>(stream));
    return launch_status();
}

size_t spec_distill_state_bytes(int64_t rows) {
    return rows < 1 ? 0 : sizeof(DistillRow) * static_cast<size_t>(rows);
}

spec_status spec_distill_loss(const void *student, const int32_t *ids, const float *logits,
                              const float *lse, const uint8_t *keep,
                              const spec_distill_params *params, float *loss, void *state,
                              void *stream) {
    const spec_status s = check_distill(student, ids, logits, params);
    if (s != SPEC_OK || params->rows == 0) return s;
    if (!loss || !aligned16(state)) return SPEC_ERR_ARG;
    DistillArgs a = distill_args(student, ids, logits, params);
    a.lse = lse;
    a.keep = keep;
    a.loss = loss;
    a.state = static_cast<DistillRow *>(state);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (params->dtype == SPEC_DTYPE_BF16)
        launch_loss_t<uint16_t>(a, params->rows, st);
    else
        launch_loss_t<float>(a, params->rows, st);
    return launch_status();
}

spec_status spec_distill_grad(const void *student, const int32_t *ids, const float *logits,
                              const void *state, const float *grad_loss,
                              const spec_distill_params *params, void *grad, void *stream) {
    const spec_status s = check_distill(student, ids, logits, params);
    if (s != SPEC_OK || params->rows == 0) return s;
    if (!state || !aligned16(state) || !grad || !aligned16(grad) ||
        overlaps_partly(student, grad, params))
        return SPEC_ERR_ARG;
    DistillArgs a = distill_args(student, ids, logits, params);
    a.state = const_cast<DistillRow *>(static_cast<const DistillRow *>(state));
    a.grad_loss = grad_loss;
    a.grad = grad;
    a.seg_vecs = kGradVecs;
    const int64_t vecs = params->row_stride * elem_size(params->dtype) / 16;
    const int segs = static_cast<int>((vecs + kGradVecs - 1) / kGradVecs);
    if (!grid_fits(params->rows * segs, kGradBlock)) return SPEC_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(params->rows * segs));
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (params->dtype == SPEC_DTYPE_BF16)
        distill_grad_kernel<uint16_t, kGradBlock, kGradUnroll><<<grid, dim3(kGradBlock), 0, st>>>(a, segs);
    else
        distill_grad_kernel<float, kGradBlock, kGradUnroll><<<grid, dim3(kGradBlock), 0, st>>>(a, segs);
    return launch_status();
}

spec_status spec_distill_step(const void *student, const int32_t *ids, const float *logits,
                              const float *lse, const uint8_t *keep, const float *grad_loss,
                              const spec_distill_params *params, float *loss, void *grad,
                              void *stream) {
    const spec_status s = check_distill(student, ids, logits, params);
    if (s != SPEC_OK || params->rows == 0) return s;
    if (!loss || !grad || !aligned16(grad) || overlaps_partly(student, grad, params))
        return SPEC_ERR_ARG;
    DistillArgs a = distill_args(student, ids, logits, params);
    a.lse = lse;
    a.keep = keep;
    a.grad_loss = grad_loss;
    a.loss = loss;
    a.grad = grad;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (params->dtype == SPEC_DTYPE_BF16)
        launch_step_t<uint16_t>(a, params->rows, st);
    else
        launch_step_t<float>(a, params->rows, st);
    return launch_status();
}

size_t spec_beam_workspace_bytes(int32_t batch, int32_t num_beams, int32_t vocab, int32_t dtype,
                                 int32_t num_out) {
    if (check_beam(batch, num_beams, vocab, dtype, num_out) != SPEC_OK || batch == 0) return 0;
    return plan_beam(static_cast<int64_t>(batch) * num_beams, vocab, dtype, num_beams, num_out)
        .total;
}

spec_status spec_beam_select(const void *logits, int64_t row_stride, const float *scores,
                             const uint8_t *ended, int32_t batch, int32_t num_beams,
                             int32_t vocab, int32_t dtype, float temperature, int32_t num_out,
                             int32_t eos, float *out_scores, int32_t *parents, int32_t *tokens,
                             uint8_t *ended_out, void *workspace, size_t workspace_bytes,
                             void *stream) {
    spec_status s = check_logits_shape(vocab, row_stride, dtype, temperature);
    if (s != SPEC_OK) return s;
    if ((s = check_beam(batch, num_beams, vocab, dtype, num_out)) != SPEC_OK) return s;
    if (batch == 0) return SPEC_OK;
    if (!logits || !aligned16(logits) || !scores || !out_scores || !parents || !tokens)
        return SPEC_ERR_ARG;
    const int64_t rows = static_cast<int64_t>(batch) * num_beams;
    const BeamPlan p = plan_beam(rows, vocab, dtype, num_beams, num_out);
    if (!grid_fits(rows * p.segs, 1024)) return SPEC_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < p.total) return SPEC_ERR_WORKSPACE;
    if (!aligned16(workspace)) return SPEC_ERR_ARG;
    char *w = static_cast<char *>(workspace);
    TopkArgs t = topk_args(logits, row_stride, vocab, dtype, temperature, num_out);
    t.segs = p.segs;
    t.seg_vecs = p.seg_vecs;
    t.list = reinterpret_cast<unsigned long long *>(w + p.list);
    t.seg_lse = reinterpret_cast<double *>(w + p.seg_lse);
    t.ended = ended;
    t.scores = scores;
    hipStream_t st = static_cast<hipStream_t>(stream);
    launch_topk(t, rows, dtype, st);
    if ((s = launch_status()) != SPEC_OK) return s;
    BeamArgs a{};
    a.base = logits;
    a.scores = scores;
    a.ended = ended;
    a.list = t.list;
    a.seg_lse = t.seg_lse;
    a.out_scores = out_scores;
    a.parents = parents;
    a.tokens = tokens;
    a.ended_out = ended_out;
    a.stride = row_stride;
    a.V = vocab;
    a.W = num_beams;
    a.n = num_out;
    a.segs = p.segs;
    a.eos = eos;
    a.inv_t = t.inv_t;
    a.near = near_bound(vocab, temperature);
    if (dtype == SPEC_DTYPE_BF16)
        beam_merge_kernel<uint16_t, kBeamMergeBlock>
            <<<dim3(batch), dim3(kBeamMergeBlock), 0, st>>>(a);
    else
        beam_merge_kernel<float, kBeamMergeBlock>
            <<<dim3(batch), dim3(kBeamMergeBlock), 0, st>>>(a);
    return launch_status();
}

spec_status spec_beam_reorder(const int32_t *parents, const int32_t *lengths, int32_t batch,
                              int32_t num_beams, int32_t num_out, const spec_beam_state *states,
                              int32_t num_states, void *stream) {
    if (batch < 0 || num_beams < 1 || num_out < 1 || num_states < 0) return SPEC_ERR_ARG;
    if (num_beams > kMaxBeams || num_out > kMaxBeamOut) return SPEC_ERR_UNSUPPORTED;
    if (batch == 0 || num_states == 0) return SPEC_OK;
    if (!parents || !states) return SPEC_ERR_ARG;
    // every state is checked before anything is enqueued
    uint64_t bits = 0;
    bool in_place = false;
    for (int i = 0; i < num_states; ++i) {
        const spec_beam_state &s = states[i];
        if (!s.src || !s.dst || s.segments < 1 || s.positions < 0 || s.position_bytes < 1)
            return SPEC_ERR_ARG;
        if (s.position_bytes > INT32_MAX ||
            s.segments > (int64_t{1} << 44) / (s.position_bytes * (int64_t{s.positions} + 1)))
            return SPEC_ERR_UNSUPPORTED;
        const int64_t beam = s.position_bytes * s.positions * s.segments;
        if (beam > (int64_t{1} << 54) / batch) return SPEC_ERR_UNSUPPORTED;
        const char *src = static_cast<const char *>(s.src), *dst = static_cast<char *>(s.dst);
        const Span from{src, src + beam * num_beams * batch}, to{dst, dst + beam * num_out * batch};
        if (src == dst ? num_out != num_beams : from.meets(to))
            return SPEC_ERR_ARG;  // in place means beam for beam
        for (int j = 0; j < i; ++j) {  // what one state writes no other state holds
            const spec_beam_state &o = states[j];
            const int64_t other = o.position_bytes * o.positions * o.segments;
            const char *osrc = static_cast<const char *>(o.src);
            const char *odst = static_cast<char *>(o.dst);
            const Span ofrom{osrc, osrc + other * num_beams * batch};
            const Span oto{odst, odst + other * num_out * batch};
            if (to.meets(oto) || to.meets(ofrom) || from.meets(oto)) return SPEC_ERR_ARG;
        }
        if (!grid_fits(reorder_blocks(s, reorder_unit(reorder_bits(s)), batch), kReorderBlock))
            return SPEC_ERR_UNSUPPORTED;  // a launch takes whole states
        in_place = in_place || src == dst;
        bits |= reorder_bits(s);
    }
    const int group = !in_place || num_beams <= 8 ? 8 : num_beams <= 16 ? 16 : 32;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int common = reorder_unit(bits);
    int64_t all = 0;
    for (int i = 0; i < num_states && all <= kOneUnitWork; ++i)
        all += reorder_blocks(states[i], common, batch);
    const bool together = reorder_together(all, common, num_beams);
    for (const int unit : {16, 4, 1}) {
        ReorderArgs a{};
        a.parents = parents;
        a.lengths = lengths;
        a.W = num_beams;
        a.n = num_out;
        int64_t blocks = 0;
        for (int i = 0; i < num_states; ++i) {
            const spec_beam_state &s = states[i];
            const bool shared =
                together && grid_fits(reorder_blocks(s, common, batch), kReorderBlock);
            if (unit != (shared ? common : reorder_unit(reorder_bits(s)))) continue;
            const int64_t more = reorder_blocks(s, unit, batch);
            if (more == 0) continue;
            if (a.count == kMaxReorder || !grid_fits(blocks + more, kReorderBlock)) {
                launch_reorder(a, unit, group, blocks, st);
                const spec_status r = launch_status();
                if (r != SPEC_OK) return r;
                a.count = 0;
                blocks = 0;
            }
            ReorderState &r = a.st[a.count++];
            r.src = static_cast<const char *>(s.src);
            r.dst = static_cast<char *>(s.dst);
            r.pos_bytes = s.position_bytes;
            r.segments = s.segments;
            r.positions = s.positions;
            r.chunks = static_cast<int32_t>(reorder_chunks(s, unit));
            r.first = static_cast<uint32_t>(blocks);
            blocks += more;
        }
        if (a.count == 0) continue;
        launch_reorder(a, unit, group, blocks, st);
        const spec_status r = launch_status();
        if (r != SPEC_OK) return r;
    }
    return SPEC_OK;
}

}  // extern "C"
