// ssd_linear_attn.h -- launch arguments shared by the linear-attention C entry points and kernels.
//
// Every pass over a sequence here is one scan of the same shape.  With the roles query, key, value of
// width Dk, Dk, Dv and the rows taken in time order i = 0 .. n-1 (against the time when `reverse`):
//   o_i = qk_scale sum_{j<=i} e^{l(i-j)} (query_i . key_j) value_j + inter_scale e^{l(i+s)} query_i S_0
//   S_n = e^{l n} S_0 + w_scale sum_j e^{l(n-1-j+1-s)} key_j value_j^T
// The forward is s = 1, inter_scale = qk_scale = scale, w_scale = 1.  With (q, k, v) the forward's rows,
// d(o) its gradient, the gradients are three more such scans, because the decay is a constant of the head:
//   dq: roles (do, v, k), s = 1, S_0 the transposed initial state, as the forward;
//   dk: roles (v, do, q) and dv: roles (k, q, do), against the time, s = 0, inter_scale = 1,
//       w_scale = scale, S_0 = the final state's gradient (transposed for dk); the state that the dv
//       scan ends with is the initial state's gradient.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace ssd {
namespace la {

struct ScanArgs {
    const void *q, *k, *v;       // rows of the three roles
    int64_t rs_q, rs_k, rs_v;    // elements between consecutive rows
    int gq, gk, gv;              // scan heads that share one stored head of the role
    int H, Dk, Dv;               // scan heads, widths
    const float* log_decay;      // [H]
    float qk_scale, inter_scale, w_scale;
    bool bf16;                   // the rows' type (else fp32)
    bool reverse;                // s = 0 and rows against the time
    const float* init;           // [batch][H][Dk][Dv] ([Dv][Dk] when init_t), or nullptr: zeros
    bool init_t;
    float* final_state;          // [batch][H][Dk][Dv] or nullptr
    void* o;                     // [rows][H][Dv]; fp32 when o_f32, else the activation type
    bool o_f32;
    int64_t batch, L, rows;      // sequences; rows of each (cu == nullptr); all rows
    const int64_t* cu;           // device, batch + 1 row offsets of packed sequences, or nullptr
    int* err;                    // device error word
    // The sequence axis cut into segments of seg_len rows (0: whole sequences), see Segment.
    int64_t seg_len, slots;
    float* seg_state;            // [slots][H][Dk][Dv] ([Dv][Dk] when seg_t: another scan's, joined there)
    bool seg_t;
};

// What a launch of a scan kernel does with its rows.
//   kWhole   the whole of each sequence: outputs and the final state
//   kStates  the state that each segment alone leaves (from zero) into seg_state
//   kOutputs the outputs of each segment from the state in seg_state
enum Mode { kWhole = 0, kStates = 1, kOutputs = 2 };

// One block's rows: row0 .. row0 + n of sequence `seq`; ok: anything to do.
struct Segment {
    int64_t row0, n, seq;
    bool ok;
};

// Segments live in `slots`.  Without packing, sequence b has the slots b * ceil(L / seg_len) + 0, 1, ..; packed,
// sequence b has cu[b] / seg_len + b + 0, 1, .., which leaves every sequence room for its segments
// (ceil(len / seg) <= (c + len) / seg - c / seg + 1) and needs no prefix sum of segment counts.
__host__ __device__ inline int64_t slot_count(int64_t batch, int64_t L, int64_t rows, bool packed, int64_t seg) {
    return packed ? rows / seg + batch : batch * ((L + seg - 1) / seg);
}

struct Span {
    int64_t start, len;
    bool ok;
};
__device__ inline Span sequence_span(const ScanArgs& a, int64_t b) {
    if (!a.cu) return Span{b * a.L, a.L, true};
    const int64_t r0 = a.cu[b], r1 = a.cu[b + 1];
    if (r0 < 0 || r1 < r0 || r1 > a.rows) return Span{0, 0, false};
    return Span{r0, r1 - r0, true};
}
// Segments of a sequence that is not packed: 32-bit arithmetic (rows < 2^31), for this is on the way to a block's first load.
__device__ inline uint32_t segments_each(const ScanArgs& a) {
    return ((uint32_t)a.L + (uint32_t)a.seg_len - 1) / (uint32_t)a.seg_len;
}
__device__ inline int64_t first_slot(const ScanArgs& a, int64_t b, const Span& s) {
    return a.cu ? s.start / a.seg_len + b : b * segments_each(a);
}
__device__ inline Segment segment_of(const ScanArgs& a, int64_t slot) {
    if (a.seg_len == 0) {
        const Span s = sequence_span(a, slot);
        return Segment{s.start, s.len, slot, true};
    }
    int64_t b;
    if (a.cu) {  // the last sequence whose first slot is not behind this one
        int64_t lo = 0, hi = a.batch - 1;
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) / 2;
            if (a.cu[mid] / a.seg_len + mid <= slot) lo = mid;
            else hi = mid - 1;
        }
        b = lo;
    } else {
        b = (uint32_t)slot / segments_each(a);
    }
    const Span s = sequence_span(a, b);
    const int64_t i = slot - first_slot(a, b, s), r = i * a.seg_len;
    if (!s.ok || i < 0 || r >= s.len) return Segment{0, 0, b, false};
    return Segment{s.start + r, s.len - r < a.seg_len ? s.len - r : a.seg_len, b, true};
}

// e^{l n} of a head; -inf (a head that keeps nothing) gives e^{l 0} = 1 like every other decay.
__device__ __forceinline__ float decay_pow(float l, int64_t n) { return n == 0 ? 1.f : expf(l * (float)n); }

// CUDA-core scan (fp32 rows).
cudaError_t launch_scan_simt(const ScanArgs* scans, int count, Mode mode, cudaStream_t st);
// Tensor-core scan (bf16 rows), up to three in one launch.
cudaError_t launch_scan_tc(const ScanArgs* scans, int count, Mode mode, cudaStream_t st);

// Runs the segments' states into one another: seg_state[i] becomes the state before segment i (in scan
// order, from init), final_state the state behind the last one.
// One or two scans of a call in one launch.
cudaError_t launch_combine(const ScanArgs* scans, int count, cudaStream_t st);
// dst[row][head][:] = sum over the `group` scan heads that share the head of src[row][head * group + g][:]; two
// such sums (of keys and of values) in one launch.  Rows outside every packed sequence, whose src nobody wrote, are left
// out.
struct GroupSum {
    const float* src;
    void* dst;
    int width;
    int64_t quads;    // set by the launch
    unsigned blocks;
};
struct GroupSums {
    GroupSum sum[2];
    int group, heads;         // scan heads to a head of dst; heads of dst
    const int64_t* cu;        // offsets of packed sequences or nullptr
    int64_t batch;
};
cudaError_t launch_group_sums(GroupSums a, int64_t rows, bool bf16, cudaStream_t st);

struct DecodeArgs {
    int64_t batch;
    int H, Hk, Dk, Dv;
    const float* log_decay;
    float scale;
    bool bf16;
    const void *q, *k, *v;
    float* state;
    void* o;
};
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t st);

}  // namespace la
}  // namespace ssd
