// ssd_linear_attn.cu -- decayed linear attention: the single-token step, the joining of segment states, the
// sum of shared heads' gradients, and the C entry points (ssd_linear_attn_*).
#include <math.h>

#include "ssd.h"
#include "ssd_common.cuh"
#include "ssd_internal.h"
#include "ssd_linear_attn.h"

namespace ssd {
namespace la {
namespace {

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xFFFF0000u), __uint_as_float(a.y << 16),
                       __uint_as_float(a.y & 0xFFFF0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&b));
}

// ---- one token ----------------------------------------------------------------------------------------------
// S <- e^l S + k v^T, o = scale q S: every state element is read once and written once, two FMAs each, so the
// step is bound by HBM (256 sequences of 128 heads 128 x 64: 355 us, 6.1 TB/s).  One block per (sequence, head); a thread
// holds four value channels and walks the key rows with eight 16-byte loads in flight; the rows' partial outputs are
// joined in shared memory in a fixed order.
constexpr int kDecThreads = 256, kDecRows = 8;

template <typename T>
__global__ void __launch_bounds__(kDecThreads) decode_kernel(DecodeArgs a) {
    __shared__ float4 red[kDecThreads];
    __shared__ float sq[128], sk[128];
    const int64_t b = blockIdx.x / a.H;
    const int h = (int)(blockIdx.x - b * a.H), hk = h / (a.H / a.Hk), tid = threadIdx.x;
    const int nq = a.Dv / 4, per = kDecThreads / nq;  // threads across a row, rows of a pass
    const int r = tid / nq, c = (tid - r * nq) * 4;
    const bool live = r < per;
    float* S = a.state + (size_t)blockIdx.x * a.Dk * a.Dv;
    if (tid < a.Dk) {
        sq[tid] = to_f32(static_cast<const T*>(a.q)[(size_t)blockIdx.x * a.Dk + tid]) * a.scale;
        sk[tid] = to_f32(static_cast<const T*>(a.k)[((size_t)b * a.Hk + hk) * a.Dk + tid]);
    }
    const float4 v = load4(static_cast<const T*>(a.v) + ((size_t)b * a.Hk + hk) * a.Dv + (live ? c : 0));
    const float decay = decay_pow(a.log_decay[h], 1);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    for (int r0 = live ? r : a.Dk; r0 < a.Dk; r0 += per * kDecRows) {
        float4 x[kDecRows];
#pragma unroll
        for (int i = 0; i < kDecRows; ++i)
            if (r0 + i * per < a.Dk) x[i] = load4(S + (size_t)(r0 + i * per) * a.Dv + c);
#pragma unroll
        for (int i = 0; i < kDecRows; ++i) {
            const int d = r0 + i * per;
            if (d < a.Dk) {
                const float kd = sk[d], qd = sq[d];
                x[i].x = fmaf(decay, x[i].x, kd * v.x);
                x[i].y = fmaf(decay, x[i].y, kd * v.y);
                x[i].z = fmaf(decay, x[i].z, kd * v.z);
                x[i].w = fmaf(decay, x[i].w, kd * v.w);
                store4(S + (size_t)d * a.Dv + c, x[i]);
                o.x = fmaf(qd, x[i].x, o.x);
                o.y = fmaf(qd, x[i].y, o.y);
                o.z = fmaf(qd, x[i].z, o.z);
                o.w = fmaf(qd, x[i].w, o.w);
            }
        }
    }
    red[tid] = o;
    __syncthreads();
    if (tid < nq) {
        float4 t = red[tid];
        for (int i = 1; i < per; ++i) {
            const float4 u = red[i * nq + tid];
            t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
        }
        store4(static_cast<T*>(a.o) + (size_t)blockIdx.x * a.Dv + c, t);
    }
}

// ---- joining segments ---------------------------------------------------------------------------------------
// R <- e^{l n_i} R + (state of segment i alone), in scan order; four state elements per thread.
struct CombineArgs {
    ScanArgs scan[2];
};
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ CombineArgs both) {
    const ScanArgs& a = both.scan[blockIdx.x >= both.scan[0].batch];
    const int64_t b = blockIdx.x % a.batch;
    const int h = blockIdx.y, e = (blockIdx.z * 256 + threadIdx.x) * 4, size = a.Dk * a.Dv;
    const Span s = sequence_span(a, b);
    if (!s.ok && h == 0 && e == 0) atomicOr(a.err, kErrBadSeqlens);
    if (e >= size) return;
    const float l = a.log_decay[h];
    float4 R = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.init) {
        const float* src = a.init + ((size_t)b * a.H + h) * size;
        if (a.init_t) {
            const float* t = src + (size_t)(e % a.Dv) * a.Dk + e / a.Dv;
            R = make_float4(t[0], t[a.Dk], t[2 * a.Dk], t[3 * a.Dk]);
        } else {
            R = load4(src + e);
        }
    }
    const int64_t nseg = (s.len + a.seg_len - 1) / a.seg_len, slot0 = first_slot(a, b, s);
    const float whole = decay_pow(l, a.seg_len);
    const float last = decay_pow(l, s.len - (nseg - 1) * a.seg_len);
    // eight segments' states are loaded before the first is overwritten: one after the other would be a chain of latencies
    float* first = a.seg_state + (size_t)h * size + e;
    const int64_t pitch = (int64_t)a.H * size;
    for (int64_t j0 = 0; j0 < nseg; j0 += 8) {
        float4 x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j0 + j < nseg) x[j] = load4(first + (slot0 + (a.reverse ? nseg - 1 - j0 - j : j0 + j)) * pitch);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j0 + j < nseg) {
                const int64_t i = a.reverse ? nseg - 1 - j0 - j : j0 + j;
                const float d = i == nseg - 1 ? last : whole;
                store4(first + (slot0 + i) * pitch, R);
                R.x = fmaf(d, R.x, x[j].x);
                R.y = fmaf(d, R.y, x[j].y);
                R.z = fmaf(d, R.z, x[j].z);
                R.w = fmaf(d, R.w, x[j].w);
            }
        }
    }
    if (a.final_state) store4(a.final_state + ((size_t)b * a.H + h) * size + e, R);
}

// ---- gradients of shared heads ------------------------------------------------------------------------------
template <typename T> __global__ void __launch_bounds__(256) group_sum_kernel(GroupSums a) {
    const int which = blockIdx.x >= a.sum[0].blocks;
    const GroupSum& g = a.sum[which];
    const int64_t i = (int64_t)(blockIdx.x - (which ? a.sum[0].blocks : 0)) * 256 + threadIdx.x;
    if (i >= g.quads) return;
    const int per = g.width / 4;
    const int64_t head = i / per;  // (row, head) of dst
    if (a.cu && ((uint64_t)head < (uint64_t)a.cu[0] * a.heads || (uint64_t)head >= (uint64_t)a.cu[a.batch] * a.heads)) return;
    const float* p = g.src + (head * a.group * per + (i - head * per)) * 4;
    float4 t = load4(p);
    for (int k = 1; k < a.group; ++k) {
        const float4 u = load4(p + (size_t)k * g.width);
        t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
    }
    store4(static_cast<T*>(g.dst) + i * 4, t);
}

}  // namespace

cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t st) {
    const unsigned blocks = (unsigned)(a.batch * a.H);
    if (a.bf16)
        decode_kernel<__nv_bfloat16><<<blocks, kDecThreads, 0, st>>>(a);
    else
        decode_kernel<float><<<blocks, kDecThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_combine(const ScanArgs* scans, int count, cudaStream_t st) {
    const ScanArgs& a = scans[0];  // the scans of one call have the same number of states of the same size
    const dim3 grid((unsigned)(a.batch * count), a.H, (a.Dk * a.Dv + 1023) / 1024);
    combine_kernel<<<grid, 256, 0, st>>>(CombineArgs{{scans[0], scans[count - 1]}});
    return cudaGetLastError();
}

cudaError_t launch_group_sums(GroupSums a, int64_t rows, bool bf16, cudaStream_t st) {
    int64_t blocks = 0;
    for (GroupSum& g : a.sum) {
        g.quads = rows * a.heads * (g.width / 4);
        g.blocks = (unsigned)((g.quads + 255) / 256);
        blocks += (g.quads + 255) / 256;
    }
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    if (bf16)
        group_sum_kernel<__nv_bfloat16><<<(unsigned)blocks, 256, 0, st>>>(a);
    else
        group_sum_kernel<float><<<(unsigned)blocks, 256, 0, st>>>(a);
    return cudaGetLastError();
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Read one value at a time, so their own alignment is enough.
bool offsets_aligned(const float* log_decay, const int64_t* cu_seqlens) {
    return !(reinterpret_cast<uintptr_t>(log_decay) & 3u) && !(reinterpret_cast<uintptr_t>(cu_seqlens) & 7u);
}

ssd_status check_dims(const ssd_linear_attn_dims* d, ssd_dtype dtype) {
    if (!d) return SSD_ERR_NULL;
    if (dtype != SSD_F32 && dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (d->batch < 0 || d->seqlen < 0) return SSD_ERR_SHAPE;
    if (d->nheads <= 0 || d->kv_heads <= 0 || d->nheads % d->kv_heads != 0 || d->nheads > 65535) return SSD_ERR_SHAPE;
    for (int w : {d->key_dim, d->value_dim})
        if (w < 8 || w > 128 || w % 8 != 0) return SSD_ERR_SHAPE;
    if (d->batch > (1LL << 31) - 1 || d->batch * (int64_t)d->nheads > (1LL << 28)) return SSD_ERR_SHAPE;
    return SSD_OK;
}

// Rows of all sequences; tensor-map row coordinates and the launches' slot counts are 32-bit.
ssd_status count_rows(const ssd_linear_attn_dims* d, bool packed, int64_t* rows) {
    constexpr int64_t most = (1LL << 31) - 256;
    if (d->seqlen > most || (!packed && d->seqlen > 0 && d->batch > most / d->seqlen)) return SSD_ERR_SHAPE;
    *rows = packed ? d->seqlen : d->batch * d->seqlen;
    return SSD_OK;
}

struct Buffer {
    const void* p;
    uint64_t n;  // bytes
};
// A role's rows as the caller's buffer: `rows` rows `stride` elements apart, the last one `width` long.
Buffer row_buffer(const void* p, int64_t rows, int64_t stride, int64_t width, uint64_t esize) {
    return Buffer{p, rows > 0 ? ((uint64_t)(rows - 1) * stride + width) * esize : 0};
}
bool overlap(const Buffer& a, const Buffer& b) {
    if (!a.p || !b.p || !a.n || !b.n) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n && y < x + a.n;
}
template <int NO, int NI> bool outputs_alias(const Buffer (&outs)[NO], const Buffer (&ins)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = i + 1; j < NO; ++j)
            if (overlap(outs[i], outs[j])) return true;
        for (int j = 0; j < NI; ++j)
            if (overlap(outs[i], ins[j])) return true;
    }
    return false;
}

cudaError_t launch_scans(const ScanArgs* scans, int count, Mode mode, cudaStream_t st) {
    return scans[0].bf16 ? launch_scan_tc(scans, count, mode, st) : launch_scan_simt(scans, count, mode, st);
}

// ---- cutting the sequence axis ------------------------------------------------------------------------------
// A scan walks its rows one chunk behind the other, so a call with few (sequence, head) pairs leaves SMs
// idle.  Cut into segments it takes two passes (the state each segment leaves, joined, then the outputs from
// the joined states), which read keys and values twice.  The choice compares modelled times in microseconds: a block
// costs `start`, and per row `row` for outputs and state or `state_row` for states alone; an SM runs `resident` blocks
// (`state_resident` of states alone) side by side, each of which slows the others by `beside`; the cut adds two launches
// (`extra`) and the writing, joining and reading of its states at `state_rate` bytes a microsecond.  The first cut has to
// gain what `cut` says, a shorter one what `shorter` says over a longer.
//
// The lengths of a packed batch are not known here (they are on the device): its longest sequence is taken to be `spread`
// times the mean, each sequence to need `more` segments beside those of its rows.  The constants are fitted to 229 measured
// cases (B200, every cut of 32 to 8192 rows; sizes drawn at random, packed rows cut at random places): in 224 of
// them the choice is within 10 % of the fastest, the worst is 22 % off (bf16 backward, 2 sequences of 4932 rows, 8 heads of
// 64 x 96: 54 us, 44 whole).  Both sides of some, in us, whole against the chosen cut, three replays from an idle GPU (the
// power cap, which makes the 289 below 333 in a long run, does not bite yet):
// bf16, 1 x 8191 rows, 16 heads of 128 x 128, 120 against 72 (2048 rows; 90 at 512); 9000 rows in 12, 10 heads of
// 64 x 64, 37 whole (51 at 512); 4 x 8192 rows, 64 heads of 128 x 64, 289 whole (459 at 2048).  fp32, 1 x 256 rows, 4 heads
// of 32 x 64, 33 against 17 (32 rows); 4636 rows in 15, 16 heads of 64 x 96, 308 against 253 (128; 321 at 512);
// backward of 4 x 1000 rows, 16 heads of 128 x 64, 736 against 598 (128; 575 at 256, 704 at 512); 4 x 1000 rows, 32 heads of
// 128 x 128, 446 whole (705 at 256).
//
// A packed batch of one long sequence among many short ones looks like an even one from here, and stays whole where that
// would be right: 32768 rows and 63 single ones, 8 heads of 128 x 64, 426 us whole (156 at 2048), but 32831 rows in 64 even
// ones 66 whole (158 at 1024); 16384 rows and 31 single ones, 4 heads of 64 x 64, 203 (48 at 1024), even ones 33 (47).
struct Cost {
    double start, row, state_row, extra, state_rate, beside, resident, state_resident, spread, more, cut, shorter;
    int64_t least;  // rows of a segment: a chunk of the kernel
    bool together;  // a pass's scans are one launch
};
Cost cost_of(bool bf16, int Dk) {
    if (bf16) return Cost{3.3, 1.46 / 128, 0.8 / 128, 6.0, 7.6e6, 0.0, 1.0, 1.0, 3.4, 0.68, 0.87, 0.84, 256, true};
    const double row = 0.031 + 0.004 * Dk;
    return Cost{0.9, row, 0.73 * row, 5.0, 2.6e6, 0.136, 2.0, 16.0, 4.4, 0.65, 0.8, 0.957, 32, false};
}
constexpr double kSms = 148.0;
// Rows of a segment, or 0: whole sequences.  `blocks`: blocks of the output pass for each sequence, of `scans` scans;
// `state_blocks`, `state_scans`: of the states' pass.
int64_t segment_rows(int64_t batch, int64_t L, int64_t rows, bool packed, bool bf16, int Dk, int Dv, int64_t H,
                     int64_t blocks, int scans, int64_t state_blocks, int state_scans) {
    if (batch == 0 || rows == 0) return 0;
    const Cost k = cost_of(bf16, Dk);
    const double mean = (double)rows / batch, longest = packed ? fmin((double)rows, k.spread * mean) : (double)L;
    // n blocks of `of` scans, rows_each rows in the mean and rows_most in the longest
    auto pass = [&](double n, int of, double per_row, double rows_each, double rows_most, double resident) {
        const int launches = k.together ? 1 : of;
        const double on_sm = fmax(1.0, n / launches / kSms);
        const double slower = 1.0 + k.beside * (fmin(on_sm, resident) - 1.0);
        const double turns = fmax(1.0, on_sm / resident);
        return launches * fmax((packed ? turns : ceil(turns)) * slower * (k.start + rows_each * per_row),
                               k.start + rows_most * per_row);
    };
    double best = pass((double)batch * blocks, scans, k.row, mean, longest, k.resident);
    int64_t seg = 0;
    int64_t m = k.least;
    while (m * 2 < longest) m *= 2;
    for (; m >= k.least && m < longest; m /= 2) {
        const double slots = packed ? rows / (double)m + k.more * batch : batch * ceil((double)L / m);
        const double bytes = slots * H * Dk * Dv * 4 * 4 * state_scans;  // written, read and written, read
        const double part = fmin((double)m, mean), most = fmin((double)m, longest);
        const double t = pass(slots * state_blocks, state_scans, k.state_row, part, most, k.state_resident) +
                         pass(slots * blocks, scans, k.row, part, most, k.resident) + k.extra + bytes / k.state_rate;
        if (t < (seg ? k.shorter : k.cut) * best) {
            best = t;
            seg = m;
        }
    }
    return seg;
}
int64_t value_blocks(int64_t H, int Dv) { return H * ((Dv + 63) / 64); }

int64_t prefill_segment(const ssd_linear_attn_dims* d, bool bf16, bool packed, int64_t rows) {
    const int64_t b = value_blocks(d->nheads, d->value_dim);
    return segment_rows(d->batch, d->seqlen, rows, packed, bf16, d->key_dim, d->value_dim, d->nheads, b, 1, b, 1);
}
int64_t backward_segment(const ssd_linear_attn_dims* d, bool bf16, bool packed, int64_t rows) {
    const int64_t k = value_blocks(d->nheads, d->key_dim), v = value_blocks(d->nheads, d->value_dim);
    return segment_rows(d->batch, d->seqlen, rows, packed, bf16, d->key_dim, d->value_dim, d->nheads, 2 * k + v, 3,
                        k + v, 2);
}
// Bytes of one scan's segment states.
size_t segment_bytes(const ssd_linear_attn_dims* d, bool packed, int64_t rows, int64_t seg) {
    if (seg == 0) return 0;
    return (size_t)slot_count(d->batch, d->seqlen, rows, packed, seg) * d->nheads * d->key_dim * d->value_dim * 4;
}

}  // namespace
}  // namespace la
}  // namespace ssd

using namespace ssd;
using namespace ssd::la;

extern "C" {

size_t ssd_linear_attn_prefill_workspace_bytes(const ssd_linear_attn_dims* d, ssd_dtype dtype, int packed) {
    int64_t rows;
    if (la::check_dims(d, dtype) != SSD_OK || count_rows(d, packed != 0, &rows) != SSD_OK) return 0;
    return segment_bytes(d, packed != 0, rows, prefill_segment(d, dtype == SSD_BF16, packed != 0, rows));
}

ssd_status ssd_linear_attn_prefill(const ssd_linear_attn_dims* d, ssd_dtype dtype, const float* log_decay, float scale,
                                   const ssd_linear_attn_strides* strides, const int64_t* cu_seqlens, const void* q,
                                   const void* k, const void* v, const float* init_state, void* o, float* final_state,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    ssd_status st = la::check_dims(d, dtype);
    if (st != SSD_OK) return st;
    const bool packed = cu_seqlens != nullptr;
    int64_t rows;
    if ((st = count_rows(d, packed, &rows)) != SSD_OK) return st;
    if (!isfinite(scale)) return SSD_ERR_SHAPE;
    if (!log_decay || (d->batch > 0 && !final_state)) return SSD_ERR_NULL;
    if (d->batch > 0 && rows > 0 && (!q || !k || !v || !o)) return SSD_ERR_NULL;
    for (const void* p : {q, k, v, (const void*)o, (const void*)init_state, (const void*)final_state,
                          (const void*)workspace})
        if (!aligned16(p)) return SSD_ERR_ALIGN;
    if (!offsets_aligned(log_decay, cu_seqlens)) return SSD_ERR_ALIGN;
    const int64_t H = d->nheads, Hk = d->kv_heads, Dk = d->key_dim, Dv = d->value_dim;
    const uint64_t es = dtype == SSD_F32 ? 4 : 2;
    ssd_linear_attn_strides rs{H * Dk, Hk * Dk, Hk * Dv};
    if (strides) {
        if (strides->q < rs.q || strides->k < rs.k || strides->v < rs.v) return SSD_ERR_SHAPE;
        if (strides->q > (1LL << 32) || strides->k > (1LL << 32) || strides->v > (1LL << 32)) return SSD_ERR_SHAPE;
        if (((strides->q | strides->k | strides->v) * (int64_t)es) & 15) return SSD_ERR_ALIGN;
        rs = *strides;
    }
    const uint64_t state = (uint64_t)d->batch * H * Dk * Dv * 4;
    const size_t need = ssd_linear_attn_prefill_workspace_bytes(d, dtype, packed);
    {
        const Buffer ins[] = {row_buffer(q, rows, rs.q, H * Dk, es), row_buffer(k, rows, rs.k, Hk * Dk, es),
                              row_buffer(v, rows, rs.v, Hk * Dv, es), {log_decay, (uint64_t)H * 4},
                              {cu_seqlens, ((uint64_t)d->batch + 1) * 8}};
        const Buffer outs[] = {{o, (uint64_t)rows * H * Dv * es}, {final_state, state}, {workspace, need}};
        if (outputs_alias(outs, ins)) return SSD_ERR_UNSUPPORTED;
        if (init_state && init_state != final_state && overlap({init_state, state}, outs[1])) return SSD_ERR_UNSUPPORTED;
        if (overlap({init_state, state}, outs[0]) || overlap({init_state, state}, outs[2])) return SSD_ERR_UNSUPPORTED;
    }
    if (need > 0 && (!workspace || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
    if (d->batch == 0) return SSD_OK;
    ScanArgs a{};
    a.q = q; a.k = k; a.v = v;
    a.rs_q = rs.q; a.rs_k = rs.k; a.rs_v = rs.v;
    a.gq = 1; a.gk = a.gv = (int)(H / Hk);
    a.H = (int)H; a.Dk = (int)Dk; a.Dv = (int)Dv;
    a.log_decay = log_decay;
    a.qk_scale = a.inter_scale = scale;
    a.w_scale = 1.f;
    a.bf16 = dtype == SSD_BF16;
    a.init = init_state;
    a.final_state = final_state;
    a.o = o;
    a.batch = d->batch; a.L = d->seqlen; a.rows = rows;
    a.cu = cu_seqlens;
    if (!(a.err = device_error_flag())) return SSD_ERR_CUDA;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    a.seg_len = prefill_segment(d, a.bf16, packed, rows);
    if (a.seg_len == 0) return launch_scans(&a, 1, kWhole, cs) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    a.slots = slot_count(a.batch, a.L, rows, packed, a.seg_len);
    a.seg_state = static_cast<float*>(workspace);
    cudaError_t e = launch_scans(&a, 1, kStates, cs);
    if (e == cudaSuccess) e = launch_combine(&a, 1, cs);
    if (e == cudaSuccess) e = launch_scans(&a, 1, kOutputs, cs);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

// Bytes of the fp32 per-head gradients of shared keys and values (none when every head has its own).
static size_t group_bytes(const ssd_linear_attn_dims* d, int64_t rows) {
    if (d->nheads == d->kv_heads) return 0;
    return (size_t)rows * d->nheads * (d->key_dim + d->value_dim) * 4;
}

size_t ssd_linear_attn_backward_workspace_bytes(const ssd_linear_attn_dims* d, ssd_dtype dtype, int packed) {
    int64_t rows;
    if (la::check_dims(d, dtype) != SSD_OK || count_rows(d, packed != 0, &rows) != SSD_OK) return 0;
    return group_bytes(d, rows) +
           2 * segment_bytes(d, packed != 0, rows, backward_segment(d, dtype == SSD_BF16, packed != 0, rows));
}

ssd_status ssd_linear_attn_backward(const ssd_linear_attn_dims* d, ssd_dtype dtype, const float* log_decay, float scale,
                                    const int64_t* cu_seqlens, const void* q, const void* k, const void* v,
                                    const float* init_state, const void* d_o, const float* d_final_state, void* dq,
                                    void* dk, void* dv, float* d_init_state, void* workspace, size_t workspace_bytes,
                                    void* stream) {
    ssd_status st = la::check_dims(d, dtype);
    if (st != SSD_OK) return st;
    const bool packed = cu_seqlens != nullptr;
    int64_t rows;
    if ((st = count_rows(d, packed, &rows)) != SSD_OK) return st;
    if (!isfinite(scale)) return SSD_ERR_SHAPE;
    if (!log_decay) return SSD_ERR_NULL;
    if (d->batch > 0 && rows > 0 && (!q || !k || !v || !d_o || !dq || !dk || !dv)) return SSD_ERR_NULL;
    for (const void* p : {q, k, v, d_o, (const void*)dq, (const void*)dk, (const void*)dv, (const void*)init_state,
                          (const void*)d_final_state, (const void*)d_init_state, (const void*)workspace})
        if (!aligned16(p)) return SSD_ERR_ALIGN;
    if (!offsets_aligned(log_decay, cu_seqlens)) return SSD_ERR_ALIGN;
    const int64_t H = d->nheads, Hk = d->kv_heads, Dk = d->key_dim, Dv = d->value_dim;
    const uint64_t es = dtype == SSD_F32 ? 4 : 2, n = (uint64_t)rows;
    const uint64_t state = (uint64_t)d->batch * H * Dk * Dv * 4;
    const size_t need = ssd_linear_attn_backward_workspace_bytes(d, dtype, packed);
    {
        const Buffer ins[] = {{q, n * H * Dk * es}, {k, n * Hk * Dk * es}, {v, n * Hk * Dv * es}, {d_o, n * H * Dv * es},
                              {init_state, state}, {d_final_state, state}, {log_decay, (uint64_t)H * 4},
                              {cu_seqlens, ((uint64_t)d->batch + 1) * 8}};
        const Buffer outs[] = {{dq, n * H * Dk * es}, {dk, n * Hk * Dk * es}, {dv, n * Hk * Dv * es},
                               {d_init_state, state}, {workspace, need}};
        if (outputs_alias(outs, ins)) return SSD_ERR_UNSUPPORTED;
    }
    if (need > 0 && (!workspace || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
    if (d->batch == 0) return SSD_OK;

    const int group = (int)(H / Hk);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    ScanArgs base{};
    base.H = (int)H;
    base.log_decay = log_decay;
    base.qk_scale = scale;
    base.bf16 = dtype == SSD_BF16;
    base.batch = d->batch; base.L = d->seqlen; base.rows = rows;
    base.cu = cu_seqlens;
    if (!(base.err = device_error_flag())) return SSD_ERR_CUDA;
    // workspace: the shared heads' dk and dv, then the segment states of the dq scan and of the dv scan
    float* ws = static_cast<float*>(workspace);
    float* dk_heads = group > 1 ? ws : nullptr;
    float* dv_heads = group > 1 ? ws + (size_t)rows * H * Dk : nullptr;
    base.seg_len = backward_segment(d, base.bf16, packed, rows);
    if (base.seg_len) base.slots = slot_count(base.batch, base.L, rows, packed, base.seg_len);
    float* states = ws + group_bytes(d, rows) / 4;

    ScanArgs a[3];
    ScanArgs& sq = a[0] = base;  // dq
    sq.q = d_o; sq.rs_q = H * Dv; sq.gq = 1;
    sq.k = v; sq.rs_k = Hk * Dv; sq.gk = group;
    sq.v = k; sq.rs_v = Hk * Dk; sq.gv = group;
    sq.Dk = (int)Dv; sq.Dv = (int)Dk;
    sq.inter_scale = scale; sq.w_scale = 1.f;
    sq.init = init_state; sq.init_t = true;
    sq.o = dq;
    sq.o_f32 = dtype == SSD_F32;
    sq.seg_state = states;

    ScanArgs& sv = a[1] = base;  // dv, and the initial state's gradient
    sv.reverse = true;
    sv.inter_scale = 1.f; sv.w_scale = scale;
    sv.q = k; sv.rs_q = Hk * Dk; sv.gq = group;
    sv.k = q; sv.rs_k = H * Dk; sv.gk = 1;
    sv.v = d_o; sv.rs_v = H * Dv; sv.gv = 1;
    sv.Dk = (int)Dk; sv.Dv = (int)Dv;
    sv.init = d_final_state;
    sv.final_state = d_init_state;
    sv.o = group > 1 ? dv_heads : dv;
    sv.o_f32 = group > 1 || dtype == SSD_F32;
    sv.seg_state = base.seg_len ? states + segment_bytes(d, packed, rows, base.seg_len) / 4 : nullptr;

    ScanArgs& sk = a[2] = base;  // dk: the dv scan's states, transposed
    sk.reverse = true;
    sk.inter_scale = 1.f; sk.w_scale = scale;
    sk.q = v; sk.rs_q = Hk * Dv; sk.gq = group;
    sk.k = d_o; sk.rs_k = H * Dv; sk.gk = 1;
    sk.v = q; sk.rs_v = H * Dk; sk.gv = 1;
    sk.Dk = (int)Dv; sk.Dv = (int)Dk;
    sk.init = d_final_state; sk.init_t = true;
    sk.o = group > 1 ? dk_heads : dk;
    sk.o_f32 = group > 1 || dtype == SSD_F32;
    sk.seg_state = sv.seg_state;
    sk.seg_t = true;

    cudaError_t e;
    if (base.seg_len) {
        e = launch_scans(a, 2, kStates, cs);
        if (e == cudaSuccess) e = launch_combine(a, 2, cs);
        if (e == cudaSuccess) e = launch_scans(a, 3, kOutputs, cs);
    } else {
        e = launch_scans(a, 3, kWhole, cs);
    }
    if (e == cudaSuccess && group > 1)
        e = launch_group_sums(
            GroupSums{{{dk_heads, dk, (int)Dk}, {dv_heads, dv, (int)Dv}}, group, (int)Hk, cu_seqlens, d->batch}, rows,
            base.bf16, cs);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_linear_attn_decode_step(const ssd_linear_attn_dims* d, ssd_dtype dtype, const float* log_decay,
                                       float scale, const void* q, const void* k, const void* v, float* state, void* o,
                                       void* stream) {
    if (!d) return SSD_ERR_NULL;
    ssd_linear_attn_dims one = *d;
    one.seqlen = 1;
    const ssd_status st = la::check_dims(&one, dtype);
    if (st != SSD_OK) return st;
    if (!isfinite(scale)) return SSD_ERR_SHAPE;
    if (!log_decay || (d->batch > 0 && (!q || !k || !v || !state || !o))) return SSD_ERR_NULL;
    for (const void* p : {q, k, v, (const void*)state, (const void*)o})
        if (!aligned16(p)) return SSD_ERR_ALIGN;
    if (!offsets_aligned(log_decay, nullptr)) return SSD_ERR_ALIGN;
    const uint64_t es = dtype == SSD_F32 ? 4 : 2, H = d->nheads, Hk = d->kv_heads, Dk = d->key_dim, Dv = d->value_dim;
    const uint64_t b = d->batch;
    const Buffer ins[] = {{q, b * H * Dk * es}, {k, b * Hk * Dk * es}, {v, b * Hk * Dv * es}, {log_decay, H * 4}};
    const Buffer outs[] = {{state, b * H * Dk * Dv * 4}, {o, b * H * Dv * es}};
    if (outputs_alias(outs, ins)) return SSD_ERR_UNSUPPORTED;
    if (d->batch == 0) return SSD_OK;
    la::DecodeArgs a{};
    a.batch = d->batch;
    a.H = (int)H; a.Hk = (int)Hk; a.Dk = (int)Dk; a.Dv = (int)Dv;
    a.log_decay = log_decay;
    a.scale = scale;
    a.bf16 = dtype == SSD_BF16;
    a.q = q; a.k = k; a.v = v;
    a.state = state;
    a.o = o;
    return la::launch_decode(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
