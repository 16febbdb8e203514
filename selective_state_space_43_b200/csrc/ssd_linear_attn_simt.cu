// ssd_linear_attn_simt.cu -- decayed linear attention on the CUDA cores (fp32 rows).
//
// One block per (64 value channels, head, sequence or segment) walks its rows in chunks of C = 32:
//   P  = (Q K^T) . D,  D_ij = qk_scale e^{l(i-j)} for j <= i, else 0      [C x C]
//   O  = P V + inter_scale e^{l(i+s)} Q S                                  [C x 64]
//   S <- e^{lC} S + (K . w)^T V,  w_j = w_scale e^{l(C-j-s)}               [Dk x 64]
// in fp32 throughout.  The state lives in registers (Dk/16 x 8 per thread) and is copied to shared memory
// for the Q S product of the next chunk.  Two groups of warps side by side: scores and outputs, and the state.  Bound by
// fp32 FMAs, 2 Dk + C per row and value channel and C Dk / 64 for the scores, and the shared-memory reads that feed them:
// 4 x 1000 rows of 32 heads 128 x 128, 446 us (579 with one group for both).
#include "ssd_common.cuh"
#include "ssd_linear_attn.h"
#include "ssd_internal.h"

namespace ssd {
namespace la {
namespace {

constexpr int kGroup = 128, C = 32, DVB = 64;
// Row lengths (floats): K's rows are read by lanes of different rows, so they are padded; the scores take the place of Q,
// which has been read by then.
constexpr int PV = DVB, PP = C + 4;

template <int DKP> constexpr int q_floats() { return C * (DKP > PP ? DKP : PP); }
template <int DKP> constexpr size_t smem_bytes() {
    return sizeof(float) * (q_floats<DKP>() + C * (DKP + 4) + C * PV + DKP * PV + 2 * C);
}

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ float4 lds4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void st4(float* p, float a, float b, float c, float d) {
    *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
// Two multiply-adds to an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 dot4(float4 a, float4 b, float2 s) {
    return fma2(make_float2(a.z, a.w), make_float2(b.z, b.w), fma2(make_float2(a.x, a.y), make_float2(b.x, b.y), s));
}
__device__ __forceinline__ void axpy4(float2 (&o)[2], float a, float4 x) {
    o[0] = fma2(both(a), make_float2(x.x, x.y), o[0]);
    o[1] = fma2(both(a), make_float2(x.z, x.w), o[1]);
}

__device__ __forceinline__ void group_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }  // the outputs' group

// Two groups of 128 threads, the outputs of a chunk and its state side by side (both start from the state before it); for
// states alone the second group is the block.
template <int MODE> constexpr int threads() { return MODE == kStates ? kGroup : 2 * kGroup; }

template <int DKP, int MODE>
__global__ void __launch_bounds__(threads<MODE>(), 2) scan_simt_kernel(ScanArgs a) {
    constexpr int kThreads = threads<MODE>();
    extern __shared__ __align__(16) float sm[];
    constexpr int PK = DKP + 4, TK = DKP / 16;  // state rows of a thread
    float* sQ = sm;
    float* sK = sQ + q_floats<DKP>();
    float* sV = sK + C * PK;
    float* sS = sV + C * PV;
    float* sP = sQ;
    float* sPow = sS + DKP * PV;  // e^{l n}, n = 0 .. C
    const int tid = threadIdx.x, t = tid % kGroup, h = blockIdx.y, dv0 = blockIdx.z * DVB;
    const int nv = min(DVB, a.Dv - dv0);
    const Segment g = segment_of(a, blockIdx.x);
    if (a.cu && tid == 0 && h == 0 && blockIdx.z == 0 && !sequence_span(a, g.seq).ok)
        atomicOr(a.err, kErrBadSeqlens);
    if (!g.ok) return;
    const float l = a.log_decay[h];
    if (tid <= C) sPow[tid] = tid == 0 ? 1.f : expf(l * (float)tid);
    const int s = a.reverse ? 0 : 1;

    const float* q = static_cast<const float*>(a.q) + (size_t)(h / a.gq) * a.Dk;
    const float* k = static_cast<const float*>(a.k) + (size_t)(h / a.gk) * a.Dk;
    const float* v = static_cast<const float*>(a.v) + (size_t)(h / a.gv) * a.Dv + dv0;
    auto row = [&](int64_t c0, int i) { return a.reverse ? g.row0 + g.n - 1 - (c0 + i) : g.row0 + c0 + i; };
    auto load_tiles = [&](int64_t c0, int n) {  // both groups
        for (int i = tid; i < C * (DKP / 4); i += kThreads) {
            const int r = i / (DKP / 4), d = (i % (DKP / 4)) * 4;
            float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
            if (r < n && d < a.Dk) {
                if (MODE != kStates) load4(q + row(c0, r) * a.rs_q + d, x);
                load4(k + row(c0, r) * a.rs_k + d, y);
            }
            if (MODE != kStates) st4(sQ + r * DKP + d, x[0], x[1], x[2], x[3]);
            st4(sK + r * PK + d, y[0], y[1], y[2], y[3]);
        }
        for (int i = tid; i < C * (DVB / 4); i += kThreads) {
            const int r = i / (DVB / 4), d = (i % (DVB / 4)) * 4;
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            if (r < n && d < nv) load4(v + row(c0, r) * a.rs_v + d, x);
            st4(sV + r * PV + d, x[0], x[1], x[2], x[3]);
        }
    };

    if (MODE != kStates && tid < kGroup) {
        // ---- outputs.  P: rows i0, i0 + 16, columns j0 + {0, 8, 16, 24}; O: rows r0 .. r0+3, channels c4 .. c4+3
        const int i0 = t >> 3, j0 = t & 7, r0 = (t >> 4) * 4, c4 = (t & 15) * 4;
        float* o = static_cast<float*>(a.o) + (size_t)h * a.Dv + dv0;
        for (int64_t c0 = 0; c0 < g.n; c0 += C) {
            const int n = (int)min((int64_t)C, g.n - c0);
            __syncthreads();  // the last chunk's reads are done
            load_tiles(c0, n);
            __syncthreads();
            float2 p[2][4] = {};
#pragma unroll 2
            for (int d = 0; d < a.Dk; d += 4) {
                const float4 qa = lds4(sQ + i0 * DKP + d), qb = lds4(sQ + (i0 + 16) * DKP + d);
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    const float4 kk = lds4(sK + (j0 + 8 * jj) * PK + d);
                    p[0][jj] = dot4(qa, kk, p[0][jj]);
                    p[1][jj] = dot4(qb, kk, p[1][jj]);
                }
            }
            float2 out[4][2] = {};
#pragma unroll 2
            for (int d = 0; d < a.Dk; d += 4) {
                float4 qq[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) qq[i] = lds4(sQ + (r0 + i) * DKP + d);
                const float4 s0 = lds4(sS + d * PV + c4), s1 = lds4(sS + (d + 1) * PV + c4);
                const float4 s2 = lds4(sS + (d + 2) * PV + c4), s3 = lds4(sS + (d + 3) * PV + c4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    axpy4(out[i], qq[i].x, s0);
                    axpy4(out[i], qq[i].y, s1);
                    axpy4(out[i], qq[i].z, s2);
                    axpy4(out[i], qq[i].w, s3);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 e = both(a.inter_scale * sPow[r0 + i + s]);
                out[i][0] = __fmul2_rn(e, out[i][0]);
                out[i][1] = __fmul2_rn(e, out[i][1]);
            }
            group_sync();  // Q has been read
#pragma unroll
            for (int ii = 0; ii < 2; ++ii)
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    const int i = i0 + 16 * ii, j = j0 + 8 * jj;
                    sP[i * PP + j] = j <= i ? (p[ii][jj].x + p[ii][jj].y) * a.qk_scale * sPow[i - j] : 0.f;
                }
            group_sync();
            for (int j = 0; j < r0; j += 4) {
                float4 pp[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) pp[i] = lds4(sP + (r0 + i) * PP + j);
                const float4 x0 = lds4(sV + j * PV + c4), x1 = lds4(sV + (j + 1) * PV + c4);
                const float4 x2 = lds4(sV + (j + 2) * PV + c4), x3 = lds4(sV + (j + 3) * PV + c4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    axpy4(out[i], pp[i].x, x0);
                    axpy4(out[i], pp[i].y, x1);
                    axpy4(out[i], pp[i].z, x2);
                    axpy4(out[i], pp[i].w, x3);
                }
            }
            // the diagonal's four: a later row's value is not multiplied by zero but left out, since it may not be finite
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 x = lds4(sV + (r0 + j) * PV + c4);
#pragma unroll
                for (int i = j; i < 4; ++i) axpy4(out[i], sP[(r0 + i) * PP + r0 + j], x);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r0 + i < n && c4 < nv)
                    st4(o + row(c0, r0 + i) * (int64_t)a.H * a.Dv + c4, out[i][0].x, out[i][0].y, out[i][1].x,
                        out[i][1].y);
        }
        return;
    }

    // ---- the state: rows k0 .. , channels v0 .. v0+7
    const int k0 = (t >> 3) * TK, v0 = (t & 7) * 8;
    const size_t at_state = (size_t)a.Dk * a.Dv;
    const float* init = MODE == kOutputs ? a.seg_state + ((size_t)blockIdx.x * a.H + h) * at_state
                        : MODE == kStates || !a.init ? nullptr
                                                     : a.init + ((size_t)g.seq * a.H + h) * at_state;
    const bool init_t = MODE == kWhole ? a.init_t : a.seg_t;
    float2 S[TK][4];
#pragma unroll
    for (int r = 0; r < TK; ++r)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int kk = k0 + r, vv = v0 + c;
            const float x = init && kk < a.Dk && vv < nv
                                ? init[init_t ? (size_t)(dv0 + vv) * a.Dk + kk : (size_t)kk * a.Dv + dv0 + vv]
                                : 0.f;
            (c & 1 ? S[r][c / 2].y : S[r][c / 2].x) = x;
        }
    for (int64_t c0 = 0; c0 < g.n; c0 += C) {
        const int n = (int)min((int64_t)C, g.n - c0);
        __syncthreads();
        load_tiles(c0, n);
        if (MODE != kStates) {
#pragma unroll
            for (int r = 0; r < TK; ++r) {
                st4(sS + (k0 + r) * PV + v0, S[r][0].x, S[r][0].y, S[r][1].x, S[r][1].y);
                st4(sS + (k0 + r) * PV + v0 + 4, S[r][2].x, S[r][2].y, S[r][3].x, S[r][3].y);
            }
        }
        __syncthreads();
        // rows behind n are zero in shared memory
        const float2 e = both(sPow[n]);
#pragma unroll
        for (int r = 0; r < TK; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) S[r][c] = __fmul2_rn(e, S[r][c]);
#pragma unroll 2
        for (int j = 0; j < n; ++j) {
            const float w = a.w_scale * sPow[n - j - s];
            const float4 x = lds4(sV + j * PV + v0), y = lds4(sV + j * PV + v0 + 4);
            const float2 v2[4] = {make_float2(x.x, x.y), make_float2(x.z, x.w), make_float2(y.x, y.y), make_float2(y.z, y.w)};
            float kj[TK];
            if constexpr (TK % 4 == 0) {
#pragma unroll
                for (int r = 0; r < TK; r += 4) {
                    const float4 z = lds4(sK + j * PK + k0 + r);
                    kj[r] = z.x; kj[r + 1] = z.y; kj[r + 2] = z.z; kj[r + 3] = z.w;
                }
            } else {
#pragma unroll
                for (int r = 0; r < TK; ++r) kj[r] = sK[j * PK + k0 + r];
            }
#pragma unroll
            for (int r = 0; r < TK; ++r) {
                const float2 kk = both(w * kj[r]);
#pragma unroll
                for (int c = 0; c < 4; ++c) S[r][c] = fma2(kk, v2[c], S[r][c]);
            }
        }
    }
    float* fin = MODE == kStates  ? a.seg_state + ((size_t)blockIdx.x * a.H + h) * at_state
                 : MODE == kWhole ? (a.final_state ? a.final_state + ((size_t)g.seq * a.H + h) * at_state : nullptr)
                                  : nullptr;
    if (fin) {
#pragma unroll
        for (int r = 0; r < TK; ++r)
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (k0 + r < a.Dk && v0 + c < nv)
                    fin[(size_t)(k0 + r) * a.Dv + dv0 + v0 + c] = c & 1 ? S[r][c / 2].y : S[r][c / 2].x;
    }
}

template <int DKP, int MODE>
cudaError_t launch(const ScanArgs& a, cudaStream_t st) {
    const cudaError_t e = allow_smem<scan_simt_kernel<DKP, MODE>>((int)smem_bytes<DKP>());
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.seg_len ? a.slots : a.batch), a.H, (a.Dv + DVB - 1) / DVB);
    scan_simt_kernel<DKP, MODE><<<grid, threads<MODE>(), smem_bytes<DKP>(), st>>>(a);
    return cudaGetLastError();
}

template <int MODE>
cudaError_t launch_dk(const ScanArgs& a, cudaStream_t st) {
    if (a.Dk <= 32) return launch<32, MODE>(a, st);
    if (a.Dk <= 64) return launch<64, MODE>(a, st);
    return launch<128, MODE>(a, st);
}

}  // namespace

cudaError_t launch_scan_simt(const ScanArgs* scans, int count, Mode mode, cudaStream_t st) {
    for (int i = 0; i < count; ++i) {
        const ScanArgs& a = scans[i];
        const cudaError_t e = mode == kStates    ? launch_dk<kStates>(a, st)
                              : mode == kOutputs ? launch_dk<kOutputs>(a, st)
                                                 : launch_dk<kWhole>(a, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace la
}  // namespace ssd
