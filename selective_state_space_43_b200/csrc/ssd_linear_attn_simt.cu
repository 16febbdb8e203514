// ssd_linear_attn_simt.cu -- decayed linear attention on the CUDA cores (fp32 rows).
//
// One block per (64 value channels, head, sequence or segment) walks its rows in chunks of C = 32:
//   P  = (Q K^T) . D,  D_ij = qk_scale e^{l(i-j)} for j <= i, else 0      [C x C]
//   O  = P V + inter_scale e^{l(i+s)} Q S                                  [C x 64]
//   S <- e^{lC} S + (K . w)^T V,  w_j = w_scale e^{l(C-j-s)}               [Dk x 64]
// in fp32 throughout.  The state lives in registers (Dk/16 x 8 per thread) and is copied to shared memory
// for the Q S product of the next chunk.  Bound by fp32 FMAs: 4 Dk + 2 C per row and value channel.
#include "ssd_common.cuh"
#include "ssd_linear_attn.h"
#include "ssd_internal.h"

namespace ssd {
namespace la {
namespace {

constexpr int kThreads = 128, C = 32, DVB = 64;
constexpr int PV = DVB + 4, PP = C + 4;  // padded row lengths (floats), 16-byte multiples

template <int DKP> constexpr size_t smem_bytes() {
    return sizeof(float) * (2 * C * (DKP + 4) + C * PV + DKP * PV + C * PP + 3 * C);
}

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ float4 lds4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void st4(float* p, float a, float b, float c, float d) {
    *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ float dot4(float4 a, float4 b, float s) {
    return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, s))));
}
__device__ __forceinline__ void axpy4(float (&o)[4], float a, float4 x) {
    o[0] = fmaf(a, x.x, o[0]); o[1] = fmaf(a, x.y, o[1]); o[2] = fmaf(a, x.z, o[2]); o[3] = fmaf(a, x.w, o[3]);
}

template <int DKP, int MODE>
__global__ void __launch_bounds__(kThreads) scan_simt_kernel(ScanArgs a) {
    extern __shared__ __align__(16) float sm[];
    constexpr int PK = DKP + 4, TK = DKP / 16;  // state rows of a thread
    float* sQ = sm;
    float* sK = sQ + C * PK;
    float* sV = sK + C * PK;
    float* sS = sV + C * PV;
    float* sP = sS + DKP * PV;
    float* sPow = sP + C * PP;  // e^{l n}, n = 0 .. C
    const int tid = threadIdx.x, h = blockIdx.y, dv0 = blockIdx.z * DVB;
    const int nv = min(DVB, a.Dv - dv0);
    const Segment g = segment_of(a, blockIdx.x);
    if (a.cu && tid == 0 && h == 0 && blockIdx.z == 0 && !sequence_span(a, g.seq).ok)
        atomicOr(a.err, kErrBadSeqlens);
    if (!g.ok) return;
    const float l = a.log_decay[h];
    if (tid <= C) sPow[tid] = tid == 0 ? 1.f : expf(l * (float)tid);
    const int s = a.reverse ? 0 : 1;

    const int k0 = (tid >> 3) * TK, v0 = (tid & 7) * 8;  // this thread's state rows and channels
    float S[TK][8];
    const size_t at_state = (size_t)a.Dk * a.Dv;
    const float* init = MODE == kOutputs ? a.seg_state + ((size_t)blockIdx.x * a.H + h) * at_state
                        : MODE == kStates || !a.init ? nullptr
                                                     : a.init + ((size_t)g.seq * a.H + h) * at_state;
    const bool init_t = MODE == kWhole ? a.init_t : a.seg_t;
#pragma unroll
    for (int r = 0; r < TK; ++r)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int kk = k0 + r, vv = v0 + c;
            S[r][c] = init && kk < a.Dk && vv < nv
                          ? init[init_t ? (size_t)(dv0 + vv) * a.Dk + kk : (size_t)kk * a.Dv + dv0 + vv]
                          : 0.f;
        }
    const float* q = static_cast<const float*>(a.q) + (size_t)(h / a.gq) * a.Dk;
    const float* k = static_cast<const float*>(a.k) + (size_t)(h / a.gk) * a.Dk;
    const float* v = static_cast<const float*>(a.v) + (size_t)(h / a.gv) * a.Dv + dv0;
    float* o = static_cast<float*>(a.o) + (size_t)h * a.Dv + dv0;

    for (int64_t c0 = 0; c0 < g.n; c0 += C) {
        const int n = (int)min((int64_t)C, g.n - c0);
        auto row = [&](int i) { return a.reverse ? g.row0 + g.n - 1 - (c0 + i) : g.row0 + c0 + i; };
        __syncthreads();  // the last chunk's reads are done
        for (int i = tid; i < C * (DKP / 4); i += kThreads) {
            const int r = i / (DKP / 4), d = (i % (DKP / 4)) * 4;
            float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
            if (r < n && d < a.Dk) {
                if (MODE != kStates) load4(q + row(r) * a.rs_q + d, x);
                load4(k + row(r) * a.rs_k + d, y);
            }
            if (MODE != kStates) st4(sQ + r * PK + d, x[0], x[1], x[2], x[3]);
            st4(sK + r * PK + d, y[0], y[1], y[2], y[3]);
        }
        for (int i = tid; i < C * (DVB / 4); i += kThreads) {
            const int r = i / (DVB / 4), d = (i % (DVB / 4)) * 4;
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            if (r < n && d < nv) load4(v + row(r) * a.rs_v + d, x);
            st4(sV + r * PV + d, x[0], x[1], x[2], x[3]);
        }
        if (MODE != kStates) {
#pragma unroll
            for (int r = 0; r < TK; ++r) {
                st4(sS + (k0 + r) * PV + v0, S[r][0], S[r][1], S[r][2], S[r][3]);
                st4(sS + (k0 + r) * PV + v0 + 4, S[r][4], S[r][5], S[r][6], S[r][7]);
            }
        }
        __syncthreads();
        if (MODE != kStates) {
            // P: rows i0, i0 + 16, columns j0 + {0, 8, 16, 24}
            const int i0 = tid >> 3, j0 = tid & 7;
            float p[2][4] = {};
            for (int d = 0; d < a.Dk; d += 4) {
                const float4 qa = lds4(sQ + i0 * PK + d), qb = lds4(sQ + (i0 + 16) * PK + d);
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    const float4 kk = lds4(sK + (j0 + 8 * jj) * PK + d);
                    p[0][jj] = dot4(qa, kk, p[0][jj]);
                    p[1][jj] = dot4(qb, kk, p[1][jj]);
                }
            }
#pragma unroll
            for (int ii = 0; ii < 2; ++ii)
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    const int i = i0 + 16 * ii, j = j0 + 8 * jj;
                    sP[i * PP + j] = j <= i ? p[ii][jj] * a.qk_scale * sPow[i - j] : 0.f;
                }
            __syncthreads();
            // O: rows r0 .. r0+3, channels c4 .. c4+3
            const int r0 = (tid >> 4) * 4, c4 = (tid & 15) * 4;
            float out[4][4] = {}, in[4][4] = {};
            for (int d = 0; d < a.Dk; d += 4) {
                float4 qq[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) qq[i] = lds4(sQ + (r0 + i) * PK + d);
                const float4 s0 = lds4(sS + d * PV + c4), s1 = lds4(sS + (d + 1) * PV + c4);
                const float4 s2 = lds4(sS + (d + 2) * PV + c4), s3 = lds4(sS + (d + 3) * PV + c4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    axpy4(in[i], qq[i].x, s0);
                    axpy4(in[i], qq[i].y, s1);
                    axpy4(in[i], qq[i].z, s2);
                    axpy4(in[i], qq[i].w, s3);
                }
            }
            for (int j = 0; j < r0 + 4; j += 4) {
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
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (r0 + i < n && c4 < nv) {
                    const float e = a.inter_scale * sPow[r0 + i + s];
                    float* dst = o + row(r0 + i) * (int64_t)a.H * a.Dv + c4;
                    st4(dst, fmaf(e, in[i][0], out[i][0]), fmaf(e, in[i][1], out[i][1]), fmaf(e, in[i][2], out[i][2]),
                         fmaf(e, in[i][3], out[i][3]));
                }
            }
        }
        // S: rows behind n are zero in shared memory
        const float e = sPow[n];
#pragma unroll
        for (int r = 0; r < TK; ++r)
#pragma unroll
            for (int c = 0; c < 8; ++c) S[r][c] *= e;
        for (int j = 0; j < n; ++j) {
            const float w = a.w_scale * sPow[n - j - s];
            const float4 x = lds4(sV + j * PV + v0), y = lds4(sV + j * PV + v0 + 4);
#pragma unroll
            for (int r = 0; r < TK; ++r) {
                const float kk = w * sK[j * PK + k0 + r];
                S[r][0] = fmaf(kk, x.x, S[r][0]); S[r][1] = fmaf(kk, x.y, S[r][1]);
                S[r][2] = fmaf(kk, x.z, S[r][2]); S[r][3] = fmaf(kk, x.w, S[r][3]);
                S[r][4] = fmaf(kk, y.x, S[r][4]); S[r][5] = fmaf(kk, y.y, S[r][5]);
                S[r][6] = fmaf(kk, y.z, S[r][6]); S[r][7] = fmaf(kk, y.w, S[r][7]);
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
                if (k0 + r < a.Dk && v0 + c < nv) fin[(size_t)(k0 + r) * a.Dv + dv0 + v0 + c] = S[r][c];
    }
}

template <int DKP, int MODE>
cudaError_t launch(const ScanArgs& a, cudaStream_t st) {
    const cudaError_t e = allow_smem<scan_simt_kernel<DKP, MODE>>((int)smem_bytes<DKP>());
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.seg_len ? a.slots : a.batch), a.H, (a.Dv + DVB - 1) / DVB);
    scan_simt_kernel<DKP, MODE><<<grid, kThreads, smem_bytes<DKP>(), st>>>(a);
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
