// ssd_qk_norm_rope.cu -- RMSNorm of each query and key head with the position rotation in the same pass, and
// its gradients.
//
// Per token t and head row x of width D, with r = rsqrt(mean(x^2) + eps):
//   n = x r w                                 (w: one weight per channel, queries' and keys' apart)
//   (y_a, y_b) = (n_a cos - n_b sin, n_b cos + n_a sin) for the pairs (a, b) of the first `rot` channels,
//   y = n elsewhere; the angle of pair p is positions[t] * inv_freq[p].
// Pairs are (p, p + rot/2), or (2p, 2p + 1) when interleaved.  The gradient turns dy back by the same angle
// into dn, then dw = sum dn x r, dx = r (w dn - x r mean(w dn x r)).
//
// A lane takes 8 channels of a row, as two quads placed so that both channels of a pair are its own: no
// exchange for the rotation, only the row sum crosses lanes (2^ceil(log2(D/8)) lanes to a row).  The angle is
// taken in fp64, reduced by whole turns there, and its sine and cosine in fp32 (far positions keep
// their digits); a token's rot/2 angles are computed once per block and shared by its heads through shared
// memory.  HBM-bound: each row is read once and written once.
#include <math.h>

#include "ssd.h"
#include "ssd_common.cuh"

namespace ssd {
namespace rope {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

struct Args {
    int64_t tokens;
    int heads[2], dim, rot;  // queries, keys
    int interleaved;
    float eps;
    int64_t rs[2];           // elements between tokens of q and k
    const void* x[2];
    const float* w[2];
    const int64_t* positions;
    const float* inv_freq;
    void* y[2];              // forward outputs; backward: dx
    const void* dy[2];       // backward: gradients of the outputs
    float* part;             // backward: [blocks][2][dim] partial weight gradients
    float* dw[2];
};

__device__ __forceinline__ void load4(const float* p, float* v) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* v) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xFFFF0000u);
    v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store4(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&b));
}

// cos and sin of position * frequency: the product and the removal of whole turns in fp64 (two-part 2 pi), the
// functions in fp32 on the remainder in [-pi, pi].
__device__ __forceinline__ float2 turn(int64_t position, float inv_freq) {
    const double a = (double)position * (double)inv_freq;
    const double n = rint(a * 0.15915494309189535);  // 1 / (2 pi)
    const double r = fma(-n, 2.4492935982947064e-16, fma(-n, 6.283185307179586, a));
    float s, c;
    sincosf((float)r, &s, &c);
    return make_float2(c, s);
}

// The lane's channels: quads at lo and hi; `turned` when they are pairs of the rotated part.
struct Lane {
    int lo, hi, angle;  // first channels of the two quads, index of their first angle
    bool live, turned;
};
__device__ __forceinline__ Lane lane_of(int item, int dim, int rot, bool interleaved) {
    Lane l;
    l.live = item < dim / 8;
    l.turned = item < rot / 8;
    const bool halves = l.turned && !interleaved;
    l.lo = halves ? 4 * item : 8 * item;
    l.hi = halves ? rot / 2 + 4 * item : 8 * item + 4;
    l.angle = 4 * item;
    return l;
}
// Turns the lane's two quads by its four angles (c, s); dir = -1 turns back.
__device__ __forceinline__ void rotate(float* lo, float* hi, const float2* cs, bool interleaved, float dir) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float& a = interleaved ? (e < 2 ? lo[2 * e] : hi[2 * e - 4]) : lo[e];
        float& b = interleaved ? (e < 2 ? lo[2 * e + 1] : hi[2 * e - 3]) : hi[e];
        const float c = cs[e].x, s = dir * cs[e].y, x = a, y = b;
        a = x * c - y * s;
        b = y * c + x * s;
    }
}
template <int LPR> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Blocks walk the tokens; a block's warps share a token's head rows, 32 / LPR rows to a warp at a time.
template <typename T, int LPR, bool kInter, bool kBackward>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(Args a) {
    constexpr int RPW = 32 / LPR, RPB = RPW * kWarps;
    __shared__ float2 turns[128];
    __shared__ float sred[kBackward ? kThreads * 8 : 1];
    const int tid = threadIdx.x, lane = tid & 31;
    const int sub = (tid >> 5) * RPW + lane / LPR;  // this lane's row within a pass of the block
    const Lane at = lane_of(lane % LPR, a.dim, a.rot, kInter);
    float w[2][8], dw[2][8];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[p][e] = at.live ? a.w[p][(e < 4 ? at.lo : at.hi - 4) + e] : 0.f;
            dw[p][e] = 0.f;
        }
    const float inv_dim = 1.f / (float)a.dim;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        __syncthreads();
        if (tid < a.rot / 2) turns[tid] = turn(a.positions[t], a.inv_freq[tid]);
        __syncthreads();
        float2 cs[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) cs[e] = at.turned ? turns[at.angle + e] : make_float2(1.f, 0.f);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const T* x = static_cast<const T*>(a.x[p]) + t * a.rs[p];
            const int64_t out = t * a.heads[p] * a.dim;
            T* y = static_cast<T*>(a.y[p]) + out;
            const T* dy = kBackward ? static_cast<const T*>(a.dy[p]) + out : nullptr;
            for (int h0 = 0; h0 < a.heads[p]; h0 += RPB) {
                const int h = h0 + sub;
                const bool live = at.live && h < a.heads[p];
                float v[8], g[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = g[e] = 0.f;
                if (live) {
                    load4(x + h * a.dim + at.lo, v);
                    load4(x + h * a.dim + at.hi, v + 4);
                    if (kBackward) {
                        load4(dy + h * a.dim + at.lo, g);
                        load4(dy + h * a.dim + at.hi, g + 4);
                    }
                }
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
                const float r = rsqrtf(row_sum<LPR>(ss) * inv_dim + a.eps);
                if (!kBackward) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = v[e] * r * w[p][e];
                    if (at.turned) rotate(v, v + 4, cs, kInter, 1.f);
                } else {
                    if (at.turned) rotate(g, g + 4, cs, kInter, -1.f);
                    float m = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[e] *= r;
                        dw[p][e] = fmaf(g[e], v[e], dw[p][e]);
                        g[e] *= w[p][e];
                        m = fmaf(g[e], v[e], m);
                    }
                    m = row_sum<LPR>(m) * inv_dim;
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = r * (g[e] - v[e] * m);
                }
                if (live) {
                    store4(y + h * a.dim + at.lo, v);
                    store4(y + h * a.dim + at.hi, v + 4);
                }
            }
        }
    }
    if (kBackward) {
        // the block's weight gradients: rows in order, one channel of one tensor per thread
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (at.live) sred[sub * a.dim + (e < 4 ? at.lo : at.hi - 4) + e] = dw[p][e];
            __syncthreads();
            for (int c = tid; c < a.dim; c += kThreads) {
                float s = 0.f;
                for (int i = 0; i < RPB; ++i) s += sred[i * a.dim + c];
                a.part[((size_t)blockIdx.x * 2 + p) * a.dim + c] = s;
            }
        }
    }
}

// dw[p][c] = sum of the blocks' partials in order: 8 warps take a share of the blocks each, then are joined.
__global__ void __launch_bounds__(256) weight_grad_kernel(const float* part, int blocks, int dim, float* dwq,
                                                          float* dwk) {
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, p = blockIdx.y;
    float t = 0.f;
    if (c < dim)
        for (int b = warp; b < blocks; b += 8) t += part[((size_t)b * 2 + p) * dim + c];
    s[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && c < dim) {
        for (int i = 1; i < 8; ++i) t += s[i][lane];
        (p == 0 ? dwq : dwk)[c] = t;
    }
}

// Blocks of a backward launch: a few per SM, each over a share of the tokens, so that the partial sums stay few.
constexpr int kBackwardBlocks = 148 * 4;
int backward_blocks(int64_t tokens) { return (int)(tokens < kBackwardBlocks ? tokens : kBackwardBlocks); }

template <typename T, bool kBackward, bool kInter>
cudaError_t launch_lpr(const Args& a, unsigned blocks, cudaStream_t st) {
    if (a.dim <= 8) qk_norm_rope_kernel<T, 1, kInter, kBackward><<<blocks, kThreads, 0, st>>>(a);
    else if (a.dim <= 16) qk_norm_rope_kernel<T, 2, kInter, kBackward><<<blocks, kThreads, 0, st>>>(a);
    else if (a.dim <= 32) qk_norm_rope_kernel<T, 4, kInter, kBackward><<<blocks, kThreads, 0, st>>>(a);
    else if (a.dim <= 64) qk_norm_rope_kernel<T, 8, kInter, kBackward><<<blocks, kThreads, 0, st>>>(a);
    else if (a.dim <= 128) qk_norm_rope_kernel<T, 16, kInter, kBackward><<<blocks, kThreads, 0, st>>>(a);
    else qk_norm_rope_kernel<T, 32, kInter, kBackward><<<blocks, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}
template <bool kBackward> cudaError_t launch(const Args& a, ssd_dtype dtype, cudaStream_t st) {
    const unsigned blocks = kBackward ? backward_blocks(a.tokens)
                                      : (unsigned)(a.tokens < 148 * 64 ? a.tokens : 148 * 64);
    cudaError_t e;
    if (dtype == SSD_F32)
        e = a.interleaved ? launch_lpr<float, kBackward, true>(a, blocks, st)
                          : launch_lpr<float, kBackward, false>(a, blocks, st);
    else
        e = a.interleaved ? launch_lpr<__nv_bfloat16, kBackward, true>(a, blocks, st)
                          : launch_lpr<__nv_bfloat16, kBackward, false>(a, blocks, st);
    if (e != cudaSuccess || !kBackward) return e;
    weight_grad_kernel<<<dim3((a.dim + 31) / 32, 2), 256, 0, st>>>(a.part, (int)blocks, a.dim, a.dw[0], a.dw[1]);
    return cudaGetLastError();
}

bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && na && nb && x < y + nb && y < x + na;
}

ssd_status check(const ssd_qk_dims* d, ssd_dtype dtype, float eps, const ssd_qk_strides* strides, Args* a) {
    if (!d) return SSD_ERR_NULL;
    if (dtype != SSD_F32 && dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (d->tokens < 0 || d->q_heads <= 0 || d->k_heads <= 0) return SSD_ERR_SHAPE;
    if (d->head_dim < 8 || d->head_dim > 256 || d->head_dim % 8 != 0) return SSD_ERR_SHAPE;
    if (d->rot_dim < 0 || d->rot_dim > d->head_dim || d->rot_dim % 8 != 0) return SSD_ERR_SHAPE;
    if ((int64_t)d->q_heads * d->head_dim > (1 << 24) || (int64_t)d->k_heads * d->head_dim > (1 << 24))
        return SSD_ERR_SHAPE;
    if (d->tokens > (1LL << 31) - 1 || !(eps >= 0.f) || !isfinite(eps)) return SSD_ERR_SHAPE;
    *a = Args{};
    a->tokens = d->tokens;
    a->heads[0] = d->q_heads; a->heads[1] = d->k_heads;
    a->dim = d->head_dim; a->rot = d->rot_dim;
    a->interleaved = d->interleaved != 0;
    a->eps = eps;
    a->rs[0] = (int64_t)d->q_heads * d->head_dim;
    a->rs[1] = (int64_t)d->k_heads * d->head_dim;
    if (strides) {
        const int64_t es = dtype == SSD_F32 ? 4 : 2;
        if (strides->q < a->rs[0] || strides->k < a->rs[1]) return SSD_ERR_SHAPE;
        if (strides->q > (1LL << 31) || strides->k > (1LL << 31)) return SSD_ERR_SHAPE;
        if (((strides->q | strides->k) * es) & 15) return SSD_ERR_ALIGN;
        a->rs[0] = strides->q;
        a->rs[1] = strides->k;
    }
    return SSD_OK;
}

}  // namespace
}  // namespace rope
}  // namespace ssd

using namespace ssd::rope;

extern "C" {

ssd_status ssd_qk_norm_rope(const ssd_qk_dims* d, ssd_dtype dtype, float eps, const ssd_qk_strides* strides,
                            const void* q, const void* k, const float* q_weight, const float* k_weight,
                            const int64_t* positions, const float* inv_freq, void* q_out, void* k_out, void* stream) {
    Args a;
    const ssd_status st = check(d, dtype, eps, strides, &a);
    if (st != SSD_OK) return st;
    if (!q_weight || !k_weight || (d->rot_dim > 0 && !inv_freq)) return SSD_ERR_NULL;
    if (d->tokens > 0 && (!q || !k || !q_out || !k_out || (d->rot_dim > 0 && !positions))) return SSD_ERR_NULL;
    for (const void* p : {q, k, (const void*)q_weight, (const void*)k_weight, (const void*)q_out, (const void*)k_out})
        if (reinterpret_cast<uintptr_t>(p) & 15u) return SSD_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(positions) & 7u) || (reinterpret_cast<uintptr_t>(inv_freq) & 3u))
        return SSD_ERR_ALIGN;
    if (d->tokens == 0) return SSD_OK;
    const uint64_t es = dtype == SSD_F32 ? 4 : 2, T = d->tokens;
    const uint64_t wq = (uint64_t)d->q_heads * d->head_dim, wk = (uint64_t)d->k_heads * d->head_dim;
    const uint64_t nq = ((T - 1) * a.rs[0] + wq) * es, nk = ((T - 1) * a.rs[1] + wk) * es;
    // a contiguous input may be its own output; any other overlap is refused
    const bool same_q = q == q_out && a.rs[0] == (int64_t)wq, same_k = k == k_out && a.rs[1] == (int64_t)wk;
    const struct { const void* p; uint64_t n; } out[2] = {{q_out, T * wq * es}, {k_out, T * wk * es}};
    if (overlap(out[0].p, out[0].n, out[1].p, out[1].n)) return SSD_ERR_UNSUPPORTED;
    for (int i = 0; i < 2; ++i)
        if ((overlap(out[i].p, out[i].n, q, nq) && !(i == 0 && same_q)) ||
            (overlap(out[i].p, out[i].n, k, nk) && !(i == 1 && same_k)) ||
            overlap(out[i].p, out[i].n, q_weight, d->head_dim * 4) ||
            overlap(out[i].p, out[i].n, k_weight, d->head_dim * 4) ||
            overlap(out[i].p, out[i].n, positions, T * 8) || overlap(out[i].p, out[i].n, inv_freq, d->rot_dim * 2))
            return SSD_ERR_UNSUPPORTED;
    a.x[0] = q; a.x[1] = k;
    a.w[0] = q_weight; a.w[1] = k_weight;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.y[0] = q_out; a.y[1] = k_out;
    return launch<false>(a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

size_t ssd_qk_norm_rope_backward_workspace_bytes(const ssd_qk_dims* d) {
    Args a;
    if (check(d, SSD_F32, 0.f, nullptr, &a) != SSD_OK) return 0;
    return (size_t)backward_blocks(d->tokens) * 2 * d->head_dim * 4;
}

ssd_status ssd_qk_norm_rope_backward(const ssd_qk_dims* d, ssd_dtype dtype, float eps, const ssd_qk_strides* strides,
                                     const void* dq_out, const void* dk_out, const void* q, const void* k,
                                     const float* q_weight, const float* k_weight, const int64_t* positions,
                                     const float* inv_freq, void* dq, void* dk, float* dq_weight, float* dk_weight,
                                     void* workspace, size_t workspace_bytes, void* stream) {
    Args a;
    const ssd_status st = check(d, dtype, eps, strides, &a);
    if (st != SSD_OK) return st;
    if (!q_weight || !k_weight || !dq_weight || !dk_weight || (d->rot_dim > 0 && !inv_freq)) return SSD_ERR_NULL;
    if (d->tokens > 0 && (!q || !k || !dq_out || !dk_out || !dq || !dk || (d->rot_dim > 0 && !positions)))
        return SSD_ERR_NULL;
    for (const void* p : {dq_out, dk_out, q, k, (const void*)q_weight, (const void*)k_weight, (const void*)dq,
                          (const void*)dk, (const void*)dq_weight, (const void*)dk_weight, (const void*)workspace})
        if (reinterpret_cast<uintptr_t>(p) & 15u) return SSD_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(positions) & 7u) || (reinterpret_cast<uintptr_t>(inv_freq) & 3u))
        return SSD_ERR_ALIGN;
    const uint64_t es = dtype == SSD_F32 ? 4 : 2, T = d->tokens;
    const uint64_t wq = (uint64_t)d->q_heads * d->head_dim, wk = (uint64_t)d->k_heads * d->head_dim;
    const uint64_t nw = (uint64_t)d->head_dim * 4;
    const size_t need = ssd_qk_norm_rope_backward_workspace_bytes(d);
    const struct { const void* p; uint64_t n; } in[] = {
        {q, T ? ((T - 1) * a.rs[0] + wq) * es : 0}, {k, T ? ((T - 1) * a.rs[1] + wk) * es : 0},
        {dq_out, T * wq * es}, {dk_out, T * wk * es}, {q_weight, nw}, {k_weight, nw}, {positions, T * 8},
        {inv_freq, (uint64_t)d->rot_dim * 2}, {workspace, need}},
        out[] = {{dq, T * wq * es}, {dk, T * wk * es}, {dq_weight, nw}, {dk_weight, nw}};
    for (int i = 0; i < 4; ++i) {
        for (int j = i + 1; j < 4; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return SSD_ERR_UNSUPPORTED;
        for (const auto& x : in)
            if (overlap(out[i].p, out[i].n, x.p, x.n)) return SSD_ERR_UNSUPPORTED;
    }
    if (need > 0 && (!workspace || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (d->tokens == 0) {  // no rows: the weight gradients are zero
        if (cudaMemsetAsync(dq_weight, 0, nw, cs) != cudaSuccess) return SSD_ERR_CUDA;
        return cudaMemsetAsync(dk_weight, 0, nw, cs) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    }
    a.x[0] = q; a.x[1] = k;
    a.w[0] = q_weight; a.w[1] = k_weight;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.y[0] = dq; a.y[1] = dk;
    a.dy[0] = dq_out; a.dy[1] = dk_out;
    a.part = static_cast<float*>(workspace);
    a.dw[0] = dq_weight; a.dw[1] = dk_weight;
    return launch<true>(a, dtype, cs) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
