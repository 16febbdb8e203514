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
// A lane takes 16 (or 8) channels of a row, as two runs placed so that both channels of a pair are its own: no
// exchange for the rotation, only the row sum crosses lanes.  Arithmetic is on pairs of fp32 values.  The angle is
// taken in fp64, reduced by whole turns there, and its sine and cosine in fp32 (far positions keep
// their digits); a token's rot/2 angles are computed once per block and shared by its heads through shared
// memory.  HBM-bound: each row is read once and written once.  32768 tokens x 128 rows of 64, bf16: 181 us, 5.9 TB/s (at
// two blocks to an SM instead of three 190); backward, 4096 tokens x 256 rows of 128: 152 us, 5.3 TB/s.
#include <math.h>

#include "ssd.h"
#include "ssd_common.cuh"
#include "ssd_internal.h"

namespace ssd {
namespace rope {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

struct Args {
    int64_t tokens;
    int heads[2], dim, rot;  // queries, keys
    int per;                 // tokens a block takes at a time
    uint32_t magic[2];       // ceil(2^32 / heads): row / heads by a multiplication (2 heads or more)
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

// A lane's channels: two runs of kRun at lo and hi, half of the rotated (or of the plain) part apart, so that the runs of
// neighbouring lanes lie side by side.  It holds them as kRun pairs (A_i, B_i): neighbours within a run when interleaved,
// else A the first run and B the second.
struct Lane {
    int lo, hi;
    bool live, turned;
};
template <int kRun> __device__ __forceinline__ Lane lane_of(int item, int dim, int rot) {
    Lane l;
    l.live = item < dim / (2 * kRun);
    l.turned = item < rot / (2 * kRun);
    const int base = l.turned ? 0 : rot, size = l.turned ? rot : dim - rot;
    l.lo = base + kRun * (item - (l.turned ? 0 : rot / (2 * kRun)));
    l.hi = l.lo + size / 2;
    return l;
}
// Channel of A_i (b = 0) or B_i (b = 1).
template <int kRun, bool kInter> __device__ __forceinline__ int channel(const Lane& l, int i, int b) {
    if (!kInter) return (b ? l.hi : l.lo) + i;
    const int e = 2 * i + b;
    return e < kRun ? l.lo + e : l.hi + e - kRun;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// A lane's values as loaded: 2 kRun of them.
template <typename T, int kRun> struct Raw {
    static constexpr int kWords = kRun * (int)sizeof(T) / 4;  // of a run
    uint32_t w[2][kWords];
    // The two runs on their way to this thread's place in shared memory (pieces of 16 or 8 bytes, those of the block's
    // threads side by side), and from there.
    static constexpr int kPiece = kWords == 2 ? 8 : 16, kPieces = 2 * kWords * 4 / kPiece;
    static constexpr int kBytes = 2 * kWords * 4;
    static __device__ __forceinline__ void fetch(uint8_t* place, const T* p, int lo, int hi) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            constexpr int per = kPieces / 2;
            const uint8_t* src = reinterpret_cast<const uint8_t*>(p + (i < per ? lo : hi)) + (i % per) * kPiece;
            const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(place + i * kThreads * kPiece));
            if constexpr (kPiece == 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
        }
    }
    __device__ __forceinline__ void take(const uint8_t* place) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            constexpr int per = kPieces / 2, words = kPiece / 4;
            const uint8_t* q = place + i * kThreads * kPiece;
            uint32_t* d = &w[i / per][(i % per) * words];
            if constexpr (kPiece == 16) {
                const uint4 x = *reinterpret_cast<const uint4*>(q);
                d[0] = x.x; d[1] = x.y; d[2] = x.z; d[3] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(q);
                d[0] = x.x; d[1] = x.y;
            }
        }
    }
    __device__ __forceinline__ void store(T* p, int lo, int hi) const {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            T* q = p + (r ? hi : lo);
            if constexpr (kWords == 2) {
                *reinterpret_cast<uint2*>(q) = make_uint2(w[r][0], w[r][1]);
            } else {
#pragma unroll
                for (int i = 0; i < kWords; i += 4)
                    reinterpret_cast<uint4*>(q)[i / 4] = make_uint4(w[r][i], w[r][i + 1], w[r][i + 2], w[r][i + 3]);
            }
        }
    }
    __device__ __forceinline__ float get(int r, int i) const {  // value i of run r
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[r][i]);
        else return __uint_as_float(i & 1 ? w[r][i / 2] & 0xFFFF0000u : w[r][i / 2] << 16);
    }
    // As pairs: v[i] = (A_2i, A_2i+1), v[kRun / 2 + i] = (B_2i, B_2i+1).
    template <bool kInter> __device__ __forceinline__ void pairs(float2* v) const {
#pragma unroll
        for (int i = 0; i < kRun / 2; ++i) {
            if constexpr (kInter) {
                const int r = 4 * i >= kRun, e = 4 * i - r * kRun;
                v[i] = make_float2(get(r, e), get(r, e + 2));
                v[kRun / 2 + i] = make_float2(get(r, e + 1), get(r, e + 3));
            } else {
                v[i] = make_float2(get(0, 2 * i), get(0, 2 * i + 1));
                v[kRun / 2 + i] = make_float2(get(1, 2 * i), get(1, 2 * i + 1));
            }
        }
    }
    __device__ __forceinline__ void put2(int r, int e, float x, float y) {  // values e, e + 1 of run r (e even)
        if constexpr (sizeof(T) == 4) {
            w[r][e] = __float_as_uint(x);
            w[r][e + 1] = __float_as_uint(y);
        } else {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
            w[r][e / 2] = *reinterpret_cast<const uint32_t*>(&p);
        }
    }
    template <bool kInter> __device__ __forceinline__ void from(const float2* v) {
#pragma unroll
        for (int i = 0; i < kRun / 2; ++i) {
            const float2 a = v[i], b = v[kRun / 2 + i];
            if constexpr (kInter) {
                const int r = 4 * i >= kRun, e = 4 * i - r * kRun;
                put2(r, e, a.x, b.x);
                put2(r, e + 2, a.y, b.y);
            } else {
                put2(0, 2 * i, a.x, a.y);
                put2(1, 2 * i, b.x, b.y);
            }
        }
    }
};
// Turns the pairs by their angles; kBack turns back.
template <int kRun, bool kInter, bool kBack>
__device__ __forceinline__ void rotate(float2* v, const Lane& at, const float* cos, const float* sin) {
#pragma unroll
    for (int i = 0; i < kRun / 2; ++i) {
        const int r = 4 * i >= kRun, e = kInter ? (r ? at.hi : at.lo) / 2 + 2 * i - r * (kRun / 2) : at.lo + 2 * i;
        const float2 c = *reinterpret_cast<const float2*>(cos + e), s = *reinterpret_cast<const float2*>(sin + e);
        const float2 n = make_float2(-s.x, -s.y), a = v[i], b = v[kRun / 2 + i];
        v[i] = fma2(b, kBack ? s : n, mul2(a, c));
        v[kRun / 2 + i] = fma2(a, kBack ? n : s, mul2(b, c));
    }
}
template <int LPR> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

constexpr int kMaxTokens = 16;  // of a block at a time
constexpr int kAhead = 4;       // rows of a thread on their way or in work

template <typename T, int kRun, bool kBackward> constexpr int smem_bytes() {
    return kAhead * kThreads * Raw<T, kRun>::kBytes * (kBackward ? 2 : 1);
}

// Blocks with y = 0 take the queries, y = 1 the keys: `per` tokens at a time, their angles once, then all their head
// rows, 32 / LPR rows to a warp.  Rows come through shared memory by asynchronous copies, each thread's
// own kAhead rows deep: registers would hold too few loads in flight for HBM's latency.
template <typename T, int kRun, int LPR, bool kInter, bool kBackward>
__global__ void __launch_bounds__(kThreads, kBackward ? 2 : 3) qk_norm_rope_kernel(Args a) {
    constexpr int RPW = 32 / LPR, RPB = RPW * kWarps, N = kRun;  // N packed pairs of values in a lane
    using Row = Raw<T, kRun>;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ __align__(16) float cosv[kMaxTokens][128], sinv[kMaxTokens][128];
    const int tid = threadIdx.x, lane = tid & 31, p = blockIdx.y;
    const int sub = (tid >> 5) * RPW + lane / LPR;  // this lane's row within a pass of the block
    const Lane at = lane_of<kRun>(lane % LPR, a.dim, a.rot);
    const int half = a.rot / 2, heads = a.heads[p];
    const int64_t rs = a.rs[p];
    float2 w[N], dw[kBackward ? N : 1] = {};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int b = i >= N / 2, e = 2 * (i - b * (N / 2));
        w[i] = at.live ? make_float2(a.w[p][channel<kRun, kInter>(at, e, b)], a.w[p][channel<kRun, kInter>(at, e + 1, b)])
                       : both(0.f);
    }
    const float inv_dim = 1.f / (float)a.dim;
    auto place = [&](int i) { return ring + (i % kAhead) * kThreads * Row::kBytes * (kBackward ? 2 : 1) + tid * Row::kPiece; };
    for (int64_t t0 = (int64_t)blockIdx.x * a.per; t0 < a.tokens; t0 += (int64_t)gridDim.x * a.per) {
        const int nt = (int)min((int64_t)a.per, a.tokens - t0), rows = nt * heads, passes = (rows + RPB - 1) / RPB;
        const T* x = static_cast<const T*>(a.x[p]) + t0 * rs;
        const int64_t out = t0 * heads * a.dim;
        T* y = static_cast<T*>(a.y[p]) + out;
        const T* dy = kBackward ? static_cast<const T*>(a.dy[p]) + out : nullptr;
        auto token_of = [&](int r) { return nt == 1 ? 0 : heads == 1 ? r : (int)__umulhi((uint32_t)r, a.magic[p]); };
        auto fetch = [&](int i) {
            const int r = sub + i * RPB;
            if (at.live && r < rows) {
                const int t = token_of(r);
                Row::fetch(place(i), x + t * rs + (int64_t)(r - t * heads) * a.dim, at.lo, at.hi);
                if (kBackward) Row::fetch(place(i) + kThreads * Row::kBytes, dy + (int64_t)r * a.dim, at.lo, at.hi);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        for (int i = 0; i < kAhead - 1; ++i) fetch(i);
        __syncthreads();  // the angles before have been used
        for (int i = tid; i < nt * half; i += kThreads) {
            const int t = i / half, e = i - t * half;
            const float2 cs = turn(a.positions[t0 + t], a.inv_freq[e]);
            cosv[t][e] = cs.x;
            sinv[t][e] = cs.y;
        }
        __syncthreads();
        for (int i = 0; i < passes; ++i) {
            fetch(i + kAhead - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
            const int row = sub + i * RPB;
            const bool live = at.live && row < rows;
            float2 v[N], g[kBackward ? N : 1];
            if (live) {
                Row raw;
                raw.take(place(i));
                raw.template pairs<kInter>(v);
                if constexpr (kBackward) {
                    raw.take(place(i) + kThreads * Row::kBytes);
                    raw.template pairs<kInter>(g);
                }
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    v[e] = both(0.f);
                    if (kBackward) g[kBackward ? e : 0] = both(0.f);
                }
            }
            const int tk = live ? token_of(row) : 0;
            float2 ss = both(0.f);
#pragma unroll
            for (int e = 0; e < N; ++e) ss = fma2(v[e], v[e], ss);
            const float mean2 = row_sum<LPR>(ss.x + ss.y) * inv_dim;  // by all lanes: it shuffles
            const float r = row < rows ? rsqrtf(mean2 + a.eps) : 0.f;  // a place without a row stays zero where eps is
            if constexpr (!kBackward) {
#pragma unroll
                for (int e = 0; e < N; ++e) v[e] = mul2(mul2(v[e], both(r)), w[e]);
                if (at.turned) rotate<kRun, kInter, false>(v, at, cosv[tk], sinv[tk]);
            } else {
                if (at.turned) rotate<kRun, kInter, true>(g, at, cosv[tk], sinv[tk]);
                float2 m2 = both(0.f);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    v[e] = mul2(v[e], both(r));
                    dw[e] = fma2(g[e], v[e], dw[e]);
                    g[e] = mul2(g[e], w[e]);
                    m2 = fma2(g[e], v[e], m2);
                }
                const float m = -row_sum<LPR>(m2.x + m2.y) * inv_dim;
#pragma unroll
                for (int e = 0; e < N; ++e) v[e] = mul2(fma2(v[e], both(m), g[e]), both(r));
            }
            if (live) {
                Row o;
                o.template from<kInter>(v);
                o.store(y + (int64_t)row * a.dim, at.lo, at.hi);
            }
        }
    }
    if constexpr (kBackward) {
        // the block's weight gradients: rows in order, one channel per thread; the ring has room for a float of every
        // channel of every lane
        float* sred = reinterpret_cast<float*>(ring);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int b = i >= N / 2, e = 2 * (i - b * (N / 2));
            if (at.live) {
                sred[sub * a.dim + channel<kRun, kInter>(at, e, b)] = dw[i].x;
                sred[sub * a.dim + channel<kRun, kInter>(at, e + 1, b)] = dw[i].y;
            }
        }
        __syncthreads();
        for (int c = tid; c < a.dim; c += kThreads) {
            float s = 0.f;
            for (int i = 0; i < RPB; ++i) s += sred[i * a.dim + c];
            a.part[((size_t)blockIdx.x * 2 + p) * a.dim + c] = s;
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
// Tokens of a block at a time: more share the start of a group (its angles, its first rows' latency), but not at the cost
// of idle SMs; few enough for row / heads by multiplication (rows * heads < 2^32).
int tokens_per_block(int64_t tokens, int heads) {
    const int64_t n = tokens / (148 * 4);
    if (heads > 8192 || n < 1) return 1;
    return n > kMaxTokens ? kMaxTokens : (int)n;
}

template <typename T, int kRun, int LPR, bool kInter, bool kBackward>
cudaError_t launch_one(const Args& a, unsigned blocks, cudaStream_t st) {
    constexpr int bytes = smem_bytes<T, kRun, kBackward>();
    const cudaError_t e = allow_smem<qk_norm_rope_kernel<T, kRun, LPR, kInter, kBackward>>(bytes);
    if (e != cudaSuccess) return e;
    qk_norm_rope_kernel<T, kRun, LPR, kInter, kBackward><<<dim3(blocks, 2), kThreads, bytes, st>>>(a);
    return cudaGetLastError();
}
// Runs of 8 channels where the head and its rotated part are made of them, else of 4 (twice the lanes to a row).
template <typename T, bool kBackward, bool kInter>
cudaError_t launch_lpr(const Args& a, unsigned blocks, cudaStream_t st) {
#define SSD_QK_CASE(RUN, LPR) \
    if (a.dim <= 2 * RUN * LPR) return launch_one<T, RUN, LPR, kInter, kBackward>(a, blocks, st);
    if (sizeof(T) == 2 && a.dim % 16 == 0 && a.rot % 16 == 0) {
        constexpr int run = sizeof(T) == 2 ? 8 : 4;
        SSD_QK_CASE(run, 2)
        SSD_QK_CASE(run, 4)
        SSD_QK_CASE(run, 8)
        SSD_QK_CASE(run, 16)
    }
    SSD_QK_CASE(4, 4)
    SSD_QK_CASE(4, 8)
    SSD_QK_CASE(4, 16)
    SSD_QK_CASE(4, 32)
#undef SSD_QK_CASE
    return cudaErrorInvalidValue;
}
template <bool kBackward> cudaError_t launch(const Args& a, ssd_dtype dtype, cudaStream_t st) {
    const int64_t groups = (a.tokens + a.per - 1) / a.per;
    const unsigned blocks = kBackward ? backward_blocks(a.tokens) : (unsigned)(groups < 148 * 64 ? groups : 148 * 64);
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
    a->per = tokens_per_block(d->tokens, d->q_heads > d->k_heads ? d->q_heads : d->k_heads);
    for (int i = 0; i < 2; ++i) a->magic[i] = (uint32_t)(((1ull << 32) + a->heads[i] - 1) / a->heads[i]);
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
        {inv_freq, (uint64_t)d->rot_dim * 2}},
        out[] = {{dq, T * wq * es}, {dk, T * wk * es}, {dq_weight, nw}, {dk_weight, nw}, {workspace, need}};
    for (int i = 0; i < 5; ++i) {
        for (int j = i + 1; j < 5; ++j)
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
