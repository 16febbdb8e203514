// ssd_linear_attn_tc.cu -- decayed linear attention on the sm_100a tensor cores (bf16 rows).
//
// One CTA per (64 value channels, head, sequence or segment) walks its rows in chunks of C = 128:
//   P  = (Q K^T) . D,  D_ij = qk_scale e^{l(i-j)} for j <= i, else 0      [C x C]    tcgen05, K = Dk
//   Y1 = P V                                                              [C x 64]   tcgen05, K = C
//   Y2 = Q S                                                              [C x 64]   tcgen05, K = Dk
//   dS = K^T V',  V'_j = w_scale e^{l(C-j-s)} v_j                         [Dk x 64]  tcgen05, K = C
//   o_i = Y1_i + inter_scale e^{l(i+s)} Y2_i,   S <- e^{lC} S + dS
// (rows i counted in time order; against the time the tile's rows are counted from its end and the mask is
// the upper triangle).  Widths below 128 run in the same tiles: the tensor maps fill with zeros.
//
// Because the decay is a constant of the head, D, w and the output coefficients are the same for every chunk:
// each thread computes its 64 mask entries, its row weight and its coefficient once and keeps them in
// registers, so a score costs one multiply and half a conversion.  The state S is held in fp32 in the
// registers of two warpgroups (32 channels of a key row per thread), dS is computed from zero each chunk: no
// accumulator is carried through the tensor cores, and nothing but those warps' multiply-adds depends on the
// chunk before.
//
// Roundings: scores (times their decay) to bf16, the A operand of Y1; the copy of S that Y2 reads to bf16 (S itself stays
// fp32); both to two bf16 parts in a sequence or segment of one chunk, whose few outputs may share their errors; o once.  V' is cut
// into bf16 parts of 8 bits (v w = hi + mid + lo): two (16 bits) where S only feeds bf16 outputs, all three (24 bits)
// where what the second leaves would show in a state that the caller gets, so that such a state is as exact as fp32 sums.
//
// Values that are not finite: what the mask multiplies by zero (scores behind the diagonal, and in P V the rows behind an
// output's own) may be NaN or infinite, and would make outputs NaN that do not depend on it.  A product of such a value with
// zero is NaN, so no output that is finite is wrong: the warps that write them watch for NaN, and an item that had one is done
// again carefully.  There the warps of the scores take what is not finite out of V before P V, start Y1 as NaN where an output
// depends on it, else as zero, and make the scores behind the diagonal zero before the mask (4 x 8192 rows of 64 heads, the
// second half of them NaN: 974 us, 299 without).
//
// 28 warps, one CTA per SM (224 KB of shared memory, 512 TMEM columns):
//   0-7   P: two warpgroups, 64 columns each: TMEM -> mask -> bf16 back into the same TMEM columns (A operand)
//   8-15  V' (shared memory -> shared memory), 32 channels each; the same threads zero the rows behind a sequence's end
//         in K and V.  Where states alone are wanted there are no scores, so 0-15 make V', 16 channels each, and it has two
//         places, so that the next is made while the product reads the last (one prompt of 8191 rows: 78 -> 76 us)
//   16-23 S: TMEM -> registers -> shared memory, and o: TMEM -> registers -> global, a row per thread in 32-byte stores;
//         32 channels each
//   24    TMA: K, V, Q of a chunk, two or three stages
//   25    tcgen05.mma
//   26    the CTA's items
//   27    tells where V is, for the items that are done again
// Q, K, V are read once (Q and K once for each 64 value channels, the second time from L2), o written once.  Where heads
// are many the power limit bounds it: 2 x 8192 rows of 74 heads 128 x 64 take 182 us (5.1 TB/s) at the 1365 MHz that it
// leaves, and 151 us (6.2 TB/s) on zeros, which draw less, at 1965 MHz; 4 x 8192 rows of 64 heads 333 us.  Where they are
// few, the chain scores - mask - products - outputs of a chunk does: one prompt of 8191 rows, 16 heads 128 x 128, 74 us.
#include "ssd_common.cuh"
#include "ssd_internal.h"
#include "ssd_linear_attn.h"
#include "ssd_sm100.cuh"

extern __shared__ __align__(1024) unsigned char ssd_la_smem[];

namespace ssd {
namespace la {
namespace {

using namespace ssd::sm100;

constexpr int C = 128, DVB = 64, kHalf = 32;
constexpr int kWarpOut = 16, kWarpTma = 24, kWarpMma = 25, kWarpItem = 26, kThreads = 28 * 32;
constexpr int kRegisters = 72;  // of a thread at launch
constexpr uint32_t kBox = 16384;                 // 128 rows of 128 bytes
constexpr uint32_t OFF_VP = 10 * kBox;           // behind the stages; V': up to three boxes
constexpr uint32_t OFF_S = OFF_VP + 3 * kBox;    // bf16 copy of S, [128 key rows][64 channels]
// Without outputs the stages end at 9 boxes and there is no copy of S: two places of two boxes for V', one of its third part.
constexpr uint32_t OFF_VP2 = 9 * kBox, OFF_V3 = OFF_S;
constexpr uint32_t OFF_BAR = OFF_S + kBox;
constexpr uint32_t OFF_STOP = OFF_BAR + 256, OFF_TMEM = OFF_BAR + 264, OFF_ANSWER = OFF_BAR + 272, OFF_ITEM = OFF_BAR + 288;
constexpr uint32_t OFF_ORDER = OFF_BAR + 512;
constexpr int kSorted = 64;   // packed sequences that are taken longest first
// The first row of a chunk, in scan order, with a value in a channel of V that is not finite (C: none); how many items are to be
// done again, how many of them were while others were left, four items' notes of it (an item's is cleared by the one
// before it), and the queue of them.
constexpr uint32_t OFF_WILD = OFF_ORDER + kSorted, OFF_REDO = OFF_WILD + DVB * 4, OFF_QUEUE = OFF_REDO + 48;
constexpr int kQueue = 8;     // no more than the ring's places are unfinished when the item warp looks, and as many when it has
constexpr uint32_t kSmemBytes = OFF_QUEUE + kQueue * 52 + 1024;  // + alignment of the base
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a block");
// KFREE, QFREE, VFREE: the products that read a stage's tile are complete.
// PREADY: without outputs, where there are no scores, V' is ready in its second place (VREADY: in its first).  One barrier for
// both would be completed twice before the products' warp looks, and take a fast warp's arrival for a slow one's.
constexpr int kStages = 3;  // at most
enum Bar { FULL = 0, KFREE = 3, QFREE = 6, VFREE = 9, DSFULL = 12, DSREAD = 14, PFULL = 16, PREADY, VREADY, SREADY, Y2DONE, YFULL,
           EPI, MMADONE, NEXT, LASTLOAD, IFULL, IEMPTY = IFULL + 3, kBars = IEMPTY + 3,
           GUARD = DSREAD, AGREE };  // with outputs, where dS is not waited for
static_assert(kBars * 8 <= 256, "the barriers' place");
// TMEM columns: scores (their bf16 form takes the place of each 16), Y1, Y2, dS (two buffers of two parts)
constexpr uint32_t COL_P = 0, COL_Y1 = 128, COL_Y2 = 192, COL_DS = 256;

// Up to three scans in one launch (a gradient's), their blocks one behind the other.
constexpr int kMaxScans = 3;
struct Scan {
    CUtensorMap tq, tk, tv;
    ScanArgs a;
    unsigned blocks;
};
struct Params {
    Scan scan[kMaxScans];
};

// Moves registers between warpgroups.  Launched with 896 x 72; with outputs 256 x 112 (scores) + 256 x 40 (V') + 256 x 80
// (S and outputs) + 128 x 40, without them 512 x 64 (V') + 256 x 88 + 128 x 72: never more than launched.
template <int N> __device__ __forceinline__ void regs_more() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void regs_fewer() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// Waits for the phase of `parity`, for so many clock cycles at most; false when they have passed, or at once when *stop is set.
// The roles wait at some forty places, each a copy of this: the kernel's speed depends on its code's size (with a wait of
// twice the instructions 4 x 1000 rows of 32 heads 128 x 128 take 46 us instead of 44).
constexpr int64_t kWait = 4000000000;        // 2 s at 1965 MHz
constexpr int64_t kItemWait = 50 * kWait;    // the longest item is a whole sequence
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int* stop, int64_t cycles = kWait) {
    if (mbar_try_wait(bar, parity)) return true;
    const int64_t t0 = clock64();
    while (!mbar_try_wait(bar, parity))
        if ((stop && *stop) || clock64() - t0 > cycles) return false;
    return true;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* stop) {
    return __all_sync(0xffffffffu, bar_wait(bar, parity, stop));
}
// A CTA's work: one (64 value channels, head, sequence or segment) behind the other.  The item warp announces
// them in a ring of kItems places that the other roles read in the same order, each at its own pace.
constexpr int kItems = 3;
struct Item {
    int scan, h, dv0;  // scan < 0: no more
    int slot, seq;
    int row0, nc, last;  // first row, chunks, rows of the chunk that ends the sequence (or segment)
    int third;           // the last chunks, in scan order, whose V' needs its third part
    int rev;
    int careful;         // done again, see above
    int index;           // among the CTA's items that have chunks
    float l;
};
static_assert(sizeof(Item) * kItems <= 512 - 288 && sizeof(Item) <= 52, "the ring's place and the queue's");
// The ring of tile stages, as each role follows it.  A stage is the K boxes (one per 64 of Dk), the V box and the Q
// boxes of a chunk: three boxes or fewer leave room for three stages, Q and K of Dk > 64 for two.  Where the next
// item's stages are cut differently the ring starts over at stage 0, when the loads have seen all others out.
struct Ring {
    int s = 0, kb = 0, count = 0;  // stage, K boxes, stages
    uint32_t phases = 0;           // a bit for each stage
    __device__ __forceinline__ bool cut(int Dk, bool q) {  // whether the cut changed
        const int k = Dk > 64 ? 2 : 1;
        if (k == kb) return false;
        kb = k;
        count = (q && k == 2) ? 2 : 3;
        s = 0;
        return true;
    }
    __device__ __forceinline__ uint32_t phase() const { return (phases >> s) & 1; }
    __device__ __forceinline__ int after() const { return s + 1 == count ? 0 : s + 1; }
    __device__ __forceinline__ void step() {
        phases ^= 1u << s;
        s = after();
    }
    __device__ __forceinline__ uint32_t k(bool q) const { return (uint32_t)s * (kb + 1 + (q ? kb : 0)) * kBox; }
    __device__ __forceinline__ uint32_t v(bool q) const { return k(q) + kb * kBox; }
    __device__ __forceinline__ uint32_t q(bool has) const { return v(has) + kBox; }
};
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}
// D[tmem] (+)= A[tmem] * B[smem]^T: the A operand's rows are TMEM lanes, two bf16 to a column.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}
// D (+)= A B over K = 64: a K-major A of one 64-wide box, B alike or (kBmn) MN-major with 128-byte rows.
template <bool kBmn>
__device__ __forceinline__ void mma_k64(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) mma_bf16(d, a + k * 2, b + k * (kBmn ? 128 : 2), idesc, accumulate || k > 0);
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void store32(void* p, const uint32_t (&r)[8]) {  // 32-byte aligned
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// Stores the first `n` (a multiple of 8, or none) of 16 channels.
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&v)[16], int n, bool wide) {
    uint32_t r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = pack_bf2(v[2 * j], v[2 * j + 1]);
    if (wide && n >= 16) {
        store32(p, r);
    } else {
        if (n >= 8) *reinterpret_cast<uint4*>(p) = make_uint4(r[0], r[1], r[2], r[3]);
        if (n >= 16) *reinterpret_cast<uint4*>(p + 8) = make_uint4(r[4], r[5], r[6], r[7]);
    }
}
__device__ __forceinline__ void store16(float* p, const float (&v)[16], int n, bool wide) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        uint32_t r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(v[8 * b + j]);
        if (n < 8 * b + 8) break;
        if (wide) {
            store32(p + 8 * b, r);
        } else {
            *reinterpret_cast<uint4*>(p + 8 * b) = make_uint4(r[0], r[1], r[2], r[3]);
            *reinterpret_cast<uint4*>(p + 8 * b + 4) = make_uint4(r[4], r[5], r[6], r[7]);
        }
    }
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Asks the hardware for a block of this grid that has not started (its 16-byte answer arrives on `bar`); the running
// CTA then does that block's work and the block is never launched.
__device__ __forceinline__ void ask_next_block(void* answer, uint64_t* bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(answer)),
                 "r"(smem_u32(bar))
                 : "memory");
}
// The block's index, or -1 when none is left.
__device__ __forceinline__ int64_t next_block(const void* answer) {
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
        : "=r"(got), "=r"(x)
        : "r"(smem_u32(answer))
        : "memory");
    return got ? (int64_t)x : -1;
}

// For items that are done again, by the eight warps of the scores.  16 rows of a V tile: what is not finite becomes zero, and
// `first` the first row, in scan order, that had such a value in each channel (C before).
__device__ __forceinline__ void tame(uint8_t* tv, int* first, int warp, int lane, bool rev) {
    int a = C, b = C;  // of this lane's two channels
    const int word = (lane & 3) * 4;
#pragma unroll 1
    for (int r0 = warp * 16; r0 < warp * 16 + 16; r0 += 4) {
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const uint32_t*>(tv + sw128_off(r0 + i, lane / 4) + word);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = rev ? C - 1 - r0 - i : r0 + i;
            const bool lo = (x[i] & 0x7F80u) == 0x7F80u, hi = (x[i] & 0x7F800000u) == 0x7F800000u;
            a = lo ? min(a, at) : a;
            b = hi ? min(b, at) : b;
            if (lo || hi)
                *reinterpret_cast<uint32_t*>(tv + sw128_off(r0 + i, lane / 4) + word) =
                    x[i] & ((lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u));
        }
    }
    if (a < C) atomicMin(first + 2 * lane, a);
    if (b < C) atomicMin(first + 2 * lane + 1, b);
}
// Then Y1 (32 of its channels): NaN where an output depends on such a value, else zero.
__device__ __forceinline__ void start_y1(uint32_t y1, const int* first, int at) {
#pragma unroll 1
    for (int d = 0; d < 32; d += 8) {
        uint32_t r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = first[d + i] <= at ? 0x7FC00000u : 0u;
        tmem_st8(y1 + d, r);
    }
}
// And of 64 columns of the scores, from tile column j0 on, those behind the diagonal and those from n on become zero (rows behind
// the sequence's end: elsewhere the zeros in V's place are enough).
__device__ __forceinline__ void trim(uint32_t p, int row, int j0, int n, bool rev) {
#pragma unroll 1
    for (int j = 0; j < 64; j += 8) {
        float v[8];
        tmem_ld8(p + j, v);
        tmem_wait_ld();
        uint32_t r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = j0 + j + i;
            r[i] = c < n && (rev ? c >= row : c <= row) ? __float_as_uint(v[i]) : 0u;
        }
        tmem_st8(p + j, r);
    }
    tmem_wait_st();
}

// kMode: see Mode.
template <int kMode>
__global__ void __launch_bounds__(kThreads, 1) scan_tc_kernel(const __grid_constant__ Params prm) {
    uint8_t* sm = ssd_la_smem + ((1024u - (smem_u32(ssd_la_smem) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
    volatile int* stop = reinterpret_cast<volatile int*>(sm + OFF_STOP);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + OFF_TMEM);
    uint8_t* answer = sm + OFF_ANSWER;
    Item* items = reinterpret_cast<Item*>(sm + OFF_ITEM);
    Item* queue = reinterpret_cast<Item*>(sm + OFF_QUEUE);
    volatile int* posted = reinterpret_cast<volatile int*>(sm + OFF_REDO);
    volatile int *odd = posted + 4, *served = posted + 1, *indexed = posted + 8;
    // Barriers of the items that are done again: the warps of the scores ask where V is; all of them have done their rows of it.
    uint64_t *asked = reinterpret_cast<uint64_t*>(sm + OFF_REDO + 8), *tamed = reinterpret_cast<uint64_t*>(sm + OFF_REDO + 40);
    volatile uint32_t* where = reinterpret_cast<volatile uint32_t*>(sm + OFF_REDO + 36);
    int* wild = reinterpret_cast<int*>(sm + OFF_WILD);
    constexpr bool kOut = kMode != kStates;
    constexpr int kMaxParts = kMode == kOutputs ? 2 : 3;  // of V'
    constexpr int kVWarps = kOut ? 8 : 16;

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (warp == kWarpMma) {
        if (lane == 0) {
            for (int i = 0; i < kBars; ++i)
                mbar_init(&bars[i], i == VREADY || (!kOut && i == PREADY) ? kVWarps
                                    : i == PREADY || i == SREADY || i == EPI || i == AGREE || (!kOut && i == DSREAD) ? 8
                                    : i >= IEMPTY ? (kOut ? 27 : 26)  // warps that read an item
                                                  : 1);
            mbar_init(asked, 8);
            mbar_init(tamed, 8);
            *stop = 0;
            *posted = *served = *indexed = 0;
            for (int i = 0; i < 4; ++i) odd[i] = 0;
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const int row = (warp & 3) * 32 + lane;  // TMEM lane of a worker thread
    const uint32_t lane_base = tmem + ((uint32_t)(warp & 3) << 21);

    // The end of a lap, for all warps; true: of the last.  The second lap is for the items that are to be done again and were
    // not yet when the first ended.
    int lap = 0;
    auto over = [&] {
        __syncwarp();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        return !kOut || lap++ == 1 || *posted == *served || *stop;
    };
    // Gives back a place of the ring, after the role has copied what it needs.
    auto leave = [&](int number) { warp_arrive(&bars[IEMPTY + number % kItems], lane); };
    // A place of the ring, or nullptr: no more, and the last lap is over.
    auto enter = [&](int& number) -> const Item* {
        for (;; ++number) {
            const int i = number % kItems;
            const bool ok = __all_sync(0xffffffffu, bar_wait(&bars[IFULL + i], (number / kItems) & 1, stop, kItemWait));
            if (ok && items[i].scan >= 0) return &items[i];
            if (!ok) *stop = 1;
            if (over()) return nullptr;
            leave(number);
        }
    };
    // Of a role one of whose waits gave up.
    auto give_up = [&] {
        *stop = 1;
        over();
    };
    // Whether the scores are kept in two bf16 parts: a lone chunk may have few outputs, which all share a score's error.
    auto two_parts = [](int nc) { return nc == 1; };
    // Whether the same holds for the state that its outputs start from: the copy of S is then written twice, what the first
    // leaves after the product with the first.
    auto two_copies = [&](const ScanArgs& a, int nc) { return kOut && two_parts(nc) && (kMode == kOutputs || a.init); };
    // the place of chunk c, in scan order, among the item's chunks; the rows of the chunk at a place
    auto place_of = [](bool rev, int nc, int c) { return rev ? nc - 1 - c : c; };
    auto rows_of = [](int place, int nc, int last) { return place == nc - 1 ? last : C; };

    if (warp >= kWarpTma) {
        if constexpr (kOut) regs_fewer<40>();
        if (warp == kWarpItem) {
            // ---- items ----
            const ScanArgs& call = prm.scan[0].a;  // a launch's scans have the same sequences
            const bool sorted = call.cu && call.seg_len == 0 && call.batch <= kSorted && gridDim.x > 148;
            uint8_t* order = sm + OFF_ORDER;
            if (sorted) {
                // Packed sequences are taken longest first, so that no long one starts when the other SMs run out of work (24
                // ragged prompts of 16384 rows in all, 40 heads: 137 -> 119 us when this was added): sequence i goes to the
                // place that the number of longer ones (and equal ones before it) gives.  More than kSorted are taken as they
                // come: of prompts of 200 rows and one of 4000, 16 heads, 64 take 75 us wherever it stands, 65 take 69 us
                // with it in front and 111 with it at the end.
                const int n = (int)call.batch;
                for (int i = lane; i < n; i += 32) {
                    const int len = (int)sequence_span(call, i).len;
                    int rank = 0;
                    for (int j = 0; j < n; ++j) {
                        const int other = (int)sequence_span(call, j).len;
                        rank += other > len || (other == len && j < i);
                    }
                    order[rank] = (uint8_t)i;
                }
                __syncwarp();
            }
            int put = 0, taken = 0;  // announced (the first lap's end too), and of the queue of items to be done again
            do {
                if (lane != 0) continue;
                int64_t block = blockIdx.x;
                auto announce = [&](const Item& it) {
                    const int i = put % kItems;
                    if (put >= kItems && !bar_wait(&bars[IEMPTY + i], ((put / kItems) - 1) & 1, stop, kItemWait)) return false;
                    items[i] = it;
                    items[i].index = *indexed;
                    if (it.nc > 0) *indexed = *indexed + 1;
                    mbar_arrive(&bars[IFULL + i]);
                    ++put;
                    return true;
                };
                // the loads of the item announced last are due to end
                auto loaded = [&] { return bar_wait(&bars[LASTLOAD], (put - lap - 1) & 1, stop, kItemWait); };
                auto again = [&] {
                    while (kOut && taken != *posted) {
                        __threadfence_block();
                        Item it = queue[taken++ % kQueue];
                        it.careful = 1;
                        if (!announce(it) || !loaded()) return false;
                    }
                    return true;
                };
                bool ok = true;
                if (lap == 1) ok = again();
                for (int asks = 0; lap == 0; ++asks) {
                    Item it;
                    it.scan = 0;
                    unsigned b = (unsigned)block;
                    while (b >= prm.scan[it.scan].blocks) b -= prm.scan[it.scan++].blocks;
                    const ScanArgs& a = prm.scan[it.scan].a;
                    const unsigned ndvb = (a.Dv + DVB - 1) / DVB;
                    it.dv0 = (int)(b % ndvb) * DVB;
                    it.h = (int)(b / ndvb % a.H);
                    it.slot = (int)(b / (ndvb * (unsigned)a.H));
                    if (sorted) it.slot = order[it.slot];
                    const Segment g = segment_of(a, it.slot);
                    if (a.cu && a.seg_len == 0 && it.h == 0 && it.dv0 == 0 && !sequence_span(a, it.slot).ok)
                        atomicOr(a.err, kErrBadSeqlens);
                    it.seq = (int)g.seq;
                    it.row0 = (int)g.row0;
                    it.nc = (int)((g.n + C - 1) / C);
                    it.last = (int)(g.n - (int64_t)(it.nc - 1) * C);
                    it.l = a.log_decay[it.h];
                    it.rev = a.reverse;
                    it.careful = 0;
                    // What the second part leaves (2^-16) shows in a state that the caller gets unless at least d rows follow
                    // with e^{l d} < 2^-8: l d < -6.
                    it.third = kMode == kOutputs || (kMode == kWhole && !a.final_state) ? 0
                               : it.l < 0.f ? (int)fminf(6.f / (C * -it.l) + 2.f, 1e9f)
                                            : 1 << 30;
                    // the next block is taken only when this item's last three loads are due: early enough to be announced
                    // by then, late enough that none waits here while another SM is idle
                    ok = (!g.ok || (announce(it) && loaded())) && again();
                    if (ok) {
                        mbar_arrive_expect_tx(&bars[NEXT], 16);
                        ask_next_block(answer, &bars[NEXT]);
                        ok = bar_wait(&bars[NEXT], asks & 1, nullptr);
                        block = next_block(answer);
                        fence_async_smem();  // read before the next answer is written
                    }
                    if (!ok || block < 0) break;
                }
                *served = taken;
                if (!ok) *stop = 1;
                Item end;
                end.scan = -1;
                end.nc = 0;
                if (!announce(end)) *stop = 1;
            } while (!over());
        } else if (warp == kWarpTma) {
            // ---- tile loads.  The whole warp runs this loop, so that addresses stay in uniform registers; one elected lane
            // issues.
            Ring ring;
            const Item* it;
            // a place's products are complete (at once where there were none)
            auto freed = [&](int bar, int i) { return warp_wait(&bars[bar + i], ((ring.phases >> i) & 1) ^ 1, stop); };
            bool ok = true;
            for (int k = 0; ok && (it = enter(k)) != nullptr; ++k) {
                const Scan& scan = prm.scan[__shfl_sync(0xffffffffu, it->scan, 0)];
                const ScanArgs& a = scan.a;
                const int dv0 = __shfl_sync(0xffffffffu, it->dv0, 0), nc = __shfl_sync(0xffffffffu, it->nc, 0);
                const int row0 = __shfl_sync(0xffffffffu, it->row0, 0), h = __shfl_sync(0xffffffffu, it->h, 0);
                auto stored = [&](int group) { return group == 1 ? h : h / group; };  // the stored head of a role
                const int hk = stored(a.gk), hv = a.gv == a.gk ? hk : stored(a.gv), hq = kOut ? stored(a.gq) : 0;
                const bool rev = a.reverse;
                leave(k);
                if (ring.cut(a.Dk, kOut) && k > 0)
                    for (int i = 0; i < kStages; ++i)
                        ok = ok && freed(KFREE, i) && (!kOut || freed(QFREE, i)) && freed(VFREE, i);
                if (nc == 0 && elect_one()) mbar_arrive(&bars[LASTLOAD]);
                for (int c = 0; ok && c < nc; ++c) {
                    const int s = ring.s, r = row0 + place_of(rev, nc, c) * C;
                    ok = freed(KFREE, s);
                    // each tile as soon as its place is free (and in any case: the bytes are expected)
                    if (elect_one()) {
                        if (c == max(0, nc - 3)) mbar_arrive(&bars[LASTLOAD]);
                        mbar_arrive_expect_tx(&bars[FULL + s], (ring.kb + 1 + (kOut ? ring.kb : 0)) * kBox);
                        tma_load_3d(sm + ring.k(kOut), &scan.tk, &bars[FULL + s], 0, hk, r);
                        if (ring.kb == 2) tma_load_3d(sm + ring.k(kOut) + kBox, &scan.tk, &bars[FULL + s], 64, hk, r);
                    }
                    __syncwarp();
                    if (kOut) {
                        ok = ok && freed(QFREE, s);
                        if (elect_one()) {
                            tma_load_3d(sm + ring.q(kOut), &scan.tq, &bars[FULL + s], 0, hq, r);
                            if (ring.kb == 2) tma_load_3d(sm + ring.q(kOut) + kBox, &scan.tq, &bars[FULL + s], 64, hq, r);
                        }
                        __syncwarp();
                    }
                    ok = ok && freed(VFREE, s);
                    if (elect_one()) tma_load_3d(sm + ring.v(kOut), &scan.tv, &bars[FULL + s], dv0, hv, r);
                    __syncwarp();
                    ring.step();
                }
            }
            if (!ok) give_up();
            // no load may be in flight when the CTA exits (each was consumed, unless a wait gave up)
            for (int i = 0; i < kStages; ++i) bar_wait(&bars[FULL + i], ((ring.phases >> i) & 1) ^ 1, nullptr, kWait / 20);
        } else if (warp == kWarpMma) {
            // ---- products.  The whole warp runs this loop, so that descriptors stay in uniform registers; one elected
            // lane issues.
            constexpr uint32_t ID_P = idesc_bf16_f32(128, 128, false, false);
            constexpr uint32_t ID_Y = idesc_bf16_f32(128, 64, false, true);
            constexpr uint32_t ID_DS = idesc_bf16_f32(128, 128, true, true), ID_DS3 = idesc_bf16_f32(128, 64, true, true);
            uint32_t base = smem_u32(sm);
            int cc = 0;  // the CTA's chunks over all its items
            int sc = 0;  // copies of S
            Ring ring;
            const Item* it;
            bool ok = true;
            for (int k = 0; ok && (it = enter(k)) != nullptr; ++k) {
                ring.cut(prm.scan[it->scan].a.Dk, kOut);
                const bool wide = ring.kb == 2;
                const int nc = it->nc, third = it->third;
                const bool twice = two_copies(prm.scan[it->scan].a, nc), careful = it->careful;
                leave(k);
                for (int c = 0; ok && c < nc; ++c, ++cc, ring.step()) {
                    const int s = ring.s;
                    // opaque to the compiler: descriptors are made where they are used, a few uniform adds each, instead
                    // of being kept (and spilled) over the loop
                    asm volatile("" : "+r"(base));
                    const uint32_t tk = base + ring.k(kOut), tv = base + ring.v(kOut), ds = tmem + COL_DS + (cc & 1) * 128;
                    const uint64_t dQ = sw128_desc(base + ring.q(kOut), 16, 1024);
                    if (!(ok = warp_wait(&bars[FULL + s], ring.phase(), stop))) break;
                    tc_fence_after();
                    if (kOut) {  // P = Q K^T (the product that read the scores before was issued before)
                        const uint64_t dK = sw128_desc(tk, 16, 1024);
                        if (elect_one()) {
                            mma_k64<false>(tmem + COL_P, dQ, dK, ID_P, 0);
                            if (wide) mma_k64<false>(tmem + COL_P, dQ + (kBox >> 4), dK + (kBox >> 4), ID_P, 1);
                            mma_commit(&bars[PFULL]);
                        }
                        __syncwarp();
                    }
                    // dS = K^T V' (its buffer was read before the S that the last Y2 waited for, if there is one): the parts lie one box
                    // behind the other, the first two are one product with 64 columns each, so that K is read once; the
                    // third adds to the second
                    ok = warp_wait(&bars[kOut || !(cc & 1) ? VREADY : PREADY], (kOut ? cc : cc >> 1) & 1, stop) &&
                         (kOut || cc < 2 || warp_wait(&bars[DSREAD + (cc & 1)], ((cc >> 1) - 1) & 1, stop));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t dKt = sw128_desc(tk, 16384, 1024);
                    const uint64_t dVP = sw128_desc(base + (kOut ? OFF_VP : OFF_VP2 + (cc & 1) * 2 * kBox), 16384, 1024);
                    const uint64_t dV3 = kOut ? dVP + 16 * 128 : sw128_desc(base + OFF_V3, 16384, 1024);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_bf16(ds, dKt + k * 128, dVP + k * 128, ID_DS, k > 0);
                        if (kMaxParts == 3 && nc - c <= third) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                mma_bf16(ds + 64, dKt + k * 128, dV3 + k * 128, ID_DS3, 1);
                        }
                        mma_commit(&bars[DSFULL + (cc & 1)]);
                        mma_commit(&bars[KFREE + s]);
                    }
                    __syncwarp();
                    if (kOut) {
                        // Y2 = Q S, once S is written and the outputs before have been read
                        ok = warp_wait(&bars[SREADY], sc & 1, stop) && (cc == 0 || warp_wait(&bars[EPI], (cc - 1) & 1, stop));
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t dS = sw128_desc(base + OFF_S, 16384, 1024);
                        if (elect_one()) {
                            mma_k64<true>(tmem + COL_Y2, dQ, dS, ID_Y, 0);
                            if (wide) mma_k64<true>(tmem + COL_Y2, dQ + (kBox >> 4), dS + 4 * 128, ID_Y, 1);
                            mma_commit(&bars[Y2DONE]);
                            if (!twice) mma_commit(&bars[QFREE + s]);
                        }
                        __syncwarp();
                        ++sc;
                        // Y1 = P V
                        if (!(ok = warp_wait(&bars[PREADY], cc & 1, stop))) break;
                        tc_fence_after();
                        const uint64_t dV = sw128_desc(tv, 16384, 1024);
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)  // the bf16 scores: 16 to the first 8 of every 16 columns
                                mma_bf16_ts(tmem + COL_Y1, tmem + COL_P + k * 16, dV + k * 128, ID_Y, k > 0 || careful);
                            if (two_parts(nc)) {  // and what they leave, in the other 8
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    mma_bf16_ts(tmem + COL_Y1, tmem + COL_P + k * 16 + 8, dV + k * 128, ID_Y, 1);
                            }
                            if (!twice) mma_commit(&bars[YFULL]);
                        }
                        __syncwarp();
                        if (twice) {  // Y2 += Q (what the first copy left of S)
                            if (!(ok = warp_wait(&bars[SREADY], sc & 1, stop))) break;
                            tc_fence_after();
                            if (elect_one()) {
                                mma_k64<true>(tmem + COL_Y2, dQ, dS, ID_Y, 1);
                                if (wide) mma_k64<true>(tmem + COL_Y2, dQ + (kBox >> 4), dS + 4 * 128, ID_Y, 1);
                                mma_commit(&bars[Y2DONE]);
                                mma_commit(&bars[QFREE + s]);
                                mma_commit(&bars[YFULL]);
                            }
                            __syncwarp();
                            ++sc;
                        }
                    }
                    if (elect_one()) mma_commit(&bars[VFREE + s]);
                    __syncwarp();
                }
            }
            if (!ok) give_up();
            // nothing may still be running on the tensor cores when TMEM is released
            if (elect_one()) mma_commit(&bars[MMADONE]);
            __syncwarp();
            bar_wait(&bars[MMADONE], 0, nullptr, kWait / 20);
        } else if (kOut) {
            // ---- where V is, of items that are done again, when the warps of the scores ask: they follow every chunk, while this one
            // skips other items' and is ahead of them, so that the parity of another barrier would tell it nothing
            int gc = 0;  // chunks of such items
            Ring ring;
            const Item* it;
            bool ok = true;
            for (int k = 0; ok && (it = enter(k)) != nullptr; ++k) {
                ring.cut(prm.scan[it->scan].a.Dk, kOut);
                const int nc = it->nc, careful = it->careful;
                leave(k);
                for (int c = 0; ok && c < nc; ++c, ring.step()) {
                    if (!careful) continue;
                    if (!(ok = warp_wait(asked, gc++ & 1, stop))) break;
                    wild[lane] = wild[lane + 32] = C;
                    if (lane == 0) *where = ring.v(kOut);
                    warp_arrive(&bars[GUARD], lane);
                }
            }
            if (!ok) give_up();
        } else {
            over();
        }
    } else if (kOut && warp < 8) {
        if constexpr (kOut) {
            regs_more<112>();
            // ---- scores: row `row`, columns 64 half .. 64 half + 63 ----
            const int j0 = (warp >> 2) * 64;
            int cc = 0, gc = 0;  // chunks, those of items that are done again
            const Item* it;
            bool ok = true;
            for (int k = 0; ok && (it = enter(k)) != nullptr; ++k) {
                const ScanArgs& a = prm.scan[it->scan].a;
                const int nc = it->nc, last = it->last;
                const float l = it->l;
                const bool rev = a.reverse, careful = it->careful;
                leave(k);
                // one factor e^l per step away from the diagonal (off by 127 fp32 roundings at most, far below bf16's)
                float m[64];
                const float el = decay_pow(l, 1);
                // distance of the half's column nearest the diagonal: the last one, against the time the first
                const int near = rev ? j0 - row : row - (j0 + 63);
                float cur = near > 0 ? a.qk_scale * decay_pow(l, near) : 0.f;
                auto next = [&](int i) {  // the factor i columns from there; 0 until the diagonal is reached
                    if (near + i == 0) cur = a.qk_scale;
                    else if (i > 0) cur *= el;
                    return cur;
                };
                if (rev) {
#pragma unroll
                    for (int i = 0; i < 64; ++i) m[i] = next(i);
                } else {
#pragma unroll
                    for (int i = 0; i < 64; ++i) m[63 - i] = next(i);
                }
                for (int c = 0; ok && c < nc; ++c, ++cc) {
                    const int n = rows_of(place_of(rev, nc, c), nc, last);
                    if (!(ok = warp_wait(&bars[PFULL], cc & 1, stop))) break;
                    tc_fence_after();
                    const uint32_t col = lane_base + COL_P + j0;
                    if (careful) {  // V' is made of V (dS is complete), and the outputs before have been read from Y1
                        ok = warp_wait(&bars[DSFULL + (cc & 1)], (cc >> 1) & 1, stop) &&
                             (cc == 0 || warp_wait(&bars[EPI], (cc - 1) & 1, stop));
                        if (!ok) break;
                        warp_arrive(asked, lane);
                        if (!(ok = warp_wait(&bars[GUARD], gc++ & 1, stop))) break;
                        tame(sm + *where, wild, warp, lane, rev);
                        fence_async_smem();
                        warp_arrive(tamed, lane);
                        if (!(ok = warp_wait(tamed, (gc - 1) & 1, stop))) break;
                        tc_fence_after();
                        start_y1(lane_base + COL_Y1 + j0 / 2, wild + j0 / 2, rev ? C - 1 - row : row);
                        trim(col, row, j0, n, rev);
                    }
#pragma unroll
                    for (int b = 0; b < 4; b += 2) {
                        float v[2][16];
                        tmem_ld16(col + b * 16, v[0]);
                        tmem_ld16(col + b * 16 + 16, v[1]);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t p[8];
                            const int j1 = (b + i) * 16;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float2 f = __fmul2_rn(make_float2(v[i][2 * j], v[i][2 * j + 1]),
                                                            make_float2(m[j1 + 2 * j], m[j1 + 2 * j + 1]));
                                v[i][2 * j] = f.x;
                                v[i][2 * j + 1] = f.y;
                                p[j] = pack_bf2(f.x, f.y);
                            }
                            tmem_st8(col + j1, p);  // over the columns just read
                            if (two_parts(nc)) {
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    p[j] = pack_bf2(v[i][2 * j] - bf_lo(p[j]), v[i][2 * j + 1] - bf_hi(p[j]));
                                tmem_st8(col + j1 + 8, p);
                            }
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    warp_arrive(&bars[PREADY], lane);
                }
            }
            if (!ok) give_up();
        }
    } else if (warp < kWarpOut) {
        // ---- V': tile row `row`, 64 * 4 / kVWarps of the 64 channels ----
        regs_fewer<kOut ? 40 : 64>();
        constexpr int kPieces = 32 / kVWarps;  // of 8 channels
        const int share = (warp >> 2) & (kVWarps / 4 - 1);
        int cc = 0;
        Ring ring;
        const Item* it;
        bool ok = true;
        for (int k = 0; ok && (it = enter(k)) != nullptr; ++k) {
            const ScanArgs& a = prm.scan[it->scan].a;
            ring.cut(a.Dk, kOut);
            const int nc = it->nc, last = it->last, third = it->third;
            const float l = it->l, w_scale = a.w_scale;
            const bool rev = a.reverse;
            leave(k);
            // weight of tile row `row` in the state behind a chunk of n rows
            auto weight = [&](int n) { return row < n ? w_scale * decay_pow(l, rev ? row + 1 : n - 1 - row) : 0.f; };
            const float w_full = weight(C);
            for (int c = 0; ok && c < nc; ++c, ++cc, ring.step()) {
                const int n = rows_of(place_of(rev, nc, c), nc, last);
                const bool three = kMaxParts == 3 && nc - c <= third;
                const float w = n == C ? w_full : weight(n);
                ok = warp_wait(&bars[FULL + ring.s], ring.phase(), stop);
                if (!ok) break;
                uint8_t* tv = sm + ring.v(kOut);
                if (row >= n) {  // behind the sequence's end: zeros
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t o = sw128_off(row, i);
                        const uint4 z = make_uint4(0, 0, 0, 0);
                        if (share < ring.kb) *reinterpret_cast<uint4*>(sm + ring.k(kOut) + share * kBox + o) = z;
                        if (i / kPieces == share) *reinterpret_cast<uint4*>(tv + o) = z;
                    }
                }
                // the product that reads the V' in this place is complete
                auto multiplied = [&](int chunk) {
                    return chunk < 0 || warp_wait(&bars[DSFULL + (chunk & 1)], (chunk >> 1) & 1, stop);
                };
                if (!(ok = multiplied(kOut ? cc - 1 : cc - 2))) break;
                uint8_t* vp = sm + (kOut ? OFF_VP : OFF_VP2 + (cc & 1) * 2 * kBox);
                auto piece = [&](int i, auto write) {  // 8 channels of V', cut into parts
                    const uint32_t o = sw128_off(row, share * kPieces + i);
                    const uint4 x = *reinterpret_cast<const uint4*>(tv + o);
                    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
                    uint32_t part[kMaxParts][4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float2 f = __fmul2_rn(make_float2(bf_lo(in[k]), bf_hi(in[k])), make_float2(w, w));
                        // a part is the upper half of the word: 8 bits cut off, the rest exact
#pragma unroll
                        for (int t = 0; t < kMaxParts; ++t) {
                            const uint32_t x0 = __float_as_uint(f.x), x1 = __float_as_uint(f.y);
                            part[t][k] = __byte_perm(x0, x1, 0x7632);
                            if (t + 1 < kMaxParts) f = __fadd2_rn(f, make_float2(-bf_hi(x0), -bf_hi(x1)));
                        }
                    }
#pragma unroll
                    for (int t = 0; t < kMaxParts; ++t)
                        write(t, o, make_uint4(part[t][0], part[t][1], part[t][2], part[t][3]));
                };
#pragma unroll 2
                for (int i = 0; i < kPieces; ++i)
                    piece(i, [&](int t, uint32_t o, uint4 p) {
                        if (t < 2 || (kOut && three)) *reinterpret_cast<uint4*>(vp + t * kBox + o) = p;
                    });
                if (!kOut && three) {  // the third part has one place, so it is made (anew) when that is free
                    if (!(ok = multiplied(cc - 1))) break;
#pragma unroll
                    for (int i = 0; i < kPieces; ++i)
                        piece(i, [&](int t, uint32_t o, uint4 p) {
                            if (t == 2) *reinterpret_cast<uint4*>(sm + OFF_V3 + o) = p;
                        });
                }
                fence_async_smem();
                warp_arrive(&bars[kOut || !(cc & 1) ? VREADY : PREADY], lane);
            }
        }
        if (!ok) give_up();
    } else {
        // ---- S: key row `row`, and the outputs: tile row `row`; 32 of the 64 channels ----
        regs_more<kOut ? 80 : 88>();
        const int half = (warp >> 2) & 1;
        float S[kHalf];
        int cc = 0, sc = 0;  // chunks, copies of S
        const Item* it;
        bool ok = true;
        auto publish = [&](bool rest) {  // the bf16 copy that Y2 reads, or what it leaves of S
            // over the copy before, once the product has read it
            ok = sc == 0 || warp_wait(&bars[Y2DONE], (sc - 1) & 1, stop);
            if (!ok) return;
            uint8_t* p = sm + OFF_S;
#pragma unroll
            for (int i = 0; i < kHalf / 8; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x = S[8 * i + 2 * j], y = S[8 * i + 2 * j + 1];
                    w[j] = pack_bf2(x, y);
                    if (rest) w[j] = pack_bf2(x - bf_lo(w[j]), y - bf_hi(w[j]));
                }
                *reinterpret_cast<uint4*>(p + sw128_off(row, half * 4 + i)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            fence_async_smem();
            warp_arrive(&bars[SREADY], lane);
            ++sc;
        };
        // the item is read from its place in the ring wherever it is needed, not kept in registers
        for (int k = 0; ok && (it = enter(k)) != nullptr; ++k) {
            bool finite = true;  // this thread's outputs
            const float decay_full = decay_pow(it->l, C);
            // this row of the state, where it is kept: among the sequences' or the segments'
            auto state_row = [&](const float* base, bool transposed) {
                const ScanArgs& a = prm.scan[it->scan].a;
                const int d0 = it->dv0 + half * kHalf;
                return base + (size_t)((kMode == kWhole ? it->seq : it->slot) * a.H + it->h) * a.Dk * a.Dv +
                       (transposed ? (size_t)d0 * a.Dk + row : (size_t)row * a.Dv + d0);
            };
            const int live = prm.scan[it->scan].a.Dv - (it->dv0 + half * kHalf);  // channels of this half
#pragma unroll
            for (int d = 0; d < kHalf; ++d) S[d] = 0.f;
            float e_full = 0.f;  // the outputs' coefficient of S
            if (kOut) {
                const ScanArgs& a = prm.scan[it->scan].a;
                e_full = a.inter_scale * decay_pow(it->l, it->rev ? C - 1 - row : row + 1);
                const float* init = kMode == kOutputs ? a.seg_state : a.init;
                const bool init_t = kMode == kWhole ? a.init_t : a.seg_t;
                if (init && row < a.Dk) {
                    const float* src = state_row(init, init_t);
                    if (init_t) {  // neighbouring lanes' values lie side by side
#pragma unroll
                        for (int d = 0; d < kHalf; ++d)
                            if (d < live) S[d] = src[d * a.Dk];
                    } else {  // a row per lane: the memory pipe takes a pass for each lane, so as few accesses as can be
#pragma unroll
                        for (int d = 0; d < kHalf; d += 4)
                            if (d < live) {
                                const float4 x = *reinterpret_cast<const float4*>(src + d);
                                S[d] = x.x; S[d + 1] = x.y; S[d + 2] = x.z; S[d + 3] = x.w;
                            }
                    }
                }
                if (it->nc > 0) publish(false);
                if (ok && two_copies(a, it->nc)) publish(true);
            }
            for (int c = 0; ok && c < it->nc; ++c, ++cc) {
                if (!(ok = warp_wait(&bars[DSFULL + (cc & 1)], (cc >> 1) & 1, stop))) break;
                tc_fence_after();
                const int place = place_of(it->rev, it->nc, c), n = rows_of(place, it->nc, it->last);
                const float decay = n == C ? decay_full : decay_pow(it->l, n);
#pragma unroll
                for (int b = 0; b < kHalf / 8; ++b) {
                    const uint32_t col = lane_base + COL_DS + (cc & 1) * 128 + half * kHalf + b * 8;
                    float x[8], y[8];
                    tmem_ld8(col, x);
                    tmem_ld8(col + 64, y);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        const float2 d = __fadd2_rn(make_float2(x[j], x[j + 1]), make_float2(y[j], y[j + 1]));
                        const float2 f = __ffma2_rn(make_float2(decay, decay), make_float2(S[b * 8 + j], S[b * 8 + j + 1]), d);
                        S[b * 8 + j] = f.x;
                        S[b * 8 + j + 1] = f.y;
                    }
                }
                tc_fence_before();
                if constexpr (!kOut) {
                    warp_arrive(&bars[DSREAD + (cc & 1)], lane);
                } else {
                    if (c + 1 < it->nc) {
                        publish(false);
                        if (!ok) break;
                    }
                    if (!(ok = warp_wait(&bars[YFULL], cc & 1, stop))) break;
                    tc_fence_after();
                    const ScanArgs& a = prm.scan[it->scan].a;
                    const float e = n == C  ? e_full
                                    : row < n ? a.inter_scale * decay_pow(it->l, it->rev ? n - 1 - row : row + 1)
                                              : 0.f;
                    // a thread stores its own row: 32-byte stores fill whole sectors where the rows allow them
                    const int esize = a.o_f32 ? 4 : 2, stored = row < n ? live : 0;
                    const bool wide = a.Dv * esize % 32 == 0 && (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0;
                    float2 zero = make_float2(0.f, 0.f);  // sums of 0 x output: NaN where one is not finite
                    uint8_t* dst = static_cast<uint8_t*>(a.o) +
                                   (((int64_t)it->row0 + place * C + row) * a.H * a.Dv + (int64_t)it->h * a.Dv + it->dv0 +
                                    half * kHalf) * esize;
#pragma unroll 1
                    for (int b = 0; b < kHalf / 16; ++b) {
                        float x[16], y[16];
                        tmem_ld16(lane_base + COL_Y1 + half * kHalf + b * 16, x);
                        tmem_ld16(lane_base + COL_Y2 + half * kHalf + b * 16, y);
                        tmem_wait_ld();
                        if (b == kHalf / 16 - 1) {
                            tc_fence_before();
                            warp_arrive(&bars[EPI], lane);
                        }
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const float2 f =
                                __ffma2_rn(make_float2(e, e), make_float2(y[j], y[j + 1]), make_float2(x[j], x[j + 1]));
                            x[j] = f.x;
                            x[j + 1] = f.y;
                            zero = __ffma2_rn(f, make_float2(0.f, 0.f), zero);
                        }
                        if (a.o_f32)
                            store16(reinterpret_cast<float*>(dst) + b * 16, x, stored - b * 16, wide);
                        else
                            store16(reinterpret_cast<__nv_bfloat16*>(dst) + b * 16, x, stored - b * 16, wide);
                    }
                    finite = finite && (stored <= 0 || zero.x + zero.y == 0.f);
                }
            }
            if (kOut && ok && it->nc > 0) {
                // One warp decides for all whether the item is done again.  Where the final state takes the initial one's place they
                // wait for that, and leave the state until then (in segments, which write none, they wait too: it spills less).  No
                // warp is here for the next item before all were for this one: its chunks wait for all their copies of S.
                const bool wait = kMode == kOutputs || prm.scan[it->scan].a.init == prm.scan[it->scan].a.final_state;
                const int item = it->index;
                if (!__all_sync(0xffffffffu, finite) && lane == 0) odd[item & 3] = 1;
                if (warp == kWarpOut && lane == 0) odd[(item + 1) & 3] = 0;
                warp_arrive(&bars[AGREE], lane);
                if (wait || warp == kWarpOut) {
                    ok = warp_wait(&bars[AGREE], item & 1, stop);
                    if (ok && odd[item & 3] && !it->careful) {
                        if (warp == kWarpOut && lane == 0) {
                            queue[*posted % kQueue] = *it;
                            __threadfence_block();
                            *posted = *posted + 1;
                        }
                        if (wait) {
                            leave(k);
                            continue;
                        }
                    }
                }
            }
            if (kMode != kOutputs) {
                const ScanArgs& a = prm.scan[it->scan].a;
                float* fin = kMode == kStates ? a.seg_state : a.final_state;
                if (ok && fin && row < a.Dk) {
                    float* dst = const_cast<float*>(state_row(fin, false));
#pragma unroll
                    for (int d = 0; d < kHalf; d += 4)
                        if (d < live) *reinterpret_cast<float4*>(dst + d) = make_float4(S[d], S[d + 1], S[d + 2], S[d + 3]);
                }
            }
            leave(k);
        }
        if (!ok) give_up();
    }
    if (warp == kWarpMma) tmem_dealloc(tmem, 512);
    if (tid == 0 && *stop) atomicOr(prm.scan[0].a.err, kErrTimeout);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                       q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<EncodeTiledFn>(p)
                   : nullptr;
    }();
    return fn;
}

// Rows of one role: [rows][heads][width] with rows `stride` elements apart; boxes of 128 rows x 128 bytes of a head,
// 128-byte swizzle, zeros outside.
bool make_map(CUtensorMap* m, const void* base, int width, int heads, int64_t rows, int64_t stride) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, 128};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kMode> cudaError_t launch(const Params& prm, unsigned blocks, cudaStream_t st) {
    const cudaError_t e = allow_smem<scan_tc_kernel<kMode>>((int)kSmemBytes);
    if (e != cudaSuccess) return e;
    // the warpgroups' shares add up to what 72 registers a thread give; from fewer a warpgroup would wait for ever
    static const int regs = [] {
        cudaFuncAttributes f{};
        return cudaFuncGetAttributes(&f, scan_tc_kernel<kMode>) == cudaSuccess ? f.numRegs : 0;
    }();
    if (regs != kRegisters) return cudaErrorInvalidConfiguration;
    scan_tc_kernel<kMode><<<blocks, kThreads, kSmemBytes, st>>>(prm);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scan_tc(const ScanArgs* scans, int count, Mode mode, cudaStream_t st) {
    Params prm;
    int64_t blocks = 0;
    for (int i = 0; i < count; ++i) {
        const ScanArgs& a = scans[i];
        Scan& s = prm.scan[i];
        s.a = a;
        const int64_t n = (a.seg_len ? a.slots : a.batch) * a.H * ((a.Dv + DVB - 1) / DVB);
        if ((blocks += n) > 0x7fffffff) return cudaErrorInvalidValue;
        s.blocks = (unsigned)n;
        if (a.rows > 0 && (!make_map(&s.tk, a.k, a.Dk, a.H / a.gk, a.rows, a.rs_k) ||
                           !make_map(&s.tv, a.v, a.Dv, a.H / a.gv, a.rows, a.rs_v) ||
                           (mode != kStates && !make_map(&s.tq, a.q, a.Dk, a.H / a.gq, a.rows, a.rs_q))))
            return cudaErrorInvalidValue;
    }
    if (blocks == 0) return cudaSuccess;
    if (mode == kStates) return launch<kStates>(prm, (unsigned)blocks, st);
    return mode == kOutputs ? launch<kOutputs>(prm, (unsigned)blocks, st) : launch<kWhole>(prm, (unsigned)blocks, st);
}

}  // namespace la
}  // namespace ssd
