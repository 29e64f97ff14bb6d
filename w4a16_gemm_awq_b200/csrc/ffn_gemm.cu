// ffn_gemm.cu -- the feed-forward products for more than a few tokens, on the 5th-generation tensor
// cores (tcgen05 over CTA pairs, TMEM, TMA).
//
//   LINEAR    y[m][n] = bf16( act( sum_k x[m][k] w[n][k] + bias[n] ) + residual[m][n] )
//   GATED     h[m][f] = bf16( act( sum_k x[m][k] wg[f][k] ) * sum_k x[m][k] wu[f][k] )
//   BACKWARD  dx[m][k] = bf16( sum_n dp[m][n] w[n][k] (+ sum_n dp[m][N + n] w2[n][k]) )
//   w = (q - z) scale, rounded once: to bf16 for LINEAR, whose activations are taken as they are, and to
//   fp16 for the others, whose activations are fp16 scaled by a power of two per token (ffn.cu), which
//   keeps every bit of theirs that fp32 sums can show; the epilogue undoes the scale.  The others have
//   several rounded factors per output: with bf16 the relative 2-norm against 64 bits was 2.9e-3 for the
//   gated output and for dx, where their own rounding to bf16 makes 1.7e-3; with fp16 it is 1.7e-3.
//   LINEAR is at 2.3e-3, and a pass over x to convert it would cost up to a tenth of the call (2048
//   tokens, K 14336: 18 us of 200).
//
// Design (B200):
//   - A CTA pair computes a tile of 256 output channels x BN tokens (BN a multiple of 32 up to 256)
//     with tcgen05.mma.cta_group::2 (M = 256: 128 channels in each CTA's TMEM).  Each CTA stages its
//     own 128 dequantized weight rows and half of the tokens: half the L2 and shared-memory traffic
//     per product of a single-CTA tile of the same width.
//   - The two accumulators (BN fp32 columns each, at TMEM columns 0 and 256) are used in turn, so the
//     epilogue of one tile runs while the next one accumulates.
//   - Warp roles (768 threads): 0 TMA of the activations, 1 MMA issue (leader CTA), 2 TMA of the packed
//     weights, 3 their scales and zero points (and the TMEM), 4-11 epilogue (a TMEM lane quarter and half
//     of the columns each), 12-23 dequant: three groups of four warps, which take the packed entries, two
//     stages of 64 contraction steps each, in turn.
//   - Dequant.  A ring entry holds the packed weights of 128 x 128 codes (8 KB, 64-byte rows, 64-byte
//     swizzle).  A thread turns 8 words into 64 weights and stores them as 16-byte chunks of the A stage
//     in the layout that the MMA reads, conflict-free.  Forward products contract over k, so a packed
//     row becomes a row of A (K-major).  The backward product contracts over n, so a packed row
//     becomes a column of A: it is stored as it lies and the MMA reads A channel-major (MN-major).
//   - fp16: a packed word becomes 8 weights in 13 operations: nibble pairs 0 and 1 are masked in place
//     into the mantissa of 1024 (as q and 16 q), 2 and 3 after one shift by 8; one subtraction or fused
//     multiply-add gives q - z exactly, one multiplication by the scale rounds.  bf16 has no room for the
//     second nibble and not for an fp16 scale: 19 operations, with scale = hi + lo, hi = bf16(scale); lo
//     has at most 3 bits and q - z 4, so (q - z) lo is exact and fma(q - z, hi, (q - z) lo) rounds once.
//   - GATED interleaves gate and up rows in sixteens, so the two sums of a channel sit in one warp's
//     lanes l and l + 16 and meet in its transposing buffer.
//   - Whole tiles go round the pairs; the tiles that do not fill a round are cut along the contraction
//     into equal runs, one per pair, whose fp32 partial tiles meet in the workspace: the last to arrive
//     (at a half of the columns, where the contributors end together) adds them in the order of the runs,
//     so the bits do not depend on which that is.  The cut tiles come first, so that joining them hides
//     behind whole tiles.  No pair waits for another.
//   - Bound: with many tokens the tensor pipe, 96 % busy (4096 tokens, K 4096, F 14336: 598 us alone, 1.61
//     PFLOP/s; 706 to 742 us in a row of calls, at the clock that the power limit leaves).  With few, the
//     loads and the dequant, about as long as one another (32 tokens, 16384 x 18944: 67 us, 2.4 TB/s of
//     packed weights; an early form 61 us, and 56 us with the dequant's arithmetic left out).
//   - Every wait on an mbarrier is bounded; one that runs out records kErrTimeout and its role stops.  The
//     epilogue warps, which also meet at a barrier of their own, stop together.  All roles of both CTAs then
//     meet at the closing cluster barrier.
#include <algorithm>
#include <cmath>

#include "act.cuh"
#include "common.cuh"
#include "internal.h"

namespace w4a16 {

namespace {

constexpr int kGroups = 3;               // dequant groups of four warps
constexpr int kEpilogue0 = 4, kDequant0 = 12;
constexpr int kThreads = 32 * (kDequant0 + 4 * kGroups);
constexpr int kS = 6;                    // stages of 64 contraction steps
constexpr int kABytes = 128 * 128;       // 128 channels x 64 steps, 16 bits each
constexpr int kEntryBytes = 128 * 64;    // 128 packed rows of 16 words: 128 contraction steps
constexpr int kParBytes = 512;           // their 128 scales (256 bytes) and 16 words of zero points
constexpr int kOutCols = 8;              // columns (tokens) an epilogue warp finishes at a time
constexpr int kOutStride = 36;           // floats per token in its transposing buffer: 32 channels, padded
constexpr int kOutBytes = kOutCols * kOutStride * 4;

// Shared memory.  NARROW: tiles of up to 128 tokens, half of the memory per stage of the activations, which
// goes to the ring of packed weights: with few tokens a stage is short and the weights come from device
// memory, so more of them have to be on their way (32 tokens, 16384 x 18944: 70.4 us with three entries, 66.3
// with six and no less with nine, before the dequant took whole entries).
template <bool NARROW>
struct Smem {
    static constexpr int kP = NARROW ? 6 : 3;               // packed entries
    static constexpr int kBBytes = (NARROW ? 64 : 128) * 128;  // this CTA's half of the tokens x 64 steps, 16 bits each
    static constexpr int kAOff = 0;
    static constexpr int kBOff = kAOff + kS * kABytes;
    static constexpr int kPOff = kBOff + kS * kBBytes;
    static constexpr int kParOff = kPOff + kP * kEntryBytes;
    static constexpr int kOutOff = kParOff + kP * kParBytes;
    static constexpr int kBarOff = kOutOff + 8 * kOutBytes;
    static constexpr int kBytes = kBarOff + 256;
    static_assert(kBytes <= 227 * 1024 && 8 * (2 * kS + 2 * kP + 5) + 8 <= 256, "shared memory of one CTA");
    // A wait by parity takes a phase for the one two before it.  So a dequant group that uses a slot uses it
    // in every phase: having waited for each phase in turn it can never pass on an old one, in whatever
    // order the copies land.
    static_assert(kP % kGroups == 0 && kS == 2 * kGroups, "the groups meet their slots in every phase");
};
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemSecond = 256;    // columns of the second accumulator

enum { kLinear = 0, kGated = 1, kBackward = 2 };

struct GemmArgs2 {
    PackedWeights w, w2;
    const uint16_t* bias;
    const uint16_t* residual;
    uint16_t* y;
    uint16_t* pre;
    uint16_t* pre2;
    float* partials;
    unsigned* counters;
    unsigned* err;
    const float* sums;       // BACKWARD: [sum_rows][N] column sums, added up into dbias; or sum_rows = 0
    float* dbias;
    int sum_rows;
    const float* row_scale;  // [M] what a token's sums are multiplied by (not for LINEAR)
    int M, N, K;       // N: rows of one weight matrix
    int gr;            // group size / 128
    int act;
    int bn;            // tokens per tile
    int entries;       // contraction / 128, both matrices of a gated backward product together
    int entries1;      // entries of the first matrix
    int tiles_c;       // tiles along the output channels
    int tiles;
    int cut;           // tiles 0 .. cut - 1 are cut into runs
    int runs;          // runs over the cut tiles' entries
    int halves;        // cut tiles are joined by halves of their columns
};

// Unit u of `units`, cut into `runs` equal runs: run p starts at p * units / runs.
__device__ __forceinline__ int run_begin(int p, int units, int runs) { return (int)((long long)units * p / runs); }
__device__ __forceinline__ int run_of(int u, int units, int runs) {
    return (int)((((long long)u + 1) * runs - 1) / units);
}

// A pair's pieces of work in order: its run over the cut tiles, tile by tile, then its whole tiles.
struct Walk {
    int u, u_end;   // rest of the run
    int whole;      // next whole tile
    int tile, e0, e1;
    bool partial;   // the tile has several contributors
    int first, count, index;  // of those: the first run, how many, this one's place
};

__device__ __forceinline__ Walk walk_start(const GemmArgs2& p, int pair) {
    Walk w;
    const int units = p.cut * p.entries;
    w.u = w.u_end = 0;
    if (pair < p.runs) {
        w.u = run_begin(pair, units, p.runs);
        w.u_end = run_begin(pair + 1, units, p.runs);
    }
    w.whole = p.cut + pair;
    w.first = w.index = 0;
    w.count = 1;
    return w;
}

__device__ __forceinline__ bool walk_step(Walk& w, const GemmArgs2& p, int pair, int pairs) {
    if (w.u < w.u_end) {
        const int units = p.cut * p.entries;
        w.tile = w.u / p.entries;
        const int t0 = w.tile * p.entries;
        w.e0 = w.u - t0;
        w.e1 = min(w.u_end, t0 + p.entries) - t0;
        w.u = t0 + w.e1;
        w.first = run_of(t0, units, p.runs);
        w.count = run_of(t0 + p.entries - 1, units, p.runs) - w.first + 1;
        w.index = pair - w.first;
        w.partial = w.count > 1;
        return true;
    }
    if (w.whole < p.tiles) {
        w.tile = w.whole;
        w.whole += pairs;
        w.e0 = 0;
        w.e1 = p.entries;
        w.partial = false;
        return true;
    }
    return false;
}

// Shared-memory operand descriptors, 128-byte swizzle.  K-major: rows of 128 bytes, 8-row groups 1024
// bytes apart.  MN-major: 64 channels x 8 steps in 1024 bytes; the next 8 steps 1024 bytes on, the next
// 64 channels 8192 bytes on.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t leading, uint32_t stride) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(leading >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on the barrier at this offset in both CTAs of the pair when the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(smem_u32(bar)), "h"((uint16_t)3)
        : "memory");
}

// TMA tile into this CTA's shared memory that completes on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4}], [%2];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
    const __half2 r = __hfma2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b), *reinterpret_cast<__half2*>(&c));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Arrivals on the leader's barriers from either CTA of the pair; what one CTA of the pair does for the other is
// waited for with acquire at cluster scope.  mbar_arrive_written releases this CTA's shared memory (the A stage,
// which its writers have passed to the async proxy) at cluster scope and nothing else: a release of all memory is
// a barrier behind the SM's global accesses too (gated, 4096 tokens, K 4096, F 14336: 1394 us with it, 707 us
// without any).  This one takes 4 us of 63 at 32 tokens, 16384 x 18944, 1 of 28 at 77, 8192 x 8192, and nothing of
// the long products.  mbar_arrive_read needs no release: the reads of an accumulator are ordered by the tcgen05
// fences on both sides.
__device__ __forceinline__ void mbar_arrive_written(uint32_t bar) {
    asm volatile(
        "fence.release.sync_restrict::shared::cta.cluster;\n\t"
        "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];"
        ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ void mbar_arrive_read(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// w & MASK over the bits of MAGIC.
template <uint32_t MASK, uint32_t MAGIC>
__device__ __forceinline__ uint32_t mask_into(uint32_t w) {
    uint32_t t;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(t) : "r"(w), "n"(MASK), "r"(MAGIC));
    return t;
}

// A packed row's scale and zero point in one group, and the 8 weights of a packed word in element order.
struct HalfRow {
    uint32_t scale, low, high;  // pairs: scale; 1024 + z; -(64 + z)

    __device__ __forceinline__ HalfRow(uint32_t s, uint32_t z)
        : scale(s | (s << 16)), low(0x64006400u | z | (z << 16)), high((0xD400u | (z << 4)) * 0x10001u) {}

    __device__ __forceinline__ uint4 operator()(uint32_t w) const {
        const uint32_t w8 = w >> 8, sixteenth = 0x2C002C00u;
        const uint32_t a = h2_sub(mask_into<0x000F000Fu, 0x64006400u>(w), low);
        const uint32_t b = h2_fma(mask_into<0x00F000F0u, 0x64006400u>(w), sixteenth, high);
        const uint32_t c = h2_sub(mask_into<0x000F000Fu, 0x64006400u>(w8), low);
        const uint32_t d = h2_fma(mask_into<0x00F000F0u, 0x64006400u>(w8), sixteenth, high);
        return make_uint4(h2_mul(a, scale), h2_mul(b, scale), h2_mul(c, scale), h2_mul(d, scale));
    }
};

struct Bf16Row {
    uint32_t hi, lo, zero;  // pairs: the scale's leading part and its rest; 128 + z

    __device__ __forceinline__ Bf16Row(uint32_t s, uint32_t z) {
        const float f = fp16_bits_to_float((uint16_t)s);
        hi = float_to_bf16_bits(f);
        lo = (uint32_t)float_to_bf16_bits(f - bf16_bits_to_float((uint16_t)hi)) * 0x10001u;
        hi *= 0x10001u;
        zero = 0x43004300u | z | (z << 16);
    }

    __device__ __forceinline__ uint32_t pair(uint32_t w) const {
        uint32_t t = bf16x2_sub(mask_into<0x000F000Fu, 0x43004300u>(w), zero);
        uint32_t l = bf16x2_mul(t, lo);
        const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&t), *reinterpret_cast<const __nv_bfloat162*>(&hi),
                                         *reinterpret_cast<const __nv_bfloat162*>(&l));
        return *reinterpret_cast<const uint32_t*>(&r);
    }

    __device__ __forceinline__ uint4 operator()(uint32_t w) const {
        return make_uint4(pair(w), pair(w >> 4), pair(w >> 8), pair(w >> 12));
    }
};

template <int MODE>
struct Dequant {
    using Row = HalfRow;
};
template <>
struct Dequant<kLinear> {
    using Row = Bf16Row;
};

__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// The whole warp waits for a barrier phase, bounded in time.  Every branch goes by a vote, so the lanes
// stay converged, as the .aligned instructions after a wait require.  CLUSTER: a phase on which the other CTA
// arrives too; acquires at cluster scope.
template <bool CLUSTER>
__device__ __forceinline__ bool warp_wait_in(uint64_t* bar, uint32_t parity) {
    auto done = [&]() {
        return __all_sync(0xffffffffu, CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) != 0;
    };
    if (done()) return true;
    const unsigned long long t0 = global_timer_ns();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (done()) return true;
        if (__any_sync(0xffffffffu, global_timer_ns() - t0 > kWaitLimitNs)) return false;
    }
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) { return warp_wait_in<false>(bar, parity); }
__device__ __forceinline__ bool warp_wait_cluster(uint64_t* bar, uint32_t parity) { return warp_wait_in<true>(bar, parity); }

// Barrier among the epilogue warps.
__device__ __forceinline__ void epilogue_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// The same, and whether all of them came with true.
__device__ __forceinline__ bool epilogue_all(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
}

template <int MODE, bool NARROW>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
ffn_gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                const __grid_constant__ CUtensorMap map_w2, const GemmArgs2 p) {
    using S = Smem<NARROW>;
    constexpr int kP = S::kP;
    // Pointers derive from the array itself, so that the compiler keeps the shared address space.
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {  // the swizzled stages need 1024-byte alignment
        if (threadIdx.x == 0) record_error(p.err, kErrShape);
        return;
    }
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBarOff);  // leader: activations landed, weights written
    uint64_t* empty = full + kS;     // the MMAs have read the stage
    uint64_t* pfull = empty + kS;    // a packed entry has landed
    uint64_t* pempty = pfull + kP;   // the dequant warps have read it
    uint64_t* dfull = pempty + kP;   // an accumulator is complete
    uint64_t* dempty = dfull + 2;    // leader: both CTAs' epilogues have read it
    uint64_t* drain = dempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    int* last_flag = reinterpret_cast<int*>(tmem_slot + 1);

    // From blockIdx and a broadcast, so that the compiler sees them as the same in a whole warp.
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x & 1);
    const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);
    const int half_bn = p.bn >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kS; ++i) {
            mbar_init(&full[i], 1 + 8);  // the leader's expected bytes, four dequant warps of each CTA
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kP; ++i) {
            mbar_init(&pfull[i], 2);  // rows and parameters
            mbar_init(&pempty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dempty[i], 16);  // eight epilogue warps of each CTA
        }
        mbar_init(drain, 1);
        fence_mbarrier_init();
    }
    if (warp == 0) prefetch_tensormap(&map_x);
    if (warp == 2) prefetch_tensormap(&map_w);
    if (warp == 2 && MODE != kLinear) prefetch_tensormap(&map_w2);
    if (warp == 3) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    // The next kernel on the stream may be scheduled as this one's CTAs leave; what it must not do before
    // this one is complete comes after its own griddepcontrol.wait.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    auto fail = [&]() { record_error(p.err, kErrTimeout); };
    Walk w = walk_start(p, pair);

    // One packed entry: warp 2 loads its 128 packed rows, warp 3 their scales and zero points (one warp for
    // both held few-token calls back: backward 32 tokens, 16384 x 18432, 60.6 us instead of 57.0).
    auto load_rows = [&](unsigned slot, int tc, int e) {
        uint8_t* dst = smem + S::kPOff + slot * kEntryBytes;
        const int n = tc * 256 + rank * 128;
        if (MODE == kLinear && n >= p.N) {  // the last pair's second half is past N: its rows go nowhere
            mbar_arrive(&pfull[slot]);
            return;
        }
        mbar_arrive_expect_tx(&pfull[slot], kEntryBytes);
        if (MODE == kLinear) {
            tma_load_2d(dst, &map_w, &pfull[slot], e * 16, n);
        } else if (MODE == kGated) {
            tma_load_2d(dst, &map_w, &pfull[slot], e * 16, n >> 1);
            tma_load_2d(dst + kEntryBytes / 2, &map_w2, &pfull[slot], e * 16, n >> 1);
        } else {
            const bool first = e < p.entries1;
            tma_load_2d(dst, first ? &map_w : &map_w2, &pfull[slot], n >> 3, (first ? e : e - p.entries1) * 128);
        }
    };
    auto load_params = [&](unsigned slot, int tc, int e) {
        uint8_t* par = smem + S::kParOff + slot * kParBytes;
        auto load = [&](const PackedWeights& q, int g, int n, int count, int at) {
            bulk_load(par + 2 * at, q.scales + (size_t)g * p.N + n, 2 * count, &pfull[slot]);
            bulk_load(par + 256 + at / 2, q.zeros + (size_t)g * (p.N >> 3) + (n >> 3), count / 2, &pfull[slot]);
        };
        const int n = tc * 256 + rank * 128;
        if (MODE == kLinear && n >= p.N) {
            mbar_arrive(&pfull[slot]);
            return;
        }
        mbar_arrive_expect_tx(&pfull[slot], 320);
        if (MODE == kLinear) {
            load(p.w, e / p.gr, n, 128, 0);
        } else if (MODE == kGated) {
            load(p.w, e / p.gr, n >> 1, 64, 0);
            load(p.w2, e / p.gr, n >> 1, 64, 64);
        } else {
            const bool first = e < p.entries1;
            load(first ? p.w : p.w2, (n >> 7) / p.gr, (first ? e : e - p.entries1) * 128, 128, 0);
        }
    };
    auto load_entry = [&](unsigned slot, int tc, int e) {
        if (elect_one()) {
            if (warp == 2)
                load_rows(slot, tc, e);
            else
                load_params(slot, tc, e);
        }
        __syncwarp();
    };
    // The first packed entries are what a call waits for first, and they need only this CTA's barriers.
    // The kernel before a GATED or BACKWARD product is its operand's, which nothing on the stream precedes
    // unfinished; before LINEAR it may be one that writes the weights (not waiting here is 1.3 us of 27 faster
    // at 77 tokens, 8192 x 8192).
    if (warp == 2 || warp == 3) {
        if (MODE == kLinear) griddep_wait();
        Walk first = w;
        if (walk_step(first, p, pair, pairs)) {
            const int tc = first.tile % p.tiles_c;
            for (int i = 0; i < kP && first.e0 + i < first.e1; ++i) load_entry(i, tc, first.e0 + i);
        }
    }
    cluster_sync_all();  // the other CTA's barriers are initialised too
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    // The TMA and MMA warps run their loops as whole warps and issue from one elected lane: the operands
    // of those instructions sit in uniform registers, and a loop that one lane runs alone moves each of
    // them there every time (385 to 480 cycles to issue a stage's four MMAs).
    if (warp == 0) {
        // ---------------------------------------------------------------- activations
        griddep_wait();  // the activations belong to the stream order
        bool ok = true;
        unsigned s = 0;
        while (ok && walk_step(w, p, pair, pairs)) {
            const int m0 = (w.tile / p.tiles_c) * p.bn + rank * half_bn;
            for (int c = 2 * w.e0; c < 2 * w.e1; ++c, ++s) {
                const unsigned slot = s % kS;
                if (s >= kS && !warp_wait_cluster(&empty[slot], (s / kS - 1) & 1)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(&full[slot], (uint32_t)p.bn * 128u);
                    tma_load_2d_pair(smem + S::kBOff + slot * S::kBBytes, &map_x, cluster_map(&full[slot], 0), c * 64, m0);
                }
                __syncwarp();
            }
        }
        // every MMA has read its stage and said so in both CTAs before either may leave
        for (unsigned i = s > kS ? s - kS : 0; ok && i < s; ++i) ok = warp_wait_cluster(&empty[i % kS], (i / kS) & 1);
        if (!ok && lane == 0) fail();
    } else if (warp == 2 || warp == 3) {
        // ---------------------------------------------------------------- packed weights
        bool ok = true;
        unsigned i = 0;
        for (bool begun = false; ok && walk_step(w, p, pair, pairs); begun = true) {
            const int tc = w.tile % p.tiles_c;
            for (int e = w.e0; e < w.e1; ++e, ++i) {
                if (!begun && i < kP) continue;  // loaded above
                const unsigned slot = i % kP;
                if (i >= kP && !warp_wait(&pempty[slot], (i / kP - 1) & 1)) {
                    ok = false;
                    break;
                }
                load_entry(slot, tc, e);
            }
        }
        if (!ok && lane == 0) fail();
        // The copies that this warp started must land before the CTA may leave, also where their readers gave up.  A
        // wait that runs out gave them that time.
        for (unsigned j = i > kP ? i - kP : 0; j < i && warp_wait(&pfull[j % kP], (j / kP) & 1); ++j) {
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issue
        if (rank == 0) {
            // D fp32, A and B fp16 (LINEAR: bf16), B K-major, A K-major or (backward) MN-major, M = 256, N = bn
            const uint32_t idesc = (1u << 4) | (MODE == kLinear ? 1u << 7 | 1u << 10 : 0u) | (MODE == kBackward ? 1u << 15 : 0u) |
                                   ((uint32_t)(p.bn >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
            const uint32_t base = smem_u32(smem);
            const uint64_t a0 = MODE == kBackward ? smem_desc(base + S::kAOff, 8192, 1024) : smem_desc(base + S::kAOff, 16, 1024);
            const uint64_t b0 = smem_desc(base + S::kBOff, 16, 1024);
            constexpr uint32_t kAStep = (MODE == kBackward ? 2048 : 32) >> 4, kBStep = 32 >> 4;  // 16 steps, as descriptors count
            bool ok = true;
            uint32_t slot = 0, phase = 0;
            unsigned t = 0;
            for (; ok && walk_step(w, p, pair, pairs); ++t) {
                const unsigned buf = t & 1;
                const uint32_t d = tmem + buf * kTmemSecond;
                if (t >= 2 && !warp_wait_cluster(&dempty[buf], (t / 2 - 1) & 1)) {
                    ok = false;
                    break;
                }
                const int stages = 2 * (w.e1 - w.e0);
                for (int c = 0; c < stages; ++c) {
                    if (!warp_wait_cluster(&full[slot], phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t a = a0 + slot * (kABytes >> 4), b = b0 + slot * (S::kBBytes >> 4);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_pair(d, a + kk * kAStep, b + kk * kBStep, idesc, (c > 0 || kk > 0) ? 1u : 0u);
                        commit_pair(&empty[slot]);
                        if (c == stages - 1) commit_pair(&dfull[buf]);
                    }
                    __syncwarp();
                    if (++slot == kS) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            }
            // the other CTA's last arrivals are here before this one may leave
            for (unsigned i = t > 2 ? t - 2 : 0; ok && i < t; ++i) ok = warp_wait_cluster(&dempty[i & 1], (i / 2) & 1);
            if (!ok) {
                if (lane == 0) fail();
                if (elect_one()) commit_pair(drain);  // MMAs in flight finish first
                (void)warp_wait_cluster(drain, 0);
            }
        }
    } else if (warp >= kDequant0) {
        // ---------------------------------------------------------------- dequant
        // The groups take the packed entries, two stages each, in turn.  A thread's packed words of its next
        // stage are read before it dequantizes the current one, so that the wait for them and the loads stay
        // out of the chain.
        const int group = (warp - kDequant0) >> 2;
        const int t = threadIdx.x & 127;  // the first dequant warp is the first of four
        int entries = 0;
        while (walk_step(w, p, pair, pairs)) entries += w.e1 - w.e0;
        // forward: row t of A (for GATED 16 gate rows, 16 up rows, ...), the half of its 64 bytes that is the
        // stage's; backward: step t % 64 of the stage's half of the packed rows, channels 64 (t / 64) .. + 63
        const int arow = MODE == kBackward ? (t & 63) : t;   // 128-byte row of the A stage
        const uint32_t dst = (MODE == kBackward ? (t >> 6) * 8192 : 0) + arow * 128;
        const uint32_t sw = (arow & 7) << 4;
        struct Packed {
            uint4 a, b;
            uint32_t scale, zword;
        };
        auto read = [&](int i, int h, Packed& q) {
            const unsigned ps = (unsigned)i % kP;
            const int prow = MODE == kLinear ? t
                             : MODE == kGated ? ((t >> 4) & 1) * 64 + 16 * (t >> 5) + (t & 15)
                                              : 64 * h + (t & 63);
            const int half = MODE == kBackward ? t >> 6 : h;
            const uint8_t* src = smem + S::kPOff + ps * kEntryBytes + prow * 64;
            const int x = (prow >> 1) & 3;
            q.a = *reinterpret_cast<const uint4*>(src + (((2 * half) ^ x) << 4));
            q.b = *reinterpret_cast<const uint4*>(src + (((2 * half + 1) ^ x) << 4));
            if (MODE != kBackward && h == 1) return;  // the same row, the same group
            const uint8_t* par = smem + S::kParOff + ps * kParBytes;
            q.scale = reinterpret_cast<const uint16_t*>(par)[prow];
            q.zword = reinterpret_cast<const uint32_t*>(par + 256)[prow >> 3] >> (4 * (prow & 7));
        };
        auto landed = [&](int i) { return warp_wait(&pfull[(unsigned)i % kP], ((unsigned)i / kP) & 1); };
        using Row = typename Dequant<MODE>::Row;
        bool ok = true;
        Packed cur{}, next{};
        if (group < entries) {
            ok = landed(group);
            if (ok) read(group, 0, cur);
        }
        for (int i = group; ok && i < entries; i += kGroups) {
            Row weights(cur.scale, cur.zword & 15u);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h == 0) {
                    read(i, 1, next);
                    // The refill writes the slot through the async proxy, which only this fence orders behind reads
                    // that are still in flight (they queue behind the epilogue's loads).  Without it the second half
                    // held codes of the entry kP further on, in one call of a hundred with a residual or bias sums.
                    // It costs nothing: 1023 tokens, 5120 x 5120 backward 53.1 us, 53.0 with the reads merely complete.
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&pempty[(unsigned)i % kP]);
                } else {
                    if (MODE == kBackward) weights = Row(cur.scale, cur.zword & 15u);
                    if (i + kGroups < entries) {
                        ok = landed(i + kGroups);
                        if (!ok) break;
                        read(i + kGroups, 0, next);
                    }
                }
                const unsigned s = 2 * (unsigned)i + h, slot = s % kS;
                if (s >= kS && !warp_wait_cluster(&empty[slot], (s / kS - 1) & 1)) {
                    ok = false;
                    break;
                }
                uint8_t* a = smem + S::kAOff + slot * kABytes + dst;
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    *reinterpret_cast<uint4*>(a + ((c << 4) ^ sw)) =
                        weights(c < 4 ? u4_get(cur.a, c) : u4_get(cur.b, c - 4));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_written(cluster_map(&full[slot], 0));
                cur = next;
            }
        }
        if (!ok && lane == 0) fail();
    } else if (warp >= kEpilogue0) {
        // ---------------------------------------------------------------- epilogue
        const int quarter = warp & 3;
        const int row = 32 * quarter + lane;  // TMEM lane
        const uint32_t t_lane = (uint32_t)(32 * quarter) << 16;
        const int side = (warp - kEpilogue0) >> 2;  // which half of the columns
        float* const out = reinterpret_cast<float*>(smem + S::kOutOff + (warp - kEpilogue0) * kOutBytes);
        griddep_wait();  // the residual, the outputs and the workspace belong to the stream order
        if (MODE == kBackward && p.sum_rows > 0) {
            // the bias gradient, while the first tile accumulates: 32 columns per CTA, the rows shared by the warps
            const int first = warp - kEpilogue0;
            for (int n = (int)blockIdx.x * 32; n < p.N; n += (int)gridDim.x * 32) {
                float s = 0.0f;
#pragma unroll 8
                for (int r = first; r < p.sum_rows; r += 8) s += __ldcg(p.sums + (size_t)r * p.N + n + lane);
                out[lane] = s;
                epilogue_barrier();
                if (first == 0) {
#pragma unroll
                    for (int i = 1; i < 8; ++i) s += out[i * (kOutBytes / 4) + lane];
                    p.dbias[n + lane] = s;
                }
                epilogue_barrier();
            }
        }
        bool ok = true;
        for (unsigned t = 0; walk_step(w, p, pair, pairs); ++t) {
            const unsigned buf = t & 1;
            ok = warp_wait_cluster(&dfull[buf], (t / 2) & 1);
            // The warps meet at barriers over a cut tile, so there all of them go on or none does: a completion
            // near the limit is seen by some of their waits only.
            if (w.partial) ok = epilogue_all(ok);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem + t_lane + buf * kTmemSecond;
            const int tc = w.tile % p.tiles_c;
            const int m0 = (w.tile / p.tiles_c) * p.bn;
            const int mtile = min(p.bn, p.M - m0);  // tokens of this tile
            // partial tiles, token-major: [run + tile][rank][bn][128]
            float* part0 = p.partials + ((size_t)(w.first + w.tile) * 2 + rank) * p.bn * 128 + row;
            const size_t part_step = (size_t)2 * p.bn * 128;
            // Where the contributors of a cut tile end together (plan.halves), they take its columns by halves,
            // the odd ones the second half first: each then finds one half of the others published and joins
            // it, instead of all publishing all and one joining all.
            const int mid = min(((mtile + 31) >> 5) << 4, mtile);  // a multiple of 16, or all
            const bool halves = w.partial && p.halves;
#pragma unroll 1
            for (int part = 0; part < (halves ? 2 : 1); ++part) {
                const int half = halves ? part ^ (w.index & 1) : 0;
                const int lo = half ? mid : 0, len = (halves && !half ? mid : mtile) - lo;
                const int cut = lo + min(((len + 31) >> 5) << 4, len);  // between the sides
                const int cb = side ? cut : lo, mlim = side ? lo + len : cut;  // this warp's columns
                if (w.partial) {
                    // A contributor that finds all the others counted joins them with its own accumulator; any
                    // other publishes its partial tile first and then counts itself, and joins if that made it
                    // the last.  The sum goes by the order of the runs either way, so its bits do not depend on
                    // who joins.
                    unsigned* counter = p.counters + 4 * w.tile + 2 * rank + half;
                    const unsigned others = (unsigned)(w.count - 1);
                    if (warp == kEpilogue0 && lane == 0) *last_flag = ld_acquire_gpu(counter) == others;
                    epilogue_barrier();
                    bool last = *reinterpret_cast<volatile int*>(last_flag) != 0;
                    epilogue_barrier();
                    if (!last) {
                        float* mine = part0 + w.index * part_step;
#pragma unroll 1
                        for (int c0 = cb; c0 < mlim; c0 += 16) {
                            uint32_t r[16];
                            tmem_ld_32x32b_x16(d + (uint32_t)c0, r);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) __stcg(mine + (size_t)(c0 + j) * 128, __uint_as_float(r[j]));
                        }
                        __threadfence();
                        epilogue_barrier();
                        if (warp == kEpilogue0 && lane == 0) *last_flag = atomic_add_acq_rel_gpu(counter, 1u) == others;
                        epilogue_barrier();
                        last = *reinterpret_cast<volatile int*>(last_flag) != 0;
                        epilogue_barrier();
                        if (!last) continue;
                    }
                    if (warp == kEpilogue0 && lane == 0) atomicExch(counter, 0u);  // all have counted themselves
                    __threadfence();
                }
                // A lane holds one channel of 8 tokens; through the warp's buffer it gets 4 neighbouring channels
                // of one token at a time, so that the outputs and the residual move 8 bytes at a time: LINEAR and
                // BACKWARD 8 lanes per token (32 channels), GATED 4 (16 channels, gate and up).
                constexpr int kLanes = MODE == kGated ? 4 : 8, kTok = 32 / kLanes, kIts = kOutCols / kTok;
                const int ch = 4 * (lane % kLanes), tk = lane / kLanes;
                const int n = MODE == kGated ? tc * 128 + rank * 64 + 16 * quarter + ch : tc * 256 + rank * 128 + 32 * quarter + ch;
                const int ld = MODE == kBackward ? p.K : p.N;
                const bool in = n < ld;  // the last pair's second half may be past N (whole warps)
                float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (MODE == kLinear && p.bias != nullptr && in) {
                    const uint2 b = *reinterpret_cast<const uint2*>(p.bias + n);
                    bias[0] = __uint_as_float(b.x << 16);
                    bias[1] = __uint_as_float(b.x & 0xFFFF0000u);
                    bias[2] = __uint_as_float(b.y << 16);
                    bias[3] = __uint_as_float(b.y & 0xFFFF0000u);
                }
                // the partial tiles of the first two other contributors, fetched one chunk ahead (those after them
                // are rare)
                float x0[kOutCols], x1[kOutCols];
                const float* s0 = part0 + (w.index == 0 ? part_step : 0);
                const float* s1 = part0 + (w.index <= 1 ? 2 * part_step : part_step);
                auto fetch = [&](int c0) {
                    if (!w.partial || c0 >= mlim) return;
#pragma unroll
                    for (int j = 0; j < kOutCols; ++j) x0[j] = __ldcg(s0 + (size_t)(c0 + j) * 128);
                    if (w.count > 2) {
#pragma unroll
                        for (int j = 0; j < kOutCols; ++j) x1[j] = __ldcg(s1 + (size_t)(c0 + j) * 128);
                    }
                };
                fetch(cb);
#pragma unroll 1
                for (int c0 = cb; c0 < mlim; c0 += kOutCols) {
                    const size_t o0 = (size_t)(m0 + c0 + tk) * ld + n;
                    const size_t step = (size_t)kTok * ld;
                    float token[kIts];  // the tokens' scales
#pragma unroll
                    for (int i = 0; i < kIts; ++i)
                        token[i] = MODE == kLinear                ? 1.0f
                                   : c0 + tk + i * kTok < mlim ? __ldcg(p.row_scale + m0 + c0 + tk + i * kTok)
                                                               : 0.0f;
                    uint2 res[kIts];
                    if (MODE == kLinear && p.residual != nullptr && in) {
#pragma unroll
                        for (int i = 0; i < kIts; ++i)
                            if (c0 + tk + i * kTok < mlim) res[i] = *reinterpret_cast<const uint2*>(p.residual + o0 + i * step);
                    }
                    float acc[kOutCols];
                    {
                        uint32_t r[kOutCols];
                        tmem_ld_32x32b_x8(d + (uint32_t)c0, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < kOutCols; ++j) acc[j] = __uint_as_float(r[j]);
                    }
                    if (w.partial) {
                        float own[kOutCols];
#pragma unroll
                        for (int j = 0; j < kOutCols; ++j) {
                            own[j] = acc[j];
                            acc[j] = w.index == 0 ? own[j] : x0[j];
                            acc[j] += w.index == 0 ? x0[j] : w.index == 1 ? own[j] : x1[j];
                            if (w.count > 2 && w.index <= 1) acc[j] += x1[j];
                        }
                        fetch(c0 + kOutCols);
#pragma unroll 1
                        for (int q = 2; q < w.count; ++q) {
                            if (q == 2 && w.index <= 1) continue;  // added above
#pragma unroll
                            for (int j = 0; j < kOutCols; ++j)
                                acc[j] += q == w.index ? own[j] : __ldcg(part0 + q * part_step + (size_t)(c0 + j) * 128);
                        }
                    }
                    __syncwarp();  // the previous columns have left the buffer
#pragma unroll
                    for (int j = 0; j < kOutCols; ++j) out[j * kOutStride + lane] = acc[j];
                    __syncwarp();
                    float v[4 * kIts];
#pragma unroll
                    for (int i = 0; i < kIts; ++i) {
                        const float4 a = *reinterpret_cast<const float4*>(out + (tk + i * kTok) * kOutStride + ch);
                        v[4 * i] = fmaf(a.x, token[i], bias[0]);
                        v[4 * i + 1] = fmaf(a.y, token[i], bias[1]);
                        v[4 * i + 2] = fmaf(a.z, token[i], bias[2]);
                        v[4 * i + 3] = fmaf(a.w, token[i], bias[3]);
                    }
                    auto put = [&](uint16_t* dst, const float (&f)[4 * kIts]) {
#pragma unroll
                        for (int i = 0; i < kIts; ++i)
                            if (in && c0 + tk + i * kTok < mlim)
                                *reinterpret_cast<uint2*>(dst + o0 + i * step) =
                                    make_uint2(bf16x2_of(f[4 * i], f[4 * i + 1]), bf16x2_of(f[4 * i + 2], f[4 * i + 3]));
                    };
                    if constexpr (MODE == kGated) {
                        float u[4 * kIts];
#pragma unroll
                        for (int i = 0; i < kIts; ++i) {
                            const float4 a = *reinterpret_cast<const float4*>(out + (tk + i * kTok) * kOutStride + 16 + ch);
                            u[4 * i] = a.x * token[i];
                            u[4 * i + 1] = a.y * token[i];
                            u[4 * i + 2] = a.z * token[i];
                            u[4 * i + 3] = a.w * token[i];
                        }
                        if (p.pre != nullptr) {
                            put(p.pre, v);
                            put(p.pre2, u);
                        }
                        act_values(p.act, v);
#pragma unroll
                        for (int i = 0; i < 4 * kIts; ++i) v[i] *= u[i];
                    } else if constexpr (MODE == kLinear) {
                        if (p.pre != nullptr) put(p.pre, v);
                        act_values(p.act, v);
                        if (p.residual != nullptr) {
#pragma unroll
                            for (int i = 0; i < kIts; ++i) {
                                v[4 * i] += __uint_as_float(res[i].x << 16);
                                v[4 * i + 1] += __uint_as_float(res[i].x & 0xFFFF0000u);
                                v[4 * i + 2] += __uint_as_float(res[i].y << 16);
                                v[4 * i + 3] += __uint_as_float(res[i].y & 0xFFFF0000u);
                            }
                        }
                    }
                    put(p.y, v);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_read(cluster_map(&dempty[buf], 0));
        }
        if (!ok && lane == 0) fail();
    }

    tc_fence_before();
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while the other may still use its memory
    if (warp == 3) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

}  // namespace

FfnPlan ffn_plan(int64_t M, int rows, int entries, int num_sms) {
    FfnPlan g{};
    const int64_t tm = (M + 255) / 256;
    g.bn = (int)(((M + tm - 1) / tm + 31) / 32 * 32);
    g.pairs = std::max(1, num_sms / 2);
    g.tiles_c = (rows + 255) / 256;
    g.tiles = (int64_t)g.tiles_c * ((M + g.bn - 1) / g.bn);
    const int rest = (int)(g.tiles % g.pairs);
    // Cycles that the last round and the cut tiles add: a stage takes the longer of its MMAs and its
    // dequant; joining c contributors about (30 bn + 800) c + 3000, half of that by halves, which hides
    // behind the whole tiles that follow the cut ones, if there are any.  Either the rest alone is cut (n
    // runs per tile, at most one per pair), or the rest and one full round (one run per pair).
    const double stage = std::max(1.45 * g.bn + 130.0, 440.0), tile = 2.0 * entries * stage;
    auto join = [&](int c, bool halves, bool hidden) {
        const double cost = ((halves ? 15.0 : 30.0) * g.bn + 800.0) * c + (halves ? 4500.0 : 3000.0);
        return hidden ? std::max(0.0, cost - tile) : cost;
    };
    // By halves pays where every run lies in one tile, so that a tile's contributors end together, with wide
    // tiles and few contributors (1023 tokens, 5120 x 5120 backward, 4 contributors: 51.7 -> 45.8 us; 300, 4096 x
    // 4096, 2: 26.1 -> 21.9); elsewhere the second count costs more (20 tokens, 4096 x 4096, 5 contributors: 13.5
    // -> 15.7 us; 512, 4096 x 14336, 112 tiles in 74 runs: 55.1 -> 60.9).  As many parts as contributors: the same.
    auto by_halves = [&](int runs, int cut) { return runs % cut == 0 && runs / cut <= 4 && g.bn >= 96; };
    double best = rest > 0 ? tile : 0.0;
    for (int n = 2; rest > 0 && n <= 16; ++n) {
        const int runs = std::min(g.pairs, rest * n);
        const int units = rest * entries;
        if (units / runs < 2) break;
        const int c = runs % rest == 0 ? runs / rest : runs / rest + 2;  // most contributors of a tile
        const double cost = 2.0 * stage * units / runs + join(c, by_halves(runs, rest), g.tiles > g.pairs);
        if (cost < best) {
            best = cost;
            g.cut = rest;
            g.runs = runs;
        }
    }
    if (rest > 0 && g.tiles > g.pairs) {
        const double cost = tile * rest / g.pairs + join(3, false, g.tiles > 2 * g.pairs);
        if (cost < best) {
            g.cut = rest + g.pairs;
            g.runs = g.pairs;
        }
    }
    g.halves = g.cut > 0 && by_halves(g.runs, g.cut);
    g.partial_bytes = (size_t)(g.cut + g.runs) * 2 * 128 * g.bn * 4;
    return g;
}

cudaError_t launch_ffn_gemm(const FfnMaps& maps, const FfnPlan& plan, const FfnArgs& a, bool back, bool two,
                            float* partials, unsigned* counters, unsigned* err, cudaStream_t stream) {
    GemmArgs2 g{};
    g.w = a.w;
    g.w2 = a.w2;
    g.bias = a.bias;
    g.residual = a.residual;
    g.y = a.y;
    g.pre = a.pre;
    g.pre2 = a.pre2;
    g.partials = partials;
    g.counters = counters;
    g.err = err;
    g.row_scale = a.row_scale;
    g.sums = a.sums;
    g.dbias = a.dbias;
    g.sum_rows = a.sum_rows;
    g.M = (int)a.M;
    g.N = a.N;
    g.K = a.K;
    g.gr = a.group_size / 128;
    g.act = a.act;
    g.bn = plan.bn;
    g.entries1 = (back ? a.N : a.K) / 128;
    g.entries = g.entries1 * (back && two ? 2 : 1);
    g.tiles_c = plan.tiles_c;
    g.tiles = (int)plan.tiles;
    g.cut = plan.cut;
    g.runs = plan.runs;
    g.halves = plan.halves;
    const bool narrow = plan.bn <= 128;
    auto* fn = back  ? (narrow ? ffn_gemm_kernel<kBackward, true> : ffn_gemm_kernel<kBackward, false>)
               : two ? (narrow ? ffn_gemm_kernel<kGated, true> : ffn_gemm_kernel<kGated, false>)
                     : (narrow ? ffn_gemm_kernel<kLinear, true> : ffn_gemm_kernel<kLinear, false>);
    const int smem = narrow ? Smem<true>::kBytes : Smem<false>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t busy = plan.tiles > plan.cut ? std::max<int64_t>(plan.tiles - plan.cut, plan.runs) : plan.runs;
    const int pairs = (int)std::min<int64_t>(plan.pairs, busy);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * pairs, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, maps.x, maps.w, maps.w2, g);
}

}  // namespace w4a16
