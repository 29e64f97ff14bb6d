// rmsnorm.cu -- residual addition + root-mean-square norm + AWQ fold, its 8-bit output and its
// backward pass.
//
//   h = bf16(x + r);  rstd = rsqrt(mean h^2 + eps);  v = h * rstd * weight / s
//   y = bf16(v), or per group sc = max(max |v|, 1e-12) / 448 and q = e4m3(v / sc)
//   backward: xhat = h rstd;  w = dy weight / s;  dx = dh + rstd (w - xhat mean(w xhat));
//             dweight = sum over rows of dy xhat / s
//
// Memory bound: every input is read once and every output written once; sums are fp32.
//   - Many rows: a block walks rows that bulk copies bring into a ring in shared memory, so the loads of
//     the next rows are in flight whatever the threads do with the current one (loads issued by the
//     threads themselves, one row at a time: e4m3 1999 x 5120 26.6 us, backward 4096 x 4096 38.8 us;
//     with the ring 16.4 us and 32.7 us, 4.4 and 4.1 TB/s; 8192 x 8192 in bf16 94 us, 5.7 TB/s of the
//     6.55 that a copy reaches).  A thread holds 4 chunks of 8 channels of the row (backward 2 or 4),
//     packed as bf16 (the sum h is exact there), and weight / s.
//   - Few rows: one block per row with as many threads as it has chunks, which shortens its latency.
//   - The backward pass runs several rows per block side by side (one group of warps each, with its own
//     ring and barrier), so that few partial sums of dweight are left.
#include "common.cuh"
#include "internal.h"

namespace w4a16 {

namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kTiny = 1e-12f;

struct NormArgs {
    const uint16_t* x;
    const uint16_t* residual;  // or nullptr
    const uint16_t* weight;
    const float* s;            // or nullptr
    float eps;
    uint16_t* h;               // or nullptr
    uint16_t* y;               // bf16 output, or nullptr
    uint8_t* q;                // e4m3 output, or nullptr
    float* scales;
    int group;                 // channels per scale
    long long M;
    int K;
    int depth;                 // rows in the ring (many rows)
    unsigned* err;
};

struct NormBwdArgs {
    const uint16_t* dy;
    const uint16_t* h;
    const uint16_t* weight;
    const float* s;    // or nullptr
    const uint16_t* dh;  // or nullptr
    float eps;
    uint16_t* dx;
    float* partials;   // [gridDim.x][K] sums of dy xhat / s, or nullptr
    long long M;
    int K;
    int depth;         // rows in a group's ring (many rows)
    unsigned* err;
};

constexpr int kMaxDepth = 4;

__device__ __forceinline__ void unpack8(const uint4& v, float f[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = u4_get(v, i);
        f[2 * i] = __uint_as_float(w << 16);
        f[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ uint4 pack8(const float f[8]) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// weight / s of a thread's 8 channels from k
__device__ __forceinline__ void load_ws(const uint16_t* weight, const float* s, int k, float ws[8]) {
    unpack8(*reinterpret_cast<const uint4*>(weight + k), ws);
    if (s != nullptr) {
        const float4 a = *reinterpret_cast<const float4*>(s + k), b = *reinterpret_cast<const float4*>(s + k + 4);
        ws[0] /= a.x; ws[1] /= a.y; ws[2] /= a.z; ws[3] /= a.w;
        ws[4] /= b.x; ws[5] /= b.y; ws[6] /= b.z; ws[7] /= b.w;
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums of N values over a group of `threads` threads (whole warps) in a fixed order.  buf: [N][32]
// floats; two buffers used in turn need no second barrier.  bar: the group's barrier.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*buf)[32], int t, int threads, int bar) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
    const int warps = threads >> 5;
    if (warps == 1) {
        __syncwarp();  // orders memory as the barrier does for more warps: a ring slot may be refilled after it
        return;
    }
    if ((t & 31) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) buf[i][t >> 5] = v[i];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
    const int l = t & 31;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(l < warps ? buf[i][l] : 0.0f);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Waits for a row of the ring.  A thread whose wait runs out records it and goes on without waiting (on
// what lies in the ring), since the others may already be at a barrier.
__device__ __forceinline__ void row_wait(uint64_t* bar, uint32_t phase, bool& dead, unsigned* err) {
    if (!dead && !mbar_wait_bounded(bar, phase)) {
        dead = true;
        record_error(err, kErrTimeout);
    }
}

// max(m, |v|) with NaN above everything.
__device__ __forceinline__ float max_abs_nan(float m, float v) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
    return r;
}

__device__ __forceinline__ uint32_t bf16x2_add(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hadd2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// V: chunks of 8 channels per thread.  MAXT: most threads.  Q8: the e4m3 output.  RING: rows come through
// the ring of bulk copies.  FULL: every thread has all its V chunks (K = 8 V T).
//
// The e4m3 output needs no second pass for the maximum: rstd is the same for the whole row, so with
// u = h weight / s and G = max |u| of a group, scale = rstd G / 448 and v / scale = u (448 / G); G is
// taken together with the sum of squares.
template <int V, int MAXT, bool Q8, bool RING, bool FULL>
__global__ void __launch_bounds__(MAXT) rmsnorm_kernel(const NormArgs p) {
    constexpr bool kKeep = V * MAXT <= 2048;  // weight / s stay in registers
    __shared__ float buf[2][1][32];
    __shared__ uint32_t gmax[2][Q8 ? 256 : 1];  // per group of a row, as bits of |u|: NaN > inf > finite
    __shared__ __align__(8) uint64_t full[kMaxDepth];
    extern __shared__ __align__(128) uint16_t ring[];  // [depth][x row, residual row]
    const int T = blockDim.x, t = threadIdx.x, K = p.K;
    const bool add = p.residual != nullptr;
    const int srcs = add ? 2 : 1;
    // Thread 0 brings row m into slot `slot`.  Its earlier contents have been read: a barrier lies between.
    auto load_row = [&](int slot, long long m) {
        mbar_arrive_expect_tx(&full[slot], (uint32_t)(2 * K * srcs));
        uint16_t* dst = ring + (size_t)slot * srcs * K;
        bulk_load(dst, p.x + (size_t)m * K, (uint32_t)(2 * K), &full[slot]);
        if (add) bulk_load(dst + K, p.residual + (size_t)m * K, (uint32_t)(2 * K), &full[slot]);
    };
    if constexpr (RING) {
        if (t == 0) {
            for (int i = 0; i < p.depth; ++i) mbar_init(&full[i], 1);
            fence_mbarrier_init();
            for (int i = 0; i < p.depth; ++i) {
                const long long m = blockIdx.x + (long long)i * gridDim.x;
                if (m < p.M) load_row(i, m);
            }
        }
        __syncthreads();
    }
    float ws[kKeep ? V : 1][8];
    int group[V];       // the scale that a chunk belongs to, and whether it writes it
    bool first[V];
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int k = (c * T + t) * 8;
        if (kKeep && (FULL || k < K)) load_ws(p.weight, p.s, k, ws[c]);
        group[c] = Q8 ? k / p.group : 0;
        first[c] = Q8 && k == group[c] * p.group;
    }
    auto weight_of = [&](int c, int k, float w[8]) {
        if constexpr (kKeep) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = ws[c][e];
        } else {
            load_ws(p.weight, p.s, k, w);
        }
    };
    const int groups = Q8 ? K / p.group : 0;
    const bool shared_max = Q8 && p.group != 128;  // a group of 128 is 16 lanes of one warp
    if (shared_max) {
        for (int i = t; i < groups; i += T) gmax[0][i] = 0u;
        __syncthreads();
    }
    const float inv_k = 1.0f / (float)K;
    int flip = 0, slot = 0;
    uint32_t phase = 0;
    bool dead = false;
    for (long long m = blockIdx.x; m < p.M; m += gridDim.x, flip ^= 1) {
        const size_t row = (size_t)m * K;
        const uint16_t* src = RING ? ring + (size_t)slot * srcs * K : p.x + row;
        const uint16_t* src2 = RING ? src + K : p.residual + row;
        if constexpr (RING) row_wait(&full[slot], phase, dead, p.err);
        uint4 a[V], r[V];
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + t) * 8;
            if (FULL || k < K) {
                a[c] = RING ? *reinterpret_cast<const uint4*>(src + k) : __ldcs(reinterpret_cast<const uint4*>(src + k));
                if (add)
                    r[c] = RING ? *reinterpret_cast<const uint4*>(src2 + k) : __ldcs(reinterpret_cast<const uint4*>(src2 + k));
            }
        }
        // the row stays packed in a: h is exact there (the bf16 addition rounds the exact sum once), and
        // the norm is that of h
        float ss[1] = {0.0f};
        float lane_max[V];
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + t) * 8;
            lane_max[c] = 0.0f;
            if (FULL || k < K) {
                if (add)
                    a[c] = make_uint4(bf16x2_add(a[c].x, r[c].x), bf16x2_add(a[c].y, r[c].y), bf16x2_add(a[c].z, r[c].z),
                                      bf16x2_add(a[c].w, r[c].w));
                if (p.h != nullptr) *reinterpret_cast<uint4*>(p.h + row + k) = a[c];
                float f[8], w[8];
                unpack8(a[c], f);
                if constexpr (Q8) weight_of(c, k, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ss[0] = fmaf(f[e], f[e], ss[0]);
                    if constexpr (Q8) lane_max[c] = max_abs_nan(lane_max[c], f[e] * w[e]);
                }
            }
        }
        if constexpr (Q8) {
#pragma unroll
            for (int c = 0; c < V; ++c) {
                // 16 lanes hold 128 channels, all of one group
                uint32_t u = __float_as_uint(lane_max[c]);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) u = max(u, __shfl_xor_sync(0xffffffffu, u, o));
                lane_max[c] = __uint_as_float(u);
                if (shared_max && (t & 15) == 0 && (FULL || (c * T + t) * 8 < K)) atomicMax(&gmax[flip][group[c]], u);
            }
        }
        if constexpr (RING) fence_proxy_async_smem();  // this thread's reads of the slot, before its refill
        group_sum<1>(ss, buf[flip], t, T, 1);
        if constexpr (RING) {  // every thread has its part of the row: the slot takes the row `depth` further on
            const long long next = m + (long long)p.depth * gridDim.x;
            if (t == 0 && next < p.M) load_row(slot, next);
            if (++slot == p.depth) {
                slot = 0;
                phase ^= 1;
            }
        }
        const float rstd = rsqrtf(fmaf(ss[0], inv_k, p.eps));
        if constexpr (Q8) {
            if (shared_max) {
                __syncthreads();  // all maxima are in (one warp: group_sum has no barrier)
                // the other buffer: read last in the previous row, used next in the next one
                for (int i = t; i < groups; i += T) gmax[flip ^ 1][i] = 0u;
            }
        }
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + t) * 8;
            if (FULL || k < K) {
                float f[8], w[8];
                unpack8(a[c], f);
                weight_of(c, k, w);
                if constexpr (Q8) {
                    const float g = shared_max ? __uint_as_float(gmax[flip][group[c]]) : lane_max[c];
                    const float am = g * rstd;  // max |v|
                    float sc = am / kE4m3Max, mul = kE4m3Max / g;
                    if (!(am >= kTiny)) {  // below the least maximum, or a NaN, which spoils the whole group
                        sc = am < kTiny ? kTiny / kE4m3Max : am;
                        mul = am < kTiny ? rstd * (kE4m3Max / kTiny) : am;
                    }
                    uint32_t q[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        q[i] = e4m3x2(f[4 * i] * w[4 * i] * mul, f[4 * i + 1] * w[4 * i + 1] * mul) |
                               (e4m3x2(f[4 * i + 2] * w[4 * i + 2] * mul, f[4 * i + 3] * w[4 * i + 3] * mul) << 16);
                    *reinterpret_cast<uint2*>(p.q + row + k) = make_uint2(q[0], q[1]);
                    if (first[c]) p.scales[(size_t)m * groups + group[c]] = sc;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * w[e];
                    *reinterpret_cast<uint4*>(p.y + row + k) = pack8(f);
                }
            }
        }
        if constexpr (Q8) {
            if (shared_max) __syncthreads();  // the cleared maxima are seen before the next row's
        }
    }
}

// A block holds blockDim.x / T groups of T threads, each on a row of its own.  With c = rstd^3 sum(v h) / K
// the gradient is dx = dh + rstd v - c h, and dweight's terms are rstd (dy h) / s.
template <int V, int MAXT, bool RING, bool FULL>
__global__ void __launch_bounds__(MAXT) rmsnorm_backward_kernel(const NormBwdArgs p, int T) {
    constexpr bool kKeep = V * MAXT <= 2048;
    constexpr int kGroups = 8;
    __shared__ float buf[kGroups][2][2][32];
    __shared__ __align__(8) uint64_t full[kGroups][kMaxDepth];
    // RING: [group][depth][dy row, h row, dh row]; at the end [groups - 1][K] sums of the other groups
    extern __shared__ __align__(128) uint8_t dyn[];
    float4* part = reinterpret_cast<float4*>(dyn);
    const int K = p.K, grp = threadIdx.x / T, t = threadIdx.x - grp * T, groups = blockDim.x / T;
    const bool stream = p.dh != nullptr;
    const int srcs = stream ? 3 : 2;
    const long long step = (long long)gridDim.x * groups;
    uint16_t* ring = reinterpret_cast<uint16_t*>(dyn) + (size_t)grp * p.depth * srcs * K;
    auto load_row = [&](int slot, long long m) {  // thread 0 of the group; the slot's earlier row has been read
        mbar_arrive_expect_tx(&full[grp][slot], (uint32_t)(2 * K * srcs));
        uint16_t* dst = ring + (size_t)slot * srcs * K;
        bulk_load(dst, p.dy + (size_t)m * K, (uint32_t)(2 * K), &full[grp][slot]);
        bulk_load(dst + K, p.h + (size_t)m * K, (uint32_t)(2 * K), &full[grp][slot]);
        if (stream) bulk_load(dst + 2 * K, p.dh + (size_t)m * K, (uint32_t)(2 * K), &full[grp][slot]);
    };
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the sums' kernel waits for this one's end
    if constexpr (RING) {
        if (t == 0) {
            for (int i = 0; i < p.depth; ++i) mbar_init(&full[grp][i], 1);
            fence_mbarrier_init();
            for (int i = 0; i < p.depth; ++i) {
                const long long m = (long long)blockIdx.x * groups + grp + i * step;
                if (m < p.M) load_row(i, m);
            }
        }
        __syncthreads();
    }
    float dw[V][8], ws[kKeep ? V : 1][8];
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int k = (c * T + t) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[c][e] = 0.0f;
        if (kKeep && (FULL || k < K)) load_ws(p.weight, p.s, k, ws[c]);
    }
    auto weight_of = [&](int c, int k, float w[8]) {
        if constexpr (kKeep) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = ws[c][e];
        } else {
            load_ws(p.weight, p.s, k, w);
        }
    };
    const float inv_k = 1.0f / (float)K;
    int flip = 0, slot = 0;
    uint32_t phase = 0;
    bool dead = false;
    for (long long m = (long long)blockIdx.x * groups + grp; m < p.M; m += step, flip ^= 1) {
        const size_t row = (size_t)m * K;
        const uint16_t* src = ring + (size_t)slot * srcs * K;
        if constexpr (RING) row_wait(&full[grp][slot], phase, dead, p.err);
        // The ring's rows are read twice from shared memory instead of being kept: three rows, the weights
        // and the sums do not fit in the registers together.
        uint4 g[RING ? 1 : V], hv[RING ? 1 : V];
        float s[2] = {0.0f, 0.0f};  // h^2, v h
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + t) * 8;
            if (FULL || k < K) {
                uint4& gc = g[RING ? 0 : c];
                uint4& hc = hv[RING ? 0 : c];
                gc = RING ? *reinterpret_cast<const uint4*>(src + k) : __ldcs(reinterpret_cast<const uint4*>(p.dy + row + k));
                hc = RING ? *reinterpret_cast<const uint4*>(src + K + k) : __ldcs(reinterpret_cast<const uint4*>(p.h + row + k));
                float a[8], h[8], w[8];
                unpack8(gc, a);
                unpack8(hc, h);
                weight_of(c, k, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s[0] = fmaf(h[e], h[e], s[0]);
                    s[1] = fmaf(a[e] * w[e], h[e], s[1]);
                }
            }
        }
        group_sum<2>(s, buf[grp][flip], t, T, 1 + grp);
        if constexpr (RING) {
            // every thread has come past the previous row: its slot takes the row `depth` further on
            const long long next = m + (long long)(p.depth - 1) * step;
            if (t == 0 && m >= step && next < p.M) load_row(slot == 0 ? p.depth - 1 : slot - 1, next);
        }
        const float rstd = rsqrtf(fmaf(s[0], inv_k, p.eps));
        const float c2 = -(rstd * rstd) * (rstd * (s[1] * inv_k));
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + t) * 8;
            if (FULL || k < K) {
                float a[8], h[8], w[8], d[8];
                unpack8(RING ? *reinterpret_cast<const uint4*>(src + k) : g[RING ? 0 : c], a);
                unpack8(RING ? *reinterpret_cast<const uint4*>(src + K + k) : hv[RING ? 0 : c], h);
                if (stream) {
                    unpack8(RING ? *reinterpret_cast<const uint4*>(src + 2 * K + k)
                                 : __ldcs(reinterpret_cast<const uint4*>(p.dh + row + k)), d);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) d[e] = 0.0f;
                }
                weight_of(c, k, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dw[c][e] = fmaf(rstd, a[e] * h[e], dw[c][e]);
                    d[e] = fmaf(c2, h[e], fmaf(rstd, a[e] * w[e], d[e]));
                }
                *reinterpret_cast<uint4*>(p.dx + row + k) = pack8(d);
            }
        }
        if constexpr (RING) {
            fence_proxy_async_smem();  // this thread's reads of the slot, before its refill
            if (++slot == p.depth) {
                slot = 0;
                phase ^= 1;
            }
        }
    }
    if (p.partials == nullptr) return;
    // the groups' sums in group order, then one row of partials per block
    __syncthreads();  // the rings are done: their memory takes the sums
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int k = (c * T + t) * 8;
        if ((FULL || k < K) && grp > 0) {
            float4* dst = part + ((size_t)(grp - 1) * K + k) / 4;
            dst[0] = make_float4(dw[c][0], dw[c][1], dw[c][2], dw[c][3]);
            dst[1] = make_float4(dw[c][4], dw[c][5], dw[c][6], dw[c][7]);
        }
    }
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int k = (c * T + t) * 8;
        if (FULL || k < K) {
            float4 a = make_float4(dw[c][0], dw[c][1], dw[c][2], dw[c][3]);
            float4 b = make_float4(dw[c][4], dw[c][5], dw[c][6], dw[c][7]);
            for (int q = 0; q < groups - 1; ++q) {
                const float4* src = part + ((size_t)q * K + k) / 4;
                a.x += src[0].x; a.y += src[0].y; a.z += src[0].z; a.w += src[0].w;
                b.x += src[1].x; b.y += src[1].y; b.z += src[1].z; b.w += src[1].w;
            }
            float4* dst = reinterpret_cast<float4*>(p.partials + (size_t)blockIdx.x * K + k);
            dst[0] = a;
            dst[1] = b;
        }
    }
}

// dweight[k] = (sum over the R rows of partials) / s[k]: 32 columns per block, kSumRows row strides side by
// side, joined in a fixed order.
constexpr int kSumRows = 16;

__global__ void __launch_bounds__(32 * kSumRows) rmsnorm_dweight_kernel(const float* partials, const float* s,
                                                                        float* dweight, int R, int K) {
    __shared__ float part[kSumRows][32];
    const int lane = threadIdx.x & 31, rt = threadIdx.x >> 5;
    const int k = blockIdx.x * 32 + lane;
    const float scale = s != nullptr && rt == 0 && k < K ? s[k] : 1.0f;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial sums are complete
    float a = 0.0f;
    if (k < K) {
#pragma unroll 10
        for (int r = rt; r < R; r += kSumRows) a += __ldcg(partials + (size_t)r * K + k);
    }
    part[rt][lane] = a;
    __syncthreads();
    if (rt != 0 || k >= K) return;
#pragma unroll
    for (int r = 1; r < kSumRows; ++r) a += part[r][lane];
    dweight[k] = s != nullptr ? a / scale : a;
}

int up32(int v) { return (v + 31) / 32 * 32; }

// Threads per row for V chunks each.
int norm_threads(int K, int V) { return up32((K + 8 * V - 1) / (8 * V)); }

// Many rows: enough that each SM walks several.
bool norm_many(int64_t M, int num_sms) { return M > 2 * num_sms; }

constexpr size_t kRingBytes = kRingSmemBytes;  // ring memory of an SM

// Forward launch.
struct NormPlan {
    int V, T, grid, depth;
    size_t smem;
};

NormPlan norm_plan(int64_t M, int K, int srcs, int num_sms) {
    NormPlan b{};
    const bool many = norm_many(M, num_sms);
    b.V = many || K > 16384 ? 4 : K > 8192 ? 2 : 1;
    b.T = norm_threads(K, b.V);
    b.grid = (int)(M < (int64_t)num_sms * 65536 ? M : (int64_t)num_sms * 65536);
    if (!many) return b;
    // resident blocks by threads (at up to 112 registers each), then the ring's depth by shared memory: where an
    // SM has several blocks, two rows of each fit (32 channels per thread, two sources of 2 bytes)
    static_assert(2 * 576 * 32 * 4 <= kRingBytes, "two rows of every block");
    int blocks = 576 / b.T < 1 ? 1 : 576 / b.T > 8 ? 8 : 576 / b.T;
    const size_t row = (size_t)2 * K * srcs;
    b.depth = (int)(kRingBytes / blocks / row);
    b.depth = b.depth < 1 ? 1 : b.depth > kMaxDepth ? kMaxDepth : b.depth;
    b.smem = b.depth * row;
    const int64_t cap = (int64_t)num_sms * blocks;
    b.grid = (int)(M < cap ? M : cap);
    return b;
}

template <int V, int MAXT, bool Q8, bool RING>
cudaError_t norm_launch(const NormArgs& a, const NormPlan& b, cudaStream_t stream) {
    auto* fn = a.K == 8 * V * b.T ? rmsnorm_kernel<V, MAXT, Q8, RING, true> : rmsnorm_kernel<V, MAXT, Q8, RING, false>;
    if (RING) {
        const cudaError_t e = allow_ring_smem(fn);
        if (e != cudaSuccess) return e;
    }
    fn<<<b.grid, b.T, b.smem, stream>>>(a);
    return cudaGetLastError();
}

template <bool Q8>
cudaError_t norm_dispatch(const NormArgs& a, const NormPlan& b, cudaStream_t stream) {
    if (b.depth > 0) {
        if (b.T <= 256) return norm_launch<4, 256, Q8, true>(a, b, stream);
        if (b.T <= 512) return norm_launch<4, 512, Q8, true>(a, b, stream);
        return norm_launch<4, 1024, Q8, true>(a, b, stream);
    }
    if (b.V == 1) return norm_launch<1, 1024, Q8, false>(a, b, stream);
    if (b.V == 2) return norm_launch<2, 1024, Q8, false>(a, b, stream);
    return norm_launch<4, 1024, Q8, false>(a, b, stream);
}

// The backward launch: chunks and threads per row, rows side by side per block, blocks, ring.
struct NormBwdPlan {
    int V, T, groups, grid, depth;
    size_t smem;
};

// Many rows with V chunks per thread.
NormBwdPlan norm_backward_many(int64_t M, int K, int srcs, int num_sms, int V) {
    NormBwdPlan b{};
    b.V = V;
    b.T = norm_threads(K, V);
    b.groups = b.T <= 256 ? (512 / b.T < 8 ? 512 / b.T : 8) : 1;
    const int64_t need = (M + b.groups - 1) / b.groups;
    b.grid = (int)(need < num_sms ? need : num_sms);
    const size_t row = (size_t)2 * K * srcs;
    // at least two rows, one filled while the other is read: several groups always have them (32 channels per
    // thread at most, three sources of 2 bytes)
    static_assert(2 * 512 * 32 * 6 <= kRingBytes, "two rows of every group");
    b.depth = (int)(kRingBytes / b.groups / row);
    b.depth = b.depth > kMaxDepth ? kMaxDepth : b.depth;
    if (b.depth < 2) b.depth = 0;  // rows too long: the threads load them themselves
    b.smem = b.groups * b.depth * row;
    return b;
}

NormBwdPlan norm_backward_plan(int64_t M, int K, int srcs, int num_sms) {
    if (norm_many(M, num_sms)) {
        // Four chunks; two where four leave each group one row ahead of the one it reads and two leave no
        // fewer threads: fewer groups, each with more rows on their way (4096 rows with dh: K 4096 33.9 -> 31.1
        // us, K 8192 55.4 -> 53.5; without dh, three rows per group: K 4096 25.7 -> 28.2, K 8192 39 -> 47; K
        // 5120 with dh, 320 threads instead of 480: 40.6 -> 45.2).
        const NormBwdPlan b = norm_backward_many(M, K, srcs, num_sms, 4);
        if (b.depth != 2) return b;
        const NormBwdPlan c = norm_backward_many(M, K, srcs, num_sms, 2);
        return c.depth > 2 && c.T <= 512 && c.T * c.groups >= b.T * b.groups ? c : b;
    }
    NormBwdPlan b{};
    b.V = K > 16384 ? 4 : K > 8192 ? 2 : 1;
    b.T = norm_threads(K, b.V);
    b.groups = 1;
    b.grid = (int)(M < num_sms ? M : num_sms);
    return b;
}

}  // namespace

int rmsnorm_backward_rows(int64_t M, int K, int num_sms) {
    const int a = norm_backward_plan(M, K, 2, num_sms).grid, b = norm_backward_plan(M, K, 3, num_sms).grid;
    return a > b ? a : b;
}

cudaError_t launch_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, const float* s,
                           float eps, uint16_t* h, uint16_t* y, uint8_t* q, float* scales, int group, int64_t M, int K,
                           int num_sms, unsigned* err, cudaStream_t stream) {
    const NormPlan b = norm_plan(M, K, residual != nullptr ? 2 : 1, num_sms);
    const NormArgs a{x, residual, weight, s, eps, h, y, q, scales, group, M, K, b.depth, err};
    return q != nullptr ? norm_dispatch<true>(a, b, stream) : norm_dispatch<false>(a, b, stream);
}

cudaError_t launch_rmsnorm_backward(const uint16_t* dy, const uint16_t* h, const uint16_t* weight, const float* s,
                                    const uint16_t* dh, float eps, uint16_t* dx, float* dweight, float* partials,
                                    int64_t M, int K, int num_sms, unsigned* err, cudaStream_t stream) {
    const NormBwdPlan b = norm_backward_plan(M, K, dh != nullptr ? 3 : 2, num_sms);
    const NormBwdArgs a{dy, h, weight, s, dh, eps, dx, dweight != nullptr ? partials : nullptr, M, K, b.depth, err};
    const int threads = b.T * b.groups;
    const size_t sums = (size_t)(b.groups - 1) * K * 4;
    const size_t smem = b.smem > sums ? b.smem : sums;
    const bool exact = K == 8 * b.V * b.T;
    auto* fn = b.depth > 0 && b.V == 2 ? (exact ? rmsnorm_backward_kernel<2, 512, true, true>
                                                : rmsnorm_backward_kernel<2, 512, true, false>)
               : b.depth > 0           ? (threads > 512 ? rmsnorm_backward_kernel<4, 1024, true, false>
                                          : exact       ? rmsnorm_backward_kernel<4, 512, true, true>
                                                        : rmsnorm_backward_kernel<4, 512, true, false>)
               : b.V == 1              ? rmsnorm_backward_kernel<1, 1024, false, false>
               : b.V == 2              ? rmsnorm_backward_kernel<2, 1024, false, false>
                                       : rmsnorm_backward_kernel<4, 1024, false, false>;
    cudaError_t e;
    if (b.depth > 0) {
        e = allow_ring_smem(fn);
        if (e != cudaSuccess) return e;
    }
    fn<<<b.grid, threads, smem, stream>>>(a, b.T);
    e = cudaGetLastError();
    if (e != cudaSuccess || dweight == nullptr) return e;
    // the sums' kernel is scheduled while the rows are still walked and waits for their end
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((K + 31) / 32, 1, 1);
    cfg.blockDim = dim3(32 * kSumRows, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rmsnorm_dweight_kernel, (const float*)partials, s, dweight, b.grid, K);
}

}  // namespace w4a16
