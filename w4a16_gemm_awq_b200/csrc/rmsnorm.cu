// rmsnorm.cu -- residual addition + root-mean-square norm + AWQ fold, its 8-bit output and its
// backward pass.
//
//   h = bf16(x + r);  rstd = rsqrt(mean h^2 + eps);  v = h * rstd * weight / s
//   y = bf16(v), or per group sc = max(max |v|, 1e-12) / 448 and q = e4m3(v / sc)
//   backward: xhat = h rstd;  w = dy weight / s;  dx = dh + rstd (w - xhat mean(w xhat));
//             dweight = sum over rows of dy xhat / s
//
// Memory bound: a row sits in registers (8 channels per thread and chunk), so every input is read
// once and every output written once; sums are fp32.  Many rows: 4 chunks per thread, so that a block
// has up to 8 independent 16-byte loads per thread in flight and several rows share an SM; each block
// walks rows and keeps weight / s in registers.  Few rows: as many threads per row as it has chunks,
// which shortens the one row's latency.  The backward pass runs several rows per block side by side
// (one group of warps each, with its own barrier) so that few partial sums of dweight are left.
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
};

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
    if (warps == 1) return;
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

// V: chunks of 8 channels per thread.  MAXT: most threads.  Q8: the e4m3 output.
template <int V, int MAXT, bool Q8>
__global__ void __launch_bounds__(MAXT) rmsnorm_kernel(const NormArgs p) {
    constexpr bool kKeep = V * MAXT <= 2048;  // weight / s stay in registers
    __shared__ float buf[2][1][32];
    __shared__ uint32_t amax[2][Q8 ? 256 : 1];  // per group of a row, as bits of |v|: NaN > inf > finite
    const int T = blockDim.x, t = threadIdx.x, K = p.K;
    float ws[kKeep ? V : 1][8];
    if constexpr (kKeep) {
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + t) * 8;
            if (k < K) load_ws(p.weight, p.s, k, ws[c]);
        }
    }
    const int groups = Q8 ? K / p.group : 0;
    const bool shared_max = Q8 && p.group != 128;  // a group of 128 is 16 lanes of one warp
    if (shared_max) {
        for (int i = t; i < groups; i += T) amax[0][i] = 0u;
        __syncthreads();
    }
    int flip = 0;
    for (long long m = blockIdx.x; m < p.M; m += gridDim.x, flip ^= 1) {
        const size_t row = (size_t)m * K;
        uint4 a[V], r[V];
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + t) * 8;
            if (k < K) {
                a[c] = __ldcs(reinterpret_cast<const uint4*>(p.x + row + k));
                if (p.residual != nullptr) r[c] = __ldcs(reinterpret_cast<const uint4*>(p.residual + row + k));
            }
        }
        // the row as rounded to bf16 stays packed in a: h is exact there, and the norm is that of h
        float ss[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + t) * 8;
            if (k < K) {
                float f[8];
                unpack8(a[c], f);
                if (p.residual != nullptr) {
                    float g[8];
                    unpack8(r[c], g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] += g[e];
                    a[c] = pack8(f);
                    unpack8(a[c], f);
                }
                if (p.h != nullptr) *reinterpret_cast<uint4*>(p.h + row + k) = a[c];
#pragma unroll
                for (int e = 0; e < 8; ++e) ss[0] = fmaf(f[e], f[e], ss[0]);
            }
        }
        group_sum<1>(ss, buf[flip], t, T, 1);
        const float rstd = rsqrtf(ss[0] / (float)K + p.eps);
        auto scaled = [&](int c, int k, float f[8]) {  // v of chunk c
            float w[8];
            if constexpr (kKeep) {
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = ws[c][e];
            } else {
                load_ws(p.weight, p.s, k, w);
            }
            unpack8(a[c], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * w[e];
        };
        uint32_t lane_max[V];
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + t) * 8;
            lane_max[c] = 0u;
            if (k < K) {
                float f[8];
                scaled(c, k, f);
                if constexpr (Q8) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) lane_max[c] = max(lane_max[c], __float_as_uint(f[e]) & 0x7FFFFFFFu);
                } else {
                    *reinterpret_cast<uint4*>(p.y + row + k) = pack8(f);
                }
            }
        }
        if constexpr (Q8) {
#pragma unroll
            for (int c = 0; c < V; ++c) {
                // 16 lanes hold 128 channels, all of one group
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) lane_max[c] = max(lane_max[c], __shfl_xor_sync(0xffffffffu, lane_max[c], o));
                const int k = (c * T + t) * 8;
                if (shared_max && (t & 15) == 0 && k < K) atomicMax(&amax[flip][k / p.group], lane_max[c]);
            }
            if (shared_max) {
                __syncthreads();
                // the other buffer: read last in the previous row, used next in the next one
                for (int i = t; i < groups; i += T) amax[flip ^ 1][i] = 0u;
            }
#pragma unroll
            for (int c = 0; c < V; ++c) {
                const int k = (c * T + t) * 8;
                if (k < K) {
                    const int g = k / p.group;
                    const float am = __uint_as_float(shared_max ? amax[flip][g] : lane_max[c]);
                    const float sc = (am < kTiny ? kTiny : am) / kE4m3Max;
                    const float inv = 1.0f / sc;
                    float f[8];
                    scaled(c, k, f);
                    uint32_t w[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        w[i] = e4m3x2(f[4 * i] * inv, f[4 * i + 1] * inv) |
                               (e4m3x2(f[4 * i + 2] * inv, f[4 * i + 3] * inv) << 16);
                    *reinterpret_cast<uint2*>(p.q + row + k) = make_uint2(w[0], w[1]);
                    if (k % p.group == 0) p.scales[(size_t)m * groups + g] = sc;
                }
            }
            if (shared_max) __syncthreads();  // the cleared maxima are seen before the next row's
        }
    }
}

// A block holds blockDim.x / T groups of T threads, each on a row of its own.
template <int V, int MAXT>
__global__ void __launch_bounds__(MAXT) rmsnorm_backward_kernel(const NormBwdArgs p, int T) {
    constexpr bool kKeep = V * MAXT <= 2048;
    constexpr int kGroups = 8;
    __shared__ float buf[kGroups][2][2][32];
    extern __shared__ float4 part[];  // [groups - 1][K] sums of the other groups, when there are several
    const int K = p.K, grp = threadIdx.x / T, t = threadIdx.x - grp * T, groups = blockDim.x / T;
    float dw[V][8], ws[kKeep ? V : 1][8];
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int k = (c * T + t) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[c][e] = 0.0f;
        if constexpr (kKeep) {
            if (k < K) load_ws(p.weight, p.s, k, ws[c]);
        }
    }
    int flip = 0;
    const long long step = (long long)gridDim.x * groups;
    for (long long m = (long long)blockIdx.x * groups + grp; m < p.M; m += step, flip ^= 1) {
        const size_t row = (size_t)m * K;
        uint4 g[V], hv[V], d4[V];
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + t) * 8;
            if (k < K) {
                g[c] = __ldcs(reinterpret_cast<const uint4*>(p.dy + row + k));
                hv[c] = __ldcs(reinterpret_cast<const uint4*>(p.h + row + k));
                if (p.dh != nullptr) d4[c] = __ldcs(reinterpret_cast<const uint4*>(p.dh + row + k));
            }
        }
        float s[2] = {0.0f, 0.0f};  // h^2, v h
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + t) * 8;
            if (k < K) {
                float a[8], h[8], w[8];
                unpack8(g[c], a);
                unpack8(hv[c], h);
                if constexpr (kKeep) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = ws[c][e];
                } else {
                    load_ws(p.weight, p.s, k, w);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s[0] = fmaf(h[e], h[e], s[0]);
                    s[1] = fmaf(a[e] * w[e], h[e], s[1]);
                }
            }
        }
        group_sum<2>(s, buf[grp][flip], t, T, 1 + grp);
        const float rstd = rsqrtf(s[0] / (float)K + p.eps);
        const float mean = s[1] * rstd / (float)K;  // mean of v xhat
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + t) * 8;
            if (k < K) {
                float a[8], h[8], w[8], d[8];
                unpack8(g[c], a);
                unpack8(hv[c], h);
                if constexpr (kKeep) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = ws[c][e];
                } else {
                    load_ws(p.weight, p.s, k, w);
                }
                if (p.dh != nullptr) {
                    unpack8(d4[c], d);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) d[e] = 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float xh = h[e] * rstd;
                    dw[c][e] = fmaf(a[e], xh, dw[c][e]);
                    d[e] = fmaf(rstd, a[e] * w[e] - xh * mean, d[e]);
                }
                *reinterpret_cast<uint4*>(p.dx + row + k) = pack8(d);
            }
        }
    }
    if (p.partials == nullptr) return;
    // the groups' sums in group order, then one row of partials per block
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int k = (c * T + t) * 8;
        if (k < K && grp > 0) {
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
        if (k < K) {
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

// dweight[k] = (sum over the R rows of partials) / s[k]: 32 columns per block, 8 row strides side by
// side, joined in a fixed order.
__global__ void __launch_bounds__(256) rmsnorm_dweight_kernel(const float* partials, const float* s, float* dweight,
                                                              int R, int K) {
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, rt = threadIdx.x >> 5;
    const int k = blockIdx.x * 32 + lane;
    float a = 0.0f;
    if (k < K) {
#pragma unroll 8
        for (int r = rt; r < R; r += 8) a += partials[(size_t)r * K + k];
    }
    part[rt][lane] = a;
    __syncthreads();
    if (rt != 0 || k >= K) return;
#pragma unroll
    for (int r = 1; r < 8; ++r) a += part[r][lane];
    dweight[k] = s != nullptr ? a / s[k] : a;
}

int up32(int v) { return (v + 31) / 32 * 32; }

// Threads per row for V chunks each.
int norm_threads(int K, int V) { return up32((K + 8 * V - 1) / (8 * V)); }

// Many rows: more than the SMs hold with one row each and 1024 threads per row.
bool norm_many(int64_t M, int num_sms) { return M > 2 * num_sms; }

template <bool Q8>
void norm_launch(const NormArgs& a, int num_sms, cudaStream_t stream) {
    const bool many = norm_many(a.M, num_sms);
    const int V = many || a.K > 16384 ? 4 : a.K > 8192 ? 2 : 1;
    const int T = norm_threads(a.K, V);
    const int64_t cap = (int64_t)num_sms * (1024 / T > 1 ? 1024 / T : 1);
    const int grid = (int)(a.M < cap || !many ? a.M : cap);
    if (V == 1) rmsnorm_kernel<1, 1024, Q8><<<grid, T, 0, stream>>>(a);
    else if (V == 2) rmsnorm_kernel<2, 1024, Q8><<<grid, T, 0, stream>>>(a);
    else if (T <= 256) rmsnorm_kernel<4, 256, Q8><<<grid, T, 0, stream>>>(a);
    else if (T <= 512) rmsnorm_kernel<4, 512, Q8><<<grid, T, 0, stream>>>(a);
    else rmsnorm_kernel<4, 1024, Q8><<<grid, T, 0, stream>>>(a);
}

// The backward launch: chunks and threads per row, rows side by side per block, blocks.
struct NormBwdPlan {
    int V, T, groups, grid;
};

NormBwdPlan norm_backward_plan(int64_t M, int K, int num_sms) {
    NormBwdPlan b;
    const bool many = norm_many(M, num_sms);
    b.V = many || K > 16384 ? 4 : K > 8192 ? 2 : 1;
    b.T = norm_threads(K, b.V);
    b.groups = many && b.T <= 256 ? (512 / b.T < 4 ? 512 / b.T : 4) : 1;
    const int64_t need = (M + b.groups - 1) / b.groups;
    b.grid = (int)(need < num_sms ? need : num_sms);
    return b;
}

}  // namespace

int rmsnorm_backward_rows(int64_t M, int K, int num_sms) { return norm_backward_plan(M, K, num_sms).grid; }

cudaError_t launch_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, const float* s,
                           float eps, uint16_t* h, uint16_t* y, uint8_t* q, float* scales, int group, int64_t M, int K,
                           int num_sms, cudaStream_t stream) {
    const NormArgs a{x, residual, weight, s, eps, h, y, q, scales, group, M, K};
    if (q != nullptr) norm_launch<true>(a, num_sms, stream);
    else norm_launch<false>(a, num_sms, stream);
    return cudaGetLastError();
}

cudaError_t launch_rmsnorm_backward(const uint16_t* dy, const uint16_t* h, const uint16_t* weight, const float* s,
                                    const uint16_t* dh, float eps, uint16_t* dx, float* dweight, float* partials,
                                    int64_t M, int K, int num_sms, cudaStream_t stream) {
    const NormBwdArgs a{dy, h, weight, s, dh, eps, dx, dweight != nullptr ? partials : nullptr, M, K};
    const NormBwdPlan b = norm_backward_plan(M, K, num_sms);
    const int threads = b.T * b.groups;
    const size_t smem = (size_t)(b.groups - 1) * K * 4;
    auto* fn = b.V == 1 ? rmsnorm_backward_kernel<1, 1024>
               : b.V == 2 ? rmsnorm_backward_kernel<2, 1024>
               : threads <= 512 ? rmsnorm_backward_kernel<4, 512>
                                : rmsnorm_backward_kernel<4, 1024>;
    cudaError_t e;
    if (smem > 32 * 1024) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    fn<<<b.grid, threads, smem, stream>>>(a, b.T);
    e = cudaGetLastError();
    if (e != cudaSuccess || dweight == nullptr) return e;
    rmsnorm_dweight_kernel<<<(K + 31) / 32, 256, 0, stream>>>(partials, s, dweight, b.grid, K);
    return cudaGetLastError();
}

}  // namespace w4a16
