// rmsnorm.cu -- residual addition + root-mean-square norm + AWQ fold, its 8-bit output and its
// backward pass.
//
//   h = bf16(x + r);  rstd = rsqrt(mean h^2 + eps);  v = h * rstd * weight / s
//   y = bf16(v), or per group sc = max(max |v|, 1e-12) / 448 and q = e4m3(v / sc)
//   backward: xhat = h rstd;  w = dy weight / s;  dx = dh + rstd (w - xhat mean(w xhat));
//             dweight = sum over rows of dy xhat / s
//
// One block per row at a time, the row in registers (8 channels per thread and chunk), so every
// input is read once and every output written once: memory bound.  Sums are fp32.
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

// Sum over the block in a fixed order.  buf: 32 floats; two buffers used in turn need no second
// barrier.
__device__ __forceinline__ float block_sum(float v, float* buf) {
    v = warp_sum(v);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    const int l = threadIdx.x & 31;
    return warp_sum(l < warps ? buf[l] : 0.0f);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// V: chunks of 8 channels per thread.  Q8: the e4m3 output.
template <int V, bool Q8>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const NormArgs p) {
    __shared__ float buf[2][32];
    __shared__ uint32_t amax[Q8 ? 256 : 1];  // per group of a row, as bits of |v|: NaN > inf > finite
    const int T = blockDim.x, K = p.K;
    float ws[V][8];
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int k = (c * T + threadIdx.x) * 8;
        if (k < K) load_ws(p.weight, p.s, k, ws[c]);
    }
    int flip = 0;
    for (long long m = blockIdx.x; m < p.M; m += gridDim.x, flip ^= 1) {
        float f[V][8];
        float ss = 0.0f;
        if constexpr (Q8) {
            __syncthreads();  // the previous row's maxima have been read
            for (int i = threadIdx.x; i < K / p.group; i += T) amax[i] = 0u;
        }
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + threadIdx.x) * 8;
            if (k < K) {
                uint4 a = *reinterpret_cast<const uint4*>(p.x + m * K + k);
                unpack8(a, f[c]);
                if (p.residual != nullptr) {
                    float r[8];
                    unpack8(*reinterpret_cast<const uint4*>(p.residual + m * K + k), r);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[c][e] += r[e];
                    a = pack8(f[c]);
                    unpack8(a, f[c]);  // the norm is that of the rounded sum
                }
                if (p.h != nullptr) *reinterpret_cast<uint4*>(p.h + m * K + k) = a;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(f[c][e], f[c][e], ss);
            }
        }
        const float rstd = rsqrtf(block_sum(ss, buf[flip]) / (float)K + p.eps);
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + threadIdx.x) * 8;
            if (k < K) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[c][e] = f[c][e] * rstd * ws[c][e];
                if constexpr (!Q8) *reinterpret_cast<uint4*>(p.y + m * K + k) = pack8(f[c]);
            }
        }
        if constexpr (Q8) {
            if ((T >> 5) == 1) __syncthreads();  // block_sum had no barrier after amax was cleared
#pragma unroll
            for (int c = 0; c < V; ++c) {
                const int k = (c * T + threadIdx.x) * 8;
                uint32_t a = 0;
                if (k < K) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) a = max(a, __float_as_uint(f[c][e]) & 0x7FFFFFFFu);
                    atomicMax(&amax[k / p.group], a);
                }
            }
            __syncthreads();
#pragma unroll
            for (int c = 0; c < V; ++c) {
                const int k = (c * T + threadIdx.x) * 8;
                if (k < K) {
                    const float am = __uint_as_float(amax[k / p.group]);
                    const float sc = (am < kTiny ? kTiny : am) / kE4m3Max;
                    uint32_t w[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        w[i] = e4m3x2(f[c][4 * i] / sc, f[c][4 * i + 1] / sc) |
                               (e4m3x2(f[c][4 * i + 2] / sc, f[c][4 * i + 3] / sc) << 16);
                    *reinterpret_cast<uint2*>(p.q + m * K + k) = make_uint2(w[0], w[1]);
                    if (k % p.group == 0) p.scales[m * (K / p.group) + k / p.group] = sc;
                }
            }
        }
    }
}

template <int V>
__global__ void __launch_bounds__(1024) rmsnorm_backward_kernel(const NormBwdArgs p) {
    __shared__ float buf[2][2][32];
    const int T = blockDim.x, K = p.K;
    float dw[V][8];
#pragma unroll
    for (int c = 0; c < V; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[c][e] = 0.0f;
    int flip = 0;
    for (long long m = blockIdx.x; m < p.M; m += gridDim.x, flip ^= 1) {
        uint4 g[V], hv[V];
        float ss = 0.0f, sv = 0.0f;
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + threadIdx.x) * 8;
            if (k < K) {
                g[c] = *reinterpret_cast<const uint4*>(p.dy + m * K + k);
                hv[c] = *reinterpret_cast<const uint4*>(p.h + m * K + k);
                float a[8], h[8], ws[8];
                unpack8(g[c], a);
                unpack8(hv[c], h);
                load_ws(p.weight, p.s, k, ws);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ss = fmaf(h[e], h[e], ss);
                    sv = fmaf(a[e] * ws[e], h[e], sv);
                }
            }
        }
        ss = block_sum(ss, buf[flip][0]);
        sv = block_sum(sv, buf[flip][1]);
        const float rstd = rsqrtf(ss / (float)K + p.eps);
        const float mean = sv * rstd / (float)K;  // mean of v xhat
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + threadIdx.x) * 8;
            if (k < K) {
                float a[8], h[8], ws[8], d[8];
                unpack8(g[c], a);
                unpack8(hv[c], h);
                load_ws(p.weight, p.s, k, ws);
                if (p.dh != nullptr) {
                    unpack8(*reinterpret_cast<const uint4*>(p.dh + m * K + k), d);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) d[e] = 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float xh = h[e] * rstd;
                    dw[c][e] = fmaf(a[e], xh, dw[c][e]);
                    d[e] = fmaf(rstd, a[e] * ws[e] - xh * mean, d[e]);
                }
                *reinterpret_cast<uint4*>(p.dx + m * K + k) = pack8(d);
            }
        }
    }
    if (p.partials != nullptr) {
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + threadIdx.x) * 8;
            if (k < K) {
                float4* dst = reinterpret_cast<float4*>(p.partials + (size_t)blockIdx.x * K + k);
                dst[0] = make_float4(dw[c][0], dw[c][1], dw[c][2], dw[c][3]);
                dst[1] = make_float4(dw[c][4], dw[c][5], dw[c][6], dw[c][7]);
            }
        }
    }
}

// dweight[k] = (sum over rows of partials[r][k], in row order) / s[k]
__global__ void __launch_bounds__(256) rmsnorm_dweight_kernel(const float* partials, const float* s, float* dweight,
                                                              int R, int K) {
    const int k = blockIdx.x * 256 + threadIdx.x;
    if (k >= K) return;
    float a = 0.0f;
    for (int r = 0; r < R; ++r) a += partials[(size_t)r * K + k];
    dweight[k] = s != nullptr ? a / s[k] : a;
}

int norm_threads(int K) {
    const int t = (K / 8 + 31) / 32 * 32;
    return t < 1024 ? t : 1024;
}

int norm_chunks(int K) { return (K / 8 + norm_threads(K) - 1) / norm_threads(K); }

int norm_grid(int64_t M, int threads, int num_sms) {
    const int64_t cap = (int64_t)num_sms * (2048 / threads < 8 ? 2048 / threads : 8);
    return (int)(M < cap ? M : cap);
}

}  // namespace

int rmsnorm_backward_rows(int64_t M, int K, int num_sms) { return norm_grid(M, norm_threads(K), num_sms); }

cudaError_t launch_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, const float* s,
                           float eps, uint16_t* h, uint16_t* y, uint8_t* q, float* scales, int group, int64_t M, int K,
                           int num_sms, cudaStream_t stream) {
    const NormArgs a{x, residual, weight, s, eps, h, y, q, scales, group, M, K};
    const int T = norm_threads(K), V = norm_chunks(K);
    const int grid = norm_grid(M, T, num_sms);
    if (q != nullptr) {
        if (V == 1) rmsnorm_kernel<1, true><<<grid, T, 0, stream>>>(a);
        else if (V == 2) rmsnorm_kernel<2, true><<<grid, T, 0, stream>>>(a);
        else rmsnorm_kernel<4, true><<<grid, T, 0, stream>>>(a);
    } else {
        if (V == 1) rmsnorm_kernel<1, false><<<grid, T, 0, stream>>>(a);
        else if (V == 2) rmsnorm_kernel<2, false><<<grid, T, 0, stream>>>(a);
        else rmsnorm_kernel<4, false><<<grid, T, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_rmsnorm_backward(const uint16_t* dy, const uint16_t* h, const uint16_t* weight, const float* s,
                                    const uint16_t* dh, float eps, uint16_t* dx, float* dweight, float* partials,
                                    int64_t M, int K, int num_sms, cudaStream_t stream) {
    const NormBwdArgs a{dy, h, weight, s, dh, eps, dx, dweight != nullptr ? partials : nullptr, M, K};
    const int T = norm_threads(K), V = norm_chunks(K);
    const int grid = rmsnorm_backward_rows(M, K, num_sms);
    if (V == 1) rmsnorm_backward_kernel<1><<<grid, T, 0, stream>>>(a);
    else if (V == 2) rmsnorm_backward_kernel<2><<<grid, T, 0, stream>>>(a);
    else rmsnorm_backward_kernel<4><<<grid, T, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || dweight == nullptr) return e;
    rmsnorm_dweight_kernel<<<(K + 255) / 256, 256, 0, stream>>>(partials, s, dweight, grid, K);
    return cudaGetLastError();
}

}  // namespace w4a16
