// ffn.cu -- the elementwise steps of the feed-forward operators' backward passes: the gradient before
// the activation, rounded to bf16 as the product's operand, and the bias gradient from the unrounded
// values.
//
// Memory bound: 16-byte loads and stores, every element read and written once.  The bias sums are
// taken in the same pass: a block covers 256 columns x a run of rows and leaves its fp32 column sums
// in the workspace; the last block of a column range to arrive (a counter, reset to zero) adds them in
// the order of the runs, so no second launch is needed and the bits do not depend on which is last.
#include "act.cuh"
#include "common.cuh"
#include "internal.h"

namespace w4a16 {

namespace {

constexpr int kDpCols = 256;  // columns per block: 32 threads x 8
constexpr int kDpRowThreads = 8;

__device__ __forceinline__ void unpack8(const uint4& v, float f[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = u4_get(v, i);
        f[2 * i] = __uint_as_float(w << 16);
        f[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float f[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// dp = dy * act'(pre) over `rows` rows per block; dp nullptr: only the bias sums are wanted (no
// activation).  sums: [gridDim.y][N], nullptr without a bias gradient.
template <int ACT>
__global__ void __launch_bounds__(32 * kDpRowThreads) linear_dp_kernel(const uint16_t* dy, const uint16_t* pre,
                                                                       uint16_t* dp, float* sums, float* dbias,
                                                                       unsigned* counters, long long M, int N, int rows) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the product may set up meanwhile
    __shared__ float part[kDpRowThreads][kDpCols];
    __shared__ int last;
    const int lane = threadIdx.x & 31, rt = threadIdx.x >> 5;
    const int n = blockIdx.x * kDpCols + lane * 8;
    const bool in = n < N;
    float a[8] = {};
    if (in) {
        const long long m1 = min((long long)(blockIdx.y + 1) * rows, M);
#pragma unroll 2
        for (long long m = (long long)blockIdx.y * rows + rt; m < m1; m += kDpRowThreads) {
            float v[8];
            unpack8(__ldcs(reinterpret_cast<const uint4*>(dy + m * N + n)), v);
            if constexpr (ACT != W4A16_ACT_NONE) {
                float p[8];
                unpack8(__ldcs(reinterpret_cast<const uint4*>(pre + m * N + n)), p);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= act_grad<ACT>(p[e]);
                *reinterpret_cast<uint4*>(dp + m * N + n) = pack8(v);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] += v[e];
        }
    }
    if (sums == nullptr) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) part[rt][lane * 8 + e] = a[e];
    __syncthreads();
    const int c = threadIdx.x, nc = blockIdx.x * kDpCols + c;  // one column per thread
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < kDpRowThreads; ++r) s += part[r][c];
    if (gridDim.y == 1) {
        if (nc < N) dbias[nc] = s;
        return;
    }
    if (nc < N) __stcg(sums + (size_t)blockIdx.y * N + nc, s);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        last = atomic_add_acq_rel_gpu(counters + blockIdx.x, 1u) == gridDim.y - 1;
        if (last) atomicExch(counters + blockIdx.x, 0u);
    }
    __syncthreads();
    if (!last || nc >= N) return;
    __threadfence();
    s = 0.0f;
#pragma unroll 8
    for (int r = 0; r < (int)gridDim.y; ++r) s += __ldcg(sums + (size_t)r * N + nc);
    dbias[nc] = s;
}

// dg = dh u act'(g), du = dh act(g); n: elements / 8.
template <int ACT>
__global__ void __launch_bounds__(256) gated_dp_kernel(const uint4* dh, const uint4* g, const uint4* u, uint4* dg,
                                                       uint4* du, long long n) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the product may set up meanwhile
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
        float d[8], a[8], b[8], x[8], y[8];
        unpack8(__ldcs(dh + i), d);
        unpack8(__ldcs(g + i), a);
        unpack8(__ldcs(u + i), b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = d[e] * b[e] * act_grad<ACT>(a[e]);
            y[e] = d[e] * act_value<ACT>(a[e]);
        }
        dg[i] = pack8(x);
        du[i] = pack8(y);
    }
}

}  // namespace

// Runs of rows: at least 16 rows each, and few enough that adding the runs up (N threads, one load per
// run) stays short.  (64 runs at 1023 x 5120 took 20 us, most of it in the last blocks' sums.)
int linear_dp_blocks(int64_t M) { return (int)((M + 15) / 16 < 32 ? (M + 15) / 16 : 32); }

cudaError_t launch_linear_dp(const uint16_t* dy, const uint16_t* pre, uint16_t* dp, float* dbias, float* sums,
                             unsigned* counters, int64_t M, int N, int act, cudaStream_t stream) {
    const int runs = linear_dp_blocks(M);
    const int rows = (int)((M + runs - 1) / runs);
    const dim3 grid((N + kDpCols - 1) / kDpCols, (unsigned)((M + rows - 1) / rows));
    float* s = dbias != nullptr ? sums : nullptr;
#define W4A16_DP(ACT) \
    case ACT: linear_dp_kernel<ACT><<<grid, 32 * kDpRowThreads, 0, stream>>>(dy, pre, dp, s, dbias, counters, M, N, rows); break
    switch (act) {
        W4A16_DP(W4A16_ACT_NONE);
        W4A16_DP(W4A16_ACT_RELU);
        W4A16_DP(W4A16_ACT_SILU);
        W4A16_DP(W4A16_ACT_GELU);
        W4A16_DP(W4A16_ACT_GELU_TANH);
        default: return cudaErrorInvalidValue;
    }
#undef W4A16_DP
    return cudaGetLastError();
}

cudaError_t launch_gated_dp(const uint16_t* dh, const uint16_t* g, const uint16_t* u, uint16_t* dg, uint16_t* du,
                            int64_t M, int F, int act, int num_sms, cudaStream_t stream) {
    const long long n = (long long)M * F / 8;
    const long long blocks = (n + 255) / 256;
    const int grid = (int)(blocks < (long long)num_sms * 8 ? blocks : (long long)num_sms * 8);
    auto v = [](const uint16_t* p) { return reinterpret_cast<const uint4*>(p); };
    auto w = [](uint16_t* p) { return reinterpret_cast<uint4*>(p); };
#define W4A16_DP(ACT) \
    case ACT: gated_dp_kernel<ACT><<<grid, 256, 0, stream>>>(v(dh), v(g), v(u), w(dg), w(du), n); break
    switch (act) {
        W4A16_DP(W4A16_ACT_NONE);
        W4A16_DP(W4A16_ACT_RELU);
        W4A16_DP(W4A16_ACT_SILU);
        W4A16_DP(W4A16_ACT_GELU);
        W4A16_DP(W4A16_ACT_GELU_TANH);
        default: return cudaErrorInvalidValue;
    }
#undef W4A16_DP
    return cudaGetLastError();
}

}  // namespace w4a16
