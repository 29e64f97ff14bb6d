// ffn.cu -- the elementwise steps of the feed-forward operators' backward passes: the gradient before
// the activation, in bf16 for the product, and the bias gradient.
#include "act.cuh"
#include "common.cuh"
#include "internal.h"

namespace w4a16 {

namespace {

// dp = dy * act'(pre), rounded to bf16 for the product (dp may be nullptr: only the bias sum is
// wanted), and the column sums of the unrounded dp over this block's rows.
__global__ void __launch_bounds__(256) linear_dp_kernel(const uint16_t* dy, const uint16_t* pre, uint16_t* dp,
                                                        float* sums, long long M, int N, int act, int rows) {
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= N) return;
    float a = 0.0f;
    const long long m0 = (long long)blockIdx.y * rows, m1 = m0 + rows < M ? m0 + rows : M;
    for (long long m = m0; m < m1; ++m) {
        float v = bf16_bits_to_float(dy[m * N + n]);
        if (act != W4A16_ACT_NONE) v *= act_grad(act, bf16_bits_to_float(pre[m * N + n]));
        if (dp != nullptr) dp[m * N + n] = float_to_bf16_bits(v);
        a += v;
    }
    if (sums != nullptr) sums[(size_t)blockIdx.y * N + n] = a;
}

__global__ void __launch_bounds__(256) column_sum_kernel(const float* sums, float* out, int R, int N) {
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= N) return;
    float a = 0.0f;
    for (int r = 0; r < R; ++r) a += sums[(size_t)r * N + n];
    out[n] = a;
}

// dg = dh u act'(g), du = dh act(g), rounded to bf16 for the product.
__global__ void __launch_bounds__(256) gated_dp_kernel(const uint16_t* dh, const uint16_t* g, const uint16_t* u,
                                                       uint16_t* dg, uint16_t* du, long long n, int act) {
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
        const float d = bf16_bits_to_float(dh[i]), a = bf16_bits_to_float(g[i]), b = bf16_bits_to_float(u[i]);
        dg[i] = float_to_bf16_bits(d * b * act_grad(act, a));
        du[i] = float_to_bf16_bits(d * act_value(act, a));
    }
}

}  // namespace

int linear_dp_blocks(int64_t M) { return (int)((M + 255) / 256 < 64 ? (M + 255) / 256 : 64); }

cudaError_t launch_linear_dp(const uint16_t* dy, const uint16_t* pre, uint16_t* dp, float* dbias, float* sums,
                             int64_t M, int N, int act, cudaStream_t stream) {
    const int R = linear_dp_blocks(M);
    const int rows = (int)((M + R - 1) / R);
    linear_dp_kernel<<<dim3((N + 255) / 256, R), 256, 0, stream>>>(dy, pre, dp, dbias != nullptr ? sums : nullptr, M, N,
                                                                   act, rows);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || dbias == nullptr) return e;
    column_sum_kernel<<<(N + 255) / 256, 256, 0, stream>>>(sums, dbias, R, N);
    return cudaGetLastError();
}

cudaError_t launch_gated_dp(const uint16_t* dh, const uint16_t* g, const uint16_t* u, uint16_t* dg, uint16_t* du,
                            int64_t M, int F, int act, int num_sms, cudaStream_t stream) {
    gated_dp_kernel<<<num_sms * 8, 256, 0, stream>>>(dh, g, u, dg, du, (long long)M * F, act);
    return cudaGetLastError();
}

}  // namespace w4a16
