// ffn.cu -- the products of the feed-forward operators: y = act(x W^T + b) + r, h = act(x Wg^T) (x Wu^T)
// and their backward products dx = dp W (contraction over the output channels).
//
// fp32 throughout: weights are dequantized to fp32 in shared memory, 64 x 64 output tiles, 4 x 4
// outputs per thread, 32 deep.
#include "act.cuh"
#include "common.cuh"
#include "internal.h"

namespace w4a16 {

namespace {

constexpr int kTile = 64, kDepth = 32;

__device__ __forceinline__ float weight_at(const PackedWeights& w, int n, int k, int N, int K, int gs) {
    const uint32_t word = w.qweight[(size_t)n * (K / 8) + k / 8];
    const int e = k & 7;
    const int nib = (e >> 1) + 4 * (e & 1);  // nibble of element e: ORDER = 0 2 4 6 1 3 5 7
    const int g = k / gs;
    const uint32_t z = (w.zeros[(size_t)g * (N / 8) + n / 8] >> (4 * (n & 7))) & 15u;
    return ((float)((word >> (4 * nib)) & 15u) - (float)z) * fp16_bits_to_float(w.scales[(size_t)g * N + n]);
}

// BACK: out[m][k] = sum_n a[m][n] W[n][k]; else out[m][n] = sum_k a[m][k] W[n][k].
// TWO: two weight matrices: gated forward (two sums), or both summed (backward, a and a2).
template <bool BACK, bool TWO>
__global__ void __launch_bounds__(256) ffn_simple_kernel(const FfnArgs p) {
    __shared__ float As[kDepth][kTile + 1], As2[BACK && TWO ? kDepth : 1][kTile + 1];
    __shared__ float Ws[kDepth][kTile + 1], Ws2[TWO ? kDepth : 1][kTile + 1];
    const int cols = BACK ? p.K : p.N, depth = BACK ? p.N : p.K;
    const int c0 = blockIdx.x * kTile;
    const long long m0 = (long long)blockIdx.y * kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {}, acc2[4][4] = {};
    for (int d0 = 0; d0 < depth; d0 += kDepth) {
        for (int i = threadIdx.x; i < kTile * kDepth; i += 256) {
            const int d = i % kDepth, m = i / kDepth;
            const bool in = m0 + m < p.M;
            As[d][m] = in ? bf16_bits_to_float(p.a[(size_t)(m0 + m) * depth + d0 + d]) : 0.0f;
            if constexpr (BACK && TWO) As2[d][m] = in ? bf16_bits_to_float(p.a2[(size_t)(m0 + m) * depth + d0 + d]) : 0.0f;
            const int c = BACK ? i % kTile : i / kDepth, dw = BACK ? i / kTile : i % kDepth;
            const int n = BACK ? d0 + dw : c0 + c, k = BACK ? c0 + c : d0 + dw;
            Ws[dw][c] = weight_at(p.w, n, k, p.N, p.K, p.group_size);
            if constexpr (TWO) Ws2[dw][c] = weight_at(p.w2, n, k, p.N, p.K, p.group_size);
        }
        __syncthreads();
        for (int d = 0; d < kDepth; ++d) {
            float a[4], b[4], a2[4], b2[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = As[d][ty + 16 * i];
                b[i] = Ws[d][tx + 16 * i];
                if constexpr (TWO) b2[i] = Ws2[d][tx + 16 * i];
                if constexpr (BACK && TWO) a2[i] = As2[d][ty + 16 * i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
                    if constexpr (BACK && TWO) acc[i][j] = fmaf(a2[i], b2[j], acc[i][j]);
                    if constexpr (!BACK && TWO) acc2[i][j] = fmaf(a[i], b2[j], acc2[i][j]);
                }
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long m = m0 + ty + 16 * i;
        if (m >= p.M) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = c0 + tx + 16 * j;
            const size_t o = (size_t)m * cols + c;
            float v = acc[i][j];
            if constexpr (!BACK && TWO) {
                if (p.pre != nullptr) {
                    p.pre[o] = float_to_bf16_bits(v);
                    p.pre2[o] = float_to_bf16_bits(acc2[i][j]);
                }
                v = act_value(p.act, v) * acc2[i][j];
            } else if constexpr (!BACK) {
                if (p.bias != nullptr) v += bf16_bits_to_float(p.bias[c]);
                if (p.pre != nullptr) p.pre[o] = float_to_bf16_bits(v);
                v = act_value(p.act, v);
                if (p.residual != nullptr) v += bf16_bits_to_float(p.residual[o]);
            }
            p.y[o] = float_to_bf16_bits(v);
        }
    }
}

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

cudaError_t launch_ffn(const FfnArgs& a, bool back, bool two, cudaStream_t stream) {
    const dim3 grid((back ? a.K : a.N) / kTile, (unsigned)((a.M + kTile - 1) / kTile));
    if (back && two) ffn_simple_kernel<true, true><<<grid, 256, 0, stream>>>(a);
    else if (back) ffn_simple_kernel<true, false><<<grid, 256, 0, stream>>>(a);
    else if (two) ffn_simple_kernel<false, true><<<grid, 256, 0, stream>>>(a);
    else ffn_simple_kernel<false, false><<<grid, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace w4a16
