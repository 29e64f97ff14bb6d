// ffn.cu -- the activations of the feed-forward products as their kernel takes them, and the elementwise
// steps of the backward passes.
//
// The products' operand is fp16 with a scale per token: x' = fp16(x 2^-e), e such that the token's
// largest |x'| lies in [2^14, 2^15); backward, x is the gradient behind the activation's derivative.  bf16
// values keep all their 8 bits down to 2^-28 of the token's largest one, and below that an error
// of at most 2^-39 of it is left, under the fp32 sums' own; gradients are rounded to 11 bits.
//
// Memory bound: 16-byte loads and stores, each row read from device memory once (a second pass over a
// row comes from the caches).  The bias gradient's column sums are taken in the same pass as the gradients:
// each block leaves its rows' fp32 sums in the workspace, and the product's epilogue warps add them up while
// its first tile accumulates.  The order of the additions is fixed.
#include "act.cuh"
#include "common.cuh"
#include "internal.h"

namespace w4a16 {

namespace {

constexpr int kDpCols = 256;  // columns per block: 32 threads x 8
constexpr int kDpRowThreads = 16;

__device__ __forceinline__ void unpack8(const uint4& v, float f[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = u4_get(v, i);
        f[2 * i] = __uint_as_float(w << 16);
        f[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8_half(const float f[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 b = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// e for a token whose largest magnitude has the fp32 bits `bits`: over 2^e it lies in [2^top, 2^(top+1)).
// e is kept in the range of the normal numbers.  With an infinity or a NaN in the token, e is that of the
// largest finite value, so that no finite one becomes infinite beside it.
__device__ __forceinline__ int token_exponent(uint32_t bits, int top) {
    const int E = (int)(bits >> 23);
    if (bits == 0u) return 0;
    return max(min(E, 254) - 127 - top, -110);
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ uint32_t max_abs8(const uint4& v, uint32_t m) {  // of packed bf16, as bf16 bits in both halves
    m = __vmaxu2(m, v.x & 0x7FFF7FFFu);
    m = __vmaxu2(m, v.y & 0x7FFF7FFFu);
    m = __vmaxu2(m, v.z & 0x7FFF7FFFu);
    return __vmaxu2(m, v.w & 0x7FFF7FFFu);
}

// The block's largest value; buf: 32 words.
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* buf) {
    v = __reduce_max_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    const int l = threadIdx.x & 31;
    v = __reduce_max_sync(0xffffffffu, l < (int)(blockDim.x >> 5) ? buf[l] : 0u);
    __syncthreads();  // buf may be used again
    return v;
}

// Waits for the previous kernel on the stream, which the launch overlapped, and lets the next one be scheduled: in
// this order, so that whatever was complete before this kernel is so for the product, which fetches weights at
// once.
__device__ __forceinline__ void stream_order() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// One block per row: row_scale[m] = 2^e and out = fp16(x 2^-e).
__global__ void __launch_bounds__(256) half_rows_kernel(const uint16_t* x, uint16_t* out, float* row_scale, long long M,
                                                        int K) {
    __shared__ uint32_t buf[32];
    stream_order();
    constexpr int V = 4;  // chunks of a row that stay in registers
    for (long long m = blockIdx.x; m < M; m += gridDim.x) {
        const uint16_t* row = x + m * K;
        uint4 a[V];
        uint32_t mx = 0u;
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * 256 + threadIdx.x) * 8;
            if (k < K) {
                a[c] = *reinterpret_cast<const uint4*>(row + k);
                mx = max_abs8(a[c], mx);
            }
        }
        for (int k = (V * 256 + threadIdx.x) * 8; k < K; k += 2048) mx = max_abs8(*reinterpret_cast<const uint4*>(row + k), mx);
        mx = block_max(max(mx & 0xFFFFu, mx >> 16), buf);
        const int e = token_exponent(mx << 16, 14);
        if (threadIdx.x == 0) row_scale[m] = exp2_int(e);
        const float s = exp2_int(-e);
        auto put = [&](const uint4& v, int k) {
            float f[8];
            unpack8(v, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= s;
            *reinterpret_cast<uint4*>(out + m * K + k) = pack8_half(f);
        };
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * 256 + threadIdx.x) * 8;
            if (k < K) put(a[c], k);
        }
        for (int k = (V * 256 + threadIdx.x) * 8; k < K; k += 2048) put(*reinterpret_cast<const uint4*>(row + k), k);
    }
}

// One block per row: row_scale[m] = 2^e for dp = dy * act'(pre).  The largest dp may be far below the largest dy, whose
// unit may be a dead one.
template <int ACT>
__global__ void __launch_bounds__(512) dp_scale_kernel(const uint16_t* dy, const uint16_t* pre, float* row_scale, long long M,
                                                       int N) {
    __shared__ uint32_t buf[32];
    stream_order();
    for (long long m = blockIdx.x; m < M; m += gridDim.x) {
        uint32_t mx = 0u;
#pragma unroll 4
        for (int k = threadIdx.x * 8; k < N; k += 512 * 8) {
            float v[8];
            unpack8(*reinterpret_cast<const uint4*>(dy + m * N + k), v);
            if constexpr (ACT != W4A16_ACT_NONE) {
                float p[8];
                unpack8(*reinterpret_cast<const uint4*>(pre + m * N + k), p);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= act_grad<ACT>(p[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) mx = max(mx, __float_as_uint(v[e]) & 0x7FFFFFFFu);
        }
        const int e = token_exponent(block_max(mx, buf), 14);
        if (threadIdx.x == 0) row_scale[m] = exp2_int(e);
    }
}

// Rows too long for linear_dp_kernel's registers: dp = fp16(dy * act'(pre) / row_scale), with the scales from
// dp_scale_kernel, over `rows` rows per block.  sums: [gridDim.y][N], nullptr without a bias gradient.
template <int ACT>
__global__ void __launch_bounds__(32 * kDpRowThreads) linear_dp_long_kernel(const uint16_t* dy, const uint16_t* pre,
                                                                            uint16_t* dp, const float* row_scale,
                                                                            float* sums, long long M, int N, int rows) {
    __shared__ float part[kDpRowThreads][kDpCols];
    stream_order();  // the rows' scales come from the kernel before
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
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] += v[e];
            const float s = 1.0f / row_scale[m];  // a power of two: exact
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= s;
            *reinterpret_cast<uint4*>(dp + m * N + n) = pack8_half(v);
        }
    }
    if (sums == nullptr) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) part[rt][lane * 8 + e] = a[e];
    __syncthreads();
    const int c = threadIdx.x & (kDpCols - 1), nc = blockIdx.x * kDpCols + c;  // one column per thread
    if (threadIdx.x >= kDpCols || nc >= N) return;
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < kDpRowThreads; ++r) s += part[r][c];
    sums[(size_t)blockIdx.y * N + nc] = s;
}

constexpr int kDpDepth = 4;

// dp = fp16(dy * act'(pre) / row_scale), one row per block at a time, V chunks of 8 columns per thread.  Rows
// come through a ring of `depth` as in gated_dp_kernel; a row's values and the block's column sums stay in
// registers.  sums: [gridDim.x][N], nullptr without a bias gradient.  (1023 x 5120 with GELU: 13 us from
// device memory; the second of the two kernels for longer rows alone takes 17 us.)
template <int ACT, int V>
__global__ void __launch_bounds__(512) linear_dp_kernel(const uint16_t* dy, const uint16_t* pre, uint16_t* dp,
                                                        float* row_scale, float* sums, long long M, int N, int depth,
                                                        unsigned* err) {
    constexpr int kSrcs = ACT == W4A16_ACT_NONE ? 1 : 2;
    __shared__ uint32_t buf[32];
    __shared__ __align__(8) uint64_t full[kDpDepth];
    extern __shared__ __align__(128) uint16_t ring[];  // [depth][dy row, pre row]
    stream_order();
    const int T = blockDim.x;
    auto load_row = [&](int slot, long long m) {  // thread 0; the slot's earlier row has been read
        mbar_arrive_expect_tx(&full[slot], (uint32_t)(2 * N * kSrcs));
        uint16_t* dst = ring + (size_t)slot * kSrcs * N;
        bulk_load(dst, dy + (size_t)m * N, (uint32_t)(2 * N), &full[slot]);
        if (kSrcs == 2) bulk_load(dst + N, pre + (size_t)m * N, (uint32_t)(2 * N), &full[slot]);
    };
    if (threadIdx.x == 0) {
        for (int i = 0; i < depth; ++i) mbar_init(&full[i], 1);
        fence_mbarrier_init();
        for (int i = 0; i < depth; ++i) {
            const long long m = blockIdx.x + (long long)i * gridDim.x;
            if (m < M) load_row(i, m);
        }
    }
    __syncthreads();
    float acc[V][8] = {};
    int slot = 0;
    uint32_t phase = 0;
    bool dead = false;
    for (long long m = blockIdx.x; m < M; m += gridDim.x) {
        const uint16_t* src = ring + (size_t)slot * kSrcs * N;
        if (!dead && !mbar_wait_bounded(&full[slot], phase)) {  // as in gated_dp_kernel
            dead = true;
            record_error(err, kErrTimeout);
        }
        float v[V][8];
        uint32_t mx = 0u;
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + threadIdx.x) * 8;
            if (k < N) {
                unpack8(*reinterpret_cast<const uint4*>(src + k), v[c]);
                if constexpr (kSrcs == 2) {
                    float q[8];
                    unpack8(*reinterpret_cast<const uint4*>(src + N + k), q);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[c][e] *= act_grad<ACT>(q[e]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    acc[c][e] += v[c][e];
                    mx = max(mx, __float_as_uint(v[c][e]) & 0x7FFFFFFFu);
                }
            }
        }
        fence_proxy_async_smem();  // this thread's reads of the slot, before its refill
        const int e = token_exponent(block_max(mx, buf), 14);
        const long long next = m + (long long)depth * gridDim.x;  // every thread has its part of the row
        if (threadIdx.x == 0 && next < M) load_row(slot, next);
        if (++slot == depth) {
            slot = 0;
            phase ^= 1;
        }
        if (threadIdx.x == 0) row_scale[m] = exp2_int(e);
        const float s = exp2_int(-e);
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int k = (c * T + threadIdx.x) * 8;
            if (k < N) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[c][i] *= s;
                *reinterpret_cast<uint4*>(dp + (size_t)m * N + k) = pack8_half(v[c]);
            }
        }
    }
    if (sums == nullptr) return;
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int k = (c * T + threadIdx.x) * 8;
        if (k < N) {
            float4* dst = reinterpret_cast<float4*>(sums + (size_t)blockIdx.x * N + k);
            dst[0] = make_float4(acc[c][0], acc[c][1], acc[c][2], acc[c][3]);
            dst[1] = make_float4(acc[c][4], acc[c][5], acc[c][6], acc[c][7]);
        }
    }
}

// dg = dh u act'(g), du = dh act(g), both in fp16 over the row's scale, side by side in dp [M][2 F]; one
// row per block at a time.  KEEP (F <= 32 threads): rows come by bulk copies through a ring of `depth`,
// so that the next rows are on their way while one is computed (a block's threads loading row by row
// took 76 us instead of 51 us at 2048 x 14336, 294 MB), and a row's values stay in registers between the
// maximum and the rounding.  Longer rows are read and computed twice.
template <int ACT, bool KEEP>
__global__ void __launch_bounds__(512) gated_dp_kernel(const uint16_t* dh, const uint16_t* g, const uint16_t* u,
                                                       uint16_t* dp, float* row_scale, long long M, int F, int depth,
                                                       unsigned* err) {
    constexpr int V = KEEP ? 4 : 1;
    __shared__ uint32_t buf[32];
    __shared__ __align__(8) uint64_t full[kDpDepth];
    extern __shared__ __align__(128) uint16_t ring[];  // KEEP: [depth][dh row, g row, u row]
    stream_order();
    const int T = blockDim.x;
    auto load_row = [&](int slot, long long m) {  // thread 0; the slot's earlier row has been read
        mbar_arrive_expect_tx(&full[slot], (uint32_t)(6 * F));
        uint16_t* dst = ring + (size_t)slot * 3 * F;
        bulk_load(dst, dh + (size_t)m * F, (uint32_t)(2 * F), &full[slot]);
        bulk_load(dst + F, g + (size_t)m * F, (uint32_t)(2 * F), &full[slot]);
        bulk_load(dst + 2 * F, u + (size_t)m * F, (uint32_t)(2 * F), &full[slot]);
    };
    if constexpr (KEEP) {
        if (threadIdx.x == 0) {
            for (int i = 0; i < depth; ++i) mbar_init(&full[i], 1);
            fence_mbarrier_init();
            for (int i = 0; i < depth; ++i) {
                const long long m = blockIdx.x + (long long)i * gridDim.x;
                if (m < M) load_row(i, m);
            }
        }
        __syncthreads();
    }
    int slot = 0;
    uint32_t phase = 0;
    bool dead = false;
    for (long long m = blockIdx.x; m < M; m += gridDim.x) {
        const size_t row = (size_t)m * F;
        const uint16_t* s0 = KEEP ? ring + (size_t)slot * 3 * F : dh + row;
        const uint16_t* s1 = KEEP ? s0 + F : g + row;
        const uint16_t* s2 = KEEP ? s0 + 2 * F : u + row;
        // a wait that runs out is recorded, and the thread goes on without waiting: the others may already be
        // at a barrier
        if (KEEP && !dead && !mbar_wait_bounded(&full[slot], phase)) {
            dead = true;
            record_error(err, kErrTimeout);
        }
        float x[V][8], y[V][8];
        auto values = [&](int k, float (&xv)[8], float (&yv)[8]) {
            float d[8], a[8], b[8];
            unpack8(*reinterpret_cast<const uint4*>(s0 + k), d);
            unpack8(*reinterpret_cast<const uint4*>(s1 + k), a);
            unpack8(*reinterpret_cast<const uint4*>(s2 + k), b);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xv[e] = d[e] * b[e] * act_grad<ACT>(a[e]);
                yv[e] = d[e] * act_value<ACT>(a[e]);
            }
        };
        uint32_t mx = 0u;
        auto largest = [&](const float (&xv)[8], const float (&yv)[8]) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                mx = max(mx, max(__float_as_uint(xv[e]) & 0x7FFFFFFFu, __float_as_uint(yv[e]) & 0x7FFFFFFFu));
        };
        if constexpr (KEEP) {
#pragma unroll
            for (int c = 0; c < V; ++c) {
                const int k = (c * T + threadIdx.x) * 8;
                if (k < F) {
                    values(k, x[c], y[c]);
                    largest(x[c], y[c]);
                }
            }
        } else {
            for (int k = threadIdx.x * 8; k < F; k += T * 8) {
                values(k, x[0], y[0]);
                largest(x[0], y[0]);
            }
        }
        if constexpr (KEEP) fence_proxy_async_smem();  // this thread's reads of the slot, before its refill
        const int e = token_exponent(block_max(mx, buf), 14);
        if constexpr (KEEP) {  // every thread has its part of the row
            const long long next = m + (long long)depth * gridDim.x;
            if (threadIdx.x == 0 && next < M) load_row(slot, next);
            if (++slot == depth) {
                slot = 0;
                phase ^= 1;
            }
        }
        if (threadIdx.x == 0) row_scale[m] = exp2_int(e);
        const float s = exp2_int(-e);
        auto put = [&](int k, float (&xv)[8], float (&yv)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                xv[i] *= s;
                yv[i] *= s;
            }
            *reinterpret_cast<uint4*>(dp + 2 * row + k) = pack8_half(xv);
            *reinterpret_cast<uint4*>(dp + 2 * row + F + k) = pack8_half(yv);
        };
        if constexpr (KEEP) {
#pragma unroll
            for (int c = 0; c < V; ++c) {
                const int k = (c * T + threadIdx.x) * 8;
                if (k < F) put(k, x[c], y[c]);
            }
        } else {
            for (int k = threadIdx.x * 8; k < F; k += T * 8) {
                values(k, x[0], y[0]);
                put(k, x[0], y[0]);
            }
        }
    }
}

}  // namespace

// Rows of column sums.  Up to 16384 columns one per block; two blocks per SM where two rows each fit beside
// one another (1023 x 5120 with GELU: 13 us, 14 us with one).  Beyond, runs of rows: blocks for one round of
// two per SM, at least 16 rows each, and few enough that adding the runs up stays short.
constexpr int kDpLongest = 16384;  // 512 threads with four chunks each

int linear_dp_runs(int64_t M, int N, int num_sms) {
    if (N <= kDpLongest) {
        const int64_t blocks = (int64_t)num_sms * (N <= 8192 ? 2 : 1);
        return (int)(M < blocks ? M : blocks);
    }
    const int64_t cols = (N + kDpCols - 1) / kDpCols, most = (M + kDpRowThreads - 1) / kDpRowThreads;
    const int64_t runs = 2 * num_sms / cols;
    return (int)(runs < 1 ? 1 : runs > 32 ? (most < 32 ? most : 32) : runs > most ? most : runs);
}

namespace {

int row_blocks(int64_t M, int num_sms) { return (int)(M < (int64_t)num_sms * 16 ? M : (int64_t)num_sms * 16); }

// A launch whose setup overlaps the previous kernel on the stream; the kernel waits for that one's end.
template <typename... Args>
cudaError_t launch_after(void (*fn)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

}  // namespace

cudaError_t launch_half_rows(const uint16_t* x, uint16_t* out, float* row_scale, int64_t M, int K, int num_sms,
                             cudaStream_t stream) {
    return launch_after(half_rows_kernel, dim3(row_blocks(M, num_sms)), 256, 0, stream, x, out, row_scale, (long long)M,
                        K);
}

cudaError_t launch_linear_dp(const uint16_t* dy, const uint16_t* pre, uint16_t* dp, float* row_scale, float* sums,
                             int* sum_rows, int64_t M, int N, int act, int num_sms, unsigned* err, cudaStream_t stream) {
    *sum_rows = 0;
    if (act == W4A16_ACT_NONE && sums == nullptr) return launch_half_rows(dy, dp, row_scale, M, N, num_sms, stream);
    const int runs = linear_dp_runs(M, N, num_sms);
    if (N <= kDpLongest) {
        const int V = N <= 4096 ? 1 : N <= 8192 ? 2 : 4, threads = (N / (8 * V) + 31) / 32 * 32;
        const size_t row = (size_t)2 * N * (act == W4A16_ACT_NONE ? 1 : 2);
        const size_t ring = N <= 8192 ? kRingSmemBytes / 2 : kRingSmemBytes;
        const int depth = row * kDpDepth <= ring ? kDpDepth : (int)(ring / row);
        const size_t smem = depth * row;
        using Kernel = void (*)(const uint16_t*, const uint16_t*, uint16_t*, float*, float*, long long, int, int, unsigned*);
        Kernel fn = nullptr;
#define W4A16_DP(ACT) \
    case ACT: fn = V == 1 ? linear_dp_kernel<ACT, 1> : V == 2 ? linear_dp_kernel<ACT, 2> : linear_dp_kernel<ACT, 4>; break
        switch (act) {
            W4A16_DP(W4A16_ACT_NONE);
            W4A16_DP(W4A16_ACT_RELU);
            W4A16_DP(W4A16_ACT_SILU);
            W4A16_DP(W4A16_ACT_GELU);
            W4A16_DP(W4A16_ACT_GELU_TANH);
            default: return cudaErrorInvalidValue;
        }
#undef W4A16_DP
        const cudaError_t e = allow_ring_smem(fn);
        if (e != cudaSuccess) return e;
        if (sums != nullptr) *sum_rows = runs;
        return launch_after(fn, dim3(runs), threads, smem, stream, dy, pre, dp, row_scale, sums, (long long)M, N, depth, err);
    }
    using Scale = void (*)(const uint16_t*, const uint16_t*, float*, long long, int);
    using Long = void (*)(const uint16_t*, const uint16_t*, uint16_t*, const float*, float*, long long, int, int);
    Scale scale = nullptr;
    Long fn = nullptr;
#define W4A16_DP(ACT) \
    case ACT: scale = dp_scale_kernel<ACT>; fn = linear_dp_long_kernel<ACT>; break
    switch (act) {
        W4A16_DP(W4A16_ACT_NONE);
        W4A16_DP(W4A16_ACT_RELU);
        W4A16_DP(W4A16_ACT_SILU);
        W4A16_DP(W4A16_ACT_GELU);
        W4A16_DP(W4A16_ACT_GELU_TANH);
        default: return cudaErrorInvalidValue;
    }
#undef W4A16_DP
    const cudaError_t e = launch_after(scale, dim3(row_blocks(M, num_sms)), 512, 0, stream, dy, pre, row_scale, (long long)M, N);
    if (e != cudaSuccess) return e;
    const int rows = (int)((M + runs - 1) / runs);
    const dim3 grid((N + kDpCols - 1) / kDpCols, (unsigned)((M + rows - 1) / rows));
    if (sums != nullptr) *sum_rows = (int)grid.y;
    return launch_after(fn, grid, 32 * kDpRowThreads, 0, stream, dy, pre, dp, (const float*)row_scale, sums, (long long)M, N,
                        rows);
}

cudaError_t launch_gated_dp(const uint16_t* dh, const uint16_t* g, const uint16_t* u, uint16_t* dp, float* row_scale,
                            int64_t M, int F, int act, int num_sms, unsigned* err, cudaStream_t stream) {
    const bool keep = F <= 16384;  // 512 threads with four chunks each
    const int threads = keep ? (F / 32 + 31) / 32 * 32 : 512;
    // resident blocks by registers (128 a thread at most); two rows of each fit (32 columns per thread, three
    // sources of 2 bytes)
    constexpr size_t kRing = kRingSmemBytes;
    const size_t row = (size_t)6 * F;
    static_assert(2 * 512 * 32 * 6 <= kRing, "two rows of every block");
    const int blocks = 512 / threads > 8 ? 8 : 512 / threads;
    int depth = keep ? (int)(kRing / blocks / row) : 0;
    depth = depth > kDpDepth ? kDpDepth : depth;
    const int64_t cap = (int64_t)num_sms * (keep ? blocks : 4);
    const int grid = (int)(M < cap ? M : cap);
    const size_t smem = (size_t)depth * row;
    using Kernel = void (*)(const uint16_t*, const uint16_t*, const uint16_t*, uint16_t*, float*, long long, int, int,
                            unsigned*);
    Kernel fn = nullptr;
#define W4A16_DP(ACT) \
    case ACT: fn = keep ? gated_dp_kernel<ACT, true> : gated_dp_kernel<ACT, false>; break
    switch (act) {
        W4A16_DP(W4A16_ACT_NONE);
        W4A16_DP(W4A16_ACT_RELU);
        W4A16_DP(W4A16_ACT_SILU);
        W4A16_DP(W4A16_ACT_GELU);
        W4A16_DP(W4A16_ACT_GELU_TANH);
        default: return cudaErrorInvalidValue;
    }
#undef W4A16_DP
    if (keep) {
        const cudaError_t e = allow_ring_smem(fn);
        if (e != cudaSuccess) return e;
    }
    return launch_after(fn, dim3(grid), threads, smem, stream, dh, g, u, dp, row_scale, (long long)M, F, depth, err);
}

}  // namespace w4a16
