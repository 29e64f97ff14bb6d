/*
 * Two host threads call the same operators at different widths, each with its own stream, operands and
 * workspace, and count the calls that are refused.  The kernels behind them are the same instances with
 * different amounts of dynamic shared memory.  Prints "ok" when no call was refused.
 *   two_threads            the norms and the backward passes, at two widths
 *   two_threads quantize   the quantizer, at two group sizes
 */
#include <cuda_runtime.h>
#include <pthread.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "w4a16.h"

#define TOKENS 400
#define CALLS 2000

typedef struct {
    int64_t width;
    int refused;
} work;

static void* device_zeros(size_t bytes) {
    void* p = NULL;
    if (cudaMalloc(&p, bytes) != cudaSuccess || cudaMemset(p, 0, bytes) != cudaSuccess) return NULL;
    return p;
}

static void* run(void* arg) {
    work* w = (work*)arg;
    const int64_t n = w->width, k = 1024;
    const size_t row = (size_t)TOKENS * (size_t)n * 2;
    cudaStream_t stream;
    w4a16_weights layer;
    uint32_t* qweight = (uint32_t*)device_zeros((size_t)n * (size_t)k / 2);
    uint16_t* scales = (uint16_t*)device_zeros((size_t)n * (size_t)(k / 128) * 2);
    uint32_t* zeros = (uint32_t*)device_zeros((size_t)n * (size_t)(k / 128) / 2);
    uint16_t* a = (uint16_t*)device_zeros(row);
    uint16_t* b = (uint16_t*)device_zeros(row);
    uint16_t* c = (uint16_t*)device_zeros(row);
    uint16_t* y = (uint16_t*)device_zeros(row);
    uint16_t* h = (uint16_t*)device_zeros(row);
    uint16_t* dx = (uint16_t*)device_zeros((size_t)TOKENS * (size_t)k * 2);
    uint16_t* weight = (uint16_t*)device_zeros((size_t)n * 2);
    float* sums = (float*)device_zeros((size_t)n * 4);
    size_t need = w4a16_fused_workspace_bytes(W4A16_OP_GATED_BACKWARD, TOKENS, n, k);
    size_t more = w4a16_fused_workspace_bytes(W4A16_OP_LINEAR_BACKWARD, TOKENS, n, k);
    void* ws;
    int i;
    w->refused = -1;
    if (more > need) need = more;
    more = w4a16_fused_workspace_bytes(W4A16_OP_RMSNORM_BACKWARD, TOKENS, 0, n);
    if (more > need) need = more;
    ws = device_zeros(need);
    if (!qweight || !scales || !zeros || !a || !b || !c || !y || !h || !dx || !weight || !sums || !ws) return NULL;
    if (cudaStreamCreateWithFlags(&stream, cudaStreamNonBlocking) != cudaSuccess) return NULL;
    if (cudaDeviceSynchronize() != cudaSuccess) return NULL;
    layer.qweight = qweight;
    layer.scales = scales;
    layer.zeros = zeros;
    w->refused = 0;
    for (i = 0; i < CALLS; ++i) {
        w->refused += awq_rmsnorm(a, b, weight, NULL, 1e-6f, h, y, TOKENS, n, stream) != W4A16_OK;
        w->refused += awq_rmsnorm_backward(a, b, weight, NULL, c, 1e-6f, y, sums, TOKENS, n, ws, need, stream) != W4A16_OK;
        w->refused += w4a16_linear_fused_backward(a, b, &layer, dx, sums, TOKENS, n, k, 128, W4A16_ACT_SILU, ws, need,
                                                  stream) != W4A16_OK;
        w->refused += w4a16_gated_backward(a, b, c, &layer, &layer, dx, TOKENS, n, k, 128, W4A16_ACT_SILU, ws, need,
                                           stream) != W4A16_OK;
        if (i % 100 == 99 && cudaStreamSynchronize(stream) != cudaSuccess) w->refused += 1;
    }
    if (cudaStreamSynchronize(stream) != cudaSuccess) w->refused += 1;
    return NULL;
}

static void* quantize(void* arg) {
    work* w = (work*)arg; /* width: the group size */
    const int64_t n = 128, k = 32768;
    cudaStream_t stream;
    float* weights = (float*)device_zeros((size_t)(n * k) * 4);
    float* act = (float*)device_zeros((size_t)k * 4);
    uint32_t* qweight = (uint32_t*)device_zeros((size_t)(n * k) / 2);
    uint16_t* scales = (uint16_t*)device_zeros((size_t)(n * (k / 128)) * 2);
    uint32_t* zeros = (uint32_t*)device_zeros((size_t)(n * (k / 128)) / 2);
    float* s = (float*)device_zeros((size_t)k * 4);
    int i;
    w->refused = -1;
    if (!weights || !act || !qweight || !scales || !zeros || !s) return NULL;
    if (cudaStreamCreateWithFlags(&stream, cudaStreamNonBlocking) != cudaSuccess) return NULL;
    if (cudaDeviceSynchronize() != cudaSuccess) return NULL;
    w->refused = 0;
    for (i = 0; i < CALLS; ++i) {
        w->refused += awq_quantize(weights, act, 0.5f, n, k, w->width, qweight, scales, zeros, s, stream) != W4A16_OK;
        if (i % 100 == 99 && cudaStreamSynchronize(stream) != cudaSuccess) w->refused += 1;
    }
    if (cudaStreamSynchronize(stream) != cudaSuccess) w->refused += 1;
    return NULL;
}

int main(int argc, char** argv) {
    const int quantizes = argc > 1 && strcmp(argv[1], "quantize") == 0;
    work works[2] = {{8192, 0}, {5120, 0}};
    pthread_t threads[2];
    int i;
    if (quantizes) {
        works[0].width = 32768;
        works[1].width = 2048;
    }
    if (cudaSetDevice(0) != cudaSuccess) return 2;
    for (i = 0; i < 2; ++i)
        if (pthread_create(&threads[i], NULL, quantizes ? quantize : run, &works[i]) != 0) return 2;
    for (i = 0; i < 2; ++i) pthread_join(threads[i], NULL);
    if (w4a16_check_device_status(NULL) != W4A16_OK) return 3;
    if (works[0].refused != 0 || works[1].refused != 0) {
        printf("refused: %d and %d of %d calls each\n", works[0].refused, works[1].refused, (quantizes ? 1 : 4) * CALLS);
        return 1;
    }
    puts("ok");
    return 0;
}
