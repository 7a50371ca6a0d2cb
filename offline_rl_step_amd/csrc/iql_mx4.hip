// V(s) with the operands of both hidden layers in microscaled 4 bits:
//   h1 = relu(q(s) q(W1)^T + b1), h2 = relu(q(h1) q(W2)^T + b2), V = w3 . h2 + b3,
// the value network of iql_forward_values ("GPU IQL + HER Porting Plan",
// "Rust Integration: gpu_iql_trainer.rs", forward_values) on the 4-bit product.
#include "iqlher.h"
#include "launch.hpp"
#include "mx4_block.hpp"

namespace iqlh {

namespace {

constexpr int kChunkRows = 16384;  // rows whose activations the workspace holds at a time

// One wave per row: V = w3 . h2 + b3.
__global__ __launch_bounds__(256) void iql_mx4_head_kernel(const float* __restrict__ h2, const float* __restrict__ w3,
                                                           int H2, int rows, int row0, int g, int B, ValueOut vo) {
    const int row = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (row >= rows) return;
    const float* h = h2 + (int64_t)row * H2;
    float s = 0.f;
    for (int n = lane; n < H2; n += kWave) s = fmaf(w3[n], h[n], s);
    s = wave_sum(s);
    if (lane == 0) write_value(vo, g, B, row0 + row, s + w3[H2]);  // b3 follows w3
}

size_t up16(size_t x) { return (x + 15) / 16 * 16; }

struct Layout {
    size_t w1c, w1s, w2c, w2s, h1, h2, product, total;
    int chunk;
};

Layout layout(const IqlDims& d, int B) {
    Layout l;
    const size_t k1 = (d.S + 31) / 32, k2 = (d.H + 31) / 32;
    l.chunk = B < kChunkRows ? B : kChunkRows;
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t p = at; at += up16(bytes); return p; };
    l.w1c = take(k1 * 16 * d.H);
    l.w1s = take(k1 * d.H);
    l.w2c = take(k2 * 16 * d.H2);
    l.w2s = take(k2 * d.H2);
    l.h1 = take(sizeof(float) * (size_t)l.chunk * d.H);
    l.h2 = take(sizeof(float) * (size_t)l.chunk * d.H2);
    const size_t p1 = mx4_workspace_bytes(l.chunk, d.H, d.S), p2 = mx4_workspace_bytes(l.chunk, d.H2, d.H);
    l.product = take(p1 > p2 ? p1 : p2);
    l.total = at;
    return l;
}

}  // namespace

size_t iql_mx4_workspace_bytes(const IqlDims& d, int B) { return layout(d, B).total; }

hipError_t launch_iql_mx4_forward(const IqlDims& d, const IqlBuffers& b, const void* states, int dtype, int64_t ld,
                                  int B, const ValueOut& vo, void* workspace, hipStream_t stream) {
    const Layout l = layout(d, B);
    uint8_t* ws = (uint8_t*)workspace;
    float* h1 = (float*)(ws + l.h1);
    float* h2 = (float*)(ws + l.h2);
    const Mx4Mat w1{ws + l.w1c, ws + l.w1s, d.H, d.S}, w2{ws + l.w2c, ws + l.w2s, d.H2, d.H};
    const size_t es = dtype == IQLH_F32 ? 4 : 2;
    for (int g = 0; g < d.G; ++g) {
        const float* W1 = b.params + (int64_t)g * d.P;
        const float* b1 = W1 + (int64_t)d.H * d.S;
        const float* W2 = b1 + d.H;
        const float* b2 = W2 + (int64_t)d.H2 * d.H;
        hipError_t e = launch_mx4_quantize(W1, IQLH_F32, d.S, false, w1, stream);
        if (e == hipSuccess) e = launch_mx4_quantize(W2, IQLH_F32, d.H, false, w2, stream);
        for (int r0 = 0; r0 < B && e == hipSuccess; r0 += l.chunk) {
            const int rows = B - r0 < l.chunk ? B - r0 : l.chunk;
            const void* x = (const char*)states + (size_t)r0 * ld * es;
            e = launch_mx4_linear(x, dtype, ld, rows, w1, Mx4Out{h1, IQLH_F32, 1, d.H, b1}, ws + l.product, stream);
            if (e == hipSuccess)
                e = launch_mx4_linear(h1, IQLH_F32, d.H, rows, w2, Mx4Out{h2, IQLH_F32, 1, d.H2, b2}, ws + l.product,
                                      stream);
            if (e != hipSuccess) break;
            hipLaunchKernelGGL(iql_mx4_head_kernel, dim3((rows + 3) / 4), dim3(256), 0, stream, h2, b2 + d.H2, d.H2,
                               rows, r0, g, B, vo);
            e = hipGetLastError();
        }
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace iqlh
