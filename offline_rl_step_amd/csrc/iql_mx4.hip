// V(s) with the operands of both hidden layers in microscaled 4 bits:
//   h1 = relu(q(s) q(W1)^T + b1), h2 = relu(q(h1) q(W2)^T + b2), V = w3 . h2 + b3,
// the value network of iql_forward_values ("GPU IQL + HER Porting Plan",
// "Rust Integration: gpu_iql_trainer.rs", forward_values) on the 4-bit product.
//
// Bound by the 4-bit fragments' way from L2 and the conversions between the layers:
// S 256, H 512, B 65536 46 to 48 us (bf16 pass 61, fp32 751; the least is 6.5 us of
// bytes, 8.3 of products at 6.2 PF and two launches), S 128, H 1024 83 to 87 (677); two
// networks of H 128, S 128, B 16384 15 us, more than their bf16 pass (6.9), for the
// weights' launch.  Layer by layer: S 1100, H 1056, B 65536 576 (fp32 4029), S 256, H
// 2048, B 65536 749 (7712).
//
// Up to 1024 states and hidden units: two launches, the weights' quantisation
// and the whole network (a workgroup takes 64 or 128 rows through both layers, h1 in
// 4 bits in LDS, V from registers).  Wider: layer by layer on the linear
// product.
#include "iqlher.h"
#include "launch.hpp"
#include "mx4_rows_block.hpp"

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

// W1 and W2 of every group, blocks along their rows, as fragments (FragsOfB): a
// thread quantises one block of 32.
struct WeightArgs {
    const float* params;  // [G][P]
    int64_t P;
    uint8_t* ws;          // [G] of `stride` bytes: codes and scales at the offsets below
    size_t stride, w1c, w1s, w2c, w2s;
    int S, H, H2;
    int n1, n2;           // lanes of W1's fragments, of W2's
};
__global__ __launch_bounds__(256) void iql_mx4_weights_kernel(WeightArgs a) {
    int e = blockIdx.x * 256 + threadIdx.x;
    if (e >= a.n1 + a.n2) return;
    const bool second = e >= a.n1;
    if (second) e -= a.n1;
    const int rows = second ? a.H2 : a.H, k = second ? a.H : a.S, steps = (k + 127) / 128;
    const int lane = e & 63, group = (e >> 6) / steps, step = (e >> 6) - group * steps;
    const int row = group * 16 + (lane & 15), k0 = step * 128 + (lane >> 4) * 32;
    const float* w = a.params + blockIdx.y * a.P + (second ? (int64_t)a.H * a.S + a.H : 0) + (int64_t)row * k + k0;
    float v[32];
    uint32_t amax = 0u;
#pragma unroll
    for (int j = 0; j < 32; j += 8) {
        const int left = row < rows ? k - k0 - j : 0;
        load8<IQLH_F32>(w + j, left < 0 ? 0 : left < 8 ? left : 8, v + j);
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) amax = umax2(amax, abs_bits(v[j]));
    const uint32_t s = mx4_scale(amax);
    uint4 c{0u, 0u, 0u, 0u};
    if (s != 255u) {
        const float inv = mx4_inverse(s);
        c = uint4{mx4_codes8(v, inv), mx4_codes8(v + 8, inv), mx4_codes8(v + 16, inv), mx4_codes8(v + 24, inv)};
    }
    uint8_t* base = a.ws + blockIdx.y * a.stride;
    ((uint4*)(base + (second ? a.w2c : a.w1c)))[e] = c;
    (base + (second ? a.w2s : a.w1s))[mx4_frag_scale_at(group, step, steps, lane)] = (uint8_t)s;
}

struct NetArgs {
    const void* x;
    int64_t ld;
    const float* params;
    int64_t P;
    const uint8_t* ws;
    size_t stride, w1c, w1s, w2c, w2s;
    int S, H, H2, G, B, kb4x, kb4h;
    ValueOut vo;
};

// largest of the lanes l, l ^ 16, l ^ 32, l ^ 48, in all of them
IQLH_DEV uint32_t group_umax(uint32_t v) {
    v = umax2(v, (uint32_t)__shfl_xor((int)v, 16, kWave));
    return umax2(v, (uint32_t)__shfl_xor((int)v, 32, kWave));
}
IQLH_DEV float group_sum(float v) {
    v += __shfl_xor(v, 16, kWave);
    return v + __shfl_xor(v, 32, kWave);
}

// ROWS rows through the network of every group.  Layer 1: a wave's chunk of 32
// hidden units is one block of h1, so its scale is found and its codes go to LDS
// from the lanes that hold its sums.  Layer 2: h2 w3 summed in the lanes, over
// the wave's chunks, the lanes of a row and the waves, in that order.
template <int ROWS, int NT, int XDT>
__global__ __launch_bounds__(NT, 2) void iql_mx4_net_kernel(NetArgs a) {
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ float part[NT / 64][ROWS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, blk = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * ROWS;
    const LdsRows<ROWS> tx(lds, a.kb4x), th(lds + mx4_lds_bytes<ROWS>(a.kb4x), a.kb4h);
    mx4_rows_to_lds<ROWS, NT, XDT>((const typename MxFloat<XDT>::type*)a.x, a.ld, a.B, m0, a.S, tx);
    __syncthreads();
    for (int g = 0; g < a.G; ++g) {
        const uint8_t* ws = a.ws + g * a.stride;
        const FragsOfB w1{(const uint4*)(ws + a.w1c), (const uint32_t*)(ws + a.w1s), a.kb4x / 4};
        const FragsOfB w2{(const uint4*)(ws + a.w2c), (const uint32_t*)(ws + a.w2s), a.kb4h / 4};
        const float* b1 = a.params + g * a.P + (int64_t)a.H * a.S;
        const float* b2 = b1 + a.H + (int64_t)a.H2 * a.H;
        const float* w3 = b2 + a.H2;
        const Mx4Out o1{nullptr, IQLH_F32, 1, 0, b1}, o2{nullptr, IQLH_F32, 1, 0, b2}, o3{nullptr, IQLH_F32, 0, 0, w3};
        float bias[kFrags][4], head[kFrags][4];
        mx4_rows_chunks<ROWS, NT>(
            tx, w1, a.kb4h * 32,
            [&](int64_t n0) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < kFrags; ++j) mx4_bias4(o1, n0 + 16 * j + 4 * blk, a.H, bias[j]);
            },
            [&](int64_t n0, mx_f4(&acc)[ROWS / 16][kFrags]) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < ROWS / 16; ++i) {
                    float y[8];
                    uint32_t amax = 0u;
#pragma unroll
                    for (int j = 0; j < kFrags; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            // hidden units past the last are zeros of the block
                            const bool in = n0 + 16 * j + 4 * blk + e < a.H;
                            const float z = in ? acc[i][j][e] + bias[j][e] : 0.f;
                            y[4 * j + e] = __builtin_elementwise_maximum(z, 0.f);
                            amax = umax2(amax, abs_bits(y[4 * j + e]));
                        }
                    const uint32_t s = mx4_scale(group_umax(amax));
                    const uint32_t w = s == 255u ? 0u : mx4_codes8(y, mx4_inverse(s));
                    const int row = 16 * i + r, b = (int)(n0 / 32);
                    uint8_t* p = th.codes + row * th.rb + b * 16 + 2 * blk;
                    *(uint16_t*)p = (uint16_t)w;               // units 4 blk .. + 3
                    *(uint16_t*)(p + 8) = (uint16_t)(w >> 16);  // units 16 + 4 blk .. + 3
                    if (blk == 0) th.scales[row * th.kb4 + b] = (uint8_t)s;
                }
            });
        __syncthreads();
        float v[ROWS / 16] = {};
        mx4_rows_chunks<ROWS, NT>(
            th, w2, a.H2,
            [&](int64_t n0) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < kFrags; ++j) {
                    mx4_bias4(o2, n0 + 16 * j + 4 * blk, a.H2, bias[j]);
                    mx4_bias4(o3, n0 + 16 * j + 4 * blk, a.H2, head[j]);
                }
            },
            [&](int64_t n0, mx_f4(&acc)[ROWS / 16][kFrags]) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < ROWS / 16; ++i)
#pragma unroll
                    for (int j = 0; j < kFrags; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const bool in = n0 + 16 * j + 4 * blk + e < a.H2;
                            const float z = in ? acc[i][j][e] + bias[j][e] : 0.f;
                            v[i] = fmaf(__builtin_elementwise_maximum(z, 0.f), head[j][e], v[i]);
                        }
            });
#pragma unroll
        for (int i = 0; i < ROWS / 16; ++i) {
            const float s = group_sum(v[i]);
            if (blk == 0) part[wave][16 * i + r] = s;
        }
        __syncthreads();  // also: every wave is done with this group's h1
        if (threadIdx.x < ROWS && m0 + threadIdx.x < a.B) {
            const int row = threadIdx.x;
            float sum = part[0][row];
#pragma unroll
            for (int w = 1; w < NT / 64; ++w) sum += part[w][row];
            write_value(a.vo, g, a.B, (int)(m0 + row), sum + w3[a.H2]);
        }
        __syncthreads();
    }
}

size_t up16(size_t x) { return (x + 15) / 16 * 16; }

bool one_launch(const IqlDims& d) { return d.S <= kRowsMaxBlocks * 32 && d.H <= kRowsMaxBlocks * 32; }

struct Layout {
    size_t w1c, w1s, w2c, w2s, group, h1, h2, product, total;
    int chunk;
};

Layout layout(const IqlDims& d, int B) {
    Layout l{};
    const size_t k1 = (d.S + 31) / 32, k2 = (d.H + 31) / 32;
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t p = at; at += up16(bytes); return p; };
    if (one_launch(d)) {
        l.w1c = take(mx4_frag_code_bytes(d.H, k1));
        l.w1s = take(mx4_frag_scale_bytes(d.H, k1));
        l.w2c = take(mx4_frag_code_bytes(d.H2, k2));
        l.w2s = take(mx4_frag_scale_bytes(d.H2, k2));
        l.group = at;
        l.total = at * d.G;
        return l;
    }
    l.w1c = take(k1 * 16 * d.H);
    l.w1s = take(k1 * d.H);
    l.w2c = take(k2 * 16 * d.H2);
    l.w2s = take(k2 * d.H2);
    l.chunk = B < kChunkRows ? B : kChunkRows;
    l.h1 = take(sizeof(float) * (size_t)l.chunk * d.H);
    l.h2 = take(sizeof(float) * (size_t)l.chunk * d.H2);
    size_t product = 0;
    for (int rows : {l.chunk, B % l.chunk ? B % l.chunk : l.chunk})  // the chunks and what is left
        for (size_t bytes : {mx4_workspace_bytes(rows, d.H, d.S), mx4_workspace_bytes(rows, d.H2, d.H)})
            if (bytes > product) product = bytes;
    l.product = take(product);
    l.total = at;
    return l;
}

template <int ROWS, int NT, int XDT>
hipError_t launch_net(const NetArgs& a, hipStream_t stream) {
    const int bytes = mx4_lds_bytes<ROWS>(a.kb4x) + mx4_lds_bytes<ROWS>(a.kb4h);
    auto kernel = iql_mx4_net_kernel<ROWS, NT, XDT>;
    if (bytes > 60 << 10) {
        hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, dim3((a.B + ROWS - 1) / ROWS), dim3(NT), bytes, stream, a);
    return hipGetLastError();
}
// 128 rows a workgroup halve the weights' traffic from L2, 64 rows give twice
// the workgroups.  64 | 128 rows, us: S 256, H 512, B 65536 53.8 | 45.6, 32768 29.6 | 26.2, 16384
// 26.8 | 24.3; S 128, H 1024, B 65536 103 | 83; S 128, H 256, B 32768 16.8 | 15.5, 16384
// 14.9 | 15.2; S 64, H 192, B 65536 30.2 | 27.5; S 128, H 128, B 65536 21.5 | 23.2, two networks
// of 16384 15.2 | 18.9
template <int XDT>
hipError_t launch_net(const NetArgs& a, hipStream_t stream) {
    const bool wide = a.H >= 256 && a.B >= 128 * 256;
    return wide ? launch_net<128, 512, XDT>(a, stream) : launch_net<64, 256, XDT>(a, stream);
}

}  // namespace

size_t iql_mx4_workspace_bytes(const IqlDims& d, int B) { return layout(d, B).total; }

hipError_t launch_iql_mx4_forward(const IqlDims& d, const IqlBuffers& b, const void* states, int dtype, int64_t ld,
                                  int B, const ValueOut& vo, void* workspace, hipStream_t stream) {
    const Layout l = layout(d, B);
    uint8_t* ws = (uint8_t*)workspace;
    if (one_launch(d)) {
        const int n1 = (int)(mx4_frag_code_bytes(d.H, (d.S + 31) / 32) / 16), n2 = (int)(mx4_frag_code_bytes(d.H2, (d.H + 31) / 32) / 16);
        WeightArgs w{b.params, d.P, ws, l.group, l.w1c, l.w1s, l.w2c, l.w2s, d.S, d.H, d.H2, n1, n2};
        hipLaunchKernelGGL(iql_mx4_weights_kernel, dim3((n1 + n2 + 255) / 256, d.G), dim3(256), 0, stream, w);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const NetArgs a{states, ld, b.params, d.P, ws, l.group, l.w1c, l.w1s, l.w2c, l.w2s, d.S, d.H, d.H2, d.G, B,
                        (d.S + 127) / 128 * 4, (d.H + 127) / 128 * 4, vo};
        return dtype == IQLH_F32 ? launch_net<IQLH_F32>(a, stream) : launch_net<IQLH_BF16>(a, stream);
    }
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
