// Microscaled 4-bit matrices: quantisation along either axis, the values
// back, and the product whose left operand is quantised on the way.
#include "mx4_block.hpp"

namespace iqlh {

namespace {

constexpr int kNT = 256;

template <typename F>
hipError_t by_dtype(int dtype, F f) {
    if (dtype == IQLH_F32) f(std::integral_constant<int, IQLH_F32>());
    else if (dtype == IQLH_BF16) f(std::integral_constant<int, IQLH_BF16>());
    else f(std::integral_constant<int, IQLH_F16>());
    return hipGetLastError();
}

// ------------------------------------------------------------ quantisation
// Blocks along x's rows.  A thread converts 8 elements (one dword of codes),
// four neighbouring lanes a block; the groups of 8 are numbered over the
// padded matrix.
template <int DT>
__global__ __launch_bounds__(kNT) void mx4_quantize_kernel(const typename MxFloat<DT>::type* __restrict__ x, int64_t ld,
                                                           Mx4Mat q) {
    const int64_t gpr = q.kb() * 4;  // groups per row
    const int64_t ngroups = q.rows * gpr;
    for (int64_t g = (int64_t)blockIdx.x * kNT + threadIdx.x; g < (ngroups + 63) / 64 * 64;
         g += (int64_t)gridDim.x * kNT) {
        const bool in = g < ngroups;
        const int64_t row = in ? g / gpr : 0;
        const int64_t c0 = (in ? g - row * gpr : 0) * 8;
        const typename MxFloat<DT>::type* p = x + row * ld;
        float v[8];
        uint32_t amax = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool ok = in && c0 + j < q.cols;
            v[j] = ok ? MxFloat<DT>::get(p[c0 + j]) : 0.f;
            amax = umax2(amax, abs_bits(v[j]));
        }
        amax = quad_umax(amax);
        const uint32_t s = mx4_scale(amax);
        const uint32_t w = s == 255u ? 0u : mx4_codes8(v, mx4_inverse(s));
        if (in) {
            ((uint32_t*)q.codes)[g] = w;
            if ((g & 3) == 0) q.scales[g >> 2] = (uint8_t)s;
        }
    }
}

// Blocks along x's columns: x is [q.cols][ld].  A workgroup takes 64 columns
// of x (rows of q) and 256 of its rows: a lane reads its column, 32 rows a
// block, neighbouring lanes neighbouring addresses; the codes pass through LDS
// so that a row of q is written 128 bytes at a time.
template <int DT>
__global__ __launch_bounds__(kNT) void mx4_quantize_columns_kernel(const typename MxFloat<DT>::type* __restrict__ x,
                                                                   int64_t ld, Mx4Mat q, int row_tiles) {
    __shared__ uint4 codes[64][9];  // 9: lanes of a store to one block column fall on different banks
    __shared__ uint8_t scales[64][8];
    const int64_t kb = q.kb();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t r0 = (int64_t)(blockIdx.x % row_tiles) * 64, b0 = (int64_t)(blockIdx.x / row_tiles) * 8;
    const int64_t r = r0 + lane;
    for (int i = wave; i < 8; i += 4) {
        const int64_t k0 = (b0 + i) * 32;
        float v[32];
        uint32_t amax = 0u;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const bool ok = r < q.rows && k0 + j < q.cols;
            v[j] = ok ? MxFloat<DT>::get(x[(k0 + j) * ld + r]) : 0.f;
            amax = umax2(amax, abs_bits(v[j]));
        }
        const uint32_t s = mx4_scale(amax);
        const float inv = s == 255u ? 0.f : mx4_inverse(s);
        uint4 w{0u, 0u, 0u, 0u};
        if (s != 255u) w = uint4{mx4_codes8(v, inv), mx4_codes8(v + 8, inv), mx4_codes8(v + 16, inv), mx4_codes8(v + 24, inv)};
        codes[lane][i] = w;
        scales[lane][i] = (uint8_t)s;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 512; e += kNT) {
        const int rr = e >> 3, i = e & 7;
        if (r0 + rr < q.rows && b0 + i < kb) {
            ((uint4*)q.codes)[(r0 + rr) * kb + b0 + i] = codes[rr][i];
            q.scales[(r0 + rr) * kb + b0 + i] = scales[rr][i];
        }
    }
}

template <int DT>
__global__ __launch_bounds__(kNT) void mx4_dequantize_kernel(Mx4Mat q, typename MxFloat<DT>::type* __restrict__ out,
                                                             int64_t ld) {
    const int64_t gpr = q.kb() * 4;
    const int64_t ngroups = q.rows * gpr;
    for (int64_t g = (int64_t)blockIdx.x * kNT + threadIdx.x; g < ngroups; g += (int64_t)gridDim.x * kNT) {
        const int64_t row = g / gpr;
        const int64_t c0 = (g - row * gpr) * 8;
        const uint32_t w = ((const uint32_t*)q.codes)[g];
        const float s = mx4_scale_value(q.scales[g >> 2]);
        typename MxFloat<DT>::type* p = out + row * ld;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c0 + j < q.cols) p[c0 + j] = MxFloat<DT>::put(mx4_value(w >> (4 * j)) * s);
    }
}

int capped_blocks(int64_t threads) {
    const int64_t nb = (threads + kNT - 1) / kNT;
    return (int)(nb < 16384 ? nb : 16384);
}

}  // namespace

hipError_t launch_mx4_quantize(const void* x, int dtype, int64_t ld, bool transposed, const Mx4Mat& q,
                               hipStream_t stream) {
    return by_dtype(dtype, [&](auto dt) {
        typedef typename MxFloat<decltype(dt)::value>::type T;
        if (transposed) {
            const int64_t row_tiles = (q.rows + 63) / 64, k_tiles = (q.kb() + 7) / 8;
            hipLaunchKernelGGL(mx4_quantize_columns_kernel<decltype(dt)::value>, dim3((uint32_t)(row_tiles * k_tiles)),
                               dim3(kNT), 0, stream, (const T*)x, ld, q, (int)row_tiles);
        } else {
            hipLaunchKernelGGL(mx4_quantize_kernel<decltype(dt)::value>, dim3(capped_blocks(q.rows * q.kb() * 4)),
                               dim3(kNT), 0, stream, (const T*)x, ld, q);
        }
    });
}

hipError_t launch_mx4_dequantize(const Mx4Mat& q, void* out, int dtype, int64_t ld, hipStream_t stream) {
    return by_dtype(dtype, [&](auto dt) {
        typedef typename MxFloat<decltype(dt)::value>::type T;
        hipLaunchKernelGGL(mx4_dequantize_kernel<decltype(dt)::value>, dim3(capped_blocks(q.rows * q.kb() * 4)),
                           dim3(kNT), 0, stream, q, (T*)out, ld);
    });
}

size_t mx4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    const size_t kb = (size_t)(K + 31) / 32;
    return (size_t)M * kb * 16 + ((size_t)M * kb + 15) / 16 * 16 + mx4_matmul_workspace_bytes(M, N, K);
}

hipError_t launch_mx4_linear(const void* x, int dtype, int64_t ld, int64_t M, const Mx4Mat& b, const Mx4Out& out,
                             void* workspace, hipStream_t stream) {
    const int64_t blocks = M * b.kb();
    const Mx4Mat a{(uint8_t*)workspace, (uint8_t*)workspace + blocks * 16, M, b.cols};
    hipError_t e = launch_mx4_quantize(x, dtype, ld, false, a, stream);
    if (e != hipSuccess) return e;
    return launch_mx4_matmul(a, b, out, (uint8_t*)workspace + blocks * 16 + (blocks + 15) / 16 * 16, stream);
}

}  // namespace iqlh
