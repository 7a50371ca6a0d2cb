// A float matrix times a small microscaled 4-bit one, quantised on the way in
// one launch: out[m][n] = act(sum_k q(x)[m][k] b[n][k] + bias[n]) for many rows m
// and a b that the L2 holds.  HBM-bound on x and out: x is read once, its codes
// live in LDS only, and b comes from L2 as fragments, without LDS.  65536 x 256 fp32 ->
// 512 bf16 28.3 us, 4.8 TB/s (by quantisation and product 65).  b regrouped by
// fragments in a launch of its own: 28.9.
#include "mx4_rows_block.hpp"

namespace iqlh {

namespace {

constexpr int kRows = 64, kNT = 256;

// Four waves; wave w takes the chunks w, w + 4, .. of 32 rows of b, 64 x 32
// outputs each.
template <int XDT, int ODT>
__global__ __launch_bounds__(kNT, 4) void mx4_rows_kernel(const typename MxFloat<XDT>::type* __restrict__ x, int64_t ld,
                                                           int64_t M, Mx4Mat b, Mx4Out o, int kb4, int stream_out) {
    typedef typename MxFloat<ODT>::type T;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, blk = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * kRows;
    const LdsRows<kRows> t(lds, kb4);
    mx4_rows_to_lds<kRows, kNT, XDT>(x, ld, M, m0, b.cols, t);
    __syncthreads();
    // a chunk's outputs leave through the wave's own LDS, as rows of
    // neighbouring 16-byte units; unit v of a row lies at v ^ row, modulo the units
    uint8_t* stage = lds + mx4_lds_bytes<kRows>(kb4) + wave * (kRows * kChunk * (int)sizeof(T));
    constexpr int E = 16 / sizeof(T), UNITS = kChunk / E;
    const float lowest = o.relu ? 0.f : -__builtin_huge_valf();
    float bias[kFrags][4];
    mx4_rows_chunks<kRows, kNT>(
        t, RowsOfB{b}, b.rows,
        [&](int64_t n0) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < kFrags; ++j) mx4_bias4(o, n0 + 16 * j + 4 * blk, b.rows, bias[j]);
        },
        [&](int64_t n0, mx_f4(&acc)[4][kFrags]) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < kFrags; ++j) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 16 * i + r, c = 16 * j + 4 * blk;
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[e] = __builtin_elementwise_maximum(acc[i][j][e] + bias[j][e], lowest);  // a NaN stays
                    mx4_put4<ODT>((T*)(stage + row * (kChunk * sizeof(T)) + 16 * ((c / E) ^ (row & (UNITS - 1)))) + c % E, y);
                }
            }
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the wave's own writes
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int c = lane; c < kRows * UNITS; c += kWave) {
                const int row = c / UNITS, v = c % UNITS;
                const int64_t m = m0 + row, n = n0 + v * E;
                const uint4 w = *(const uint4*)(stage + row * (kChunk * sizeof(T)) + 16 * (v ^ (row & (UNITS - 1))));
                if (m >= M || n >= b.rows) continue;
                T* p = (T*)o.p + m * o.ld + n;
                if (n + E <= b.rows) {
                    typedef T tu __attribute__((ext_vector_type(E), aligned(sizeof(T))));
                    if (stream_out) __builtin_nontemporal_store(__builtin_bit_cast(tu, w), (tu*)p);
                    else *(tu*)p = __builtin_bit_cast(tu, w);
                } else {
                    const T* y = (const T*)&w;
                    for (int k = 0; k < E; ++k)
                        if (n + k < b.rows) p[k] = y[k];
                }
            }
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_s_waitcnt(0xC07F);
            __builtin_amdgcn_wave_barrier();
        });
}

}  // namespace

bool mx4_rows_ok(int64_t M, int64_t N, int64_t K) {
    // Rows enough for every compute unit, and less than 2^32 threads of them; a b of at
    // most 256 KB, above K 896 of 96 KB.  fp32 -> bf16, quantisation and product | one
    // launch, us, at M 16384, 65536:
    //   N 512, K 256: 19 | 14, 40 | 28 (M 4096: 12.2 | 11.5, 2048: 8.5 | 11.1); K 768:
    //   23 | 26, 71 | 72; K 1000: 28 | 40, 106 | 130; N 128, K 1024: 23 | 20, 71 | 62;
    //   N 2048, K 256: 33 | 34, 113 | 107; N 4096, K 256 (512 KB): 57 | 63, 224 | 229
    const int64_t kb = (K + 31) / 32;
    return M >= 16384 && M <= 1 << 29 && kb <= kRowsMaxBlocks && N * kb <= (kb <= 28 ? 16384 : 6144);
}

hipError_t launch_mx4_rows(const void* x, int dtype, int64_t ld, int64_t M, const Mx4Mat& b, const Mx4Out& out,
                           hipStream_t stream) {
    const int kb4 = (int)((b.kb() + 3) / 4 * 4), es = out.dtype == IQLH_F32 ? 4 : 2, bytes = mx4_lds_bytes<kRows>(kb4) + 4 * kRows * kChunk * es;
    // outputs that the L2s (8 x 4 MB) cannot keep for a reader are stored past
    // them: 64 MB of outputs 32.5 us, through them 36.0; no difference at 4 MB
    const int stream_out = M * b.rows * es > 32 << 20;
    const dim3 grid((uint32_t)((M + kRows - 1) / kRows));
    hipError_t e = hipSuccess;
    auto go = [&](auto xdt, auto odt) {
        constexpr int X = decltype(xdt)::value, O = decltype(odt)::value;
        auto kernel = mx4_rows_kernel<X, O>;
        if (bytes > 64 << 10) e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return;
        hipLaunchKernelGGL(kernel, grid, dim3(kNT), bytes, stream, (const typename MxFloat<X>::type*)x, ld, M, b, out, kb4,
                           stream_out);
        e = hipGetLastError();
    };
    auto with_out = [&](auto xdt) {
        if (out.dtype == IQLH_F32) go(xdt, std::integral_constant<int, IQLH_F32>());
        else if (out.dtype == IQLH_BF16) go(xdt, std::integral_constant<int, IQLH_BF16>());
        else go(xdt, std::integral_constant<int, IQLH_F16>());
    };
    if (dtype == IQLH_F32) with_out(std::integral_constant<int, IQLH_F32>());
    else if (dtype == IQLH_BF16) with_out(std::integral_constant<int, IQLH_BF16>());
    else with_out(std::integral_constant<int, IQLH_F16>());
    return e;
}

}  // namespace iqlh
