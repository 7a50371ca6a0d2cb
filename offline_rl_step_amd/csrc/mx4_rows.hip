// A float matrix times a small microscaled 4-bit one, quantised on the way in
// one launch: out[m][n] = act(sum_k q(x)[m][k] b[n][k] + bias[n]) for many rows m
// and a b that the L2 holds.  HBM-bound on x and out: x is read once, its codes
// live in LDS only, and b comes from L2 as fragments, without LDS.
#include "mx4_block.hpp"

namespace iqlh {

namespace {

constexpr int kNT = 256;
constexpr int kRows = 64;     // rows of x a workgroup takes
constexpr int kMaxBlocks = 32;  // K <= 1024
constexpr int kChunk = 32;    // rows of b a wave takes at a time
constexpr int kFrags = kChunk / 16;

// bytes between two rows' codes in LDS: 16 more than the codes, so that the 16
// lanes of a fragment column fall on different banks
__host__ __device__ constexpr int row_bytes(int kb4) { return kb4 * 16 + 16; }
// and each wave's stage for its outputs, element size es
__host__ __device__ constexpr int lds_bytes(int kb4, int es) {
    return kRows * (row_bytes(kb4) + kb4) + 4 * kRows * kChunk * es;
}

// Four waves; wave w takes the chunks w, w + 4, .. of 32 rows of b, 64 x 32
// outputs each.
template <int XDT, int ODT>
__global__ __launch_bounds__(kNT, 3) void mx4_rows_kernel(const typename MxFloat<XDT>::type* __restrict__ x, int64_t ld,
                                                       int64_t M, Mx4Mat b, Mx4Out o, int kb4, int stream_out) {
    typedef typename MxFloat<ODT>::type T;
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int r = lane & 15, blk = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * kRows;
    const int rb = row_bytes(kb4);
    uint8_t* scales = lds + kRows * rb;  // [kRows][kb4]
    const int gpr = kb4 * 4;             // groups of 8 a row, a multiple of 16
    constexpr int U = 4;  // groups in flight per thread
    for (int g0 = tid; g0 < kRows * gpr; g0 += kNT * U) {
        float v[U][8];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int e = g0 + i * kNT, row = e / gpr, g = e - row * gpr;
            const int64_t m = m0 + row < M ? m0 + row : M - 1;
            const int64_t left = e < kRows * gpr ? b.cols - g * 8 : 0;
            load8<XDT>(x + m * ld + g * 8, (int)(left < 0 ? 0 : left < 8 ? left : 8), v[i]);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int e = g0 + i * kNT, row = e / gpr, g = e - row * gpr;
            if (e >= kRows * gpr) break;  // the same for the whole workgroup: kRows gpr is a multiple of 256
            uint32_t amax = 0u;
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = umax2(amax, abs_bits(v[i][j]));
            const uint32_t s = mx4_scale(quad_umax(amax));
            *(uint32_t*)(lds + row * rb + g * 4) = s == 255u ? 0u : mx4_codes8(v[i], mx4_inverse(s));
            if ((g & 3) == 0) scales[row * kb4 + (g >> 2)] = (uint8_t)s;
        }
    }
    __syncthreads();
    uint8_t* stage = scales + kRows * kb4 + wave * (kRows * kChunk * (int)sizeof(T));
    constexpr int E = 16 / sizeof(T);                  // elements of a 16-byte unit
    constexpr int SN = kChunk;                         // columns staged at a time
    constexpr int UNITS = SN / E;
    const int steps = kb4 / 4;
    const float lowest = o.relu ? 0.f : -__builtin_huge_valf();
    // b's fragments one step ahead, over the chunks' ends too
    uint4 bn[kFrags];
    uint32_t bsn[kFrags];
    auto fetch = [&](int64_t n0, int s) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < kFrags; ++j) RowFrag(b, n0 + 16 * j + r).load(s * 4 + blk, bn[j], bsn[j]);
    };
    if (wave * kChunk < b.rows) fetch(wave * kChunk, 0);
    for (int64_t n0 = (int64_t)wave * kChunk; n0 < b.rows; n0 += 4 * kChunk) {
        float bias[kFrags][4];
#pragma unroll
        for (int j = 0; j < kFrags; ++j) {
            const int64_t n = n0 + 16 * j + 4 * blk;
            mx4_bias4(o, n, b.rows, bias[j]);
        }
        mx_f4 acc[4][kFrags];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < kFrags; ++j) acc[i][j] = mx_f4{0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < steps; ++s) {
            uint4 bv[kFrags], av[4];
            uint32_t bs[kFrags], as[4];
#pragma unroll
            for (int j = 0; j < kFrags; ++j) {
                bv[j] = bn[j];
                bs[j] = bsn[j];
            }
            if (s + 1 < steps) fetch(n0, s + 1);
            else if (n0 + 4 * kChunk < b.rows) fetch(n0 + 4 * kChunk, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                av[i] = *(const uint4*)(lds + (16 * i + r) * rb + (s * 4 + blk) * 16);
                as[i] = scales[(16 * i + r) * kb4 + s * 4 + blk];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < kFrags; ++j) acc[i][j] = mx4_mma(bv[j], av[i], acc[i][j], bs[j], as[i]);
        }
        // to memory through the wave's own LDS: rows of 128 neighbouring bytes.
        // Unit v of a row lies at v ^ (row & 7) (of 4 units, & 3).
        {
#pragma unroll
            for (int j = 0; j < kFrags; ++j) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 16 * i + r, c = 16 * j + 4 * blk;
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = __builtin_elementwise_maximum(acc[i][j][e] + bias[j][e], lowest);  // a NaN stays
                    mx4_put4<ODT>((T*)(stage + row * (SN * sizeof(T)) + 16 * ((c / E) ^ (row & (UNITS - 1)))) + c % E, y);
                }
            }
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the wave's own writes
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int c = lane; c < kRows * UNITS; c += kWave) {
                const int row = c / UNITS, v = c % UNITS;
                const int64_t m = m0 + row, n = n0 + v * E;
                const uint4 w = *(const uint4*)(stage + row * (SN * sizeof(T)) + 16 * (v ^ (row & (UNITS - 1))));
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
        }
    }
}

}  // namespace

bool mx4_rows_ok(int64_t M, int64_t N, int64_t K) {
    // rows enough for every compute unit, a b of at most 256 KB
    const int64_t kb = (K + 31) / 32;
    return M >= 8192 && kb <= kMaxBlocks && N * kb <= 16384;
}

hipError_t launch_mx4_rows(const void* x, int dtype, int64_t ld, int64_t M, const Mx4Mat& b, const Mx4Out& out,
                           hipStream_t stream) {
    const int kb4 = (int)((b.kb() + 3) / 4 * 4), es = out.dtype == IQLH_F32 ? 4 : 2, bytes = lds_bytes(kb4, es);
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
