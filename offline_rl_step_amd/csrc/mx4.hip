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
constexpr int kNarrowRows = 4;
constexpr int kQRows = 4;  // rows (times the workgroup's) a thread converts

// Blocks along x's rows.  HBM-bound.  A thread converts 8 elements (one dword
// of codes) of kQRows rows, all loaded before the first is used; four
// neighbouring lanes share a block.  A workgroup is 2^c_log groups of 8 wide
// and 256 / 2^c_log rows high.  (8192 x 8192 bf16 29 us, 5.9 TB/s of 170 MB, with an
// input that the Infinity Cache holds, 37 from HBM, and 48 right behind a pass whose 268
// MB of output are still on their way there; fp32, 304 MB, 49 with the same input
// again, 58 with others; 65536 x 777 with the same input fp32 35, bf16 27; a batch of
// 16384 x 128 fp32 3.2 to 3.6, where the launch counts.)
template <int DT>
__global__ __launch_bounds__(kNT) void mx4_quantize_kernel(const typename MxFloat<DT>::type* __restrict__ x, int64_t ld,
                                                           Mx4Mat q, int c_log, int col_tiles) {
    const int64_t gpr = q.kb() * 4;  // groups per row
    const int rows_high = kNT >> c_log;
    const int64_t g = ((int64_t)(blockIdx.x % col_tiles) << c_log) + (threadIdx.x & ((1 << c_log) - 1));
    const int64_t row0 = (int64_t)(blockIdx.x / col_tiles) * rows_high * kQRows + (threadIdx.x >> c_log);
    const int count = (int)(q.cols - g * 8 < 8 ? q.cols - g * 8 : 8);
    // a row's last group of a 16-bit type is one load where the matrix goes on
    // behind it (2^21 x 11 bf16: 23.6 us, element by element 32.0; fp32 25.8
    // against 20.9)
    const typename MxFloat<DT>::type* end = DT == IQLH_F32 ? nullptr : x + (q.rows - 1) * ld + q.cols;
    Eight<DT> raw[kQRows];
#pragma unroll
    for (int i = 0; i < kQRows; ++i) {
        const int64_t row = row0 + i * rows_high;
        raw[i].load(x + (row < q.rows ? row : q.rows - 1) * ld + g * 8, g < gpr ? count : 0, end);
    }
#pragma unroll
    for (int i = 0; i < kQRows; ++i) {
        const int64_t row = row0 + i * rows_high;
        float v[8];
        raw[i].get(v);
        uint32_t amax = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = umax2(amax, abs_bits(v[j]));
        const uint32_t s = mx4_scale(quad_umax(amax));
        const uint32_t w = s == 255u ? 0u : mx4_codes8(v, mx4_inverse(s));
        if (row < q.rows && g < gpr) {
            ((uint32_t*)q.codes)[row * gpr + g] = w;
            if ((g & 3) == 0) q.scales[(row * gpr + g) >> 2] = (uint8_t)s;
        }
    }
}

// The same for a matrix of one block a row and at most 8 G columns: a lane
// takes a row, so that its codes leave as 16 bytes.  (2^22 x 1 bf16 47 -> 15 us,
// 2^22 x 3 46 -> 18, 2^21 x 11 25 -> 15.5.)
template <int DT, int G>
__global__ __launch_bounds__(kNT) void mx4_quantize_narrow_kernel(const typename MxFloat<DT>::type* __restrict__ x,
                                                                  int64_t ld, Mx4Mat q) {
    const int64_t row0 = (int64_t)blockIdx.x * (kNT * kNarrowRows) + threadIdx.x;
    const int cols = (int)q.cols;
    const typename MxFloat<DT>::type* end = DT == IQLH_F32 || cols < 3 ? nullptr : x + (q.rows - 1) * ld + cols;
    Eight<DT> raw[kNarrowRows][G];
#pragma unroll
    for (int i = 0; i < kNarrowRows; ++i) {
        const int64_t row = row0 + i * kNT < q.rows ? row0 + i * kNT : q.rows - 1;
#pragma unroll
        for (int g = 0; g < G; ++g) raw[i][g].load(x + row * ld + 8 * g, cols - 8 * g < 8 ? cols - 8 * g : 8, end);
    }
#pragma unroll
    for (int i = 0; i < kNarrowRows; ++i) {
        float v[8 * G];
        uint32_t amax = 0u;
#pragma unroll
        for (int g = 0; g < G; ++g) raw[i][g].get(v + 8 * g);
#pragma unroll
        for (int j = 0; j < 8 * G; ++j) amax = umax2(amax, abs_bits(v[j]));
        const uint32_t s = mx4_scale(amax);
        const int64_t row = row0 + i * kNT;
        if (row < q.rows) {
            uint4 w{0u, 0u, 0u, 0u};
            if (s != 255u) {
                const float inv = mx4_inverse(s);
                w.x = mx4_codes8(v, inv);
                if (G > 1) w.y = mx4_codes8(v + 8, inv);
            }
            ((uint4*)q.codes)[row] = w;
            q.scales[row] = (uint8_t)s;
        }
    }
}

// Blocks along x's columns: x is [q.cols][ld].  HBM-bound.  A lane takes one
// column of x, 32 rows a block, neighbouring lanes neighbouring addresses; a
// workgroup 2^c_log columns (64, fewer of a narrow x) and 4 HALVES blocks per
// wave's worth of them.  The codes pass through LDS so that a row of q is written 64 bytes
// or more at a time.  (8192^2 bf16 from the Infinity Cache 27.0 us, 6.3 TB/s; two 16-bit columns per
// lane by dword loads 27.5, and 12.3 against 5.2 us at 5001 x 777, where they
// leave half of the compute units without a workgroup.  Runs of tiles per XCD:
// 65536 x 777 fp32 52 -> 34 us, bf16 38 -> 21.5; rows on cache lines lose by them,
// 4096 x 16384 fp32 49 -> 53.)
template <int DT, int HALVES>
__global__ __launch_bounds__(kNT) void mx4_quantize_columns_kernel(const typename MxFloat<DT>::type* __restrict__ x,
                                                                   int64_t ld, Mx4Mat q, int c_log, int row_tiles,
                                                                   int shared_lines) {
    __shared__ uint4 codes[576];  // [columns][blocks + 1]: the lanes of a store to one block fall on different banks
    __shared__ uint8_t scales[576];
    const int64_t kb = q.kb();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int columns = 1 << c_log, b_log = 7 + HALVES - c_log, blocks = 1 << b_log;
    const int c = lane & (columns - 1);
    // rows of x that do not start on cache lines: neighbouring tiles share the lines at
    // their border, so each XCD (every eighth workgroup) gets a run of tiles
    uint32_t id = blockIdx.x;
    if (shared_lines) {
        const uint32_t per = gridDim.x / 8, rest = gridDim.x % 8, xcd = id & 7;
        id = xcd * per + (xcd < rest ? xcd : rest) + (id >> 3);
    }
    const int64_t r0 = (int64_t)(id % row_tiles) * columns, b0 = (int64_t)(id / row_tiles) << b_log;
    const int64_t r = r0 + c < q.rows ? r0 + c : q.rows - 1;  // lanes past the end: not written below
#pragma unroll
    for (int half = 0; half < HALVES; ++half) {
        const int i = ((wave + 4 * half) << (6 - c_log)) + (lane >> c_log);
        const int64_t k0 = (b0 + i) * 32;
        if (b0 + i < kb) {
            // loads at clamped rows, those behind the last one masked: no branch between them
            const int left = (int)(q.cols - k0 < 32 ? q.cols - k0 : 32);
            const typename MxFloat<DT>::type* p = x + k0 * ld + r;
            float v[32];
            uint32_t amax = 0u;
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = keep_if(j < left, MxFloat<DT>::get(p[(j < left ? j : 0) * ld]));
#pragma unroll
            for (int j = 0; j < 32; ++j) amax = umax2(amax, abs_bits(v[j]));
            const uint32_t s = mx4_scale(amax);
            uint4 w{0u, 0u, 0u, 0u};
            if (s != 255u) {
                const float inv = mx4_inverse(s);
                w = uint4{mx4_codes8(v, inv), mx4_codes8(v + 8, inv), mx4_codes8(v + 16, inv), mx4_codes8(v + 24, inv)};
            }
            codes[c * (blocks + 1) + i] = w;
            scales[c * (blocks + 1) + i] = (uint8_t)s;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < HALVES * kNT; e += kNT) {
        const int rr = e >> b_log, i = e & (blocks - 1);
        if (r0 + rr < q.rows && b0 + i < kb) {
            ((uint4*)q.codes)[(r0 + rr) * kb + b0 + i] = codes[rr * (blocks + 1) + i];
            q.scales[(r0 + rr) * kb + b0 + i] = scales[rr * (blocks + 1) + i];
        }
    }
}

// HBM-bound on its stores: a thread writes 16 bytes of kQRows rows, so that
// neighbouring lanes write neighbouring 16 bytes.  (8192 x 8192 to fp32, 304 MB, 45 us
// behind the quantisation, whose codes the caches still hold, 55 otherwise; stores past
// the caches: no gain.)
template <int DT>
__global__ __launch_bounds__(kNT) void mx4_dequantize_kernel(Mx4Mat q, typename MxFloat<DT>::type* __restrict__ out,
                                                             int64_t ld, int c_log, int col_tiles) {
    typedef typename MxFloat<DT>::type T;
    constexpr int E = 16 / sizeof(T);  // elements a thread converts: a dword of codes or half of one
    const int rows_high = kNT >> c_log;
    const int64_t c0 = (((int64_t)(blockIdx.x % col_tiles) << c_log) + (threadIdx.x & ((1 << c_log) - 1))) * E;
    const int64_t row0 = (int64_t)(blockIdx.x / col_tiles) * rows_high * kQRows + (threadIdx.x >> c_log);
    if (c0 >= q.cols) return;
    const int64_t kb = q.kb();
    uint32_t w[kQRows], s[kQRows];
#pragma unroll
    for (int i = 0; i < kQRows; ++i) {
        const int64_t row = row0 + i * rows_high < q.rows ? row0 + i * rows_high : q.rows - 1;
        const uint8_t* p = q.codes + row * kb * 16 + c0 / 2;
        w[i] = E == 8 ? *(const uint32_t*)p : *(const uint16_t*)p;
        s[i] = q.scales[row * kb + c0 / 32];
    }
#pragma unroll
    for (int i = 0; i < kQRows; ++i) {
        const int64_t row = row0 + i * rows_high;
        if (row >= q.rows) break;
        const float sc = mx4_scale_value(s[i]);
        T y[E];
        static_for<E / 2>([&](auto j) __attribute__((always_inline)) {
            constexpr int J = decltype(j)::value;
            const auto v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.f, J);
            y[2 * J] = MxFloat<DT>::put(v[0] * sc);
            y[2 * J + 1] = MxFloat<DT>::put(v[1] * sc);
        });
        T* p = out + row * ld + c0;
        if (c0 + E <= q.cols) {
            typedef T tu __attribute__((ext_vector_type(E), aligned(sizeof(T))));
            tu o;
#pragma unroll
            for (int j = 0; j < E; ++j) o[j] = y[j];
            *(tu*)p = o;
        } else {
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (c0 + j < q.cols) p[j] = y[j];
        }
    }
}

// Workgroups of 2^c_log columns (at most 256) for `across` column groups a
// row, and how many of them the matrix takes.
struct Shape {
    int c_log, col_tiles;
    int64_t blocks;
};
constexpr int64_t kMostBlocks = ((int64_t)1 << 32) / kNT - 1;  // launches hold less than 2^32 threads
Shape shape_for(int64_t rows, int64_t across) {
    Shape s;
    s.c_log = 2;
    while (s.c_log < 8 && ((int64_t)1 << s.c_log) < across) ++s.c_log;
    s.col_tiles = (int)((across + (1 << s.c_log) - 1) >> s.c_log);
    const int64_t high = (int64_t)(kNT >> s.c_log) * kQRows;
    s.blocks = (rows + high - 1) / high * s.col_tiles;
    return s;
}

// Columns a workgroup (2^c_log) and workgroups of a quantisation along x's columns:
// no more columns than x has, as long as there is a workgroup for every
// compute unit (2^22 rows of 1: 10.5 us, of 64 82; 2^14: 9.4 against 4.0)
struct ColumnShape {
    int c_log, halves;
    int64_t row_tiles, blocks;
};
ColumnShape column_shape_for(int64_t rows, int64_t kb, int es, bool on_lines) {
    ColumnShape s;
    s.c_log = 0;
    while (s.c_log < 6 && ((int64_t)1 << s.c_log < rows || kb >> (9 - s.c_log) < 256)) ++s.c_log;
    s.row_tiles = (rows + (1 << s.c_log) - 1) >> s.c_log;
    // one block a lane, two of wide binary32 rows on cache lines (5001 x 777 fp16: 4.5
    // against 5.5 us, 8192 x 8192 bf16 26.8 against 27.8; fp32 57.0 against 52.5, and 262144 x
    // 200 fp32, whose rows end inside a line, 33.8 against 37.0)
    const int64_t two = s.row_tiles * ((kb + (1 << (9 - s.c_log)) - 1) >> (9 - s.c_log));
    s.halves = on_lines && es == 4 && two >= 2048 ? 2 : 1;
    const int b_log = 7 + s.halves - s.c_log;
    s.blocks = s.row_tiles * ((kb + (1 << b_log) - 1) >> b_log);
    return s;
}

int64_t dequantize_across(int64_t cols, int es) { return (cols * es + 15) / 16; }

}  // namespace

bool mx4_quantizable(int64_t rows, int64_t cols, bool transposed) {
    const int64_t kb = (cols + 31) / 32;
    return (transposed ? column_shape_for(rows, kb, 2, false).blocks : shape_for(rows, kb * 4).blocks) <= kMostBlocks;
}
bool mx4_dequantizable(int64_t rows, int64_t cols, int es) {
    return shape_for(rows, dequantize_across(cols, es)).blocks <= kMostBlocks;
}

hipError_t launch_mx4_quantize(const void* x, int dtype, int64_t ld, bool transposed, const Mx4Mat& q,
                               hipStream_t stream) {
    // a column without gaps is a row (2^26 x 1 bf16: 63 us, column by column 116)
    if (transposed && q.rows == 1 && ld == 1) return launch_mx4_quantize(x, dtype, q.cols, false, q, stream);
    return by_dtype(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        typedef typename MxFloat<DT>::type T;
        if (transposed) {
            const int shared_lines = (((uintptr_t)x | (uint64_t)ld * sizeof(T)) & 127u) != 0;
            const ColumnShape s = column_shape_for(q.rows, q.kb(), sizeof(T), !shared_lines);
            const dim3 grid((uint32_t)s.blocks);
            if (s.halves == 1)
                hipLaunchKernelGGL((mx4_quantize_columns_kernel<DT, 1>), grid, dim3(kNT), 0, stream, (const T*)x, ld, q, s.c_log,
                                   (int)s.row_tiles, shared_lines);
            else
                hipLaunchKernelGGL((mx4_quantize_columns_kernel<DT, 2>), grid, dim3(kNT), 0, stream, (const T*)x, ld, q, s.c_log,
                                   (int)s.row_tiles, shared_lines);
        } else if (q.cols <= 16) {
            const dim3 grid((uint32_t)((q.rows + kNT * kNarrowRows - 1) / (kNT * kNarrowRows)));
            if (q.cols <= 8) hipLaunchKernelGGL((mx4_quantize_narrow_kernel<DT, 1>), grid, dim3(kNT), 0, stream, (const T*)x, ld, q);
            else hipLaunchKernelGGL((mx4_quantize_narrow_kernel<DT, 2>), grid, dim3(kNT), 0, stream, (const T*)x, ld, q);
        } else {
            const Shape s = shape_for(q.rows, q.kb() * 4);
            hipLaunchKernelGGL(mx4_quantize_kernel<DT>, dim3((uint32_t)s.blocks), dim3(kNT), 0, stream, (const T*)x, ld, q,
                               s.c_log, s.col_tiles);
        }
    });
}

hipError_t launch_mx4_dequantize(const Mx4Mat& q, void* out, int dtype, int64_t ld, hipStream_t stream) {
    return by_dtype(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        typedef typename MxFloat<DT>::type T;
        const Shape s = shape_for(q.rows, dequantize_across(q.cols, sizeof(T)));
        hipLaunchKernelGGL(mx4_dequantize_kernel<DT>, dim3((uint32_t)s.blocks), dim3(kNT), 0, stream, q, (T*)out, ld, s.c_log,
                           s.col_tiles);
    });
}

size_t mx4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    const size_t kb = (size_t)(K + 31) / 32;
    return (size_t)M * kb * 16 + ((size_t)M * kb + 15) / 16 * 16 + mx4_matmul_workspace_bytes(M, N, K);
}

bool mx4_linear_launchable(int64_t M, int64_t N, int64_t K) {
    return mx4_few_ok(M, N, K) || mx4_rows_ok(M, N, K) || mx4_quantizable(M, K, false);
}

hipError_t launch_mx4_linear(const void* x, int dtype, int64_t ld, int64_t M, const Mx4Mat& b, const Mx4Out& out,
                             void* workspace, hipStream_t stream) {
    if (mx4_few_ok(M, b.rows, b.cols)) return launch_mx4_few(x, dtype, ld, M, b, out, stream);
    if (mx4_rows_ok(M, b.rows, b.cols)) return launch_mx4_rows(x, dtype, ld, M, b, out, stream);
    const int64_t blocks = M * b.kb();
    const Mx4Mat a{(uint8_t*)workspace, (uint8_t*)workspace + blocks * 16, M, b.cols};
    hipError_t e = launch_mx4_quantize(x, dtype, ld, false, a, stream);
    if (e != hipSuccess) return e;
    return launch_mx4_matmul(a, b, out, (uint8_t*)workspace + blocks * 16 + (blocks + 15) / 16 * 16, stream);
}

}  // namespace iqlh
