// Product of two microscaled 4-bit matrices,
//   out[m][n] = act(sum_k a[m][k] b[n][k] + bias[n]),
// on the scaled matrix instructions (16 x 16 outputs and 128 k, or 32 x 32 and 64 k, one
// scale byte per 32 k and row).  b is the instruction's row operand in every kernel, so
// that a lane holds four neighbouring n of one output row.
//
// Kernels by shape (pick; a rule's comment says what both sides measured):
//   few rows (M <= 16, and floats of more rows): HBM-bound on b; a workgroup takes 16
//     rows of b, the left operand lies in LDS;
//   waves that split k, where outputs are fewer than a round of workgroups;
//   straight from memory, for many outputs of short sums;
//   tiles of 128 x 128 and 256 x 256 through LDS, the rest.
#include "lds_copy.hpp"
#include "mx4_block.hpp"

namespace iqlh {

namespace {

constexpr int kNT = 256;
constexpr int kComputeUnits = 256;

template <typename F>
hipError_t by_dtype(int dtype, F f) {
    if (dtype == IQLH_F32) f(std::integral_constant<int, IQLH_F32>());
    else if (dtype == IQLH_BF16) f(std::integral_constant<int, IQLH_BF16>());
    else f(std::integral_constant<int, IQLH_F16>());
    return hipGetLastError();
}

// ------------------------------------------------------------- few rows
// HBM-bound on b, at small sizes on the latency of one pass over it.
// Workgroup: 16 rows of b and up to 16 MF rows of the left operand.  Wave w of 8 takes the k steps w, w + 8, ..; U
// steps' loads of b are in flight together, the first of them before anything
// else.  The left operand lies in LDS, as rows of whole steps: copied there, or
// (XDT >= 0, a float matrix) quantised into it by every workgroup, an eighth of a
// step per thread at 4096 elements, while b's loads are under way.  A wave's
// 16-byte loads of 16 rows are 64 lookups in the L1, so only b's are made; b's
// scales come as 4 bytes per row to 16 lanes.  The waves' sums meet in LDS, added in
// wave order.  (One row of 4096 x 4096 in bf16: 4.1 to 4.4 us, 2.2 TB/s; of 8192 x 8192
// 9.4, 3.8 TB/s, in 4 bits already 8.0; 16 rows of that in 4 bits 11.3.)
constexpr int kFewWaves = 8;
constexpr int kFewElements = 16384;  // of a workgroup's part of a float left operand, padded
template <int XDT, int ODT, int MF>
__global__ __launch_bounds__(64 * kFewWaves) void mx4_few_rows_kernel(Mx4Mat a, const void* x, int64_t ld, Mx4Mat b,
                                                                      Mx4Out o, int n_tiles) {
    constexpr int U = 4, NT = 64 * kFewWaves;
    extern __shared__ __align__(16) uint8_t lds[];
    mx_f4(*part)[MF][64] = (mx_f4(*)[MF][64])lds;    // [kFewWaves]
    uint8_t* codes = lds + kFewWaves * MF * 64 * 16;  // [rows][kb4 * 16 + 16]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, blk = lane >> 4;
    const int64_t n0 = (int64_t)(blockIdx.x % n_tiles) * 16, m0 = (int64_t)(blockIdx.x / n_tiles) * (16 * MF);
    const int rows = (int)(a.rows - m0 < 16 * MF ? a.rows - m0 : 16 * MF);
    const RowFrag fb(b, n0 + r);
    const int kb = (int)b.kb(), steps = (kb + 3) / 4;
    uint4 bv[U];
    uint32_t bw[U];
    auto load_b = [&](int s0) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u * kFewWaves;
            const int at = s * 4 + blk < kb ? s * 4 + blk : 0;  // blocks past the end: a's are zeros
            bv[u] = fb.codes[at];
        }
        if (blk == 0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int s = (s0 + u * kFewWaves) * 4;
                typedef uint32_t u1 __attribute__((aligned(1)));
                if (s + 4 <= kb) {
                    bw[u] = *(const u1*)(fb.scales + s);
                } else {
                    bw[u] = 0x7F7F7F7Fu;
                    for (int e = 0; s + e < kb; ++e) bw[u] = (bw[u] & ~(255u << (8 * e))) | (uint32_t)fb.scales[s + e] << (8 * e);
                }
            }
        }
    };
    load_b(wave);
    const int kb4 = steps * 4, rb = kb4 * 16 + 16;
    uint8_t* scales = codes + rows * rb;             // [rows][kb4]
    if constexpr (XDT >= 0) {
        const int gpr = kb4 * 4;                     // groups of 8 a row
        for (int e = threadIdx.x; e < rows * gpr; e += NT) {  // four lanes share a block: gpr is a multiple of 16
            const int row = e / gpr, g = e - row * gpr;
            const int64_t left = a.cols - g * 8;
            float v[8];
            load8<XDT>((const typename MxFloat<XDT>::type*)x + (m0 + row) * ld + g * 8, (int)(left < 0 ? 0 : left < 8 ? left : 8), v);
            uint32_t amax = 0u;
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = umax2(amax, abs_bits(v[j]));
            const uint32_t s = mx4_scale(quad_umax(amax));
            *(uint32_t*)(codes + row * rb + g * 4) = s == 255u ? 0u : mx4_codes8(v, mx4_inverse(s));
            if ((g & 3) == 0) scales[row * kb4 + (g >> 2)] = (uint8_t)s;
        }
    } else {
        for (int e0 = threadIdx.x; e0 < rows * kb4; e0 += NT * U) {
            uint4 w[U];
            uint32_t s[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int e = e0 + i * NT, row = e / kb4, k = e - row * kb4;
                const bool in = e < rows * kb4 && k < kb;
                const int64_t at = in ? (m0 + row) * kb + k : 0;
                w[i] = ((const uint4*)a.codes)[at];
                s[i] = in ? a.scales[at] : 127u;
                const uint32_t keep = in ? 0xFFFFFFFFu : 0u;
                w[i] = uint4{w[i].x & keep, w[i].y & keep, w[i].z & keep, w[i].w & keep};
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int e = e0 + i * NT, row = e / kb4, k = e - row * kb4;
                if (e >= rows * kb4) break;
                *(uint4*)(codes + row * rb + k * 16) = w[i];
                scales[e] = (uint8_t)s[i];
            }
        }
    }
    __syncthreads();
    mx_f4 acc[MF];
#pragma unroll
    for (int i = 0; i < MF; ++i) acc[i] = mx_f4{0.f, 0.f, 0.f, 0.f};
    for (int s0 = wave; s0 < steps; s0 += kFewWaves * U) {
        if (s0 != wave) load_b(s0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u * kFewWaves;
            const uint32_t bs = (uint32_t)__shfl((int)bw[u], r, kWave) >> (8 * blk) & 255u;
#pragma unroll
            for (int i = 0; i < MF; ++i) {
                const bool in = s < steps && 16 * i + r < rows;
                const int at = in ? s * 4 + blk : 0, row = in ? 16 * i + r : 0;
                const uint4 w = *(const uint4*)(codes + row * rb + at * 16);
                const uint32_t keep = in ? 0xFFFFFFFFu : 0u;
                const uint32_t as = in ? scales[row * kb4 + at] : 127u;
                acc[i] = mx4_mma(bv[u], uint4{w.x & keep, w.y & keep, w.z & keep, w.w & keep}, acc[i], bs, as);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < MF; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    if (wave < MF && 16 * wave + r < rows) {
        mx_f4 v = part[0][wave][lane];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) v += part[w][wave][lane];
        mx4_store4<ODT>(o, m0 + 16 * wave + r, n0 + 4 * blk, b.rows, v);
    }
}

// LDS of a left operand of `rows` rows and K columns, and of the sums
int64_t few_bytes(int64_t rows, int64_t K, int MF = 1) {
    return kFewWaves * 1024 * MF + rows * ((K + 127) / 128 * 68 + 16);
}

template <int XDT, int MF>
hipError_t launch_few_rows(const Mx4Mat& a, const void* x, int64_t ld, const Mx4Mat& b, const Mx4Out& out,
                           hipStream_t stream) {
    const int bytes = (int)few_bytes(a.rows < 16 * MF ? a.rows : 16 * MF, b.cols, MF);
    const int64_t nt = (b.rows + 15) / 16, mt = (a.rows + 16 * MF - 1) / (16 * MF);
    return by_dtype(out.dtype, [&](auto dt) {
        auto kernel = mx4_few_rows_kernel<XDT, decltype(dt)::value, MF>;
        if (bytes > 64 << 10)
            (void)hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        hipLaunchKernelGGL(kernel, dim3((uint32_t)(nt * mt)), dim3(64 * kFewWaves), bytes, stream, a, x, ld, b, out, (int)nt);
    });
}
template <int XDT>
hipError_t launch_few_rows_of(const Mx4Mat& a, const void* x, int64_t ld, const Mx4Mat& b, const Mx4Out& out,
                              hipStream_t stream) {
    return a.rows <= 16   ? launch_few_rows<XDT, 1>(a, x, ld, b, out, stream)
           : a.rows <= 32 ? launch_few_rows<XDT, 2>(a, x, ld, b, out, stream)
                          : launch_few_rows<XDT, 4>(a, x, ld, b, out, stream);
}

// --------------------------------------------- short sums, straight from memory
// A wave computes 64 x 64 outputs, the workgroup's four 128 x 128, fragments
// from L2: for sums of a step or two, where a ring would not fill.  Bound by the
// L1's lookups of its 16-row fragments and the stores.  (8192 x 8192, K 128: 47 us, its
// outputs alone at a copy's rate 26; 256 tiles there 52.)
template <int DT>
__global__ __launch_bounds__(kNT) void mx4_direct_kernel(Mx4Mat a, Mx4Mat b, Mx4Out o, int n_tiles) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, blk = lane >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x / n_tiles) * 128 + (wave >> 1) * 64;
    const int64_t n0 = (int64_t)(blockIdx.x % n_tiles) * 128 + (wave & 1) * 64;
    const RowFrag fa[4] = {RowFrag(a, m0 + r), RowFrag(a, m0 + 16 + r), RowFrag(a, m0 + 32 + r), RowFrag(a, m0 + 48 + r)};
    const RowFrag fb[4] = {RowFrag(b, n0 + r), RowFrag(b, n0 + 16 + r), RowFrag(b, n0 + 32 + r), RowFrag(b, n0 + 48 + r)};
    mx_f4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mx_f4{0.f, 0.f, 0.f, 0.f};
    const int64_t steps = (a.kb() + 3) / 4;
    for (int64_t s = 0; s < steps; ++s) {
        uint4 av[4], bv[4];
        uint32_t as[4], bs[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            fa[i].load(s * 4 + blk, av[i], as[i]);
            fb[i].load(s * 4 + blk, bv[i], bs[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = mx4_mma(bv[j], av[i], acc[i][j], bs[j], as[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + 16 * i + r, n = n0 + 16 * j + 4 * blk;
            if (m < a.rows) mx4_store4<DT>(o, m, n, b.rows, acc[i][j]);
        }
}

// ------------------------------------------------------- waves that split k
// The eight waves' sums of 16 MF x 16 NF outputs, through 4 MF NF KB of LDS: waves
// 4..7 add to waves 0..3, then those four are added in wave order.
template <int DT, int MF, int NF>
IQLH_DEV void add_split_waves(const Mx4Mat& a, const Mx4Mat& b, const Mx4Out& o, int64_t m0, int64_t n0, uint8_t* lds,
                              const mx_f4 (&acc)[MF][NF]) {
    mx_f4(*part)[MF * NF][64] = (mx_f4(*)[MF * NF][64])lds;  // [4]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, blk = lane >> 4;
    if (wave >= 4) {
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int j = 0; j < NF; ++j) part[wave - 4][NF * i + j][lane] = acc[i][j];
    }
    __syncthreads();
    if (wave < 4) {
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int j = 0; j < NF; ++j) part[wave][NF * i + j][lane] += acc[i][j];
    }
    __syncthreads();
    for (int e = wave; e < MF * NF; e += 8) {
        mx_f4 v = part[0][e][lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) v += part[w][e][lane];
        const int64_t m = m0 + 16 * (e / NF) + r, n = n0 + 16 * (e % NF) + 4 * blk;
        if (m < a.rows) mx4_store4<DT>(o, m, n, b.rows, v);
    }
}

// A workgroup takes 16 MF x 16 NF outputs, its eight waves every eighth k step
// each.  For few outputs, where what counts is how many loads are in flight over
// the chip, and the L1's lookups: straight from memory a fragment of 16 rows is
// 64 of them per KB, so each wave copies the rows of its step, 64 bytes each, to its
// own D buffers in LDS, 4 neighbouring lanes a row, 16 lookups per KB.  The scales of all
// rows lie in LDS before, for up to kSplitSteps steps at a time.  Within a
// wave's buffer the 16 bytes of block b of row r lie at 64 r + 16 (b ^ (r >> 2 &
// 3)), so that 16 rows' reads fall on all banks; the scales of step d at dword d ^ (r
// & 15) of the row's.  (512^3 3.4 us, straight from memory 6.2; 64 x 4096 x 4096 5.5
// against 12.9; 1024 x 1024 x 4096 10.0 against 21.0.)
template <int MF, int NF, int D>
constexpr int kSplitRing = 8 * D * (MF + NF) * 1024;
constexpr int split_scale_row(int64_t steps) { return (int)((steps + 15) / 16 * 64); }
// steps whose scales fit beside the buffers, a multiple of 16
template <int MF, int NF, int D>
constexpr int kSplitSteps = (160 * 1024 - kSplitRing<MF, NF, D>) / (16 * (MF + NF)) / 64 * 16;
template <int DT, int MF, int NF, int D>
__global__ __launch_bounds__(512, 2) void mx4_split_kernel(Mx4Mat a, Mx4Mat b, Mx4Out o, int n_tiles) {
    constexpr int P = MF + NF;           // copies a step
    extern __shared__ __align__(16) uint8_t lds[];
    uint8_t* scales = lds + kSplitRing<MF, NF, D>;  // [16 P rows][split_scale_row], b's rows, then a's
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, blk = lane >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x / n_tiles) * (16 * MF), n0 = (int64_t)(blockIdx.x % n_tiles) * (16 * NF);
    const int kb = (int)a.kb(), all = (kb + 3) / 4;
    const uint32_t ring = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds + wave * (D * P * 1024);
    const int cr = lane >> 2, u = (lane & 3) ^ (cr >> 2 & 3);  // row and block a lane copies
    const uint8_t* src[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const Mx4Mat& q = i < NF ? b : a;
        const int64_t row = (i < NF ? n0 + 16 * i : m0 + 16 * (i - NF)) + cr;
        src[i] = q.codes + (row < q.rows ? row : q.rows - 1) * kb * 16 + 16 * u;
    }
    auto issue = [&](int s, int buf) __attribute__((always_inline)) {
        const bool in = 4 * s + u < kb;
#pragma unroll
        for (int i = 0; i < P; ++i)
            copy16(in ? src[i] + (int64_t)s * 64 : (const uint8_t*)kZeroChunk, ring + (buf * P + i) * 1024);
    };
    mx_f4 acc[MF][NF];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[i][j] = mx_f4{0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < all; s0 += kSplitSteps<MF, NF, D>) {
        const int n = all - s0 < kSplitSteps<MF, NF, D> ? all - s0 : kSplitSteps<MF, NF, D>;
        const int steps = s0 + n, rs = split_scale_row(n);
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (s0 + wave + 8 * d < steps) issue(s0 + wave + 8 * d, d);
#pragma unroll 8
        for (int e = threadIdx.x; e < 16 * P * n; e += 512) {
            const int row = e / n, d = e - row * n, block = (s0 + d) * 4;
            const bool is_b = row < 16 * NF;
            const Mx4Mat& q = is_b ? b : a;
            const int64_t at = is_b ? n0 + row : m0 + row - 16 * NF;
            const uint8_t* p = q.scales + (at < q.rows ? at : q.rows - 1) * kb + block;
            uint32_t w = 0x7F7F7F7Fu;
            if (block + 4 <= kb) {
                typedef uint32_t u1 __attribute__((aligned(1)));
                w = *(const u1*)p;
            } else {
                for (int j = 0; block + j < kb; ++j) w = (w & ~(255u << (8 * j))) | (uint32_t)p[j] << (8 * j);
            }
            *(uint32_t*)(scales + row * rs + 4 * (d ^ (row & 15))) = w;
        }
        bar();
        int buf = 0;
        for (int s = s0 + wave; s < steps; s += 8) {
            const int behind = (steps - 1 - s) >> 3;  // of the wave's steps
            if (behind >= D - 1) wait_vm<(D - 1) * P>();
            else if (D > 3 && behind == 2) wait_vm<2 * P>();
            else if (D > 2 && behind == 1) wait_vm<P>();
            else wait_vm<0>();
            asm volatile("" ::: "memory");
            const uint8_t* at = lds + (wave * D + buf) * (P * 1024) + r * 64 + 16 * (blk ^ (r >> 2 & 3));
            uint4 f[P];
            uint32_t fs[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                f[i] = *(const uint4*)(at + i * 1024);
                fs[i] = *(const uint32_t*)(scales + (16 * i + r) * rs + 4 * ((s - s0) ^ r)) >> (8 * blk);
            }
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the buffer is read
            asm volatile("" ::: "memory");
            if (s + 8 * D < steps) issue(s + 8 * D, buf);
            buf = buf + 1 < D ? buf + 1 : 0;
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int j = 0; j < NF; ++j) acc[i][j] = mx4_mma(f[j], f[NF + i], acc[i][j], fs[j], fs[NF + i]);
        }
        bar();  // no wave reads its buffers or the scales any more
    }
    add_split_waves<DT, MF, NF>(a, b, o, m0, n0, lds, acc);
}

// ------------------------------------------------------- tiles through LDS
// Scales regrouped for the tile kernel: for 32 rows and the 8 blocks of a
// step one dword per lane, byte i the scale of row lane & 31, block
// 2 i + (lane >> 5), so that a lane's dword serves the step's four matrix
// instructions of a fragment (the instruction selects the byte).
// [32-row group][step][lane]; rows and blocks past the end get 127.
// A workgroup takes 32 rows and 8 steps, 64 bytes of each row.  (Both operands of
// 8192^3: 4.3 us; single bytes to LDS in the tile kernel would be 64 lookups a
// fragment.)
__global__ __launch_bounds__(kNT) void mx4_scale_groups_kernel(Mx4Mat a, Mx4Mat b, uint32_t* __restrict__ ga,
                                                               uint32_t* __restrict__ gb, int a_groups) {
    const bool is_a = (int)blockIdx.x < a_groups;
    const Mx4Mat& q = is_a ? a : b;
    const int64_t group = is_a ? blockIdx.x : blockIdx.x - a_groups;
    const int64_t kb = q.kb(), steps = (kb + 7) / 8;
    const int r = threadIdx.x & 31;
    const int64_t step = (int64_t)blockIdx.y * 8 + (threadIdx.x >> 5), row = group * 32 + r;
    if (step >= steps) return;
    const uint8_t* p = q.scales + row * kb + step * 8;
    uint32_t even = 0x7F7F7F7Fu, odd = 0x7F7F7F7Fu;
    if (row < q.rows) {
        if (step * 8 + 8 <= kb) {
            typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(1)));
            const u2 w = *(const u2*)p;
            even = __builtin_amdgcn_perm(w.y, w.x, 0x06040200u);
            odd = __builtin_amdgcn_perm(w.y, w.x, 0x07050301u);
        } else {
            even = odd = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                even |= (step * 8 + 2 * i < kb ? (uint32_t)p[2 * i] : 127u) << (8 * i);
                odd |= (step * 8 + 2 * i + 1 < kb ? (uint32_t)p[2 * i + 1] : 127u) << (8 * i);
            }
        }
    }
    uint32_t* g = (is_a ? ga : gb) + (group * steps + step) * 64;
    g[r] = even;
    g[32 + r] = odd;
}

// Workgroups of TILE x TILE outputs, 2 TILE threads
constexpr int stage_bytes(int tile) { return 2 * tile * 128; }  // codes of both operands, 256 k
constexpr int buf_bytes(int tile) { return stage_bytes(tile) + 2 * (tile / 32) * 256; }  // and scales; two in LDS
constexpr int kShortSteps = 8;
constexpr int short_bytes(int tile) { return 2 * stage_bytes(tile) + 2 * tile * 8 * kShortSteps; }
constexpr int kCodeCopies = 8;   // asynchronous copies a thread issues per step: 2 TILE 128 / 16 / (2 TILE)
constexpr int kScaleCopies = 2;  // 2 TILE 8 / 4 / (2 TILE)

struct TileArgs {
    Mx4Mat a, b;
    const uint32_t* ga;
    const uint32_t* gb;
    Mx4Out o;
    int m_tiles, n_tiles;
};

// The workgroup's sums to memory: through LDS, so that a row leaves as
// neighbouring 16-byte stores and not as the matrix instruction's 4-element
// pieces.  A 32-bit tile of 256 passes in two halves of 128 rows (one of the
// waves' rows each).  A row's 16-byte unit v lies at v ^ (row & 7).
template <int DT, int TILE, int FA>
IQLH_DEV void store_tile(const TileArgs& t, const mx_f16 (&acc)[FA][2], uint8_t* lds, int64_t m0, int64_t n0, int wm,
                         int wn) {
    typedef typename MxFloat<DT>::type T;
    constexpr int HALVES = TILE * TILE * (int)sizeof(T) > 2 * buf_bytes(TILE) ? 2 : 1, ROWS = TILE / HALVES;
    constexpr int E = 16 / sizeof(T), UNITS = TILE / E;  // elements of a unit, units of a row
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const Mx4Out& o = t.o;
#pragma unroll
    for (int half = 0; half < HALVES; ++half) {
        if (half) __syncthreads();
        if (HALVES == 1 || wm / ROWS == half) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int n = wn + 32 * j + 8 * g + 4 * h;
                    float bias[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) bias[e] = o.bias && n0 + n + e < t.b.rows ? o.bias[n0 + n + e] : 0.f;
#pragma unroll
                    for (int i = 0; i < FA; ++i) {
                        const int row = (HALVES == 1 ? wm : 0) + 32 * i + r;
                        float y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            y[e] = acc[i][j][4 * g + e] + bias[e];
                            if (o.relu && y[e] < 0.f) y[e] = 0.f;  // a NaN stays
                        }
                        uint8_t* p = lds + row * (TILE * sizeof(T)) + 16 * ((n / E) ^ (row & 7)) + (n % E) * sizeof(T);
                        mx4_put4<DT>((T*)p, y);
                    }
                }
        }
        __syncthreads();
#pragma unroll 4
        for (int c = threadIdx.x; c < ROWS * UNITS; c += 2 * TILE) {
            const int row = c / UNITS, v = c % UNITS;
            const int64_t m = m0 + half * ROWS + row, n = n0 + v * E;
            if (m >= t.a.rows || n >= t.b.rows) continue;
            const uint4 w = *(const uint4*)(lds + row * (TILE * sizeof(T)) + 16 * (v ^ (row & 7)));
            T* p = (T*)o.p + m * o.ld + n;
            if (n + E <= t.b.rows) {
                typedef T tu __attribute__((ext_vector_type(E), aligned(sizeof(T))));
                *(tu*)p = __builtin_bit_cast(tu, w);
            } else {
                const T* e = (const T*)&w;
                for (int k = 0; k < E; ++k)
                    if (n + k < t.b.rows) p[k] = e[k];
            }
        }
    }
}

// TILE 256: eight waves, 2 x 4, each 128 x 64 outputs (4 x 2 fragments of
// 32 x 32, 128 registers of sums), one workgroup to a compute unit.  TILE 128: four
// waves, 2 x 2, each 64 x 64, two workgroups.  A step is 256 k, 128 bytes of a
// row: whole cache lines per request.  Two buffers: in the last quarter of
// step s every wave waits for its copies of step s + 1, passes the barrier
// (behind which all reads of step s's buffer are done), issues step s + 2 into
// that buffer and reads the first fragments of step s + 1 while the matrix
// instructions of the quarter run.  A row's chunk u (16 bytes) lies at
// 128 row + 16 (u ^ ((row >> 1) & 7)): 16 lanes of a fragment column fall on
// all 64 banks.  8192^3 280 to 314 us, 3.5 to 3.9 PF: by the counters the matrix units
// are busy 47 % of the cycles, at 1.93 GHz.  On registers alone the instruction
// reaches 6.2 PF on random codes, for which the clock falls to 1.5 GHz, and 9.8 on zeros
// at 2.4 GHz (16 x 16 ones 6.7 and 9.4; bench.py --probe mx4-rate).  Where a tile
// has a few steps only, by the chain of first load, steps and stores: 2048^3 12.3 us,
// 8192 x 8192 x 256 52.
// SHORT: K of at most kShortSteps steps, the scales of all of it in LDS before
// the first step, [2 TILE rows][kShortSteps] of 8 bytes, step s of row r at s ^ (r >> 2
// & 7) so that 32 rows' reads fall on all banks; no launch before this one.
template <int DT, int TILE, bool SHORT>
__global__ __launch_bounds__(2 * TILE, 2) void mx4_tile_kernel(TileArgs t) {
    constexpr int NT = 2 * TILE, FA = TILE / 64, WN = TILE / 64;  // threads, row fragments a wave, waves along n
    constexpr int STAGE = stage_bytes(TILE), BUF = SHORT ? STAGE : buf_bytes(TILE);
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t lds_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    const int r = lane & 31, h = lane >> 5;
    // consecutive workgroups go to different XCDs: give each XCD a run of
    // tiles, walked in columns of 4 tile rows, so that its L2 serves a
    // patch of about 4 x 8 tiles at a time
    const int total = t.m_tiles * t.n_tiles;
    int id = blockIdx.x;
    {
        const int per = total / 8, rest = total % 8, x = id & 7, k = id >> 3;
        id = x * per + (x < rest ? x : rest) + k;
    }
    const int band = id / (4 * t.n_tiles), in_band = id - band * 4 * t.n_tiles;
    const int rows_in = t.m_tiles - band * 4 < 4 ? t.m_tiles - band * 4 : 4;
    const int tm = band * 4 + in_band % rows_in, tn = in_band / rows_in;
    const int64_t kb = t.a.kb();
    const int steps = (int)((kb + 7) / 8);
    const int64_t m0 = (int64_t)tm * TILE, n0 = (int64_t)tn * TILE;
    // copy addresses: chunk c = i NT + tid fills place c & 7 of row c >> 3
    const int u = (tid & 7) ^ ((tid >> 4) & 7);
    const uint8_t* abase = t.a.codes + m0 * kb * 16;
    const uint8_t* bbase = t.b.codes + n0 * kb * 16;
    uint32_t off[kCodeCopies];  // b's rows, then a's
#pragma unroll
    for (int i = 0; i < kCodeCopies; ++i) {
        const int row = (i & 3) * (TILE / 4) + (tid >> 3);
        const int64_t left = (i < 4 ? t.b.rows - n0 : t.a.rows - m0) - 1;
        off[i] = (uint32_t)((row < left ? row : (int)left) * kb * 16) + 16u * u;
    }
    const uint32_t* sbase[kScaleCopies];  // scale groups `wave` of b and of a
    if constexpr (!SHORT) {
        const int64_t gb = n0 / 32 + wave, ga = m0 / 32 + wave;
        const int64_t lb = (t.b.rows + 31) / 32 - 1, la = (t.a.rows + 31) / 32 - 1;
        sbase[0] = t.gb + (gb < lb ? gb : lb) * steps * 64 + lane;
        sbase[1] = t.ga + (ga < la ? ga : la) * steps * 64 + lane;
    }
    // every step issues the same copies, those behind the last one from the
    // zero chunk, so that the loop has no branch
    auto issue = [&](int s) __attribute__((always_inline)) {
        const uint32_t dst = lds_at + (s & 1) * BUF;
        const int64_t k0 = (int64_t)s * 128;
        const bool in = 8 * s + u < kb;
#pragma unroll
        for (int i = 0; i < kCodeCopies; ++i) {
            const uint8_t* src = (i < 4 ? bbase : abase) + k0 + off[i];
            copy16(in ? src : (const uint8_t*)kZeroChunk, dst + i * NT * 16 + wave * 1024);
        }
        if constexpr (!SHORT) {
#pragma unroll
            for (int i = 0; i < kScaleCopies; ++i)
                copy4(sbase[i] + (int64_t)(s < steps ? s : steps - 1) * 64, dst + STAGE + (TILE / 32 * i + wave) * 256);
        }
    };
    const int wm = wave / WN * (32 * FA), wn = wave % WN * 64;
    struct Frags {
        uint4 a[FA], b[2];
    } f[2];
    uint32_t sa[2][FA], sb[2][2];
    auto load = [&](int s, auto quarter, auto p) __attribute__((always_inline)) {
        constexpr int Q = decltype(quarter)::value;
        const uint8_t* src = lds + (s & 1) * BUF;
        const int foff = r * 128 + 16 * ((2 * Q + h) ^ ((r >> 1) & 7));
        Frags& g = f[decltype(p)::value];
#pragma unroll
        for (int i = 0; i < 2; ++i) g.b[i] = *(const uint4*)(src + (wn + 32 * i) * 128 + foff);
#pragma unroll
        for (int i = 0; i < FA; ++i) g.a[i] = *(const uint4*)(src + (TILE + wm + 32 * i) * 128 + foff);
    };
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    auto load_scales = [&](int s, uint32_t (&pa)[FA], uint32_t (&pb)[2]) __attribute__((always_inline)) {
        if constexpr (SHORT) {
            const uint8_t* src = lds + 2 * STAGE + r * (8 * kShortSteps) + 8 * ((s < steps ? s : steps - 1) ^ (r >> 2 & 7));
            const uint32_t sel = h ? 0x07050301u : 0x06040200u;  // the bytes of blocks h, 2 + h, 4 + h, 6 + h
            auto group = [&](int row) __attribute__((always_inline)) {
                const u2 w = *(const u2*)(src + row * (8 * kShortSteps));
                return __builtin_amdgcn_perm(w.y, w.x, sel);
            };
#pragma unroll
            for (int i = 0; i < 2; ++i) pb[i] = group(wn + 32 * i);
#pragma unroll
            for (int i = 0; i < FA; ++i) pa[i] = group(TILE + wm + 32 * i);
            return;
        }
        const uint8_t* src = lds + (s & 1) * BUF + STAGE + lane * 4;
#pragma unroll
        for (int i = 0; i < 2; ++i) pb[i] = *(const uint32_t*)(src + (wn / 32 + i) * 256);
#pragma unroll
        for (int i = 0; i < FA; ++i) pa[i] = *(const uint32_t*)(src + (TILE / 32 + wm / 32 + i) * 256);
    };
    mx_f16 acc[FA][2];
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mx_f16{};
    auto mma = [&](auto quarter, auto p, const uint32_t (&pa)[FA], const uint32_t (&pb)[2]) __attribute__((always_inline)) {
        constexpr int Q = decltype(quarter)::value;
        const Frags& g = f[decltype(p)::value];
#pragma unroll
        for (int i = 0; i < FA; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = mx4_mma32<Q, Q>(g.b[j], g.a[i], acc[i][j], pb[j], pa[i]);
    };
    typedef std::integral_constant<int, 0> C0;
    typedef std::integral_constant<int, 1> C1;
    typedef std::integral_constant<int, 2> C2;
    typedef std::integral_constant<int, 3> C3;
    issue(0);
    if constexpr (SHORT) {  // a thread takes a row: b's, then a's
        const Mx4Mat& q = tid < TILE ? t.b : t.a;
        const int64_t row = tid < TILE ? n0 + tid : m0 + tid - TILE;
        const uint8_t* p = q.scales + (row < q.rows ? row : q.rows - 1) * kb;
        u2 w[kShortSteps];
#pragma unroll
        for (int d = 0; d < kShortSteps; ++d) {
            w[d] = u2{0x7F7F7F7Fu, 0x7F7F7F7Fu};
            if (8 * d + 8 <= kb) {
                typedef uint32_t u2u __attribute__((ext_vector_type(2), aligned(1)));
                w[d] = *(const u2u*)(p + 8 * d);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (8 * d + j < kb) w[d][j >> 2] = (w[d][j >> 2] & ~(255u << (8 * (j & 3)))) | (uint32_t)p[8 * d + j] << (8 * (j & 3));
            }
        }
#pragma unroll
        for (int d = 0; d < kShortSteps; ++d)
            if (d < steps) *(u2*)(lds + 2 * STAGE + tid * (8 * kShortSteps) + 8 * (d ^ (tid >> 2 & 7))) = w[d];
    }
    wait_vm<0>();
    bar();
    issue(1);
    load(0, C0(), C0());
    load_scales(0, sa[0], sb[0]);
    // per quarter: the next one's LDS reads, then this one's matrix instructions
    auto reads_first = [] __attribute__((always_inline)) {
        __builtin_amdgcn_sched_group_barrier(0x100, FA + 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 2 * FA, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    for (int s = 0; s < steps; ++s) {
        load(s, C1(), C1());
        mma(C0(), C0(), sa[0], sb[0]);
        reads_first();
        load(s, C2(), C0());
        mma(C1(), C1(), sa[0], sb[0]);
        reads_first();
        load(s, C3(), C1());
        mma(C2(), C0(), sa[0], sb[0]);
        reads_first();
        wait_vm<0>();  // step s + 1 has landed
        bar();
        issue(s + 2);
        load(s + 1, C0(), C0());
        load_scales(s + 1, sa[1], sb[1]);
        mma(C3(), C1(), sa[0], sb[0]);
        __builtin_amdgcn_sched_group_barrier(0x100, 2 * FA + 4, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 2 * FA, 0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < FA; ++i) sa[0][i] = sa[1][i];
#pragma unroll
        for (int i = 0; i < 2; ++i) sb[0][i] = sb[1][i];
    }
    wait_vm<0>();  // the copies behind the last step, before their buffers are used again
    bar();
    store_tile<DT, TILE, FA>(t, acc, lds, m0, n0, wm, wn);
}

size_t group_bytes(int64_t rows, int64_t kb) { return (size_t)((rows + 31) / 32) * (size_t)((kb + 7) / 8) * 256; }

// Which kernel a product runs on.
enum class Path { few, direct, split32x16, split32, split64, tile128, tile256 };
int64_t tiles_of(int64_t M, int64_t N, int64_t T) { return ((M + T - 1) / T) * ((N + T - 1) / T); }
Path pick(int64_t M, int64_t N, int64_t K) {
    if (M <= 16 && few_bytes(M, K) <= 80 << 10) return Path::few;  // two workgroups to a compute unit
    const bool lds_tiles = K <= 1 << 22 && tiles_of(M, N, 128) < 1 << 22;  // 32-bit offsets in a tile, grid sizes
    // 256 tiles for most compute units.  128 | 256 tiles, us, at K 512, 1500, 4096: 128 of
    // the large ones 12.3 | 14.8, 18.9 | 21.9, 33.8 | 39.7; 169: 17.6 | 15.3, 26.6 | 23.7, 42.5 |
    // 42.4; 196: 19.5 | 15.9, 31.6 | 25.3, 51.4 | 43.0; 256: 20.5 | 17.1, 35.1 | 27.8, 56.1 | 47.2; 289,
    // the first of a second round: 25.2 | 26.7, 41.7 | 43.2, 68.0 | 74.7; 1024: 64.7 | 57.9, 117
    // | 97, 198 | 168
    if (lds_tiles && K >= 256 && tiles_of(M, N, 256) >= 192) return Path::tile256;
    // waves that split k, the smallest outputs a workgroup that a round of workgroups
    // covers: 32 x 16 (20 x 4096 x 4096: 4.8 us, with 32 x 32 5.2), 32 x 32, two to a
    // compute unit (512^3: 3.4, with 64 x 64 5.1; 1000^3, two rounds, 7.2 against
    // 6.0), 64 x 64 (900 x 900 x 3000: 10.5; by 128 tiles 14.9)
    if ((M + 31) / 32 * ((N + 15) / 16) <= kComputeUnits) return Path::split32x16;
    if (tiles_of(M, N, 32) <= 2 * kComputeUnits) return Path::split32;
    if (tiles_of(M, N, 64) <= kComputeUnits) return Path::split64;
    // more: straight from memory where the sums are short (1500 x 1500 x 256: 8.8
    // us, 128 tiles 9.0; K 384 8.7 against 10.0, K 512 11.7 against 9.7)
    if (K <= 384) return Path::direct;
    return lds_tiles ? Path::tile128 : Path::split64;
}

template <int TILE>
hipError_t launch_tiles(const Mx4Mat& a, const Mx4Mat& b, const Mx4Out& out, void* workspace, hipStream_t stream) {
    TileArgs t{a, b, nullptr, nullptr, out, (int)((a.rows + TILE - 1) / TILE), (int)((b.rows + TILE - 1) / TILE)};
    auto launch = [&](auto is_short) {
        constexpr bool SHORT = decltype(is_short)::value;
        return by_dtype(out.dtype, [&](auto dt) {
            constexpr int bytes = SHORT ? short_bytes(TILE) : 2 * buf_bytes(TILE);
            static_assert(bytes <= 160 * 1024, "LDS of a compute unit");
            auto kernel = mx4_tile_kernel<decltype(dt)::value, TILE, SHORT>;
            (void)hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
            hipLaunchKernelGGL(kernel, dim3((uint32_t)(t.m_tiles * t.n_tiles)), dim3(2 * TILE), bytes, stream, t);
        });
    };
    if (a.cols <= kShortSteps * 256) return launch(std::true_type());
    t.ga = (const uint32_t*)workspace;
    t.gb = (const uint32_t*)((const char*)workspace + group_bytes(a.rows, a.kb()));
    const uint32_t ag = (uint32_t)((a.rows + 31) / 32), bg = (uint32_t)((b.rows + 31) / 32);
    hipLaunchKernelGGL(mx4_scale_groups_kernel, dim3(ag + bg, (uint32_t)((a.kb() + 63) / 64)), dim3(kNT), 0, stream, a, b,
                       (uint32_t*)t.ga, (uint32_t*)t.gb, (int)ag);
    return launch(std::false_type());
}

template <int MF, int NF, int D>
hipError_t launch_split(const Mx4Mat& a, const Mx4Mat& b, const Mx4Out& out, hipStream_t stream) {
    const int64_t mt = (a.rows + 16 * MF - 1) / (16 * MF), nt = (b.rows + 16 * NF - 1) / (16 * NF);
    const int64_t steps = (a.kb() + 3) / 4;
    const int most = kSplitSteps<MF, NF, D>;
    const int bytes = kSplitRing<MF, NF, D> + 16 * (MF + NF) * split_scale_row(steps < most ? steps : most);
    static_assert(kSplitRing<MF, NF, D> + 16 * (MF + NF) * split_scale_row(kSplitSteps<MF, NF, D>) <= 160 * 1024 &&
                      4 * MF * NF * 1024 <= kSplitRing<MF, NF, D>, "LDS of a compute unit");
    return by_dtype(out.dtype, [&](auto dt) {
        auto kernel = mx4_split_kernel<decltype(dt)::value, MF, NF, D>;
        (void)hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        hipLaunchKernelGGL(kernel, dim3((uint32_t)(mt * nt)), dim3(512), bytes, stream, a, b, out, (int)nt);
    });
}

}  // namespace

size_t mx4_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    const int64_t kb = (K + 31) / 32;
    const Path p = pick(M, N, K);
    return K > kShortSteps * 256 && (p == Path::tile256 || p == Path::tile128) ? group_bytes(M, kb) + group_bytes(N, kb) : 16;
}

// Launches hold less than 2^32 threads
bool mx4_launchable(int64_t M, int64_t N, int64_t K) {
    const int64_t top = (int64_t)1 << 32;
    switch (pick(M, N, K)) {
        case Path::few: return (N + 15) / 16 * 512 < top;
        case Path::direct: return tiles_of(M, N, 128) * kNT < top;
        case Path::split32x16:
        case Path::split32: break;
        case Path::split64: return tiles_of(M, N, 64) < top / 512;
        case Path::tile128:
        case Path::tile256: break;  // bounded by pick; the scales' regrouping by their rows
    }
    return ((M + 31) / 32 + (N + 31) / 32) * kNT < top;
}

// One launch with the left operand quantised by every workgroup, which is its time
// where its part is large: for up to 16 rows (16 x 1024 x 1024 4.7 us, in two
// launches 7), and for more where the workgroups are one round (300 x 300, K 100:
// 5.0; 61 x 26, K 407, 30000 elements a workgroup: 8.3 against 6.4)
bool mx4_few_ok(int64_t M, int64_t N, int64_t K) {
    const int64_t k4 = (K + 127) / 128 * 128, nt = (N + 15) / 16;
    if (M <= 16) return M * k4 <= 2 * kFewElements;
    return (M < 64 ? M : 64) * k4 <= kFewElements && nt * ((M + 63) / 64) <= kComputeUnits;
}

hipError_t launch_mx4_few(const void* x, int dtype, int64_t ld, int64_t M, const Mx4Mat& b, const Mx4Out& out,
                          hipStream_t stream) {
    const Mx4Mat a{nullptr, nullptr, M, b.cols};
    if (dtype == IQLH_F32) return launch_few_rows_of<IQLH_F32>(a, x, ld, b, out, stream);
    if (dtype == IQLH_BF16) return launch_few_rows_of<IQLH_BF16>(a, x, ld, b, out, stream);
    return launch_few_rows_of<IQLH_F16>(a, x, ld, b, out, stream);
}

hipError_t launch_mx4_matmul(const Mx4Mat& a, const Mx4Mat& b, const Mx4Out& out, void* workspace,
                             hipStream_t stream) {
    switch (pick(a.rows, b.rows, a.cols)) {
        case Path::few: return launch_few_rows<-1, 1>(a, nullptr, 0, b, out, stream);
        case Path::tile256: return launch_tiles<256>(a, b, out, workspace, stream);
        case Path::tile128: return launch_tiles<128>(a, b, out, workspace, stream);
        case Path::split32x16: return launch_split<2, 1, 4>(a, b, out, stream);
        case Path::split32: return launch_split<2, 2, 2>(a, b, out, stream);
        case Path::split64: return launch_split<4, 4, 2>(a, b, out, stream);
        case Path::direct: break;
    }
    const int64_t mt = (a.rows + 127) / 128, nt = (b.rows + 127) / 128;
    return by_dtype(out.dtype, [&](auto dt) {
        hipLaunchKernelGGL(mx4_direct_kernel<decltype(dt)::value>, dim3((uint32_t)(mt * nt)), dim3(kNT), 0, stream, a, b,
                           out, (int)nt);
    });
}

}  // namespace iqlh
