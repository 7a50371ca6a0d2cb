// Product of two microscaled 4-bit matrices,
//   out[m][n] = act(sum_k a[m][k] b[n][k] + bias[n]),
// on v_mfma_scale_f32_16x16x128_f8f6f4 (16 x 16 outputs, 128 k, one scale byte
// per 32 k and row).  b is the instruction's row operand in every kernel, so
// that a lane holds four neighbouring n of one output row.
//
// Three kernels by shape (launch_mx4_matmul):
//   few rows (M <= 16): HBM-bound on b; a workgroup takes 16 rows of b, its
//     waves split k, and every lane has its wave's whole share in flight;
//   tiles of 256 x 256 with operands staged through LDS by asynchronous
//     copies, where there are enough of them to fill the chip;
//   tiles straight from global memory for what lies between, its waves
//     splitting k where tiles are few.
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
// wave order.
constexpr int kFewWaves = 8;
constexpr int kFewElements = 32768;  // of a workgroup's part of a float left operand, padded
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
        for (int e = threadIdx.x; e < rows * kb4; e += NT) {
            const int row = e / kb4, k = e - row * kb4;
            const bool in = k < kb;
            const int64_t at = (m0 + row) * kb + (in ? k : 0);
            const uint4 w = ((const uint4*)a.codes)[at];
            const uint32_t s = a.scales[at], keep = in ? 0xFFFFFFFFu : 0u;
            *(uint4*)(codes + row * rb + k * 16) = uint4{w.x & keep, w.y & keep, w.z & keep, w.w & keep};
            scales[e] = (uint8_t)(in ? s : 127u);
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
// from L2: for K of a step or two, where a ring would not fill.
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
// A workgroup takes 16 MF x 16 NF outputs, its eight waves every eighth k step
// each, the next step's fragments on their way while this one's are
// multiplied.  The sums meet in LDS: waves 4..7 add to waves 0..3, then those
// four are added in wave order.  For few outputs, where what counts is how
// many loads are in flight over the chip.
template <int DT, int MF, int NF>
__global__ __launch_bounds__(512) void mx4_split_kernel(Mx4Mat a, Mx4Mat b, Mx4Out o, int n_tiles) {
    extern __shared__ __align__(16) uint8_t lds[];
    mx_f4(*part)[MF * NF][64] = (mx_f4(*)[MF * NF][64])lds;  // [4]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, blk = lane >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x / n_tiles) * (16 * MF), n0 = (int64_t)(blockIdx.x % n_tiles) * (16 * NF);
    const int64_t kb = a.kb();
    const uint4* ac[MF];
    const uint8_t* as_[MF];
#pragma unroll
    for (int i = 0; i < MF; ++i) {
        const RowFrag f(a, m0 + 16 * i + r);
        ac[i] = f.codes;
        as_[i] = f.scales;
    }
    const uint4* bc[NF];
    const uint8_t* bs_[NF];
#pragma unroll
    for (int j = 0; j < NF; ++j) {
        const RowFrag f(b, n0 + 16 * j + r);
        bc[j] = f.codes;
        bs_[j] = f.scales;
    }
    struct Frags {
        uint4 a[MF], b[NF];
        uint32_t as[MF], bs[NF];
    } f[2];
    auto load = [&](int64_t s, Frags& g) __attribute__((always_inline)) {
        const int64_t block = s * 4 + blk;
        const bool in = block < kb;
        const int64_t at = in ? block : 0;
        const uint32_t keep = in ? 0xFFFFFFFFu : 0u;
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            g.b[j] = bc[j][at];
            g.bs[j] = bs_[j][at];
        }
#pragma unroll
        for (int i = 0; i < MF; ++i) {
            const uint4 v = ac[i][at];
            g.a[i] = uint4{v.x & keep, v.y & keep, v.z & keep, v.w & keep};  // zeros behind the last block
            g.as[i] = in ? as_[i][at] : 127u;
        }
#pragma unroll
        for (int j = 0; j < NF; ++j) g.bs[j] = in ? g.bs[j] : 127u;
    };
    mx_f4 acc[MF][NF];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[i][j] = mx_f4{0.f, 0.f, 0.f, 0.f};
    auto mma = [&](const Frags& g) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int j = 0; j < NF; ++j) acc[i][j] = mx4_mma(g.b[j], g.a[i], acc[i][j], g.bs[j], g.as[i]);
    };
    const int64_t steps = (kb + 3) / 4;
    load(wave, f[0]);
    int64_t s = wave;
    for (; s + 8 < steps; s += 16) {
        load(s + 8, f[1]);
        mma(f[0]);
        load(s + 16, f[0]);  // zeros behind the last step
        mma(f[1]);
    }
    if (s < steps) mma(f[0]);
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

// ------------------------------------------------------- tiles through LDS
// Scales regrouped for the tile kernel: for 32 rows and the 8 blocks of a
// step one dword per lane, byte i the scale of row lane & 31, block
// 2 i + (lane >> 5), so that a lane's dword serves the step's four matrix
// instructions of a fragment (the instruction selects the byte).
// [32-row group][step][lane]; rows and blocks past the end get 127.
// A workgroup takes 32 rows and 8 steps, 64 bytes of each row.
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

__device__ __align__(16) const uint4 kZeroChunk[1] = {};

// Workgroups of TILE x TILE outputs, 2 TILE threads
constexpr int stage_bytes(int tile) { return 2 * tile * 128; }  // codes of both operands, 256 k
constexpr int buf_bytes(int tile) { return stage_bytes(tile) + 2 * (tile / 32) * 256; }  // and scales; two in LDS
constexpr int kCodeCopies = 8;   // asynchronous copies a thread issues per step: 2 TILE 128 / 16 / (2 TILE)
constexpr int kScaleCopies = 2;  // 2 TILE 8 / 4 / (2 TILE)

template <int N>
IQLH_DEV void wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// Asynchronous copy of 16 (4) bytes per lane, global -> LDS, to lds_at + 16 (4)
// lane.  As an instruction of its own and not the compiler's builtin: behind
// the builtin the compiler waits for every copy in flight before each LDS
// read that may alias one, which is all of them, and the ring runs empty.  It
// has no output registers; wait_vm orders it against the reads.  (One wait
// state between writing M0 and its use by the copy.)
IQLH_DEV void copy16(const void* src, uint32_t lds_at) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"{m0}"(lds_at), "v"(src) : "memory");
}
IQLH_DEV void copy4(const void* src, uint32_t lds_at) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %1, off" ::"{m0}"(lds_at), "v"(src) : "memory");
}
// Workgroup barrier after this wave's LDS reads, leaving the asynchronous
// copies it has in flight
IQLH_DEV void bar() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

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
// all 64 banks.
template <int DT, int TILE>
__global__ __launch_bounds__(2 * TILE, 2) void mx4_tile_kernel(TileArgs t) {
    constexpr int NT = 2 * TILE, FA = TILE / 64, WN = TILE / 64;  // threads, row fragments a wave, waves along n
    constexpr int STAGE = stage_bytes(TILE), BUF = buf_bytes(TILE);
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
    {
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
#pragma unroll
        for (int i = 0; i < kScaleCopies; ++i)
            copy4(sbase[i] + (int64_t)(s < steps ? s : steps - 1) * 64, dst + STAGE + (TILE / 32 * i + wave) * 256);
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
    auto load_scales = [&](int s, uint32_t (&pa)[FA], uint32_t (&pb)[2]) __attribute__((always_inline)) {
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
enum class Path { few, direct, split1, split2, split4, tile128, tile256 };
int64_t tiles_of(int64_t M, int64_t N, int64_t T) { return ((M + T - 1) / T) * ((N + T - 1) / T); }
Path pick(int64_t M, int64_t N, int64_t K) {
    if (M <= 16 && few_bytes(M, K) <= 80 << 10) return Path::few;  // two workgroups to a compute unit
    const bool lds_tiles = K <= 1 << 22 && tiles_of(M, N, 128) < 1 << 22;  // 32-bit offsets in a tile, grid sizes
    // 256 tiles for most compute units (2048 x 4096 x 4096, 128 of them: 39.1 us
    // against 30.5 with 128 tiles; 4096^3, 256 of them: 45.0)
    if (lds_tiles && K >= 256 && tiles_of(M, N, 256) >= 192) return Path::tile256;
    // a step or two: the waves that split k have little to split, but eight of
    // them store a 64 x 64 tile; more tiles than two rounds go to 128 x 128 by four
    // waves (1000 x 1000 x 128: 5.4 against 6.5 us, 2000 x 2000 x 200 15.9 against 8.2)
    const int64_t tiles64 = tiles_of(M, N, 64);
    if (K <= 256) return tiles64 <= 512 ? Path::split4 : Path::direct;
    // 128 tiles against waves that split k, both as measured up to a round of
    // tiles: the tiles take 8 us and 2.1 per 1000 k whatever their number, the
    // splitting waves 3 us and 5 per 10^9 products (as many at K 1024 and below,
    // where waves go without a step).  768 x 1024 x 4096: 16.3 against 29.5 us;
    // 512 x 512 x 2048: 11.7 against 8.5; 6281 x 1202 x 454: 13.3 against 32.2
    const double split_us = 3.0 + 5e-9 * (double)M * (double)N * (double)(K < 1024 ? 1024 : K);
    if (lds_tiles && split_us > 8.0 + 2.1e-3 * (double)K) return Path::tile128;
    // the largest of the splitting tiles that gives every compute unit one,
    // where there are steps for all eight waves
    if (K <= 512 || tiles64 >= 256) return Path::split4;
    if (M > 32 && ((M + 63) / 64) * ((N + 31) / 32) >= 256) return Path::split2;
    return Path::split1;
}

template <int TILE>
hipError_t launch_tiles(const Mx4Mat& a, const Mx4Mat& b, const Mx4Out& out, void* workspace, hipStream_t stream) {
    TileArgs t{a, b, nullptr, nullptr, out, (int)((a.rows + TILE - 1) / TILE), (int)((b.rows + TILE - 1) / TILE)};
    t.ga = (const uint32_t*)workspace;
    t.gb = (const uint32_t*)((const char*)workspace + group_bytes(a.rows, a.kb()));
    const uint32_t ag = (uint32_t)((a.rows + 31) / 32), bg = (uint32_t)((b.rows + 31) / 32);
    hipLaunchKernelGGL(mx4_scale_groups_kernel, dim3(ag + bg, (uint32_t)((a.kb() + 63) / 64)), dim3(kNT), 0, stream, a, b,
                       (uint32_t*)t.ga, (uint32_t*)t.gb, (int)ag);
    return by_dtype(out.dtype, [&](auto dt) {
        constexpr int bytes = 2 * buf_bytes(TILE);
        static_assert(bytes <= 160 * 1024, "LDS of a compute unit");
        auto kernel = mx4_tile_kernel<decltype(dt)::value, TILE>;
        (void)hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        hipLaunchKernelGGL(kernel, dim3((uint32_t)(t.m_tiles * t.n_tiles)), dim3(2 * TILE), bytes, stream, t);
    });
}

template <int MF, int NF>
hipError_t launch_split(const Mx4Mat& a, const Mx4Mat& b, const Mx4Out& out, hipStream_t stream) {
    const int64_t mt = (a.rows + 16 * MF - 1) / (16 * MF), nt = (b.rows + 16 * NF - 1) / (16 * NF);
    return by_dtype(out.dtype, [&](auto dt) {
        hipLaunchKernelGGL((mx4_split_kernel<decltype(dt)::value, MF, NF>), dim3((uint32_t)(mt * nt)), dim3(512),
                           4 * MF * NF * 1024, stream, a, b, out, (int)nt);
    });
}

}  // namespace

size_t mx4_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    const int64_t kb = (K + 31) / 32;
    const Path p = pick(M, N, K);
    return p == Path::tile256 || p == Path::tile128 ? group_bytes(M, kb) + group_bytes(N, kb) : 16;
}

// Launches hold less than 2^32 threads
bool mx4_launchable(int64_t M, int64_t N, int64_t K) {
    const int64_t top = (int64_t)1 << 32;
    switch (pick(M, N, K)) {
        case Path::few: return (N + 15) / 16 * 512 < top;
        case Path::direct: return tiles_of(M, N, 128) * kNT < top;
        case Path::split1: return (M + (M <= 32 ? 31 : 63)) / (M <= 32 ? 32 : 64) * ((N + 15) / 16) < top / 512;
        case Path::split2: return (M + 63) / 64 * ((N + 31) / 32) < top / 512;
        case Path::split4: return tiles_of(M, N, 64) < top / 512;
        case Path::tile128:
        case Path::tile256: break;  // bounded by pick; the scales' regrouping by their rows
    }
    return ((M + 31) / 32 + (N + 31) / 32) * kNT < top;
}

// One launch with the left operand quantised by every workgroup: for up to 16
// rows, and for more where the workgroups are one round (61 x 26, K 407: 8.5
// us, in two launches 9.9; two and a half rounds at 33 x 5853, K 385: 12.3 against
// 10.0)
bool mx4_few_ok(int64_t M, int64_t N, int64_t K) {
    const int64_t k4 = (K + 127) / 128 * 128, nt = (N + 15) / 16;
    if ((M < 64 ? M : 64) * k4 > kFewElements) return false;
    return M <= 16 || nt * ((M + 63) / 64) <= kComputeUnits;
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
        case Path::split4: return launch_split<4, 4>(a, b, out, stream);
        case Path::split2: return launch_split<4, 2>(a, b, out, stream);
        case Path::split1: return a.rows <= 32 ? launch_split<2, 1>(a, b, out, stream) : launch_split<4, 1>(a, b, out, stream);
        case Path::direct: break;
    }
    const int64_t mt = (a.rows + 127) / 128, nt = (b.rows + 127) / 128;
    return by_dtype(out.dtype, [&](auto dt) {
        hipLaunchKernelGGL(mx4_direct_kernel<decltype(dt)::value>, dim3((uint32_t)(mt * nt)), dim3(kNT), 0, stream, a, b,
                           out, (int)nt);
    });
}

}  // namespace iqlh
