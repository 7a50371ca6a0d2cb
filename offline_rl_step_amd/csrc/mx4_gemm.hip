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
#define IQLH_LDS(p) ((__attribute__((address_space(3))) void*)(p))

template <typename F>
hipError_t by_dtype(int dtype, F f) {
    if (dtype == IQLH_F32) f(std::integral_constant<int, IQLH_F32>());
    else if (dtype == IQLH_BF16) f(std::integral_constant<int, IQLH_BF16>());
    else f(std::integral_constant<int, IQLH_F16>());
    return hipGetLastError();
}

// 16 rows from row0 on, blocks 4 step .. 4 step + 3, of a matrix in memory:
// this lane's 16 bytes and scale.  Rows past the end read the last one (their
// outputs are never stored), blocks past the end are zeros of scale 1.
struct RowFrag {
    const uint4* codes;
    const uint8_t* scales;
    int64_t kb;
    IQLH_DEV RowFrag(const Mx4Mat& q, int64_t row) : kb(q.kb()) {
        const int64_t r = row < q.rows ? row : q.rows - 1;
        codes = (const uint4*)q.codes + r * kb;
        scales = q.scales + r * kb;
    }
    IQLH_DEV void load(int64_t block, uint4& v, uint32_t& s) const {
        const bool in = block < kb;
        v = codes[in ? block : 0];
        s = scales[in ? block : 0];
        const uint32_t keep = in ? 0xFFFFFFFFu : 0u;
        v = uint4{v.x & keep, v.y & keep, v.z & keep, v.w & keep};
        s = in ? s : 127u;
    }
};

// ------------------------------------------------------------- few rows
// M <= 16.  Workgroup: 16 rows of b.  Wave w of WAVES takes the k steps w,
// w + WAVES, ..; U steps' loads are in flight together.  The waves' sums meet
// in LDS, added in wave order.
template <int DT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void mx4_few_rows_kernel(Mx4Mat a, Mx4Mat b, Mx4Out o) {
    constexpr int U = 4;
    __shared__ mx_f4 part[WAVES][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, blk = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const RowFrag fa(a, r), fb(b, n0 + r);
    const int64_t steps = (a.kb() + 3) / 4;
    mx_f4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int64_t s0 = wave; s0 < steps; s0 += WAVES * U) {
        uint4 av[U], bv[U];
        uint32_t as[U], bs[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t block = (s0 + u * WAVES) * 4 + blk;
            fb.load(block, bv[u], bs[u]);
            fa.load(block, av[u], as[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) acc = mx4_mma(bv[u], av[u], acc, bs[u], as[u]);
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave == 0 && r < a.rows) {
#pragma unroll
        for (int w = 1; w < WAVES; ++w) acc += part[w][lane];
        const int64_t n = n0 + 4 * blk;
        mx4_store4<DT>(o, r, n, (int)(b.rows - n < 4 ? b.rows - n : 4), acc, mx4_wide_rows<DT>(o));
    }
}

// ------------------------------------------------- tiles from global memory
// A wave computes 64 x 64 outputs, 4 x 4 fragments.  WK = 1: the workgroup's
// four waves take 128 x 128 outputs; WK = 4: they take the same 64 x 64 and
// every fourth k step each, and add their sums through LDS in wave order.
template <int DT, int WK>
__global__ __launch_bounds__(kNT) void mx4_direct_kernel(Mx4Mat a, Mx4Mat b, Mx4Out o, int n_tiles) {
    constexpr int T = WK == 1 ? 128 : 64;
    __shared__ mx_f4 part[WK == 1 ? 1 : 4][WK == 1 ? 1 : 16][WK == 1 ? 1 : 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, blk = lane >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x / n_tiles) * T + (WK == 1 ? (wave >> 1) * 64 : 0);
    const int64_t n0 = (int64_t)(blockIdx.x % n_tiles) * T + (WK == 1 ? (wave & 1) * 64 : 0);
    const RowFrag fa[4] = {RowFrag(a, m0 + r), RowFrag(a, m0 + 16 + r), RowFrag(a, m0 + 32 + r), RowFrag(a, m0 + 48 + r)};
    const RowFrag fb[4] = {RowFrag(b, n0 + r), RowFrag(b, n0 + 16 + r), RowFrag(b, n0 + 32 + r), RowFrag(b, n0 + 48 + r)};
    mx_f4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mx_f4{0.f, 0.f, 0.f, 0.f};
    const int64_t steps = (a.kb() + 3) / 4;
    for (int64_t s = WK == 1 ? 0 : wave; s < steps; s += WK) {
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
    const bool wide = mx4_wide_rows<DT>(o);
    auto store = [&](int i, int j, mx_f4 v) {
        const int64_t m = m0 + 16 * i + r, n = n0 + 16 * j + 4 * blk;
        if (m < a.rows) mx4_store4<DT>(o, m, n, (int)(b.rows - n < 4 ? b.rows - n : 4), v, wide);
    };
    if constexpr (WK == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) store(i, j, acc[i][j]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) part[wave][4 * i + j][lane] = acc[i][j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // wave w: fragments (w, 0..3)
            mx_f4 v = part[0][4 * wave + j][lane];
#pragma unroll
            for (int w = 1; w < 4; ++w) v += part[w][4 * wave + j][lane];
            store(wave, j, v);
        }
    }
}

// ------------------------------------------------------- tiles through LDS
// Scales regrouped for the tile kernel: for 64 rows and 4 blocks of a step one
// dword per lane, byte i the scale of row 16 i + (lane & 15), block lane >> 4, so
// that a lane's dword serves four fragments (the instruction selects the
// byte).  [64-row group][step][lane]; rows and blocks past the end get 127.
__global__ __launch_bounds__(kNT) void mx4_scale_groups_kernel(Mx4Mat a, Mx4Mat b, uint32_t* __restrict__ ga,
                                                               uint32_t* __restrict__ gb, int64_t na, int64_t nb) {
    int64_t e = (int64_t)blockIdx.x * kNT + threadIdx.x;
    if (e >= na + nb) return;
    const Mx4Mat& q = e < na ? a : b;
    uint32_t* g = e < na ? ga : gb;
    e = e < na ? e : e - na;
    const int64_t kb = q.kb(), steps = (kb + 3) / 4;
    const int lane = (int)(e & 63);
    const int64_t block = (e >> 6) % steps * 4 + (lane >> 4), row = (e >> 6) / steps * 64 + (lane & 15);
    uint32_t w = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool in = row + 16 * i < q.rows && block < kb;
        w |= (in ? (uint32_t)q.scales[(row + 16 * i) * kb + block] : 127u) << (8 * i);
    }
    g[e] = w;
}

__device__ __align__(16) const uint4 kZeroChunk[1] = {};

constexpr int kTile = 256;
constexpr int kStages = 4;                        // ring of 4 k steps, 3 in flight
constexpr int kStageBytes = 2 * kTile * 64;       // codes of both operands, 128 k
constexpr int kScaleBytes = 2 * (kTile / 64) * 256;
constexpr int kTNT = 512;
constexpr int kCodeCopies = kStageBytes / 16 / kTNT;
constexpr int kCopies = kCodeCopies + kScaleBytes / 4 / kTNT;  // asynchronous copies a thread issues per step

template <int N>
IQLH_DEV void wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// Workgroup barrier that leaves the asynchronous copies in flight
IQLH_DEV void bar() {
    asm volatile("" ::: "memory");
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

// Eight waves, 2 x 4, each 128 x 64 outputs (8 x 4 fragments, 128 registers
// of sums), two waves per SIMD.
// Ring: step s lives in buffer s % kStages; its buffer is refilled (step s +
// kStages) after the barrier of step s + 1, which every wave reaches with its
// reads of step s done.  A row's 64 bytes of a step lie at 64 row, chunk u at
// u ^ ((row >> 1) & 3): the 16 lanes of a fragment column then fall on all
// banks.
template <int DT>
__global__ __launch_bounds__(kTNT, 2) void mx4_tile_kernel(TileArgs t) {
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wbase = tid & ~63;
    const int r = lane & 15, blk = lane >> 4;
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
    const int steps = (int)((kb + 3) / 4);
    const int64_t m0 = (int64_t)tm * kTile, n0 = (int64_t)tn * kTile;
    // copy addresses: chunk c = i 512 + tid holds row c >> 2, chunk (c & 3) ^ ((row >> 1) & 3)
    const int u = (tid & 3) ^ ((tid >> 3) & 3);
    const uint8_t* abase = t.a.codes + m0 * kb * 16;
    const uint8_t* bbase = t.b.codes + n0 * kb * 16;
    uint32_t off[kCodeCopies];  // b's rows, then a's
#pragma unroll
    for (int i = 0; i < kCodeCopies; ++i) {
        const int row = (i & 1) * 128 + (tid >> 2);
        const int64_t left = (i < 2 ? t.b.rows - n0 : t.a.rows - m0) - 1;
        off[i] = (uint32_t)((row < left ? row : (int)left) * kb * 16) + 16u * u;
    }
    const uint32_t* sbase;  // scale group `wave`: b's four, then a's four
    {
        const int64_t grp = wave < 4 ? n0 / 64 + wave : m0 / 64 + wave - 4;
        const int64_t last = (wave < 4 ? t.b.rows + 63 : t.a.rows + 63) / 64 - 1;
        sbase = (wave < 4 ? t.gb : t.ga) + (grp < last ? grp : last) * steps * 64 + lane;
    }
    // every step issues the same copies, those behind the last one from the
    // zero chunk, so that the loop has no branch and one wait count
    auto issue = [&](int s) __attribute__((always_inline)) {
        uint8_t* dst = lds + (s & (kStages - 1)) * (kStageBytes + kScaleBytes);
        const int64_t k0 = (int64_t)s * 64;
        const bool in = 4 * s + u < kb;
#pragma unroll
        for (int i = 0; i < kCodeCopies; ++i) {
            const uint8_t* src = (i < 2 ? bbase : abase) + k0 + off[i];
            __builtin_amdgcn_global_load_lds((const void*)(in ? src : (const uint8_t*)kZeroChunk),
                                             IQLH_LDS(dst + (i * kTNT + wbase) * 16), 16, 0, 0);
        }
        __builtin_amdgcn_global_load_lds((const void*)(sbase + (int64_t)(s < steps ? s : steps - 1) * 64),
                                         IQLH_LDS(dst + kStageBytes + wave * 256), 4, 0, 0);
    };
    const int wm = (wave >> 2) * 128, wn = (wave & 3) * 64;
    const int foff = r * 64 + 16 * (blk ^ ((r >> 1) & 3));
    mx_f4 acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mx_f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) issue(s);
    for (int s = 0; s < steps; ++s) {
        wait_vm<(kStages - 2) * kCopies>();  // step s has landed, the two behind it may be in flight
        bar();
        issue(s + kStages - 1);
        const uint8_t* src = lds + (s & (kStages - 1)) * (kStageBytes + kScaleBytes);
        uint4 av[8], bv[4];
        uint32_t sa[2];
        const uint32_t sb = *(const uint32_t*)(src + kStageBytes + (wn / 64) * 256 + lane * 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) sa[i] = *(const uint32_t*)(src + kStageBytes + (4 + wm / 64 + i) * 256 + lane * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) bv[i] = *(const uint4*)(src + (wn + 16 * i) * 64 + foff);
#pragma unroll
        for (int i = 0; i < 8; ++i) av[i] = *(const uint4*)(src + (kTile + wm + 16 * i) * 64 + foff);
        static_for<8>([&](auto i) __attribute__((always_inline)) {
            static_for<4>([&](auto j) __attribute__((always_inline)) {
                constexpr int I = decltype(i)::value, J = decltype(j)::value;
                acc[I][J] = mx4_mma_sel<J & 3, I & 3>(bv[J], av[I], acc[I][J], sb, sa[I >> 2]);
            });
        });
        __builtin_amdgcn_sched_group_barrier(0x100, 15, 0);  // the LDS reads
        __builtin_amdgcn_sched_group_barrier(0x008, 32, 0);  // then the matrix instructions
    }
    wait_vm<0>();  // the copies behind the last step, before this workgroup's LDS is given away
    const bool wide = mx4_wide_rows<DT>(t.o);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t m = m0 + wm + 16 * i + r;
        if (m >= t.a.rows) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + wn + 16 * j + 4 * blk;
            mx4_store4<DT>(t.o, m, n, (int)(t.b.rows - n < 4 ? t.b.rows - n : 4), acc[i][j], wide);
        }
    }
}

size_t group_bytes(int64_t rows, int64_t kb) { return (size_t)((rows + 63) / 64) * (size_t)((kb + 3) / 4) * 256; }

}  // namespace

// the tile kernel: enough tiles for most compute units, and steps enough to
// fill its ring; its copies address a tile by 32-bit offsets
bool mx4_use_tiles(int64_t M, int64_t N, int64_t K) {
    const int64_t tiles = (M + kTile - 1) / kTile * ((N + kTile - 1) / kTile);
    return tiles >= 128 && tiles < (1 << 30) && K >= 1024 && K <= (1 << 22);
}

size_t mx4_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    const int64_t kb = (K + 31) / 32;
    return mx4_use_tiles(M, N, K) ? group_bytes(M, kb) + group_bytes(N, kb) : 16;
}

hipError_t launch_mx4_matmul(const Mx4Mat& a, const Mx4Mat& b, const Mx4Out& out, void* workspace,
                             hipStream_t stream) {
    if (a.rows <= 16) {
        return by_dtype(out.dtype, [&](auto dt) {
            hipLaunchKernelGGL((mx4_few_rows_kernel<decltype(dt)::value, 8>), dim3((uint32_t)((b.rows + 15) / 16)),
                               dim3(512), 0, stream, a, b, out);
        });
    }
    if (mx4_use_tiles(a.rows, b.rows, a.cols)) {
        TileArgs t{a, b, nullptr, nullptr, out, (int)((a.rows + kTile - 1) / kTile), (int)((b.rows + kTile - 1) / kTile)};
        const size_t na = group_bytes(a.rows, a.kb()), nb = group_bytes(b.rows, b.kb());
        t.ga = (const uint32_t*)workspace;
        t.gb = (const uint32_t*)((const char*)workspace + na);
        hipLaunchKernelGGL(mx4_scale_groups_kernel, dim3((uint32_t)(((na + nb) / 4 + kNT - 1) / kNT)), dim3(kNT), 0,
                           stream, a, b, (uint32_t*)t.ga, (uint32_t*)t.gb, (int64_t)na / 4, (int64_t)nb / 4);
        return by_dtype(out.dtype, [&](auto dt) {
            constexpr int bytes = kStages * (kStageBytes + kScaleBytes);
            static_assert(bytes <= 160 * 1024, "LDS of a compute unit");
            auto kernel = mx4_tile_kernel<decltype(dt)::value>;
            (void)hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
            hipLaunchKernelGGL(kernel, dim3((uint32_t)(t.m_tiles * t.n_tiles)), dim3(kTNT), bytes, stream, t);
        });
    }
    // waves split k where 128 x 128 tiles leave compute units idle and there
    // are steps to split
    const int64_t big = ((a.rows + 127) / 128) * ((b.rows + 127) / 128);
    const bool split = big < 256 && a.cols > 256;
    const int64_t T = split ? 64 : 128;
    const int64_t mt = (a.rows + T - 1) / T, nt = (b.rows + T - 1) / T;
    return by_dtype(out.dtype, [&](auto dt) {
        if (split)
            hipLaunchKernelGGL((mx4_direct_kernel<decltype(dt)::value, 4>), dim3((uint32_t)(mt * nt)), dim3(kNT), 0, stream,
                               a, b, out, (int)nt);
        else
            hipLaunchKernelGGL((mx4_direct_kernel<decltype(dt)::value, 1>), dim3((uint32_t)(mt * nt)), dim3(kNT), 0, stream,
                               a, b, out, (int)nt);
    });
}

}  // namespace iqlh
