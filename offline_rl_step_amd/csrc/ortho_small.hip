// Orthogonalised updates of matrices that fit into the LDS of a compute unit: one
// workgroup a matrix takes it through the whole step, norm, momentum, all products and the
// weights, in one launch.  (Formulas and operands as in ortho.hip.)
//
// X [rows][cols] and S = X X^T, then b S + c S S, lie in LDS as binary16 in one or two
// planes.  Eight waves take 64 x 32 outputs each at a time, with a matrix's fragments read
// straight from LDS: rows as they are, columns by the transposing read, from the same
// place.  Bound by one compute unit's matrix instructions (15 products of 128^3 in two planes 19 us at
// 2.4 GHz, in one 6.4): a product is 3.4 us, of which 1.3 are theirs, the rest reads, barriers and results.
// Four matrices of 128 x 128 among a step's list: 71 us, with a launch a product 97.
#include "iqlher.h"
#include "launch.hpp"
#include "ortho_block.hpp"
#include "tile16.hpp"

namespace iqlh {

namespace {

constexpr int kNT = 512, kWaves = kNT / 64;
constexpr int kTiles = 3;                 // most outputs of 64 x 32 a wave
constexpr int kMostElements = kTiles * kWaves * 2048;

// Chunks of 16 bytes of a row in LDS, a multiple of 16; chunk c of row r lies at c ^ place_mix(r), so that
// both 16 rows' reads of one chunk and the transposing reads of 4 rows fall on all banks
__host__ __device__ inline int row_chunks(int planes, int cols_pad) { return (planes * cols_pad / 8 + 15) / 16 * 16; }
IQLH_DEV int place_mix(int r) { return (r & 3) << 2 | (r >> 2 & 3); }

template <int PL>
struct Matrix {
    uint8_t* p;
    int chunks;  // of a row
    IQLH_DEV uint8_t* chunk(int r, int c) const { return p + (r * chunks + (c ^ place_mix(r))) * 16; }
    // chunk of column col (a multiple of 8) and plane
    static IQLH_DEV int at(int col, int plane) { return PL == 2 ? col / 32 * 8 + (col & 31) / 8 + 4 * plane : col / 8; }
    // fragment of 32 i from i0, 16 k from k0: element (i, k) in row i
    IQLH_DEV uint4 rows(int i0, int k0, int plane) const {
        const int lane = threadIdx.x & 63;
        return *(const uint4*)chunk(i0 + (lane & 31), at(k0 + 8 * (lane >> 5), plane));
    }
    // element (i, k) in column i of row k
    IQLH_DEV uint4 cols(int i0, int k0, int plane) const {
        typedef short s4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s4 lds_s4;
        const int lane = threadIdx.x & 63, li = lane & 15, half = lane >> 4 & 1, h = lane >> 5;
        const int k = k0 + 8 * h + (li >> 2), c = at(i0 + 16 * half, plane) + ((li & 3) >> 1);
        const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(chunk(k, c) + 8 * (li & 1)));
        const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(chunk(k + 4, c) + 8 * (li & 1)));
        const uint2 l = __builtin_bit_cast(uint2, lo), u = __builtin_bit_cast(uint2, hi);
        return uint4{l.x, l.y, u.x, u.y};
    }
    // four neighbouring elements of row r from column col (a multiple of 4) on
    IQLH_DEV void get4(int r, int col, float (&v)[4]) const {
        const int c = col & ~7, half = (col & 4) * 2;
        const uint2 hi = *(const uint2*)(chunk(r, at(c, 0)) + half);
        v[0] = half_of(hi.x, 0), v[1] = half_of(hi.x, 1), v[2] = half_of(hi.y, 0), v[3] = half_of(hi.y, 1);
        if (PL == 2) {
            const uint2 lo = *(const uint2*)(chunk(r, at(c, 1)) + half);
            v[0] += half_of(lo.x, 0), v[1] += half_of(lo.x, 1), v[2] += half_of(lo.y, 0), v[3] += half_of(lo.y, 1);
        }
    }
    IQLH_DEV void put4(int r, int col, const float (&v)[4]) const {
        const int c = col & ~7, half = (col & 4) * 2;
        const uint2 hi = {pack_half(v[0], v[1]), pack_half(v[2], v[3])};
        *(uint2*)(chunk(r, at(c, 0)) + half) = hi;
        if (PL == 2)
            *(uint2*)(chunk(r, at(c, 1)) + half) = uint2{pack_half(v[0] - half_of(hi.x, 0), v[1] - half_of(hi.x, 1)),
                                                        pack_half(v[2] - half_of(hi.y, 0), v[3] - half_of(hi.y, 1))};
    }
};

// One element, and four neighbouring ones of any alignment
IQLH_DEV float load1_of(int dtype, const void* p, int64_t at) {
    if (dtype == IQLH_F32) return ((const float*)p)[at];
    const uint32_t w = ((const uint16_t*)p)[at];
    return dtype == IQLH_BF16 ? brain_of(w, 0) : half_of(w, 0);
}
IQLH_DEV void store1_of(int dtype, void* p, int64_t at, float v) {
    if (dtype == IQLH_F32) ((float*)p)[at] = v;
    else ((uint16_t*)p)[at] = dtype == IQLH_BF16 ? f2bf(v) : (uint16_t)pack_half(v, 0.f);
}
typedef uint32_t u2_a2 __attribute__((ext_vector_type(2), aligned(2)));
IQLH_DEV void load4_of(int dtype, const void* p, int64_t at, float (&v)[4]) {
    if (dtype == IQLH_F32) {
        const u4_a4 w = *(const u4_a4*)((const float*)p + at);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(w[e]);
        return;
    }
    const u2_a2 w = *(const u2_a2*)((const uint16_t*)p + at);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = dtype == IQLH_BF16 ? brain_of(w[e >> 1], e & 1) : half_of(w[e >> 1], e & 1);
}
IQLH_DEV void store4_of(int dtype, void* p, int64_t at, const float (&v)[4]) {
    if (dtype == IQLH_F32) {
        *(u4_a4*)((float*)p + at) = u4_a4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    } else {
        const bool brain = dtype == IQLH_BF16;
        *(u2_a2*)((uint16_t*)p + at) = u2_a2{brain ? pack_bf2(v[0], v[1]) : pack_half(v[0], v[1]),
                                            brain ? pack_bf2(v[2], v[3]) : pack_half(v[2], v[3])};
    }
}

// acc = sum over k < K of a(m, k) b(n, k) for the wave's tiles t = wave, wave + 8, .. of 64 x 32, nt of them along n
template <int PL, bool AC, bool BC>
IQLH_DEV void product(const Matrix<PL>& a, const Matrix<PL>& b, int tiles, int nt, int K, mm_f16 (&acc)[kTiles][2]) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
    for (int f = 0; f < kTiles; ++f) {
        acc[f][0] = mm_f16{};
        acc[f][1] = mm_f16{};
        const int t = wave + kWaves * f;
        if (t >= tiles) continue;
        const int m0 = t / nt * 64, n0 = t % nt * 32;
        struct Frags {
            uint4 x[PL][2], y[PL];
        } g[2];
        auto load = [&](Frags& q, int k) __attribute__((always_inline)) {
#pragma unroll
            for (int p = PL - 1; p >= 0; --p) {
                q.y[p] = BC ? b.cols(n0, k, p) : b.rows(n0, k, p);
#pragma unroll
                for (int i = 0; i < 2; ++i) q.x[p][i] = AC ? a.cols(m0 + 32 * i, k, p) : a.rows(m0 + 32 * i, k, p);
            }
        };
        auto mma = [&](const Frags& q) __attribute__((always_inline)) {
#pragma unroll
            for (int s = PL == 2 ? 0 : 2; s < 3; ++s)  // lo hi, hi lo, hi hi
#pragma unroll
                for (int i = 0; i < 2; ++i) acc[f][i] = mma16<false>(q.y[s == 1], q.x[s == 0][i], acc[f][i]);
        };
        load(g[0], 0);
        for (int k = 0; k < K; k += 32) {  // K is a multiple of 64; the next 16 k's reads before these ones' products
            load(g[1], k + 16);
            __builtin_amdgcn_sched_barrier(0);
            mma(g[0]);
            __builtin_amdgcn_sched_barrier(0);
            load(g[0], k + 32 < K ? k + 32 : k);
            __builtin_amdgcn_sched_barrier(0);
            mma(g[1]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// f(row, column, four sums) for the wave's outputs
template <typename F>
IQLH_DEV void each4(int tiles, int nt, mm_f16 (&acc)[kTiles][2], F f) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const int tile = wave + kWaves * t;
        if (tile >= tiles) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = acc[t][i][4 * g + e];
                f(tile / nt * 64 + 32 * i + r, tile % nt * 32 + 8 * g + 4 * h, v);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[t][i][4 * g + e] = v[e];
            }
    }
}

template <int PL>
IQLH_DEV void small_step(const OrthoArgs& a, const OrthoMat& q, uint8_t* lds) {
    __shared__ double red[kWaves];
    const Matrix<PL> X{lds, row_chunks(PL, q.cols_pad)}, S{lds + q.rows_pad * X.chunks * 16, row_chunks(PL, q.k_pad)};
    const int gc = q.cols_pad / 8, groups = q.rows_pad * gc;
    // f(row, column, elements in the row, eight elements of the update, of the momentum behind it), for every group of eight; in
    // batches whose loads are made together.  Called twice, since the update would not stay in registers.
    constexpr int BATCH = 4;
    auto each8 = [&](auto f) __attribute__((always_inline)) {
        for (int e0 = threadIdx.x; e0 < groups; e0 += BATCH * kNT) {
            float u[BATCH][8], m[BATCH][8];
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const int e = e0 + j * kNT, row = e / gc, col = 8 * (e - row * gc), n = row < q.rows ? q.cols - col : 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) u[j][i] = 0.f;
                if (n <= 0) continue;
                load8_of(q.x_dtype, (const void*)q.x, row * q.ld_x + col, n, u[j]);
                if (a.h.step) load8_of(IQLH_F32, (const void*)q.momentum, row * q.ld_momentum + col, n, m[j]);
            }
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const int e = e0 + j * kNT, row = e / gc, col = 8 * (e - row * gc), n = row < q.rows ? q.cols - col : 0;
                if (e >= groups) continue;
                if (a.h.step && n > 0) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        m[j][i] = fmaf(a.h.mu, m[j][i], u[j][i]);
                        u[j][i] = a.h.nesterov ? fmaf(a.h.mu, m[j][i], u[j][i]) : m[j][i];
                    }
                }
                f(row, col, n, u[j], m[j]);
            }
        }
    };
    double sum = 0.0;
    each8([&](int, int, int, const float (&u)[8], const float (&)[8]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fma((double)u[i], (double)u[i], sum);
    });
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) sum += red[i];
    const double norm = sqrt(sum);
    const bool ok = norm < __longlong_as_double(0x7FF0000000000000ll);
    if (!ok) {  // the weights and the momentum stay; results are NaN
        if (threadIdx.x == 0) set_flag(a.h.flags, IQLH_FLAG_NONFINITE_GRAD);
        if (a.h.step) return;
    }
    const int small_by = ok ? ortho_exponent(norm, a.h.eps) : 0;
    const double scale = ok ? ldexp((double)kUp / (norm + a.h.eps), small_by) : 0.0;
    each8([&](int row, int col, int n, const float (&u)[8], const float (&m)[8]) __attribute__((always_inline)) {
        if (a.h.step && n > 0) store8_of(IQLH_F32, (void*)q.momentum, row * q.ld_momentum + col, n, m);
        float lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = (float)((double)u[i] * scale);
            hi[i] = (float)((double)u[4 + i] * scale);
        }
        X.put4(row, col, lo);
        X.put4(row, col + 4, hi);
    });
    __syncthreads();
    const bool tall = q.rows > q.cols;
    const int nts = q.k_pad / 32, ts = q.k_pad / 64 * nts, ntx = q.cols_pad / 32, tx = q.rows_pad / 64 * ntx;
    mm_f16 acc[kTiles][2];
    for (int s = 0; s < a.h.steps; ++s) {
        // X' = 2^(e' - e) (a X + 2^-2e S X) of X, S and X' as they are held
        const int e0 = ortho_exponent_at(small_by, s), e1 = s + 1 < a.h.steps ? ortho_exponent_at(small_by, s + 1) : 0;
        const float of_poly = ldexpf(kC * kDown, -2 * e0), of_sum = ldexpf(kDown, e1 - 3 * e0), of_own = ldexpf(kA, e1 - e0);
        if (tall) product<PL, true, true>(X, X, ts, nts, q.rows_pad, acc);
        else product<PL, false, false>(X, X, ts, nts, q.cols_pad, acc);
        each4(ts, nts, acc, [&](int m, int n, float (&v)[4]) __attribute__((always_inline)) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] *= kDown;
            S.put4(m, n, v);
        });
        __syncthreads();
        product<PL, false, false>(S, S, ts, nts, q.k_pad, acc);
        each4(ts, nts, acc, [&](int m, int n, float (&v)[4]) __attribute__((always_inline)) {
            float own[4];
            S.get4(m, n, own);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = fmaf(kB, own[e], of_poly * v[e]);
        });
        __syncthreads();  // S is read
        each4(ts, nts, acc, [&](int m, int n, float (&v)[4]) __attribute__((always_inline)) { S.put4(m, n, v); });
        __syncthreads();
        if (tall) product<PL, false, false>(X, S, tx, ntx, q.k_pad, acc);
        else product<PL, false, true>(S, X, tx, ntx, q.k_pad, acc);
        each4(tx, ntx, acc, [&](int m, int n, float (&v)[4]) __attribute__((always_inline)) {
            float own[4];
            X.get4(m, n, own);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = fmaf(of_own, own[e], of_sum * v[e]);
        });
        if (s + 1 == a.h.steps) break;
        __syncthreads();  // X is read
        each4(tx, ntx, acc, [&](int m, int n, float (&v)[4]) __attribute__((always_inline)) { X.put4(m, n, v); });
        __syncthreads();
    }
    const float rate = a.h.step ? (float)(a.h.lr * ortho_shape(q.rows, q.cols, a.h.scale)) : 0.f;
    each4(tx, ntx, acc, [&](int m, int n, float (&v)[4]) __attribute__((always_inline)) {
        if (m >= q.rows || n >= q.cols) return;
        const int64_t at = m * q.ld_out + n;
        const bool four = n + 4 <= q.cols;
        float old[4] = {0.f, 0.f, 0.f, 0.f}, y[4];
        if (a.h.step) {
            if (four) load4_of(q.out_dtype, (const void*)q.out, at, old);
            else
                for (int e = 0; n + e < q.cols; ++e) old[e] = load1_of(q.out_dtype, (const void*)q.out, at + e);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[e] = ok ? v[e] * kDown : __uint_as_float(0x7FC00000u);
            if (a.h.step) y[e] = ortho_weight(old[e], y[e], rate, a.h.decay);
        }
        if (four) store4_of(q.out_dtype, (void*)q.out, at, y);
        else
            for (int e = 0; n + e < q.cols; ++e) store1_of(q.out_dtype, (void*)q.out, at + e, y[e]);
    });
}

__global__ __launch_bounds__(kNT, 2) void ortho_small_kernel(OrthoArgs a) {
    extern __shared__ __align__(16) uint8_t lds[];
    const OrthoMat& q = a.mats[a.small[blockIdx.x].mat];
    if (q.planes == 2) small_step<2>(a, q, lds);
    else small_step<1>(a, q, lds);
}

}  // namespace

int64_t ortho_small_bytes(int32_t rows_pad, int32_t cols_pad, int32_t k_pad, int32_t planes) {
    return (int64_t)rows_pad * row_chunks(planes, cols_pad) * 16 + (int64_t)k_pad * row_chunks(planes, k_pad) * 16;
}
// 158 KB: what the sums take is in LDS too
constexpr int kMostBytes = 158 << 10;
bool ortho_small_ok(int32_t rows_pad, int32_t cols_pad, int32_t k_pad, int32_t planes) {
    return (int64_t)rows_pad * cols_pad <= kMostElements && (int64_t)k_pad * k_pad <= kMostElements &&
           ortho_small_bytes(rows_pad, cols_pad, k_pad, planes) <= kMostBytes;
}

hipError_t launch_ortho_small(const OrthoArgs& a, hipStream_t stream) {
    (void)hipFuncSetAttribute((const void*)ortho_small_kernel, hipFuncAttributeMaxDynamicSharedMemorySize, kMostBytes);
    hipLaunchKernelGGL(ortho_small_kernel, dim3(a.nsmall), dim3(kNT), a.small_bytes, stream, a);
    return hipGetLastError();
}

}  // namespace iqlh
