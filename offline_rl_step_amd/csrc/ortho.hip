// Orthogonalised updates of a list of weight matrices.
//
// For an update U [rows, cols] of the list, with X = U / (|U|_F + eps):
//   steps times   A = X X^T,   X <- a X + (b A + c A A) X       (X X^T on the smaller side)
// with (a, b, c) = (3.4445, -4.7750, 2.0315): every singular value s of X goes to p(s) = a s + b
// s^3 + c s^5, which five times over takes all but the smallest of (0, 1] into about [0.68, 1.2], so
// that X tends to U V^T of U = U S V^T.  With momentum the list's weights are updated by it:
//   m <- mu m + g,   U = g + mu m (Nesterov) or m,   w <- (1 - lr wd) w - lr s X.
//
// Launches, each over all matrices of the list: norms, normalisation (and momentum), then
// three products a step.  A and b A + c A A are symmetric: tiles on and below the
// diagonal only, each stored in both places, half the matrix instructions.
//
// Operands are binary16 times 2^13, not bfloat16: |X| <= 1.2025 (p's maximum on [0, 1], and p maps [0,
// 1.2025] into itself), |A| <= 1.45 and |b A + c A A| <= 2.81 bound every element, so binary16 holds
// them with three bits more than bfloat16 and down to 2^-27 at full length.  Where |U| is below eps, X, A and the
// polynomial are held times 2^e, 2^2e and 2^2e, with e from the norm and the step alone (ortho_exponent_at): 2^e |X| <= 1
// then, and |b A + c 2^-2e A A| <= 4.8.  Matrices
// whose result is binary32 or binary16 are held in two planes (tile16.hpp), 22 bits.
// p's slope at 0 is a: an error in a small singular value's direction grows up to a^5 = 485 times
// with the value itself, which is what one plane of 11 bits leaves at about 1e-3 of the result
// and two at 1e-6.
//
// Bound by the products: 8192 x 8192 in one plane 990 to 1020 us for X's (1.1 PF), 670 to 700 and 725 to 745 for the
// symmetric ones, whose 528 tiles are three rounds of 256 compute units for 2.06; four of 1024 x 1024 and three of width
// 4096 in two planes 109, 63 and 114 to 128.  Small lists by what a launch and a tile's start and results take, 9 to 11 us a
// product of 512 x 512 x 256.  Norm and start move 12 and 6 (planes: 8) bytes an element at the copy's rate.
#include "iqlher.h"
#include "launch.hpp"
#include "ortho_block.hpp"
#include "tile16.hpp"

namespace iqlh {

namespace {

constexpr int kNT = 256;

// Eight neighbouring elements of the update, and the momentum behind it
IQLH_DEV void update8(const OrthoMat& q, const OrthoHyper& h, int64_t row, int col, float (&u)[8], float (&m)[8]) {
    const int n = q.cols - col;
    load8_of(q.x_dtype, (const void*)q.x, row * q.ld_x + col, n, u);
    if (!h.step) return;
    load8_of(IQLH_F32, (const void*)q.momentum, row * q.ld_momentum + col, n, m);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m[i] = fmaf(h.mu, m[i], u[i]);
        u[i] = h.nesterov ? fmaf(h.mu, m[i], u[i]) : m[i];
    }
}

// Sum of squares of a unit (unit_rows rows of a matrix)
__global__ __launch_bounds__(kNT) void ortho_norm_kernel(OrthoArgs a) {
    __shared__ double red[kNT / kWave];
    const OrthoTile w = a.units[blockIdx.x];
    const OrthoMat& q = a.mats[w.mat];
    const int row0 = w.m * q.unit_rows, rows = q.rows - row0 < q.unit_rows ? q.rows - row0 : q.unit_rows;
    const int groups = (q.cols + 7) / 8;
    double s0 = 0.0, s1 = 0.0;
    for (int e = threadIdx.x; e < rows * groups; e += kNT) {
        const int row = e / groups, col = 8 * (e - row * groups);
        float u[8], m[8];
        update8(q, a.h, row0 + row, col, u, m);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {  // elements behind the row's end are 0
            s0 = fma((double)u[i], (double)u[i], s0);
            s1 = fma((double)u[i + 1], (double)u[i + 1], s1);
        }
    }
    s0 = block_sum64<kNT>(s0 + s1, red);
    if (threadIdx.x == 0) a.part[blockIdx.x] = s0;
}

// X of a unit, zeros in the padding, and the momentum
__global__ __launch_bounds__(kNT) void ortho_start_kernel(OrthoArgs a) {
    __shared__ double red[kNT / kWave];
    const OrthoTile w = a.units[blockIdx.x];
    const OrthoMat& q = a.mats[w.mat];
    double sum = 0.0;
    for (int i = threadIdx.x; i < q.units; i += kNT) sum += a.part[q.unit0 + i];
    const double norm = sqrt(block_sum64<kNT>(sum, red));
    const bool ok = norm < __longlong_as_double(0x7FF0000000000000ll);
    if (w.m == 0 && threadIdx.x == 0) {
        a.small_by[w.mat] = ok ? ortho_exponent(norm, a.h.eps) : -1;
        if (!ok) set_flag(a.h.flags, IQLH_FLAG_NONFINITE_GRAD);
    }
    const double scale = ok ? ldexp((double)kUp / (norm + a.h.eps), ortho_exponent(norm, a.h.eps)) : 0.0;
    const int row0 = w.m * q.unit_rows, rows = q.rows_pad - row0 < q.unit_rows ? q.rows_pad - row0 : q.unit_rows;
    const int groups = q.cols_pad / 8;
    uint16_t* x = (uint16_t*)(a.base + q.x_at[0]);
    for (int e = threadIdx.x; e < rows * groups; e += kNT) {
        const int row = row0 + e / groups, col = 8 * (e % groups);
        float u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, m[8];
        if (ok && row < q.rows && col < q.cols) {
            update8(q, a.h, row, col, u, m);
            if (a.h.step) store8_of(IQLH_F32, (void*)q.momentum, row * q.ld_momentum + col, q.cols - col, m);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = (float)((double)u[i] * scale);
        }
        put_planes(x, row, q.cols_pad, col, q.planes == 2, u);
    }
}

// X X^T and the polynomial of it (kGram, kPoly): symmetric, tiles m >= n.
// kApply: the next X.  kLast: the result.
enum { kGram, kPoly, kApply, kLast };
template <int TILE, int PHASE, int STEPS>
__global__ __launch_bounds__(Tile16<TILE>::NT, (Tile16<TILE, 1, STEPS>::PER_SIMD)) void ortho_product_kernel(OrthoArgs a, int step) {
    typedef Tile16<TILE, 1, STEPS> T;
    extern __shared__ __align__(16) uint8_t lds[];
    const OrthoTile w = (PHASE <= kPoly ? a.sym : a.rect)[blockIdx.x];
    const OrthoMat& q = a.mats[w.mat];
    const int from = step & 1, small_by = a.small_by[w.mat];
    const bool two = q.planes == 2, tall = q.rows > q.cols;
    const int64_t m0 = (int64_t)w.m * TILE, n0 = (int64_t)w.n * TILE;
    const uint16_t* x = (const uint16_t*)(a.base + q.x_at[from]);
    uint16_t* gram = (uint16_t*)(a.base + q.gram_at);
    uint16_t* poly = (uint16_t*)(a.base + q.poly_at);
    mm_f16 acc[T::FA][T::FB];
    auto product = [&](auto planes) __attribute__((always_inline)) {
        constexpr int PL = decltype(planes)::value;
        if (PHASE == kGram) {
            const Side16 s{x, 0, q.cols_pad, q.k_pad};
            if (tall) tile_product<false, TILE, true, true, PL, STEPS>(s, s, m0, n0, 0, q.rows_pad, false, lds, acc);
            else tile_product<false, TILE, false, false, PL, STEPS>(s, s, m0, n0, 0, q.cols_pad, false, lds, acc);
        } else if (PHASE == kPoly) {
            const Side16 s{gram, 0, q.k_pad, q.k_pad};
            tile_product<false, TILE, false, false, PL, STEPS>(s, s, m0, n0, 0, q.k_pad, false, lds, acc);
        } else {
            const Side16 p{poly, 0, q.k_pad, q.k_pad};
            if (tall) tile_product<false, TILE, false, false, PL, STEPS>(Side16{x, 0, q.cols_pad, q.rows_pad}, p, m0, n0, 0, q.k_pad, false, lds, acc);
            else tile_product<false, TILE, false, true, PL, STEPS>(p, Side16{x, 0, q.cols_pad, q.cols_pad}, m0, n0, 0, q.k_pad, false, lds, acc);
        }
    };
    if (two) product(std::integral_constant<int, 2>());
    else product(std::integral_constant<int, 1>());
    const int rows = PHASE <= kPoly ? q.k_pad : q.rows_pad, cols = PHASE <= kPoly ? q.k_pad : q.cols_pad;
    const bool ok = small_by >= 0;
    // X' = 2^(e' - e) (a X + 2^-2e S X) of X, S and X' as they are held
    const int e = ortho_exponent_at(small_by, step), e_next = PHASE == kLast ? 0 : ortho_exponent_at(small_by, step + 1);
    const float of_sum = PHASE == kGram ? kDown : ldexpf(PHASE == kPoly ? kC * kDown : kDown, (PHASE == kPoly ? -2 : -3) * e + e_next);
    const float of_own = PHASE == kPoly ? kB : ldexpf(kA, e_next - e);
    float rate = 0.f;
    if (PHASE == kLast) {
        if (a.h.step) {
            if (!ok) return;
            rate = (float)(a.h.lr * ortho_shape(q.rows, q.cols, a.h.scale));
        }
    }
    // What is combined with the sums: the element's own row of X X^T or X, and in a step the old weights.  All
    // of a batch's loads are made before its first use, so that their time is paid once.
    constexpr int BATCH = 4;
    struct Own {
        uint4 hi, lo;
        float old[8];
    };
    const uint16_t* own = PHASE == kPoly ? gram : x;
    const int own_ld = PHASE == kPoly ? q.k_pad : q.cols_pad;
    auto fetch = [&](int m, int n, Own& o) __attribute__((always_inline)) {
        if (PHASE == kGram) return;
        const uint16_t* p = own + (two ? planes_at(m, own_ld, n) : (int64_t)m * own_ld + n);
        o.hi = *(const uint4*)p;
        o.lo = two ? *(const uint4*)(p + 32) : uint4{0u, 0u, 0u, 0u};
        if (PHASE == kLast && a.h.step && m < q.rows && n < q.cols)
            load8_of(q.out_dtype, (const void*)q.out, (int64_t)m * q.ld_out + n, q.cols - n, o.old);
    };
    // eight neighbouring sums v of row m from column n on, as they are stored
    auto put = [&](int m, int n, const float (&v)[8], const Own& o) __attribute__((always_inline)) {
        float y[8];
        const uint32_t hw[4] = {o.hi.x, o.hi.y, o.hi.z, o.hi.w}, lw[4] = {o.lo.x, o.lo.y, o.lo.z, o.lo.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = v[i] * of_sum;
            const float e = PHASE == kGram ? 0.f : half_of(hw[i >> 1], i & 1) + half_of(lw[i >> 1], i & 1);
            y[i] = PHASE == kGram ? s : fmaf(of_own, e, s);
        }
        if (PHASE == kGram) put_planes(gram, m, q.k_pad, n, two, y);
        if (PHASE == kPoly) put_planes(poly, m, q.k_pad, n, two, y);
        if (PHASE == kApply) put_planes((uint16_t*)(a.base + q.x_at[from ^ 1]), m, q.cols_pad, n, two, y);
        if (PHASE == kLast && m < q.rows && n < q.cols) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[i] = ok ? y[i] * kDown : __uint_as_float(0x7FC00000u);
                if (a.h.step) y[i] = ortho_weight(o.old[i], y[i], rate, a.h.decay);
            }
            store8_of(q.out_dtype, (void*)q.out, (int64_t)m * q.ld_out + n, q.cols - n, y);
        }
    };
#pragma unroll
    for (int band = 0; band < T::BANDS; ++band) {
        stage_band<TILE>(acc, lds, band);
        const int mb = (int)m0 + band * T::BAND;
        constexpr int UNITS = T::BAND * (TILE / 8);
        for (int c0 = threadIdx.x; c0 < UNITS; c0 += BATCH * T::NT) {
            Own o[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int c = c0 + k * T::NT, m = mb + c / (TILE / 8), n = (int)n0 + 8 * (c % (TILE / 8));
                if (c < UNITS && m < rows && n < cols) fetch(m, n, o[k]);
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int c = c0 + k * T::NT, row = c / (TILE / 8), u = c % (TILE / 8), m = mb + row, n = (int)n0 + 8 * u;
                if (c >= UNITS || m >= rows || n >= cols) continue;
                const float4 lo = *stage_at<TILE>(lds, row, 2 * u), hi = *stage_at<TILE>(lds, row, 2 * u + 1);
                const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                put(m, n, v, o[k]);
            }
        }
        if (PHASE <= kPoly && w.m != w.n) {  // and in the mirrored place
            for (int c0 = threadIdx.x; c0 < UNITS; c0 += BATCH * T::NT) {
                Own o[BATCH];
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int c = c0 + k * T::NT, m = mb + 8 * (c % (T::BAND / 8)), n = (int)n0 + c / (T::BAND / 8);
                    if (c < UNITS && m < rows && n < cols) fetch(n, m, o[k]);
                }
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int c = c0 + k * T::NT, u = c % (T::BAND / 8), col = c / (T::BAND / 8), m = mb + 8 * u, n = (int)n0 + col;
                    if (c >= UNITS || m >= rows || n >= cols) continue;
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = ((const float*)stage_at<TILE>(lds, 8 * u + i, col / 4))[col & 3];
                    put(n, m, v, o[k]);
                }
            }
        }
    }
}

template <int PHASE>
hipError_t launch_product(const OrthoArgs& a, int step, hipStream_t stream) {
    const int n = PHASE <= kPoly ? a.nsym : a.nrect;
    auto launch = [&](auto tile, auto steps) {
        typedef Tile16<decltype(tile)::value, 1, decltype(steps)::value> T;
        auto kernel = ortho_product_kernel<decltype(tile)::value, PHASE, decltype(steps)::value>;
        (void)hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, T::LDS);
        hipLaunchKernelGGL(kernel, dim3(n), dim3(T::NT), T::LDS, stream, a, step);
    };
    typedef std::integral_constant<int, 2> Two;
    typedef std::integral_constant<int, 4> Four;
    const int tile = PHASE <= kPoly ? a.sym_tile : a.rect_tile;
    if (tile == 256) launch(std::integral_constant<int, 256>(), Two());
    else if (tile == 64) launch(std::integral_constant<int, 64>(), Four());
    else if (n <= 256) launch(std::integral_constant<int, 128>(), Four());
    else launch(std::integral_constant<int, 128>(), Two());
    return hipGetLastError();
}

}  // namespace

hipError_t launch_orthogonalize(const OrthoArgs& a, hipStream_t stream) {
    if (a.nsmall) {
        const hipError_t e = launch_ortho_small(a, stream);
        if (e != hipSuccess || !a.nunits) return e;
    }
    hipLaunchKernelGGL(ortho_norm_kernel, dim3(a.nunits), dim3(kNT), 0, stream, a);
    hipLaunchKernelGGL(ortho_start_kernel, dim3(a.nunits), dim3(kNT), 0, stream, a);
    hipError_t e = hipGetLastError();
    for (int s = 0; s < a.h.steps && e == hipSuccess; ++s) {
        e = launch_product<kGram>(a, s, stream);
        if (e == hipSuccess) e = launch_product<kPoly>(a, s, stream);
        if (e == hipSuccess) e = s + 1 < a.h.steps ? launch_product<kApply>(a, s, stream) : launch_product<kLast>(a, s, stream);
    }
    return e;
}

}  // namespace iqlh
