// Loss of a policy over many actions: softmax cross entropy of a linear head, with
// its gradients, without the logits in memory.
//
//   z = H W^T + b,  lse_r = log sum_v exp z_rv,  nll_r = lse_r - z_{r, a_r},
//   loss = s sum_r w_r nll_r,  G_rv = s w_r (exp(z_rv - lse_r) - [v = a_r]),
//   dH = G W,  dW = G^T H,  db = column sums of G.
//
// Loss: tiles of z on the matrix instructions; a tile leaves the maximum and the sum of
// exponentials of each of its rows (8 bytes for 128 or 256 logits), which a second
// launch joins.  Gradients: for one piece of the actions after another, the
// tiles of z again, now with lse known, leave G in 16 bits (a piece is chosen so that it
// stays in the Infinity Cache), and two products read it: dW of the piece, and
// dH summed over the pieces in binary32.
//
// Bfloat16 inputs: G is bfloat16.  Binary16 inputs: G is binary16 times a power of
// two by the largest |w|: 11 bits down to p |w| of 2^-27 of that, 0 below 2^-38.
//
// Binary32 inputs: H, W and G are two planes of binary16 each (tile16.hpp) behind a power of two that takes
// the largest of what shares it to [2^13, 2^14): 22 bits for what is within 2^-17 of that largest, and to 2^-38 of
// it below.  What is not summed together, or can be moved to the other side of the product, shares none.  With
// c_d the largest |W_vd| of a column, without the actions that are forbidden, as powers of two all of them:
//   z = sum_d (H_rd c_d) (W_vd / c_d)      a factor for each row and each action,
//   dH = sum_v G_rv W_vd                   for each row of G (by |w_r|) and each column of W,
//   dW = sum_r (G_rv / |w_r|) (H_rd |w_r|) for each column of H |w|, G as for dH.
// One factor for a matrix lost all bits of a column that another is 2^30 times as large as.
//
// Bound by the products, the logits' twice: 8192 x 65536 x 2048 bf16 7.1 ms, 1.17 to 1.26 PF each; 16384 x 32768 x
// 512 bf16, loss alone, 0.51 to 0.58 ms, 0.95 to 1.08 PF; 4096 x 16384 x 512 fp32 0.85 to 0.89 ms, 0.9 to 1.1 PF of binary16
// products, and 85 us for columns' magnitudes and planes.  What is not a product else: copies of rows that are not whole 16-byte
// chunks, 18 of 116 us at 777 x 10007 x 501.
#include "policy_block.hpp"

namespace iqlh {

using namespace policy;

namespace {

// Magnitude of x: b with |x| in [2^(b - 1), 2^b), subnormal ones as 2^-126; kNoBits for 0 and what is not finite
constexpr int kNoBits = -100000, kTop = 14;  // kTop: magnitude of the largest element in planes
IQLH_DEV int bits_of(float x) {
    const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
    return b == 0u || b >= 0x7F800000u ? kNoBits : b >> 23 ? (int)(b >> 23) - 126 : -125;
}
IQLH_DEV int or_zero(int bits) { return bits < -1000 ? 0 : bits; }  // of nothing but zeros: any power of two will do
// Of a row's weight, or the largest: 2^(kTop - b) is a normal binary32 number, as its inverse is
IQLH_DEV int weight_bits(int bits) { return or_zero(bits) < kTop - 126 ? kTop - 126 : or_zero(bits); }
IQLH_DEV int weight_bits(const float* row_weights, int64_t m) { return row_weights ? weight_bits(bits_of(row_weights[m])) : 1; }

// ------------------------------------------------------------ preparation
IQLH_DEV int wave_imax(int v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const int b = __shfl_xor(v, o, kWave);
        v = b > v ? b : v;
    }
    return v;
}

// Row and group of 8 columns of element group at + i (i below 2^30), `at` the same for the workgroup: one
// division of 64 bits for all of it
struct Place {
    int64_t row;
    int group;
};
IQLH_DEV Place place_of(int64_t at, int i, int groups) {
    const int64_t row = at / groups;
    const uint32_t g = (uint32_t)(at - row * groups) + (uint32_t)i, r = g / (uint32_t)groups;
    return Place{row + r, (int)(g - r * (uint32_t)groups)};
}

// Magnitude of the largest weight of a row that is on, of kAbsBlocks workgroups each
__global__ __launch_bounds__(kNT) void policy_weights_kernel(const int32_t* taken, const float* row_weights, int64_t rows, int64_t actions,
                                                             int32_t* part) {
    __shared__ int red[kNT / kWave];
    int top = kNoBits;
    for (int64_t m = (int64_t)blockIdx.x * kNT + threadIdx.x; m < rows; m += (int64_t)kAbsBlocks * kNT) {
        const int b = row_off(taken, row_weights, actions, m) ? kNoBits : bits_of(row_weights[m]);
        top = b > top ? b : top;
    }
    top = wave_imax(top);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 1; i < kNT / kWave; ++i) top = red[i] > top ? red[i] : top;
        part[blockIdx.x] = top;
    }
}

// An action that is never taken: 2^(its bias in bits) is 0
IQLH_DEV bool forbidden(const float* bias, int64_t v) { return bias && bias[v] * kLog2e == kNone; }

// Empty columns for policy_columns_kernel; and (part) whether a forbidden action was taken all the same in a row that is
// on, of each wave of kStartBlocks workgroups
constexpr int kStartBlocks = 64, kStartWaves = kStartBlocks * kNT / kWave;
static_assert(kStartWaves <= kAbsBlocks, "their place in the workspace");
struct StartArgs {
    int32_t* cols;
    int n_cols;
    int32_t* part;  // [kStartWaves], or null
    const int32_t* taken;
    const float *row_weights, *bias;
    int64_t rows, actions;
};
__global__ __launch_bounds__(kNT) void policy_start_kernel(StartArgs a) {
    const int64_t first = (int64_t)blockIdx.x * kNT + threadIdx.x, step = (int64_t)gridDim.x * kNT;
    for (int64_t i = first; i < a.n_cols; i += step) a.cols[i] = kNoBits;
    if (!a.part) return;
    bool any = false;
    constexpr int AHEAD = 8;
    for (int64_t m0 = first; m0 < a.rows; m0 += AHEAD * step) {
        int32_t t[AHEAD];
        bool on[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {  // behind the end: the first row again
            const int64_t m = m0 + k * step < a.rows ? m0 + k * step : m0;
            const float w = a.row_weights ? a.row_weights[m] : 1.f;
            t[k] = a.taken[m];
            on[k] = t[k] >= 0 && t[k] < a.actions && w != 0.f;
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) any |= on[k] & forbidden(a.bias, on[k] ? t[k] : 0);
    }
    any = __any(any);
    if ((threadIdx.x & 63) == 0) a.part[first / kWave] = any;
}
// Of a whole wave: bias, or null where forbidden actions count as others do, one of them being taken
IQLH_DEV const float* bias_that_forbids(const float* bias, const int32_t* part) {
    if (!bias || !part) return bias;
    int any = 0;
#pragma unroll
    for (int i = 0; i < kStartWaves; i += kWave) any |= part[i + (threadIdx.x & 63)];
    return __any(any) ? nullptr : bias;
}

// Magnitudes of the columns of hidden (blockIdx.z 0; its rows' weights times them, rows that are off left out) and of
// the head's weights (1; forbidden actions left out), binary32: 8 `lanes` columns a workgroup, each lane 8 of every
// (gridDim.x kNT / lanes)-th row.  gridDim.x above 1: columns that policy_start_kernel left.
struct ColumnArgs {
    PolicyMat m[2];
    int32_t* to[2];
    const int32_t* taken;
    const float *row_weights, *bias;
    const int32_t* part;  // of policy_start_kernel, or null
    int64_t actions, ld;
    int lanes;
};
__global__ __launch_bounds__(kNT) void policy_columns_kernel(ColumnArgs a) {
    constexpr int AHEAD = 8;
    __shared__ int red[kNT][8];
    const PolicyMat& q = a.m[blockIdx.z];
    if (!q.p) return;
    const float* bias = blockIdx.z ? bias_that_forbids(a.bias, a.part) : nullptr;
    const int lane = threadIdx.x % a.lanes, own = threadIdx.x / a.lanes, at_once = kNT / a.lanes;
    const int first = blockIdx.y * 8 * a.lanes, col = first + 8 * lane, n = (int)q.cols - col;
    int top[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) top[i] = kNoBits;
    auto sweep = [&](auto hidden) __attribute__((always_inline)) {
        const int64_t step = (int64_t)gridDim.x * at_once;
        for (int64_t row0 = (int64_t)blockIdx.x * at_once + own; row0 < q.rows; row0 += AHEAD * step) {
            float v[AHEAD][8];
            int32_t t[AHEAD];
            float w[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {  // behind the end: the first row again
                const int64_t row = row0 + k * step < q.rows ? row0 + k * step : row0;
                t[k] = decltype(hidden)::value ? a.taken[row] : 0;
                w[k] = decltype(hidden)::value ? (a.row_weights ? a.row_weights[row] : 1.f) : bias ? bias[row] : 0.f;
                load8_of(IQLH_F32, q.p, row * q.ld + col, n, v[k]);
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const bool off = decltype(hidden)::value ? t[k] < 0 || t[k] >= a.actions || w[k] == 0.f : w[k] * kLog2e == kNone;
                const int add = off ? kNoBits : decltype(hidden)::value ? weight_bits(bits_of(w[k])) : 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int b = bits_of(v[k][i]) + add;
                    top[i] = b > top[i] ? b : top[i];
                }
            }
        }
    };
    if (n > 0) blockIdx.z == 0 ? sweep(std::true_type()) : sweep(std::false_type());
#pragma unroll
    for (int i = 0; i < 8; ++i) red[threadIdx.x][i] = top[i];
    __syncthreads();
    const int c = threadIdx.x;
    if (c < 8 * a.lanes && first + c < a.ld) {
        int t = kNoBits;
        for (int k = 0; k < at_once; ++k) {
            const int b = red[k * a.lanes + c / 8][c % 8];
            t = b > t ? b : t;
        }
        int32_t* to = a.to[blockIdx.z] + first + c;
        if (gridDim.x == 1) *to = t;
        // mostly there already: many workgroups' atomics on one line wait for each other
        else if (t > -1000 && t > __hip_atomic_load(to, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) atomicMax(to, t);
    }
}

// Matrices as operands: rows of whole 64 16-bit elements, zeros behind the end.  Binary32 in two planes: x in row r
// and column d times 2^(kTop + sign cols[d]) and (weighted) the weight's magnitude, or, by rows, times 2^(sign cols[d] -
// row_exp[r]) with row_exp of the row's largest, which is written.
struct Convert {
    PolicyMat m;
    uint16_t* to;             // [rows][ld_to]
    int64_t ld_to;
    const int32_t* cols;      // binary32: [ld_to]
    int32_t* row_exp;         // or null: not by rows
    int sign, zero_off;       // zero_off: zeros in the place of rows that are off; -1: of forbidden actions
    int weighted;
    int lanes, blocks;        // lanes: of a row, a power of two
};
struct ConvertArgs {
    Convert c[4];
    const int32_t* part;         // binary16: [kAbsBlocks], or null
    int32_t* g_top;              // their largest
    const float* bias;           // binary32, or null
    const int32_t* forbid_part;  // of policy_start_kernel, or null
    const int32_t* taken;
    const float* row_weights;
    int64_t actions;
    int dtype;
};
__global__ __launch_bounds__(kNT) void policy_convert_kernel(ConvertArgs a) {
    const int lane = threadIdx.x & 63;
    const bool f32 = a.dtype == IQLH_F32;
    if (a.part && blockIdx.x == 0 && threadIdx.x < kWave) {
        int top = kNoBits;
        for (int i = lane; i < kAbsBlocks; i += kWave) top = a.part[i] > top ? a.part[i] : top;
        top = wave_imax(top);
        if (lane == 0) *a.g_top = weight_bits(top);
    }
    int k = 0, block = blockIdx.x;
    while (k < 3 && block >= a.c[k].blocks) block -= a.c[k++].blocks;
    const Convert& c = a.c[k];
    const PolicyMat& q = c.m;
    if (!q.p) return;
    const int groups = (int)(c.ld_to / 8);
    const float* bias = c.zero_off < 0 ? bias_that_forbids(a.bias, a.forbid_part) : nullptr;
    auto off_row = [&](int64_t row) __attribute__((always_inline)) {
        return c.zero_off < 0 ? forbidden(bias, row) : c.zero_off && row_off(a.taken, a.row_weights, a.actions, row);
    };
    auto fetch = [&](int64_t row, int col, bool off, float (&v)[8]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
        if (row < q.rows && col < q.cols && !off) load8_of(a.dtype, q.p, row * q.ld + col, q.cols - col, v);
    };
    auto column_bits = [&](int col, int (&b)[8]) __attribute__((always_inline)) {
        const int4 x = *(const int4*)(c.cols + col), y = *(const int4*)(c.cols + col + 4);
        b[0] = x.x, b[1] = x.y, b[2] = x.z, b[3] = x.w, b[4] = y.x, b[5] = y.y, b[6] = y.z, b[7] = y.w;
        // what meets nothing but zeros: 0, and of no magnitude (a division of those zeros by any power of two will do)
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = c.sign > 0 ? b[i] : -or_zero(b[i]);
    };
    // times 2^(e + b)
    auto put = [&](int64_t row, int col, float (&v)[8], int e, const int (&b)[8]) __attribute__((always_inline)) {
        if (f32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = ldexpf(v[i], e + b[i]);
            put_planes(c.to, row, c.ld_to, col, true, v);
        } else {
            store8_of(a.dtype, c.to, row * c.ld_to + col, 8, v);
        }
    };
    // By rows: as many lanes a row as it has groups, 64 at most; its largest element, then the planes.  A lane's first
    // elements stay in registers.
    if (c.row_exp) {
        const int lanes = c.lanes, in = lane & (lanes - 1), rows_at_once = kNT / lanes;
        int b0[8];
        column_bits(8 * (in < groups ? in : 0), b0);
        for (int64_t row0 = (int64_t)block * rows_at_once; row0 < q.rows; row0 += (int64_t)c.blocks * rows_at_once) {
            const int64_t row = row0 + threadIdx.x / lanes;
            const bool off = row < q.rows && off_row(row);
            float v0[8];
            fetch(row, 8 * in, off, v0);
            int top = kNoBits;
            auto largest = [&](const float (&v)[8], const int (&b)[8]) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) top = bits_of(v[i]) + b[i] > top ? bits_of(v[i]) + b[i] : top;
            };
            largest(v0, b0);
            for (int g = in + kWave; g < groups; g += kWave) {
                float v[8];
                int b[8];
                fetch(row, 8 * g, off, v);
                column_bits(8 * g, b);
                largest(v, b);
            }
            for (int o = lanes / 2; o > 0; o >>= 1) {
                const int b = __shfl_xor(top, o, kWave);
                top = b > top ? b : top;
            }
            if (row >= q.rows) continue;
            const int e = or_zero(top) - kTop;
            if (in == 0) c.row_exp[row] = e;
            if (in < groups) put(row, 8 * in, v0, -e, b0);
            for (int g = in + kWave; g < groups; g += kWave) {
                float v[8];
                int b[8];
                fetch(row, 8 * g, off, v);
                column_bits(8 * g, b);
                put(row, 8 * g, v, -e, b);
            }
        }
        return;
    }
    constexpr int AHEAD = 4;
    const int64_t total = q.rows * groups;
    if (q.cols < 8) {
        for (int64_t at = (int64_t)block * (AHEAD * kNT) + threadIdx.x; at < total; at += (int64_t)c.blocks * (AHEAD * kNT))
            for (int64_t e = at; e < total && e < at + AHEAD * kNT; e += kNT) {
                const int64_t row = e / groups;
                const int col = 8 * (int)(e - row * groups);
                float v[8];
                int b[8] = {};
                fetch(row, col, off_row(row), v);
                if (f32) column_bits(col, b);
                put(row, col, v, kTop + (c.weighted ? weight_bits(a.row_weights, row) : 0), b);
            }
        return;
    }
    // The loads of AHEAD groups with nothing between them that waits: a row's last group is read from its last 8
    // elements and moved, a row that is off is read too (10007 x 501 and 777 x 501, f16: 11 -> 7 us)
    auto sweep = [&](auto wide) __attribute__((always_inline)) {
        constexpr bool F32 = decltype(wide)::value;
        for (int64_t at = (int64_t)block * (AHEAD * kNT); at < total; at += (int64_t)c.blocks * (AHEAD * kNT)) {
            u4_a2 x[AHEAD];
            u4_a4 y[AHEAD];
            Place p[AHEAD];
            int32_t t[AHEAD];
            float w[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                p[k] = place_of(at, threadIdx.x + k * kNT, groups);
                const int64_t row = p[k].row < q.rows ? p[k].row : q.rows - 1;
                const int64_t from = row * q.ld + (8 * (int64_t)p[k].group < q.cols - 8 ? 8 * p[k].group : q.cols - 8);
                if constexpr (F32) {
                    const u4_a4* s = (const u4_a4*)((const float*)q.p + from);
                    x[k] = s[0], y[k] = s[1];
                } else {
                    x[k] = *(const u4_a2*)((const uint16_t*)q.p + from);
                }
                t[k] = c.zero_off > 0 ? a.taken[row] : 0;
                w[k] = c.zero_off > 0 && a.row_weights ? a.row_weights[row] : bias ? bias[row] : 1.f;
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                if (p[k].row >= q.rows) continue;
                const int64_t past = 8 * (int64_t)p[k].group - (q.cols - 8);
                const int move = past < 0 ? 0 : past > 8 ? 8 : (int)past;
                const bool off = t[k] < 0 || t[k] >= a.actions || (bias ? w[k] * kLog2e == kNone : w[k] == 0.f) || move == 8;
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if constexpr (F32) v[i] = __uint_as_float(i < 4 ? x[k][i] : y[k][i - 4]);
                    else v[i] = a.dtype == IQLH_BF16 ? brain_of(x[k][i >> 1], i & 1) : half_of(x[k][i >> 1], i & 1);
                    v[i] = off ? 0.f : v[i];
                }
#pragma unroll
                for (int o = 4; o > 0; o >>= 1)
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = move & o ? (i + o < 8 ? v[i + o] : 0.f) : v[i];
                int b[8] = {};
                if constexpr (F32) column_bits(8 * p[k].group, b);
                put(p[k].row, 8 * p[k].group, v, kTop + (!F32 || !c.weighted ? 0 : a.row_weights ? weight_bits(bits_of(w[k])) : 1), b);
            }
        }
    };
    f32 ? sweep(std::true_type()) : sweep(std::false_type());
}

// ------------------------------------------------------------------ tiles
// blockIdx -> tile: each XCD takes a run of tiles, walked in columns of 4 tile
// rows, so that its L2 serves a patch of about 4 x 8 tiles at a time
IQLH_DEV void tile_of(int id, int m_tiles, int n_tiles, int& tm, int& tn) {
    const int total = m_tiles * n_tiles;
    const int per = total / 8, rest = total % 8, x = id & 7, k = id >> 3;
    id = x * per + (x < rest ? x : rest) + k;
    const int band = id / (4 * n_tiles), in_band = id - band * 4 * n_tiles;
    const int rows_in = m_tiles - band * 4 < 4 ? m_tiles - band * 4 : 4;
    tm = band * 4 + in_band % rows_in;
    tn = in_band / rows_in;
}

struct LogitArgs {
    Side16 h, w;             // w: of the piece
    const float* bias;       // of the piece, or null
    const int32_t* taken;
    const float* row_weights;  // or null
    const float* lse;
    const int32_t *row_exp, *act_exp;  // binary32: exponents of the sums' rows and columns (of the piece)
    const int32_t* g_top;    // or null: of all weights
    float g_factor;          // of G without either of them
    Soft* part;              // [n_tiles][rows]
    float* z_taken;          // [rows]
    uint16_t* g;             // [rows][ldg], for binary32 in two planes; else a second matrix behind `plane`
    float* db_part;          // [m_tiles][ldg], or null
    int64_t rows, actions, first, ldg, plane;  // actions of the piece; its first one
    int64_t all_actions;
    int64_t k;               // summed elements
    int g_planes, m_tiles, n_tiles;
};

// The logits of a tile, times log2(e).  GRAD false: maxima and sums of its rows, and the taken
// actions' logits.  true: G.
template <bool BRAIN, int TILE, bool GRAD, int PL>
__global__ __launch_bounds__(Tile16<TILE>::NT, Tile16<TILE>::PER_SIMD) void policy_logits_kernel(LogitArgs a) {
    typedef Tile16<TILE, PL> T;
    constexpr int FA = T::FA, FB = T::FB;
    extern __shared__ __align__(16) uint8_t lds[];
    int tm, tn;
    tile_of(blockIdx.x, a.m_tiles, a.n_tiles, tm, tn);
    const int64_t m0 = (int64_t)tm * TILE, n0 = (int64_t)tn * TILE;
    const int there = (int)(a.actions - n0 < TILE ? a.actions - n0 : TILE);  // columns of the tile
    // of the columns: the bias, minus infinity behind the end.  Of the rows: the column of the action
    // taken (or -1), the weight and the lse
    float* col_bias = (float*)(lds + T::RING);
    int* row_col = (int*)(col_bias + TILE);
    float* row_w = (float*)(row_col + TILE);
    float* row_lse = row_w + TILE;
    int* row_exp = (int*)(row_lse + TILE);  // PL 2: exponents of the sums, and what takes G back to its size
    int* col_exp = row_exp + TILE;
    float* row_back = (float*)(col_exp + TILE);
    // (loaded before the product and put there behind it, so that the product does not wait for them)
    const int64_t mine = m0 + (threadIdx.x % TILE), mine_in = mine < a.rows ? mine : a.rows - 1;
    const int32_t t_in = a.taken[mine_in];
    const float b_in = a.bias && (int)(threadIdx.x % TILE) < there ? a.bias[n0 + threadIdx.x % TILE] : 0.f;
    const float w_in = GRAD && a.row_weights ? a.row_weights[mine_in] : 1.f, lse_in = GRAD ? a.lse[mine_in] : 0.f;
    int re_in = 0, ce_in = 0;
    float gf = a.g_factor;
    if constexpr (PL == 2) {
        re_in = a.row_exp[mine_in];
        ce_in = (int)(threadIdx.x % TILE) < there ? a.act_exp[n0 + threadIdx.x % TILE] : 0;
        if (GRAD) gf = ldexpf(1.f, kTop - (a.row_weights ? weight_bits(bits_of(w_in)) : 1));
    } else if (GRAD && a.g_top) {
        gf = ldexpf(1.f, kTop - *a.g_top);
    }
    mm_f16 acc[FA][FB];
    tile_product<BRAIN, TILE, false, false, PL>(a.h, a.w, m0, n0, 0, a.k, false, lds, acc);
    if (threadIdx.x < TILE) {
        const int n = threadIdx.x;
        const bool off = mine >= a.rows || t_in < 0 || t_in >= a.all_actions || w_in == 0.f;
        const int64_t col = t_in - a.first - n0;
        col_bias[n] = n < there ? b_in * kLog2e : kNone;
        row_col[n] = mine < a.rows && col >= 0 && col < there ? (int)col : -1;
        row_w[n] = off ? 0.f : w_in * gf;
        // no logit above minus infinity: no probabilities
        row_lse[n] = off ? __builtin_huge_valf() : lse_in == kNone ? 0.f : lse_in * kLog2e;
        if (PL == 2) row_exp[n] = re_in, col_exp[n] = ce_in;
        if (PL == 2 && GRAD) row_back[n] = 1.f / gf;
    }
    __syncthreads();
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int wm = wave_m<TILE>(), wn = wave_n<TILE>();
    float sub[FA];
    int col[FA], re[FA];
#pragma unroll
    for (int i = 0; i < FA; ++i) {
        const int row = wm + 32 * i + r;
        re[i] = PL == 2 ? row_exp[row] : 0;
        sub[i] = GRAD ? row_lse[row] : 0.f;
        col[i] = row_col[row] - wn;
    }
#pragma unroll
    for (int j = 0; j < FB; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float4 b4 = *(const float4*)(col_bias + wn + 32 * j + 8 * g + 4 * h);
            const float b[4] = {b4.x, b4.y, b4.z, b4.w};
            int ce[4] = {};
            if constexpr (PL == 2) {
                const int4 e4 = *(const int4*)(col_exp + wn + 32 * j + 8 * g + 4 * h);
                ce[0] = e4.x, ce[1] = e4.y, ce[2] = e4.z, ce[3] = e4.w;
            }
#pragma unroll
            for (int i = 0; i < FA; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float z = PL == 2 ? ldexpf(acc[i][j][4 * g + e], re[i] + ce[e]) : acc[i][j][4 * g + e];
                    acc[i][j][4 * g + e] = fmaf(z, kLog2e, GRAD ? b[e] - sub[i] : b[e]);
                }
        }
    if constexpr (!GRAD) {
        Soft(*rows)[T::WN] = (Soft(*)[T::WN])lds;  // [TILE]
#pragma unroll
        for (int i = 0; i < FA; ++i) {
            Soft v{kNone, 0.f};
#pragma unroll
            for (int j = 0; j < FB; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) v.m = fmaxf(v.m, acc[i][j][e]);
            const float top = v.m == kNone ? 0.f : v.m;
#pragma unroll
            for (int j = 0; j < FB; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) v.s += __builtin_amdgcn_exp2f(acc[i][j][e] - top);
            if (__any(col[i] >= 0 && col[i] < 32 * FB)) {
#pragma unroll
                for (int j = 0; j < FB; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (col[i] == 32 * j + 8 * (e >> 2) + 4 * h + (e & 3)) a.z_taken[m0 + wm + 32 * i + r] = acc[i][j][e];
            }
            v = soft_xor(v, 32);
            if (h == 0) rows[wm + 32 * i + r][wn / (32 * FB)] = v;
        }
        __syncthreads();
        if (threadIdx.x < TILE && m0 + threadIdx.x < a.rows) {
            Soft v = rows[threadIdx.x][0];
#pragma unroll
            for (int k = 1; k < T::WN; ++k) v.join(rows[threadIdx.x][k]);
            a.part[(int64_t)tn * a.rows + m0 + threadIdx.x] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < FA; ++i) {
            const float w = row_w[wm + 32 * i + r];
#pragma unroll
            for (int j = 0; j < FB; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = w * __builtin_amdgcn_exp2f(acc[i][j][e]);
            if (__any(w == 0.f)) {  // rows that are off, also where an infinite weight made NaN of their zeros
#pragma unroll
                for (int j = 0; j < FB; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[i][j][e] = w == 0.f ? 0.f : acc[i][j][e];
            }
            if (__any(col[i] >= 0 && col[i] < 32 * FB)) {
#pragma unroll
                for (int j = 0; j < FB; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (col[i] == 32 * j + 8 * (e >> 2) + 4 * h + (e & 3)) acc[i][j][e] -= w;
            }
        }
        if (a.db_part) {  // sums over the tile's rows
            float(*sums)[TILE] = (float(*)[TILE])lds;  // [WM]
            float back[FA];
#pragma unroll
            for (int i = 0; i < FA; ++i) back[i] = PL == 2 ? row_back[wm + 32 * i + r] : 1.f;
#pragma unroll
            for (int jj = 0; jj < FB; jj += 2) {
                float v[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    v[k] = acc[0][jj + k / 16][k % 16] * back[0];
#pragma unroll
                    for (int i = 1; i < FA; ++i) v[k] = fmaf(acc[i][jj + k / 16][k % 16], back[i], v[k]);
                }
                // 32 values of 32 lanes: each exchange halves the values a lane has; lane r ends with value r
                // (by masks: a selection of two elements becomes one of all 32)
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const uint32_t upper = r & o ? 0xFFFFFFFFu : 0u;
#pragma unroll
                    for (int k = 0; k < o; ++k) {
                        const uint32_t lo = __float_as_uint(v[k]), hi = __float_as_uint(v[k + o]);
                        const float send = __uint_as_float((lo & upper) | (hi & ~upper));
                        v[k] = __uint_as_float((hi & upper) | (lo & ~upper)) + __shfl_xor(send, o, kWave);
                    }
                }
                sums[wm / (32 * FA)][wn + 32 * (jj + (r >> 4)) + 8 * (r >> 2 & 3) + 4 * h + (r & 3)] = v[0];
            }
            __syncthreads();
            for (int n = threadIdx.x; n < TILE; n += T::NT)
                if (n0 + n < a.ldg) a.db_part[(int64_t)tm * a.ldg + n0 + n] = sums[0][n] + sums[1][n];
            __syncthreads();
        }
        // To memory through LDS, 16 bits an element, so that rows leave in 16-byte stores: the 16 bytes of columns
        // 8 u .. of row m lie at place u ^ (m & 15).  A second plane holds what the first rounds off.
        for (int plane = 0; plane < a.g_planes; ++plane) {
            const bool more = plane + 1 < a.g_planes;
            if (plane) __syncthreads();
#pragma unroll
            for (int i = 0; i < FA; ++i)
#pragma unroll
                for (int j = 0; j < FB; ++j)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int m = wm + 32 * i + r, u = (wn + 32 * j) / 8 + g;
                        const uint32_t lo = pack16<BRAIN>(acc[i][j][4 * g], acc[i][j][4 * g + 1]);
                        const uint32_t hi = pack16<BRAIN>(acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]);
                        if (more)
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[i][j][4 * g + e] -= of16<BRAIN>(e < 2 ? lo : hi, e & 1);
                        *(uint2*)(lds + m * (TILE * 2) + 16 * (u ^ (m & 15)) + 8 * h) = uint2{lo, hi};
                    }
            __syncthreads();
            uint16_t* to = a.g + (PL == 2 ? 32 * plane : plane * a.plane);
#pragma unroll 4
            for (int c = threadIdx.x; c < TILE * (TILE / 8); c += T::NT) {
                const int row = c / (TILE / 8), u = c % (TILE / 8);
                if (m0 + row >= a.rows || n0 + 8 * u >= a.ldg) continue;
                *(uint4*)(to + (PL == 2 ? planes_at(m0 + row, a.ldg, n0 + 8 * u) : (m0 + row) * a.ldg + n0 + 8 * u)) =
                    *(const uint4*)(lds + row * (TILE * 2) + 16 * (u ^ (row & 15)));
            }
        }
    }
}

// ------------------------------------------------------------ row statistics
// R rows a workgroup, 256 / R threads a row
template <int R>
__global__ __launch_bounds__(kNT) void policy_finish_kernel(FinishArgs a) {
    constexpr int S = kNT / R;
    __shared__ Soft each[S][R];
    __shared__ double red[kNT / kWave];
    const int row = threadIdx.x % R, slice = threadIdx.x / R;
    const int64_t m = (int64_t)blockIdx.x * R + row;
    Soft v{kNone, 0.f};
    if (m < a.rows)
#pragma unroll 4
        for (int k = slice; k < a.parts; k += S) v.join(a.part[(int64_t)k * a.rows + m]);
    each[slice][row] = v;
    for (int half = S / 2; half > 0; half /= 2) {
        __syncthreads();
        if (slice < half) {
            v.join(each[slice + half][row]);
            each[slice][row] = v;
        }
    }
    double term = 0.0;
    if (slice == 0 && m < a.rows) {
        const float l2 = v.s == 0.f ? kNone : v.m + log2f(v.s);
        const int32_t t = a.taken[m];
        float nll = 0.f;
        if (t >= 0 && t < a.actions) {
            const float z = a.z_taken[m];
            nll = z == kNone && l2 == l2 ? __builtin_huge_valf() : (l2 - z) * kLn2;
            const float w = a.row_weights ? a.row_weights[m] : 1.f;
            if (w != 0.f) term = (double)w * (double)nll;
        } else if (t != -1) {
            set_flag(a.flags, IQLH_FLAG_BAD_INDEX);
        }
        a.lse[m] = l2 * kLn2;
        a.nll[m] = nll;
    }
    term = block_sum64<kNT>(term, red);
    if (threadIdx.x == 0) {
        if (gridDim.x == 1) put_loss(a, term);
        else a.loss_part[blockIdx.x] = term;
    }
}
__global__ __launch_bounds__(kNT) void policy_loss_sum_kernel(FinishArgs a, int n) {
    __shared__ double red[kNT / kWave];
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kNT) s += a.loss_part[i];
    s = block_sum64<kNT>(s, red);
    if (threadIdx.x == 0) put_loss(a, s);
}
int finish_rows(int64_t rows) { return rows >= 1024 ? 64 : rows >= 64 ? 16 : 1; }
hipError_t launch_finish(const FinishArgs& a, hipStream_t stream) {
    const int R = finish_rows(a.rows);
    const uint32_t n = (uint32_t)((a.rows + R - 1) / R);
    auto kernel = R == 64 ? policy_finish_kernel<64> : R == 16 ? policy_finish_kernel<16> : policy_finish_kernel<1>;
    hipLaunchKernelGGL(kernel, dim3(n), dim3(kNT), 0, stream, a);
    if (n > 1) hipLaunchKernelGGL(policy_loss_sum_kernel, dim3(1), dim3(kNT), 0, stream, a, (int)n);
    return hipGetLastError();
}

// ----------------------------------------------------------------- products
// Sums to gradients: times mant 2^(exp + the magnitudes)
struct Back {
    float mant;
    int exp;
    const int32_t *g_top, *cols;  // or null: 0; cols [whole 8]
    const float* row_weights;     // or null: 0
    IQLH_DEV int all() const { return exp + (g_top ? *g_top : 0); }
    IQLH_DEV int row(int64_t m) const { return row_weights ? weight_bits(row_weights, m) : 0; }
    IQLH_DEV int col(int64_t n) const { return cols ? or_zero(cols[n]) : 0; }
    IQLH_DEV float apply(float v, int e) const { return ldexpf(v * mant, e); }
};
struct GradArgs {
    Side16 a, b;
    int64_t m, n, k;         // outputs, summed elements
    int64_t k_split;         // of one workgroup, a multiple of 64
    bool both;               // a's second matrix too
    int m_tiles, n_tiles, splits;
    Back back;
    float* sums;             // [splits][m][ld_sums]: partial sums
    int64_t ld_sums;
    int add;                 // to what lies in sums
    void* out;               // the result, or null: sums only
    int64_t ld_out;
    int out_dtype;
};
// One of the products of G: with `out` null, or several splits, the sums in binary32.
template <bool BRAIN, int TILE, bool AC, int PL>
__global__ __launch_bounds__(Tile16<TILE>::NT, Tile16<TILE>::PER_SIMD) void policy_grad_kernel(GradArgs a) {
    typedef Tile16<TILE, PL> T;
    extern __shared__ __align__(16) uint8_t lds[];
    const int tiles = a.m_tiles * a.n_tiles, split = blockIdx.x / tiles;
    int tm, tn;
    tile_of(blockIdx.x - split * tiles, a.m_tiles, a.n_tiles, tm, tn);
    const int64_t m0 = (int64_t)tm * TILE, n0 = (int64_t)tn * TILE;
    const int64_t k0 = split * a.k_split, k1 = k0 + a.k_split < a.k ? k0 + a.k_split : a.k;
    // exponents of the results' rows and columns, loaded before the product
    int* row_e = (int*)(lds + T::RING);
    int* col_e = row_e + TILE;
    const int all = a.back.all(), own = threadIdx.x % TILE;
    int re_in = 0, ce_in = 0;
    if (PL == 2 && a.out) {
        re_in = all + a.back.row(m0 + own < a.m ? m0 + own : a.m - 1);
        ce_in = n0 + own < a.n ? a.back.col(n0 + own) : 0;
    }
    mm_f16 acc[T::FA][T::FB];
    tile_product<BRAIN, TILE, AC, true, PL>(a.a, a.b, m0, n0, k0, k1, a.both, lds, acc);
    if (PL == 2 && threadIdx.x < TILE) row_e[own] = re_in, col_e[own] = ce_in;
    float* sums = a.sums + (int64_t)split * a.m * a.ld_sums;
#pragma unroll
    for (int band = 0; band < T::BANDS; ++band) {
        stage_band<TILE>(acc, lds, band);
#pragma unroll 2
        for (int c = threadIdx.x; c < T::BAND * (TILE / 8); c += T::NT) {
            const int row = c / (TILE / 8), u = c % (TILE / 8);
            const int64_t m = m0 + band * T::BAND + row, n = n0 + 8 * u;
            if (m >= a.m || n >= a.n) continue;
            const float4 lo = *stage_at<TILE>(lds, row, 2 * u), hi = *stage_at<TILE>(lds, row, 2 * u + 1);
            float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            float4* s = (float4*)(sums + m * a.ld_sums + n);  // rows of whole 8 elements
            if (a.add) {
                const float4 x = s[0], y = s[1];
                v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
                v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
            }
            if (a.out) {
                const int re = PL == 2 ? row_e[band * T::BAND + row] : all;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = a.back.apply(v[i], PL == 2 ? re + col_e[8 * u + i] : re);
                store8_of(a.out_dtype, a.out, m * a.ld_out + n, a.n - n, v);
            } else {
                s[0] = float4{v[0], v[1], v[2], v[3]};
                s[1] = float4{v[4], v[5], v[6], v[7]};
            }
        }
    }
}

// out = factor times the sum over the splits
__global__ __launch_bounds__(kNT) void policy_join_kernel(GradArgs a) {
    const int64_t groups = (a.n + 7) / 8, total = a.m * groups;
    const int all = a.back.all();
    for (int64_t e = (int64_t)blockIdx.x * kNT + threadIdx.x; e < total; e += (int64_t)gridDim.x * kNT) {
        const int64_t m = e / groups, n = 8 * (e - m * groups);
        const int re = all + a.back.row(m);
        int ce[8] = {};
        if (a.back.cols) {
            const int4 x = *(const int4*)(a.back.cols + n), y = *(const int4*)(a.back.cols + n + 4);
            ce[0] = x.x, ce[1] = x.y, ce[2] = x.z, ce[3] = x.w, ce[4] = y.x, ce[5] = y.y, ce[6] = y.z, ce[7] = y.w;
        }
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int k = 0; k < a.splits; ++k) {
            const float4* s = (const float4*)(a.sums + ((int64_t)k * a.m + m) * a.ld_sums + n);
            const float4 x = s[0], y = s[1];
            v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
            v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = a.back.apply(v[i], re + or_zero(ce[i]));
        store8_of(a.out_dtype, a.out, m * a.ld_out + n, a.n - n, v);
    }
}
// db of a piece
__global__ __launch_bounds__(kNT) void policy_bias_kernel(const float* part, int parts, int64_t ld, Back back, float* out,
                                                          int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * kNT + threadIdx.x;
    if (i >= n) return;
    double s = 0.0;
#pragma unroll 8
    for (int k = 0; k < parts; ++k) s += part[k * ld + i];
    out[i] = back.apply((float)s, back.all());
}

// Rows up to which G has two planes whatever its type: its rounding does not average
// out over few rows, and the products are bound by W and dW there
constexpr int64_t kFewRows = 64;

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
int64_t tiles_of(int64_t m, int64_t n, int t) { return ((m + t - 1) / t) * ((n + t - 1) / t); }
// Tiles of 256 where those of 128, two to a compute unit, would need more than one round: loss and gradients' two
// products of logits of 1280 x 8192 x 512 bf16 (160 tiles) 42 us against 48, of 2048 x 16384 x 512 87 against 106;
// but of 1024 x 8192 x 512 (128 tiles) 41 against 33.  With two planes from 192 tiles on: 1280 x 9000 x 1024 (180
// tiles) 166 against 160 us, 4096 x 16384 x 512 486 against 502.
int tile_for(int64_t m, int64_t n, int planes) { return tiles_of(m, n, 256) > (planes == 1 ? 128 : 192) ? 256 : 128; }

// Parts of the summed axis, of 512 elements or more, so that there are 384 workgroups of 128 tiles, 512 with two
// planes, and none where half as many are there without.  dH of 777 x 501 over 10007 actions: 21 us and the join 7,
// unsplit 109.  More parts gain less than their join takes: dW of 8192 x 512 over 1280 rows 20 us and the join 22 in
// two parts, 21.5 whole; dH of 4096 x 512 over 16384 actions in two planes, three parts 239 and 13, four 202 and 8.
struct Split {
    int tile, n;
    int64_t k;
};
Split split_for(int64_t m, int64_t n, int64_t k, int planes) {
    Split s{tile_for(m, n, planes), 1, up(k, 64)};
    if (s.tile == 256) return s;
    int64_t want = (planes == 1 ? 384 : 512) / tiles_of(m, n, 128), most = (k + 511) / 512;
    want = want < 1 ? 1 : want > most ? most : want;
    s.k = up((k + want - 1) / want, 64);
    s.n = (int)((k + s.k - 1) / s.k);
    return s;
}

}  // namespace

// Actions of a piece: G of 256 MB, what the Infinity Cache holds, but enough for dW to have tiles.  8192 x 65536
// x 2048 bf16, loss and gradients: four pieces 7.37 ms, one of 1 GB 7.27 ms: not worth four times the workspace.
PolicyPlan policy_plan(int64_t rows, int64_t actions, int64_t dim, int dtype, bool grad) {
    PolicyPlan p{};
    p.planes = dtype == IQLH_F32 ? 2 : 1;
    p.g_planes = dtype == IQLH_F32 || rows <= kFewRows ? 2 : 1;
    p.ld = up(dim, 64);
    int64_t piece = ((int64_t)1 << 27) / (rows * p.g_planes) / 256 * 256;
    piece = piece < 1024 ? 1024 : piece;
    p.piece = piece < actions ? piece : up(actions, 64);
    p.pieces = (int)((actions + p.piece - 1) / p.piece);
    size_t at = 0;
    auto take = [&at](size_t bytes) {
        const size_t was = at;
        at += (bytes + 255) / 256 * 256;
        return was;
    };
    p.z_taken = take((size_t)rows * 4);
    p.loss_part = take((size_t)rows * 8);
    p.few_actions = policy_few_actions_ok(actions, dim);
    p.few_rows = !p.few_actions && !grad && policy_few_rows_ok(rows, dim, dtype);
    if (p.few_actions || p.few_rows) {
        p.part = take(p.few_rows ? (size_t)policy_few_rows_parts(actions) * rows * sizeof(Soft) : 0);
        p.g = take(grad ? policy_few_actions_bytes(rows, actions, dim) : 0);
        p.bytes = at;
        return p;
    }
    p.row_exp = take(p.planes == 2 ? (size_t)rows * 4 : 0);
    p.act_exp = take(p.planes == 2 ? (size_t)actions * 4 : 0);
    p.cols = take(p.planes == 2 ? (size_t)p.ld * 8 : 0);
    p.h = take((size_t)rows * p.ld * 2 * p.planes);
    p.w = take((size_t)actions * p.ld * 2 * p.planes);
    const size_t begin = at;  // the loss's and the gradients' own
    p.part = take((size_t)((actions + 127) / 128) * rows * sizeof(Soft));
    p.bytes = at;
    if (grad) {
        at = begin;
        const Split dh = split_for(rows, dim, p.piece, p.planes);
        const int64_t full = p.pieces > 1 ? p.piece : actions, last = actions - (p.pieces - 1) * p.piece;
        // parts of dW, none where one workgroup has the whole sum
        auto dw_parts = [&](int64_t n) { const int64_t k = split_for(n, dim, rows, p.planes).n; return k > 1 ? k * n : 0; };
        const int64_t dw_full = dw_parts(full), dw_last = dw_parts(last);
        p.g_top = take(4);
        p.weight_top = take(kAbsBlocks * 4);  // or kStartWaves
        p.h_dw = take(p.planes == 2 ? (size_t)rows * p.ld * 4 : 0);
        p.w_dh = take(p.planes == 2 ? (size_t)actions * p.ld * 4 : 0);
        p.g = take((size_t)rows * p.piece * 2 * p.g_planes);
        p.db_part = take((size_t)((rows + 127) / 128) * p.piece * 4);
        p.dh_sums = take(p.pieces > 1 || dh.n > 1 ? (size_t)dh.n * rows * up(dim, 8) * 4 : 0);
        p.dw_sums = take((size_t)(dw_full > dw_last ? dw_full : dw_last) * up(dim, 8) * 4);
        if (at > p.bytes) p.bytes = at;
    }
    return p;
}

namespace {

struct Operands {
    Side16 h, w;       // of the logits
    Side16 h_dw, w_dh;  // of the gradients' products
    int64_t k;         // summed elements of the logits; columns of H and W as operands
    const int32_t *row_exp, *act_exp, *cols_h, *cols_w, *g_top;
};

bool in_place(const PolicyMat& q) {
    return q.dtype != IQLH_F32 && (uintptr_t)q.p % 16 == 0 && q.ld % 8 == 0 && q.ld < 1 << 22 && q.cols % 8 == 0;
}

// H and W as operands.  For the gradients rows of H that are off become zeros, since they would add
// 0 times what they hold to dW, NaN or infinities as it may be.
hipError_t prepare(const PolicyArgs& a, const PolicyPlan& p, bool grad, Operands* o, hipStream_t stream) {
    const bool f32 = a.h.dtype == IQLH_F32, sized = grad && a.h.dtype == IQLH_F16 && a.row_weights;
    uint8_t* base = (uint8_t*)a.workspace;
    const PolicyMat none{};
    ConvertArgs c{};
    c.dtype = a.h.dtype;
    c.taken = a.taken, c.row_weights = a.row_weights, c.actions = a.w.rows;
    *o = Operands{};
    if (sized) {
        c.part = (int32_t*)(base + p.weight_top);
        o->g_top = c.g_top = (int32_t*)(base + p.g_top);
        hipLaunchKernelGGL(policy_weights_kernel, dim3(kAbsBlocks), dim3(kNT), 0, stream, a.taken, a.row_weights, a.h.rows, a.w.rows,
                           (int32_t*)(base + p.weight_top));
    }
    if (f32) {
        ColumnArgs m{};
        m.m[0] = grad && a.d_weight ? a.h : none, m.m[1] = a.w;
        m.to[0] = (int32_t*)(base + p.cols), m.to[1] = m.to[0] + p.ld;
        m.taken = a.taken, m.row_weights = a.row_weights, m.bias = a.bias, m.actions = a.w.rows, m.ld = p.ld;
        m.lanes = a.h.cols <= 64 ? 8 : 16;
        o->cols_h = m.to[0], o->cols_w = m.to[1];
        o->row_exp = (int32_t*)(base + p.row_exp), o->act_exp = (int32_t*)(base + p.act_exp);
        // one workgroup to a column for up to 512 rows: as long as the launch that empties the columns takes
        const int64_t most = m.m[0].p && a.h.rows > a.w.rows ? a.h.rows : a.w.rows, chunks = (p.ld + 8 * m.lanes - 1) / (8 * m.lanes);
        int64_t slabs = most <= 512 ? 1 : 512 / chunks < 32 ? 32 : 512 / chunks;
        if (slabs > (most + 63) / 64) slabs = (most + 63) / 64;
        // d_hidden of a row that took a forbidden action has that action's weights
        const bool forbids = grad && a.d_hidden && a.bias;
        if (slabs > 1 || forbids) {
            StartArgs s{m.to[0], (int)(2 * p.ld), forbids ? (int32_t*)(base + p.weight_top) : nullptr, a.taken, a.row_weights, a.bias,
                        a.h.rows, a.w.rows};
            m.part = c.forbid_part = s.part;
            hipLaunchKernelGGL(policy_start_kernel, dim3(forbids ? kStartBlocks : (uint32_t)((2 * p.ld + kNT - 1) / kNT)), dim3(kNT), 0, stream, s);
        }
        c.bias = a.bias;
        hipLaunchKernelGGL(policy_columns_kernel, dim3((uint32_t)slabs, (uint32_t)chunks, 2), dim3(kNT), 0, stream, m);
    }
    int n = 0;
    auto convert = [&](const PolicyMat& q, size_t at, bool zero_off, int32_t* row_exp, const int32_t* cols, int sign,
                       bool weighted, bool forbids = false) {
        int lanes = 8;  // rows are of 8 groups or more
        while (lanes < kWave && lanes < p.ld / 8) lanes *= 2;
        const int64_t blocks = row_exp ? (q.rows * lanes + kNT - 1) / kNT : (q.rows * (p.ld / 8) + 4 * kNT - 1) / (4 * kNT);
        c.c[n++] = Convert{q,       (uint16_t*)(base + at), p.ld, cols, row_exp, sign, forbids ? -1 : zero_off, weighted, lanes,
                           (int)(blocks < 4096 ? blocks : 4096)};
        return Side16{(const uint16_t*)(base + at), 0, p.ld, q.rows};
    };
    if (f32) {
        o->k = p.ld;
        o->h = convert(a.h, p.h, grad, (int32_t*)o->row_exp, o->cols_w, 1, false);
        o->w = convert(a.w, p.w, false, (int32_t*)o->act_exp, o->cols_w, -1, false);
        if (grad && a.d_weight) o->h_dw = convert(a.h, p.h_dw, true, nullptr, o->cols_h, -1, true);
        if (grad && a.d_hidden) o->w_dh = convert(a.w, p.w_dh, false, nullptr, o->cols_w, -1, false, true);
    } else {
        // both in place or both converted, but for H of the gradients: the summed axis is as long in one as in the other
        const bool copy = !in_place(a.w) || (!grad && !in_place(a.h));
        o->k = copy ? p.ld : a.h.cols;
        o->h = copy || grad ? convert(a.h, p.h, grad, nullptr, nullptr, 0, false)
                            : Side16{(const uint16_t*)a.h.p, 0, a.h.ld, a.h.rows};
        o->w = copy ? convert(a.w, p.w, false, nullptr, nullptr, 0, false) : Side16{(const uint16_t*)a.w.p, 0, a.w.ld, a.w.rows};
        o->h_dw = o->h, o->w_dh = o->w;
    }
    if (n) {
        const uint32_t blocks = c.c[0].blocks + c.c[1].blocks + c.c[2].blocks + c.c[3].blocks;
        hipLaunchKernelGGL(policy_convert_kernel, dim3(blocks), dim3(kNT), 0, stream, c);
    }
    return hipGetLastError();
}

// f(binary16 or bfloat16, tile, planes); two planes are binary16's
template <typename F>
hipError_t by_operands(bool brain, int planes, int tile, F f) {
    typedef std::integral_constant<int, 1> One;
    typedef std::integral_constant<int, 2> Two;
    typedef std::integral_constant<int, 128> T128;
    typedef std::integral_constant<int, 256> T256;
    if (planes == 2 && tile == 256) f(std::false_type(), T256(), Two());
    else if (planes == 2) f(std::false_type(), T128(), Two());
    else if (tile == 256) brain ? f(std::true_type(), T256(), One()) : f(std::false_type(), T256(), One());
    else brain ? f(std::true_type(), T128(), One()) : f(std::false_type(), T128(), One());
    return hipGetLastError();
}

template <bool GRAD>
hipError_t launch_logits(LogitArgs a, bool brain, int planes, hipStream_t stream) {
    const int tile = tile_for(a.rows, a.actions, planes);
    a.m_tiles = (int)((a.rows + tile - 1) / tile);
    a.n_tiles = (int)(((GRAD ? a.ldg : a.actions) + tile - 1) / tile);
    return by_operands(brain, planes, tile, [&](auto is_brain, auto t, auto pl) {
        typedef Tile16<decltype(t)::value, decltype(pl)::value> T;
        auto kernel = policy_logits_kernel<decltype(is_brain)::value, decltype(t)::value, GRAD, decltype(pl)::value>;
        (void)hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, T::LDS);
        hipLaunchKernelGGL(kernel, dim3((uint32_t)(a.m_tiles * a.n_tiles)), dim3(T::NT), T::LDS, stream, a);
    });
}

// `joined`: partial sums that make up the result, at least those of this launch
template <bool AC>
hipError_t launch_grad_product(GradArgs a, const Split& s, int joined, bool brain, int planes, hipStream_t stream) {
    a.m_tiles = (int)((a.m + s.tile - 1) / s.tile);
    a.n_tiles = (int)((a.n + s.tile - 1) / s.tile);
    a.splits = s.n;
    a.k_split = s.k;
    void* out = a.out;
    if (joined > 1) a.out = nullptr;
    hipError_t e = by_operands(brain, planes, s.tile, [&](auto is_brain, auto t, auto pl) {
        typedef Tile16<decltype(t)::value, decltype(pl)::value> T;
        auto kernel = policy_grad_kernel<decltype(is_brain)::value, decltype(t)::value, AC, decltype(pl)::value>;
        (void)hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, T::LDS);
        hipLaunchKernelGGL(kernel, dim3((uint32_t)(a.m_tiles * a.n_tiles * a.splits)), dim3(T::NT), T::LDS, stream, a);
    });
    if (e == hipSuccess && joined > 1 && out) {
        a.out = out;
        a.splits = joined;
        const int64_t blocks = (a.m * ((a.n + 7) / 8) + kNT - 1) / kNT;
        hipLaunchKernelGGL(policy_join_kernel, dim3((uint32_t)(blocks < 2048 ? blocks : 2048)), dim3(kNT), 0, stream, a);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace

hipError_t launch_policy_loss(const PolicyArgs& a, hipStream_t stream) {
    const PolicyPlan p = policy_plan(a.h.rows, a.w.rows, a.h.cols, a.h.dtype, false);
    uint8_t* base = (uint8_t*)a.workspace;
    FinishArgs f{};
    f.part = (Soft*)(base + p.part), f.z_taken = (float*)(base + p.z_taken), f.taken = a.taken, f.row_weights = a.row_weights;
    f.nll = a.nll, f.lse = a.lse_out, f.loss = a.loss, f.loss_part = (double*)(base + p.loss_part), f.flags = a.flags;
    f.rows = a.h.rows, f.actions = a.w.rows, f.scale = a.scale;
    if (p.few_actions) {
        int n = 0;
        hipError_t e = launch_policy_few_actions(a, f.loss_part, &n, stream);
        if (e != hipSuccess || n == 1) return e;
        hipLaunchKernelGGL(policy_loss_sum_kernel, dim3(1), dim3(kNT), 0, stream, f, n);
        return hipGetLastError();
    }
    if (p.few_rows) {
        hipError_t e = launch_policy_few_rows(a, base + p.part, (float*)(base + p.z_taken), stream);
        if (e != hipSuccess) return e;
        f.parts = policy_few_rows_parts(a.w.rows);
        return launch_finish(f, stream);
    }
    Operands o;
    hipError_t e = prepare(a, p, false, &o, stream);
    if (e != hipSuccess) return e;
    LogitArgs l{};
    l.h = o.h, l.w = o.w, l.k = o.k, l.row_exp = o.row_exp, l.act_exp = o.act_exp;
    l.bias = a.bias, l.taken = a.taken;
    l.rows = a.h.rows, l.actions = l.all_actions = a.w.rows;
    l.part = (Soft*)(base + p.part), l.z_taken = (float*)(base + p.z_taken);
    e = launch_logits<false>(l, a.h.dtype == IQLH_BF16, p.planes, stream);
    if (e != hipSuccess) return e;
    const int tile = tile_for(l.rows, l.actions, p.planes);
    f.parts = (int)((l.actions + tile - 1) / tile);
    return launch_finish(f, stream);
}

hipError_t launch_policy_loss_grad(const PolicyArgs& a, hipStream_t stream) {
    const PolicyPlan p = policy_plan(a.h.rows, a.w.rows, a.h.cols, a.h.dtype, true);
    uint8_t* base = (uint8_t*)a.workspace;
    if (p.few_actions) return launch_policy_few_actions_grad(a, base + p.g, stream);
    const int64_t rows = a.h.rows, actions = a.w.rows, dim = a.h.cols;
    const bool brain = a.h.dtype == IQLH_BF16;
    const int es = a.h.dtype == IQLH_F32 ? 4 : 2;
    Operands o;
    hipError_t e = prepare(a, p, true, &o, stream);
    // The scale is mant 2^exp.  Bfloat16: G holds mant.  Else G is times 2^(kTop - magnitude of the weights), 1 of weights
    // that are not given, and binary32's other operands too
    const bool f32 = a.h.dtype == IQLH_F32;
    Back back{1.f, 0, o.g_top, nullptr, nullptr};
    const float mant = (float)std::frexp(a.scale, &back.exp);
    if (!brain) back.mant = mant;
    if (a.h.dtype == IQLH_F16) back.exp += (o.g_top ? 0 : 1) - kTop;
    LogitArgs l{};
    l.h = o.h, l.w = o.w, l.k = o.k, l.row_exp = o.row_exp;
    l.g_top = o.g_top, l.g_factor = brain ? mant : (float)(1 << (kTop - 1));
    l.taken = a.taken, l.row_weights = a.row_weights, l.lse = a.lse_in;
    l.rows = rows, l.all_actions = actions;
    l.g = (uint16_t*)(base + p.g), l.g_planes = p.g_planes;
    const Split dh = split_for(rows, dim, p.piece, p.planes);
    for (int k = 0; k < p.pieces && e == hipSuccess; ++k) {
        const int64_t first = k * p.piece, n = actions - first < p.piece ? actions - first : p.piece;
        l.first = first, l.actions = n, l.ldg = up(n, 64), l.plane = rows * l.ldg;
        l.w.p = o.w.p + p.planes * first * o.w.ld, l.w.n = n;
        l.act_exp = f32 ? o.act_exp + first : nullptr;
        l.bias = a.bias ? a.bias + first : nullptr;
        l.db_part = a.d_bias ? (float*)(base + p.db_part) : nullptr;
        e = launch_logits<true>(l, brain, p.planes, stream);
        if (e != hipSuccess) break;
        if (a.d_bias) {
            const int tile = tile_for(rows, n, p.planes);
            hipLaunchKernelGGL(policy_bias_kernel, dim3((uint32_t)((n + kNT - 1) / kNT)), dim3(kNT), 0, stream, l.db_part,
                               (int)((rows + tile - 1) / tile), l.ldg, back, a.d_bias + first, n);
            e = hipGetLastError();
        }
        GradArgs g{};
        g.n = dim, g.both = p.planes == 1 && p.g_planes == 2, g.ld_sums = up(dim, 8), g.out_dtype = a.h.dtype;
        const Side16 gs{l.g, l.plane, l.ldg, rows};
        if (a.d_weight && e == hipSuccess) {
            g.a = Side16{l.g, l.plane, l.ldg, l.ldg};
            g.b = o.h_dw;
            g.b.n = o.k;
            g.m = n, g.k = rows;
            g.back = back;
            if (f32) g.back.exp -= 2 * kTop, g.back.cols = o.cols_h;
            g.sums = (float*)(base + p.dw_sums);
            g.out = (uint8_t*)a.d_weight + first * a.ld_dw * es;
            g.ld_out = a.ld_dw;
            const Split s = split_for(n, dim, rows, p.planes);
            e = launch_grad_product<true>(g, s, s.n, brain, p.planes, stream);
        }
        if (a.d_hidden && e == hipSuccess) {
            g.a = gs;
            g.b = o.w_dh;
            g.b.p += p.planes * first * g.b.ld;
            g.b.n = o.k;
            g.m = rows, g.k = n;
            g.back = back;
            if (f32) g.back.exp -= 2 * kTop, g.back.cols = o.cols_w, g.back.exp += a.row_weights ? 0 : 1, g.back.row_weights = a.row_weights;
            g.sums = (float*)(base + p.dh_sums);
            g.add = k > 0;
            g.out = k + 1 == p.pieces ? a.d_hidden : nullptr;
            g.ld_out = a.ld_dh;
            Split s = dh;
            s.n = (int)((n + s.k - 1) / s.k);
            e = launch_grad_product<false>(g, s, p.pieces > 1 ? dh.n : s.n, brain, p.planes, stream);
        }
    }
    return e;
}

}  // namespace iqlh
