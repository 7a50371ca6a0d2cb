// Policy loss of few actions and of few rows.
//
// Few actions (up to 16, with the head's weights in 64 KB): a tile of the matrix
// instructions would be empty but for them, and what counts is hidden, read once for the
// loss and twice for the gradients.  16 lanes take a row, eight neighbouring elements each,
// products in binary32 from the weights in LDS.
//   1. logits, the row's statistics and the loss, or G (binary32, to the workspace);
//   2. dH, and the workgroup's part of dW and db, for 128 columns;
//   3. the parts' sum.
// 16384 rows, dim 128, nine actions in binary32, loss and gradients: 34 us, with tiles 97; hidden's three reads are
// 25 MB, 5 us: what is left are five launches, none of which fills the chip for long.
//
// Few rows (up to 16): bound by the head's weights, which a wave reads straight into the
// matrix instruction's registers, 16 actions at a time, several loads in flight; hidden
// lies in LDS.  Binary32 takes the binary32 matrix instructions, which are below the loads' time.
#include "policy_block.hpp"

namespace iqlh {

using namespace policy;

namespace {

struct FewArgs {
    PolicyMat h, w;
    const float* bias;  // or null
    const float* lse;   // gradients
    float* g;           // [rows][VM]
    float* part;        // [blocks][VM][ld] of dW, then [blocks][VM] of db
    void* d_hidden;     // or null
    void* d_weight;     // or null
    float* d_bias;      // or null
    int64_t ld_dh, ld_dw;
    int32_t blocks;     // of the rows
    FinishArgs f;
};

constexpr int kGroups = kNT / 16;  // rows a workgroup takes at a time

// ------------------------------------------------------------- few actions
template <int VM, bool GRAD>
__global__ __launch_bounds__(kNT) void policy_few_actions_kernel(FewArgs a) {
    extern __shared__ __align__(16) float w_lds[];  // [VM][ld]
    __shared__ double red[kNT / kWave];
    const int64_t rows = a.h.rows;
    const int dim = (int)a.h.cols, groups = (dim + 7) / 8, ld = 8 * groups, V = (int)a.w.rows, lane = threadIdx.x & 15;
    // the first elements of the first row, on their way while the weights come to LDS
    const int64_t m_first = (int64_t)blockIdx.x * kGroups + threadIdx.x / 16;
    float x0[8];
    if (m_first < rows && 8 * lane < dim) load8_of(a.h.dtype, a.h.p, m_first * a.h.ld + 8 * lane, dim - 8 * lane, x0);
    for (int e = threadIdx.x; e < VM * groups; e += kNT) {
        const int v = e / groups, col = 8 * (e - v * groups);
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (v < V) load8_of(a.w.dtype, a.w.p, v * a.w.ld + col, dim - col, x);
        *(float4*)(w_lds + v * ld + col) = float4{x[0], x[1], x[2], x[3]};
        *(float4*)(w_lds + v * ld + col + 4) = float4{x[4], x[5], x[6], x[7]};
    }
    __syncthreads();
    double term = 0.0;
    for (int64_t m = m_first; m < rows; m += (int64_t)gridDim.x * kGroups) {
        const int32_t t = a.f.taken[m];
        const float weight = a.f.row_weights ? a.f.row_weights[m] : 1.f;
        const float lse_in = GRAD ? a.lse[m] : 0.f;
        float z[VM];
#pragma unroll
        for (int v = 0; v < VM; ++v) z[v] = 0.f;
        for (int col = 8 * lane; col < dim; col += 128) {
            float x[8];
            if (m == m_first && col == 8 * lane) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = x0[i];
            } else {
                load8_of(a.h.dtype, a.h.p, m * a.h.ld + col, dim - col, x);
            }
#pragma unroll
            for (int v = 0; v < VM; ++v) {
                const float4 p = *(const float4*)(w_lds + v * ld + col), q = *(const float4*)(w_lds + v * ld + col + 4);
                z[v] = fmaf(x[0], p.x, fmaf(x[1], p.y, fmaf(x[2], p.z, fmaf(x[3], p.w, z[v]))));
                z[v] = fmaf(x[4], q.x, fmaf(x[5], q.y, fmaf(x[6], q.z, fmaf(x[7], q.w, z[v]))));
            }
        }
        Soft soft{kNone, 0.f};
        float taken = kNone;
#pragma unroll
        for (int v = 0; v < VM; ++v) {
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) z[v] += __shfl_xor(z[v], o, kWave);
            z[v] = v < V ? fmaf(z[v], kLog2e, a.bias ? a.bias[v] * kLog2e : 0.f) : kNone;
            soft.m = fmaxf(soft.m, z[v]);
            if (v == t) taken = z[v];
        }
        const bool there = t >= 0 && t < V, on = there && weight != 0.f;
        if constexpr (!GRAD) {
            const float top = soft.m == kNone ? 0.f : soft.m;
#pragma unroll
            for (int v = 0; v < VM; ++v) soft.s += __builtin_amdgcn_exp2f(z[v] - top);
            const float l2 = soft.s == 0.f ? kNone : soft.m + log2f(soft.s);
            const float nll = !there ? 0.f : taken == kNone && l2 == l2 ? __builtin_huge_valf() : (l2 - taken) * kLn2;
            if (lane == 0) {
                a.f.lse[m] = l2 * kLn2;
                a.f.nll[m] = nll;
                if (on) term += (double)weight * (double)nll;
                if (!there && t != -1) set_flag(a.f.flags, IQLH_FLAG_BAD_INDEX);
            }
        } else {
            const float l2 = lse_in == kNone ? 0.f : lse_in * kLog2e, scale = weight * (float)a.f.scale;
#pragma unroll
            for (int v = 0; v < VM; ++v) {
                const float g = scale * (__builtin_amdgcn_exp2f(z[v] - l2) - (v == t ? 1.f : 0.f));
                if (lane == v) a.g[m * VM + v] = on && v < V ? g : 0.f;
            }
        }
    }
    if constexpr (!GRAD) {
        term = block_sum64<kNT>(term, red);
        if (threadIdx.x == 0) {
            if (gridDim.x == 1) put_loss(a.f, term);
            else a.f.loss_part[blockIdx.x] = term;
        }
    }
}

// dH, and the parts of dW and db, of 128 columns (blockIdx.y)
template <int VM>
__global__ __launch_bounds__(kNT, 2) void policy_few_grads_kernel(FewArgs a) {
    constexpr int AHEAD = 2;
    __shared__ __align__(16) float w_lds[VM][128];
    __shared__ __align__(16) float sums[kNT / kWave][VM][128];
    __shared__ float b_sums[kNT / kWave][VM];
    const int64_t rows = a.h.rows;
    const int dim = (int)a.h.cols, ld = (dim + 7) / 8 * 8, V = (int)a.w.rows, lane = threadIdx.x & 15, wave = threadIdx.x >> 6;
    const int col = blockIdx.y * 128 + 8 * lane, n = dim - col;
    for (int e = threadIdx.x; e < VM * 16; e += kNT) {
        const int v = e / 16, c = blockIdx.y * 128 + 8 * (e % 16);
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (v < V && c < dim) load8_of(a.w.dtype, a.w.p, v * a.w.ld + c, dim - c, x);
        *(float4*)&w_lds[v][8 * (e % 16)] = float4{x[0], x[1], x[2], x[3]};
        *(float4*)&w_lds[v][8 * (e % 16) + 4] = float4{x[4], x[5], x[6], x[7]};
    }
    __syncthreads();
    float acc[VM][8], b[VM];
#pragma unroll
    for (int v = 0; v < VM; ++v) {
        b[v] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[v][i] = 0.f;
    }
    const int64_t step = (int64_t)a.blocks * kGroups;
    for (int64_t m0 = (int64_t)blockIdx.x * kGroups + threadIdx.x / 16; m0 < rows; m0 += AHEAD * step) {
        float x[AHEAD][8], g[AHEAD][VM];
        asm volatile("" ::: "memory");  // the weights stay in LDS: kept in registers they displace the sums
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int64_t m = m0 + k * step;
#pragma unroll
            for (int v = 0; v < VM; v += 4) {
                const float4 q = m < rows ? *(const float4*)(a.g + m * VM + v) : float4{0.f, 0.f, 0.f, 0.f};
                g[k][v] = q.x, g[k][v + 1] = q.y, g[k][v + 2] = q.z, g[k][v + 3] = q.w;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) x[k][i] = 0.f;
            if (m < rows && n > 0 && a.d_weight) load8_of(a.h.dtype, a.h.p, m * a.h.ld + col, n, x[k]);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int64_t m = m0 + k * step;
            float dh[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            bool any = false;  // a row that is off may hold anything
#pragma unroll
            for (int v = 0; v < VM; ++v) any |= g[k][v] != 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[k][i] = any ? x[k][i] : 0.f;
#pragma unroll
            for (int v = 0; v < VM; ++v) {
                const float4 p = *(const float4*)&w_lds[v][8 * lane], q = *(const float4*)&w_lds[v][8 * lane + 4];
                const float w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
                b[v] += g[k][v];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dh[i] = fmaf(g[k][v], w[i], dh[i]);
                    acc[v][i] = fmaf(g[k][v], x[k][i], acc[v][i]);
                }
            }
            if (!any)
#pragma unroll
                for (int i = 0; i < 8; ++i) dh[i] = 0.f;
            if (m < rows && n > 0 && a.d_hidden) store8_of(a.h.dtype, a.d_hidden, m * a.ld_dh + col, n, dh);
        }
    }
    // the four rows of a wave, then the waves
#pragma unroll
    for (int v = 0; v < VM; ++v) {
#pragma unroll
        for (int o = 16; o < 64; o <<= 1) {
            b[v] += __shfl_xor(b[v], o, kWave);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[v][i] += __shfl_xor(acc[v][i], o, kWave);
        }
        if ((threadIdx.x & 63) < 16) {
            *(float4*)&sums[wave][v][8 * lane] = float4{acc[v][0], acc[v][1], acc[v][2], acc[v][3]};
            *(float4*)&sums[wave][v][8 * lane + 4] = float4{acc[v][4], acc[v][5], acc[v][6], acc[v][7]};
            if (lane == 0) b_sums[wave][v] = b[v];
        }
    }
    __syncthreads();
    float* part = a.part + (int64_t)blockIdx.x * VM * ld;
    for (int e = threadIdx.x; e < VM * 128; e += kNT) {
        const int v = e / 128, c = e % 128;
        if (blockIdx.y * 128 + c < ld) part[v * ld + blockIdx.y * 128 + c] = sums[0][v][c] + sums[1][v][c] + sums[2][v][c] + sums[3][v][c];
    }
    if (blockIdx.y == 0 && threadIdx.x < VM)
        a.part[(int64_t)a.blocks * VM * ld + blockIdx.x * VM + threadIdx.x] =
            b_sums[0][threadIdx.x] + b_sums[1][threadIdx.x] + b_sums[2][threadIdx.x] + b_sums[3][threadIdx.x];
}

// Sum of the parts: action blockIdx.x, 128 columns blockIdx.y, 16 threads along the parts
template <int VM>
__global__ __launch_bounds__(kNT) void policy_few_join_kernel(FewArgs a) {
    __shared__ float sums[16][128];
    __shared__ double red[kNT / kWave];
    const int dim = (int)a.h.cols, ld = (dim + 7) / 8 * 8, v = blockIdx.x, lane = threadIdx.x & 15, slice = threadIdx.x / 16;
    const int col = blockIdx.y * 128 + 8 * lane;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (col < ld && a.d_weight)
#pragma unroll 4
        for (int k = slice; k < a.blocks; k += 16) {
            const float4* p = (const float4*)(a.part + ((int64_t)k * VM + v) * ld + col);
            const float4 x = p[0], y = p[1];
            s[0] += x.x, s[1] += x.y, s[2] += x.z, s[3] += x.w, s[4] += y.x, s[5] += y.y, s[6] += y.z, s[7] += y.w;
        }
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[slice][8 * lane + i] = s[i];
    __syncthreads();
    if (slice == 0 && col < dim && a.d_weight) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) y[i] += sums[k][8 * lane + i];
        }
        store8_of(a.w.dtype, a.d_weight, v * a.ld_dw + col, dim - col, y);
    }
    if (blockIdx.y == 0 && a.d_bias) {
        double b = 0.0;
        for (int k = threadIdx.x; k < a.blocks; k += kNT) b += a.part[(int64_t)a.blocks * VM * ld + k * VM + v];
        b = block_sum64<kNT>(b, red);
        if (threadIdx.x == 0) a.d_bias[v] = (float)b;
    }
}

template <typename F>
hipError_t by_actions(int64_t actions, F f) {
    if (actions <= 4) f(std::integral_constant<int, 4>());
    else if (actions <= 8) f(std::integral_constant<int, 8>());
    else if (actions <= 12) f(std::integral_constant<int, 12>());
    else f(std::integral_constant<int, 16>());
    return hipGetLastError();
}
int few_vm(int64_t actions) { return actions <= 4 ? 4 : actions <= 8 ? 8 : actions <= 12 ? 12 : 16; }
int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }

// ---------------------------------------------------------------- few rows
typedef float mm_f4 __attribute__((ext_vector_type(4)));
struct FewRowsArgs {
    PolicyMat h, w;
    const float* bias;  // or null
    const int32_t* taken;
    Soft* part;         // [workgroups][rows]
    float* z_taken;
};
// A wave takes 16 actions at a time: lane l reads the 16 bytes of its chunk l / 16 of the step's four from
// row l % 16 of W (action) and, from LDS, of hidden.
template <int DT>
__global__ __launch_bounds__(kNT) void policy_few_rows_kernel(FewRowsArgs a) {
    constexpr int E = DT == IQLH_F32 ? 4 : 8, ES = 16 / E, U = 16;  // elements of a lane and step; steps in flight
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ Soft waves[kNT / kWave][16];
    const int rows = (int)a.h.rows, dim = (int)a.h.cols, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, blk = lane >> 4, chunks = (dim + E - 1) / E, steps = (chunks + 3) / 4;
    const int pitch = steps * 64 + 16;  // bytes of a row of hidden, zeros behind its end
    // 16 bytes of a row, zeros behind its end (hidden's zeros there must not meet a NaN)
    auto load = [&](const uint8_t* row, int c) __attribute__((always_inline)) {
        const int n = dim - c * E;
        u4_a2 w = {0u, 0u, 0u, 0u};
        if (n >= E) {
            w = *(const u4_a2*)(row + (int64_t)c * 16);
        } else {
            for (int i = 0; i < n; ++i) {
                if (DT == IQLH_F32) w[i] = ((const uint32_t*)(row + (int64_t)c * 16))[i];
                else w[i >> 1] |= (uint32_t)((const uint16_t*)(row + (int64_t)c * 16))[i] << (16 * (i & 1));
            }
        }
        return w;
    };
    const int64_t actions = a.w.rows, first = ((int64_t)blockIdx.x * (kNT / kWave) + wave) * 16;
    u4_a2 w[U];
    auto load_w = [&](int64_t v0, int s0) __attribute__((always_inline)) {
        const uint8_t* p = (const uint8_t*)a.w.p + (v0 + r < actions ? v0 + r : actions - 1) * a.w.ld * ES;
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = load(p, 4 * (s0 + u) + blk);
    };
    load_w(first, 0);  // on their way while hidden comes to LDS
    for (int e = threadIdx.x; e < rows * steps * 4; e += kNT) {
        const int row = e / (steps * 4), c = e - row * (steps * 4);
        const u4_a2 x = load((const uint8_t*)a.h.p + row * a.h.ld * ES, c);
        *(uint4*)(lds + row * pitch + c * 16) = uint4{x[0], x[1], x[2], x[3]};
    }
    __syncthreads();
    const int32_t t = r < rows ? a.taken[r] : -1;
    Soft soft{kNone, 0.f};
    for (int64_t v0 = first; v0 < actions; v0 += (int64_t)gridDim.x * (kNT / kWave) * 16) {
        float bias[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) bias[e] = a.bias && v0 + 4 * blk + e < actions ? a.bias[v0 + 4 * blk + e] * kLog2e : 0.f;
        mm_f4 acc = {0.f, 0.f, 0.f, 0.f};
        for (int s0 = 0; s0 < steps; s0 += U) {
            if (v0 != first || s0) load_w(v0, s0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (s0 + u >= steps) break;
                const uint4 x = r < rows ? *(const uint4*)(lds + r * pitch + (s0 + u) * 64 + 16 * blk) : uint4{0u, 0u, 0u, 0u};
                const uint4 y = uint4{w[u][0], w[u][1], w[u][2], w[u][3]};
                if constexpr (DT == IQLH_F32) {
                    const float xs[4] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w)};
                    const float ys[4] = {__uint_as_float(y.x), __uint_as_float(y.y), __uint_as_float(y.z), __uint_as_float(y.w)};
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(ys[i], xs[i], acc, 0, 0, 0);
                } else if constexpr (DT == IQLH_BF16) {
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(mm_b8, y), __builtin_bit_cast(mm_b8, x), acc, 0, 0, 0);
                } else {
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(mm_h8, y), __builtin_bit_cast(mm_h8, x), acc, 0, 0, 0);
                }
            }
        }
        // lane: row r of hidden, actions v0 + 4 blk + e
        Soft one{kNone, 0.f};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            acc[e] = v0 + 4 * blk + e < actions ? fmaf(acc[e], kLog2e, bias[e]) : kNone;
            one.m = fmaxf(one.m, acc[e]);
            if (t >= 0 && v0 + 4 * blk + e == t && t < actions) a.z_taken[r] = acc[e];
        }
        const float top = one.m == kNone ? 0.f : one.m;
#pragma unroll
        for (int e = 0; e < 4; ++e) one.s += __builtin_amdgcn_exp2f(acc[e] - top);
        soft.join(one);
    }
    soft = soft_xor(soft_xor(soft, 16), 32);
    if (lane < 16) waves[wave][lane] = soft;
    __syncthreads();
    if ((int)threadIdx.x < rows) {
        Soft v = waves[0][threadIdx.x];
#pragma unroll
        for (int k = 1; k < kNT / kWave; ++k) v.join(waves[k][threadIdx.x]);
        a.part[(int64_t)blockIdx.x * rows + threadIdx.x] = v;
    }
}
int64_t few_rows_bytes(int64_t rows, int64_t dim, int dtype) { return rows * ((dim * (dtype == IQLH_F32 ? 4 : 2) + 63) / 64 * 64 + 16); }

}  // namespace

// The head's weights in 64 KB of LDS: 16 actions of 1024 elements.  Loss and gradients, fp32, dim 128, against tiles:
// 16 actions, 16384 rows 49 us against 126, 64 rows 34 against 55.
bool policy_few_actions_ok(int64_t actions, int64_t dim) { return actions <= 16 && few_vm(actions) * up8(dim) <= 16384; }
// Hidden in 128 KB.  Loss of 65536 actions, dim 512, bf16, against tiles: one row 22.6 us against 23.8, 16 rows 26.8
// against 28.3; where the tiles would need W in another layout (fp32, odd widths) that pass is saved too.
constexpr int kFewRowsBytes = 128 << 10;
bool policy_few_rows_ok(int64_t rows, int64_t dim, int dtype) { return rows <= 16 && few_rows_bytes(rows, dim, dtype) <= kFewRowsBytes; }
int policy_few_rows_parts(int64_t actions) {
    const int64_t n = (actions + 63) / 64;
    return (int)(n < 1024 ? n : 1024);
}

// Workgroups along the rows: four rows a 16 lanes, 512 at most
static int few_blocks(int64_t rows) {
    const int64_t n = (rows + 4 * kGroups - 1) / (4 * kGroups);
    return (int)(n < 512 ? n : 512);
}
size_t policy_few_actions_bytes(int64_t rows, int64_t actions, int64_t dim) {
    const int vm = few_vm(actions);
    return (size_t)rows * vm * 4 + (size_t)few_blocks(rows) * vm * (up8(dim) + 1) * 4 + 256;
}
static int few_loss_blocks(int64_t rows) {
    const int64_t n = (rows + kGroups - 1) / kGroups;
    return (int)(n < 2048 ? n : 2048);
}

static FewArgs few_args(const PolicyArgs& a, void* work) {
    FewArgs q{};
    q.h = a.h, q.w = a.w, q.bias = a.bias, q.lse = a.lse_in;
    q.d_hidden = a.d_hidden, q.d_weight = a.d_weight, q.d_bias = a.d_bias, q.ld_dh = a.ld_dh, q.ld_dw = a.ld_dw;
    q.blocks = few_blocks(a.h.rows);
    q.g = (float*)work;
    q.part = q.g + (a.h.rows * few_vm(a.w.rows) + 63) / 64 * 64;
    q.f.taken = a.taken, q.f.row_weights = a.row_weights, q.f.nll = a.nll, q.f.lse = a.lse_out, q.f.loss = a.loss;
    q.f.flags = a.flags, q.f.rows = a.h.rows, q.f.actions = a.w.rows, q.f.scale = a.scale;
    return q;
}

// the weights' 64 KB and the sums beside them
static void allow_weights(void (*kernel)(FewArgs)) {
    (void)hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, 64 << 10);
}

hipError_t launch_policy_few_actions(const PolicyArgs& a, double* loss_part, int* parts, hipStream_t stream) {
    FewArgs q = few_args(a, nullptr);
    q.f.loss_part = loss_part;
    const int n = few_loss_blocks(a.h.rows);
    *parts = n;
    return by_actions(a.w.rows, [&](auto vm) {
        constexpr int VM = decltype(vm)::value;
        allow_weights(policy_few_actions_kernel<VM, false>);
        hipLaunchKernelGGL((policy_few_actions_kernel<VM, false>), dim3(n), dim3(kNT), VM * up8(a.h.cols) * 4, stream, q);
    });
}

hipError_t launch_policy_few_actions_grad(const PolicyArgs& a, void* work, hipStream_t stream) {
    const FewArgs q = few_args(a, work);
    const uint32_t chunks = (uint32_t)((a.h.cols + 127) / 128);
    return by_actions(a.w.rows, [&](auto vm) {
        constexpr int VM = decltype(vm)::value;
        allow_weights(policy_few_actions_kernel<VM, true>);
        hipLaunchKernelGGL((policy_few_actions_kernel<VM, true>), dim3(few_loss_blocks(a.h.rows)), dim3(kNT), VM * up8(a.h.cols) * 4,
                           stream, q);
        hipLaunchKernelGGL(policy_few_grads_kernel<VM>, dim3(q.blocks, chunks), dim3(kNT), 0, stream, q);
        if (q.d_weight || q.d_bias)
            hipLaunchKernelGGL(policy_few_join_kernel<VM>, dim3((uint32_t)a.w.rows, chunks), dim3(kNT), 0, stream, q);
    });
}

hipError_t launch_policy_few_rows(const PolicyArgs& a, void* part, float* z_taken, hipStream_t stream) {
    const FewRowsArgs q{a.h, a.w, a.bias, a.taken, (Soft*)part, z_taken};
    const int bytes = (int)few_rows_bytes(a.h.rows, a.h.cols, a.h.dtype);
    auto launch = [&](auto dt) {
        auto kernel = policy_few_rows_kernel<decltype(dt)::value>;
        (void)hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, kFewRowsBytes);
        hipLaunchKernelGGL(kernel, dim3(policy_few_rows_parts(a.w.rows)), dim3(kNT), bytes, stream, q);
    };
    if (a.h.dtype == IQLH_F32) launch(std::integral_constant<int, IQLH_F32>());
    else if (a.h.dtype == IQLH_BF16) launch(std::integral_constant<int, IQLH_BF16>());
    else launch(std::integral_constant<int, IQLH_F16>());
    return hipGetLastError();
}

}  // namespace iqlh
