// Rows of a float matrix quantised into LDS, and their products with a matrix
// in 4 bits read from L2: the parts of the one-launch linear kernel and of the
// value network's.
#pragma once
#include "mx4_block.hpp"

namespace iqlh {

// ROWS rows and NT threads a workgroup
constexpr int kChunk = 32;    // rows of b a wave takes at a time
constexpr int kFrags = kChunk / 16;
constexpr int kRowsMaxBlocks = 32;  // K <= 1024

// ROWS rows of kb4 blocks in LDS, kb4 a multiple of 4: codes, 16 bytes more
// than they take between two rows so that the 16 lanes of a fragment column
// fall on different banks, then the scales.
__host__ __device__ constexpr int mx4_lds_row(int kb4) { return kb4 * 16 + 16; }
template <int ROWS>
__host__ __device__ constexpr int mx4_lds_bytes(int kb4) { return ROWS * (mx4_lds_row(kb4) + kb4); }
template <int ROWS>
struct LdsRows {
    uint8_t* codes;
    uint8_t* scales;
    int kb4, rb;
    IQLH_DEV LdsRows(uint8_t* at, int kb4_) : codes(at), scales(at + ROWS * mx4_lds_row(kb4_)), kb4(kb4_), rb(mx4_lds_row(kb4_)) {}
};

// Rows m0 .. m0 + ROWS - 1 of x [M][ld], `cols` wide (rows past the end: the
// last one), quantised into t.  A thread converts 8 elements at a time, four
// neighbouring lanes a block.
template <int ROWS, int NT, int XDT>
IQLH_DEV void mx4_rows_to_lds(const typename MxFloat<XDT>::type* x, int64_t ld, int64_t M, int64_t m0, int64_t cols,
                              const LdsRows<ROWS>& t) {
    const int gpr = t.kb4 * 4;  // groups of 8 a row, a multiple of 16
    constexpr int U = XDT == IQLH_F32 ? 4 : 8;  // groups in flight per thread: 128 bytes
    for (int g0 = threadIdx.x; g0 < ROWS * gpr; g0 += NT * U) {
        Eight<XDT> raw[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int e = g0 + i * NT, row = e / gpr, g = e - row * gpr;
            const int64_t m = m0 + row < M ? m0 + row : M - 1;
            const int64_t left = e < ROWS * gpr ? cols - g * 8 : 0;
            raw[i].load(x + m * ld + g * 8, (int)(left < 0 ? 0 : left < 8 ? left : 8));
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int e = g0 + i * NT, row = e / gpr, g = e - row * gpr;
            if (e >= ROWS * gpr) break;  // the same for the whole workgroup: ROWS gpr is a multiple of NT
            float v[8];
            raw[i].get(v);
            uint32_t amax = 0u;
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = umax2(amax, abs_bits(v[j]));
            const uint32_t s = mx4_scale(quad_umax(amax));
            *(uint32_t*)(t.codes + row * t.rb + g * 4) = s == 255u ? 0u : mx4_codes8(v, mx4_inverse(s));
            if ((g & 3) == 0) t.scales[row * t.kb4 + (g >> 2)] = (uint8_t)s;
        }
    }
}

// b in memory as its rows, of 32-bit extent
struct RowsOfB {
    Mx4Mat q;
    struct Step {
        uint4 v;
        uint32_t s;
    };
    IQLH_DEV void load(int64_t n0, int step, int lane, Step& f) const {
        const uint32_t n = (uint32_t)n0 + (lane & 15), kb = (uint32_t)q.kb(), block = step * 4 + (lane >> 4);
        const bool in = block < kb;
        const uint32_t at = (n < (uint32_t)q.rows ? n : (uint32_t)q.rows - 1) * kb + (in ? block : 0u);
        const uint4 v = *(const uint4*)(q.codes + at * 16u);
        const uint32_t keep = in ? 0xFFFFFFFFu : 0u;  // zeros of scale 1 behind the last block
        f.v = uint4{v.x & keep, v.y & keep, v.z & keep, v.w & keep};
        f.s = in ? q.scales[at] : 127u;
    }
    static IQLH_DEV uint32_t scale(const Step& f, int step) { return f.s; }
};

// b regrouped by fragments: the codes of 16 rows and a step as the 64 lanes
// hold them (1 KB in 16 lookups of the L1, not the 64 of a fragment of 16 rows,
// and the scale bytes' 64 more), and one dword of scales per lane for four
// steps, byte s & 3 that of step s.  Rows are padded to a multiple of 128, blocks
// to whole steps, with zeros.
struct FragsOfB {
    const uint4* codes;      // [rows128 / 16][steps][64]
    const uint32_t* scales;  // [rows128 / 16][(steps + 3) / 4][64]
    int steps;
    struct Step {
        uint4 v;
        uint32_t s;
    };
    IQLH_DEV void load(int64_t n0, int step, int lane, Step& f) const {
        f.v = codes[(n0 / 16 * steps + step) * 64 + lane];
        f.s = scales[(n0 / 16 * ((steps + 3) / 4) + step / 4) * 64 + lane];
    }
    static IQLH_DEV uint32_t scale(const Step& f, int step) { return f.s >> (8 * (step & 3)); }
};
__host__ __device__ inline int64_t mx4_frag_groups(int64_t rows) { return (rows + 127) / 128 * 8; }
__host__ __device__ inline int64_t mx4_frag_code_bytes(int64_t rows, int64_t kb) {
    return mx4_frag_groups(rows) * ((kb + 3) / 4) * 1024;
}
__host__ __device__ inline int64_t mx4_frag_scale_bytes(int64_t rows, int64_t kb) {
    return mx4_frag_groups(rows) * ((kb + 15) / 16) * 256;
}
// where the lane's scale byte of (16-row group, step) lies
IQLH_DEV int64_t mx4_frag_scale_at(int64_t group, int64_t step, int64_t steps, int lane) {
    return ((group * ((steps + 3) / 4) + step / 4) * 64 + lane) * 4 + (step & 3);
}

// For the chunks n0 = 32 wave, + 32 waves, .. below n_end: acc[i][j] (rows 16 i + (lane
// & 15) of t, rows n0 + 16 j + 4 (lane >> 4) + 0..3 of b) = the products' sums, then
// done(n0, acc).  b's fragments are loaded one step ahead, over the chunks'
// ends too; first(n0) runs before a chunk's steps (loads for done).
template <int ROWS, int NT, class B, class First, class Done>
IQLH_DEV void mx4_rows_chunks(const LdsRows<ROWS>& t, const B& b, int64_t n_end, First&& first, Done&& done) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, blk = lane >> 4;
    const int steps = t.kb4 / 4;
    typename B::Step bn[kFrags];
    auto fetch = [&](int64_t n0, int s) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < kFrags; ++j) b.load(n0 + 16 * j, s, lane, bn[j]);
    };
    if (wave * kChunk < n_end) fetch(wave * kChunk, 0);
    for (int64_t n0 = (int64_t)wave * kChunk; n0 < n_end; n0 += NT / 64 * kChunk) {
        first(n0);
        mx_f4 acc[ROWS / 16][kFrags];
#pragma unroll
        for (int i = 0; i < ROWS / 16; ++i)
#pragma unroll
            for (int j = 0; j < kFrags; ++j) acc[i][j] = mx_f4{0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < steps; ++s) {
            uint4 bv[kFrags], av[ROWS / 16];
            uint32_t bs[kFrags], as[ROWS / 16];
#pragma unroll
            for (int j = 0; j < kFrags; ++j) {
                bv[j] = bn[j].v;
                bs[j] = B::scale(bn[j], s);
            }
            if (s + 1 < steps) fetch(n0, s + 1);
            else if (n0 + NT / 64 * kChunk < n_end) fetch(n0 + NT / 64 * kChunk, 0);
#pragma unroll
            for (int i = 0; i < ROWS / 16; ++i) {
                av[i] = *(const uint4*)(t.codes + (16 * i + r) * t.rb + (s * 4 + blk) * 16);
                as[i] = t.scales[(16 * i + r) * t.kb4 + s * 4 + blk];
            }
#pragma unroll
            for (int i = 0; i < ROWS / 16; ++i)
#pragma unroll
                for (int j = 0; j < kFrags; ++j) acc[i][j] = mx4_mma(bv[j], av[i], acc[i][j], bs[j], as[i]);
        }
        done(n0, acc);
    }
}

}  // namespace iqlh
