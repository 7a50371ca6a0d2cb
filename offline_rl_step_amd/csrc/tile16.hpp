// Products of 16-bit matrices on the matrix instructions, one tile of outputs a
// workgroup:  acc[m][n] = sum_k a(m, k) b(n, k), sums in binary32.
//
// An operand is binary16 or bfloat16 and lies either with its summed axis
// along the rows (a(i, k) at p[i ld + k]) or along the columns (p[k ld + i]): rows are
// read from LDS as they are, columns through the transposing LDS read, so no
// operand is ever transposed in memory.
//
// An operand that stands for binary32 values is two binary16 matrices (planes):
// x = (hi + lo) 2^-s, hi the nearest binary16 to 2^s x and lo the nearest to the rest,
// 22 bits together.  A product of two such operands is three products, lo hi + hi lo + hi
// hi (lo lo lies below the last bit): 2.5 PF / 3 against the 0.16 PF of the binary32
// matrix instructions.  The planes lie in one matrix of twice the row length, 32 elements of hi and their 32
// of lo in turn, so that a step of 32 k reads whole cache lines.
#pragma once
#include <type_traits>

#include "lds_copy.hpp"

namespace iqlh {

// copy16 from a uniform address plus a lane's offset
IQLH_DEV void copy16(const void* base, uint32_t off, uint32_t lds_at) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(lds_at), "v"(off), "s"(base) : "memory");
}

typedef float mm_f16 __attribute__((ext_vector_type(16)));
typedef _Float16 mm_h8 __attribute__((ext_vector_type(8)));
typedef __bf16 mm_b8 __attribute__((ext_vector_type(8)));

// One operand.  n: bound of i (rows: the last row is read again behind it; columns: another element, n a
// multiple of 8).  p 16-byte aligned, ld a multiple of 8, of 64 with two planes.  plane: elements to a second
// matrix that holds what this one rounds off (tile_product's `both`).
struct Side16 {
    const uint16_t* p;
    int64_t plane, ld, n;
};
// Place of element (row, col) of two planes, ld columns; that of the rest is 32 elements behind
IQLH_DEV int64_t planes_at(int64_t row, int64_t ld, int64_t col) { return 2 * (row * ld + col) - (col & 31); }

template <bool BRAIN>
IQLH_DEV mm_f16 mma16(uint4 a, uint4 b, mm_f16 c) {
    if constexpr (BRAIN)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(mm_b8, a), __builtin_bit_cast(mm_b8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(mm_h8, a), __builtin_bit_cast(mm_h8, b), c, 0, 0, 0);
}

// TILE 256: eight waves, 2 x 4, each 128 x 64 outputs (4 x 2 fragments of 32 x 32).  TILE 128 and 64: four
// waves, 2 x 2, each 64 x 64 or 32 x 32; two workgroups to a compute unit.
template <int TILE, int PL = 1, int STEPS = TILE == 64 ? 4 : 2>
struct Tile16 {
    static constexpr int WM = 2, WN = TILE == 256 ? 4 : 2;          // waves
    static constexpr int FA = TILE / 32 / WM, FB = TILE / 32 / WN;  // fragments of 32 x 32 of a wave
    static constexpr int NT = 64 * WM * WN;
    static constexpr int BK = PL == 2 ? 32 : 64;  // k of a step
    static constexpr int SIDE = TILE * 128;       // one operand in a step
    static constexpr int STAGE = 2 * SIDE;
    static constexpr int CP = SIDE / 16 / NT;     // copies of a thread, operand and step
    static constexpr int NB = STEPS;              // steps in LDS, a power of two
    static constexpr int RING = NB * STAGE;       // also the staged sums of BAND rows
    static constexpr int LDS = RING + 28 * TILE;  // and what an epilogue keeps of rows and columns meanwhile
    static constexpr int BANDS = TILE == 256 ? 2 : 1, BAND = TILE / BANDS;
    static constexpr int PER_CU = RING > 64 << 10 ? 1 : 2, PER_SIMD = PER_CU * NT / 256;
    static_assert(BAND * TILE * 4 <= RING && PER_CU * LDS <= 160 * 1024, "LDS of a compute unit");
};

// Position of this wave's outputs in the tile
template <int TILE> IQLH_DEV int wave_m() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / Tile16<TILE>::WN * (32 * Tile16<TILE>::FA); }
template <int TILE> IQLH_DEV int wave_n() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % Tile16<TILE>::WN * (32 * Tile16<TILE>::FB); }

// The sums over k in [k0, k1): multiples of 64 but for k1, which is one of 8 for operands in rows.  PL 2: operands
// of two planes, binary16.  both: a's second matrix and a, each times b.  Lane l: acc[i][j][4 g + e] is m =
// wave_m + 32 i + (l & 31), n = wave_n + 32 j + 8 g + 4 (l >> 5) + e.  Every step of 16 k is added in
// the same order whatever the tile.  When it returns, the ring in LDS is free.
//
// NB steps in LDS, filled by asynchronous copies: in its last part of 16 k step s waits
// for the copies of step s + 1, passes the barrier (behind which all reads of its own buffer are
// done), issues those of step s + NB into that buffer and reads the first fragments of
// step s + 1 while the part's matrix instructions run.  The copies are made one at a time between the matrix
// instructions of that part and of the next step's first one; those of a 64 tile, which has few of either, at once
// (512 x 512 x 256 in two planes 9.7 against 11 us; 8192 x 65536 x 2048 / 4 on 256 tiles 499 against 528).
// Rows: 128 bytes of a row, a whole cache line, its 16-byte chunk u at u ^ ((row >> 1) & 7), so that 16
// lanes' reads fall on all banks.  Columns: TILE elements of one k, chunk u at u ^ 4 (k
// & 3) (rows of 128 bytes: u ^ 2 (k & 2)): a transposing read takes 4 k of 16 neighbouring elements in 16 lanes, 32 lanes
// all banks.
template <bool BRAIN, int TILE, bool AC, bool BC, int PL = 1, int STEPS = Tile16<TILE>::NB>
IQLH_DEV void tile_product(const Side16& a, const Side16& b, int64_t m0, int64_t n0, int64_t k0, int64_t k1, bool both,
                           uint8_t* lds, mm_f16 (&acc)[Tile16<TILE>::FA][Tile16<TILE>::FB]) {
    typedef Tile16<TILE, PL, STEPS> T;
    constexpr int NT = T::NT, FA = T::FA, FB = T::FB, BK = T::BK, CP = T::CP, NB = T::NB;
    constexpr int CPR = PL * TILE / 8, KR = NT / CPR, PARTS = BK / 16;
    auto col_mix = [](int k) __attribute__((always_inline)) { return CPR == 8 ? 2 * (k & 2) : 4 * (k & 3); };
    static_assert(CP * KR == BK && CP * (NT / 8) == TILE, "copies of a step");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 31, h = lane >> 5, li = lane & 15, half = lane >> 4 & 1;
    const uint32_t lds_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    const int per = (int)((k1 - k0 + BK - 1) / BK), steps = both ? 2 * per : per;
    // what a thread copies: chunk i NT + tid of a side
    const int ru = (tid & 7) ^ ((tid >> 4) & 7), rk = 8 * (PL == 2 ? ru & 3 : ru);  // rows: chunk of the row, its k
    const int ck = tid / CPR, cu = (tid % CPR) ^ col_mix(ck);                  // columns: k, chunk of it
    const int ci = PL == 2 ? cu / 8 * 32 + (cu & 3) * 8 : cu * 8;
    auto offset = [&](const Side16& s, bool cols, int64_t i0, int i) __attribute__((always_inline)) -> uint32_t {
        if (cols) return (uint32_t)((KR * i + ck) * s.ld * (2 * PL)) + 16u * (i0 + ci < s.n ? cu : 0);
        const int row = i * (NT / 8) + (tid >> 3);
        const int64_t left = s.n - i0 - 1;
        return (uint32_t)((row < left ? row : (int)left) * s.ld * (2 * PL)) + 16u * ru;
    };
    uint32_t offa[CP], offb[CP];
#pragma unroll
    for (int i = 0; i < CP; ++i) {
        offa[i] = offset(a, AC, m0, i);
        offb[i] = offset(b, BC, n0, i);
    }
    // the copies of one step: `next` takes it up, `copy` makes copy c of 2 CP, b's first
    int step_in = 0;
    bool rest = both;
    const uint8_t *pa = nullptr, *pb = nullptr;
    uint32_t dst = 0u;
    int64_t kk = 0;
    bool there = false, whole = false;
    auto next = [&](int s) __attribute__((always_inline)) {
        there = s < steps;
        dst = lds_at + (s & (NB - 1)) * T::STAGE + wave * 1024;
        kk = k0 + (int64_t)step_in * BK;
        whole = there && kk + BK <= k1;
        pb = (const uint8_t*)(b.p + PL * (BC ? kk * b.ld + n0 : n0 * b.ld + kk));
        pa = (const uint8_t*)(a.p + (rest ? a.plane : 0) + PL * (AC ? kk * a.ld + m0 : m0 * a.ld + kk));
        if (++step_in == per) step_in = 0, rest = false;
    };
    auto copy = [&](int c) __attribute__((always_inline)) {
        if (c < CP) copy16(pb, offb[c], dst + c * NT * 16);
        else copy16(pa, offa[c - CP], dst + c * NT * 16);
    };
    auto copy_edge = [&](int c) __attribute__((always_inline)) {  // zeros behind k1
        const bool cols = c < CP ? BC : AC;
        const bool in = cols ? kk + KR * (c % CP) + ck < k1 : kk + rk < k1;
        copy16(in ? (c < CP ? pb + offb[c] : pa + offa[c - CP]) : (const uint8_t*)kZeroChunk, dst + c * NT * 16);
    };
    auto issue = [&](int s) __attribute__((always_inline)) {
        next(s);
        if (whole) {
#pragma unroll
            for (int c = 0; c < 2 * CP; ++c) copy(c);
        } else if (there) {
#pragma unroll
            for (int c = 0; c < 2 * CP; ++c) copy_edge(c);
        }
    };
    const int wm = wave / T::WN * (32 * FA), wn = wave % T::WN * (32 * FB);
    // where a lane reads: rows, the row's start (the chunk goes by the part); columns, the fragment's chunk of the lane's k
    auto col_at = [&](int i0) __attribute__((always_inline)) {
        return (8 * h + (li >> 2)) * (2 * PL * TILE) + 16 * ((PL * i0 / 8 + 2 * half + ((li & 3) >> 1)) ^ col_mix(li >> 2)) + 8 * (li & 1);
    };
    int ca[FA], cb[FB];
#pragma unroll
    for (int i = 0; i < FA; ++i) ca[i] = T::SIDE + (AC ? col_at(wm + 32 * i) : (wm + 32 * i + r) * 128);
#pragma unroll
    for (int i = 0; i < FB; ++i) cb[i] = BC ? col_at(wn + 32 * i) : (wn + 32 * i + r) * 128;
    struct Frags {
        uint4 a[PL][FA], b[PL][FB];
    } f[2];
    typedef short s4 __attribute__((ext_vector_type(4)));
    auto read = [&](const uint8_t* buf, int at, auto cols, auto part, int p) __attribute__((always_inline)) -> uint4 {
        constexpr int Q = decltype(part)::value;
        if constexpr (decltype(cols)::value) {
            typedef __attribute__((address_space(3))) s4 lds_s4;
            const uint8_t* q = buf + (at ^ (p * 64)) + Q * (32 * PL * TILE);  // the rest: 4 chunks on
            const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)q);
            const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(q + 8 * PL * TILE));
            const uint2 l = __builtin_bit_cast(uint2, lo), u = __builtin_bit_cast(uint2, hi);
            return uint4{l.x, l.y, u.x, u.y};
        } else {
            return *(const uint4*)(buf + at + 16 * ((2 * Q + h + 4 * p) ^ ((r >> 1) & 7)));
        }
    };
    typedef std::integral_constant<bool, AC> CA;
    typedef std::integral_constant<bool, BC> CB;
    constexpr int FRAGS = PL * (FA + FB), MMAS = FA * FB * (PL == 2 ? 3 : 1);
    // fragment e of a part: the smaller plane's first, b's before a's
    auto load_one = [&](const uint8_t* buf, int e, auto part, auto set) __attribute__((always_inline)) {
        Frags& g = f[decltype(set)::value];
        const int p = PL - 1 - e / (FA + FB), i = e % (FA + FB);
        if (i < FB) g.b[p][i] = read(buf, cb[i], CB(), part, p);
        else g.a[p][i - FB] = read(buf, ca[i - FB], CA(), part, p);
    };
    auto mma_one = [&](int e, auto set) __attribute__((always_inline)) {
        const Frags& g = f[decltype(set)::value];
        const int t = PL == 2 ? e / (FA * FB) : 2, i = e / FB % FA, j = e % FB;  // lo hi, hi lo, hi hi
        acc[i][j] = mma16<BRAIN>(g.b[t == 1][j], g.a[t == 0][i], acc[i][j]);
    };
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j) acc[i][j] = mm_f16{};
    // A part's matrix instructions, with the LDS reads of part `load` of step s and a half of the copies taken up
    // (0 the first, 1 the second, 2 none) between them: neither LDS nor the path of the copies
    // takes more than one wave's at a time, and what waits for either holds up the wave.
    auto run = [&](int s, auto load, auto load_set, auto set, auto copies) __attribute__((always_inline)) {
        constexpr int H = decltype(copies)::value;
        const uint8_t* buf = lds + (s & (NB - 1)) * T::STAGE;
        if (H < 2 && there && !whole) {
#pragma unroll
            for (int c = 0; c < CP; ++c) copy_edge(H * CP + c);
        }
#pragma unroll
        for (int e = 0; e < MMAS; ++e) {
#pragma unroll
            for (int x = e * FRAGS / MMAS; x < (e + 1) * FRAGS / MMAS; ++x) load_one(buf, x, load, load_set);
            mma_one(e, set);
            if (H < 2 && e * CP / MMAS < (e + 1) * CP / MMAS && whole) {
#pragma unroll
                for (int c = e * CP / MMAS; c < (e + 1) * CP / MMAS; ++c) copy(H * CP + c);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    typedef std::integral_constant<int, 0> C0;
    typedef std::integral_constant<int, 1> C1;
    typedef std::integral_constant<int, 2> C2;
    typedef std::integral_constant<int, 3> C3;
    // the copies of step s are here; those of the NB - 2 steps behind it may be on their way
    auto landed = [&](int s) __attribute__((always_inline)) {
        if (NB == 2 || s + NB - 2 >= steps) wait_vm<0>();
        else wait_vm<(NB - 2) * 2 * CP>();
        bar();
    };
#pragma unroll
    for (int i = 0; i < NB - 1; ++i) issue(i);
    landed(0);
    issue(NB - 1);
    there = whole = false;  // all made
#pragma unroll
    for (int e = 0; e < FRAGS; ++e) load_one(lds, e, C0(), C0());
    for (int s = 0; s < steps; ++s) {
        run(s, C1(), C1(), C0(), C1());
        if constexpr (PARTS == 4) {
            run(s, C2(), C0(), C1(), C2());
            run(s, C3(), C1(), C0(), C2());
        }
        landed(s + 1);
        if constexpr (TILE == 64) {
            issue(s + NB);
            there = whole = false;
        } else {
            next(s + NB);
        }
        run(s + 1, C0(), C0(), C1(), C0());
    }
    wait_vm<0>();  // the copies behind the last step, before their buffers are used again
    bar();
}

// ------------------------------------------------------- staged sums
// A band of BAND rows of the tile's sums in LDS as binary32, rows of TILE: the 16
// bytes of columns 4 q .. of row m lie at place q ^ g(m), so that the waves' writes (32
// rows, one q), reads along rows and reads down columns (16 blocks of 8 rows, one q)
// each fall on all banks.
IQLH_DEV int stage_mix(int m) { return ((m >> 3) ^ ((m & 7) << 1)) & 15; }
template <int TILE>
IQLH_DEV float4* stage_at(uint8_t* lds, int m, int q) {
    return (float4*)(lds + (m * (TILE / 4) + (q ^ stage_mix(m))) * 16);
}
template <int TILE>
IQLH_DEV void stage_band(const mm_f16 (&acc)[Tile16<TILE>::FA][Tile16<TILE>::FB], uint8_t* lds, int band) {
    typedef Tile16<TILE> T;
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int wm = wave_m<TILE>(), wn = wave_n<TILE>();
    if (band) __syncthreads();
    if (T::BANDS == 1 || wm / T::BAND == band) {
#pragma unroll
        for (int i = 0; i < T::FA; ++i)
#pragma unroll
            for (int j = 0; j < T::FB; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    *stage_at<TILE>(lds, (T::BANDS == 1 ? wm : 0) + 32 * i + r, (wn + 32 * j) / 4 + 2 * g + h) =
                        float4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
    }
    __syncthreads();
}

// -------------------------------------------------------- element types
// Eight neighbouring elements, the first `n` of them (n >= 1; the others 0)
// there; any alignment of whole elements.
IQLH_DEV float half_of(uint32_t w, int odd) { return (float)__builtin_bit_cast(_Float16, (uint16_t)(odd ? w >> 16 : w)); }
IQLH_DEV float brain_of(uint32_t w, int odd) { return __uint_as_float(odd ? w & 0xFFFF0000u : w << 16); }
IQLH_DEV uint32_t pack_half(float a, float b) {
    return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)a) | (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)b) << 16;
}
// Two values as 16-bit ones, rounded to nearest, and back
typedef __bf16 b2_16 __attribute__((ext_vector_type(2)));
typedef float f2_16 __attribute__((ext_vector_type(2)));
template <bool BRAIN>
IQLH_DEV uint32_t pack16(float a, float b) {
    if constexpr (BRAIN) return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2_16{a, b}, b2_16));
    else return pack_half(a, b);
}
template <bool BRAIN>
IQLH_DEV float of16(uint32_t w, int odd) { return BRAIN ? brain_of(w, odd) : half_of(w, odd); }
typedef uint32_t u4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u4_a2 __attribute__((ext_vector_type(4), aligned(2)));
IQLH_DEV void load8_of(int dtype, const void* base, int64_t at, int64_t n, float (&v)[8]) {
    if (dtype == IQLH_F32) {
        const float* p = (const float*)base + at;
        if (n >= 8) {
            const u4_a4 x = *(const u4_a4*)p, y = *(const u4_a4*)(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = __uint_as_float(x[i]);
                v[4 + i] = __uint_as_float(y[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
        }
        return;
    }
    const uint16_t* p = (const uint16_t*)base + at;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (n >= 8) {
        const u4_a2 x = *(const u4_a2*)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = x[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = dtype == IQLH_BF16 ? brain_of(w[i >> 1], i & 1) : half_of(w[i >> 1], i & 1);
}
IQLH_DEV void store8_of(int dtype, void* base, int64_t at, int64_t n, const float (&v)[8]) {
    if (dtype == IQLH_F32) {
        float* p = (float*)base + at;
        if (n >= 8) {
            u4_a4 x, y;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = __float_as_uint(v[i]);
                y[i] = __float_as_uint(v[4 + i]);
            }
            *(u4_a4*)p = x;
            *(u4_a4*)(p + 4) = y;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) p[i] = v[i];
        }
        return;
    }
    uint16_t* p = (uint16_t*)base + at;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = dtype == IQLH_BF16 ? pack_bf2(v[2 * i], v[2 * i + 1]) : pack_half(v[2 * i], v[2 * i + 1]);
    if (n >= 8) {
        *(u4_a2*)p = u4_a2{w[0], w[1], w[2], w[3]};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
}

// Eight values of row `row`, columns col.. (col a multiple of 8), of a binary16 matrix of one or two
// planes.  A value that is not finite has no rest.
IQLH_DEV void put_planes(uint16_t* base, int64_t row, int64_t ld, int64_t col, bool two, const float (&v)[8]) {
    uint16_t* p = base + (two ? planes_at(row, ld, col) : row * ld + col);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        hi[i] = pack_half(v[2 * i], v[2 * i + 1]);
        if (two) {
            const float a = v[2 * i] - half_of(hi[i], 0), b = v[2 * i + 1] - half_of(hi[i], 1);
            lo[i] = pack_half(a == a ? a : 0.f, b == b ? b : 0.f);
        }
    }
    *(uint4*)p = uint4{hi[0], hi[1], hi[2], hi[3]};
    if (two) *(uint4*)(p + 32) = uint4{lo[0], lo[1], lo[2], lo[3]};
}
IQLH_DEV void get_planes(const uint16_t* base, int64_t row, int64_t ld, int64_t col, bool two, float (&v)[8]) {
    const uint16_t* p = base + (two ? planes_at(row, ld, col) : row * ld + col);
    const uint4 h = *(const uint4*)p;
    const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = half_of(hw[i >> 1], i & 1);
    if (two) {
        const uint4 l = *(const uint4*)(p + 32);
        const uint32_t lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += half_of(lw[i >> 1], i & 1);
    }
}

}  // namespace iqlh
