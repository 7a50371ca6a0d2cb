// Norm and clip of the gradients of a network held as a list of tensors.
//
//   norm = sqrt(sum_t sum_i x_ti^2)   (or max |x_ti|)
//   c    = max_norm / norm if norm > max_norm else 1,   x <- c x
//
// HBM-bound: the norm reads every element once, the clip once more (from the
// Infinity Cache where the set fits it) and writes it once.  The list is cut
// into pieces on the host (TensorPiece), so a workgroup streams whole pieces
// whatever the tensors' sizes are, and one launch serves any number of
// tensors and any mix of types.
//   1. norm pass: a workgroup takes the pieces b, b + grid, ..; block sums (and
//      with per-tensor norms each wave's sum of each piece) to the workspace,
//      added up by the workgroup that finishes last;
//   2. for many pieces a launch adds them up instead, with a workgroup per tensor
//      for the tensors' own norms;
//   3. for a clip the scale pass: every workgroup adds the block sums itself, in
//      the same order, and scales its pieces.
// No atomics on sums: every order is fixed, results repeat bit for bit.
//
// Measured: 12 tensors of two value networks, 66306 elements, 5.8 to 6.3 us in one launch;
// 537 MB of bf16 92 us, 5.8 TB/s, and 4.8 for the tensors' own norms; 1.07 GB of fp32
// into the flat vector 192 + 380 us, 5.6 TB/s of the three passes; in place, above the
// bound, 192 MB of fp16 28 + 58 us, 537 MB of bf16 290 and of fp32 286 together, 5.6 TB/s.
//
// Squares and sums are held in binary64: a product of two binary32 values is
// exact there, nothing overflows or vanishes (binary32 squares do from
// |x| = 1.8e19 up and 1e-23 down), and the norm does not depend on how the
// list is cut.  One conversion and one fma per element at half rate stay
// under the loads' time.
#include "common.hpp"
#include "iqlher.h"
#include "launch.hpp"

namespace iqlh {

namespace {

constexpr int kNT = 256;
constexpr int kAhead = 8;  // 16-byte loads in flight per thread
// most pieces whose sums, and tensors whose own norms, the last workgroup of the norm
// launch adds up (more: a launch of their own)
constexpr int kOnePieces = 256, kOneTensors = 64;

template <int DT> struct Elem;
template <> struct Elem<IQLH_F32> {
    typedef float type;
    static constexpr int kQ = 4;  // elements per 16 bytes
    static IQLH_DEV float get(uint4 q, int i) { return __uint_as_float((&q.x)[i]); }
    static IQLH_DEV float load(const void* p, int64_t i) { return ((const float*)p)[i]; }
    static IQLH_DEV void store(void* p, int64_t i, float v) { ((float*)p)[i] = v; }
    static IQLH_DEV uint4 pack(const float* v) {
        return uint4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    }
};
template <> struct Elem<IQLH_BF16> {
    typedef uint16_t type;
    static constexpr int kQ = 8;
    static IQLH_DEV float get(uint4 q, int i) {
        const uint32_t w = (&q.x)[i >> 1];
        return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
    }
    static IQLH_DEV float load(const void* p, int64_t i) { return bf2f(((const uint16_t*)p)[i]); }
    static IQLH_DEV void store(void* p, int64_t i, float v) { ((uint16_t*)p)[i] = f2bf(v); }
    static IQLH_DEV uint4 pack(const float* v) {
        return uint4{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7])};
    }
};
template <> struct Elem<IQLH_F16> {
    typedef _Float16 type;
    static constexpr int kQ = 8;
    static IQLH_DEV float get(uint4 q, int i) {
        const uint32_t w = (&q.x)[i >> 1];
        return (float)__builtin_bit_cast(_Float16, (uint16_t)(i & 1 ? w >> 16 : w));
    }
    static IQLH_DEV float load(const void* p, int64_t i) { return (float)((const _Float16*)p)[i]; }
    static IQLH_DEV void store(void* p, int64_t i, float v) { ((_Float16*)p)[i] = (_Float16)v; }
    static IQLH_DEV uint32_t pack2(float a, float b) {
        return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)a) |
               (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)b) << 16;
    }
    static IQLH_DEV uint4 pack(const float* v) {
        return uint4{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
    }
};

// Running value of a norm: the sum of squares, or the largest |x| as its
// bits (whose order is that of the values, NaN above infinity).
template <int KIND> struct Stat;
template <> struct Stat<IQLH_NORM_L2> {
    double s;
    IQLH_DEV Stat() : s(0.0) {}
    IQLH_DEV void add(float x) { s = fma((double)x, (double)x, s); }
    IQLH_DEV void join(uint64_t bits) { s += __longlong_as_double((long long)bits); }
    IQLH_DEV uint64_t bits() const { return (uint64_t)__double_as_longlong(s); }
    IQLH_DEV double norm() const { return sqrt(s); }
};
template <> struct Stat<IQLH_NORM_MAX> {
    uint32_t s;
    IQLH_DEV Stat() : s(0u) {}
    IQLH_DEV void add(float x) {
        const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
        s = b > s ? b : s;
    }
    IQLH_DEV void join(uint64_t bits) { s = (uint32_t)bits > s ? (uint32_t)bits : s; }
    IQLH_DEV uint64_t bits() const { return s; }
    IQLH_DEV double norm() const { return (double)__uint_as_float(s); }
};

// joined over 2 TOP neighbouring lanes, in all of them
template <int TOP, int KIND>
IQLH_DEV Stat<KIND> lanes_join(Stat<KIND> v) {
#pragma unroll
    for (int o = TOP; o > 0; o >>= 1) {
        const uint64_t b = v.bits();
        const uint32_t lo = __shfl_xor((uint32_t)b, o, kWave), hi = __shfl_xor((uint32_t)(b >> 32), o, kWave);
        v.join((uint64_t)hi << 32 | lo);
    }
    return v;
}

template <int KIND>
IQLH_DEV Stat<KIND> wave_join(Stat<KIND> v) { return lanes_join<32>(v); }

template <int KIND>
IQLH_DEV Stat<KIND> block_join(Stat<KIND> v, uint64_t* red) {
    v = wave_join(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x / kWave] = v.bits();
    __syncthreads();
    Stat<KIND> s;
#pragma unroll
    for (int i = 0; i < kNT / kWave; ++i) s.join(red[i]);
    return s;
}

// A piece as [head elements][nq whole 16-byte quads on a boundary][tail elements]
template <int DT>
struct Cut {
    int head, nq, tail;
    const uint4* q;
    IQLH_DEV explicit Cut(const TensorPiece& p) {
        const int to_edge = (int)((16u - (uint32_t)(p.ptr & 15u)) & 15u) / (int)sizeof(typename Elem<DT>::type);
        head = to_edge < p.n ? to_edge : p.n;
        nq = (p.n - head) / Elem<DT>::kQ;
        tail = p.n - head - nq * Elem<DT>::kQ;
        q = (const uint4*)(p.ptr + (uint64_t)head * sizeof(typename Elem<DT>::type));
    }
    // element index of the thread's edge element, or -1
    IQLH_DEV int edge() const {
        const int t = threadIdx.x;
        return t < head ? t : t < head + tail ? nq * Elem<DT>::kQ + t : -1;
    }
};

template <int DT, int KIND>
IQLH_DEV void piece_stat(const TensorPiece& p, Stat<KIND>& a0, Stat<KIND>& a1) {
    typedef Elem<DT> E;
    const Cut<DT> c(p);
    int i = threadIdx.x;
    for (; i + (kAhead - 1) * kNT < c.nq; i += kAhead * kNT) {
        uint4 x[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) x[k] = c.q[i + k * kNT];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int j = 0; j < E::kQ; ++j) (j & 1 ? a1 : a0).add(E::get(x[k], j));
    }
    for (; i < c.nq; i += kNT) {
        const uint4 x = c.q[i];
#pragma unroll
        for (int j = 0; j < E::kQ; ++j) (j & 1 ? a1 : a0).add(E::get(x, j));
    }
    const int e = c.edge();
    if (e >= 0) a0.add(E::load((const void*)p.ptr, e));
}

IQLH_DEV bool finite64(double x) { return fabs(x) < __longlong_as_double(0x7FF0000000000000ll); }

template <int KIND>
IQLH_DEV double norm_of_parts(const uint64_t* part, int nb, uint64_t* red) {
    Stat<KIND> s;
#pragma unroll 8
    for (int i = threadIdx.x; i < nb; i += kNT) s.join(part[i]);
    return block_join(s, red).norm();
}

// Workspace values that another workgroup of the same launch reads: agent-scope
// atomics, which act past the XCD's own L2.
IQLH_DEV void put_shared(uint64_t* p, uint64_t v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
IQLH_DEV uint64_t get_shared(const uint64_t* p) {
    return __hip_atomic_load((uint64_t*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The last workgroup of a norm launch: the whole norm, and with EACH the
// tensors' own, 16 lanes a tensor.
template <int KIND, bool EACH>
IQLH_DEV void finish_norm(const TensorSetArgs& a, int nb, float* out_norm, float* out_each, uint64_t* red) {
    __shared__ uint64_t all[EACH ? 4 * kOnePieces : 1];
    __shared__ int first[EACH ? kOneTensors + 1 : 1];
    Stat<KIND> s;
    if constexpr (EACH) {
        // everything that is read, in flight together
        static_assert(kOneTensors < kNT && kOnePieces <= kNT, "one load a thread");
        if ((int)threadIdx.x <= a.count) first[threadIdx.x] = a.first[threadIdx.x];
        if ((int)threadIdx.x < nb) s.join(get_shared(a.part + threadIdx.x));  // nb = npieces, or 1 without any
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if ((int)threadIdx.x < a.npieces) all[4 * threadIdx.x + i] = get_shared(a.each + 4 * threadIdx.x + i);
    } else {
#pragma unroll 8
        for (int i = threadIdx.x; i < nb; i += kNT) s.join(get_shared(a.part + i));
    }
    const double n = block_join(s, red).norm();
    if (threadIdx.x == 0) {
        *out_norm = (float)n;
        if (!finite64(n)) set_flag(a.flags, IQLH_FLAG_NONFINITE_GRAD);
    }
    if constexpr (EACH) {
        for (int t0 = 0; t0 < a.count; t0 += kNT / 16) {  // every lane takes part in the exchanges
            const int t = t0 + threadIdx.x / 16;
            Stat<KIND> v;
            if (t < a.count)
                for (int i = first[t] * 4 + (threadIdx.x & 15); i < first[t + 1] * 4; i += 16) v.join(all[i]);
            v = lanes_join<8>(v);
            if (t < a.count && (threadIdx.x & 15) == 0) out_each[t] = (float)v.norm();
        }
    }
}

// ONE: the workgroup that finishes last also adds up, so that the norm takes
// one launch.  Every wave waits for its stores to the workspace (agent scope, so
// they are in place then), the workgroup's barrier orders them before its count,
// and whoever counts last finds all of them.  The count is left at 0.  (A count with
// release and acquire instead writes an L2 back and empties it for every workgroup:
// 18 workgroups 5.0 us against 4.6, 977 23 against 16, 537 MB 184 against 97.)
template <int KIND, bool EACH, bool ONE>
__global__ __launch_bounds__(kNT) void grad_norm_kernel(TensorSetArgs a, float* __restrict__ out_norm,
                                                        float* __restrict__ out_each) {
    __shared__ uint64_t red[kNT / kWave];
    __shared__ int last;
    Stat<KIND> total;
    for (int k = blockIdx.x; k < a.npieces; k += gridDim.x) {
        const TensorPiece p = a.pieces[k];
        Stat<KIND> s0, s1;
        if (p.dtype == IQLH_F32) piece_stat<IQLH_F32>(p, s0, s1);
        else if (p.dtype == IQLH_BF16) piece_stat<IQLH_BF16>(p, s0, s1);
        else piece_stat<IQLH_F16>(p, s0, s1);
        s0.join(s1.bits());
        total.join(s0.bits());
        if (EACH) {
            const Stat<KIND> w = wave_join(s0);
            if ((threadIdx.x & 63) == 0) {
                uint64_t* e = a.each + (int64_t)k * 4 + threadIdx.x / kWave;
                if (ONE) put_shared(e, w.bits());
                else *e = w.bits();
            }
        }
    }
    total = block_join(total, red);
    if (!ONE) {
        if (threadIdx.x == 0) a.part[blockIdx.x] = total.bits();
        return;
    }
    if (threadIdx.x == 0) put_shared(a.part + blockIdx.x, total.bits());
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(a.arrived, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    if (threadIdx.x == 0) __hip_atomic_store(a.arrived, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    finish_norm<KIND, EACH>(a, gridDim.x, out_norm, out_each, red);
}

// Block 0: the whole norm.  Block 1 + t: tensor t.
template <int KIND>
__global__ __launch_bounds__(kNT) void grad_norm_finish_kernel(TensorSetArgs a, int nb, float* __restrict__ out_norm,
                                                               float* __restrict__ out_each) {
    __shared__ uint64_t red[kNT / kWave];
    if (blockIdx.x == 0) {
        const double n = norm_of_parts<KIND>(a.part, nb, red);
        if (threadIdx.x == 0) {
            *out_norm = (float)n;
            if (!finite64(n)) set_flag(a.flags, IQLH_FLAG_NONFINITE_GRAD);
        }
        return;
    }
    const int t = blockIdx.x - 1;
    const double n = norm_of_parts<KIND>(a.each + (int64_t)a.first[t] * 4, (a.first[t + 1] - a.first[t]) * 4, red);
    if (threadIdx.x == 0) out_each[t] = (float)n;
}

// Products of a clip in place are rounded once.  To binary16 the multiplication
// and the conversion are one instruction, which does so.  To bfloat16 the product
// passes through binary32, and where that puts it onto the middle of two values
// the conversion would go to the even one: the thread's products are then taken again
// from the exact ones (32 bits, exact in binary64), rounded to odd, that is cut off
// with the last bit set, so that the conversion sees the side they lie on.
// (537 MB of bf16, norm and clip: 290 us, without this 285.)
// 0 for a binary32 value in the middle of two bfloat16:
IQLH_DEV uint32_t off_middle(float f) { return (__float_as_uint(f) << 16) + 0x80000000u; }
IQLH_DEV float product_to_odd(float x, float c) {
    const double p = (double)x * (double)c;
    const float f = (float)p;
    const double d = (double)f;
    const uint32_t b = __float_as_uint(f);
    const uint32_t outward = fabs(d) < fabs(p) ? 1u : 0xFFFFFFFFu;
    return __uint_as_float(d != p && !(b & 1u) ? b + outward : b);  // an even f: its neighbour on p's side
}

// Elements [0, n) of q times c in place, whole 16-byte quads, kAhead loads in
// flight per thread.
template <int DT>
IQLH_DEV void scale_quads(uint4* q, int nq, float c) {
    typedef Elem<DT> E;
    uint32_t nearest = 1u;  // 0: one of the products below lies in the middle
    auto scaled = [&](uint4 x) __attribute__((always_inline)) {
        float v[E::kQ];
#pragma unroll
        for (int j = 0; j < E::kQ; ++j) {
            v[j] = E::get(x, j) * c;
            if constexpr (DT == IQLH_BF16) {
                const uint32_t o = off_middle(v[j]);
                nearest = o < nearest ? o : nearest;
            }
        }
        return E::pack(v);
    };
    auto exactly = [&](uint4 x) __attribute__((always_inline)) {
        float v[E::kQ];
#pragma unroll
        for (int j = 0; j < E::kQ; ++j) v[j] = product_to_odd(E::get(x, j), c);
        return E::pack(v);
    };
    int i = threadIdx.x;
    for (; i + (kAhead - 1) * kNT < nq; i += kAhead * kNT) {
        uint4 x[kAhead], y[kAhead];
        nearest = 1u;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) x[k] = q[i + k * kNT];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) y[k] = scaled(x[k]);
        if (DT == IQLH_BF16 && !nearest) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) y[k] = exactly(x[k]);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) q[i + k * kNT] = y[k];
    }
    for (; i < nq; i += kNT) {
        const uint4 x = q[i];
        nearest = 1u;
        uint4 y = scaled(x);
        if (DT == IQLH_BF16 && !nearest) y = exactly(x);
        q[i] = y;
    }
}

// Four elements of a body that starts on a 16-byte boundary, times c, to the
// flat vector: 16 bytes of it per thread whatever the source type, so that
// neighbouring lanes store neighbouring 16 bytes (which need not lie on a
// boundary of 16, only of 4).
template <int DT> struct Four;
template <> struct Four<IQLH_F32> {
    typedef uint4 type;
    static IQLH_DEV float get(uint4 w, int i) { return __uint_as_float((&w.x)[i]); }
};
template <> struct Four<IQLH_BF16> {
    typedef uint2 type;
    static IQLH_DEV float get(uint2 w, int i) { return Elem<IQLH_BF16>::get(uint4{w.x, w.y, 0u, 0u}, i); }
};
template <> struct Four<IQLH_F16> {
    typedef uint2 type;
    static IQLH_DEV float get(uint2 w, int i) { return Elem<IQLH_F16>::get(uint4{w.x, w.y, 0u, 0u}, i); }
};
typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));
template <int DT>
IQLH_DEV void scale_flat(const void* src, float* out, int n4, float c) {
    typedef Four<DT> F;
    const typename F::type* q = (const typename F::type*)src;
    auto scaled = [c](typename F::type w) __attribute__((always_inline)) {
        return f4u{F::get(w, 0) * c, F::get(w, 1) * c, F::get(w, 2) * c, F::get(w, 3) * c};
    };
    int i = threadIdx.x;
    for (; i + (kAhead - 1) * kNT < n4; i += kAhead * kNT) {
        typename F::type x[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) x[k] = q[i + k * kNT];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) *(f4u*)(out + (int64_t)(i + k * kNT) * 4) = scaled(x[k]);
    }
    for (; i < n4; i += kNT) *(f4u*)(out + (int64_t)i * 4) = scaled(q[i]);
}

template <int DT>
IQLH_DEV void scale_piece(const TensorPiece& p, float c, float* flat) {
    typedef Elem<DT> E;
    const Cut<DT> cut(p);
    const int e = cut.edge();
    if (!flat) {
        scale_quads<DT>((uint4*)cut.q, cut.nq, c);
        if (e >= 0) {
            const float x = E::load((const void*)p.ptr, e);
            E::store((void*)p.ptr, e, DT == IQLH_BF16 ? product_to_odd(x, c) : x * c);
        }
        return;
    }
    scale_flat<DT>(cut.q, flat + p.off + cut.head, cut.nq * (E::kQ / 4), c);
    if (e >= 0) flat[p.off + e] = E::load((const void*)p.ptr, e) * c;
}

template <int KIND>
__global__ __launch_bounds__(kNT) void grad_scale_kernel(TensorSetArgs a, int nb, double max_norm,
                                                         float* __restrict__ flat, float* __restrict__ out) {
    __shared__ uint64_t red[kNT / kWave];
    const double n = norm_of_parts<KIND>(a.part, nb, red);
    const bool ok = finite64(n);
    const float c = ok && n > max_norm ? (float)(max_norm / n) : 1.f;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        out[0] = (float)n;
        out[1] = c;
        if (!ok) set_flag(a.flags, IQLH_FLAG_NONFINITE_GRAD);
    }
    if (!flat && c == 1.f) return;
    // last piece first: the end of the list is what the norm pass read last
    // and what a list larger than the Infinity Cache still finds there
    for (int k = a.npieces - 1 - blockIdx.x; k >= 0; k -= gridDim.x) {
        const TensorPiece p = a.pieces[k];
        if (p.dtype == IQLH_F32) scale_piece<IQLH_F32>(p, c, flat);
        else if (p.dtype == IQLH_BF16) scale_piece<IQLH_BF16>(p, c, flat);
        else scale_piece<IQLH_F16>(p, c, flat);
    }
}

int norm_blocks(int npieces) { return npieces < 1 ? 1 : npieces < kNormBlocks ? npieces : kNormBlocks; }

template <int KIND, bool EACH, bool ONE>
hipError_t norm_pass(const TensorSetArgs& a, float* out_norm, float* out_each, hipStream_t stream) {
    hipLaunchKernelGGL((grad_norm_kernel<KIND, EACH, ONE>), dim3(norm_blocks(a.npieces)), dim3(kNT), 0, stream, a, out_norm,
                       out_each);
    return hipGetLastError();
}

// One launch up to kOnePieces, where it saves the second one: 64 pieces 4.9 us
// against 7.1, 256 6.5 against 7.6.  Above that the count of the workgroups that
// have finished, one at a time on one address, takes longer: 384 pieces 8.3 us
// against 7.5, 1024 (16 MB) 16.7 against 7.5, 2048 30 against 13.5, 512 MB 91 against 90.
template <int KIND>
hipError_t norm_launch(const TensorSetArgs& a, float* out_norm, float* out_each, hipStream_t stream) {
    if (a.npieces <= kOnePieces && (!out_each || a.count <= kOneTensors))
        return out_each ? norm_pass<KIND, true, true>(a, out_norm, out_each, stream)
                        : norm_pass<KIND, false, true>(a, out_norm, out_each, stream);
    hipError_t e = out_each ? norm_pass<KIND, true, false>(a, out_norm, out_each, stream)
                            : norm_pass<KIND, false, false>(a, out_norm, out_each, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(grad_norm_finish_kernel<KIND>, dim3(out_each ? 1 + a.count : 1), dim3(kNT), 0, stream, a,
                       norm_blocks(a.npieces), out_norm, out_each);
    return hipGetLastError();
}

template <int KIND>
hipError_t clip_launch(const TensorSetArgs& a, double max_norm, float* flat, float* out, hipStream_t stream) {
    hipError_t e = norm_pass<KIND, false, false>(a, nullptr, nullptr, stream);
    if (e != hipSuccess) return e;
    const int nb = norm_blocks(a.npieces);
    hipLaunchKernelGGL(grad_scale_kernel<KIND>, dim3(nb), dim3(kNT), 0, stream, a, nb, max_norm, flat, out);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grad_norm(const TensorSetArgs& a, int kind, float* out_norm, float* out_each, hipStream_t stream) {
    return kind == IQLH_NORM_L2 ? norm_launch<IQLH_NORM_L2>(a, out_norm, out_each, stream)
                                : norm_launch<IQLH_NORM_MAX>(a, out_norm, out_each, stream);
}

hipError_t launch_grad_clip(const TensorSetArgs& a, int kind, double max_norm, float* flat, float* out,
                            hipStream_t stream) {
    return kind == IQLH_NORM_L2 ? clip_launch<IQLH_NORM_L2>(a, max_norm, flat, out, stream)
                                : clip_launch<IQLH_NORM_MAX>(a, max_norm, flat, out, stream);
}

}  // namespace iqlh
