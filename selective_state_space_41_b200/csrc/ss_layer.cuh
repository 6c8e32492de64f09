// What the operators around the scan (normalisation, causal convolution,
// gated recurrence) share: eight-element vectors of a (batch, dim, L) tensor,
// the logistic function with its complement, masks of sequence starts, and
// the host-side checks of a descriptor.
//
// Rows of L steps start at multiples of L elements, so with an odd length no
// row but the first starts on a 16-byte boundary.  The kernels that walk rows
// therefore count "virtual" steps from the 8-element boundary at or before
// the row's start: every vector is then aligned, the first and the last one
// of a row hold a few elements of the neighbouring rows, and those are
// masked.  All tensors of a call have the same shape, so one shift serves all.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cstdint>
#include <initializer_list>

#include "selscan.h"
#include "ss_fwd_kernel.cuh"

namespace selscan {

constexpr int kV = 8;  // elements per vector: 16 bytes of bf16, 32 of fp32

// Two neighbouring elements of words as they lie in memory, as floats.
template <typename T>
__device__ __forceinline__ float2 pair_of(const uint32_t *w, int k) {
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
    else return make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, both(-1.f), a); }  // (exact: one rounding)

// Eight elements as they lie in memory.
template <typename T>
struct Vec8 {
    static constexpr int kWords = kV * sizeof(T) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ float operator[](int i) const { return Io<T>::widen(w, i); }
    __device__ __forceinline__ float2 pair(int k) const { return pair_of<T>(w, k); }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < kWords; ++k) w[k] = 0u;
    }
    // Makes the words opaque here: what was computed from them before is
    // computed anew after it, rather than kept in registers meanwhile.
    __device__ __forceinline__ void again() {
#pragma unroll
        for (int k = 0; k < kWords; ++k) asm volatile("" : "+r"(w[k]));
    }
    // The vector at an element index that is a multiple of 8 (16-byte aligned).
    __device__ __forceinline__ void load(const T *p, int64_t e) {
        const uint4 *q = reinterpret_cast<const uint4 *>(p + e);
#pragma unroll
        for (int k = 0; k < kWords / 4; ++k) {
            const uint4 u = __ldg(q + k);
            w[4 * k] = u.x, w[4 * k + 1] = u.y, w[4 * k + 2] = u.z, w[4 * k + 3] = u.w;
        }
    }
    __device__ __forceinline__ void put_bits(int i, uint32_t b) {  // into a cleared place
        if constexpr (sizeof(T) == 4) w[i] = b;
        else w[i >> 1] |= b << (16 * (i & 1));
    }
    // Elements [lo, hi) of it; the others are zero.  Loads without a branch
    // (from the nearest element of the range), so that all are in flight at
    // once, then the selection.
    __device__ __forceinline__ void load_part(const T *p, int64_t e, int lo, int hi) {
        clear();
        if (hi <= lo) return;
        uint32_t b[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) b[i] = Io<T>::bits(p, e + (i < lo ? lo : i < hi ? i : hi - 1));
#pragma unroll
        for (int i = 0; i < kV; ++i) put_bits(i, i >= lo && i < hi ? b[i] : 0u);
    }

    // Clears all but elements [lo, hi), 0 <= lo, hi <= 8.
    __device__ __forceinline__ void keep(int lo, int hi) {
        const uint32_t m = ((1u << hi) - 1u) & ~((1u << lo) - 1u);
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            if constexpr (sizeof(T) == 4) w[k] &= (uint32_t)((int)(m << (31 - k)) >> 31);
            else w[k] &= __byte_perm((uint32_t)((int)(m << (31 - 2 * k)) >> 31), (uint32_t)((int)(m << (30 - 2 * k)) >> 31), 0x7610);
        }
    }
};

// The vector at element e of a tensor of n, of which elements [lo, hi) belong
// to the row; the others are zero.  A whole vector is loaded where the tensor
// holds it, and masked.
template <typename T>
__device__ __forceinline__ void load_row8(Vec8<T> &r, const T *p, int64_t e, int64_t n, int lo, int hi, bool vec) {
    if (hi <= lo) {
        r.clear();
    } else if (vec && e >= 0 && e + kV <= n) {
        r.load(p, e);
        if (lo > 0 || hi < kV) r.keep(lo, hi);
    } else {
        r.load_part(p, e, lo, hi);
    }
}

__device__ __forceinline__ float load_elem(const float *p, int64_t i) { return __ldg(p + i); }
__device__ __forceinline__ float load_elem(const __nv_bfloat16 *p, int64_t i) {
    return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short *>(p) + i) << 16);
}

__device__ __forceinline__ void put(float *p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, int64_t i, float v) { p[i] = __float2bfloat16_rn(v); }

__device__ __forceinline__ void store_vec(float *p, const float (&v)[kV]) {
    float4 *q = reinterpret_cast<float4 *>(p);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const float (&v)[kV]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// Elements [lo, hi) of v to the vector at element e.
template <typename T>
__device__ __forceinline__ void store8(T *p, int64_t e, int lo, int hi, bool vec, const float (&v)[kV]) {
    if (vec && lo <= 0 && hi >= kV) {
        store_vec(p + e, v);
    } else if (hi > lo) {
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (i >= lo && i < hi) put(p, e + i, v[i]);
    }
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ int clamp8(int64_t v) { return v < 0 ? 0 : v > kV ? kV : (int)v; }

// exp(-v) of two values that go into results of inputs of type T.  bf16
// inputs, whose values carry 2^-9: on the SFU (2 ulp), beyond which the
// rounding of v log2 e adds |v| 2^-24.  fp32 inputs: expf, whose error does not
// grow with |v|.  (fp32 with 2^x on the SFU: 10^-6 relative at v = -20 where
// this has 2.7 10^-7; 4 x 1024 x 4096 convolution 27.0 us, backward 61.9, with
// expf 28.8 and 63.6; recurrence forward and backward with the gate 121.2, 122.7.)
template <typename T>
__device__ __forceinline__ float2 exp_neg2(float2 v) {
    if constexpr (sizeof(T) == 4) return make_float2(expf(-v.x), expf(-v.y));
    const float2 t = mul2(v, both(-kLog2e));
    return make_float2(sfu_exp2(t.x), sfu_exp2(t.y));
}
// The reciprocal on the SFU (1 ulp) for both types: an IEEE division takes
// those fp32 cases to 69.1 and 140.4 us, and the error from 2.2 to 2.0 10^-7
// for |v| <= 1.
__device__ __forceinline__ float2 rcp2(float2 u) { return make_float2(sfu_rcp(u.x), sfu_rcp(u.y)); }
// 1 / (1 + exp(-v)).  exp(-v) may overflow, to a result of zero.
template <typename T>
__device__ __forceinline__ float2 sigmoid2(float2 v) { return rcp2(add2(exp_neg2<T>(v), both(1.f))); }
template <typename T>
__device__ __forceinline__ float2 silu2(float2 v) { return mul2(v, sigmoid2<T>(v)); }
// silu'(v) = s (1 + v (1 - s)), given s = sigmoid(v).
__device__ __forceinline__ float2 silu_slope2(float2 v, float2 s) { return mul2(s, fma2(v, sub2(both(1.f), s), both(1.f))); }

// Division of n < 2^31 by a fixed d: n mul >> (32 + shift), with
// 2^(32 + shift) >= 2^31 d and mul its quotient by d rounded up: the excess
// mul d - 2^(32 + shift) is below d, so n times it stays below the power.
struct Divisor {
    uint32_t d, mul;
    int shift;
};
inline Divisor divisor_of(int64_t d) {
    Divisor r{(uint32_t)d, 0u, 0};
    if (d <= 1) return r;
    while (((int64_t)1 << (r.shift + 1)) < d) ++r.shift;  // 2^(shift + 1) >= d
    r.mul = (uint32_t)((((uint64_t)1 << (32 + r.shift)) + (uint64_t)d - 1) / (uint64_t)d);
    return r;
}
__device__ __forceinline__ uint32_t divide(uint32_t n, const Divisor &v) { return v.mul ? __umulhi(n, v.mul) >> v.shift : n; }

// Bits 0..3: whether bytes 0..3 of a word are nonzero.  The sum carries into
// a byte's top bit unless its low seven are zero; the product gathers the four
// ones into bits 24..27 (its ten partial products fall on different bits).
__device__ __forceinline__ uint32_t nonzero_bytes(uint32_t w) {
    const uint32_t top = (((w & 0x7f7f7f7fu) + 0x7f7f7f7fu) | w) & 0x80808080u;
    return (top >> 7) * 0x01020408u >> 24;
}

// Bits lo..hi-1 of the start mask of eight steps from byte m of `reset`, whose
// bytes [0, n) may be read.  Two aligned words where both lie inside, single
// bytes at the mask's ends.
__device__ __forceinline__ uint32_t start_bits(const uint8_t *reset, int64_t m, int64_t n, int lo, int hi) {
    if (hi <= lo) return 0u;
    const uint32_t keep = ((1u << hi) - 1u) & ~((1u << lo) - 1u);
    const uintptr_t at = reinterpret_cast<uintptr_t>(reset) + (uintptr_t)m;
    const int off = (int)(at & 7);
    if (m - off >= 0 && m - off + 16 <= n) {
        const uint2 *q = reinterpret_cast<const uint2 *>(at - off);
        const uint2 u = __ldg(q), v = __ldg(q + 1);
        const unsigned long long a = ((unsigned long long)u.y << 32) | u.x, b = ((unsigned long long)v.y << 32) | v.x;
        const unsigned long long x = off ? (a >> (8 * off)) | (b << (64 - 8 * off)) : a;
        return (nonzero_bytes((uint32_t)x) & 15u | nonzero_bytes((uint32_t)(x >> 32)) << 4) & keep;
    }
    uint32_t bits = 0;
    for (int i = lo; i < hi; ++i)
        if (__ldg(reset + m + i)) bits |= 1u << i;
    return bits;
}

// ------------------------------------------------------------------- host
struct LayerSizes {
    int64_t rows, elems;  // batch * dim, batch * dim * seqlen
};

// The descriptor's sizes and types, as the scan's entries check them, but
// for dstate, which these operators do not read.
inline ss_status check_layer(const ss_desc *desc, LayerSizes *s) {
    if (!desc) return SS_ERR_NULL_POINTER;
    if (desc->batch < 0 || desc->dim < 0 || desc->seqlen < 0) return SS_ERR_BAD_SHAPE;
    const bool in_ok = desc->in_dtype == SS_F32 || desc->in_dtype == SS_BF16;
    const bool out_ok = desc->out_dtype == desc->in_dtype || (desc->in_dtype == SS_BF16 && desc->out_dtype == SS_F32);
    if (!in_ok || !out_ok) return SS_ERR_UNSUPPORTED_DTYPE;
    constexpr int64_t kMost = INT64_MAX / 64;
    const int64_t d = desc->dim > 0 ? desc->dim : 1, l = desc->seqlen > 0 ? desc->seqlen : 1;
    const int64_t b = desc->batch > 0 ? desc->batch : 1;
    if (d > kMost / b || l > kMost / (b * d)) return SS_ERR_BAD_SHAPE;
    s->rows = desc->batch * desc->dim;
    s->elems = s->rows * desc->seqlen;
    return SS_OK;
}

inline size_t layer_size(ss_dtype t) { return t == SS_BF16 ? 2 : 4; }
inline bool layer_aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline bool vec_ok(std::initializer_list<const void *> ps) {  // 16-byte vectors at every base (null: absent)
    for (const void *q : ps)
        if (!layer_aligned(q, 16)) return false;
    return true;
}
inline ss_status status_of(cudaError_t e) { return e == cudaSuccess ? SS_OK : SS_ERR_CUDA; }

// SMs of the current device (asked once per device).
inline int layer_sm_count() {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> cache[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
    int v = cache[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) v = 148;
    cache[dev].store(v, std::memory_order_relaxed);
    return v;
}

}  // namespace selscan

// KERNEL<Tin, Tout> for the descriptor's type pair, as a launch of `CALL`.
#define SS_LAYER_DISPATCH(DESC, CALL)                                                     \
    ((DESC)->in_dtype == SS_F32    ? CALL<float, float>                                   \
     : (DESC)->out_dtype == SS_F32 ? CALL<__nv_bfloat16, float> : CALL<__nv_bfloat16, __nv_bfloat16>)
