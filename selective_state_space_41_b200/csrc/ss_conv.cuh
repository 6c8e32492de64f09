// The causal depthwise convolution: forward, backward and one decoding step
// (declarations and the meaning of every argument in include/selscan.h).
//
//   p_t = bias + sum_(j < W) w_j x_(t - (W-1) + j),   y_t = p_t or silu(p_t)
//
// per row (b, d), with the steps before the row taken from a state (or zero)
// and nothing read across a sequence start.
//
// Both directions take 16 steps of a row per thread: two vectors, and their
// neighbours for the taps (which other threads load too: L1 hits).  Rows are
// cut in virtual steps (see ss_layer.cuh), so every length uses whole
// vectors; what lies outside the row is masked after the load.  Steps i and
// i + 8 of a thread are worked as a pair with the packed arithmetic of two
// floats: their taps are pairs too, i + j and i + j + 8.
//
// Forward: two bytes in and two out per bf16 element against 2 W + 5
// operations.  8 x 1536 x 2048 bf16, W = 4, SiLU: 23 us (15.4 for the bytes),
// issue 66 %, half of the warps an SM can hold, mostly waiting for loads; the
// SFU's 60 % is not the limit (21.6 us without SiLU).  fp32, 4 x 1024 x 4096:
// 28.8 us (20.5 for the bytes).  With starts (2 x 1024 x 20011, W = 5, every
// 500): 62 us (25.0), the tests of the taps and the unpacking of bf16 on the
// integer pipe.
//
// Backward: with q_t = dy_t (silu'(p_t)),
//   dx_s = sum_j w_j q_(s + (W-1) - j),   dw_j = sum_t q_t x_(t - (W-1) + j),   dbias = sum_t q_t.
// p is recomputed from x; q of the W - 1 steps behind a thread's own comes
// from the next thread through shared memory, and for the block's last thread
// from the round before: a block works its spans from the last to the first
// (each thread computing them itself: 51.9 us where this takes 47, 8 x 1536 x
// 2048 bf16, W = 4, SiLU; 23.1 for the bytes; 16 warps an SM at 110 registers
// issue 53 % of the time; fp32 4 x 1024 x 4096 63.7, 30.7 for the bytes).
// dw and dbias sum over batch and steps for each channel, so a block (or a
// cluster of blocks, when the channels are few) takes one channel and all of
// its batch entries; every thread keeps its W + 1 sums in registers over all
// its vectors and they are joined once at the end, in a fixed order and
// without a second launch.
//
// A warp that sees a sequence start in any of its windows takes the path that
// tests every tap against the starts; the others do not pay for it.
#pragma once

#include <type_traits>

#include "ss_layer.cuh"

namespace selscan {

constexpr int kMinWidth = 2, kMaxWidth = 8;

struct ConvParams {
    const void *x, *dy, *dlast, *h0;
    const float *weight, *bias;
    const uint8_t *reset;
    void *y, *last, *dx, *dh0;
    float *dweight, *dbias;
    int64_t batch, dim, L;
    int silu, vec;
    int width;            // decoding step
    int64_t main_blocks;  // forward: blocks of the outputs; the rest write the last state
    Divisor by_spans, by_dim;  // spans of a row, channels
    int small;            // the spans count in 31 bits (forward: of all rows; backward: of a channel)
    int64_t chunks, groups;  // forward with starts: warps of spans to a row, groups of 8 channels to an entry
    int64_t rounds, each;    // backward: rounds of a block's threads to a channel, and to a block
};

cudaError_t conv_fwd_f32_f32(int width, cudaStream_t s, ConvParams &p);
cudaError_t conv_fwd_bf16_bf16(int width, cudaStream_t s, ConvParams &p);
cudaError_t conv_fwd_bf16_f32(int width, cudaStream_t s, ConvParams &p);
cudaError_t conv_bwd_f32_f32(int width, cudaStream_t s, ConvParams &p);
cudaError_t conv_bwd_bf16_bf16(int width, cudaStream_t s, ConvParams &p);
cudaError_t conv_bwd_bf16_f32(int width, cudaStream_t s, ConvParams &p);

// x at step t of a row (t < 0: the state), in 32 bits.
template <typename T, int W>
__device__ __forceinline__ float conv_input(const ConvParams &p, int64_t row, int64_t t) {
    if (t >= 0) return load_elem(static_cast<const T *>(p.x), row * p.L + t);
    return p.h0 ? load_elem(static_cast<const T *>(p.h0), row * (W - 1) + (W - 1) + t) : 0.f;
}

__device__ __forceinline__ bool starts_at(const ConvParams &p, int64_t b, int64_t t) {
    return p.reset && __ldg(p.reset + b * p.L + t) != 0;
}

// p_t from single loads: the places where no vector serves.
template <typename T, int W>
__device__ __forceinline__ float conv_at(const ConvParams &p, int64_t row, int64_t t, const float (&w)[W], float bias) {
    const int64_t b = row / p.dim;
    float acc = bias;
    bool seen = true;
    float xs[W];
#pragma unroll
    for (int j = W - 1; j >= 0; --j) {  // from step t back
        const int64_t s = t - (W - 1) + j;
        xs[j] = seen ? conv_input<T, W>(p, row, s) : 0.f;
        if (s >= 0 && starts_at(p, b, s)) seen = false;
    }
#pragma unroll
    for (int j = 0; j < W; ++j) acc = fmaf(w[j], xs[j], acc);
    return acc;
}

// dy silu'(p).
template <typename T>
__device__ __forceinline__ float2 conv_slope(float2 pre, float2 dy) { return mul2(dy, silu_slope2(pre, sigmoid2<T>(pre))); }

constexpr int kSpan = 16;  // steps of a thread

// Where a thread's steps lie: step t0 of the row, element e; head and tail
// are the steps from the row's start and to its end, counted up to 64.
struct Span {
    int64_t t0, e;
    int head, tail;
    __device__ __forceinline__ int lo(int i) const { return min(max(-(head + i), 0), kV); }  // of the vector at t0 + i
    __device__ __forceinline__ int hi(int i) const { return min(max(tail - i, 0), kV); }
};
__device__ __forceinline__ Span span_of(int64_t e0, int64_t v, int64_t L) {
    Span s;
    s.t0 = v * kSpan - (e0 & (kV - 1));
    s.e = e0 + s.t0;
    s.head = (int)min(s.t0, (int64_t)64);
    s.tail = (int)min(L - s.t0, (int64_t)64);  // -6 at the least
    return s;
}
// Spans of a row: the largest shift of a row's start is 8 less the largest
// power of two in L (8 at most).
__host__ __device__ __forceinline__ int64_t spans_of(int64_t L) {
    const int64_t two = L % 8 == 0 ? 8 : L % 4 == 0 ? 4 : L % 2 == 0 ? 2 : 1;
    return (L + kV - two + kSpan - 1) / kSpan;
}

// x at steps t0 - (W-1) .. of a thread, kN vectors of its own and behind:
// pairs (k, k + 8).  Outside the row: the state before it, zero behind.
template <typename T, int W, int kVecs>
struct Window {
    static constexpr int kN = W - 1 + kV * (kVecs - 1) + (kVecs == 2 ? kV : W - 1);  // values
    static constexpr int kPairs = kN - kV;
    float2 v[kPairs];
    // value k is v[k].x (k < kPairs) and v[k - 8].y (k >= 8)
    __device__ __forceinline__ void set(int k, float f) {
        if (k < kPairs) v[k].x = f;
        if (k >= kV) v[k - kV].y = f;
    }
    __device__ __forceinline__ float get(int k) const { return k < kPairs ? v[k].x : v[k - kV].y; }
    // From its vectors, the one before the thread's steps first.
    __device__ __forceinline__ void take(const ConvParams &p, const Vec8<T> (&q)[kVecs + 1], const Span &s, int64_t row) {
#pragma unroll
        for (int k = 0; k < kN; ++k) set(k, q[(k + kV - (W - 1)) / kV][(k + kV - (W - 1)) % kV]);
        if (p.h0 && s.head < W - 1) {
#pragma unroll
            for (int k = 0; k < 2 * (W - 1) + kV - 1 && k < kN; ++k) {  // head >= -7: steps -(W-1) .. -1 lie here
                const int t = s.head - (W - 1) + k;
                if (t < 0 && t >= -(W - 1)) set(k, load_elem(static_cast<const T *>(p.h0), row * (W - 1) + (W - 1) + t));
            }
        }
    }
    // inner: all of its vectors lie in the row and are whole
    __device__ __forceinline__ void load(const ConvParams &p, const T *x, const Span &s, int64_t row, int64_t n, bool inner) {
        Vec8<T> q[kVecs + 1];
        if (inner) {
#pragma unroll
            for (int i = 0; i <= kVecs; ++i) q[i].load(x + s.e, (i - 1) * kV);
        } else {
#pragma unroll
            for (int i = 0; i <= kVecs; ++i)
                load_row8(q[i], x, s.e + (i - 1) * kV, n, s.lo((i - 1) * kV), s.hi((i - 1) * kV), p.vec);
        }
        take(p, q, s, row);
    }
};

// Bits of the starts at steps t0 + i of a span, i = first .. first + 7.
__device__ __forceinline__ uint32_t span_starts(const ConvParams &p, int64_t b, const Span &s, int first) {
    return start_bits(p.reset, b * p.L + s.t0 + first, p.batch * p.L, s.lo(first), s.hi(first));
}

// cut[j], bit k: a start lies between tap j of output k and the output's own
// step (window positions k + j + 1 .. k + W - 1).  The result is the same in
// all lanes: bit k is set where any of them has a tap cut in outputs k, k + 8.
// Only those pairs of outputs test their taps (packed sequences of 500 steps
// cut four pairs in a warp's 512 steps).
template <int W>
__device__ __forceinline__ uint32_t cuts_of(uint32_t m, uint32_t (&cut)[W]) {
    cut[W - 1] = 0;
#pragma unroll
    for (int j = W - 2; j >= 0; --j) cut[j] = cut[j + 1] | m >> (j + 1);
    return __reduce_or_sync(0xffffffffu, cut[0] | cut[0] >> kV);
}
// v, of a tap with these cuts of outputs k and k + 8, or zero behind a start.
__device__ __forceinline__ float2 seen(float2 v, uint32_t cut, int k) {
    if (cut >> k & 1u) v.x = 0.f;
    if (cut >> (k + kV) & 1u) v.y = 0.f;
    return v;
}

template <typename Tin, typename Tout, int W, bool kR>
__global__ void __launch_bounds__(256) conv_fwd_kernel(const ConvParams p) {
    const int64_t L = p.L, rows = p.batch * p.dim, n = rows * L;
    if (blockIdx.x >= p.main_blocks) {
        // the last W - 1 inputs, those of the last sequence alone
        const int64_t i = (blockIdx.x - p.main_blocks) * (int64_t)blockDim.x + threadIdx.x;
        if (i >= rows * (W - 1)) return;
        const int64_t row = i / (W - 1), t = L - (W - 1) + i % (W - 1), b = row / p.dim;
        bool seen = true;
        for (int64_t s = L - 1; s > t && s >= 0; --s) seen = seen && !starts_at(p, b, s);
        put(static_cast<Tin *>(p.last), i, seen ? conv_input<Tin, W>(p, row, t) : 0.f);
        return;
    }
    const int64_t nv = spans_of(L);
    bool there;  // (the threads behind the end stay for their warp's vote)
    uint32_t row, b, d;
    int64_t v;
    uint32_t m = 0;  // bit k: a sequence starts at step t0 - (W-1) + k
    if constexpr (kR) {
        // A warp's 32 spans of a row, and 8 channels that share their starts
        // in a block: the mask's bytes become bits once for all of them.
        constexpr int kAhead = 16, kWords = 32 * kSpan / 32 + 2;  // from 16 steps before the warp's spans
        __shared__ uint32_t bits[kWords];
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int64_t chunk = blockIdx.x % p.chunks, group = blockIdx.x / p.chunks;
        b = (uint32_t)(group / p.groups);
        d = (uint32_t)(group - (int64_t)b * p.groups) * 8 + warp;
        const int64_t first = chunk * 32 * kSpan - kAhead;
        for (int k = warp; k < kWords; k += 8) {
            const int64_t t = first + k * 32 + lane;
            const uint32_t w = __ballot_sync(0xffffffffu, t >= 0 && t < L && __ldg(p.reset + b * L + max(t, (int64_t)0)) != 0);
            if (lane == 0) bits[k] = w;
        }
        __syncthreads();
        v = chunk * 32 + lane;
        there = d < p.dim && v < nv;
        if (!there) d = 0, v = 0;
        row = b * (uint32_t)p.dim + d;
        const int at = kAhead + lane * kSpan - (int)(row * L & (kV - 1)) - (W - 1);
        if (there) m = __funnelshift_r(bits[at >> 5], bits[(at >> 5) + 1], at & 31) & ((1u << (W - 1 + kSpan)) - 1u);
    } else {
        const int64_t q = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
        there = q < rows * nv;
        row = !there ? 0u : p.small ? divide((uint32_t)q, p.by_spans) : (uint32_t)(q / nv);
        b = divide(row, p.by_dim), d = row - b * p.by_dim.d;
        v = there ? q - row * nv : 0;
    }
    Span s = span_of(row * L, v, L);
    if (!there) s.tail = -kSpan;
    const bool whole = p.vec && s.head >= 0 && s.tail >= kSpan, inner = whole && s.head >= kV;
    float w[W];
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = __ldg(p.weight + (int64_t)d * W + j);
    const float bias = p.bias ? __ldg(p.bias + d) : 0.f;
    Window<Tin, W, 2> x;
    x.load(p, static_cast<const Tin *>(p.x), s, row, n, inner);
    float2 out[kV];
    uint32_t cut[W];
    const uint32_t slow = kR ? cuts_of<W>(m, cut) : 0u;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        out[i] = both(bias);
        if (kR && (slow >> i & 1u)) {
#pragma unroll
            for (int j = 0; j < W; ++j) out[i] = fma2(both(w[j]), seen(x.v[i + j], cut[j], i), out[i]);
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) out[i] = fma2(both(w[j]), x.v[i + j], out[i]);
        }
    }
    if (p.silu) {
#pragma unroll
        for (int i = 0; i < kV; ++i) out[i] = silu2<Tin>(out[i]);
    }
    float y0[kV], y1[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) y0[i] = out[i].x, y1[i] = out[i].y;
    Tout *y = static_cast<Tout *>(p.y) + s.e;
    if (whole) {
        store_vec(y, y0);
        store_vec(y + kV, y1);
    } else {
        store8(y, 0, s.lo(0), s.hi(0), p.vec, y0);
        store8(y, kV, s.lo(kV), s.hi(kV), p.vec, y1);
    }
}

constexpr int kConvBwdThreads = 128;  // of a block, at most: fewer where a channel has fewer spans

// The backward's next spans, copied in while the present ones are worked on:
// a slot for each thread's 16 elements of a tensor, and one before them.
template <typename T>
struct Slots {
    static constexpr int kQ = sizeof(T) / 2;  // 16-byte words of a vector
    uint4 w[(kConvBwdThreads + 1) * 2 * kQ];
    // Both vectors of a thread whose steps all lie in the row.
    __device__ __forceinline__ void fill_whole(int t, const T *p) {
#pragma unroll
        for (int k = 0; k < 2 * kQ; ++k) cp_async16(w + (t + 1) * 2 * kQ + k, p + k * (16 / sizeof(T)));
    }
    // Vector i of the tensor's spans, counted from the slot before thread 0's.
    __device__ __forceinline__ void fill(int i, const T *p, int64_t e, int64_t n, int lo, int hi, bool vec) {
        uint4 *to = w + i * kQ;
        if (hi > lo && vec && e >= 0 && e + kV <= n) {
#pragma unroll
            for (int k = 0; k < kQ; ++k) cp_async16(to + k, p + e + k * (16 / sizeof(T)));
        } else if (hi > lo) {
            Vec8<T> v;
            v.load_part(p, e, lo, hi);
#pragma unroll
            for (int k = 0; k < kQ; ++k) to[k] = make_uint4(v.w[4 * k], v.w[4 * k + 1], v.w[4 * k + 2], v.w[4 * k + 3]);
        }
    }
    __device__ __forceinline__ void read(Vec8<T> &v, int i) const {
#pragma unroll
        for (int k = 0; k < kQ; ++k) {
            const uint4 u = w[i * kQ + k];
            v.w[4 * k] = u.x, v.w[4 * k + 1] = u.y, v.w[4 * k + 2] = u.z, v.w[4 * k + 3] = u.w;
        }
    }
};

// Clears what of the vector at step t0 + i is not in the row.
template <typename T>
__device__ __forceinline__ void trim(Vec8<T> &v, const Span &s, int i) {
    const int lo = s.lo(i), hi = s.hi(i);
    if (hi <= lo) v.clear();
    else if (lo > 0 || hi < kV) v.keep(lo, hi);
}

template <typename Tin, typename Tout, int W, bool kR>
__global__ void __launch_bounds__(kConvBwdThreads, 4) conv_bwd_kernel(const ConvParams p, int nblk) {
    const int64_t L = p.L, n = p.batch * p.dim * L;
    const int64_t d = blockIdx.x / nblk;  // the blocks of a channel follow one another: one cluster
    const int rank = (int)(blockIdx.x % nblk);
    const Tin *x = static_cast<const Tin *>(p.x);
    const Tout *dy = static_cast<const Tout *>(p.dy);
    Tin *dx = static_cast<Tin *>(p.dx);
    const bool silu = p.silu, vec = p.vec;
    float w[W];
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = __ldg(p.weight + d * W + j);
    const float bias = p.bias ? __ldg(p.bias + d) : 0.f;

    float2 sum2[W + 1];  // dw_j, dbias, of the two halves of the thread's steps
#pragma unroll
    for (int j = 0; j <= W; ++j) sum2[j] = both(0.f);

    __shared__ Slots<Tin> xs[2];
    __shared__ Slots<Tout> gs[2];
    __shared__ uint32_t starts[kR ? kConvBwdThreads + 2 : 1];
    __shared__ float heads[2][W - 1][kConvBwdThreads];  // q of each thread's outputs 0 .. W-2
    const int t = threadIdx.x;
    const int64_t nv = spans_of(L), total = p.batch * nv;
    // The block's rounds of blockDim spans, worked from the last to the first.
    const int64_t first = rank * p.each, behind = min(first + p.each, p.rounds);
    // Span q of the channel; one behind the last has no step.
    const auto place = [&](int64_t q, int64_t &b) {
        const bool there = q < total;
        b = !there ? 0 : p.small ? (int64_t)divide((uint32_t)q, p.by_spans) : q / nv;
        Span s = span_of((b * p.dim + d) * L, there ? q - b * nv : 0, L);
        if (!there) s.tail = -kSpan;
        return s;
    };
    const bool whole_rows = L % kV == 0;
    const auto fill = [&](const Span &s, int buf) {
        if (vec && s.head >= 0 && s.tail >= kSpan) {
            xs[buf].fill_whole(t, x + s.e);
            gs[buf].fill_whole(t, dy + s.e);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                xs[buf].fill(2 * t + 2 + i, x, s.e + i * kV, n, s.lo(i * kV), s.hi(i * kV), vec);
                gs[buf].fill(2 * t + 2 + i, dy, s.e + i * kV, n, s.lo(i * kV), s.hi(i * kV), vec);
            }
        }
        if (t == 0 && s.head > 0) xs[buf].fill(1, x, s.e - kV, n, s.lo(-kV), s.hi(-kV), vec);
        cp_async_commit();
    };
    int buf = 0;
    int64_t b, next_b;
    Span s, next = place((behind - 1) * blockDim.x + t, next_b);
    if (first < behind) {
        fill(next, 0);
        // What later rounds leave for the last thread, for the first of them:
        // steps behind the row's end have a slope of zero here as there.
        if (t == (int)blockDim.x - 1 && next.tail > kSpan) {
            const int64_t row = next_b * p.dim + d;
#pragma unroll 1
            for (int k = 0; k < W - 1; ++k) {
                const int64_t at = next.t0 + kSpan + k;
                float q = 0.f;
                if (k < next.tail - kSpan) {
                    q = load_elem(dy, row * L + at);
                    if (silu) q = conv_slope<Tin>(both(conv_at<Tin, W>(p, row, at, w, bias)), both(q)).x;
                }
                heads[1][k][0] = q;
            }
        }
    }
    for (int64_t round = behind - 1; round >= first; --round, buf ^= 1) {
        const int64_t q = round * blockDim.x + t;
        const bool there = q < total;
        s = next, b = next_b;
        if (round > first) {
            next = place(q - blockDim.x, next_b);
            fill(next, buf ^ 1);
            cp_async_wait_one();
        } else {
            cp_async_wait_all();
        }
        uint32_t m = 0;  // bit k: a sequence starts at step t0 - (W-1) + k
        if constexpr (kR) {
            // each thread's own 16 steps, and those of its neighbours
            m = span_starts(p, b, s, 0) | span_starts(p, b, s, kV) << kV;
            starts[t + 1] = m;
            if (t == 0) starts[0] = span_starts(p, b, s, -kV) << kV;
            if (t == (int)blockDim.x - 1) starts[t + 2] = span_starts(p, b, s, kSpan);
        }
        __syncthreads();
        if constexpr (kR) {
            const uint32_t before = s.head > 0 ? starts[t] : 0u, behind = s.tail > kSpan ? starts[t + 2] : 0u;
            m = (before & 0xffffu) >> (kSpan - (W - 1)) | m << (W - 1) | behind << (W - 1 + kSpan);
            m &= (1u << (2 * (W - 1) + kSpan)) - 1u;
        }
        const int64_t row = b * p.dim + d;
        const bool whole = vec && s.head >= 0 && s.tail >= kSpan;
        Window<Tin, W, 2> win;
        float2 slope[kV];  // first dy: outputs k and k + 8
        {
            Vec8<Tin> v[3];
            Vec8<Tout> u[2];
#pragma unroll
            for (int i = 0; i < 3; ++i) xs[buf].read(v[i], 2 * t + 1 + i);
#pragma unroll
            for (int i = 0; i < 2; ++i) gs[buf].read(u[i], 2 * t + 2 + i);
            // what is not in the row: it was not copied, or belongs to a neighbouring one
            if (whole_rows) {
                if (s.head <= 0) v[0].clear();
                if (s.tail <= 0) v[1].clear(), u[0].clear();  // (a thread without a span)
                if (s.tail <= kV) v[2].clear(), u[1].clear();
            } else if (s.head < kV || s.tail < kSpan) {
#pragma unroll
                for (int i = 0; i < 3; ++i) trim(v[i], s, (i - 1) * kV);
#pragma unroll
                for (int i = 0; i < 2; ++i) trim(u[i], s, i * kV);
            }
            win.take(p, v, s, row);
            // outputs outside the row have dy = 0, and with it no part in anything
#pragma unroll
            for (int k = 0; k < kV; ++k) slope[k] = make_float2(u[0][k], u[1][k]);
        }
        uint32_t cut[W];
        const uint32_t slow = kR ? cuts_of<W>(m, cut) : 0u;
        // Output by output: p, q, and what q adds to the sums and to the steps
        // of its taps.  Tap j of output k reads window position k + j, step
        // k + j - (W-1) of the thread.
        float2 g[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) g[i] = both(0.f);
        const auto spread = [&](int k, float2 q, auto cutting) {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const int i = k + j - (W - 1);
                if (i >= 0 && i < kV) g[i] = fma2(both(w[j]), cutting.value ? seen(q, cut[j], k) : q, g[i]);
            }
        };
        const auto output = [&](int k, auto cutting) {
            float2 tap[W];
#pragma unroll
            for (int j = 0; j < W; ++j) tap[j] = cutting.value ? seen(win.v[k + j], cut[j], k) : win.v[k + j];
            if (silu) {
                float2 pre = both(bias);
#pragma unroll
                for (int j = 0; j < W; ++j) pre = fma2(both(w[j]), tap[j], pre);
                slope[k] = conv_slope<Tin>(pre, slope[k]);
            }
#pragma unroll
            for (int j = 0; j < W; ++j) sum2[j] = fma2(slope[k], tap[j], sum2[j]);
            sum2[W] = add2(sum2[W], slope[k]);
            spread(k, slope[k], cutting);
        };
#pragma unroll
        for (int k = 0; k < kV; ++k) {
            if (kR && (slow >> k & 1u)) output(k, std::true_type{});
            else output(k, std::false_type{});
        }
        // The W - 1 outputs behind: the second halves' firsts, and those of the
        // next thread, for the last one thread 0's of the round before.
#pragma unroll
        for (int k = 0; k < W - 1; ++k) heads[buf][k][t] = slope[k].x;
        __syncthreads();  // (and the slots of this half may be filled again)
        const float *next_heads = t + 1 < (int)blockDim.x ? &heads[buf][0][t + 1] : &heads[buf ^ 1][0][0];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            float2 q2 = make_float2(slope[k].y, next_heads[k * kConvBwdThreads]);
            if (s.tail <= kSpan) q2.y = 0.f;
            if (kR && (slow >> (k + kV) & 1u)) spread(k + kV, q2, std::true_type{});
            else spread(k + kV, q2, std::false_type{});
        }
        if (p.dlast && there && s.t0 + kSpan > L - (W - 1)) {  // the last state's elements are inputs too
            bool seen = true;
            for (int64_t t = L - 1; t >= s.t0 && t >= 0 && t >= L - (W - 1); --t) {
                const int i = (int)(t - s.t0);
                if (i < kSpan && seen) {
                    const float f = load_elem(static_cast<const Tin *>(p.dlast), row * (W - 1) + t - (L - (W - 1)));
#pragma unroll
                    for (int k = 0; k < kV; ++k) {
                        if (k == i) g[k].x += f;
                        if (k + kV == i) g[k].y += f;
                    }
                }
                if (starts_at(p, b, t)) seen = false;
            }
        }
        float g0[kV], g1[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) g0[i] = g[i].x, g1[i] = g[i].y;
        if (whole) {
            store_vec(dx + s.e, g0);
            store_vec(dx + s.e + kV, g1);
        } else {
            store8(dx + s.e, 0, s.lo(0), s.hi(0), vec, g0);
            store8(dx + s.e, kV, s.lo(kV), s.hi(kV), vec, g1);
        }
    }
    float sum[W + 1];
#pragma unroll
    for (int j = 0; j <= W; ++j) sum[j] = sum2[j].x + sum2[j].y;
    // Outputs outside the row have dy = 0, but their taps are the state, or the
    // row's last inputs, and zero times an infinity or a NaN there is a NaN.  So
    // a thread that had such outputs and ends with a NaN adds up anew, over the
    // row's outputs alone.  (Clearing those outputs' taps as they are met would
    // cost every row end some 20 selects an output; this changes calls without
    // a NaN by 1.5 % at most, 8 x 1536 x 2047 64.1 to 65.1 us.  Calls full of
    // NaN take 0.45 ms there, four to nine times as long as others.)
    bool nan = false;
#pragma unroll
    for (int j = 0; j <= W; ++j) nan |= sum[j] != sum[j];
    bool cut_short = false;
    if (nan)
        for (int64_t round = first; round < behind; ++round) {
            s = place(round * blockDim.x + t, b);
            cut_short |= s.head < 0 || s.tail < kSpan;
        }
    if (cut_short) {
#pragma unroll
        for (int j = 0; j <= W; ++j) sum[j] = 0.f;
#pragma unroll 1
        for (int64_t round = first; round < behind; ++round) {
            s = place(round * blockDim.x + t, b);
#pragma unroll 1
            for (int k = max(-s.head, 0); k < min(s.tail, kSpan); ++k) {
                const int64_t row = b * p.dim + d, at = s.t0 + k;
                float q = load_elem(dy, row * L + at);
                if (silu) q = conv_slope<Tin>(both(conv_at<Tin, W>(p, row, at, w, bias)), both(q)).x;
                bool seen = true;
#pragma unroll
                for (int j = W - 1; j >= 0; --j) {  // from step `at` back
                    const int64_t u = at - (W - 1) + j;
                    sum[j] = fmaf(q, seen ? conv_input<Tin, W>(p, row, u) : 0.f, sum[j]);
                    if (u >= 0 && starts_at(p, b, u)) seen = false;
                }
                sum[W] += q;
            }
        }
    }

    // the state's gradient: outputs 0 .. W-2 reach it
    if (p.dh0) {
        for (int64_t i = (int64_t)rank * blockDim.x + threadIdx.x; i < p.batch * (W - 1); i += (int64_t)nblk * blockDim.x) {
            const int64_t b = i / (W - 1), row = b * p.dim + d;
            const int k = (int)(i % (W - 1));  // step k - (W-1)
            float acc = 0.f;
            bool seen = true;
            for (int64_t t = 0; t <= k && t < L && seen; ++t) {
                if (starts_at(p, b, t)) seen = false;
                if (!seen) break;
                const float pre = silu ? conv_at<Tin, W>(p, row, t, w, bias) : 0.f;
                const float dyt = load_elem(dy, row * L + t);
                const float slope = silu ? conv_slope<Tin>(both(pre), both(dyt)).x : dyt;
#pragma unroll
                for (int j = 0; j < W; ++j)
                    if (j == k - t) acc = fmaf(w[j], slope, acc);
            }
            // the steps before a short row stay in its last state
            if (p.dlast && k >= L) {
                bool kept = true;
                for (int64_t t = 0; t < L; ++t) kept = kept && !starts_at(p, b, t);
                if (kept) acc += load_elem(static_cast<const Tin *>(p.dlast), row * (W - 1) + k - L);
            }
            put(static_cast<Tin *>(p.dh0), row * (W - 1) + k, acc);
        }
    }

    // threads -> warps -> block -> cluster
    __shared__ float part[kConvBwdThreads / 32][kMaxWidth + 1];
    __shared__ float mine[kMaxWidth + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
#pragma unroll
        for (int o = 16; o >= 1; o /= 2) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
        if (lane == 0) part[warp][j] = sum[j];
    }
    __syncthreads();
    if (threadIdx.x <= W) {
        float s = 0.f;
        for (int k = 0; k < (int)blockDim.x / 32; ++k) s += part[k][threadIdx.x];
        mine[threadIdx.x] = s;
    }
    if (nblk > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (rank == 0 && threadIdx.x <= W) {
            float s = 0.f;
            for (int k = 0; k < nblk; ++k) {
                uint32_t at = smem_addr(&mine[threadIdx.x]), peer;
                float v;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(at), "r"(k));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer) : "memory");
                s += v;
            }
            mine[threadIdx.x] = s;
        }
        // no block leaves while its sums are read (and rank 0 read its own before writing it above)
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
        __syncthreads();
    }
    if (rank == 0 && threadIdx.x <= W) {
        if (threadIdx.x < W) {
            if (p.dweight) p.dweight[d * W + threadIdx.x] = mine[threadIdx.x];
        } else if (p.dbias) {
            p.dbias[d] = mine[W];
        }
    }
}

}  // namespace selscan
