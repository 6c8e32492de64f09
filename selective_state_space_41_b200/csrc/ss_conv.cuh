// The causal depthwise convolution: forward, backward and one decoding step
// (declarations and the meaning of every argument in include/selscan.h).
//
//   p_t = bias + sum_(j < W) w_j x_(t - (W-1) + j),   y_t = p_t or silu(p_t)
//
// per row (b, d), with the steps before the row taken from a state (or zero)
// and nothing read across a sequence start.
//
// Forward: two bytes in and two out per bf16 element against 2 W + 5
// operations, so it is bound by memory.  The outputs of all rows form one
// flat array, eight of them per thread, so every length fills the warps and
// every access is an aligned vector; the W - 1 steps before a thread's own
// come from the vector before, which its neighbour loads too (an L1 hit).
// A vector that spans two rows (odd lengths) is worked element by element.
//
// Backward: with q_t = dy_t (silu'(p_t)),
//   dx_s = sum_j w_j q_(s + (W-1) - j),   dw_j = sum_t q_t x_(t - (W-1) + j),   dbias = sum_t q_t.
// p is recomputed from x.  dw and dbias sum over batch and steps for each
// channel, so a block (or a cluster of blocks, when the channels are few)
// takes one channel and all of its batch entries; every thread keeps its W + 1
// sums in registers over all its vectors and they are joined once at the end,
// in a fixed order and without a second launch.
#pragma once

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
};

cudaError_t conv_fwd_f32_f32(int width, cudaStream_t s, ConvParams &p);
cudaError_t conv_fwd_bf16_bf16(int width, cudaStream_t s, ConvParams &p);
cudaError_t conv_fwd_bf16_f32(int width, cudaStream_t s, ConvParams &p);
cudaError_t conv_bwd_f32_f32(int width, cudaStream_t s, const ConvParams &p);
cudaError_t conv_bwd_bf16_bf16(int width, cudaStream_t s, const ConvParams &p);
cudaError_t conv_bwd_bf16_f32(int width, cudaStream_t s, const ConvParams &p);

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

template <bool kFast>
__device__ __forceinline__ float silu_of(float v) {
    float s, c;
    sigmoid2<kFast>(v, s, c);
    return v * s;
}

template <typename Tin, typename Tout, int W, bool kR>
__global__ void __launch_bounds__(256) conv_fwd_kernel(const ConvParams p) {
    constexpr bool kFast = sizeof(Tin) == 2;
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
    const int64_t e = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * kV;
    if (e >= n) return;
    const int64_t row = n <= INT_MAX ? (int64_t)((uint32_t)e / (uint32_t)L) : e / L;
    const int64_t t0 = e - row * L;
    const int64_t b = rows <= INT_MAX ? (int64_t)((uint32_t)row / (uint32_t)p.dim) : row / p.dim;
    const int64_t d = row - b * p.dim;
    const Tin *x = static_cast<const Tin *>(p.x);
    Tout *y = static_cast<Tout *>(p.y);
    float out[kV];
    if (t0 + kV <= L) {
        float w[W];
#pragma unroll
        for (int j = 0; j < W; ++j) w[j] = __ldg(p.weight + d * W + j);
        const float bias = p.bias ? __ldg(p.bias + d) : 0.f;
        float win[W - 1 + kV];  // steps t0 - (W-1) .. t0 + 7
        Vec8<Tin> own;
        load8(own, x, e, 0, kV, p.vec);
        if (t0 >= W - 1) {
            Vec8<Tin> prev;
            if (p.vec) prev.load(x, e - kV);
            else prev.load_part(x, e - kV, kV - (W - 1), kV);
#pragma unroll
            for (int k = 0; k < W - 1; ++k) win[k] = prev[kV - (W - 1) + k];
        } else {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) win[k] = conv_input<Tin, W>(p, row, t0 - (W - 1) + k);
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) win[W - 1 + i] = own[i];
        if constexpr (kR) {
            // bit k: a sequence starts at step t0 - (W-1) + k
            const int lo = t0 >= kV ? 0 : (int)(kV - t0);
            const uint32_t before = start_bits(p.reset, b * L + t0 - kV, p.batch * L, lo, kV) >> (kV - (W - 1));
            const uint32_t m = before | start_bits(p.reset, b * L + t0, p.batch * L, 0, kV) << (W - 1);
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                float acc = bias;
                bool seen = true;
                float xs[W];
#pragma unroll
                for (int j = W - 1; j >= 0; --j) {
                    xs[j] = seen ? win[i + j] : 0.f;
                    seen = seen && !(m >> (i + j) & 1u);
                }
#pragma unroll
                for (int j = 0; j < W; ++j) acc = fmaf(w[j], xs[j], acc);
                out[i] = acc;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                float acc = bias;
#pragma unroll
                for (int j = 0; j < W; ++j) acc = fmaf(w[j], win[i + j], acc);
                out[i] = acc;
            }
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < kV; ++i) {
            if (e + i >= n) break;
            const int64_t r = (e + i) / L, c = r % p.dim;
            float w[W];
#pragma unroll
            for (int j = 0; j < W; ++j) w[j] = __ldg(p.weight + c * W + j);
            const float v = conv_at<Tin, W>(p, r, e + i - r * L, w, p.bias ? __ldg(p.bias + c) : 0.f);
            put(y, e + i, p.silu ? silu_of<kFast>(v) : v);
        }
        return;
    }
    if (p.silu) {
#pragma unroll
        for (int i = 0; i < kV; ++i) out[i] = silu_of<kFast>(out[i]);
    }
    store8(y, e, 0, kV, p.vec, out);
}

// q_t from p_t and dy_t.
template <bool kFast>
__device__ __forceinline__ float conv_slope(float pre, float dy, bool silu) {
    if (!silu) return dy;
    float s, c;
    sigmoid2<kFast>(pre, s, c);
    return dy * (s * fmaf(pre, c, 1.f));
}

constexpr int kConvBwdThreads = 256;

template <typename Tin, typename Tout, int W, bool kR>
__global__ void __launch_bounds__(kConvBwdThreads) conv_bwd_kernel(const ConvParams p, int nblk) {
    constexpr bool kFast = sizeof(Tin) == 2;
    const int64_t L = p.L;
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

    float sum[W + 1];  // dw_j, dbias
#pragma unroll
    for (int j = 0; j <= W; ++j) sum[j] = 0.f;

    // Vectors of the channel's rows, in virtual steps: nv for each batch entry.
    const int64_t nv = (L + 2 * kV - 2) / kV;
    const int64_t total = p.batch * nv, stride = (int64_t)nblk * blockDim.x;
    for (int64_t q = (int64_t)rank * blockDim.x + threadIdx.x; q < total; q += stride) {
        const int64_t b = q / nv;
        const int64_t row = b * p.dim + d, e0 = row * L;
        const int64_t t0 = (q - b * nv) * kV - (e0 & (kV - 1)), e = e0 + t0;
        const int lo = clamp8(-t0), hi = clamp8(L - t0);
        if (hi <= lo) continue;
        constexpr int kWin = kV + 2 * (W - 1);  // x at steps t0 - (W-1) .. t0 + 7 + (W-1)
        constexpr int kOut = kV + W - 1;        // q at steps t0 .. t0 + 7 + (W-1)
        float win[kWin], slope[kOut];
        {
            Vec8<Tin> v;
            const bool in = vec && t0 >= kV && t0 + 2 * kV <= L;  // all three vectors lie in the row
            if (in) {
                v.load(x, e - kV);
#pragma unroll
                for (int k = 0; k < W - 1; ++k) win[k] = v[kV - (W - 1) + k];
                v.load(x, e);
#pragma unroll
                for (int k = 0; k < kV; ++k) win[W - 1 + k] = v[k];
                v.load(x, e + kV);
#pragma unroll
                for (int k = 0; k < W - 1; ++k) win[W - 1 + kV + k] = v[k];
                Vec8<Tout> u;
                u.load(dy, e);
#pragma unroll
                for (int k = 0; k < kV; ++k) slope[k] = u[k];
                u.load(dy, e + kV);
#pragma unroll
                for (int k = 0; k < W - 1; ++k) slope[kV + k] = u[k];
            } else {
#pragma unroll
                for (int k = 0; k < kWin; ++k) {
                    const int64_t t = t0 - (W - 1) + k;
                    win[k] = t >= -(W - 1) && t < L ? conv_input<Tin, W>(p, row, t) : 0.f;
                }
#pragma unroll
                for (int k = 0; k < kOut; ++k) {
                    const int64_t t = t0 + k;
                    slope[k] = t >= 0 && t < L ? load_elem(dy, e0 + t) : 0.f;
                }
            }
        }
        uint32_t m = 0;  // bit k: a sequence starts at step t0 - (W-1) + k
        if constexpr (kR) {
#pragma unroll
            for (int k = 0; k < kWin; ++k) {
                const int64_t t = t0 - (W - 1) + k;
                if (t >= 0 && t < L && starts_at(p, b, t)) m |= 1u << k;
            }
        }
        // p_t and q_t; a tap j of output k reads win[k + j] unless a start lies behind it
        const auto cut = [&](int k, int j) {  // a start in the steps after win[k + j] up to output k's own
            return kR && (m >> (k + j + 1) & ((1u << (W - 1 - j)) - 1u)) != 0;
        };
#pragma unroll
        for (int k = 0; k < kOut; ++k) {
            if (silu) {
                float pre = bias;
#pragma unroll
                for (int j = 0; j < W; ++j) pre = fmaf(w[j], cut(k, j) ? 0.f : win[k + j], pre);
                const bool inside = t0 + k >= 0 && t0 + k < L;
                slope[k] = inside ? conv_slope<kFast>(pre, slope[k], true) : 0.f;
            }
        }
        float g[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            float acc = 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) {  // output step i + j, whose tap W-1-j reads step i
                const int k = i + j;
                acc = cut(k, W - 1 - j) ? acc : fmaf(w[W - 1 - j], slope[k], acc);
            }
            g[i] = acc;
        }
        if (p.dlast && t0 + kV > L - (W - 1)) {
            bool seen = true;
            for (int64_t s = L - 1; s >= t0 && s >= 0 && s >= L - (W - 1); --s) {
                const int64_t i = s - t0;
                if (i < kV && seen) {
#pragma unroll
                    for (int k = 0; k < kV; ++k)
                        if (k == i) g[k] += load_elem(static_cast<const Tin *>(p.dlast), row * (W - 1) + s - (L - (W - 1)));
                }
                if (starts_at(p, b, s)) seen = false;
            }
        }
        store8(dx, e, lo, hi, vec, g);
        // the channel's sums, over this vector's own outputs
#pragma unroll
        for (int i = 0; i < kV; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) sum[j] = cut(i, j) ? sum[j] : fmaf(slope[i], win[i + j], sum[j]);
            sum[W] += slope[i];
        }
    }

    // the state's gradient: outputs 0 .. W-2 reach it
    if (p.dh0) {
        for (int64_t i = (int64_t)rank * blockDim.x + threadIdx.x; i < p.batch * (W - 1); i += stride) {
            const int64_t b = i / (W - 1), row = b * p.dim + d;
            const int k = (int)(i % (W - 1));  // step k - (W-1)
            float acc = 0.f;
            bool seen = true;
            for (int64_t t = 0; t <= k && t < L && seen; ++t) {
                if (starts_at(p, b, t)) seen = false;
                if (!seen) break;
                const float pre = silu ? conv_at<Tin, W>(p, row, t, w, bias) : 0.f;
                const float slope = conv_slope<kFast>(pre, load_elem(dy, row * L + t), silu);
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
        for (int k = 0; k < kConvBwdThreads / 32; ++k) s += part[k][threadIdx.x];
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
