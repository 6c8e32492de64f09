// Layer norm (and its RMS form) over the channels, forward and backward
// (declarations and the meaning of every argument in include/selscan.h).
//
//   m = sum_d x / D,  r = (sum_d (x - m)^2 / D + eps)^(-1/2),  xh = (x - m) r,
//   y = xh w + b                                     (RMS form: m = 0)
//   dx = r (v - sum_d v / D - xh sum_d v xh / D) with v = dy w   (RMS: without the middle term)
//   dw = sum dy xh,  db = sum dy  over all steps of the batch
//
// All four kernels are bound by memory: x is read once (backward: x and dy)
// and a result written once, against some ten operations an element.  What a
// row needs twice therefore stays in registers between its sums and its
// results.
//
// seqlen = 1 (rows of dim contiguous elements): a warp or a block takes a
// row, 8-element vectors dealt out over its threads.  In the backward the
// blocks stay and walk over the rows, so a thread keeps its columns, and
// their parts of dw and db are sums in its registers.
//
// seqlen > 1: the channels of a step lie L elements apart.  A lane takes one
// step, a warp 32 steps of kNch channels: every access is then 32
// neighbouring elements whatever L is, and the sums over channels stay
// within the lane but for one exchange between the warps, and between the
// blocks of a cluster when one block's registers do not hold dim channels.
// The backward needs sums over the steps as well; those of 32 channels come
// out of 31 shuffles (each round halves the values a lane still holds and
// doubles the lanes they sum over) and stay with lane i for channel i.
//
// dw and db leave each block (or cluster) as one row of partial sums in the
// workspace; a second kernel adds the rows in a fixed order, so the results
// do not change from run to run.
#include "ss_layer.cuh"

namespace selscan {
namespace {

struct NormParams {
    const void *x, *dy;
    const float *weight, *bias, *mean_in, *rstd_in;
    void *y, *dx;
    float *mean, *rstd;
    float *part;  // backward: parts x 2 x dim (dw, db)
    int64_t batch, dim, L;
    float eps, inv_dim;
    int rms;
    int sums;     // backward: dw and db wanted
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum of a and b over the T threads of a row (T = 32: a warp; else the block).
template <int kN>
__device__ __forceinline__ void row_sum(float (&v)[kN], int T, float (*red)[kN]) {
#pragma unroll
    for (int k = 0; k < kN; ++k) v[k] = warp_sum(v[k]);
    if (T == 32) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
#pragma unroll
        for (int k = 0; k < kN; ++k) red[warp][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        float s = 0.f;
        for (int i = 0; i < (T >> 5); ++i) s += red[i][k];
        v[k] = s;
    }
}

// ------------------------------------------------------------------- rows

// Column of element i of a thread's vector k: vectors of 8, or single
// elements where rows are not whole vectors or a base is not on 16 bytes.
template <bool kVec>
__device__ __forceinline__ int64_t column(int k, int i, int t, int T) {
    return kVec ? ((int64_t)k * T + t) * kV + i : ((int64_t)k * kV + i) * T + t;
}

template <typename T, int kNv, bool kVec>
__device__ __forceinline__ void load_row(Vec8<T> (&r)[kNv], const T *row, int t, int T_, int64_t dim) {
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
        r[k].clear();
        if constexpr (kVec) {
            const int64_t c = column<true>(k, 0, t, T_);
            if (c < dim) r[k].load(row, c);
        } else {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const int64_t c = column<false>(k, i, t, T_);
                if (c < dim) r[k].set(row, c, i);
            }
        }
    }
}

template <bool kVec>
__device__ __forceinline__ void load_cols(float (&w)[kV], const float *p, int k, int t, int T, int64_t dim, float none) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < kV; ++i) w[i] = none;
    } else if constexpr (kVec) {
        const int64_t c = column<true>(k, 0, t, T);
        if (c >= dim) return;
#pragma unroll
        for (int i = 0; i < kV; ++i) w[i] = __ldg(p + c + i);
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int64_t c = column<false>(k, i, t, T);
            w[i] = c < dim ? __ldg(p + c) : 0.f;
        }
    }
}

template <typename T, bool kVec>
__device__ __forceinline__ void store_cols(T *row, const float (&v)[kV], int k, int t, int T_, int64_t dim) {
    if constexpr (kVec) {
        const int64_t c = column<true>(k, 0, t, T_);
        if (c < dim) store_vec(row + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int64_t c = column<false>(k, i, t, T_);
            if (c < dim) put(row, c, v[i]);
        }
    }
}

// T threads a row; with T = 32 each of the block's warps has a row.
template <typename Tin, typename Tout, int kNv, bool kVec>
__global__ void __launch_bounds__(512) norm_rows_fwd_kernel(const NormParams p, int T) {
    __shared__ float red[2][32][1];
    const int t = T == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = T == 32 ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= p.batch) return;
    Vec8<Tin> x[kNv];
    load_row<Tin, kNv, kVec>(x, static_cast<const Tin *>(p.x) + row * p.dim, t, T, p.dim);
    float mean = 0.f;
    if (!p.rms) {
        float s[1] = {0.f};
#pragma unroll
        for (int k = 0; k < kNv; ++k)
#pragma unroll
            for (int i = 0; i < kV; ++i) s[0] += x[k][i];
        row_sum<1>(s, T, red[0]);
        mean = s[0] * p.inv_dim;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int k = 0; k < kNv; ++k)
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const float c = x[k][i] - mean;
            if (column<kVec>(k, i, t, T) < p.dim) q[0] = fmaf(c, c, q[0]);
        }
    row_sum<1>(q, T, red[1]);
    const float rstd = rsqrtf(fmaf(q[0], p.inv_dim, p.eps));
    if (t == 0) {
        if (p.mean && !p.rms) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    Tout *y = static_cast<Tout *>(p.y) + row * p.dim;
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
        float w[kV], b[kV], v[kV];
        load_cols<kVec>(w, p.weight, k, t, T, p.dim, 1.f);
        load_cols<kVec>(b, p.bias, k, t, T, p.dim, 0.f);
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = fmaf((x[k][i] - mean) * rstd, w[i], b[i]);
        store_cols<Tout, kVec>(y, v, k, t, T, p.dim);
    }
}

// Rows too wide for a block's registers: three passes over the row (the
// later ones from the caches).
template <typename Tin, typename Tout>
__global__ void __launch_bounds__(1024) norm_rows_fwd_wide_kernel(const NormParams p) {
    __shared__ float red[2][32][1];
    const int64_t row = blockIdx.x;
    const Tin *x = static_cast<const Tin *>(p.x) + row * p.dim;
    float s[1] = {0.f}, q[1] = {0.f};
    if (!p.rms)
        for (int64_t c = threadIdx.x; c < p.dim; c += blockDim.x) s[0] += load_elem(x, c);
    row_sum<1>(s, blockDim.x, red[0]);
    const float mean = s[0] * p.inv_dim;
    for (int64_t c = threadIdx.x; c < p.dim; c += blockDim.x) {
        const float v = load_elem(x, c) - mean;
        q[0] = fmaf(v, v, q[0]);
    }
    row_sum<1>(q, blockDim.x, red[1]);
    const float rstd = rsqrtf(fmaf(q[0], p.inv_dim, p.eps));
    if (threadIdx.x == 0) {
        if (p.mean && !p.rms) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    Tout *y = static_cast<Tout *>(p.y) + row * p.dim;
    for (int64_t c = threadIdx.x; c < p.dim; c += blockDim.x)
        put(y, c, fmaf((load_elem(x, c) - mean) * rstd, p.weight ? __ldg(p.weight + c) : 1.f, p.bias ? __ldg(p.bias + c) : 0.f));
}

template <typename Tin, typename Tout, int kNv, bool kVec>
__global__ void __launch_bounds__(512) norm_rows_bwd_kernel(const NormParams p, int T) {
    extern __shared__ float acc[];  // T = 32: the warps' sums, joined at the end
    __shared__ float red[2][32][2];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
    const int t = T == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t step = T == 32 ? (int64_t)gridDim.x * warps : gridDim.x;
    float dw[kNv][kV], db[kNv][kV];
#pragma unroll
    for (int k = 0; k < kNv; ++k)
#pragma unroll
        for (int i = 0; i < kV; ++i) dw[k][i] = db[k][i] = 0.f;
    int buf = 0;
    for (int64_t row = T == 32 ? (int64_t)blockIdx.x * warps + warp : blockIdx.x; row < p.batch; row += step, buf ^= 1) {
        Vec8<Tin> x[kNv];
        Vec8<Tout> dy[kNv];
        load_row<Tin, kNv, kVec>(x, static_cast<const Tin *>(p.x) + row * p.dim, t, T, p.dim);
        load_row<Tout, kNv, kVec>(dy, static_cast<const Tout *>(p.dy) + row * p.dim, t, T, p.dim);
        const float mean = p.mean_in ? __ldg(p.mean_in + row) : 0.f, rstd = __ldg(p.rstd_in + row);
        float c[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < kNv; ++k) {
            float w[kV];
            load_cols<kVec>(w, p.weight, k, t, T, p.dim, 1.f);
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                if (column<kVec>(k, i, t, T) < p.dim) {
                    const float g = dy[k][i], xh = (x[k][i] - mean) * rstd, v = g * w[i];
                    c[0] += v;
                    c[1] = fmaf(v, xh, c[1]);
                    dw[k][i] = fmaf(g, xh, dw[k][i]);
                    db[k][i] += g;
                }
            }
        }
        row_sum<2>(c, T, red[buf]);
        const float c1 = p.mean_in ? c[0] * p.inv_dim : 0.f, c2 = c[1] * p.inv_dim;
        Tin *dx = static_cast<Tin *>(p.dx) + row * p.dim;
#pragma unroll
        for (int k = 0; k < kNv; ++k) {
            float w[kV], v[kV];
            load_cols<kVec>(w, p.weight, k, t, T, p.dim, 1.f);
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const float xh = (x[k][i] - mean) * rstd;
                v[i] = (fmaf(dy[k][i], w[i], -c1) - xh * c2) * rstd;
            }
            store_cols<Tin, kVec>(dx, v, k, t, T, p.dim);
        }
    }
    if (!p.sums) return;
    float *out = p.part + (int64_t)blockIdx.x * 2 * p.dim;
    if (T == 32) {
        // the block's warps hold the same columns
        for (int w = 0; w < warps; ++w) {
            if (warp == w) {
#pragma unroll
                for (int k = 0; k < kNv; ++k)
#pragma unroll
                    for (int i = 0; i < kV; ++i) {
                        const int64_t c = column<kVec>(k, i, t, 32);
                        if (c < p.dim) {
                            acc[c] = w ? acc[c] + dw[k][i] : dw[k][i];
                            acc[p.dim + c] = w ? acc[p.dim + c] + db[k][i] : db[k][i];
                        }
                    }
            }
            __syncthreads();
        }
        for (int64_t c = threadIdx.x; c < 2 * p.dim; c += blockDim.x) out[c] = acc[c];
    } else {
#pragma unroll
        for (int k = 0; k < kNv; ++k) {
            store_cols<float, kVec>(out, dw[k], k, t, T, p.dim);
            store_cols<float, kVec>(out + p.dim, db[k], k, t, T, p.dim);
        }
    }
}

// Rows too wide for a block's registers: a block per group of rows, its sums
// kept in its own row of partial sums.
template <typename Tin, typename Tout>
__global__ void __launch_bounds__(1024) norm_rows_bwd_wide_kernel(const NormParams p) {
    __shared__ float red[2][32][2];
    float *out = p.part + (int64_t)blockIdx.x * 2 * p.dim;
    int buf = 0;
    bool first = true;
    for (int64_t row = blockIdx.x; row < p.batch; row += gridDim.x, buf ^= 1, first = false) {
        const Tin *x = static_cast<const Tin *>(p.x) + row * p.dim;
        const Tout *dy = static_cast<const Tout *>(p.dy) + row * p.dim;
        Tin *dx = static_cast<Tin *>(p.dx) + row * p.dim;
        const float mean = p.mean_in ? __ldg(p.mean_in + row) : 0.f, rstd = __ldg(p.rstd_in + row);
        float c[2] = {0.f, 0.f};
        for (int64_t d = threadIdx.x; d < p.dim; d += blockDim.x) {
            const float g = load_elem(dy, d), xh = (load_elem(x, d) - mean) * rstd;
            const float v = p.weight ? g * __ldg(p.weight + d) : g;
            c[0] += v;
            c[1] = fmaf(v, xh, c[1]);
            if (p.sums) {  // this thread's columns alone
                out[d] = first ? g * xh : fmaf(g, xh, out[d]);
                out[p.dim + d] = first ? g : out[p.dim + d] + g;
            }
        }
        row_sum<2>(c, blockDim.x, red[buf]);
        const float c1 = p.mean_in ? c[0] * p.inv_dim : 0.f, c2 = c[1] * p.inv_dim;
        for (int64_t d = threadIdx.x; d < p.dim; d += blockDim.x) {
            const float w = p.weight ? __ldg(p.weight + d) : 1.f, xh = (load_elem(x, d) - mean) * rstd;
            put(dx, d, (fmaf(load_elem(dy, d), w, -c1) - xh * c2) * rstd);
        }
    }
}

// ------------------------------------------------------------------ steps

constexpr int kNch = 32;  // channels a lane holds

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float peer_load(const float *p, int rank) {
    uint32_t peer;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer) : "memory");
    return v;
}

// A step's place: element of channel 0, and whether there is such a step.
struct Step {
    int64_t at, index;
    bool in;
};
__device__ __forceinline__ Step step_of(const NormParams &p, int64_t tile, int lane) {
    const int64_t s = tile * 32 + lane, n = p.batch * p.L;
    Step r;
    r.in = s < n;
    r.index = r.in ? s : n - 1;
    const int64_t b = r.index / p.L;
    r.at = b * p.dim * p.L + (r.index - b * p.L);
    return r;
}

// Forward over steps: nblk blocks of a cluster share the channels.
template <typename Tin, typename Tout>
__global__ void __launch_bounds__(512) norm_steps_fwd_kernel(const NormParams p, int nblk) {
    __shared__ float sm[2][16][32];  // per warp: mean and squares about it
    __shared__ float all[2][32];     // the block's
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int rank = (int)(blockIdx.x % nblk);
    const int64_t c0 = ((int64_t)rank * warps + warp) * kNch;
    const Step st = step_of(p, blockIdx.x / nblk, lane);
    const Tin *x = static_cast<const Tin *>(p.x) + st.at;
    const int have = c0 >= p.dim ? 0 : p.dim - c0 < kNch ? (int)(p.dim - c0) : kNch;
    float v[kNch];
#pragma unroll
    for (int i = 0; i < kNch; ++i) v[i] = i < have ? load_elem(x, (c0 + i) * p.L) : 0.f;

    // Mean and squares about it, joined from parts (n, m, S):
    // m = sum n_i m_i / n,  S = sum S_i + sum n_i (m_i - m)^2.
    const auto count = [&](int64_t first, int64_t width) {  // channels of a part
        const int64_t k = p.dim - first;
        return k <= 0 ? 0.f : (float)(k < width ? k : width);
    };
    float m = 0.f, S = 0.f;
    if (!p.rms && have) {
#pragma unroll
        for (int i = 0; i < kNch; ++i) m += v[i];
        m /= (float)have;
    }
#pragma unroll
    for (int i = 0; i < kNch; ++i) {
        const float c = v[i] - m;
        if (i < have) S = fmaf(c, c, S);
    }
    sm[0][warp][lane] = m, sm[1][warp][lane] = S;
    __syncthreads();
    const int64_t b0 = (int64_t)rank * warps * kNch;
    if (warp == 0) {
        float n = 0.f, mb = 0.f, Sb = 0.f;
        for (int k = 0; k < warps; ++k) {
            const float nk = count(b0 + k * kNch, kNch);
            mb = fmaf(nk, sm[0][k][lane], mb);
            n += nk;
        }
        mb = n > 0.f ? mb / n : 0.f;
        for (int k = 0; k < warps; ++k) {
            const float d = sm[0][k][lane] - mb;
            Sb += fmaf(count(b0 + k * kNch, kNch) * d, d, sm[1][k][lane]);
        }
        all[0][lane] = mb, all[1][lane] = Sb;
    }
    if (nblk > 1) cluster_sync();
    else __syncthreads();
    float mean = 0.f, sq = 0.f;
    if (nblk > 1) {
        const int64_t wide = (int64_t)warps * kNch;
        for (int k = 0; k < nblk; ++k) mean = fmaf(count(k * wide, wide), peer_load(&all[0][lane], k), mean);
        mean *= p.inv_dim;
        for (int k = 0; k < nblk; ++k) {
            const float d = peer_load(&all[0][lane], k) - mean;
            sq += fmaf(count(k * wide, wide) * d, d, peer_load(&all[1][lane], k));
        }
    } else {
        mean = all[0][lane], sq = all[1][lane];
    }
    if (p.rms) mean = 0.f;
    const float rstd = rsqrtf(fmaf(sq, p.inv_dim, p.eps));
    if (st.in && rank == 0 && warp == 0) {
        if (p.mean && !p.rms) p.mean[st.index] = mean;
        if (p.rstd) p.rstd[st.index] = rstd;
    }
    Tout *y = static_cast<Tout *>(p.y) + st.at;
#pragma unroll
    for (int i = 0; i < kNch; ++i) {
        if (i < have) {
            const float w = p.weight ? __ldg(p.weight + c0 + i) : 1.f, b = p.bias ? __ldg(p.bias + c0 + i) : 0.f;
            if (st.in) put(y, (c0 + i) * p.L, fmaf((v[i] - mean) * rstd, w, b));
        }
    }
    if (nblk > 1) cluster_sync();  // no block leaves while its sums may be read
}

// Sums over the 32 lanes of kNch values each: value i to lane i.
__device__ __forceinline__ float lane_sums(float (&v)[kNch], int lane) {
#pragma unroll
    for (int o = 16; o >= 1; o /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int k = 0; k < o; ++k) {
            const float send = up ? v[k] : v[k + o], keep = up ? v[k + o] : v[k];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return v[0];
}

template <typename Tin, typename Tout>
__global__ void __launch_bounds__(512) norm_steps_bwd_kernel(const NormParams p, int nblk) {
    __shared__ float sm[2][16][32];
    __shared__ float all[2][2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int rank = (int)(blockIdx.x % nblk);
    const int64_t group = blockIdx.x / nblk, groups = gridDim.x / nblk;
    const int64_t c0 = ((int64_t)rank * warps + warp) * kNch;
    const int have = c0 >= p.dim ? 0 : p.dim - c0 < kNch ? (int)(p.dim - c0) : kNch;
    const int64_t tiles = (p.batch * p.L + 31) / 32;
    float dw = 0.f, db = 0.f;  // of channel c0 + lane
    int buf = 0;
    for (int64_t tile = group; tile < tiles; tile += groups, buf ^= 1) {
        const Step st = step_of(p, tile, lane);
        const Tin *x = static_cast<const Tin *>(p.x) + st.at;
        const Tout *dy = static_cast<const Tout *>(p.dy) + st.at;
        float xh[kNch], g[kNch];
#pragma unroll
        for (int i = 0; i < kNch; ++i) {
            xh[i] = i < have ? load_elem(x, (c0 + i) * p.L) : 0.f;
            g[i] = i < have && st.in ? load_elem(dy, (c0 + i) * p.L) : 0.f;
        }
        const float mean = p.mean_in ? __ldg(p.mean_in + st.index) : 0.f, rstd = __ldg(p.rstd_in + st.index);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < kNch; ++i) {
            if (i < have) {
                xh[i] = (xh[i] - mean) * rstd;
                const float v = p.weight ? g[i] * __ldg(p.weight + c0 + i) : g[i];
                s1 += v;
                s2 = fmaf(v, xh[i], s2);
            }
        }
        sm[0][warp][lane] = s1, sm[1][warp][lane] = s2;
        __syncthreads();
        if (warp < 2) {
            float s = 0.f;
            for (int k = 0; k < warps; ++k) s += sm[warp][k][lane];
            all[buf][warp][lane] = s;
        }
        // one barrier a tile: the two buffers keep a slow block's reads apart from the next tile's sums
        if (nblk > 1) cluster_sync();
        else __syncthreads();
        float c1 = 0.f, c2 = 0.f;
        if (nblk > 1) {
            for (int k = 0; k < nblk; ++k) {
                c1 += peer_load(&all[buf][0][lane], k);
                c2 += peer_load(&all[buf][1][lane], k);
            }
        } else {
            c1 = all[buf][0][lane], c2 = all[buf][1][lane];
        }
        c1 = p.mean_in ? c1 * p.inv_dim : 0.f;
        c2 *= p.inv_dim;
        Tin *dx = static_cast<Tin *>(p.dx) + st.at;
#pragma unroll
        for (int i = 0; i < kNch; ++i) {
            if (i < have) {
                const float w = p.weight ? __ldg(p.weight + c0 + i) : 1.f;
                if (st.in) put(dx, (c0 + i) * p.L, (fmaf(g[i], w, -c1) - xh[i] * c2) * rstd);
            }
        }
        if (p.sums) {
#pragma unroll
            for (int i = 0; i < kNch; ++i) xh[i] = st.in ? xh[i] * g[i] : 0.f;
            dw += lane_sums(xh, lane);
            db += lane_sums(g, lane);
        }
    }
    if (p.sums && lane < have) {
        float *out = p.part + group * 2 * p.dim;
        out[c0 + lane] = dw;
        out[p.dim + c0 + lane] = db;
    }
    if (nblk > 1) cluster_sync();
}

// More channels than a cluster's registers hold: passes over the tile, the
// later ones from the caches.
template <typename Tin, typename Tout>
__global__ void __launch_bounds__(512) norm_steps_fwd_wide_kernel(const NormParams p) {
    __shared__ float sm[2][16][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const Step st = step_of(p, blockIdx.x, lane);
    const Tin *x = static_cast<const Tin *>(p.x) + st.at;
    float mean = 0.f, s = 0.f;
    if (!p.rms) {
        for (int64_t c = warp; c < p.dim; c += warps) s += load_elem(x, c * p.L);
        sm[0][warp][lane] = s;
        __syncthreads();
        for (int k = 0; k < warps; ++k) mean += sm[0][k][lane];
        mean *= p.inv_dim;
    }
    s = 0.f;
    for (int64_t c = warp; c < p.dim; c += warps) {
        const float v = load_elem(x, c * p.L) - mean;
        s = fmaf(v, v, s);
    }
    sm[1][warp][lane] = s;
    __syncthreads();
    float sq = 0.f;
    for (int k = 0; k < warps; ++k) sq += sm[1][k][lane];
    const float rstd = rsqrtf(fmaf(sq, p.inv_dim, p.eps));
    if (!st.in) return;
    if (warp == 0) {
        if (p.mean && !p.rms) p.mean[st.index] = mean;
        if (p.rstd) p.rstd[st.index] = rstd;
    }
    Tout *y = static_cast<Tout *>(p.y) + st.at;
    for (int64_t c = warp; c < p.dim; c += warps)
        put(y, c * p.L, fmaf((load_elem(x, c * p.L) - mean) * rstd, p.weight ? __ldg(p.weight + c) : 1.f,
                             p.bias ? __ldg(p.bias + c) : 0.f));
}

template <typename Tin, typename Tout>
__global__ void __launch_bounds__(512) norm_steps_bwd_wide_kernel(const NormParams p) {
    __shared__ float sm[2][2][16][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t tiles = (p.batch * p.L + 31) / 32;
    float *out = p.part + (int64_t)blockIdx.x * 2 * p.dim;
    int buf = 0;
    bool first = true;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1, first = false) {
        const Step st = step_of(p, tile, lane);
        const Tin *x = static_cast<const Tin *>(p.x) + st.at;
        const Tout *dy = static_cast<const Tout *>(p.dy) + st.at;
        Tin *dx = static_cast<Tin *>(p.dx) + st.at;
        const float mean = p.mean_in ? __ldg(p.mean_in + st.index) : 0.f, rstd = __ldg(p.rstd_in + st.index);
        float c[2] = {0.f, 0.f};
        for (int64_t d = warp; d < p.dim; d += warps) {
            const float g = st.in ? load_elem(dy, d * p.L) : 0.f, xh = (load_elem(x, d * p.L) - mean) * rstd;
            const float v = p.weight ? g * __ldg(p.weight + d) : g;
            c[0] += v;
            c[1] = fmaf(v, xh, c[1]);
            if (p.sums) {
                const float sw = warp_sum(st.in ? g * xh : 0.f), sb = warp_sum(g);
                if (lane == 0) {  // this warp's channels alone
                    out[d] = first ? sw : out[d] + sw;
                    out[p.dim + d] = first ? sb : out[p.dim + d] + sb;
                }
            }
        }
        sm[buf][0][warp][lane] = c[0], sm[buf][1][warp][lane] = c[1];
        __syncthreads();
        float c1 = 0.f, c2 = 0.f;
        for (int k = 0; k < warps; ++k) c1 += sm[buf][0][k][lane], c2 += sm[buf][1][k][lane];
        c1 = p.mean_in ? c1 * p.inv_dim : 0.f;
        c2 *= p.inv_dim;
        if (st.in)
            for (int64_t d = warp; d < p.dim; d += warps) {
                const float w = p.weight ? __ldg(p.weight + d) : 1.f, xh = (load_elem(x, d * p.L) - mean) * rstd;
                put(dx, d * p.L, (fmaf(load_elem(dy, d * p.L), w, -c1) - xh * c2) * rstd);
            }
    }
}

// dw and db from the rows of partial sums, in order: 32 columns by 8 runs of
// rows per block, the runs joined in shared memory.
__global__ void __launch_bounds__(256) norm_sums_kernel(const float *part, int64_t parts, int64_t dim, float *dweight,
                                                        float *dbias) {
    __shared__ float sm[8][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + tx;
    float s = 0.f;
    if (c < 2 * dim) {
#pragma unroll 4
        for (int64_t k = ty; k < parts; k += 8) s += part[k * 2 * dim + c];
    }
    sm[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < 2 * dim) {
        float v = 0.f;
        for (int k = 0; k < 8; ++k) v += sm[k][tx];
        if (c < dim) {
            if (dweight) dweight[c] = v;
        } else if (dbias) {
            dbias[c - dim] = v;
        }
    }
}

// ------------------------------------------------------------------- host

// The launch of a shape: kernel family, threads and blocks.
struct NormPlan {
    bool rows, wide;
    int T, nv;         // rows: threads per row, vectors per thread
    int warps, nblk;   // steps: warps per block, blocks per cluster
    int64_t parts;     // backward: rows of partial sums (blocks or clusters)
};

constexpr int kRowWarps = 4;  // rows per block where a warp takes a row

NormPlan norm_plan(const ss_desc *desc) {
    NormPlan pl{};
    const int64_t sms = layer_sm_count();
    pl.rows = desc->seqlen == 1;
    if (pl.rows) {
        // The fewest threads whose vectors (four each at most) hold the row.
        const int64_t vecs = (desc->dim + kV - 1) / kV;
        pl.T = 32;
        while (pl.T < 512 && vecs > (int64_t)pl.T * 4) pl.T *= 2;
        pl.nv = (int)((vecs + pl.T - 1) / pl.T);
        pl.wide = pl.nv > 4;
        const int per = !pl.wide && pl.T == 32 ? kRowWarps : 1;
        const int64_t blocks = (desc->batch + per - 1) / per;
        const int64_t most = pl.wide ? sms : sms * (pl.T <= 64 ? 8 : pl.T <= 128 ? 6 : pl.T <= 256 ? 3 : 1);
        pl.parts = blocks < most ? blocks : most;
    } else {
        // The channels over the warps of up to 8 blocks, 8 warps each or 16.
        const int64_t need = (desc->dim + kNch - 1) / kNch;
        pl.warps = need <= 8 ? (int)need : need <= 64 ? 8 : 16;
        if (pl.warps < 2) pl.warps = 2;
        const int64_t nblk = (need + pl.warps - 1) / pl.warps;
        pl.wide = nblk > 8;
        pl.nblk = pl.wide ? 1 : (int)nblk;
        const int64_t tiles = (desc->batch * desc->seqlen + 31) / 32;
        const int64_t most = pl.wide ? sms : (sms * 2 * 8 / pl.warps + pl.nblk - 1) / pl.nblk;
        pl.parts = tiles < most ? tiles : most;
    }
    return pl;
}

template <typename K>
cudaError_t launch_cluster(K kernel, int64_t grid, int threads, int nblk, cudaStream_t s, const NormParams &p) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)nblk;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, nblk);
}

template <typename Tin, typename Tout, int kNv, bool kVec>
cudaError_t launch_rows(bool back, const NormPlan &pl, cudaStream_t s, const NormParams &p) {
    const int threads = pl.T == 32 ? 32 * kRowWarps : pl.T;
    if (back) {
        const size_t smem = pl.T == 32 ? (size_t)p.dim * 2 * sizeof(float) : 0;
        norm_rows_bwd_kernel<Tin, Tout, kNv, kVec><<<(unsigned)pl.parts, threads, smem, s>>>(p, pl.T);
    } else {
        const int64_t grid = pl.T == 32 ? (p.batch + kRowWarps - 1) / kRowWarps : p.batch;
        norm_rows_fwd_kernel<Tin, Tout, kNv, kVec><<<(unsigned)grid, threads, 0, s>>>(p, pl.T);
    }
    return cudaGetLastError();
}

template <typename Tin, typename Tout>
cudaError_t dispatch_norm(bool back, bool vec, const NormPlan &pl, cudaStream_t s, const NormParams &p) {
    if (pl.rows && pl.wide) {
        if (back) norm_rows_bwd_wide_kernel<Tin, Tout><<<(unsigned)pl.parts, 1024, 0, s>>>(p);
        else norm_rows_fwd_wide_kernel<Tin, Tout><<<(unsigned)p.batch, 1024, 0, s>>>(p);
        return cudaGetLastError();
    }
    if (pl.rows) {
        switch (pl.nv) {
            case 1: return vec ? launch_rows<Tin, Tout, 1, true>(back, pl, s, p) : launch_rows<Tin, Tout, 1, false>(back, pl, s, p);
            case 2: return vec ? launch_rows<Tin, Tout, 2, true>(back, pl, s, p) : launch_rows<Tin, Tout, 2, false>(back, pl, s, p);
            case 3: return vec ? launch_rows<Tin, Tout, 3, true>(back, pl, s, p) : launch_rows<Tin, Tout, 3, false>(back, pl, s, p);
            default: return vec ? launch_rows<Tin, Tout, 4, true>(back, pl, s, p) : launch_rows<Tin, Tout, 4, false>(back, pl, s, p);
        }
    }
    const int64_t tiles = (p.batch * p.L + 31) / 32;
    if (pl.wide) {
        if (back) norm_steps_bwd_wide_kernel<Tin, Tout><<<(unsigned)pl.parts, 512, 0, s>>>(p);
        else norm_steps_fwd_wide_kernel<Tin, Tout><<<(unsigned)tiles, 512, 0, s>>>(p);
        return cudaGetLastError();
    }
    if (back) return launch_cluster(norm_steps_bwd_kernel<Tin, Tout>, pl.parts * pl.nblk, 32 * pl.warps, pl.nblk, s, p);
    return launch_cluster(norm_steps_fwd_kernel<Tin, Tout>, tiles * pl.nblk, 32 * pl.warps, pl.nblk, s, p);
}

ss_status check_norm(const ss_desc *desc, LayerSizes *sz) {
    const ss_status st = check_layer(desc, sz);
    if (st != SS_OK) return st;
    // blocks are counted by rows, or by 32 steps times up to 8 blocks
    if (desc->dim > INT_MAX || (desc->seqlen == 1 ? desc->batch > INT_MAX : desc->batch * desc->seqlen > (int64_t)INT_MAX * 2))
        return SS_ERR_BAD_SHAPE;
    return SS_OK;
}

NormParams norm_params(const ss_desc *desc) {
    NormParams p{};
    p.batch = desc->batch, p.dim = desc->dim, p.L = desc->seqlen;
    p.inv_dim = (float)(1.0 / (double)desc->dim);
    return p;
}

}  // namespace
}  // namespace selscan

using namespace selscan;

extern "C" {

ss_status ss_norm_fwd(const ss_desc *desc, const void *x, const float *weight, const float *bias, float eps, int rms,
                      void *y, float *mean, float *rstd, ss_stream_t stream) {
    LayerSizes sz;
    const ss_status st = check_norm(desc, &sz);
    if (st != SS_OK) return st;
    if (sz.elems == 0) return SS_OK;
    if (!x || !y) return SS_ERR_NULL_POINTER;
    const size_t ein = layer_size(desc->in_dtype), eout = layer_size(desc->out_dtype);
    if (!layer_aligned(x, ein) || !layer_aligned(y, eout)) return SS_ERR_MISALIGNED;
    for (const void *q : {(const void *)weight, (const void *)bias, (const void *)mean, (const void *)rstd})
        if (!layer_aligned(q, 4)) return SS_ERR_MISALIGNED;
    NormParams p = norm_params(desc);
    p.x = x, p.weight = weight, p.bias = bias, p.y = y, p.mean = mean, p.rstd = rstd;
    p.eps = eps, p.rms = rms != 0;
    const bool vec = desc->dim % kV == 0 && vec_ok({x, y});
    return status_of(SS_LAYER_DISPATCH(desc, dispatch_norm)(false, vec, norm_plan(desc),
                                                            reinterpret_cast<cudaStream_t>(stream), p));
}

size_t ss_norm_bwd_workspace_bytes(const ss_desc *desc) {
    LayerSizes sz;
    if (check_norm(desc, &sz) != SS_OK || sz.elems == 0) return 0;
    return (size_t)norm_plan(desc).parts * 2 * (size_t)desc->dim * sizeof(float);
}

ss_status ss_norm_bwd(const ss_desc *desc, const void *x, const float *weight, const float *mean, const float *rstd,
                      const void *dy, void *dx, float *dweight, float *dbias, void *workspace, size_t workspace_bytes,
                      ss_stream_t stream) {
    LayerSizes sz;
    const ss_status st = check_norm(desc, &sz);
    if (st != SS_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    for (const void *q : {(const void *)weight, (const void *)mean, (const void *)rstd, (const void *)dweight, (const void *)dbias})
        if (!layer_aligned(q, 4)) return SS_ERR_MISALIGNED;
    if (sz.elems == 0) {
        const size_t d = (size_t)desc->dim * 4;
        cudaError_t e = cudaSuccess;
        if (dweight && d) e = cudaMemsetAsync(dweight, 0, d, s);
        if (e == cudaSuccess && dbias && d) e = cudaMemsetAsync(dbias, 0, d, s);
        return status_of(e);
    }
    if (!x || !rstd || !dy || !dx) return SS_ERR_NULL_POINTER;
    const size_t ein = layer_size(desc->in_dtype), eout = layer_size(desc->out_dtype);
    if (!layer_aligned(x, ein) || !layer_aligned(dy, eout) || !layer_aligned(dx, ein)) return SS_ERR_MISALIGNED;
    const NormPlan pl = norm_plan(desc);
    NormParams p = norm_params(desc);
    p.sums = dweight || dbias;
    if (p.sums) {
        if (!workspace || workspace_bytes < ss_norm_bwd_workspace_bytes(desc)) return SS_ERR_WORKSPACE;
        if (!layer_aligned(workspace, 16)) return SS_ERR_MISALIGNED;
    }
    p.x = x, p.weight = weight, p.mean_in = mean, p.rstd_in = rstd, p.dy = dy, p.dx = dx;
    p.part = static_cast<float *>(workspace);
    const bool vec = desc->dim % kV == 0 && vec_ok({x, dy, dx});
    cudaError_t e = SS_LAYER_DISPATCH(desc, dispatch_norm)(true, vec, pl, s, p);
    if (e == cudaSuccess && p.sums) {
        norm_sums_kernel<<<(unsigned)((2 * p.dim + 31) / 32), 256, 0, s>>>(p.part, pl.parts, p.dim, dweight, dbias);
        e = cudaGetLastError();
    }
    return status_of(e);
}

}  // extern "C"
