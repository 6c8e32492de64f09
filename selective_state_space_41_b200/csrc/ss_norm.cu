// Layer norm (and its RMS form) over the channels, forward and backward
// (declarations and the meaning of every argument in include/selscan.h).
//
//   m = sum_d x / D,  r = (sum_d (x - m)^2 / D + eps)^(-1/2),  xh = (x - m) r,
//   y = xh w + b                                     (RMS form: m = 0)
//   dx = r (v - sum_d v / D - xh sum_d v xh / D) with v = dy w   (RMS: without the middle term)
//   dw = sum dy xh,  db = sum dy  over all steps of the batch
//
// The traffic sets the floor: x is read once (backward: x and dy) and a result
// written once, against some ten operations an element.  What a step needs
// twice therefore stays on the chip between its sums and its results.  Which
// kernel runs is a matter of shape (norm_plan):
//
// Rows (seqlen = 1: dim contiguous elements): 32 to 512 threads take a row,
// 8-element vectors dealt out over them.  In the backward the blocks stay and
// walk over the rows, so a thread keeps its columns, and their parts of dw and
// db are sums in its registers.
//
// Tiles (seqlen > 1, rows of whole vectors, all channels of 64 bytes' worth of
// steps fit into shared memory): a block copies its next tile in under the
// results of the present one.
//
// Clusters (seqlen > 1 otherwise; in words of two steps where that pays): the
// channels of a step lie L elements apart.  A warp takes 32 channels of 32 steps (or of 64 or 32 in vectors)
// into registers; the sums over channels need one exchange between the warps
// and one between the blocks of a cluster, where one block's registers do not
// hold dim channels.  The backward's sums over the steps come out of shuffles
// that halve the values a lane still holds and double the lanes they sum over.
//
// Wide (dim beyond what a block or a cluster holds): passes over the row or
// tile, the later ones from the caches.
//
// dw and db leave each block (or cluster) as one row of partial sums in the
// workspace; a second kernel adds the rows in a fixed order, so the results
// do not change from run to run.
#include <type_traits>

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

// Sums over the T threads of a row: a warp, or T / 32 warps of the block,
// which meet at a barrier of their own (`group` counts such groups).
template <int kN>
__device__ __forceinline__ void row_sum(float (&v)[kN], int T, int group, float (*red)[kN]) {
#pragma unroll
    for (int k = 0; k < kN; ++k) v[k] = warp_sum(v[k]);
    if (T == 32) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = T >> 5, first = group * n;
    if (lane == 0) {
#pragma unroll
        for (int k = 0; k < kN; ++k) red[warp][k] = v[k];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(T) : "memory");
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        float s = 0.f;
        for (int i = 0; i < n; ++i) s += red[first + i][k];
        v[k] = s;
    }
}

// ------------------------------------------------------------------- rows

// Column of element i of a thread's vector k: vectors of 8, or single
// elements where rows are not whole vectors or a base is not on 16 bytes.
template <bool kVec>
__device__ __forceinline__ int column(int k, int i, int t, int T) {
    return kVec ? (k * T + t) * kV + i : (k * kV + i) * T + t;
}

template <typename T, int kNv, bool kVec>
__device__ __forceinline__ void load_row(Vec8<T> (&r)[kNv], const T *row, int t, int T_, int dim) {
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
        r[k].clear();
        if constexpr (kVec) {
            const int c = column<true>(k, 0, t, T_);
            if (c < dim) r[k].load(row, c);
        } else {
            // no branch around a load: all of them are in flight at once
            uint32_t b[kV];
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const int c = column<false>(k, i, t, T_);
                b[i] = Io<T>::bits(row, c < dim ? c : dim - 1);
            }
#pragma unroll
            for (int i = 0; i < kV; ++i) r[k].put_bits(i, column<false>(k, i, t, T_) < dim ? b[i] : 0u);
        }
    }
}

template <bool kVec>
__device__ __forceinline__ void load_cols(float2 (&w)[kV / 2], const float *p, int k, int t, int T, int dim, float none) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < kV / 2; ++i) w[i] = both(none);
    } else if constexpr (kVec) {
        int c = column<true>(k, 0, t, T);
        c = c < dim ? c : dim - kV;
        const float4 a = __ldg(reinterpret_cast<const float4 *>(p + c)), b = __ldg(reinterpret_cast<const float4 *>(p + c) + 1);
        w[0] = make_float2(a.x, a.y), w[1] = make_float2(a.z, a.w);
        w[2] = make_float2(b.x, b.y), w[3] = make_float2(b.z, b.w);
    } else {
        float v[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = __ldg(p + min(column<false>(k, i, t, T), dim - 1));
#pragma unroll
        for (int i = 0; i < kV / 2; ++i) w[i] = make_float2(v[2 * i], v[2 * i + 1]);
    }
}

template <typename T, bool kVec>
__device__ __forceinline__ void store_cols(T *row, const float (&v)[kV], int k, int t, int T_, int dim) {
    if constexpr (kVec) {
        const int c = column<true>(k, 0, t, T_);
        if (c < dim) store_vec(row + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int c = column<false>(k, i, t, T_);
            if (c < dim) put(row, c, v[i]);
        }
    }
}

// Which of a thread's elements there are: all of a vector or none, or one by one.
template <bool kVec>
__device__ __forceinline__ float2 there(float2 v, int k, int i, int t, int T, int dim) {
    if constexpr (kVec) {
        if (column<true>(k, 0, t, T) >= dim) v = both(0.f);
    } else {
        if (column<false>(k, 2 * i, t, T) >= dim) v.x = 0.f;
        if (column<false>(k, 2 * i + 1, t, T) >= dim) v.y = 0.f;
    }
    return v;
}

// T threads a row, blockDim / T rows a block at a time; the next row is on
// its way while one is worked on.  8 rows of 768 bf16: 4.1 us, a launch and a
// chain of two sums; 16384 rows: 14.4 us (3.5 TB/s), the latency of a
// row's loads and sums.
template <typename Tin, typename Tout, int kNv, bool kVec>
__global__ void __launch_bounds__(512) norm_rows_fwd_kernel(const NormParams p, int T) {
    __shared__ float red[2][2][16][1];
    const int groups = blockDim.x / T, group = threadIdx.x / T, t = threadIdx.x - group * T, dim = (int)p.dim;
    const int64_t step = (int64_t)gridDim.x * groups;
    int64_t row = (int64_t)blockIdx.x * groups + group;
    if (row >= p.batch) return;  // a whole group, and with it its barrier
    float2 w[kNv][kV / 2], b[kNv][kV / 2];
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
        load_cols<kVec>(w[k], p.weight, k, t, T, dim, 1.f);
        load_cols<kVec>(b[k], p.bias, k, t, T, dim, 0.f);
    }
    Vec8<Tin> x[kNv], next[kNv];
    load_row<Tin, kNv, kVec>(next, static_cast<const Tin *>(p.x) + row * p.dim, t, T, dim);
    for (int buf = 0; row < p.batch; row += step, buf ^= 1) {
#pragma unroll
        for (int k = 0; k < kNv; ++k) x[k] = next[k];
        if (row + step < p.batch)
            load_row<Tin, kNv, kVec>(next, static_cast<const Tin *>(p.x) + (row + step) * p.dim, t, T, dim);
        float2 nm = both(0.f);
        if (!p.rms) {
            float2 s = both(0.f);
#pragma unroll
            for (int k = 0; k < kNv; ++k)
#pragma unroll
                for (int i = 0; i < kV / 2; ++i) s = add2(s, x[k].pair(i));
            float v[1] = {s.x + s.y};
            row_sum<1>(v, T, group, red[buf][0]);
            nm = both(-v[0] * p.inv_dim);
        }
        float2 q = both(0.f);
#pragma unroll
        for (int k = 0; k < kNv; ++k)
#pragma unroll
            for (int i = 0; i < kV / 2; ++i) {
                const float2 c = there<kVec>(add2(x[k].pair(i), nm), k, i, t, T, dim);
                q = fma2(c, c, q);
            }
        float v[1] = {q.x + q.y};
        row_sum<1>(v, T, group, red[buf][1]);
        const float rstd = rsqrtf(fmaf(v[0], p.inv_dim, p.eps));
        if (t == 0) {
            if (p.mean && !p.rms) p.mean[row] = -nm.x;
            if (p.rstd) p.rstd[row] = rstd;
        }
        Tout *y = static_cast<Tout *>(p.y) + row * p.dim;
#pragma unroll
        for (int k = 0; k < kNv; ++k) {
            float o[kV];
#pragma unroll
            for (int i = 0; i < kV / 2; ++i) {
                const float2 r = fma2(mul2(add2(x[k].pair(i), nm), both(rstd)), w[k][i], b[k][i]);
                o[2 * i] = r.x, o[2 * i + 1] = r.y;
            }
            store_cols<Tout, kVec>(y, o, k, t, T, dim);
        }
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
    row_sum<1>(s, blockDim.x, 0, red[0]);
    const float mean = s[0] * p.inv_dim;
    for (int64_t c = threadIdx.x; c < p.dim; c += blockDim.x) {
        const float v = load_elem(x, c) - mean;
        q[0] = fmaf(v, v, q[0]);
    }
    row_sum<1>(q, blockDim.x, 0, red[1]);
    const float rstd = rsqrtf(fmaf(q[0], p.inv_dim, p.eps));
    if (threadIdx.x == 0) {
        if (p.mean && !p.rms) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    Tout *y = static_cast<Tout *>(p.y) + row * p.dim;
    for (int64_t c = threadIdx.x; c < p.dim; c += blockDim.x)
        put(y, c, fmaf((load_elem(x, c) - mean) * rstd, p.weight ? __ldg(p.weight + c) : 1.f, p.bias ? __ldg(p.bias + c) : 0.f));
}

// Blocks stay and walk over the rows.  A thread's columns are the same in
// every row, so their parts of dw and db are sums in its registers, joined
// over the block's groups at the end.  16384 rows of 768 bf16: 25 us with
// the second kernel's 5 or so, against 11.6 for the bytes: 16 warps an SM (128
// registers) do not cover the loads, and their sums issue 47 % of the time.
template <typename Tin, typename Tout, int kNv, bool kVec>
__global__ void __launch_bounds__(512) norm_rows_bwd_kernel(const NormParams p, int T) {
    extern __shared__ float acc[];  // groups x 2 x dim
    __shared__ float red[2][16][2];
    const int groups = blockDim.x / T, group = threadIdx.x / T, t = threadIdx.x - group * T, dim = (int)p.dim;
    const int64_t step = (int64_t)gridDim.x * groups;
    float2 dw[kNv][kV / 2], db[kNv][kV / 2], w[kNv][kV / 2];
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
        load_cols<kVec>(w[k], p.weight, k, t, T, dim, 1.f);
#pragma unroll
        for (int i = 0; i < kV / 2; ++i) dw[k][i] = db[k][i] = both(0.f);
    }
    int buf = 0;
    int64_t row = (int64_t)blockIdx.x * groups + group;
    // The next row is on its way while one is worked on, where the registers
    // hold both (8192 rows of 4096 bf16: 64 us against 76 without).
    constexpr bool kAhead = kNv <= (kVec ? 2 : 1);
    Vec8<Tin> x[kNv], nx[kNv];
    Vec8<Tout> dy[kNv], ny[kNv];
    if (kAhead && row < p.batch) {
        load_row<Tin, kNv, kVec>(nx, static_cast<const Tin *>(p.x) + row * p.dim, t, T, dim);
        load_row<Tout, kNv, kVec>(ny, static_cast<const Tout *>(p.dy) + row * p.dim, t, T, dim);
    }
    for (; row < p.batch; row += step, buf ^= 1) {
        if constexpr (kAhead) {
#pragma unroll
            for (int k = 0; k < kNv; ++k) x[k] = nx[k], dy[k] = ny[k];
            if (row + step < p.batch) {
                load_row<Tin, kNv, kVec>(nx, static_cast<const Tin *>(p.x) + (row + step) * p.dim, t, T, dim);
                load_row<Tout, kNv, kVec>(ny, static_cast<const Tout *>(p.dy) + (row + step) * p.dim, t, T, dim);
            }
        } else {
            load_row<Tin, kNv, kVec>(x, static_cast<const Tin *>(p.x) + row * p.dim, t, T, dim);
            load_row<Tout, kNv, kVec>(dy, static_cast<const Tout *>(p.dy) + row * p.dim, t, T, dim);
        }
        const float2 nm = both(p.mean_in ? -__ldg(p.mean_in + row) : 0.f);
        const float rstd = __ldg(p.rstd_in + row);
        // elements that are not there have dy = 0, and count in no sum
        float2 c1 = both(0.f), c2 = both(0.f);
#pragma unroll
        for (int k = 0; k < kNv; ++k)
#pragma unroll
            for (int i = 0; i < kV / 2; ++i) {
                const float2 g = dy[k].pair(i), h = mul2(g, mul2(add2(x[k].pair(i), nm), both(rstd)));
                c1 = fma2(g, w[k][i], c1);
                c2 = fma2(h, w[k][i], c2);
                dw[k][i] = add2(dw[k][i], h);
                db[k][i] = add2(db[k][i], g);
            }
        float c[2] = {c1.x + c1.y, c2.x + c2.y};
        row_sum<2>(c, T, group, red[buf]);
#pragma unroll
        for (int k = 0; k < kNv; ++k) x[k].again(), dy[k].again();
        // dx = rstd v - rstd c1 - (x - m) rstd^2 c2
        const float f = -rstd * p.inv_dim;
        const float2 a1 = both(p.mean_in ? c[0] * f : 0.f), a2 = both(c[1] * f * rstd);
        Tin *dx = static_cast<Tin *>(p.dx) + row * p.dim;
#pragma unroll
        for (int k = 0; k < kNv; ++k) {
            float o[kV];
#pragma unroll
            for (int i = 0; i < kV / 2; ++i) {
                const float2 r = fma2(add2(x[k].pair(i), nm), a2, fma2(mul2(dy[k].pair(i), w[k][i]), both(rstd), a1));
                o[2 * i] = r.x, o[2 * i + 1] = r.y;
            }
            store_cols<Tin, kVec>(dx, o, k, t, T, dim);
        }
    }
    if (!p.sums) return;
    float *out = p.part + (int64_t)blockIdx.x * 2 * p.dim;
    float *to = groups > 1 ? acc + group * 2 * dim : out;
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
        float o[kV], u[kV];
#pragma unroll
        for (int i = 0; i < kV / 2; ++i) {
            o[2 * i] = dw[k][i].x, o[2 * i + 1] = dw[k][i].y;
            u[2 * i] = db[k][i].x, u[2 * i + 1] = db[k][i].y;
        }
        store_cols<float, kVec>(to, o, k, t, T, dim);
        store_cols<float, kVec>(to + dim, u, k, t, T, dim);
    }
    if (groups > 1) {
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * dim; c += blockDim.x) {
            float v = 0.f;
            for (int g = 0; g < groups; ++g) v += acc[g * 2 * dim + c];
            out[c] = v;
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
        row_sum<2>(c, blockDim.x, 0, red[buf]);
        const float c1 = p.mean_in ? c[0] * p.inv_dim : 0.f, c2 = c[1] * p.inv_dim;
        for (int64_t d = threadIdx.x; d < p.dim; d += blockDim.x) {
            const float w = p.weight ? __ldg(p.weight + d) : 1.f, xh = (load_elem(x, d) - mean) * rstd;
            put(dx, d, (fmaf(load_elem(dy, d), w, -c1) - xh * c2) * rstd);
        }
    }
}

// ------------------------------------------------------------------ steps

constexpr int kWarpCh = 32;  // channels of a warp

// v into the same place of block `rank`'s shared memory.
__device__ __forceinline__ void peer_store(float2 *p, int rank, float2 v) {
    uint32_t peer;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(peer), "f"(v.x), "f"(v.y) : "memory");
}

// How a warp covers its 32 channels: kLs lanes along the steps, V steps each
// (16 bytes of the input), and kLc lanes by kN channels.  V = 1 where rows
// are not whole vectors: then every lane has a step and all 32 channels.
// A thread's elements are worked in pairs, with the packed arithmetic of two
// floats: neighbouring steps of a channel, or with V = 1 neighbouring
// channels.  Pair q belongs to channel chan(q) (and the next one with V = 1)
// and to the statistics stat(q).
template <int V>
struct Tile {
    static constexpr int kLc = V == 1 ? 1 : 4, kLs = 32 / kLc, kN = kWarpCh / kLc, kSteps = kLs * V;
    static constexpr int kPairs = kN * V / 2, kStats = V == 1 ? 1 : V / 2;
    __device__ static constexpr int chan(int q) { return V == 1 ? 2 * q : q / kStats; }
    __device__ static constexpr int stat(int q) { return V == 1 ? 0 : q % kStats; }
};

// A thread's elements as they lie in memory.
template <typename T, int V>
struct Patch {
    using G = Tile<V>;
    static constexpr int kWords = G::kPairs * sizeof(T) / 2;
    uint32_t w[kWords];
    __device__ __forceinline__ float2 pair(int q) const { return pair_of<T>(w, q); }
    // Channels 0 .. kN-1, `apart` elements from one to the next; those from
    // `have` on are read from the last one there is, and cleared.
    __device__ __forceinline__ void load(const T *p, int64_t apart, int have) {
        if constexpr (V == 1) {
            uint32_t b[G::kN];
            if (have == G::kN) {
#pragma unroll
                for (int i = 0; i < G::kN; ++i, p += apart) b[i] = Io<T>::bits(p, 0);
            } else {
#pragma unroll
                for (int i = 0; i < G::kN; ++i) b[i] = Io<T>::bits(p + min(i, max(have - 1, 0)) * apart, 0);
            }
#pragma unroll
            for (int i = 0; i < G::kN; ++i) {
                if constexpr (sizeof(T) == 4) w[i] = b[i];
                else if (i % 2) w[i / 2] = __byte_perm(b[i - 1], b[i], 0x5410);
            }
        } else {
            constexpr int kQ = V * sizeof(T) / 16;
#pragma unroll
            for (int i = 0; i < G::kN; ++i) {
                const uint4 *q = reinterpret_cast<const uint4 *>(p + min(i, max(have - 1, 0)) * apart);
#pragma unroll
                for (int k = 0; k < kQ; ++k) {
                    const uint4 u = __ldg(q + k);
                    uint32_t *v = w + (i * kQ + k) * 4;
                    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
                }
            }
        }
    }
    __device__ __forceinline__ void keep(int have) {  // clears the channels from `have` on
        if (have >= G::kN) return;
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            if (V == 1 && sizeof(T) == 2) w[k] &= 2 * k + 1 < have ? ~0u : 2 * k < have ? 0xffffu : 0u;
            else if (k * G::kN / kWords >= have) w[k] = 0u;
        }
    }
    __device__ __forceinline__ void again() {  // as Vec8::again
#pragma unroll
        for (int k = 0; k < kWords; ++k) asm volatile("" : "+r"(w[k]));
    }
};

// The pairs of channel i (with V = 1: i and i + 1) to p.
template <int V>
__device__ __forceinline__ void store_pairs(float *p, int64_t apart, const float2 *v, bool second) {
    if constexpr (V == 1) {
        p[0] = v[0].x;
        if (second) p[apart] = v[0].y;
    } else {
#pragma unroll
        for (int k = 0; k < V / 4; ++k)
            reinterpret_cast<float4 *>(p)[k] = make_float4(v[2 * k].x, v[2 * k].y, v[2 * k + 1].x, v[2 * k + 1].y);
    }
}
template <int V>
__device__ __forceinline__ void store_pairs(__nv_bfloat16 *p, int64_t apart, const float2 *v, bool second) {
    if constexpr (V == 1) {
        p[0] = __float2bfloat16_rn(v[0].x);
        if (second) p[apart] = __float2bfloat16_rn(v[0].y);
    } else {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                                   pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
    }
}

// A per-channel parameter for the pairs of channel c0 + i kLc (null: `none`).
template <int V>
__device__ __forceinline__ float2 param(const float *p, int64_t c, bool second, float none) {
    if (!p) return both(none);
    const float v = __ldg(p + c);
    return V == 1 ? make_float2(v, __ldg(p + c + (second ? 1 : 0))) : both(v);
}

// Where a lane's steps lie: element of channel 0, index among all steps (the
// last ones again for a lane behind the end).
struct Place {
    int64_t at, index;
    bool in;
};
template <int V>
__device__ __forceinline__ Place place_of(const NormParams &p, int64_t tile, int sl) {
    const int64_t s = tile * Tile<V>::kSteps + sl * V, n = p.batch * p.L;
    Place r;
    r.in = s < n;
    r.index = r.in ? s : n - V;
    const int64_t b = n <= INT_MAX ? (int64_t)((uint32_t)r.index / (uint32_t)p.L) : r.index / p.L;
    r.at = b * p.dim * p.L + (r.index - b * p.L);
    return r;
}

__device__ __forceinline__ float clamp_count(int64_t n, int64_t most) { return n <= 0 ? 0.f : (float)(n < most ? n : most); }

// Channels of a thread that there are, of c0, c0 + kLc, ...
template <int V>
__device__ __forceinline__ int have_of(const NormParams &p, int64_t c0) {
    using G = Tile<V>;
    return c0 >= p.dim ? 0 : (int)min((int64_t)G::kN, (p.dim - c0 + G::kLc - 1) / G::kLc);
}

// Makes a value opaque: what depends on it is computed anew from here, rather
// than kept in registers.
__device__ __forceinline__ void again(int64_t &v) { asm volatile("" : "+l"(v)); }

// Sums over the kLc lanes that share a step, and over a pair with V = 1.
template <int V>
__device__ __forceinline__ void lanes_sum(float2 (&v)[Tile<V>::kStats]) {
    if constexpr (V == 1) {
        v[0] = both(v[0].x + v[0].y);
    } else {
#pragma unroll
        for (int o = Tile<V>::kLs; o < 32; o *= 2)
#pragma unroll
            for (int k = 0; k < Tile<V>::kStats; ++k)
                v[k] = add2(v[k], make_float2(__shfl_xor_sync(0xffffffffu, v[k].x, o), __shfl_xor_sync(0xffffffffu, v[k].y, o)));
    }
}

// Means and squares about them of parts of n(k) channels each into those of
// all:  m = sum n m_k / sum n,  S = sum S_k + n (m_k - m)^2.
template <typename N>
__device__ __forceinline__ float2 join(const float2 *part, int stride, int parts, N n) {
    float all = 0.f, m = 0.f, S = 0.f;
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
        m = fmaf(n(k), part[k * stride].x, m);
        all += n(k);
    }
    m = all > 0.f ? m / all : 0.f;
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
        const float2 v = part[k * stride];
        const float d = v.x - m;
        S += fmaf(n(k) * d, d, v.y);
    }
    return make_float2(m, S);
}

// Forward over steps.  The statistics of a step come together in three
// stages, always as mean and squares about it (no difference of large sums):
// a warp's channels, the block's warps, the cluster's blocks; each block
// writes its own into every other's shared memory, so one cluster barrier is
// all they wait for.  Single steps (fp32 3 x 1000 x 4099): 35 us,
// 15 for the bytes, the instructions of four-byte accesses and the barriers
// (issue 53 %); in vectors 36 us for 8 x 1536 x 2048 bf16, where the tiles
// below take 30.
template <typename Tin, typename Tout, int V, int kMaxW>
__global__ void __launch_bounds__(32 * kMaxW, kMaxW <= 8 ? 3 : 1) norm_steps_fwd_kernel(const NormParams p, int nblk) {
    using G = Tile<V>;
    __shared__ float2 part[kMaxW][G::kSteps], slot[8][G::kSteps];
    __shared__ __align__(16) float stat[2][G::kSteps];  // -mean, 1 / deviation
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int rank = (int)(blockIdx.x % nblk), sl = lane % G::kLs, cl = lane / G::kLs;
    if (nblk > 1) cluster_arrive();  // waited for before the first remote store
    const int64_t w0 = ((int64_t)rank * warps + warp) * kWarpCh, c0 = w0 + cl;  // channels c0 + i kLc
    const Place at = place_of<V>(p, blockIdx.x / nblk, sl);
    const int have = have_of<V>(p, c0);
    const int64_t first = at.at + min(c0, p.dim - 1) * p.L;
    int64_t apart = G::kLc * p.L;
    Patch<Tin, V> x;
    x.load(static_cast<const Tin *>(p.x) + first, apart, have);
    x.keep(have);

    float2 nm[G::kStats], S[G::kStats];
#pragma unroll
    for (int k = 0; k < G::kStats; ++k) nm[k] = S[k] = both(0.f);
    const float nw = clamp_count(p.dim - w0, kWarpCh);
    if (!p.rms && nw > 0.f) {
#pragma unroll
        for (int q = 0; q < G::kPairs; ++q) nm[G::stat(q)] = add2(nm[G::stat(q)], x.pair(q));
        lanes_sum<V>(nm);
        const float2 f = both(-1.f / nw);
#pragma unroll
        for (int k = 0; k < G::kStats; ++k) nm[k] = mul2(nm[k], f);
    }
    if (nw == kWarpCh) {
#pragma unroll
        for (int q = 0; q < G::kPairs; ++q) {
            const float2 d = add2(x.pair(q), nm[G::stat(q)]);
            S[G::stat(q)] = fma2(d, d, S[G::stat(q)]);
        }
    } else {
#pragma unroll
        for (int q = 0; q < G::kPairs; ++q) {
            float2 d = add2(x.pair(q), nm[G::stat(q)]);
            if (G::chan(q) >= have) d = both(0.f);
            if (V == 1 && G::chan(q) + 1 >= have) d.y = 0.f;
            S[G::stat(q)] = fma2(d, d, S[G::stat(q)]);
        }
    }
    lanes_sum<V>(S);
    if (cl == 0) {
        if constexpr (V == 1) {
            part[warp][sl] = make_float2(-nm[0].x, S[0].x);
        } else {
#pragma unroll
            for (int k = 0; k < G::kStats; ++k) {
                part[warp][sl * V + 2 * k] = make_float2(-nm[k].x, S[k].x);
                part[warp][sl * V + 2 * k + 1] = make_float2(-nm[k].y, S[k].y);
            }
        }
    }
    __syncthreads();
    const int t = threadIdx.x;
    const int64_t wide = (int64_t)warps * kWarpCh;
    float2 all = make_float2(0.f, 0.f);
    if (t < G::kSteps)
        all = join(&part[0][t], G::kSteps, warps,
                          [&](int k) { return clamp_count(p.dim - (rank * wide + k * kWarpCh), kWarpCh); });
    if (nblk > 1) {
        cluster_wait();  // every block has begun
        if (t < G::kSteps)
            for (int k = 0; k < nblk; ++k) peer_store(&slot[rank][t], k, all);
        cluster_arrive();
        cluster_wait();
        if (t < G::kSteps)
            all = join(&slot[0][t], G::kSteps, nblk, [&](int k) { return clamp_count(p.dim - k * wide, wide); });
    }
    if (t < G::kSteps) {
        const float rstd = rsqrtf(fmaf(all.y, p.inv_dim, p.eps));
        stat[0][t] = -all.x, stat[1][t] = rstd;
        const int64_t s = (blockIdx.x / nblk) * (int64_t)G::kSteps + t;
        if (rank == 0 && s < p.batch * p.L) {
            if (p.mean && !p.rms) p.mean[s] = all.x;
            if (p.rstd) p.rstd[s] = rstd;
        }
    }
    __syncthreads();
    if (!at.in) return;
    x.again(), again(apart);
#pragma unroll
    for (int k = 0; k < G::kStats; ++k) {
        if constexpr (V == 1) {
            nm[0] = both(stat[0][sl]), S[0] = both(stat[1][sl]);
        } else {
            nm[k] = *reinterpret_cast<const float2 *>(&stat[0][sl * V + 2 * k]);
            S[k] = *reinterpret_cast<const float2 *>(&stat[1][sl * V + 2 * k]);
        }
    }
    Tout *y = static_cast<Tout *>(p.y) + first;
    constexpr int kRun = V == 1 ? 1 : V / 2;  // pairs stored together
#pragma unroll
    for (int q = 0; q < G::kPairs; q += kRun) {
        const int i = G::chan(q);
        if (i < have) {
            const bool second = V == 1 && i + 1 < have;
            const float2 w = param<V>(p.weight, c0 + i * G::kLc, second, 1.f), b = param<V>(p.bias, c0 + i * G::kLc, second, 0.f);
            float2 v[kRun];
#pragma unroll
            for (int k = 0; k < kRun; ++k) v[k] = fma2(mul2(add2(x.pair(q + k), nm[k]), S[k]), w, b);
            store_pairs<V>(y + i * apart, apart, v, second);
        }
    }
}

// Sums over kN neighbouring lanes of kN values each, value i to lane i of them:
// each round halves the values a lane still holds.
template <int kN>
__device__ __forceinline__ float lane_sums(float (&v)[kN], int lane) {
#pragma unroll
    for (int o = kN / 2; o >= 1; o /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int k = 0; k < o; ++k) {
            const float send = up ? v[k] : v[k + o], keep = up ? v[k + o] : v[k];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return v[0];
}

// Backward over steps: clusters stay and walk over the tiles.  3 x 1000 x 4099
// fp32: 55 us with the second kernel's 5 or so, against 22.5 for the bytes:
// 16 warps an SM and a cluster barrier for each 32 steps (issue 45 %).  8 x
// 1536 x 2047 bf16: 80 us (95 where full warps too ask which channels there are).
// bf16 x with fp32 dy: 82 us there; in vectors, where a lane's registers spill,
// 95 us for 8 x 1536 x 2048.
template <typename Tin, typename Tout, int V, int kMaxW>
__global__ void __launch_bounds__(32 * kMaxW, kMaxW <= 8 ? 2 : 1) norm_steps_bwd_kernel(const NormParams p, int nblk) {
    using G = Tile<V>;
    static_assert(G::kN == G::kLs, "one channel's sum for each step lane");
    __shared__ float2 part[kMaxW][G::kSteps], slot[2][8][G::kSteps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int rank = (int)(blockIdx.x % nblk), sl = lane % G::kLs, cl = lane / G::kLs;
    const int64_t group = blockIdx.x / nblk, groups = gridDim.x / nblk;
    const int64_t c0 = ((int64_t)rank * warps + warp) * kWarpCh + cl;
    const int have = have_of<V>(p, c0);
    const int64_t tiles = (p.batch * p.L + G::kSteps - 1) / G::kSteps;
    constexpr int kRun = V == 1 ? 1 : V / 2;
    if (nblk > 1) cluster_arrive();
    bool begun = nblk == 1;
    float dw = 0.f, db = 0.f;  // of channel c0 + sl kLc
    int buf = 0;
    for (int64_t tile = group; tile < tiles; tile += groups, buf ^= 1) {
        const Place at = place_of<V>(p, tile, sl);
        const int64_t first = at.at + min(c0, p.dim - 1) * p.L;
        int64_t apart = G::kLc * p.L, wc = c0;
        again(apart), again(wc);  // nothing of them is kept from tile to tile
        Patch<Tin, V> x;
        Patch<Tout, V> g;
        x.load(static_cast<const Tin *>(p.x) + first, apart, have);
        g.load(static_cast<const Tout *>(p.dy) + first, apart, have);
        float2 nm[G::kStats], r[G::kStats], s1[G::kStats], s2[G::kStats];
#pragma unroll
        for (int k = 0; k < G::kStats; ++k) {
            const int64_t s = at.index + 2 * k;
            constexpr int kNext = V == 1 ? 0 : 1;
            nm[k] = p.mean_in ? make_float2(-__ldg(p.mean_in + s), -__ldg(p.mean_in + s + kNext)) : both(0.f);
            r[k] = make_float2(__ldg(p.rstd_in + s), __ldg(p.rstd_in + s + kNext));
            s1[k] = s2[k] = both(0.f);
        }
        x.keep(have);
        g.keep(at.in ? have : 0);
        float term[G::kN];
        // (all: every channel of the thread is there)
        const auto to_sums = [&](auto all) {
#pragma unroll
            for (int q = 0; q < G::kPairs; q += kRun) {
                const int i = G::chan(q);
                const bool second = V == 1 && (all.value || i + 1 < have);
                const float2 w = param<V>(p.weight, all.value || i < have ? wc + i * G::kLc : min(c0, p.dim - 1), second, 1.f);
                float2 sum = both(0.f);
#pragma unroll
                for (int k = 0; k < kRun; ++k) {
                    const float2 gv = g.pair(q + k), t = mul2(gv, mul2(add2(x.pair(q + k), nm[k]), r[k]));
                    s1[k] = fma2(gv, w, s1[k]);
                    s2[k] = fma2(t, w, s2[k]);
                    sum = add2(sum, t);
                }
                if constexpr (V == 1) term[i] = sum.x, term[i + 1] = sum.y;
                else term[i] = sum.x + sum.y;
            }
        };
        if (have == G::kN) to_sums(std::true_type{});
        else to_sums(std::false_type{});
        if (p.sums) dw += lane_sums<G::kN>(term, lane);
        lanes_sum<V>(s1), lanes_sum<V>(s2);
        if (cl == 0) {
            if constexpr (V == 1) {
                part[warp][sl] = make_float2(s1[0].x, s2[0].x);
            } else {
#pragma unroll
                for (int k = 0; k < G::kStats; ++k) {
                    part[warp][sl * V + 2 * k] = make_float2(s1[k].x, s2[k].x);
                    part[warp][sl * V + 2 * k + 1] = make_float2(s1[k].y, s2[k].y);
                }
            }
        }
        __syncthreads();
        const int t = threadIdx.x;
        float2 all = make_float2(0.f, 0.f);
        if (t < G::kSteps)
            for (int k = 0; k < warps; ++k) all = add2(all, part[k][t]);
        if (nblk > 1) {
            if (!begun) cluster_wait();  // every block has begun
            begun = true;
            if (t < G::kSteps)
                for (int k = 0; k < nblk; ++k) peer_store(&slot[buf][rank][t], k, all);
            // One barrier a tile: a block that is ahead writes the other
            // half of `slot`, and cannot come back to this one before all
            // have read it and arrived at the next tile's barrier.
            cluster_arrive();
            cluster_wait();
        } else {
            if (t < G::kSteps) slot[buf][0][t] = all;
            __syncthreads();
        }
        x.again(), g.again(), again(apart), again(wc);
        // dx = rstd v - rstd c1 - (x - m) rstd^2 c2, with the step's factors
        // made once; s1, s2: -rstd c1, -rstd^2 c2
#pragma unroll
        for (int k = 0; k < G::kStats; ++k) {
            float2 c = both(0.f), d = both(0.f);  // the sums of both steps of the pair
            for (int b = 0; b < nblk; ++b) {
                c = add2(c, slot[buf][b][V == 1 ? sl : sl * V + 2 * k]);
                if (V > 1) d = add2(d, slot[buf][b][sl * V + 2 * k + (V > 1)]);
            }
            if (V == 1) d = c;
            const float2 f = mul2(r[k], both(-p.inv_dim));
            s1[k] = p.mean_in ? mul2(make_float2(c.x, d.x), f) : both(0.f);
            s2[k] = mul2(mul2(make_float2(c.y, d.y), f), r[k]);
        }
        Tin *dx = static_cast<Tin *>(p.dx) + first;
        const auto to_dx = [&](auto all) {
            Tin *to = dx;
#pragma unroll
            for (int q = 0; q < G::kPairs; q += kRun) {
                const int i = G::chan(q);
                const bool second = V == 1 && (all.value || i + 1 < have);
                const float2 w = param<V>(p.weight, all.value || i < have ? wc + i * G::kLc : min(c0, p.dim - 1), second, 1.f);
                float2 v[kRun], sum = both(0.f);
#pragma unroll
                for (int k = 0; k < kRun; ++k) {
                    const float2 gv = g.pair(q + k);
                    sum = add2(sum, gv);
                    v[k] = fma2(add2(x.pair(q + k), nm[k]), s2[k], fma2(mul2(gv, w), r[k], s1[k]));
                }
                if ((all.value || i < have) && at.in) store_pairs<V>(to, apart, v, second);
                to += (V == 1 ? 2 : (q + kRun) % G::kStats ? 0 : 1) * apart;
                if constexpr (V == 1) term[i] = sum.x, term[i + 1] = sum.y;
                else term[i] = sum.x + sum.y;
            }
        };
        if (have == G::kN) to_dx(std::true_type{});
        else to_dx(std::false_type{});
        if (p.sums) db += lane_sums<G::kN>(term, lane);
    }
    if (p.sums && sl < have) {
        float *out = p.part + group * 2 * p.dim;
        out[c0 + sl * G::kLc] = dw;
        out[p.dim + c0 + sl * G::kLc] = db;
    }
}

// ---------------------------------------------------------- steps in pairs
//
// The forward of bf16 rows that are not whole vectors, in words of two steps: a
// lane takes a word of each of its warp's channels.  With an odd L the rows of
// every other channel start in the middle of a word, so their words lie one
// step earlier: those of channels c0, c0 + 2, ... cover steps 2i - sh[0] and
// the next one, those of the others 2i - sh[1] (each 0 or 1).  Sums over
// channels are kept for the two kinds apart and brought to steps 2i, 2i + 1 by
// one shuffle at the end.  32 words so cover 63 steps of both kinds; tiles do
// not cross batch entries, where a word's two steps are not neighbours.
// (8 x 1536 x 2047: 53 us, 64 in single steps; fp32 3 x 1000 x 4099 took 41
// against 35, and the backward, whose words fill the registers, 98 against 80:
// those stay with single steps.)
constexpr int kPairSteps = 63, kPairWarps = 8;
using Half = __nv_bfloat16;

// Where a warp's words lie.
struct PairTile {
    int64_t e0, index;  // element of channel c0 at the tile's first step; that step among all
    int n, sh[2];       // steps of the tile, shifts of the two kinds of channels
    bool last;          // the tensor's last step is in the tile
    // Whether the steps of this lane's words of kind k are the tile's.
    __device__ __forceinline__ bool x(int k, int lane) const { return 2 * lane >= sh[k] && 2 * lane - sh[k] < n; }
    __device__ __forceinline__ bool y(int k, int lane) const { return 2 * lane - sh[k] + 1 < n; }
    __device__ __forceinline__ int step(int k, int lane, int i) const { return min(max(2 * lane - sh[k] + i, 0), n - 1); }
    // The lane's word of channel c0 + i, or the row's last one for a lane behind it.
    __device__ __forceinline__ int64_t word(int i, int lane, int64_t L) const {
        const int s = sh[i & 1];
        return e0 + i * L - s + 2 * min(lane, (n - 1 + s) >> 1);
    }
};
__device__ __forceinline__ PairTile pair_tile(const NormParams &p, uint32_t tile, int64_t c0) {
    const uint32_t per = (uint32_t)((p.L + kPairSteps - 1) / kPairSteps), b = tile / per;
    const int64_t s0 = (int64_t)(tile - b * per) * kPairSteps;
    PairTile t;
    t.e0 = ((int64_t)b * p.dim + c0) * p.L + s0;
    t.index = b * p.L + s0;
    t.n = (int)min((int64_t)kPairSteps, p.L - s0);
    t.sh[0] = (int)(t.e0 & 1), t.sh[1] = (int)((t.e0 + p.L) & 1);
    t.last = t.index + t.n == p.batch * p.L;
    return t;
}

// The words of a warp's channels; zero where there is none.
__device__ __forceinline__ void load_words(uint32_t (&r)[kWarpCh], const Half *p, const PairTile &t, int lane, int have,
                                           const NormParams &q) {
    if (have == kWarpCh && !t.last) {
        const Half *a = p + t.word(0, lane, q.L), *b = p + t.word(1, lane, q.L);
#pragma unroll
        for (int i = 0; i < kWarpCh; ++i) r[i] = __ldg(reinterpret_cast<const uint32_t *>((i % 2 ? b : a) + (i / 2) * 2 * q.L));
        return;
    }
    const int64_t n = q.batch * q.dim * q.L;
#pragma unroll
    for (int i = 0; i < kWarpCh; ++i) {
        r[i] = 0u;
        if (i < have) {
            const int64_t e = t.word(i, lane, q.L);
            if (e + 1 < n) r[i] = __ldg(reinterpret_cast<const uint32_t *>(p + e));
            else r[i] = Io<Half>::bits(p, e);  // the tensor's last element has no next one
        }
    }
}

// Values of the words' steps 2 lane - sh, and one on, to those of steps
// 2 lane, 2 lane + 1, and back (the last and the first are not the tile's).
__device__ __forceinline__ float2 to_steps(float2 v, int sh) {
    const float next = __shfl_down_sync(0xffffffffu, v.x, 1);
    return sh ? make_float2(v.y, next) : v;
}
__device__ __forceinline__ float2 to_words(float2 v, int sh) {
    const float before = __shfl_up_sync(0xffffffffu, v.y, 1);
    return sh ? make_float2(before, v.x) : v;
}

__device__ __forceinline__ void put_word(float *p, float2 v, bool x, bool y) {
    if (x && y) *reinterpret_cast<float2 *>(p) = v;
    else if (x || y) put(p, y ? 1 : 0, y ? v.y : v.x);
}
__device__ __forceinline__ void put_word(Half *p, float2 v, bool x, bool y) {
    if (x && y) *reinterpret_cast<uint32_t *>(p) = pack_bf16x2(v.x, v.y);
    else if (x || y) put(p, y ? 1 : 0, y ? v.y : v.x);
}

// Forward, as norm_steps_fwd_kernel.  No step of a word is the other's
// business, so nothing is masked before the results.
template <typename Tout>
__global__ void __launch_bounds__(32 * kPairWarps, 3) norm_pairs_fwd_kernel(const NormParams p, int nblk) {
    constexpr int kN = kWarpCh;
    __shared__ float2 part[kPairWarps][64], slot[8][64];
    __shared__ float stat[2][64];  // -mean, 1 / deviation
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, rank = (int)(blockIdx.x % nblk);
    if (nblk > 1) cluster_arrive();  // waited for before the first remote store
    const int64_t wide = (int64_t)warps * kN, c0 = rank * wide + warp * kN;
    const int have = (int)clamp_count(p.dim - c0, kN);
    const PairTile at = pair_tile(p, blockIdx.x / nblk, c0);
    uint32_t x[kN];
    load_words(x, static_cast<const Half *>(p.x), at, lane, have, p);
    const float2 none[2] = {both(0.f), both(0.f)};
    float2 nm[2] = {none[0], none[1]}, S[2] = {none[0], none[1]};
    float2 mean = both(0.f);
    if (!p.rms && have > 0) {
        float2 A[2] = {none[0], none[1]};
#pragma unroll
        for (int i = 0; i < kN; ++i) A[i & 1] = add2(A[i & 1], pair_of<Half>(x, i));
        mean = mul2(add2(to_steps(A[0], at.sh[0]), to_steps(A[1], at.sh[1])), both(1.f / (float)have));
        nm[0] = mul2(to_words(mean, at.sh[0]), both(-1.f)), nm[1] = mul2(to_words(mean, at.sh[1]), both(-1.f));
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        float2 d = add2(pair_of<Half>(x, i), nm[i & 1]);
        if (i >= have) d = both(0.f);
        S[i & 1] = fma2(d, d, S[i & 1]);
    }
    S[0] = add2(to_steps(S[0], at.sh[0]), to_steps(S[1], at.sh[1]));
    part[warp][2 * lane] = make_float2(mean.x, S[0].x);
    part[warp][2 * lane + 1] = make_float2(mean.y, S[0].y);
    __syncthreads();
    const int t = threadIdx.x;
    float2 all = both(0.f);
    if (t < 64) all = join(&part[0][t], 64, warps, [&](int k) { return clamp_count(p.dim - (rank * wide + k * kN), kN); });
    if (nblk > 1) {
        cluster_wait();  // every block has begun
        if (t < 64)
            for (int k = 0; k < nblk; ++k) peer_store(&slot[rank][t], k, all);
        cluster_arrive();
        cluster_wait();
        if (t < 64) all = join(&slot[0][t], 64, nblk, [&](int k) { return clamp_count(p.dim - k * wide, wide); });
    }
    if (t < 64) {
        const float rstd = rsqrtf(fmaf(all.y, p.inv_dim, p.eps));
        stat[0][t] = -all.x, stat[1][t] = rstd;
        if (rank == 0 && t < at.n) {
            if (p.mean && !p.rms) p.mean[at.index + t] = all.x;
            if (p.rstd) p.rstd[at.index + t] = rstd;
        }
    }
    __syncthreads();
    bool in_x[2], in_y[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int a = at.step(k, lane, 0), b = at.step(k, lane, 1);
        nm[k] = make_float2(stat[0][a], stat[0][b]), S[k] = make_float2(stat[1][a], stat[1][b]);
        in_x[k] = at.x(k, lane), in_y[k] = at.y(k, lane);
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) asm volatile("" : "+r"(x[i]));
    Tout *y = static_cast<Tout *>(p.y);
    Tout *to[2] = {y + at.word(0, lane, p.L), y + at.word(1, lane, p.L)};
    int64_t apart = 2 * p.L;
    again(apart);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        if (i < have) {
            const float2 w = both(p.weight ? __ldg(p.weight + c0 + i) : 1.f), b = both(p.bias ? __ldg(p.bias + c0 + i) : 0.f);
            put_word(to[i & 1] + (i / 2) * apart, fma2(mul2(add2(pair_of<Half>(x, i), nm[i & 1]), S[i & 1]), w, b), in_x[i & 1], in_y[i & 1]);
        }
    }
}

// ---------------------------------------------------------- steps in shared memory
//
// Where rows are whole vectors and a tile of all channels fits into shared
// memory, no cluster is needed: a block takes 64 bytes of every channel (32
// steps of bf16, 16 of fp32), goes over them once for the statistics and once
// for the results.  Every thread copies in the very units of 16 bytes that it
// reads later, so the copies need no barrier, and as soon as it has read a
// unit for the last time it starts the copy of the same unit of the block's
// next tile: the loads of the next tile run under the results of this one.
//
// A warp covers 4 lanes along the steps by 8 channels; a batch is 4 of a
// thread's units, as many as there are lanes along the steps, so that the
// sums over the steps of a batch (backward) come out one unit to each lane.
template <typename T>
struct Geo {
    static constexpr int kE = 16 / (int)sizeof(T), kLs = 4, kLc = 8, kB = 4, kSteps = kLs * kE;
    static constexpr int kStats = kE / 2;  // pairs of a unit
};

template <typename T>
struct Batch {
    uint32_t w[4 * Geo<T>::kB];
    __device__ __forceinline__ float2 pair(int j, int k) const { return pair_of<T>(w + 4 * j, k); }
    __device__ __forceinline__ void read(const unsigned char *sm, int step) {  // units `step` bytes apart
#pragma unroll
        for (int j = 0; j < Geo<T>::kB; ++j) {
            const uint4 u = *reinterpret_cast<const uint4 *>(sm + j * step);
            w[4 * j] = u.x, w[4 * j + 1] = u.y, w[4 * j + 2] = u.z, w[4 * j + 3] = u.w;
        }
    }
};

// p + j distances of `apart` bytes (32 bits: one multiply-add an address).
template <typename T>
__device__ __forceinline__ T *at_unit(T *p, uint32_t apart, int j) {
    return reinterpret_cast<T *>(reinterpret_cast<uintptr_t>(p) + (uint64_t)apart * (uint32_t)j);
}

// Starts the copy of a batch of a tile, channels c, c + each, ... below dim
// (kFull: all of them are); a lane without a step gets zeros.
template <typename T, bool kFull>
__device__ __forceinline__ void copy_batch(unsigned char *sm, int step, const T *src, uint32_t apart, int c, int each, int dim,
                                           bool in) {
#pragma unroll
    for (int j = 0; j < Geo<T>::kB; ++j) {
        if (kFull || c + j * each < dim) {
            if (in) cp_async16(sm + j * step, at_unit(src, apart, j));
            else *reinterpret_cast<uint4 *>(sm + j * step) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
}

template <typename T>
__device__ __forceinline__ Place place_in(const NormParams &p, int64_t tile, int sl) {
    using G = Geo<T>;
    const int64_t s = tile * G::kSteps + sl * G::kE, n = p.batch * p.L;
    Place r;
    r.in = s < n;
    r.index = r.in ? s : n - G::kE;
    const int64_t b = n <= INT_MAX ? (int64_t)((uint32_t)r.index / (uint32_t)p.L) : r.index / p.L;
    r.at = b * p.dim * p.L + (r.index - b * p.L);
    return r;
}

template <int kN>
__device__ __forceinline__ void store_unit(float *p, const float2 (&v)[kN]) {
#pragma unroll
    for (int k = 0; k < kN / 2; ++k)
        reinterpret_cast<float4 *>(p)[k] = make_float4(v[2 * k].x, v[2 * k].y, v[2 * k + 1].x, v[2 * k + 1].y);
}
__device__ __forceinline__ void store_unit(__nv_bfloat16 *p, const float2 (&v)[4]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                               pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
}

// Sums over the 8 lanes of a warp that share a step.
template <int kN>
__device__ __forceinline__ void step_sums(float2 (&v)[kN]) {
#pragma unroll
    for (int o = 4; o < 32; o *= 2)
#pragma unroll
        for (int k = 0; k < kN; ++k)
            v[k] = add2(v[k], make_float2(__shfl_xor_sync(0xffffffffu, v[k].x, o), __shfl_xor_sync(0xffffffffu, v[k].y, o)));
}

// A warp's statistics of its steps to a row of `to`.
template <int kN>
__device__ __forceinline__ void write_steps(float2 *to, int sl, const float2 (&a)[kN], const float2 (&b)[kN]) {
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        to[(sl * kN + k) * 2] = make_float2(a[k].x, b[k].x);
        to[(sl * kN + k) * 2 + 1] = make_float2(a[k].y, b[k].y);
    }
}

template <int kN>
__device__ __forceinline__ void read_steps(const float *from, int sl, float2 (&v)[kN]) {
#pragma unroll
    for (int k = 0; k < kN; ++k) v[k] = reinterpret_cast<const float2 *>(from)[sl * kN + k];
}

constexpr int kTileWarps = 16;  // of a block, at most

// Calls f(batch, whole) for every batch; whole: every thread has all of its units.
template <typename F>
__device__ __forceinline__ void for_batches(int batches, int full, F f) {
    int b = 0;
    for (; b < full; ++b) f(b, std::true_type{});
    for (; b < batches; ++b) f(b, std::false_type{});
}

// batches: a thread's units, in batches.  Shared memory: batches * 4 * T units.
//
// Statistics in one pass: differences d to a pivot, the mean of the thread's
// first batch; then m = pivot + sum d / n and S = sum d^2 - (sum d)^2 / n.
// The pivot is a mean of n0 of the thread's own n values, so its square
// distance from their mean is at most S / n0: sum d^2 is at most
// (1 + n / n0) S, and nothing is lost in the difference, whatever the values.
//
// 8 x 1536 x 2048 bf16: 30 us (15.4 for the bytes).  Two blocks an SM have
// 512 tiles in 2 rounds where 1.73 would be even, and issue 52 % of the time.
template <typename Tin, typename Tout>
__global__ void __launch_bounds__(32 * kTileWarps, 2) norm_tile_fwd_kernel(const NormParams p, int batches) {
    using G = Geo<Tin>;
    extern __shared__ __align__(16) unsigned char units[];
    __shared__ float2 part[kTileWarps][G::kSteps];
    __shared__ __align__(8) float stat[2][G::kSteps];  // -mean, 1 / deviation
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, warps = blockDim.x >> 5, sl = lane % G::kLs;
    const int each = blockDim.x / G::kLs, c0 = t / G::kLs, dim = (int)p.dim;  // channels c0, c0 + each, ...
    const int64_t tiles = (p.batch * p.L + G::kSteps - 1) / G::kSteps;
    const uint32_t apart = (uint32_t)(each * p.L * (int)sizeof(Tin)), apart_y = (uint32_t)(each * p.L * (int)sizeof(Tout));
    const int step = blockDim.x * 16, span = G::kB * step;  // bytes from unit to unit, batch to batch
    unsigned char *mine = units + t * 16;
    const int full = dim / each / G::kB;  // batches whose units all threads have
    const Tin *x = static_cast<const Tin *>(p.x);
    Tout *y = static_cast<Tout *>(p.y);

    Place at = place_in<Tin>(p, blockIdx.x, sl);
    for_batches(batches, full, [&](int b, auto whole) {
        const int c = c0 + b * G::kB * each;
        copy_batch<Tin, whole.value>(mine + b * span, step, x + at.at + c * p.L, apart, c, each, dim, at.in);
    });
    cp_async_commit();
    // channels of a warp: 8 of every `each` ones
    const auto channels = [&](int w) {
        const int k = dim / each, rest = dim - k * each - w * G::kLc;
        return (float)(k * G::kLc + min(max(rest, 0), G::kLc));
    };
    const int have = c0 < dim ? (dim - c0 + each - 1) / each : 0;
    const float nt = (float)have, inv_n = have ? 1.f / nt : 0.f, inv_w = channels(warp) > 0.f ? 1.f / channels(warp) : 0.f;
    const float inv_0 = have ? 1.f / (float)min(have, G::kB) : 0.f;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        cp_async_wait_all();
        float2 np[G::kStats], D[G::kStats], S[G::kStats];  // -pivot, sums of d and d^2
#pragma unroll
        for (int k = 0; k < G::kStats; ++k) np[k] = D[k] = S[k] = both(0.f);
        for_batches(batches, full, [&](int b, auto whole) {
            Batch<Tin> v;
            v.read(mine + b * span, step);
            const int c = c0 + b * G::kB * each;
            if (b == 0 && !p.rms) {
#pragma unroll
                for (int j = 0; j < G::kB; ++j)
                    if (whole.value || c + j * each < dim) {
#pragma unroll
                        for (int k = 0; k < G::kStats; ++k) np[k] = add2(np[k], v.pair(j, k));
                    }
#pragma unroll
                for (int k = 0; k < G::kStats; ++k) np[k] = mul2(np[k], both(-inv_0));
            }
#pragma unroll
            for (int j = 0; j < G::kB; ++j)
                if (whole.value || c + j * each < dim) {
#pragma unroll
                    for (int k = 0; k < G::kStats; ++k) {
                        const float2 d = add2(v.pair(j, k), np[k]);
                        D[k] = add2(D[k], d);
                        S[k] = fma2(d, d, S[k]);
                    }
                }
        });
        if (!p.rms) {
            // the thread's mean and squares about it, then the warp's
            float2 m[G::kStats], mw[G::kStats];
#pragma unroll
            for (int k = 0; k < G::kStats; ++k) {
                const float2 e = mul2(D[k], both(inv_n));
                S[k] = fma2(mul2(D[k], both(-1.f)), e, S[k]);
                m[k] = sub2(e, np[k]);
                mw[k] = mul2(m[k], both(nt));
            }
            step_sums(mw);
#pragma unroll
            for (int k = 0; k < G::kStats; ++k) {
                D[k] = mul2(mw[k], both(inv_w));
                const float2 d = sub2(m[k], D[k]);
                S[k] = fma2(mul2(d, both(nt)), d, S[k]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < G::kStats; ++k) D[k] = both(0.f);
        }
        step_sums(S);
        if (lane < G::kLs) write_steps(part[warp], sl, D, S);
        __syncthreads();
        if (t < G::kSteps) {
            const float2 all = join(&part[0][t], G::kSteps, warps, channels);
            const float S2 = all.y < 0.f ? 0.f : all.y;  // (a NaN passes)
            const float rstd = rsqrtf(fmaf(S2, p.inv_dim, p.eps));
            stat[0][t] = -all.x, stat[1][t] = rstd;
            const int64_t s = tile * G::kSteps + t;
            if (s < p.batch * p.L) {
                if (p.mean && !p.rms) p.mean[s] = all.x;
                if (p.rstd) p.rstd[s] = rstd;
            }
        }
        __syncthreads();
        read_steps(stat[0], sl, np);
        read_steps(stat[1], sl, S);
        const Place now = at;
        const bool more = tile + gridDim.x < tiles;
        if (more) at = place_in<Tin>(p, tile + gridDim.x, sl);
        for_batches(batches, full, [&](int b, auto whole) {
            const int c = c0 + b * G::kB * each;
            Batch<Tin> v;
            v.read(mine + b * span, step);
            Tout *to = y + now.at + c * p.L;
#pragma unroll
            for (int j = 0; j < G::kB; ++j) {
                if (whole.value || c + j * each < dim) {
                    const float2 w = both(p.weight ? __ldg(p.weight + c + j * each) : 1.f),
                                 bi = both(p.bias ? __ldg(p.bias + c + j * each) : 0.f);
                    float2 r[G::kStats];
#pragma unroll
                    for (int k = 0; k < G::kStats; ++k) r[k] = fma2(mul2(add2(v.pair(j, k), np[k]), S[k]), w, bi);
                    if (now.in) store_unit(at_unit(to, apart_y, j), r);
                }
            }
            if (more) copy_batch<Tin, whole.value>(mine + b * span, step, x + at.at + c * p.L, apart, c, each, dim, at.in);
        });
        cp_async_commit();
    }
}

// Backward: x and dy, and the block's sums of dw and db per channel, in
// shared memory, which leaves one block an SM: 8 x 1536 x 2048 bf16 53 us
// with the second kernel (23.1 for the bytes).
template <typename T>
__global__ void __launch_bounds__(32 * kTileWarps, 1) norm_tile_bwd_kernel(const NormParams p, int batches) {
    using G = Geo<T>;
    extern __shared__ __align__(16) unsigned char units[];
    __shared__ float2 part[kTileWarps][G::kSteps];
    __shared__ __align__(8) float stat[2][G::kSteps];  // sums of v, of v xh
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, warps = blockDim.x >> 5, sl = lane % G::kLs;
    const int each = blockDim.x / G::kLs, c0 = t / G::kLs, dim = (int)p.dim;
    const int64_t tiles = (p.batch * p.L + G::kSteps - 1) / G::kSteps;
    const uint32_t apart = (uint32_t)(each * p.L * (int)sizeof(T));
    const int step = blockDim.x * 16, span = G::kB * step;
    unsigned char *mx = units + t * 16, *mg = mx + batches * span;
    float *acc = reinterpret_cast<float *>(units + 2 * batches * span);  // dw, db
    const int full = dim / each / G::kB;
    const T *x = static_cast<const T *>(p.x), *dy = static_cast<const T *>(p.dy);
    T *dx = static_cast<T *>(p.dx);

    Place at = place_in<T>(p, blockIdx.x, sl);
    for_batches(batches, full, [&](int b, auto whole) {
        const int c = c0 + b * G::kB * each;
        const int64_t from = at.at + c * p.L;
        if (!whole.value) {  // units of channels that are not there stay zero
            for (int j = 0; j < G::kB; ++j) {
                *reinterpret_cast<uint4 *>(mx + b * span + j * step) = make_uint4(0u, 0u, 0u, 0u);
                *reinterpret_cast<uint4 *>(mg + b * span + j * step) = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        copy_batch<T, whole.value>(mx + b * span, step, x + from, apart, c, each, dim, at.in);
        copy_batch<T, whole.value>(mg + b * span, step, dy + from, apart, c, each, dim, at.in);
    });
    cp_async_commit();
    for (int c = t; c < 2 * dim; c += blockDim.x) acc[c] = 0.f;
    __syncthreads();
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        float2 nm[G::kStats], r[G::kStats], s1[G::kStats], s2[G::kStats];
#pragma unroll
        for (int k = 0; k < G::kStats; ++k) {
            const int64_t s = at.index + 2 * k;
            nm[k] = p.mean_in ? make_float2(-__ldg(p.mean_in + s), -__ldg(p.mean_in + s + 1)) : both(0.f);
            r[k] = make_float2(__ldg(p.rstd_in + s), __ldg(p.rstd_in + s + 1));
            s1[k] = s2[k] = both(0.f);
        }
        cp_async_wait_all();
        for_batches(batches, full, [&](int b, auto whole) {
            const int c = c0 + b * G::kB * each;
            Batch<T> vx, vg;
            vx.read(mx + b * span, step);
            vg.read(mg + b * span, step);
            float term[G::kB];
#pragma unroll
            for (int j = 0; j < G::kB; ++j) {
                const int cj = whole.value ? c + j * each : min(c + j * each, dim - 1);
                const float2 w = both(p.weight ? __ldg(p.weight + cj) : 1.f);
                float2 sum = both(0.f);
#pragma unroll
                for (int k = 0; k < G::kStats; ++k) {
                    const float2 g = vg.pair(j, k), h = mul2(g, mul2(add2(vx.pair(j, k), nm[k]), r[k]));
                    s1[k] = fma2(g, w, s1[k]);
                    s2[k] = fma2(h, w, s2[k]);
                    sum = add2(sum, h);
                }
                term[j] = sum.x + sum.y;
            }
            if (p.sums) {
                const float v = lane_sums<G::kB>(term, lane);
                const int cs = c + sl * each;  // this lane's unit of the batch
                if (whole.value || cs < dim) acc[cs] += v;
            }
        });
        step_sums(s1), step_sums(s2);
        if (lane < G::kLs) write_steps(part[warp], sl, s1, s2);
        __syncthreads();
        if (t < G::kSteps) {
            float2 all = both(0.f);
            for (int k = 0; k < warps; ++k) all = add2(all, part[k][t]);
            stat[0][t] = all.x, stat[1][t] = all.y;
        }
        __syncthreads();
        // dx = rstd v - rstd c1 - (x - m) rstd^2 c2, with the step's factors
        // made once; s1, s2: -rstd c1, -rstd^2 c2
        read_steps(stat[0], sl, s1);
        read_steps(stat[1], sl, s2);
#pragma unroll
        for (int k = 0; k < G::kStats; ++k) {
            const float2 f = mul2(r[k], both(-p.inv_dim));
            s1[k] = p.mean_in ? mul2(s1[k], f) : both(0.f);
            s2[k] = mul2(mul2(s2[k], f), r[k]);
        }
        const Place now = at;
        const bool more = tile + gridDim.x < tiles;
        if (more) at = place_in<T>(p, tile + gridDim.x, sl);
        for_batches(batches, full, [&](int b, auto whole) {
            const int c = c0 + b * G::kB * each;
            Batch<T> vx, vg;
            vx.read(mx + b * span, step);
            vg.read(mg + b * span, step);
            T *to = dx + now.at + c * p.L;
            float term[G::kB];
#pragma unroll
            for (int j = 0; j < G::kB; ++j) {
                const int cj = whole.value ? c + j * each : min(c + j * each, dim - 1);
                const float2 w = both(p.weight ? __ldg(p.weight + cj) : 1.f);
                float2 v[G::kStats], sum = both(0.f);
#pragma unroll
                for (int k = 0; k < G::kStats; ++k) {
                    const float2 g = vg.pair(j, k);
                    sum = add2(sum, g);
                    v[k] = fma2(add2(vx.pair(j, k), nm[k]), s2[k], fma2(mul2(g, w), r[k], s1[k]));
                }
                if (now.in && (whole.value || c + j * each < dim)) store_unit(at_unit(to, apart, j), v);
                term[j] = sum.x + sum.y;
            }
            if (more) {
                copy_batch<T, whole.value>(mx + b * span, step, x + at.at + c * p.L, apart, c, each, dim, at.in);
                copy_batch<T, whole.value>(mg + b * span, step, dy + at.at + c * p.L, apart, c, each, dim, at.in);
            }
            if (p.sums) {
                const float v = lane_sums<G::kB>(term, lane);
                const int cs = c + sl * each;
                if (whole.value || cs < dim) acc[dim + cs] += v;
            }
        });
        cp_async_commit();
    }
    if (p.sums) {
        __syncthreads();
        float *out = p.part + (int64_t)blockIdx.x * 2 * p.dim;
        for (int c = t; c < 2 * dim; c += blockDim.x) out[c] = acc[c];
    }
}

// More channels than a cluster's registers hold: passes over the tile, the
// later ones from the caches.
template <typename Tin, typename Tout>
__global__ void __launch_bounds__(512) norm_steps_fwd_wide_kernel(const NormParams p) {
    __shared__ float sm[2][16][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const Place st = place_of<1>(p, blockIdx.x, lane);
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
        const Place st = place_of<1>(p, tile, lane);
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

// dw and db from the rows of partial sums: 32 columns by 32 runs of rows per
// block, each run and then the runs added in order.
__global__ void __launch_bounds__(1024) norm_sums_kernel(const float *part, int64_t parts, int64_t dim, float *dweight,
                                                         float *dbias) {
    __shared__ float sm[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + tx;
    float s = 0.f;
    if (c < 2 * dim) {
        constexpr int kAt = 10;  // loads in flight
        for (int64_t k = ty; k < parts; k += 32 * kAt) {
            float v[kAt];
#pragma unroll
            for (int i = 0; i < kAt; ++i) v[i] = part[min(k + 32 * i, parts - 1) * 2 * dim + c];
#pragma unroll
            for (int i = 0; i < kAt; ++i) s += k + 32 * i < parts ? v[i] : 0.f;
        }
    }
    sm[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < 2 * dim) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) v += sm[k][tx];
        if (c < dim) {
            if (dweight) dweight[c] = v;
        } else if (dbias) {
            dbias[c - dim] = v;
        }
    }
}

// ------------------------------------------------------------------- host

// The launch of a shape: kernel family, threads and blocks.
enum NormKind { kRows, kRowsWide, kTile, kPairs, kCluster, kStepsWide };
struct NormPlan {
    NormKind kind;
    bool vec;
    int T, nv, per;    // rows: threads per row, vectors per thread, rows per block; tile: threads
    int batches;       // tile: batches of a thread
    int V, warps, max_warps, nblk;  // cluster: steps of a lane's run, warps per block and at most, blocks
    int64_t blocks, parts;          // blocks (clusters); rows of partial sums of the backward
};

constexpr int kRowThreads = 256;          // of a block, unless one row takes more
constexpr int64_t kSmMost = 228 * 1024;   // shared memory of an SM, and of a block with its reserve of 1 KB
constexpr int64_t kBlockMost = 227 * 1024;
constexpr int64_t kTileOwn = 5 * 1024;    // the tile kernels' static shared memory, rounded up
constexpr int kSmDefault = 40 * 1024;     // dynamic shared memory that needs no attribute beside a kernel's own

// The most dynamic shared memory that any launch of the kernel asks for: one
// value for all of them, as calls from other threads set it too.
template <typename K>
cudaError_t allow_smem(K kernel, int most) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

// Dynamic shared memory of the tile kernels.
int64_t tile_smem(int64_t dim, const NormPlan &pl, bool back) {
    const int64_t units = (int64_t)pl.batches * pl.T * 64;
    return back ? 2 * units + 8 * dim : units;
}

// What the innermost axis allows at every base: whole vectors, words of two steps.
enum NormWords { kSingle, kWords, kVectors };
NormPlan norm_plan(const ss_desc *desc, NormWords words, bool back) {
    const bool vec = words == kVectors;
    NormPlan pl{};
    const int64_t sms = layer_sm_count();
    pl.vec = vec;
    if (desc->seqlen == 1) {
        // The fewest threads that hold a row with three vectors each at most
        // (two where elements are loaded one by one and cost more registers):
        // the backward's sums, parameters and inputs then stay in 128 registers.
        // (Backward of 16384 rows of 768 bf16: 25 us, 31 with two vectors at
        // most, 43 with one; 16001 rows of 1001, element by element: 59, 67
        // with one.)
        const int64_t vecs = (desc->dim + kV - 1) / kV, most = vec ? 3 : 2;
        pl.T = 32;
        while (pl.T < 512 && vecs > (int64_t)pl.T * most) pl.T *= 2;
        pl.nv = (int)((vecs + pl.T - 1) / pl.T);
        pl.kind = pl.nv > most ? kRowsWide : kRows;
        pl.per = pl.kind == kRowsWide || pl.T > kRowThreads ? 1 : kRowThreads / pl.T;
        const int64_t blocks = (desc->batch + pl.per - 1) / pl.per;
        const int64_t resident = pl.kind == kRowsWide || pl.T > kRowThreads ? sms : 2 * sms;
        pl.blocks = pl.parts = blocks < resident ? blocks : resident;
        return pl;
    }
    const int64_t n = desc->batch * desc->seqlen;
    // Tiles of 64 bytes of every channel in shared memory, while they fit:
    // the channels over T threads, in batches of T.  (8 x 1536 x 2048 bf16:
    // forward 30 us against 36 in clusters, backward 53 against 69, with 256
    // threads 35 and 67; fp32 4 x 1024 x 4096 forward 33 against 41; 4 x 256 x
    // 16384 backward 38 against 36; with rows
    // that are not whole vectors the same scheme with 4- or 2-byte units took
    // 69 against 67 and 148 against 137, fp32 of 1000 x 4099 backward 65
    // against 55: those go to the clusters.)  The backward has dy in x's type;
    // the bytes between a thread's channels are counted in 32 bits.
    const int64_t steps = desc->in_dtype == SS_BF16 ? 32 : 16, tiles = (n + steps - 1) / steps;
    pl.batches = (int)((desc->dim + 511) / 512);
    pl.T = (int)(((desc->dim + pl.batches - 1) / pl.batches + 31) / 32 * 32);
    const int64_t smem = tile_smem(desc->dim, pl, back) + kTileOwn;
    if (vec && smem <= kBlockMost && !(back && desc->in_dtype != desc->out_dtype) && desc->seqlen <= 1 << 20) {
        pl.kind = kTile;
        int64_t resident = 65536 / (pl.T * (back ? 128 : 64));
        if (resident > kSmMost / (smem + 1024)) resident = kSmMost / (smem + 1024);
        if (resident < 1) resident = 1;
        pl.blocks = pl.parts = tiles < resident * sms ? tiles : resident * sms;
        return pl;
    }
    // Words of two steps, the channels in the registers of up to 8 blocks of 8
    // warps, unless tiles that end with the row leave over a fifth of the lanes
    // without a step, or there are too few of them to go round (1 x 500 x 1001:
    // 10.4 us against 8.3 in single steps, whose tiles are half as long).
    const int64_t need = (desc->dim + kWarpCh - 1) / kWarpCh;
    const int64_t row_tiles = (desc->seqlen + kPairSteps - 1) / kPairSteps;
    pl.blocks = desc->batch * row_tiles, pl.nblk = (int)((need + kPairWarps - 1) / kPairWarps);
    if (words == kWords && !back && desc->in_dtype == SS_BF16 && pl.nblk <= 8 &&
        row_tiles * kPairSteps * 4 <= desc->seqlen * 5 && pl.blocks * pl.nblk >= 2 * sms) {
        pl.kind = kPairs;
        pl.warps = (int)((need + pl.nblk - 1) / pl.nblk);
        if (pl.warps < 2) pl.warps = 2;  // a thread for each step of the tile
        return pl;
    }
    // The channels in the registers of up to 8 blocks of 8 warps, or of 16
    // where 8 do not hold them (8 x 1536 x 2047 bf16, forward in single steps:
    // 90 us with blocks of 16, 64 with 8).
    pl.max_warps = need <= 64 ? 8 : 16;
    const int64_t nblk = (need + pl.max_warps - 1) / pl.max_warps;
    if (nblk <= 8) {
        pl.kind = kCluster;
        pl.nblk = (int)nblk;
        pl.warps = (int)((need + nblk - 1) / nblk);
        if (pl.warps < 2) pl.warps = 2;  // a thread for each step of the tile
        pl.V = !vec ? 1 : desc->in_dtype == SS_BF16 ? 8 : 4;
        const int64_t wide = pl.V == 8 ? 64 : 32, count = (n + wide - 1) / wide;
        // Clusters that run at the same time: a cluster lies within one of the
        // eight groups of SMs, which are not all of a size, hence a margin (one
        // cluster too many runs alone after all the others: 71 us, not 55, for
        // 3 x 1000 x 4099 fp32).
        const int64_t resident = nblk <= 2 ? sms * (pl.max_warps == 8 ? 2 : 1) / nblk
                                           : sms / 8 * (pl.max_warps == 8 ? 2 : 1) / nblk * 8 * 92 / 100;
        pl.blocks = count;
        pl.parts = count < resident ? count : resident;
        return pl;
    }
    pl.kind = kStepsWide;
    pl.blocks = (n + 31) / 32;
    pl.parts = pl.blocks < sms ? pl.blocks : sms;
    return pl;
}

// Whole vectors: rows of dim elements, or steps of each channel.  (The kernels
// over the steps read their parameters one by one, the row kernels in vectors.)
NormWords norm_words(const ss_desc *desc, std::initializer_list<const void *> tensors, std::initializer_list<const void *> params) {
    const int64_t inner = desc->seqlen == 1 ? desc->dim : desc->seqlen;
    const int64_t whole = desc->seqlen == 1 || desc->in_dtype == SS_BF16 ? 8 : 4;
    if (inner % whole == 0 && vec_ok(tensors) && (desc->seqlen > 1 || vec_ok(params))) return kVectors;
    for (const void *q : tensors)
        if (!layer_aligned(q, 2 * layer_size(desc->out_dtype))) return kSingle;
    return kWords;
}

template <typename K>
cudaError_t launch_cluster(K kernel, int64_t grid, int threads, int nblk, cudaStream_t s, const NormParams &p) {
    if (nblk == 1) {
        kernel<<<(unsigned)grid, (unsigned)threads, 0, s>>>(p, nblk);
        return cudaGetLastError();
    }
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
    const int threads = pl.T * pl.per;
    if (back) {
        const size_t smem = pl.per > 1 ? (size_t)pl.per * p.dim * 2 * sizeof(float) : 0;  // 48 KB at most: 256 threads of 24 columns
        if (smem > kSmDefault) {
            const cudaError_t e = allow_smem(norm_rows_bwd_kernel<Tin, Tout, kNv, kVec>, 48 * 1024);
            if (e != cudaSuccess) return e;
        }
        norm_rows_bwd_kernel<Tin, Tout, kNv, kVec><<<(unsigned)pl.parts, threads, smem, s>>>(p, pl.T);
    } else {
        norm_rows_fwd_kernel<Tin, Tout, kNv, kVec><<<(unsigned)pl.parts, threads, 0, s>>>(p, pl.T);
    }
    return cudaGetLastError();
}

template <typename Tin, typename Tout, int V, int kMaxW>
cudaError_t launch_steps(bool back, const NormPlan &pl, cudaStream_t s, const NormParams &p) {
    if (back)
        return launch_cluster(norm_steps_bwd_kernel<Tin, Tout, V, kMaxW>, pl.parts * pl.nblk, 32 * pl.warps, pl.nblk, s, p);
    return launch_cluster(norm_steps_fwd_kernel<Tin, Tout, V, kMaxW>, pl.blocks * pl.nblk, 32 * pl.warps, pl.nblk, s, p);
}

template <typename Tin, typename Tout>
cudaError_t launch_tile(bool back, const NormPlan &pl, cudaStream_t s, const NormParams &p) {
    const auto kernel = back ? norm_tile_bwd_kernel<Tin> : norm_tile_fwd_kernel<Tin, Tout>;
    const int smem = (int)tile_smem(p.dim, pl, back);
    if (smem > kSmDefault) {
        const cudaError_t e = allow_smem(kernel, (int)(kBlockMost - kTileOwn));
        if (e != cudaSuccess) return e;
    }
    kernel<<<(unsigned)pl.blocks, pl.T, smem, s>>>(p, pl.batches);
    return cudaGetLastError();
}

template <typename Tin, typename Tout>
cudaError_t dispatch_norm(bool back, const NormPlan &pl, cudaStream_t s, const NormParams &p) {
    constexpr int kWhole = sizeof(Tin) == 2 ? 8 : 4;
    switch (pl.kind) {
        case kRowsWide:
            if (back) norm_rows_bwd_wide_kernel<Tin, Tout><<<(unsigned)pl.parts, 1024, 0, s>>>(p);
            else norm_rows_fwd_wide_kernel<Tin, Tout><<<(unsigned)p.batch, 1024, 0, s>>>(p);
            return cudaGetLastError();
        case kStepsWide:
            if (back) norm_steps_bwd_wide_kernel<Tin, Tout><<<(unsigned)pl.parts, 512, 0, s>>>(p);
            else norm_steps_fwd_wide_kernel<Tin, Tout><<<(unsigned)pl.blocks, 512, 0, s>>>(p);
            return cudaGetLastError();
        case kRows:
            if (!pl.vec)
                return pl.nv == 1 ? launch_rows<Tin, Tout, 1, false>(back, pl, s, p)
                                  : launch_rows<Tin, Tout, 2, false>(back, pl, s, p);
            return pl.nv == 1   ? launch_rows<Tin, Tout, 1, true>(back, pl, s, p)
                   : pl.nv == 2 ? launch_rows<Tin, Tout, 2, true>(back, pl, s, p)
                                : launch_rows<Tin, Tout, 3, true>(back, pl, s, p);
        case kTile: return launch_tile<Tin, Tout>(back, pl, s, p);
        case kPairs:
            if constexpr (sizeof(Tin) == 2)
                return launch_cluster(norm_pairs_fwd_kernel<Tout>, pl.blocks * pl.nblk, 32 * pl.warps, pl.nblk, s, p);
            break;
        default: break;
    }
    if (pl.max_warps == 8)
        return pl.V == 1 ? launch_steps<Tin, Tout, 1, 8>(back, pl, s, p) : launch_steps<Tin, Tout, kWhole, 8>(back, pl, s, p);
    return pl.V == 1 ? launch_steps<Tin, Tout, 1, 16>(back, pl, s, p) : launch_steps<Tin, Tout, kWhole, 16>(back, pl, s, p);
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
    const NormPlan pl = norm_plan(desc, norm_words(desc, {x, y}, {weight, bias}), false);
    return status_of(SS_LAYER_DISPATCH(desc, dispatch_norm)(false, pl, reinterpret_cast<cudaStream_t>(stream), p));
}

size_t ss_norm_bwd_workspace_bytes(const ss_desc *desc) {
    LayerSizes sz;
    if (check_norm(desc, &sz) != SS_OK || sz.elems == 0) return 0;
    // the largest of the shapes: which one runs depends on the pointers too
    int64_t most = 0;
    for (const NormWords w : {kSingle, kVectors}) {  // (words of two steps: the forward alone)
        const int64_t parts = norm_plan(desc, w, true).parts;
        most = parts > most ? parts : most;
    }
    return (size_t)most * 2 * (size_t)desc->dim * sizeof(float);
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
    NormParams p = norm_params(desc);
    p.sums = dweight || dbias;
    if (p.sums) {
        if (!workspace || workspace_bytes < ss_norm_bwd_workspace_bytes(desc)) return SS_ERR_WORKSPACE;
        if (!layer_aligned(workspace, 16)) return SS_ERR_MISALIGNED;
    }
    p.x = x, p.weight = weight, p.mean_in = mean, p.rstd_in = rstd, p.dy = dy, p.dx = dx;
    p.part = static_cast<float *>(workspace);
    const NormPlan pl = norm_plan(desc, norm_words(desc, {x, dy, dx}, {weight}), true);  // the workspace is aligned
    cudaError_t e = SS_LAYER_DISPATCH(desc, dispatch_norm)(true, pl, s, p);
    if (e == cudaSuccess && p.sums) {
        norm_sums_kernel<<<(unsigned)((2 * p.dim + 31) / 32), 1024, 0, s>>>(p.part, pl.parts, p.dim, dweight, dbias);
        e = cudaGetLastError();
    }
    return status_of(e);
}

}  // extern "C"
