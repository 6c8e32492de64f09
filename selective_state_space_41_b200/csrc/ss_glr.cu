// The gated linear recurrence: forward, backward and one decoding step
// (declarations and the meaning of every argument in include/selscan.h).
//
//   a_t = g_t or sigmoid(g_t),  b_t = x_t or (1 - a_t) x_t
//   h_t = a_t h_(t-1) + b_t     (nothing carried into a sequence start)
//   y_t = h_t or h_t silu(z_t)
//
// One state per row (b, d), so a step costs two or three reads and a write
// and some twenty operations: the kernels are bound by memory, and what the
// design has to do is to keep enough loads in flight and the serial chain of
// the recurrence short.  A warp takes 256 steps of a row at a time, eight per
// lane.  Each lane folds its steps into one pair (A, B): the map h -> A h + B
// of its eight steps.  The pairs compose as (A2, B2) o (A1, B1) = (A2 A1,
// A2 B1 + B2), so five shuffle rounds give every lane the map of all lanes
// before it; applied to the state entering the 256 steps it gives the state
// entering the lane's own, from which the lane runs its steps again, now one
// after the other as the formula has them.  W warps share a row when there
// are few rows: each folds its own 256 steps, and W pairs in shared memory
// join them.  The loads of the next piece are issued before the current one
// is worked on.
//
// Sequence starts cut the maps: behind a start the entering state does not
// count, whatever it is (an infinity or a NaN of another sequence included),
// so a cut is carried as a bit and selects instead of multiplying by zero.
//
// Backward: with dh = dy (silu(z)) the adjoint obeys lam_t = dh_t + m_(t+1),
// m_t = a_t lam_t, where m_t is what reaches the step before.  In m it is a
// recurrence of the same form, m_t = a_t m_(t+1) + a_t dh_t, with the step's
// own decay, run from the last step back over the same pieces of 256 steps.
// The forward kept the state entering every piece (4 bytes per 256 steps),
// so each warp recomputes its states from registers alone, and no second
// pass over the sequence is needed.
//   dx = lam (1 - a) or lam;  da = lam (h_(t-1) - x) or lam h_(t-1);
//   dg = da a (1 - a) or da;  dz = dy h silu'(z)
#include "ss_layer.cuh"

namespace selscan {
namespace {

constexpr int kPiece = 256;   // steps a warp takes at a time; also the checkpoint stride
constexpr int kMaxWarps = 16; // warps sharing a row

struct GlrParams {
    const void *x, *g, *z, *dy;
    const uint8_t *reset;
    const float *h0;      // state before step 0 (forward), or null
    const float *dlast;   // gradient of the state after the last step (backward), or null
    const float *ckpt_in; // the forward's checkpoints (backward)
    void *y, *dx, *dg, *dz;
    float *last, *ckpt, *dh0;
    int64_t rows, dim, L, nck;
    int sigmoid, couple, vec;
};

// a, 1 - a of a step's gate input.
template <bool kFast>
__device__ __forceinline__ void gate(float g, bool sigmoid, float &a, float &keep) {
    if (sigmoid) {
        sigmoid2<kFast>(g, a, keep);
    } else {
        a = g;
        keep = 1.f - g;
    }
}

// Lanes lane-d+1 .. lane as a mask (the lanes a pair stands for before the
// shuffle round of distance d), and lane .. lane+d-1.
__device__ __forceinline__ uint32_t lanes_up_to(int lane, int d) { return ((1u << d) - 1u) << (lane - d + 1); }
__device__ __forceinline__ uint32_t lanes_from(int lane, int d) { return ((1u << d) - 1u) << lane; }

// Inclusive composition over lanes 0..lane.  cuts: lanes that hold a start.
template <bool kR>
__device__ __forceinline__ void scan_up(float &A, float &B, int lane, uint32_t cuts) {
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const float Ao = __shfl_up_sync(0xffffffffu, A, d), Bo = __shfl_up_sync(0xffffffffu, B, d);
        if (lane >= d && !(kR && (cuts & lanes_up_to(lane, d)))) {
            B = fmaf(A, Bo, B);
            A *= Ao;
        }
    }
}

// Inclusive composition over lanes 31..lane (the adjoint's direction).
template <bool kR>
__device__ __forceinline__ void scan_down(float &A, float &B, int lane, uint32_t cuts) {
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const float Ao = __shfl_down_sync(0xffffffffu, A, d), Bo = __shfl_down_sync(0xffffffffu, B, d);
        if (lane + d < 32 && !(kR && (cuts & lanes_from(lane, d)))) {
            B = fmaf(A, Bo, B);
            A *= Ao;
        }
    }
}

struct Pair {
    float A, B;
    int cut;
};

// kMulti: one warp per row, several rows per block; otherwise the block's
// warps share its row.
template <typename Tin, typename Tout, bool kZ, bool kR, bool kMulti>
__global__ void __launch_bounds__(512) glr_fwd_kernel(const GlrParams p) {
    constexpr bool kFast = sizeof(Tin) == 2;
    __shared__ Pair pairs[2][kMaxWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int W = kMulti ? 1 : warps, w = kMulti ? 0 : warp;
    const int64_t row = kMulti ? (int64_t)blockIdx.x * warps + warp : blockIdx.x;
    if (row >= p.rows) return;  // a whole warp of a kMulti block, which has no barrier
    const int64_t e0 = row * p.L;
    const int shift = (int)(e0 & (kV - 1));
    const int64_t base = e0 - shift, steps = shift + p.L;
    const int64_t bl = kR ? row / p.dim * p.L - shift : 0, bl_all = kR ? p.rows / p.dim * p.L : 0;
    const Tin *x = static_cast<const Tin *>(p.x), *g = static_cast<const Tin *>(p.g), *z = static_cast<const Tin *>(p.z);
    Tout *y = static_cast<Tout *>(p.y);
    const bool vec = p.vec, sigmoid = p.sigmoid, couple = p.couple;

    Vec8<Tin> nx, ng, nz;
    uint32_t ncut = 0;
    const auto fetch = [&](int64_t v) {
        const int lo = clamp8(shift - v), hi = clamp8(steps - v);
        load8(ng, g, base + v, lo, hi, vec);
        load8(nx, x, base + v, lo, hi, vec);
        if constexpr (kZ) load8(nz, z, base + v, lo, hi, vec);
        if constexpr (kR) ncut = start_bits(p.reset, bl + v, bl_all, lo, hi);
    };

    float carry = p.h0 ? p.h0[row] : 0.f;
    int buf = 0;
    fetch((int64_t)w * kPiece + lane * kV);
    for (int64_t v0 = 0; v0 < steps; v0 += (int64_t)W * kPiece, buf ^= 1) {
        const int64_t v = v0 + (int64_t)w * kPiece + lane * kV;
        const int lo = clamp8(shift - v), hi = clamp8(steps - v);
        float a[kV], b[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            float keep;
            gate<kFast>(ng[i], sigmoid, a[i], keep);
            b[i] = couple ? keep * nx[i] : nx[i];
        }
        if (lo > 0 || hi < kV) {
#pragma unroll
            for (int i = 0; i < kV; ++i)
                if (i < lo || i >= hi) a[i] = 1.f, b[i] = 0.f;
        }
        const Vec8<Tin> cz = nz;
        const uint32_t cut = ncut;
        if (v0 + (int64_t)W * kPiece < steps) fetch(v + (int64_t)W * kPiece);

        // the lane's map, then the maps of the lanes before it
        float A = 1.f, B = 0.f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const bool c = kR && (cut >> i & 1u);
            B = c ? b[i] : fmaf(a[i], B, b[i]);
            A = c ? 0.f : A * a[i];
        }
        const uint32_t cuts = kR ? __ballot_sync(0xffffffffu, cut != 0) : 0u;
        scan_up<kR>(A, B, lane, cuts);
        const float Aw = __shfl_sync(0xffffffffu, A, 31), Bw = __shfl_sync(0xffffffffu, B, 31);
        float Ax = __shfl_up_sync(0xffffffffu, A, 1), Bx = __shfl_up_sync(0xffffffffu, B, 1);
        if (lane == 0) Ax = 1.f, Bx = 0.f;

        float in = carry;  // the state entering this warp's piece
        if constexpr (kMulti) {
            carry = kR && cuts ? Bw : fmaf(Aw, carry, Bw);
        } else {
            if (lane == 0) pairs[buf][w] = {Aw, Bw, kR && cuts ? 1 : 0};
            __syncthreads();
            float c = carry;
            for (int k = 0; k < W; ++k) {
                if (k == w) in = c;
                const Pair q = pairs[buf][k];
                c = kR && q.cut ? q.B : fmaf(q.A, c, q.B);
            }
            carry = c;
        }
        const int64_t piece = v0 / kPiece + w;
        if (p.ckpt && lane == 0 && piece * kPiece < steps) p.ckpt[row * p.nck + piece] = in;
        float h = kR && (cuts & ((1u << lane) - 1u)) ? Bx : fmaf(Ax, in, Bx);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            h = kR && (cut >> i & 1u) ? b[i] : fmaf(a[i], h, b[i]);
            b[i] = h;
        }
        if (y) {
            if constexpr (kZ) {
#pragma unroll
                for (int i = 0; i < kV; ++i) {
                    float s, c;
                    sigmoid2<kFast>(cz[i], s, c);
                    b[i] *= cz[i] * s;
                }
            }
            store8(y, base + v, lo, hi, vec, b);
        }
    }
    if (p.last && lane == 0 && w == 0) p.last[row] = carry;
}

template <typename Tin, typename Tout, bool kZ, bool kR, bool kMulti>
__global__ void __launch_bounds__(512) glr_bwd_kernel(const GlrParams p) {
    constexpr bool kFast = sizeof(Tin) == 2;
    __shared__ Pair pairs[2][kMaxWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int W = kMulti ? 1 : warps, w = kMulti ? 0 : warp;
    const int64_t row = kMulti ? (int64_t)blockIdx.x * warps + warp : blockIdx.x;
    if (row >= p.rows) return;
    const int64_t e0 = row * p.L;
    const int shift = (int)(e0 & (kV - 1));
    const int64_t base = e0 - shift, steps = shift + p.L;
    const int64_t bl = kR ? row / p.dim * p.L - shift : 0, bl_all = kR ? p.rows / p.dim * p.L : 0;
    const Tin *x = static_cast<const Tin *>(p.x), *g = static_cast<const Tin *>(p.g), *z = static_cast<const Tin *>(p.z);
    const Tout *dy = static_cast<const Tout *>(p.dy);
    const bool vec = p.vec, sigmoid = p.sigmoid, couple = p.couple;

    Vec8<Tin> nx, ng, nz;
    Vec8<Tout> nd;
    uint32_t ncut = 0;
    float nin = 0.f;
    const auto fetch = [&](int64_t v) {
        const int lo = clamp8(shift - v), hi = clamp8(steps - v);
        load8(ng, g, base + v, lo, hi, vec);
        load8(nx, x, base + v, lo, hi, vec);
        load8(nd, dy, base + v, lo, hi, vec);
        if constexpr (kZ) load8(nz, z, base + v, lo, hi, vec);
        if constexpr (kR) ncut = start_bits(p.reset, bl + v, bl_all, lo, hi);
        const int64_t piece = v / kPiece;
        nin = piece * kPiece < steps ? __ldg(p.ckpt_in + row * p.nck + piece) : 0.f;
    };

    const int64_t stride = (int64_t)W * kPiece;
    float carry = p.dlast ? p.dlast[row] : 0.f;
    int buf = 0;
    int64_t v0 = (steps - 1) / stride * stride;
    fetch(v0 + (int64_t)w * kPiece + lane * kV);
    for (; v0 >= 0; v0 -= stride, buf ^= 1) {
        const int64_t v = v0 + (int64_t)w * kPiece + lane * kV;
        const int lo = clamp8(shift - v), hi = clamp8(steps - v);
        const Vec8<Tin> cx = nx, cz = nz, cg = ng;
        const Vec8<Tout> cd = nd;
        const uint32_t cut = ncut;
        const float in = nin;
        if (v0 > 0) fetch(v - stride);

        float a[kV], keep[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) gate<kFast>(cg[i], sigmoid, a[i], keep[i]);
        if (lo > 0 || hi < kV) {
#pragma unroll
            for (int i = 0; i < kV; ++i)
                if (i < lo || i >= hi) a[i] = 1.f, keep[i] = 0.f;
        }
        // the state entering the lane's steps; masked steps have zero inputs
        float A = 1.f, B = 0.f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const bool c = kR && (cut >> i & 1u);
            const float b = couple ? keep[i] * cx[i] : cx[i];
            B = c ? b : fmaf(a[i], B, b);
            A = c ? 0.f : A * a[i];
        }
        const uint32_t cuts = kR ? __ballot_sync(0xffffffffu, cut != 0) : 0u;
        float M = 0.f, Am = A;
        // dh, and the lane's map of the adjoint
        float dh[kV], dzv[kV];
#pragma unroll
        for (int i = kV - 1; i >= 0; --i) {
            dh[i] = cd[i];
            if constexpr (kZ) {
                float s, c;
                sigmoid2<kFast>(cz[i], s, c);
                dzv[i] = dh[i] * (s * fmaf(cz[i], c, 1.f));
                dh[i] *= cz[i] * s;
            }
            M = kR && (cut >> i & 1u) ? 0.f : a[i] * (dh[i] + M);
        }
        scan_up<kR>(A, B, lane, cuts);
        scan_down<kR>(Am, M, lane, cuts);
        float Ax = __shfl_up_sync(0xffffffffu, A, 1), Bx = __shfl_up_sync(0xffffffffu, B, 1);
        if (lane == 0) Ax = 1.f, Bx = 0.f;
        const float Aw = __shfl_sync(0xffffffffu, Am, 0), Mw = __shfl_sync(0xffffffffu, M, 0);
        float Amx = __shfl_down_sync(0xffffffffu, Am, 1), Mx = __shfl_down_sync(0xffffffffu, M, 1);
        if (lane == 31) Amx = 1.f, Mx = 0.f;

        float from = carry;  // the adjoint reaching this warp's piece from behind
        if constexpr (kMulti) {
            carry = kR && cuts ? Mw : fmaf(Aw, carry, Mw);
        } else {
            if (lane == 0) pairs[buf][w] = {Aw, Mw, kR && cuts ? 1 : 0};
            __syncthreads();
            float c = carry;
            for (int k = W - 1; k >= 0; --k) {
                if (k == w) from = c;
                const Pair q = pairs[buf][k];
                c = kR && q.cut ? q.B : fmaf(q.A, c, q.B);
            }
            carry = c;
        }
        float h = kR && (cuts & ((1u << lane) - 1u)) ? Bx : fmaf(Ax, in, Bx);
        float before[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const bool c = kR && (cut >> i & 1u);
            const float b = couple ? keep[i] * cx[i] : cx[i];
            before[i] = c ? 0.f : h;
            h = c ? b : fmaf(a[i], h, b);
            if constexpr (kZ) dzv[i] *= h;
        }
        if constexpr (kZ) store8(static_cast<Tin *>(p.dz), base + v, lo, hi, vec, dzv);
        const uint32_t behind = lane == 31 ? 0u : ~((2u << lane) - 1u);
        float m = kR && (cuts & behind) ? Mx : fmaf(Amx, from, Mx);
#pragma unroll
        for (int i = kV - 1; i >= 0; --i) {
            const float lam = dh[i] + m;
            const float da = lam * (couple ? before[i] - cx[i] : before[i]);
            dh[i] = couple ? lam * keep[i] : lam;
            before[i] = sigmoid ? da * (a[i] * keep[i]) : da;
            m = kR && (cut >> i & 1u) ? 0.f : a[i] * lam;
        }
        store8(static_cast<Tin *>(p.dx), base + v, lo, hi, vec, dh);
        store8(static_cast<Tin *>(p.dg), base + v, lo, hi, vec, before);
    }
    if (p.dh0 && lane == 0 && w == 0) p.dh0[row] = carry;
}

// One step: a thread per row, the state read and written in place.
template <typename Tin, typename Tout>
__global__ void __launch_bounds__(256) glr_step_kernel(const GlrParams p) {
    constexpr bool kFast = sizeof(Tin) == 2;
    const int64_t row = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (row >= p.rows) return;
    float a, keep;
    gate<kFast>(load_elem(static_cast<const Tin *>(p.g), row), p.sigmoid, a, keep);
    const float xv = load_elem(static_cast<const Tin *>(p.x), row);
    const float h = fmaf(a, p.last[row], p.couple ? keep * xv : xv);
    p.last[row] = h;
    float yv = h;
    if (p.z) {
        const float zv = load_elem(static_cast<const Tin *>(p.z), row);
        float s, c;
        sigmoid2<kFast>(zv, s, c);
        yv *= zv * s;
    }
    put(static_cast<Tout *>(p.y), row, yv);
}

int64_t pieces(int64_t L) { return (L + kV - 1 + kPiece - 1) / kPiece; }

// Warps per row: as many as bring the GPU to about kWant warps per SM, no
// more than the row has pieces.
int glr_warps(int64_t rows, int64_t L) {
    constexpr int kWant = 32;
    const int64_t want = (int64_t)layer_sm_count() * kWant, n = pieces(L);
    int w = 1;
    while (w < kMaxWarps && rows * w < want && w < n) w *= 2;
    return w;
}

template <typename Tin, typename Tout, bool kZ, bool kR>
cudaError_t launch_glr(bool back, cudaStream_t s, const GlrParams &p) {
    const int w = glr_warps(p.rows, p.L);
    if (w == 1) {
        constexpr int kRows = 4;
        const unsigned grid = (unsigned)((p.rows + kRows - 1) / kRows);
        if (back) glr_bwd_kernel<Tin, Tout, kZ, kR, true><<<grid, 32 * kRows, 0, s>>>(p);
        else glr_fwd_kernel<Tin, Tout, kZ, kR, true><<<grid, 32 * kRows, 0, s>>>(p);
    } else {
        if (back) glr_bwd_kernel<Tin, Tout, kZ, kR, false><<<(unsigned)p.rows, 32 * w, 0, s>>>(p);
        else glr_fwd_kernel<Tin, Tout, kZ, kR, false><<<(unsigned)p.rows, 32 * w, 0, s>>>(p);
    }
    return cudaGetLastError();
}

template <typename Tin, typename Tout>
cudaError_t dispatch_glr(bool back, cudaStream_t s, const GlrParams &p) {
    if (p.z) return p.reset ? launch_glr<Tin, Tout, true, true>(back, s, p) : launch_glr<Tin, Tout, true, false>(back, s, p);
    return p.reset ? launch_glr<Tin, Tout, false, true>(back, s, p) : launch_glr<Tin, Tout, false, false>(back, s, p);
}

template <typename Tin, typename Tout>
cudaError_t launch_glr_step(cudaStream_t s, const GlrParams &p) {
    glr_step_kernel<Tin, Tout><<<(unsigned)((p.rows + 255) / 256), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace
}  // namespace selscan

using namespace selscan;

extern "C" {

size_t ss_glr_ckpt_elems(const ss_desc *desc) {
    LayerSizes sz;
    if (check_layer(desc, &sz) != SS_OK || sz.elems == 0) return 0;
    return (size_t)sz.rows * (size_t)pieces(desc->seqlen);
}

ss_status ss_glr_fwd(const ss_desc *desc, const void *x, const void *g, const void *z, int gate_sigmoid, int couple,
                     const float *initial_state, const uint8_t *reset, void *y, float *last_state, float *ckpt,
                     ss_stream_t stream) {
    LayerSizes sz;
    const ss_status st = check_layer(desc, &sz);
    if (st != SS_OK) return st;
    if (sz.rows > INT_MAX) return SS_ERR_BAD_SHAPE;
    if (sz.rows == 0) return SS_OK;
    if (!layer_aligned(initial_state, 4) || !layer_aligned(last_state, 4) || !layer_aligned(ckpt, 4)) return SS_ERR_MISALIGNED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (desc->seqlen == 0) {
        if (!last_state || last_state == initial_state) return SS_OK;
        const size_t n = (size_t)sz.rows * 4;
        return status_of(initial_state ? cudaMemcpyAsync(last_state, initial_state, n, cudaMemcpyDeviceToDevice, s)
                                       : cudaMemsetAsync(last_state, 0, n, s));
    }
    if (!x || !g || (!y && !ckpt && !last_state)) return SS_ERR_NULL_POINTER;
    const size_t ein = layer_size(desc->in_dtype), eout = layer_size(desc->out_dtype);
    if (!layer_aligned(x, ein) || !layer_aligned(g, ein) || !layer_aligned(z, ein) || !layer_aligned(y, eout))
        return SS_ERR_MISALIGNED;
    GlrParams p{};
    p.x = x, p.g = g, p.z = z, p.reset = reset, p.h0 = initial_state;
    p.y = y, p.last = last_state, p.ckpt = ckpt;
    p.rows = sz.rows, p.dim = desc->dim, p.L = desc->seqlen, p.nck = pieces(desc->seqlen);
    p.sigmoid = gate_sigmoid != 0, p.couple = couple != 0;
    p.vec = vec_ok({x, g, z, y});
    return status_of(SS_LAYER_DISPATCH(desc, dispatch_glr)(false, s, p));
}

ss_status ss_glr_bwd(const ss_desc *desc, const void *x, const void *g, const void *z, int gate_sigmoid, int couple,
                     const uint8_t *reset, const float *ckpt, const void *dy, const float *d_last_state, void *dx,
                     void *dg, void *dz, float *d_initial_state, ss_stream_t stream) {
    LayerSizes sz;
    const ss_status st = check_layer(desc, &sz);
    if (st != SS_OK) return st;
    if (sz.rows > INT_MAX) return SS_ERR_BAD_SHAPE;
    if (sz.rows == 0) return SS_OK;
    if (!layer_aligned(d_last_state, 4) || !layer_aligned(d_initial_state, 4) || !layer_aligned(ckpt, 4))
        return SS_ERR_MISALIGNED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (desc->seqlen == 0) {
        if (!d_initial_state || d_initial_state == d_last_state) return SS_OK;
        const size_t n = (size_t)sz.rows * 4;
        return status_of(d_last_state ? cudaMemcpyAsync(d_initial_state, d_last_state, n, cudaMemcpyDeviceToDevice, s)
                                      : cudaMemsetAsync(d_initial_state, 0, n, s));
    }
    if (!x || !g || !ckpt || !dy || !dx || !dg || !z != !dz) return SS_ERR_NULL_POINTER;
    const size_t ein = layer_size(desc->in_dtype), eout = layer_size(desc->out_dtype);
    for (const void *q : {x, g, z, (const void *)dx, (const void *)dg, (const void *)dz})
        if (!layer_aligned(q, ein)) return SS_ERR_MISALIGNED;
    if (!layer_aligned(dy, eout)) return SS_ERR_MISALIGNED;
    GlrParams p{};
    p.x = x, p.g = g, p.z = z, p.reset = reset, p.ckpt_in = ckpt, p.dy = dy, p.dlast = d_last_state;
    p.dx = dx, p.dg = dg, p.dz = dz, p.dh0 = d_initial_state;
    p.rows = sz.rows, p.dim = desc->dim, p.L = desc->seqlen, p.nck = pieces(desc->seqlen);
    p.sigmoid = gate_sigmoid != 0, p.couple = couple != 0;
    p.vec = vec_ok({x, g, z, dy, dx, dg, dz});
    return status_of(SS_LAYER_DISPATCH(desc, dispatch_glr)(true, s, p));
}

ss_status ss_glr_step(const ss_desc *desc, const void *x, const void *g, const void *z, int gate_sigmoid, int couple,
                      float *state, void *y, ss_stream_t stream) {
    LayerSizes sz;
    const ss_status st = check_layer(desc, &sz);
    if (st != SS_OK) return st;
    if (desc->seqlen != 1 || sz.rows > INT_MAX) return SS_ERR_BAD_SHAPE;
    if (sz.rows == 0) return SS_OK;
    if (!x || !g || !state || !y) return SS_ERR_NULL_POINTER;
    const size_t ein = layer_size(desc->in_dtype), eout = layer_size(desc->out_dtype);
    if (!layer_aligned(x, ein) || !layer_aligned(g, ein) || !layer_aligned(z, ein) || !layer_aligned(y, eout) ||
        !layer_aligned(state, 4))
        return SS_ERR_MISALIGNED;
    GlrParams p{};
    p.x = x, p.g = g, p.z = z, p.y = y, p.last = state;
    p.rows = sz.rows, p.dim = desc->dim, p.L = 1;
    p.sigmoid = gate_sigmoid != 0, p.couple = couple != 0;
    return status_of(SS_LAYER_DISPATCH(desc, launch_glr_step)(reinterpret_cast<cudaStream_t>(stream), p));
}

}  // extern "C"
