// The gated linear recurrence: forward, backward and one decoding step
// (declarations and the meaning of every argument in include/selscan.h).
//
//   a_t = g_t or sigmoid(g_t),  b_t = x_t or (1 - a_t) x_t
//   h_t = a_t h_(t-1) + b_t     (nothing carried into a sequence start)
//   y_t = h_t or h_t silu(z_t)
//
// One state per row (b, d), so a step costs two or three reads and a write
// and some twenty operations: the kernels are bound by memory, and close
// behind it by the instructions they issue.  What the design has to do is to
// keep enough loads in flight, the serial chain of the recurrence short and
// the work per step small (4 x 1024 x 100000 bf16: 460 us, 375 for the
// bytes; 8 x 1536 x 2048 with the output gate, forward 41 and backward 73,
// 30.7 and 53.7 for the bytes; issue 55 to 60 %; fp32 4 x 1024 x 4096 with the
// gate, forward 47, 41.0 for the bytes).  G lanes take a row (32, or fewer for short rows),
// 16 steps each at a time forward and 8 backward.  Each lane folds its steps
// into one pair (A, B): the map h -> A h + B.  The pairs compose as
// (A2, B2) o (A1, B1) = (A2 A1, A2 B1 + B2), so log2 G shuffle rounds give
// every lane the map of all lanes before it; applied to the state entering
// the G lanes' steps it gives the state entering the lane's own, from which
// the lane runs its steps again, now one after the other as the formula has
// them.  W warps share a row when there are few rows: each folds its own
// steps, and W pairs in shared memory join them (of a cluster's blocks, where
// rows are very few: each warp writes its pair to all of them).  The loads of the next steps
// are issued before the current ones are worked on; gates and products are
// computed in pairs of steps with the packed arithmetic of two floats.
//
// The A of a map is a product of up to 512 decays.  With decays of at most one
// in size it cannot overflow, and an A that underflows to zero loses no more
// than the state's own decay does; larger ones are outside the operator's
// domain (an infinite A and a state of zero give NaN).
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
#include <type_traits>

#include "ss_layer.cuh"

namespace selscan {
namespace {

constexpr int kPiece = 256;    // steps between two checkpoints of a row
constexpr int kMaxWarps = 16;  // warps of a block sharing a row
constexpr int kMaxBlocks = 8;  // blocks sharing one: a cluster

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

// Calls f with the two flags as constants: what depends on them is then
// decided once, not at every step.
template <typename F>
__device__ __forceinline__ void with_flags(bool sigmoid, bool couple, F f) {
    if (sigmoid) {
        if (couple) f(std::true_type{}, std::true_type{});
        else f(std::true_type{}, std::false_type{});
    } else {
        if (couple) f(std::false_type{}, std::true_type{});
        else f(std::false_type{}, std::false_type{});
    }
}

// a, 1 - a of two gate inputs.  With g held from -87 on (a NaN passes),
// e = exp(-g) stays below 2^126, so 1 / (1 + e) and e / (1 + e) are finite and
// not flushed, and each has its full relative precision: 1 - a of a slow decay
// does not come from a subtraction.  (The least a is some 10^-38.)
template <typename T>
__device__ __forceinline__ void gate2(float2 g, bool sigmoid, float2 &a, float2 &keep) {
    if (!sigmoid) {
        a = g;
        keep = sub2(both(1.f), g);
    } else {
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(g.x) : "f"(g.x), "f"(-87.f));
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(g.y) : "f"(g.y), "f"(-87.f));
        const float2 e = exp_neg2<T>(g);
        a = rcp2(add2(e, both(1.f)));
        keep = mul2(e, a);
    }
}

// The lanes that a pair stands for before the shuffle round of distance d:
// lane-d+1 .. lane, and lane .. lane+d-1, as masks.
__device__ __forceinline__ uint32_t lanes_up_to(int lane, int d) { return ((1u << d) - 1u) << (lane - d + 1); }
__device__ __forceinline__ uint32_t lanes_from(int lane, int d) { return ((1u << d) - 1u) << lane; }

// Inclusive composition over the row's lanes up to this one.  G: its lanes
// (kG of them, or `lanes` where kG is 0); cuts: lanes that hold a start.
template <bool kR, int kG>
__device__ __forceinline__ void scan_up(float &A, float &B, int lane, int lanes, uint32_t cuts) {
    const int G = kG ? kG : lanes, in = lane & (G - 1);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        if (d >= G) break;
        const float Ao = __shfl_up_sync(0xffffffffu, A, d), Bo = __shfl_up_sync(0xffffffffu, B, d);
        if (in >= d && !(kR && (cuts & lanes_up_to(lane, d)))) {
            B = fmaf(A, Bo, B);
            A *= Ao;
        }
    }
}

// Inclusive composition over the row's lanes from the last to this one (the
// adjoint's direction).
template <bool kR, int kG>
__device__ __forceinline__ void scan_down(float &A, float &B, int lane, int lanes, uint32_t cuts) {
    const int G = kG ? kG : lanes, in = lane & (G - 1);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        if (d >= G) break;
        const float Ao = __shfl_down_sync(0xffffffffu, A, d), Bo = __shfl_down_sync(0xffffffffu, B, d);
        if (in + d < G && !(kR && (cuts & lanes_from(lane, d)))) {
            B = fmaf(A, Bo, B);
            A *= Ao;
        }
    }
}

enum Share { kOwn, kBlock, kCluster };  // who shares a row

struct Pair {
    float A, B;
    int cut;
};

// A warp's pair (from its first lanes) to all blocks that share its row, and
// the meeting of their warps.
template <int kShare>
__device__ __forceinline__ void share(Pair *to, const Pair &q, int lane, int nblk) {
    if constexpr (kShare == kBlock) {
        if (lane == 0) *to = q;
        __syncthreads();
        return;
    }
    if (lane < nblk) {
        uint32_t at;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(to)), "r"(lane));
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(q.A) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 4), "f"(q.B) : "memory");
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at + 8), "r"(q.cut) : "memory");
    }
    cluster_arrive();
    cluster_wait();
}

// Vectors of a lane in the forward: 16 steps of bf16 halve what the scan over
// the lanes costs a step (8 x 1536 x 2048: 37.5 us against 39), and would
// take all the registers with fp32 (3 x 1000 x 4099: 45 us against 41).
template <typename T>
constexpr int kGlrVecs = sizeof(T) == 2 ? 2 : 1;

// Where a row lies, in virtual steps from the 8-element boundary before it.
struct Row {
    int64_t row, base, steps;
    int shift;
    bool there;
};
template <int kShare>
__device__ __forceinline__ Row row_of(const GlrParams &p, int lanes, int nblk) {
    Row r;
    const int per = kShare != kOwn ? 1 : (int)blockDim.x / lanes;  // rows of a block
    r.row = kShare == kCluster ? blockIdx.x / nblk : kShare == kBlock ? blockIdx.x : (int64_t)blockIdx.x * per + (int)threadIdx.x / lanes;
    r.there = r.row < p.rows;
    if (!r.there) r.row = p.rows - 1;  // lanes that only take part in their warp's shuffles
    const int64_t e0 = r.row * p.L;
    r.shift = (int)(e0 & (kV - 1));
    r.base = e0 - r.shift;
    r.steps = r.shift + p.L;
    return r;
}

// Steps [lo, hi) of the kV at virtual step v that are the row's.
__device__ __forceinline__ void bounds_of(const Row &r, int64_t v, int &lo, int &hi) {
    const int64_t left = r.steps - v;
    lo = v == 0 ? r.shift : 0;
    hi = left >= kV ? kV : left > 0 ? (int)left : 0;
}

// kShare: the warps of a block, or of a cluster of nblk, share a row; otherwise every kG lanes (kG 0:
// `lanes`) have a row of their own.
template <typename Tin, typename Tout, bool kZ, bool kR, int kShare, int kG>
__global__ void __launch_bounds__(512) glr_fwd_kernel(const GlrParams p, int lanes, int nblk) {
    constexpr int kVecs = kGlrVecs<Tin>, kE = kVecs * kV;  // steps of a lane
    __shared__ Pair pairs[2][kShare == kCluster ? kMaxWarps * kMaxBlocks : kMaxWarps];
    const int G = kG ? kG : lanes, lane = threadIdx.x & 31, in = lane & (G - 1);
    const int wb = (int)blockDim.x >> 5, W = kShare == kOwn ? 1 : kShare == kBlock ? wb : wb * nblk;
    const int w = (kShare == kOwn ? 0 : (int)threadIdx.x >> 5) + (kShare == kCluster ? (int)(blockIdx.x % nblk) * wb : 0);
    const Row r = row_of<kShare>(p, G, nblk);
    if constexpr (kShare == kCluster) {  // every block has begun before the first remote store
        cluster_arrive();
        cluster_wait();
    }
    const int64_t bl = kR ? r.row / p.dim * p.L - r.shift : 0, bl_all = kR ? p.rows / p.dim * p.L : 0;
    const Tin *x = static_cast<const Tin *>(p.x) + r.base, *g = static_cast<const Tin *>(p.g) + r.base;
    const Tin *z = kZ ? static_cast<const Tin *>(p.z) + r.base : nullptr;
    Tout *y = static_cast<Tout *>(p.y) + r.base;
    const bool vec = p.vec, sigmoid = p.sigmoid, couple = p.couple;
    const int64_t span = (int64_t)G * kE, stride = W * span;  // steps of the row's lanes in a warp, in the block

    Vec8<Tin> nx[kVecs], ng[kVecs], nz[kVecs];
    uint32_t ncut = 0;
    const auto fetch = [&](int64_t v) {
        ncut = 0;
        if (vec && v >= r.shift && v + kE <= r.steps) {
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                ng[k].load(g, v + k * kV);
                nx[k].load(x, v + k * kV);
                if constexpr (kZ) nz[k].load(z, v + k * kV);
                if constexpr (kR) ncut |= start_bits(p.reset, bl + v + k * kV, bl_all, 0, kV) << (k * kV);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                int lo, hi;
                bounds_of(r, v + k * kV, lo, hi);
                const int64_t e = v + k * kV, n = p.rows * p.L - r.base;  // (elements from r.base to the tensor's end)
                load_row8(ng[k], g, e, n, lo, hi, vec);
                load_row8(nx[k], x, e, n, lo, hi, vec);
                if constexpr (kZ) load_row8(nz[k], z, e, n, lo, hi, vec);
                if constexpr (kR) ncut |= start_bits(p.reset, bl + v + k * kV, bl_all, lo, hi) << (k * kV);
            }
        }
    };

    float carry = p.h0 ? p.h0[r.row] : 0.f;
    int buf = 0;
    const int64_t mine = w * span + (int64_t)in * kE;
    // (rows that share a warp have one turn, whatever their shifts: glr_shape)
    fetch(mine);
    for (int64_t v0 = 0; v0 < r.steps; v0 += stride, buf ^= 1) {
        const int64_t v = v0 + mine;
        float a[kE], b[kE];
        with_flags(sigmoid, couple, [&](auto sig, auto cpl) {
#pragma unroll
            for (int i = 0; i < kE; i += 2) {
                float2 a2, k2, b2 = nx[i / kV].pair(i % kV / 2);
                gate2<Tin>(ng[i / kV].pair(i % kV / 2), sig.value, a2, k2);
                if (cpl.value) b2 = mul2(k2, b2);
                a[i] = a2.x, a[i + 1] = a2.y, b[i] = b2.x, b[i + 1] = b2.y;
            }
        });
        const bool inner = v >= r.shift && v + kE <= r.steps;  // all of the lane's steps are the row's
        if (!inner) {
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                int lo, hi;
                bounds_of(r, v + k * kV, lo, hi);
#pragma unroll
                for (int i = 0; i < kV; ++i)
                    if (i < lo || i >= hi) a[k * kV + i] = 1.f, b[k * kV + i] = 0.f;
            }
        }
        Vec8<Tin> cz[kVecs];
#pragma unroll
        for (int k = 0; k < kVecs; ++k) cz[k] = nz[k];
        const uint32_t cut = ncut;
        if (v0 + stride < r.steps) fetch(v + stride);

        // the lane's map, then the maps of the lanes before it
        float A = 1.f, B = 0.f;
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            const bool c = kR && (cut >> i & 1u);
            B = c ? b[i] : fmaf(a[i], B, b[i]);
            A = c ? 0.f : A * a[i];
        }
        const uint32_t cuts = kR ? __ballot_sync(0xffffffffu, cut != 0) : 0u;
        scan_up<kR, kG>(A, B, lane, lanes, cuts);
        const int last = lane | (G - 1);  // the row's last lane in the warp
        const uint32_t row_cuts = kR ? cuts & lanes_up_to(last, G == 32 ? 31 : G) : 0u;
        const bool any = kR && (G == 32 ? cuts != 0 : row_cuts != 0);
        const float Aw = __shfl_sync(0xffffffffu, A, last), Bw = __shfl_sync(0xffffffffu, B, last);
        float Ax = __shfl_up_sync(0xffffffffu, A, 1), Bx = __shfl_up_sync(0xffffffffu, B, 1);
        if (in == 0) Ax = 1.f, Bx = 0.f;

        float from = carry;  // the state entering this warp's steps
        if constexpr (kShare != kOwn) {
            share<kShare>(&pairs[buf][w], {Aw, Bw, any ? 1 : 0}, lane, nblk);
            float c = carry;
            for (int k = 0; k < W; ++k) {
                if (k == w) from = c;
                const Pair q = pairs[buf][k];
                c = kR && q.cut ? q.B : fmaf(q.A, c, q.B);
            }
            carry = c;
        } else {
            carry = any ? Bw : fmaf(Aw, carry, Bw);
        }
        float h = kR && in > 0 && (cuts & lanes_up_to(lane - 1, in)) ? Bx : fmaf(Ax, from, Bx);
        if (p.ckpt && v % kPiece == 0 && v < r.steps && r.there) p.ckpt[r.row * p.nck + v / kPiece] = h;
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            h = kR && (cut >> i & 1u) ? b[i] : fmaf(a[i], h, b[i]);
            b[i] = h;
        }
        if (!p.y || !r.there) continue;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            float o[kV];
#pragma unroll
            for (int i = 0; i < kV; i += 2) {
                float2 h2 = make_float2(b[k * kV + i], b[k * kV + i + 1]);
                if constexpr (kZ) h2 = mul2(h2, silu2<Tin>(cz[k].pair(i / 2)));
                o[i] = h2.x, o[i + 1] = h2.y;
            }
            if (inner && vec) {
                store_vec(y + v + k * kV, o);
            } else {
                int lo, hi;
                bounds_of(r, v + k * kV, lo, hi);
                store8(y, v + k * kV, lo, hi, vec, o);
            }
        }
    }
    if (p.last && r.there && in == 0 && w == 0) p.last[r.row] = carry;
}

template <typename Tin, typename Tout, bool kZ, bool kR, int kShare, int kG>
__global__ void __launch_bounds__(512) glr_bwd_kernel(const GlrParams p, int lanes, int nblk) {
    __shared__ Pair pairs[2][kShare == kCluster ? kMaxWarps * kMaxBlocks : kMaxWarps];
    const int G = kG ? kG : lanes, lane = threadIdx.x & 31, in = lane & (G - 1);
    const int wb = (int)blockDim.x >> 5, W = kShare == kOwn ? 1 : kShare == kBlock ? wb : wb * nblk;
    const int w = (kShare == kOwn ? 0 : (int)threadIdx.x >> 5) + (kShare == kCluster ? (int)(blockIdx.x % nblk) * wb : 0);
    const Row r = row_of<kShare>(p, G, nblk);
    if constexpr (kShare == kCluster) {  // every block has begun before the first remote store
        cluster_arrive();
        cluster_wait();
    }
    const int64_t bl = kR ? r.row / p.dim * p.L - r.shift : 0, bl_all = kR ? p.rows / p.dim * p.L : 0;
    const Tin *x = static_cast<const Tin *>(p.x) + r.base, *g = static_cast<const Tin *>(p.g) + r.base;
    const Tin *z = kZ ? static_cast<const Tin *>(p.z) + r.base : nullptr;
    const Tout *dy = static_cast<const Tout *>(p.dy) + r.base;
    Tin *dx = static_cast<Tin *>(p.dx) + r.base, *dg = static_cast<Tin *>(p.dg) + r.base;
    Tin *dz = kZ ? static_cast<Tin *>(p.dz) + r.base : nullptr;
    const float *ckpt = p.ckpt_in + r.row * p.nck;
    const bool vec = p.vec, sigmoid = p.sigmoid, couple = p.couple;
    const int64_t span = (int64_t)G * kV, stride = W * span;  // (span divides kPiece: one checkpoint a span)

    Vec8<Tin> nx, ng, nz;
    Vec8<Tout> nd;
    uint32_t ncut = 0;
    float nin = 0.f;
    const auto fetch = [&](int64_t v, int64_t start) {  // the lane's steps, and where the row's lanes begin
        if (vec && v >= r.shift && v + kV <= r.steps) {
            ng.load(g, v);
            nx.load(x, v);
            nd.load(dy, v);
            if constexpr (kZ) nz.load(z, v);
            if constexpr (kR) ncut = start_bits(p.reset, bl + v, bl_all, 0, kV);
        } else {
            int lo, hi;
            bounds_of(r, v, lo, hi);
            const int64_t n = p.rows * p.L - r.base;  // elements from r.base to the tensor's end
            load_row8(ng, g, v, n, lo, hi, vec);
            load_row8(nx, x, v, n, lo, hi, vec);
            load_row8(nd, dy, v, n, lo, hi, vec);
            if constexpr (kZ) load_row8(nz, z, v, n, lo, hi, vec);
            if constexpr (kR) ncut = start_bits(p.reset, bl + v, bl_all, lo, hi);
        }
        nin = start < r.steps ? __ldg(ckpt + start / kPiece) : 0.f;
    };

    float carry = p.dlast ? p.dlast[r.row] : 0.f;
    int buf = 0;
    int64_t v0 = (r.steps - 1) / stride * stride;
    fetch(v0 + w * span + in * kV, v0 + w * span);
    for (; v0 >= 0; v0 -= stride, buf ^= 1) {
        const int64_t v = v0 + w * span + in * kV;
        const bool inner = v >= r.shift && v + kV <= r.steps;
        float2 a[kV / 2], keep[kV / 2];
        if (sigmoid) {
#pragma unroll
            for (int i = 0; i < kV / 2; ++i) gate2<Tin>(ng.pair(i), true, a[i], keep[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kV / 2; ++i) gate2<Tin>(ng.pair(i), false, a[i], keep[i]);
        }
        if (!inner) {
            int lo, hi;
            bounds_of(r, v, lo, hi);
#pragma unroll
            for (int i = 0; i < kV / 2; ++i) {
                if (2 * i < lo || 2 * i >= hi) a[i].x = 1.f, keep[i].x = 0.f;
                if (2 * i + 1 < lo || 2 * i + 1 >= hi) a[i].y = 1.f, keep[i].y = 0.f;
            }
        }
        // masked steps have inputs of zero
        float2 xv[kV / 2], b[kV / 2], dh[kV / 2], dzv[kV / 2];
#pragma unroll
        for (int i = 0; i < kV / 2; ++i) {
            xv[i] = b[i] = nx.pair(i);
            dh[i] = nd.pair(i);
            if constexpr (kZ) {
                // dy silu(z) and dy silu'(z)
                const float2 zv = nz.pair(i);
                const float2 s = sigmoid2<Tin>(zv);
                dzv[i] = mul2(dh[i], silu_slope2(zv, s));
                dh[i] = mul2(dh[i], mul2(s, zv));
            }
        }
        if (couple) {
#pragma unroll
            for (int i = 0; i < kV / 2; ++i) b[i] = mul2(keep[i], xv[i]);
        }
        const uint32_t cut = ncut;
        const float from_state = nin;
        if (v0 > 0) fetch(v - stride, v0 + w * span - stride);

        // the lane's maps of the state and of the adjoint
        float A = 1.f, B = 0.f, M = 0.f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const bool c = kR && (cut >> i & 1u);
            const float ai = i % 2 ? a[i / 2].y : a[i / 2].x, bi = i % 2 ? b[i / 2].y : b[i / 2].x;
            B = c ? bi : fmaf(ai, B, bi);
            A = c ? 0.f : A * ai;
        }
#pragma unroll
        for (int i = kV - 1; i >= 0; --i) {
            const float ai = i % 2 ? a[i / 2].y : a[i / 2].x, di = i % 2 ? dh[i / 2].y : dh[i / 2].x;
            M = kR && (cut >> i & 1u) ? 0.f : ai * (di + M);
        }
        float Am = A;
        const uint32_t cuts = kR ? __ballot_sync(0xffffffffu, cut != 0) : 0u;
        scan_up<kR, kG>(A, B, lane, lanes, cuts);
        scan_down<kR, kG>(Am, M, lane, lanes, cuts);
        const int first = lane & ~(G - 1), last = lane | (G - 1);
        const bool any = kR && (G == 32 ? cuts != 0 : (cuts & lanes_up_to(last, G == 32 ? 31 : G)) != 0);
        float Ax = __shfl_up_sync(0xffffffffu, A, 1), Bx = __shfl_up_sync(0xffffffffu, B, 1);
        if (in == 0) Ax = 1.f, Bx = 0.f;
        const float Aw = __shfl_sync(0xffffffffu, Am, first), Mw = __shfl_sync(0xffffffffu, M, first);
        float Amx = __shfl_down_sync(0xffffffffu, Am, 1), Mx = __shfl_down_sync(0xffffffffu, M, 1);
        if (lane == last) Amx = 1.f, Mx = 0.f;

        float from = carry;  // the adjoint reaching this warp's steps from behind
        if constexpr (kShare != kOwn) {
            share<kShare>(&pairs[buf][w], {Aw, Mw, any ? 1 : 0}, lane, nblk);
            float c = carry;
            for (int k = W - 1; k >= 0; --k) {
                if (k == w) from = c;
                const Pair q = pairs[buf][k];
                c = kR && q.cut ? q.B : fmaf(q.A, c, q.B);
            }
            carry = c;
        } else {
            carry = any ? Mw : fmaf(Aw, carry, Mw);
        }
        // the states, from the one before the lane's steps
        float h = kR && in > 0 && (cuts & lanes_up_to(lane - 1, in)) ? Bx : fmaf(Ax, from_state, Bx);
        float2 before[kV / 2];
#pragma unroll
        for (int i = 0; i < kV / 2; ++i) {
            float2 hv;
            before[i].x = kR && (cut >> (2 * i) & 1u) ? 0.f : h;
            hv.x = kR && (cut >> (2 * i) & 1u) ? b[i].x : fmaf(a[i].x, h, b[i].x);
            before[i].y = kR && (cut >> (2 * i + 1) & 1u) ? 0.f : hv.x;
            hv.y = kR && (cut >> (2 * i + 1) & 1u) ? b[i].y : fmaf(a[i].y, hv.x, b[i].y);
            h = hv.y;
            if constexpr (kZ) dzv[i] = mul2(dzv[i], hv);
        }
        // the adjoints, from the one behind them
        const int after = last - lane;  // the row's lanes behind this one
        float m = kR && after > 0 && (cuts & lanes_from(lane + 1, after)) ? Mx : fmaf(Amx, from, Mx);
        float ox[kV], og[kV];
        with_flags(sigmoid, couple, [&](auto sig, auto cpl) {
#pragma unroll
            for (int i = kV / 2 - 1; i >= 0; --i) {
                float2 lam;
                lam.y = dh[i].y + m;
                m = kR && (cut >> (2 * i + 1) & 1u) ? 0.f : a[i].y * lam.y;
                lam.x = dh[i].x + m;
                m = kR && (cut >> (2 * i) & 1u) ? 0.f : a[i].x * lam.x;
                float2 da = mul2(lam, cpl.value ? sub2(before[i], xv[i]) : before[i]);
                if (sig.value) da = mul2(da, mul2(a[i], keep[i]));
                if (cpl.value) lam = mul2(lam, keep[i]);
                ox[2 * i] = lam.x, ox[2 * i + 1] = lam.y, og[2 * i] = da.x, og[2 * i + 1] = da.y;
            }
        });
        if (!r.there) continue;
        float oz[kV];
        if constexpr (kZ) {
#pragma unroll
            for (int i = 0; i < kV / 2; ++i) oz[2 * i] = dzv[i].x, oz[2 * i + 1] = dzv[i].y;
        }
        if (inner && vec) {
            store_vec(dx + v, ox);
            store_vec(dg + v, og);
            if constexpr (kZ) store_vec(dz + v, oz);
        } else {
            int lo, hi;
            bounds_of(r, v, lo, hi);
            store8(dx, v, lo, hi, vec, ox);
            store8(dg, v, lo, hi, vec, og);
            if constexpr (kZ) store8(dz, v, lo, hi, vec, oz);
        }
    }
    if (p.dh0 && r.there && in == 0 && w == 0) p.dh0[r.row] = carry;
}

// One step: a thread per row, the state read and written in place.
template <typename Tin, typename Tout>
__global__ void __launch_bounds__(256) glr_step_kernel(const GlrParams p) {
    const int64_t row = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (row >= p.rows) return;
    float2 a2, keep2;
    gate2<Tin>(both(load_elem(static_cast<const Tin *>(p.g), row)), p.sigmoid, a2, keep2);
    const float a = a2.x, keep = keep2.x;
    const float xv = load_elem(static_cast<const Tin *>(p.x), row);
    const float h = fmaf(a, p.last[row], p.couple ? keep * xv : xv);
    p.last[row] = h;
    float yv = h;
    if (p.z) {
        yv *= silu2<Tin>(both(load_elem(static_cast<const Tin *>(p.z), row))).x;
    }
    put(static_cast<Tout *>(p.y), row, yv);
}

int64_t pieces(int64_t L) { return (L + kV - 1 + kPiece - 1) / kPiece; }

// How rows are dealt out: `lanes` lanes each (a power of two) where a row is
// short (256 x 1536 x 50, forward and backward: 235 us, 565 where such rows
// take warps), else whole warps, as many as bring the GPU to about kWant warps
// per SM (3 x 1000 x 4099 fp32: 40 us, 48 with 16 warps wanted, 45 with 64; 4 x
// 1024 x 100000 bf16: 463, 521, 458), no more than the row feeds with
// `per_lane` steps a lane.
struct GlrShape {
    int lanes, warps, nblk;
};
GlrShape glr_shape(int64_t rows, int64_t L, int per_lane) {
    constexpr int kWant = 32;
    const int64_t steps = L + kV - 1, want = (int64_t)layer_sm_count() * kWant;
    GlrShape s{32, 1, 1};
    if (steps <= 16 * per_lane) {  // a row's steps in one turn
        s.lanes = 4;
        while (s.lanes * per_lane < steps) s.lanes *= 2;
        return s;
    }
    while (s.warps < kMaxWarps && rows * s.warps < want && (int64_t)s.warps * 32 * per_lane < steps) s.warps *= 2;
    // Rows too few for the SMs are cut further, over a cluster of blocks, while
    // all clusters run at once (one lies within one of the eight groups of SMs,
    // which are not all of a size) and each block keeps three rounds of steps.
    // (1 x 16 x 100000 bf16 with the gate, forward: 16.5 us, 31 with a block to
    // a row; 1 x 64 x 300000: 57, 74; 1 x 4 x 200000, forward and backward: 52,
    // 125; with fewer rounds, 1 x 37 x 20000: 27, 19.)
    const int64_t sms = layer_sm_count();
    while (s.warps == kMaxWarps && s.nblk < kMaxBlocks) {
        const int64_t n = s.nblk * 2, resident = n == 2 ? sms / 2 : sms / 8 / n * 8 * 92 / 100;
        if (rows > resident || n * kMaxWarps * 32 * per_lane * 3 > steps) break;
        s.nblk = (int)n;
    }
    return s;
}

template <typename Tin, typename Tout, bool kZ, bool kR>
cudaError_t launch_glr(bool back, cudaStream_t s, const GlrParams &p) {
    const GlrShape q = glr_shape(p.rows, p.L, back ? kV : kGlrVecs<Tin> * kV);
    constexpr int kThreads = 128;
    const int64_t per = kThreads / q.lanes;
    const unsigned grid = (unsigned)(q.warps > 1 ? p.rows * q.nblk : (p.rows + per - 1) / per);
    const int threads = q.warps > 1 ? 32 * q.warps : kThreads;
    if (q.lanes < 32) {
        if (back) glr_bwd_kernel<Tin, Tout, kZ, kR, kOwn, 0><<<grid, threads, 0, s>>>(p, q.lanes, 1);
        else glr_fwd_kernel<Tin, Tout, kZ, kR, kOwn, 0><<<grid, threads, 0, s>>>(p, q.lanes, 1);
    } else if (q.warps == 1) {
        if (back) glr_bwd_kernel<Tin, Tout, kZ, kR, kOwn, 32><<<grid, threads, 0, s>>>(p, 32, 1);
        else glr_fwd_kernel<Tin, Tout, kZ, kR, kOwn, 32><<<grid, threads, 0, s>>>(p, 32, 1);
    } else if (q.nblk > 1) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3((unsigned)threads);
        cfg.stream = s;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)q.nblk;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        return back ? cudaLaunchKernelEx(&cfg, glr_bwd_kernel<Tin, Tout, kZ, kR, kCluster, 32>, p, 32, q.nblk)
                    : cudaLaunchKernelEx(&cfg, glr_fwd_kernel<Tin, Tout, kZ, kR, kCluster, 32>, p, 32, q.nblk);
    } else {
        if (back) glr_bwd_kernel<Tin, Tout, kZ, kR, kBlock, 32><<<grid, threads, 0, s>>>(p, 32, 1);
        else glr_fwd_kernel<Tin, Tout, kZ, kR, kBlock, 32><<<grid, threads, 0, s>>>(p, 32, 1);
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
