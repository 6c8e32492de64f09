// The convolution's kernels for one type pair: compiled once per
// (SS_INST_TIN, SS_INST_TOUT) with SS_INST_NAME as the launchers' suffix.
#include "ss_conv.cuh"

#if !defined(SS_INST_TIN) || !defined(SS_INST_TOUT) || !defined(SS_INST_NAME)
#error "compile with -DSS_INST_TIN=... -DSS_INST_TOUT=... -DSS_INST_NAME=..."
#endif

#define SS_CAT2(A, B) A##_##B
#define SS_CAT(A, B) SS_CAT2(A, B)

namespace selscan {
namespace {

using Tin = SS_INST_TIN;
using Tout = SS_INST_TOUT;

template <int W>
cudaError_t fwd(cudaStream_t s, ConvParams &p) {
    const int64_t spans = p.batch * p.dim * spans_of(p.L);
    p.main_blocks = (spans + 255) / 256;
    p.small = spans <= INT_MAX;
    p.by_spans = divisor_of(spans_of(p.L)), p.by_dim = divisor_of(p.dim);
    if (p.reset) {
        p.chunks = (spans_of(p.L) + 31) / 32, p.groups = (p.dim + 7) / 8;
        p.main_blocks = p.batch * p.groups * p.chunks;
    }
    const int64_t tail = p.last ? (p.batch * p.dim * (W - 1) + 255) / 256 : 0;
    if (p.main_blocks + tail > INT_MAX) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)(p.main_blocks + tail);
    if (p.reset) conv_fwd_kernel<Tin, Tout, W, true><<<grid, 256, 0, s>>>(p);
    else conv_fwd_kernel<Tin, Tout, W, false><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}

template <int W>
cudaError_t bwd(cudaStream_t s, ConvParams &p) {
    // Blocks per channel: enough for four blocks per SM, which is what runs at
    // once, no more than the channel's spans feed.  (fp32 4 x 1024 x 4096: 64
    // us, 68 with eight per SM wanted and 79 with sixteen; bf16 2 x 1024 x 20011
    // with starts 145, 169 and 198; 4 x 64 x 65536: 38 with each.)
    const int64_t vecs = p.batch * spans_of(p.L);
    p.small = vecs <= INT_MAX;
    p.by_spans = divisor_of(spans_of(p.L));
    int nblk = 1;
    while (nblk < 8 && p.dim * nblk < (int64_t)layer_sm_count() * 4 && vecs > (int64_t)nblk * kConvBwdThreads) nblk *= 2;
    const int threads = vecs < kConvBwdThreads ? (int)(vecs + 31) / 32 * 32 : kConvBwdThreads;
    p.rounds = (vecs + threads - 1) / threads;
    p.each = (p.rounds + nblk - 1) / nblk;
    if (nblk == 1) {
        if (p.reset) conv_bwd_kernel<Tin, Tout, W, true><<<(unsigned)p.dim, threads, 0, s>>>(p, nblk);
        else conv_bwd_kernel<Tin, Tout, W, false><<<(unsigned)p.dim, threads, 0, s>>>(p, nblk);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.dim * nblk));
    cfg.blockDim = dim3(kConvBwdThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)nblk;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return p.reset ? cudaLaunchKernelEx(&cfg, conv_bwd_kernel<Tin, Tout, W, true>, p, nblk)
                   : cudaLaunchKernelEx(&cfg, conv_bwd_kernel<Tin, Tout, W, false>, p, nblk);
}

}  // namespace

#define SS_WIDTHS(F)                    \
    switch (width) {                    \
        case 2: return F<2>(s, p);      \
        case 3: return F<3>(s, p);      \
        case 4: return F<4>(s, p);      \
        case 5: return F<5>(s, p);      \
        case 6: return F<6>(s, p);      \
        case 7: return F<7>(s, p);      \
        case 8: return F<8>(s, p);      \
        default: return cudaErrorInvalidValue; \
    }

cudaError_t SS_CAT(conv_fwd, SS_INST_NAME)(int width, cudaStream_t s, ConvParams &p) { SS_WIDTHS(fwd) }
cudaError_t SS_CAT(conv_bwd, SS_INST_NAME)(int width, cudaStream_t s, ConvParams &p) { SS_WIDTHS(bwd) }

}  // namespace selscan
