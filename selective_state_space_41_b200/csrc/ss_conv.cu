// C entries of the causal depthwise convolution (include/selscan.h) and its
// decoding step; the other kernels are in ss_conv.cuh.
#include "ss_conv.cuh"

namespace selscan {
namespace {

// One step: a thread per row.  The W - 1 kept inputs move up by one place and
// the new one takes the last.
template <typename Tin, typename Tout>
__global__ void __launch_bounds__(128) conv_step_kernel(const ConvParams p) {
    const int64_t row = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (row >= p.batch * p.dim) return;
    const int W = p.width;
    const int64_t d = row % p.dim;
    Tin *state = static_cast<Tin *>(p.last) + row * (W - 1);
    const float *w = p.weight + d * W;
    float v[kMaxWidth - 1], wv[kMaxWidth];
#pragma unroll
    for (int j = 0; j < kMaxWidth - 1; ++j) v[j] = static_cast<float>(state[min(j, W - 2)]);  // all in flight at once
#pragma unroll
    for (int j = 0; j < kMaxWidth; ++j) wv[j] = __ldg(w + min(j, W - 1));
    const float xv = load_elem(static_cast<const Tin *>(p.x), row);
    float acc = p.bias ? __ldg(p.bias + d) : 0.f;
#pragma unroll
    for (int j = 0; j < kMaxWidth - 1; ++j) {
        if (j >= W - 1) break;
        acc = fmaf(wv[j], v[j], acc);
        if (j > 0) put(state, j - 1, v[j]);
    }
#pragma unroll
    for (int j = 1; j < kMaxWidth; ++j)
        if (j == W - 1) acc = fmaf(wv[j], xv, acc);
    put(state, W - 2, xv);
    put(static_cast<Tout *>(p.y), row, p.silu ? silu2<Tin>(both(acc)).x : acc);
}

template <typename Tin, typename Tout>
cudaError_t launch_conv_step(cudaStream_t s, const ConvParams &p) {
    conv_step_kernel<Tin, Tout><<<(unsigned)((p.batch * p.dim + 127) / 128), 128, 0, s>>>(p);
    return cudaGetLastError();
}

// What the three entries check alike.
ss_status check_conv(const ss_desc *desc, int width, LayerSizes *sz) {
    const ss_status st = check_layer(desc, sz);
    if (st != SS_OK) return st;
    if (width < kMinWidth || width > kMaxWidth || sz->rows > INT_MAX / kMaxWidth) return SS_ERR_BAD_SHAPE;
    return SS_OK;
}

}  // namespace
}  // namespace selscan

using namespace selscan;

extern "C" {

ss_status ss_conv_fwd(const ss_desc *desc, int width, const void *x, const float *weight, const float *bias, int silu,
                      const void *initial_state, const uint8_t *reset, void *y, void *last_state, ss_stream_t stream) {
    LayerSizes sz;
    const ss_status st = check_conv(desc, width, &sz);
    if (st != SS_OK) return st;
    if (sz.rows == 0) return SS_OK;
    const size_t ein = layer_size(desc->in_dtype), eout = layer_size(desc->out_dtype);
    if (!layer_aligned(initial_state, ein) || !layer_aligned(last_state, ein)) return SS_ERR_MISALIGNED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (desc->seqlen == 0) {
        if (!last_state || last_state == initial_state) return SS_OK;
        const size_t n = (size_t)sz.rows * (size_t)(width - 1) * ein;
        return status_of(initial_state ? cudaMemcpyAsync(last_state, initial_state, n, cudaMemcpyDeviceToDevice, s)
                                       : cudaMemsetAsync(last_state, 0, n, s));
    }
    if (!x || !weight || !y) return SS_ERR_NULL_POINTER;
    if (y == x || (last_state && last_state == initial_state)) return SS_ERR_OVERLAP;
    if (!layer_aligned(x, ein) || !layer_aligned(y, eout) || !layer_aligned(weight, 4) || !layer_aligned(bias, 4))
        return SS_ERR_MISALIGNED;
    ConvParams p{};
    p.x = x, p.weight = weight, p.bias = bias, p.h0 = initial_state, p.reset = reset, p.y = y, p.last = last_state;
    p.batch = desc->batch, p.dim = desc->dim, p.L = desc->seqlen;
    p.silu = silu != 0, p.vec = vec_ok({x, y});
    const auto launch = desc->in_dtype == SS_F32    ? conv_fwd_f32_f32
                        : desc->out_dtype == SS_F32 ? conv_fwd_bf16_f32
                                                    : conv_fwd_bf16_bf16;
    return status_of(launch(width, s, p));
}

ss_status ss_conv_bwd(const ss_desc *desc, int width, const void *x, const float *weight, const float *bias, int silu,
                      const void *initial_state, const uint8_t *reset, const void *dy, const void *d_last_state,
                      void *dx, float *dweight, float *dbias, void *d_initial_state, ss_stream_t stream) {
    LayerSizes sz;
    const ss_status st = check_conv(desc, width, &sz);
    if (st != SS_OK) return st;
    const size_t ein = layer_size(desc->in_dtype), eout = layer_size(desc->out_dtype);
    if (!layer_aligned(initial_state, ein) || !layer_aligned(d_last_state, ein) || !layer_aligned(d_initial_state, ein) ||
        !layer_aligned(dweight, 4) || !layer_aligned(dbias, 4))
        return SS_ERR_MISALIGNED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (sz.elems == 0) {  // no steps: the sums are zero, the state passes through
        const size_t n = (size_t)sz.rows * (size_t)(width - 1) * ein, d = (size_t)desc->dim * 4;
        cudaError_t e = cudaSuccess;
        if (d_initial_state && n && d_initial_state != d_last_state)
            e = d_last_state ? cudaMemcpyAsync(d_initial_state, d_last_state, n, cudaMemcpyDeviceToDevice, s)
                             : cudaMemsetAsync(d_initial_state, 0, n, s);
        if (e == cudaSuccess && dweight && d) e = cudaMemsetAsync(dweight, 0, d * (size_t)width, s);
        if (e == cudaSuccess && dbias && d) e = cudaMemsetAsync(dbias, 0, d, s);
        return status_of(e);
    }
    if (!x || !weight || !dy || !dx) return SS_ERR_NULL_POINTER;
    if (dx == x || dx == dy || (d_initial_state && d_initial_state == d_last_state)) return SS_ERR_OVERLAP;
    if (!layer_aligned(x, ein) || !layer_aligned(dx, ein) || !layer_aligned(dy, eout) || !layer_aligned(weight, 4) ||
        !layer_aligned(bias, 4))
        return SS_ERR_MISALIGNED;
    ConvParams p{};
    p.x = x, p.weight = weight, p.bias = bias, p.h0 = initial_state, p.reset = reset, p.dy = dy, p.dlast = d_last_state;
    p.dx = dx, p.dweight = dweight, p.dbias = dbias, p.dh0 = d_initial_state;
    p.batch = desc->batch, p.dim = desc->dim, p.L = desc->seqlen;
    p.silu = silu != 0, p.vec = vec_ok({x, dy, dx});
    const auto launch = desc->in_dtype == SS_F32    ? conv_bwd_f32_f32
                        : desc->out_dtype == SS_F32 ? conv_bwd_bf16_f32
                                                    : conv_bwd_bf16_bf16;
    return status_of(launch(width, s, p));
}

ss_status ss_conv_step(const ss_desc *desc, int width, const void *x, const float *weight, const float *bias, int silu,
                       void *state, void *y, ss_stream_t stream) {
    LayerSizes sz;
    const ss_status st = check_conv(desc, width, &sz);
    if (st != SS_OK) return st;
    if (desc->seqlen != 1) return SS_ERR_BAD_SHAPE;
    if (sz.rows == 0) return SS_OK;
    if (!x || !weight || !state || !y) return SS_ERR_NULL_POINTER;
    const size_t ein = layer_size(desc->in_dtype), eout = layer_size(desc->out_dtype);
    if (!layer_aligned(x, ein) || !layer_aligned(state, ein) || !layer_aligned(y, eout) || !layer_aligned(weight, 4) ||
        !layer_aligned(bias, 4))
        return SS_ERR_MISALIGNED;
    ConvParams p{};
    p.x = x, p.weight = weight, p.bias = bias, p.last = state, p.y = y;
    p.batch = desc->batch, p.dim = desc->dim, p.L = 1;
    p.silu = silu != 0, p.width = width;
    return status_of(SS_LAYER_DISPATCH(desc, launch_conv_step)(reinterpret_cast<cudaStream_t>(stream), p));
}

}  // extern "C"
