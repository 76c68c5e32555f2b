// Prefill products with what stands around them: bias, activation and
// residual in the epilogue (aq_gemm_fused), the gated feed-forward block
// (aq_glu_gemm), and the backward passes of both (aq_gemm_fused_grad,
// aq_glu_grad), which compute the projections again and take the gradient in
// the epilogue, then multiply it back (input_grad.cu).
//
// All run on the warp-specialised kernel of gemm_ws.cuh.  TMA needs rows of
// 16-byte multiples; for T not a multiple of 8 the activations are first
// copied to rows of T rounded up to 8 in the workspace.
#include "gemm_ws.cuh"
#include "layer_ops.cuh"

namespace aqk {

// x [rows][T] -> rows of `pitch` (T rounded up to 8) elements; the elements
// past T are left alone (the tensor maps end at T).  A thread writes one
// 16-byte piece; a warp's reads cover 512 consecutive bytes.
constexpr int kPadThreads = 256;

__global__ void __launch_bounds__(kPadThreads)
pad_rows_kernel(const uint16_t *__restrict__ x, int rows, int T, int pitch, uint16_t *__restrict__ out)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int per_row = pitch / 8;
    const size_t n = (size_t)rows * per_row;
    for (size_t i = (size_t)blockIdx.x * kPadThreads + threadIdx.x; i < n; i += (size_t)gridDim.x * kPadThreads) {
        const size_t r = i / per_row;
        const int c = (int)(i - r * per_row) * 8;
        const uint16_t *src = x + r * T + c;
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = c + j < T ? (uint32_t)__ldg(src + j) : 0u;
        *reinterpret_cast<uint4 *>(out + r * pitch + c) =
            make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
    }
}

// grad_bias[o] = sums[0][o] + sums[1][o] + ..., in that order within each of
// eight interleaved parts, the parts then in order: 32 rows per CTA, one
// warp per part.
__global__ void __launch_bounds__(256) bias_grad_kernel(const float *__restrict__ sums, int blocks, int out,
                                                        float *__restrict__ grad_bias)
{
    __shared__ float part[8][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, p = threadIdx.x >> 5, o = blockIdx.x * 32 + lane;
    float a = 0.f;
    if (o < out) {
#pragma unroll 4
        for (int b = p; b < blocks; b += 8) a += __ldcg(sums + (size_t)b * out + o);
    }
    part[p][lane] = a;
    __syncthreads();
    if (p == 0 && o < out) {
#pragma unroll
        for (int i = 1; i < 8; ++i) a += part[i][lane];
        grad_bias[o] = a;
    }
}

}  // namespace aqk

namespace aqh {
using namespace aqk;

cudaError_t pad_rows(const uint16_t *x, int rows, int T, uint16_t *out, cudaStream_t s)
{
    const int pitch = padded_tokens(T);
    const size_t pieces = (size_t)rows * (pitch / 8);
    const unsigned grid = (unsigned)std::min<size_t>((pieces + kPadThreads - 1) / kPadThreads, 16 * kNumSMs);
    return launch_programmatic(pad_rows_kernel, dim3(grid), dim3(kPadThreads), s, x, rows, T, pitch, out);
}

namespace {

// Workspace of a product: the plan's, then (T ragged) the padded input.
struct Layout {
    GemmPlan p;
    size_t x_pad;   // offset of the padded input
    size_t end;
};

template <class Op>
Layout layout_of(const Geom &g, int T)
{
    Layout l;
    l.p = plan_ws(ws_mtiles<Op>(g), ws_layer_stages<Op>(g), T, ws_max_bn<Op>(g), Op::kPairs);
    l.x_pad = align_up(l.p.ws_bytes);
    l.end = T % 8 ? l.x_pad + padded_bytes(g.in, T) : l.p.ws_bytes;
    return l;
}

// Pads x where T asks for it and launches the product.
template <class Op>
cudaError_t product(const Geom &g, const Layout &l, const uint16_t *x, int T, const Op &op, char *ws, cudaStream_t s)
{
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    if (T % 8) {
        uint16_t *xp = reinterpret_cast<uint16_t *>(ws + l.x_pad);
        const cudaError_t e = pad_rows(x, g.in, T, xp, s);
        if (e != cudaSuccess) return e;
        x = xp;
    }
    TensorMaps<Op::kMaps> maps{};
    if (!token_map(encode, &maps.m[0], x, g.in, T, padded_tokens(T)) || !io_maps(encode, &maps, op, g, T))
        return cudaErrorInvalidValue;
    return launch_ws(g, l.p, maps, op, T, ws, s, true);
}

// The backward passes: the product's part (later the transposed product's
// plan works there: it follows the product on the stream), then the sums of
// the bias gradient and the padded copies of the gradients.
struct GradLayout {
    Layout l;
    size_t sums, pad0, pad1, end;
};

template <class Op>
GradLayout grad_layout(const Geom &g, int T)
{
    constexpr bool kBias = !Op::kGated;
    const size_t pad = T % 8 ? align_up(padded_bytes(g.out, T)) : 0;
    GradLayout r;
    r.l = layout_of<Op>(g, T);
    r.sums = align_up(std::max(r.l.end, back_plan_bytes(g, Op::kLayers, T)));
    r.pad0 = r.sums + (kBias ? align_up((size_t)((T + 15) / 16) * g.out * sizeof(float)) : 0);
    r.pad1 = r.pad0 + pad;
    r.end = r.pad1 + (Op::kLayers > 1 ? pad : 0);
    return r;
}

}  // namespace

size_t gemm_fused_workspace_bytes(const Geom &g, int T) { return layout_of<FusedOp>(g, T).end; }

cudaError_t launch_gemm_fused(const Geom &g, const LayerWeights &w, const uint16_t *x, int T, const EpilogueArgs &ep,
                              uint16_t *y, void *ws, cudaStream_t s)
{
    const FusedOp op{{w}, ep.act, ep.bias, ep.residual, y, false, nullptr, nullptr};
    return product(g, layout_of<FusedOp>(g, T), x, T, op, reinterpret_cast<char *>(ws), s);
}

size_t glu_gemm_workspace_bytes(const Geom &g, int T) { return layout_of<GatedOp>(g, T).end; }

cudaError_t launch_glu_gemm(const Geom &g, const LayerWeights &gate, const LayerWeights &up, const uint16_t *x, int T,
                            int act, uint16_t *y, void *ws, cudaStream_t s)
{
    const GatedOp op{{gate, up}, act, nullptr, y, nullptr, nullptr, nullptr};
    return product(g, layout_of<GatedOp>(g, T), x, T, op, reinterpret_cast<char *>(ws), s);
}

size_t gemm_fused_grad_workspace_bytes(const Geom &g, int T)
{
    return grad_layout<FusedOp>(g, T).end;
}

cudaError_t launch_gemm_fused_grad(const Geom &g, const LayerWeights &w, const uint16_t *x, const uint16_t *gy, int T,
                                   const EpilogueArgs &ep, uint16_t *grad_z, float *grad_bias, uint16_t *grad_x,
                                   void *ws, cudaStream_t s)
{
    const GradLayout r = grad_layout<FusedOp>(g, T);
    char *base = reinterpret_cast<char *>(ws);
    float *sums = grad_bias ? reinterpret_cast<float *>(base + r.sums) : nullptr;
    uint16_t *pad = (T % 8 && grad_x) ? reinterpret_cast<uint16_t *>(base + r.pad0) : nullptr;
    const FusedOp op{{w}, ep.act, ep.bias, gy, grad_z, true, pad, sums};
    cudaError_t e = product(g, r.l, x, T, op, base, s);
    if (e == cudaSuccess && grad_bias)
        e = launch_programmatic(bias_grad_kernel, dim3((g.out + 31) / 32), dim3(256), s, (const float *)sums,
                                (T + 15) / 16, g.out, grad_bias);
    if (e != cudaSuccess || !grad_x) return e;
    return launch_back(g, 1, w, pad ? pad : grad_z, w, nullptr, T, grad_x, ws, s);
}

size_t glu_grad_workspace_bytes(const Geom &g, int T)
{
    return grad_layout<GatedOp>(g, T).end;
}

cudaError_t launch_glu_grad(const Geom &g, const LayerWeights &gate, const LayerWeights &up, const uint16_t *x,
                            const uint16_t *gy, int T, int act, uint16_t *grad_gate, uint16_t *grad_up,
                            uint16_t *grad_x, void *ws, cudaStream_t s)
{
    const GradLayout r = grad_layout<GatedOp>(g, T);
    char *base = reinterpret_cast<char *>(ws);
    const bool pad = T % 8 && grad_x;
    uint16_t *p0 = pad ? reinterpret_cast<uint16_t *>(base + r.pad0) : nullptr;
    uint16_t *p1 = pad ? reinterpret_cast<uint16_t *>(base + r.pad1) : nullptr;
    const GatedOp op{{gate, up}, act, gy, grad_gate, grad_up, p0, p1};
    const cudaError_t e = product(g, r.l, x, T, op, base, s);
    if (e != cudaSuccess || !grad_x) return e;
    return launch_back(g, 2, gate, pad ? p0 : grad_gate, up, pad ? p1 : grad_up, T, grad_x, ws, s);
}

}  // namespace aqh
