// Input gradient of a quantised layer, gx = W^T (s gy), and of the gated
// block's two layers at once: the transposed product on the warp-specialised
// kernel of gemm_ws.cuh (BackOp).
//
// A CTA takes 128 input features and 256 or 512 tokens and walks the layer's
// rows, 64 a stage: the codewords of 8 rows x 16 groups are laid along M
// (MN-major A), gy rows come by TMA.  Two layers follow one another in the
// same accumulator.  4096 x 4096 1x16, 512 tokens: 39 us in series, of which
// finding the largest product and scaling gy take 8, the main loop 14 (32 tiles,
// the layer's rows split over clusters of four) and the joined finish 11; 11008 x
// 4096 2x8, 2048 tokens: 173 us (1065 TFLOP/s), 2047 tokens 207.
#include "gemm_ws.cuh"
#include "layer_ops.cuh"

namespace aqh {
using namespace aqk;

using AnyBack = BackOp<true>;  // both forms have the same plan

static GemmPlan plan_back(const Geom &g, int layers, int T)
{
    return plan_ws(ws_mtiles<AnyBack>(g), layers * ws_layer_stages<AnyBack>(g), T, ws_max_bn<AnyBack>(g), AnyBack::kPairs);
}

size_t back_plan_bytes(const Geom &g, int layers, int T) { return plan_back(g, layers, T).ws_bytes; }

template <bool ScaleW>
static cudaError_t launch(const Geom &g, int layers, const LayerWeights &w0, const uint16_t *g0, const LayerWeights &w1,
                          const uint16_t *g1, int T, const float *factor, uint16_t *gx, void *ws, cudaStream_t s)
{
    using Op = BackOp<ScaleW>;
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    TensorMaps<Op::kMaps> maps{};
    const Op op{{w0, layers > 1 ? w1 : w0}, layers, gx, factor, ws_top(ws)};
    const int pitch = padded_tokens(T);
    if (!token_map(encode, &maps.m[0], g0, g.out, T, pitch) ||
        !token_map(encode, &maps.m[1], layers > 1 ? g1 : g0, g.out, T, pitch) ||
        !io_maps(encode, &maps, op, g, T, pitch))
        return cudaErrorInvalidValue;
    const GemmPlan p = plan_back(g, layers, T);
    return with_scheme(g, [&](auto sch) {
        using S = decltype(sch);
        if constexpr ((S::B == 8 && S::K <= 2) != ScaleW) return cudaErrorInvalidValue;  // see back_scales_weights
        else return launch_ws_scheme<S>(g, p, maps, op, T, ws, s, true);
    });
}

cudaError_t launch_back(const Geom &g, int layers, const LayerWeights &w0, const uint16_t *g0, const LayerWeights &w1,
                        const uint16_t *g1, int T, const float *factor, uint16_t *gx, void *ws, cudaStream_t s)
{
    return back_scales_weights(g) ? launch<true>(g, layers, w0, g0, w1, g1, T, nullptr, gx, ws, s)
                                  : launch<false>(g, layers, w0, g0, w1, g1, T, factor, gx, ws, s);
}

}  // namespace aqh
