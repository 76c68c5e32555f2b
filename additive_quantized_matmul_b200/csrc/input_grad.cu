// Input gradient of a quantised layer, gx = W^T (s gy), and of the gated
// block's two layers at once: the transposed product on the warp-specialised
// kernel of gemm_ws.cuh (BackOp), which takes s gy (gemm_fused.cu).
//
// A CTA takes 128 input features and 256 or 512 tokens and walks the layer's
// rows, 64 a stage: the codewords of 8 rows x 16 groups are laid along M
// (MN-major A), gy rows come by TMA.  Two layers follow one another in the
// same accumulator.
#include "gemm_ws.cuh"
#include "layer_ops.cuh"

namespace aqh {
using namespace aqk;

static GemmPlan plan_back(const Geom &g, int layers, int T)
{
    return plan_ws(ws_mtiles<BackOp>(g), layers * ws_layer_stages<BackOp>(g), T, ws_max_bn<BackOp>(g), BackOp::kPairs);
}

size_t back_plan_bytes(const Geom &g, int layers, int T) { return plan_back(g, layers, T).ws_bytes; }

cudaError_t launch_back(const Geom &g, int layers, const LayerWeights &w0, const uint16_t *g0, const LayerWeights &w1,
                        const uint16_t *g1, int T, const float *factor, uint16_t *gx, void *ws, cudaStream_t s)
{
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    TensorMaps<BackOp::kMaps> maps{};
    const BackOp op{{w0, layers > 1 ? w1 : w0}, layers, gx, factor, ws_top(ws)};
    const int pitch = padded_tokens(T);
    if (!token_map(encode, &maps.m[0], g0, g.out, T, pitch) ||
        !token_map(encode, &maps.m[1], layers > 1 ? g1 : g0, g.out, T, pitch) ||
        !io_maps(encode, &maps, op, g, T, pitch))
        return cudaErrorInvalidValue;
    return launch_ws(g, plan_back(g, layers, T), maps, op, T, ws, s, true);
}

}  // namespace aqh
