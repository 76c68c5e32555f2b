// Decode-time products with what stands around them: bias, activation and
// residual (aq_gemv_fused), and the gated feed-forward block (aq_glu_gemv).
//
// The kernels and plans are aq_gemv's with another output.  A gated block is
// planned as one layer of twice the rows: its two projections' CTAs fill the
// GPU in one launch and meet in the split-K finish.
//
// The bound is aq_gemv's: random codeword reads (1x16) or shared-memory
// wavefronts (8-bit codebooks), then the fixed cost of the split's finish.
// Inside a graph of cold layers, beside the plain product: 4096 x 4096 1x16 at
// one token with residual 11.5 us (plain 11.5), 4096 x 11008 2x8 at eight 14.0
// (13.8); gated 11008 x 4096: 2x8 at one token 13.7 us, at eight 33.6, 1x16 at
// one 45.2, at sixteen 63.1 (the codeword reads alone take 40).
#include "gemv_plan.cuh"

namespace aqh {
using namespace aqk;

cudaError_t launch_gemv_fused(const Geom &g, const LayerWeights &w, const uint16_t *x, int batch,
                              const EpilogueArgs &ep, uint16_t *y, void *ws, cudaStream_t s)
{
    const GemvPlan p = plan_gemv(g, batch);
    if (ep.act == AQ_ACT_NONE) return launch_plan(g, p, GemvFusedOut<false>{{w}, y, ep}, x, batch, ws, s, true);
    return launch_plan(g, p, GemvFusedOut<true>{{w}, y, ep}, x, batch, ws, s, true);
}

static GemvPlan plan_glu(const Geom &g, int batch) { return plan_gemv(g, batch, ~(size_t)0, 2); }

size_t glu_gemv_workspace_bytes(const Geom &g, int batch) { return plan_glu(g, batch).ws_bytes; }

cudaError_t launch_glu_gemv(const Geom &g, const LayerWeights &gate, const LayerWeights &up, const uint16_t *x,
                            int batch, int act, uint16_t *y, void *ws, cudaStream_t s)
{
    return launch_plan(g, plan_glu(g, batch), GemvGatedOut{{gate, up}, y, act}, x, batch, ws, s, true);
}

}  // namespace aqh
