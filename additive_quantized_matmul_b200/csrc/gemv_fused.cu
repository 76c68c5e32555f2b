// Decode-time products with what stands around them: bias, activation and
// residual (aq_gemv_fused), and the gated feed-forward block (aq_glu_gemv).
//
// The kernels and plans are aq_gemv's with another output.  A gated block is
// planned as one layer of twice the rows: its two projections' CTAs fill the
// GPU in one launch and meet in the split-K finish.
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
