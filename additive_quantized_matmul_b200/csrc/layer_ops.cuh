// Host helpers shared by the layer operators' translation units.
#pragma once

#include "epilogue.cuh"

namespace aqh {

// Row pitch that TMA accepts (16-byte rows).
inline int padded_tokens(int T) { return (T + 7) / 8 * 8; }
inline size_t align_up(size_t v) { return (v + 127) / 128 * 128; }
inline size_t padded_bytes(int rows, int T) { return (size_t)rows * padded_tokens(T) * sizeof(uint16_t); }

// Rows of T elements from one pitch to another (the padding is left alone).
struct RowCopy {
    const uint16_t *src;
    uint16_t *dst;
    int rows, src_pitch, dst_pitch;
    const uint16_t *scales;  // or null: 1
};
constexpr int kMaxRowCopies = 3;

// Up to three arrays in one launch.
cudaError_t copy_rows(const RowCopy *jobs, int n, int T, cudaStream_t s);

// The same with row r multiplied by scales[r] / 2^E on the way, for arrays of
// the same number of rows, E the same for all of them: the largest finite
// |scales[r] src[r][t]|, divided by 2^E, is 2^14 to 2^15.  2^E goes to *factor.
// The largest stands in *top already (`known`), or a launch finds it first
// (*top zero before).
cudaError_t scale_rows(const RowCopy *jobs, int n, int T, float *factor, unsigned *top, bool known, cudaStream_t s);

// The transposed product over one or two layers, gx = sum of W^T g, g0 and g1
// [out] rows of padded_tokens(T) elements, gx likewise.  Layers with one or two
// 8-bit codebooks have their scales multiplied into the weights; the others'
// are in g already: with `factor`, the result is multiplied by *factor, and the
// workspace's ws_top is cleared.  Its plan works in the first back_plan_bytes of
// ws.
inline bool back_scales_weights(const aqk::Geom &g) { return g.B == 8 && g.K <= 2; }
size_t back_plan_bytes(const aqk::Geom &g, int layers, int T);
cudaError_t launch_back(const aqk::Geom &g, int layers, const aqk::LayerWeights &w0, const uint16_t *g0,
                        const aqk::LayerWeights &w1, const uint16_t *g1, int T, const float *factor, uint16_t *gx,
                        void *ws, cudaStream_t s);

// Launch with programmatic stream serialisation: the kernel waits
// (griddepcontrol.wait) before it touches memory that others write.
template <class... KArgs, class... Args>
cudaError_t launch_programmatic(void (*kern)(KArgs...), dim3 grid, dim3 block, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace aqh
