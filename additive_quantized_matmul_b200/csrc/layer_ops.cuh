// Host helpers shared by the layer operators' translation units.
#pragma once

#include "epilogue.cuh"

namespace aqh {

// Row pitch that TMA accepts (16-byte rows).
inline int padded_tokens(int T) { return (T + 7) / 8 * 8; }
inline size_t align_up(size_t v) { return (v + 127) / 128 * 128; }
inline size_t padded_bytes(int rows, int T) { return (size_t)rows * padded_tokens(T) * sizeof(uint16_t); }

// Rows of T elements from one pitch to another (the padding is left alone),
// row r multiplied by scales[r] / 2^E on the way where `scales` is given
// (see scale_exponent in epilogue.cuh).
struct RowCopy {
    const uint16_t *src;
    uint16_t *dst;
    int rows, src_pitch, dst_pitch;
    const uint16_t *scales;  // or null: a plain copy
};
constexpr int kMaxRowCopies = 3;

// Up to three arrays in one launch; E is that of the largest scale of any of
// them, and 2^E goes to *factor.
cudaError_t copy_rows(const RowCopy *jobs, int n, int T, float *factor, cudaStream_t s);

// The transposed product over one or two layers, g0 and g1 [out] rows of
// padded_tokens(T) elements, gx likewise; its plan works in the first
// back_plan_bytes of ws.  1x16 layers (back_takes_scaled) want g0 and g1
// multiplied by their layer's scales / 2^E already, and 2^E in *factor; the
// others apply the scales themselves.
inline bool back_takes_scaled(const aqk::Geom &g) { return g.K == 1 && g.B == 16; }
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
