// What stands around a quantised product in a transformer block: activation
// functions, their slopes, and the host declarations of the layer operators.
//
// All of it is evaluated in fp32 on fp32 sums; the results are rounded once,
// where they are written.  The exponential is the fast one (ex2.approx,
// relative error about 2^-22 per unit of its argument's magnitude, far below
// the binary16 results' 2^-11).
#pragma once

#include <type_traits>

#include "aq_common.cuh"

namespace aqk {

constexpr float kSqrt2OverPi = 0.7978845608028654f;
constexpr float kSqrtHalf = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// 1 / (1 + e^-v): 0 at -infinity (e^-v is infinite), 1 at infinity.
__device__ __forceinline__ float logistic(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// The tanh form of GELU is v * logistic(2 t) with this t: (1 + tanh t) / 2 =
// logistic(2 t), which loses no bits where tanh is near -1.
__device__ __forceinline__ float gelu_tanh_arg(float v) { return 2.f * kSqrt2OverPi * fmaf(0.044715f * v * v, v, v); }

__device__ __forceinline__ float act_value(int act, float v)
{
    switch (act) {
    case AQ_ACT_RELU: return v < 0.f ? 0.f : v;  // a NaN stays one
    case AQ_ACT_GELU: return v * 0.5f * erfcf(-v * kSqrtHalf);
    case AQ_ACT_GELU_TANH: return v * logistic(gelu_tanh_arg(v));
    case AQ_ACT_SILU: return v * logistic(v);
    default: return v;
    }
}

// act(v), and its derivative in `slope`.
__device__ __forceinline__ float act_value_slope(int act, float v, float &slope)
{
    switch (act) {
    case AQ_ACT_RELU: slope = v > 0.f ? 1.f : 0.f; return v < 0.f ? 0.f : v;
    case AQ_ACT_GELU: {
        const float cdf = 0.5f * erfcf(-v * kSqrtHalf);
        slope = fmaf(v * kInvSqrt2Pi, __expf(-0.5f * v * v), cdf);
        return v * cdf;
    }
    case AQ_ACT_GELU_TANH: {
        const float p = logistic(gelu_tanh_arg(v));
        slope = fmaf(2.f * v * p * (1.f - p), kSqrt2OverPi * fmaf(3.f * 0.044715f * v, v, 1.f), p);
        return v * p;
    }
    case AQ_ACT_SILU: {
        const float p = logistic(v);
        slope = fmaf(v * p, 1.f - p, p);
        return v * p;
    }
    default: slope = 1.f; return v;
    }
}

// v[i] = act(v[i]), with one branch on the activation for all of them.
template <int N>
__device__ __forceinline__ void act_values(int act, float (&v)[N])
{
    auto all = [&](auto kind) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = act_value(decltype(kind)::value, v[i]);
    };
    switch (act) {
    case AQ_ACT_RELU: all(std::integral_constant<int, AQ_ACT_RELU>{}); break;
    case AQ_ACT_GELU: all(std::integral_constant<int, AQ_ACT_GELU>{}); break;
    case AQ_ACT_GELU_TANH: all(std::integral_constant<int, AQ_ACT_GELU_TANH>{}); break;
    case AQ_ACT_SILU: all(std::integral_constant<int, AQ_ACT_SILU>{}); break;
    }
}

// v[i] = act(v[i]) and d[i] = act'(v[i]), likewise.
template <int N>
__device__ __forceinline__ void act_values_slopes(int act, float (&v)[N], float (&d)[N])
{
    auto all = [&](auto kind) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = act_value_slope(decltype(kind)::value, v[i], d[i]);
    };
    switch (act) {
    case AQ_ACT_RELU: all(std::integral_constant<int, AQ_ACT_RELU>{}); break;
    case AQ_ACT_GELU: all(std::integral_constant<int, AQ_ACT_GELU>{}); break;
    case AQ_ACT_GELU_TANH: all(std::integral_constant<int, AQ_ACT_GELU_TANH>{}); break;
    case AQ_ACT_SILU: all(std::integral_constant<int, AQ_ACT_SILU>{}); break;
    default: all(std::integral_constant<int, AQ_ACT_NONE>{}); break;
    }
}

__device__ __forceinline__ float half_bits_to_float(uint16_t h) { return __half2float(__ushort_as_half(h)); }
__device__ __forceinline__ uint16_t float_to_half_bits(float f) { return __half_as_ushort(__float2half_rn(f)); }

// One layer's stored weights on the device.
struct LayerWeights {
    const uint8_t *packed;
    const uint4 *cb;
    const uint16_t *scales;  // or null: s = 1
};

// Epilogue of a product: y = RN16(act(z + bias) + residual).
struct EpilogueArgs {
    int act;
    const uint16_t *bias;      // [out] or null
    const uint16_t *residual;  // [out][n] or null
};

}  // namespace aqk

namespace aqh {
size_t gemm_fused_workspace_bytes(const aqk::Geom &g, int T);
cudaError_t launch_gemv_fused(const aqk::Geom &g, const aqk::LayerWeights &w, const uint16_t *x, int batch,
                              const aqk::EpilogueArgs &ep, uint16_t *y, void *ws, cudaStream_t s);
cudaError_t launch_gemm_fused(const aqk::Geom &g, const aqk::LayerWeights &w, const uint16_t *x, int T,
                              const aqk::EpilogueArgs &ep, uint16_t *y, void *ws, cudaStream_t s);
size_t input_grad_workspace_bytes(const aqk::Geom &g, int T);
cudaError_t launch_input_grad(const aqk::Geom &g, const aqk::LayerWeights &w, const uint16_t *gy, int T,
                              uint16_t *gx, void *ws, cudaStream_t s);
size_t gemm_fused_grad_workspace_bytes(const aqk::Geom &g, int T);
cudaError_t launch_gemm_fused_grad(const aqk::Geom &g, const aqk::LayerWeights &w, const uint16_t *x,
                                   const uint16_t *gy, int T, const aqk::EpilogueArgs &ep, uint16_t *grad_z,
                                   float *grad_bias, uint16_t *grad_x, void *ws, cudaStream_t s);
size_t glu_gemv_workspace_bytes(const aqk::Geom &g, int batch);
size_t glu_gemm_workspace_bytes(const aqk::Geom &g, int T);
cudaError_t launch_glu_gemv(const aqk::Geom &g, const aqk::LayerWeights &gate, const aqk::LayerWeights &up,
                            const uint16_t *x, int batch, int act, uint16_t *y, void *ws, cudaStream_t s);
cudaError_t launch_glu_gemm(const aqk::Geom &g, const aqk::LayerWeights &gate, const aqk::LayerWeights &up,
                            const uint16_t *x, int T, int act, uint16_t *y, void *ws, cudaStream_t s);
size_t glu_grad_workspace_bytes(const aqk::Geom &g, int T);
cudaError_t launch_glu_grad(const aqk::Geom &g, const aqk::LayerWeights &gate, const aqk::LayerWeights &up,
                            const uint16_t *x, const uint16_t *gy, int T, int act, uint16_t *grad_gate,
                            uint16_t *grad_up, uint16_t *grad_x, void *ws, cudaStream_t s);
}  // namespace aqh
