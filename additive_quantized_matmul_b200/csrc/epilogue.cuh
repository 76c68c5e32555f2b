// What stands around a quantised product in a transformer block: activation
// functions, their slopes, and the host declarations of the layer operators.
//
// All of it is evaluated in fp32 on fp32 sums; the results are rounded once,
// where they are written.  Exponential and reciprocal are the approximate
// instructions (relative errors about 2^-22), far below the binary16
// results' 2^-11.
#pragma once

#include <type_traits>

#include "aq_common.cuh"

namespace aqk {

// Activations by family, so that an epilogue chooses its code once and not
// per element: SiLU and the tanh form of GELU are both v p with p the
// logistic function of v (k1 + k2 v^2) -- (1 + tanh t) / 2 = logistic(2 t),
// which loses no bits where tanh is near -1 -- and differ in k1, k2 alone.
constexpr int kActLinear = 0;    // none, ReLU
constexpr int kActLogistic = 1;  // SiLU, GELU (tanh)
constexpr int kActErf = 2;       // GELU

struct ActParams {
    bool relu;
    float k1, k2;
};

__host__ __device__ __forceinline__ constexpr int act_family(int act)
{
    return act == AQ_ACT_GELU ? kActErf : act >= AQ_ACT_GELU_TANH ? kActLogistic : kActLinear;
}

__device__ __forceinline__ ActParams act_params(int act)
{
    const bool tanh_form = act == AQ_ACT_GELU_TANH;  // 2 sqrt(2 / pi) (1 + 0.044715 v^2)
    return ActParams{act == AQ_ACT_RELU, tanh_form ? 1.5957691216057308f : 1.f, tanh_form ? 0.0713548162726009f : 0.f};
}

// act(v) of a family, and its derivative.
template <int F>
__device__ __forceinline__ float act_value(const ActParams &k, float v, float &slope)
{
    if constexpr (F == kActLinear) {
        slope = !k.relu || v > 0.f ? 1.f : v <= 0.f ? 0.f : v;
        return (k.relu && v < 0.f) ? 0.f : v;  // (a NaN stays one in both)
    } else if constexpr (F == kActLogistic) {
        constexpr float kLog2E = 1.4426950408889634f;
        const float v2 = fminf(v * v, 1e30f);  // finite: 0 times it stays 0 where v is infinite
        float e, p;
        // 1 / (1 + 2^(-log2(e) a)): 0 where the power is infinite
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-kLog2E * v * fmaf(k.k2, v2, k.k1)));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(1.f + e));
        const float y = v * p;
        slope = fmaf(y * (1.f - p), fmaf(3.f * k.k2, v2, k.k1), p);
        return y;
    } else {
        // Phi(v) = erfc(-v / sqrt(2)) / 2, erfc by the rational-argument
        // Chebyshev fit of "Numerical Recipes" (Press et al., section
        // "Incomplete gamma function, error function"): t exp(-x^2 + P(t)),
        // t = 1 / (1 + x / 2), x >= 0, relative error below 1.2e-7 everywhere
        // -- the tail of negative v keeps its bits
        constexpr float kLog2E = 1.4426950408889634f, kInvSqrt2Pi = 0.3989422804014327f;
        const float x = fabsf(v) * 0.7071067811865476f;
        float t, e, g;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.5f, x, 1.f)));
        float q = fmaf(t, 0.17087277f, -0.82215223f);
        q = fmaf(t, q, 1.48851587f);
        q = fmaf(t, q, -1.13520398f);
        q = fmaf(t, q, 0.27886807f);
        q = fmaf(t, q, -0.18628806f);
        q = fmaf(t, q, 0.09678418f);
        q = fmaf(t, q, 0.37409196f);
        q = fmaf(t, q, 1.00002368f);
        q = fmaf(t, q, -1.26551223f);
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(g) : "f"(-kLog2E * x * x));      // exp(-v^2 / 2)
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(kLog2E * q));
        const float tail = 0.5f * t * e * g;                                     // Phi(-|v|)
        const float cdf = v < 0.f ? tail : 1.f - tail;
        slope = fmaf(v * kInvSqrt2Pi, g, cdf);
        return v * cdf;
    }
}
template <int F>
__device__ __forceinline__ float act_value(const ActParams &k, float v)
{
    float unused;
    return act_value<F>(k, v, unused);
}

// f(std::integral_constant<int, family>) for an activation.
template <class F>
__device__ __forceinline__ void with_act_family(int act, F &&f)
{
    switch (act_family(act)) {
    case kActLinear: f(std::integral_constant<int, kActLinear>{}); break;
    case kActLogistic: f(std::integral_constant<int, kActLogistic>{}); break;
    default: f(std::integral_constant<int, kActErf>{}); break;
    }
}

// v[i] = act(v[i]).
template <int N>
__device__ __forceinline__ void act_values(int act, float (&v)[N])
{
    const ActParams k = act_params(act);
    with_act_family(act, [&](auto family) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = act_value<decltype(family)::value>(k, v[i]);
    });
}

__device__ __forceinline__ float half_bits_to_float(uint16_t h) { return __half2float(__ushort_as_half(h)); }
__device__ __forceinline__ uint16_t float_to_half_bits(float f) { return __half_as_ushort(__float2half_rn(f)); }

// Largest finite magnitude of pairs of binary16 values, per half; and the float
// it stands for in a row of scale s (0 where s is not finite: the whole row's
// products are not, whatever is made of them).
__device__ __forceinline__ void finite_absmax_h2(uint32_t &m, uint32_t w)
{
    const __half2 a = __habs2(*reinterpret_cast<const __half2 *>(&w));
    uint32_t b = *reinterpret_cast<const uint32_t *>(&a);
    b &= __hlt2_mask(a, __half2half2(__ushort_as_half(0x7c00)));  // false for infinities and NaN
    const __half2 r = __hmax2(*reinterpret_cast<const __half2 *>(&m), *reinterpret_cast<const __half2 *>(&b));
    m = *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ void finite_absmax_h8(uint32_t &m, uint4 v)
{
    finite_absmax_h2(m, v.x), finite_absmax_h2(m, v.y), finite_absmax_h2(m, v.z), finite_absmax_h2(m, v.w);
}
__device__ __forceinline__ float scaled_top(uint32_t m, float s)
{
    const float2 f = h2f2(m);
    return fabsf(s) < 65536.f ? fabsf(s) * fmaxf(f.x, f.y) : 0.f;
}

// Largest finite |v| (as the bits of a binary16) of this thread's share of
// v[0 .. n), `threads` threads in all.
__device__ __forceinline__ uint32_t finite_absmax_share(const uint16_t *__restrict__ v, int n, int thread, int threads)
{
    uint32_t m = 0;
    // 16-byte pieces between the ragged ends (v has 2-byte alignment)
    const int head = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(v) & 15)) & 15) / 2);
    const int nv = (n - head) / 8;
    const uint4 *v4 = reinterpret_cast<const uint4 *>(v + head);
#pragma unroll 8
    for (int i = thread; i < nv; i += threads) finite_absmax_h8(m, __ldg(v4 + i));
    if (thread < head) finite_absmax_h2(m, v[thread]);
    if (head + nv * 8 + thread < n && thread < 8) finite_absmax_h2(m, v[head + nv * 8 + thread]);
    return max(m & 0xffffu, m >> 16);
}

// The transposed product of layers with one or two 8-bit codebooks multiplies the
// scales into the weights, divided by 2^E: of the largest scale (bits `s`) and the
// largest entry of a codebook (bits `c`), E is the smallest for which no |W s| / 2^E
// reaches 2^15 (|W| <= K c, but for infinite weights; with c of 2^14 and more, none
// reaches 65504), nor any s / 2^E.  What is subnormal then, a scale or a weight
// times a scale, is less than 2^-14 2^E; with codebook entries up to 1/2 or 1/4
// that is 2^-29 of the largest scale.
__device__ __forceinline__ int weight_exponent(uint32_t s, uint32_t c, int K)
{
    if (s == 0) return 0;
    const int es = ilogbf(half_bits_to_float((uint16_t)s)) + 1;
    const int ec = c ? ilogbf((float)K * half_bits_to_float((uint16_t)c)) + 1 : 0;
    return es - max(0, 15 - max(ec, 0));
}

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
