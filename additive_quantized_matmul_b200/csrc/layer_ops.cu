// Layer operators around the quantised product, in their simplest form: fp32
// sums on the CUDA cores, one thread per output token (see include/aq.h for
// what each computes).
//
// A CTA decodes a strip of one layer's rows into shared memory (each weight
// group the sum of its K codewords, rounded once to binary16) and its
// threads, one per token, multiply it with the activations.  The strip is
// read by 128 tokens; nothing is staged ahead, so the kernels are bound by
// the latency of their own loads.
#include <algorithm>

#include "epilogue.cuh"
#include "scheme.cuh"

namespace aqk {

constexpr int kSimpleTokens = 128;   // tokens (threads) per CTA
constexpr int kSimpleChunk = 128;    // groups (product) or rows (transposed) decoded at a time

// The weights of group g of row o.
template <class S>
__device__ __forceinline__ uint4 decode_group(const Geom &L, const LayerWeights &w, int o, int g)
{
    const Chunk<S> c = load_chunk<S>(w.packed, (size_t)(o >> 3) * L.gp + g, true);
    uint4 t[S::K];
    uint32_t code[S::K];
#pragma unroll
    for (int r = 0; r < 8; ++r)
        if (r == (o & 7)) {
#pragma unroll
            for (int k = 0; k < S::K; ++k) code[k] = c.code(r, k);
        }
#pragma unroll
    for (int k = 0; k < S::K; ++k) t[k] = ldg_nc_v4(w.cb + ((size_t)k << S::B) + code[k]);
    return sum_round_exact_h8<S::K>(t);
}

// sum_i W[o][i] x[i][t] of row o, this thread's token t.
template <class S>
__device__ float simple_row(const Geom &L, const LayerWeights &w, int o, const uint16_t *__restrict__ x, int T, int t,
                            uint4 *strip)
{
    float acc = 0.f;
    for (int g0 = 0; g0 < L.G; g0 += kSimpleChunk) {
        const int ng = min(kSimpleChunk, L.G - g0);
        __syncthreads();
        for (int i = threadIdx.x; i < ng; i += blockDim.x) strip[i] = decode_group<S>(L, w, o, g0 + i);
        __syncthreads();
        if (t < T)
            for (int i = 0; i < ng; ++i) {
                const uint4 v = strip[i];
                const uint16_t *xp = x + (size_t)(g0 + i) * 8 * T + t;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const float2 f = h2f2(u4_at(v, h));
                    acc = fmaf(f.x, half_bits_to_float(xp[(size_t)(2 * h) * T]), acc);
                    acc = fmaf(f.y, half_bits_to_float(xp[(size_t)(2 * h + 1) * T]), acc);
                }
            }
    }
    return acc * (w.scales ? half_bits_to_float(w.scales[o]) : 1.f);
}

// y = act(z) + residual; with gy: grad_z = gy act'(z), and its sum over tokens
template <class S>
__global__ void simple_fused_kernel(Geom L, LayerWeights w, const uint16_t *x, int T, EpilogueArgs ep,
                                    uint16_t *y, const uint16_t *gy, uint16_t *grad_z, float *grad_bias)
{
    __shared__ uint4 strip[kSimpleChunk];
    __shared__ float s_sum[kSimpleTokens];
    const int o = blockIdx.x;
    float sum = 0.f;
    for (int t0 = blockIdx.y * kSimpleTokens; t0 < T; t0 += gridDim.y * kSimpleTokens) {
        const int t = t0 + threadIdx.x;
        const float v = simple_row<S>(L, w, o, x, T, t, strip) + (ep.bias ? half_bits_to_float(ep.bias[o]) : 0.f);
        if (t >= T) continue;
        const size_t at = (size_t)o * T + t;
        if (!gy) {
            y[at] = float_to_half_bits(act_value(ep.act, v) + (ep.residual ? half_bits_to_float(ep.residual[at]) : 0.f));
        } else {
            float slope;
            act_value_slope(ep.act, v, slope);
            const float gz = half_bits_to_float(gy[at]) * slope;
            grad_z[at] = float_to_half_bits(gz);
            sum += gz;
        }
    }
    if (grad_bias) {
        s_sum[threadIdx.x] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kSimpleTokens; ++i) sum += s_sum[i];
            grad_bias[o] = sum;
        }
    }
}

// y = act(g) u; with gy: the gradients of g and u
template <class S>
__global__ void simple_glu_kernel(Geom L, LayerWeights gate, LayerWeights up, const uint16_t *x, int T, int act,
                                  uint16_t *y, const uint16_t *gy, uint16_t *grad_gate, uint16_t *grad_up)
{
    __shared__ uint4 strip[kSimpleChunk];
    const int o = blockIdx.x, t = blockIdx.y * kSimpleTokens + threadIdx.x;
    const float g = simple_row<S>(L, gate, o, x, T, t, strip), u = simple_row<S>(L, up, o, x, T, t, strip);
    if (t >= T) return;
    const size_t at = (size_t)o * T + t;
    float slope;
    const float a = act_value_slope(act, g, slope);
    if (!gy) {
        y[at] = float_to_half_bits(a * u);
    } else {
        const float d = half_bits_to_float(gy[at]);
        grad_gate[at] = float_to_half_bits(d * u * slope);
        grad_up[at] = float_to_half_bits(d * a);
    }
}

// gx = W^T (s gy) of one group of 8 features, over one or two layers
template <class S>
__global__ void simple_input_grad_kernel(Geom L, LayerWeights w0, const uint16_t *gy0, LayerWeights w1,
                                         const uint16_t *gy1, int T, uint16_t *gx)
{
    __shared__ uint4 strip[kSimpleChunk];
    __shared__ float s_sc[kSimpleChunk];
    const int g = blockIdx.x, t = blockIdx.y * kSimpleTokens + threadIdx.x;
    float acc[8] = {};
    for (int src = 0; src < (gy1 ? 2 : 1); ++src) {
        const LayerWeights w = src ? w1 : w0;
        const uint16_t *gy = src ? gy1 : gy0;
        for (int o0 = 0; o0 < L.out; o0 += kSimpleChunk) {
            const int no = min(kSimpleChunk, L.out - o0);
            __syncthreads();
            for (int i = threadIdx.x; i < no; i += blockDim.x) {
                strip[i] = decode_group<S>(L, w, o0 + i, g);
                s_sc[i] = w.scales ? half_bits_to_float(w.scales[o0 + i]) : 1.f;
            }
            __syncthreads();
            if (t < T)
                for (int i = 0; i < no; ++i) {
                    const uint4 v = strip[i];
                    const float d = s_sc[i] * half_bits_to_float(gy[(size_t)(o0 + i) * T + t]);
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const float2 f = h2f2(u4_at(v, h));
                        acc[2 * h] = fmaf(f.x, d, acc[2 * h]);
                        acc[2 * h + 1] = fmaf(f.y, d, acc[2 * h + 1]);
                    }
                }
        }
    }
    if (t >= T) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) gx[(size_t)(8 * g + j) * T + t] = float_to_half_bits(acc[j]);
}

}  // namespace aqk

namespace aqh {
using namespace aqk;

size_t gemm_fused_workspace_bytes(const Geom &, int) { return kWsHeader; }
size_t input_grad_workspace_bytes(const Geom &, int) { return kWsHeader; }
size_t gemm_fused_grad_workspace_bytes(const Geom &, int) { return kWsHeader; }
size_t glu_gemv_workspace_bytes(const Geom &, int) { return kWsHeader; }
size_t glu_gemm_workspace_bytes(const Geom &, int) { return kWsHeader; }
size_t glu_grad_workspace_bytes(const Geom &, int) { return kWsHeader; }

static dim3 simple_grid(int rows, int T) { return dim3(rows, std::min(65535, (T + kSimpleTokens - 1) / kSimpleTokens)); }

static cudaError_t simple_fused(const Geom &g, const LayerWeights &w, const uint16_t *x, int T, const EpilogueArgs &ep,
                                uint16_t *y, const uint16_t *gy, uint16_t *grad_z, float *grad_bias, cudaStream_t s)
{
    dim3 grid = simple_grid(g.out, T);
    if (grad_bias) grid.y = 1;
    return with_scheme(g, [&](auto sch) {
        simple_fused_kernel<decltype(sch)><<<grid, kSimpleTokens, 0, s>>>(g, w, x, T, ep, y, gy, grad_z, grad_bias);
        return cudaGetLastError();
    });
}

cudaError_t launch_gemv_fused(const Geom &g, const LayerWeights &w, const uint16_t *x, int batch,
                              const EpilogueArgs &ep, uint16_t *y, void *, cudaStream_t s)
{
    return simple_fused(g, w, x, batch, ep, y, nullptr, nullptr, nullptr, s);
}

cudaError_t launch_gemm_fused(const Geom &g, const LayerWeights &w, const uint16_t *x, int T, const EpilogueArgs &ep,
                              uint16_t *y, void *, cudaStream_t s)
{
    return simple_fused(g, w, x, T, ep, y, nullptr, nullptr, nullptr, s);
}

static cudaError_t simple_input_grad(const Geom &g, const LayerWeights &w0, const uint16_t *gy0,
                                     const LayerWeights &w1, const uint16_t *gy1, int T, uint16_t *gx, cudaStream_t s)
{
    return with_scheme(g, [&](auto sch) {
        simple_input_grad_kernel<decltype(sch)><<<simple_grid(g.G, T), kSimpleTokens, 0, s>>>(g, w0, gy0, w1, gy1, T, gx);
        return cudaGetLastError();
    });
}

cudaError_t launch_input_grad(const Geom &g, const LayerWeights &w, const uint16_t *gy, int T, uint16_t *gx, void *,
                              cudaStream_t s)
{
    return simple_input_grad(g, w, gy, w, nullptr, T, gx, s);
}

cudaError_t launch_gemm_fused_grad(const Geom &g, const LayerWeights &w, const uint16_t *x, const uint16_t *gy, int T,
                                   const EpilogueArgs &ep, uint16_t *grad_z, float *grad_bias, uint16_t *grad_x,
                                   void *, cudaStream_t s)
{
    cudaError_t e = simple_fused(g, w, x, T, ep, nullptr, gy, grad_z, grad_bias, s);
    if (e != cudaSuccess || !grad_x) return e;
    return simple_input_grad(g, w, grad_z, w, nullptr, T, grad_x, s);
}

static cudaError_t simple_glu(const Geom &g, const LayerWeights &gate, const LayerWeights &up, const uint16_t *x,
                              int T, int act, uint16_t *y, const uint16_t *gy, uint16_t *gg, uint16_t *gu,
                              cudaStream_t s)
{
    return with_scheme(g, [&](auto sch) {
        simple_glu_kernel<decltype(sch)><<<simple_grid(g.out, T), kSimpleTokens, 0, s>>>(g, gate, up, x, T, act, y, gy, gg, gu);
        return cudaGetLastError();
    });
}

cudaError_t launch_glu_gemv(const Geom &g, const LayerWeights &gate, const LayerWeights &up, const uint16_t *x,
                            int batch, int act, uint16_t *y, void *, cudaStream_t s)
{
    return simple_glu(g, gate, up, x, batch, act, y, nullptr, nullptr, nullptr, s);
}

cudaError_t launch_glu_gemm(const Geom &g, const LayerWeights &gate, const LayerWeights &up, const uint16_t *x, int T,
                            int act, uint16_t *y, void *, cudaStream_t s)
{
    return simple_glu(g, gate, up, x, T, act, y, nullptr, nullptr, nullptr, s);
}

cudaError_t launch_glu_grad(const Geom &g, const LayerWeights &gate, const LayerWeights &up, const uint16_t *x,
                            const uint16_t *gy, int T, int act, uint16_t *grad_gate, uint16_t *grad_up,
                            uint16_t *grad_x, void *, cudaStream_t s)
{
    cudaError_t e = simple_glu(g, gate, up, x, T, act, nullptr, gy, grad_gate, grad_up, s);
    if (e != cudaSuccess || !grad_x) return e;
    return simple_input_grad(g, gate, grad_gate, up, grad_up, T, grad_x, s);
}

}  // namespace aqh
