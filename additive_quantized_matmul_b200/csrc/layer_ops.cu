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

template <class S>
__global__ void simple_fused_kernel(Geom L, LayerWeights w, const uint16_t *x, int T, EpilogueArgs ep, uint16_t *y)
{
    __shared__ uint4 strip[kSimpleChunk];
    const int o = blockIdx.x, t = threadIdx.x;
    const float v = simple_row<S>(L, w, o, x, T, t, strip) + (ep.bias ? half_bits_to_float(ep.bias[o]) : 0.f);
    if (t >= T) return;
    const size_t at = (size_t)o * T + t;
    y[at] = float_to_half_bits(act_value(ep.act, v) + (ep.residual ? half_bits_to_float(ep.residual[at]) : 0.f));
}

template <class S>
__global__ void simple_glu_kernel(Geom L, LayerWeights gate, LayerWeights up, const uint16_t *x, int T, int act,
                                  uint16_t *y)
{
    __shared__ uint4 strip[kSimpleChunk];
    const int o = blockIdx.x, t = threadIdx.x;
    const float g = simple_row<S>(L, gate, o, x, T, t, strip), u = simple_row<S>(L, up, o, x, T, t, strip);
    if (t >= T) return;
    y[(size_t)o * T + t] = float_to_half_bits(act_value(act, g) * u);
}

}  // namespace aqk

namespace aqh {
using namespace aqk;

size_t glu_gemv_workspace_bytes(const Geom &, int) { return kWsHeader; }

cudaError_t launch_gemv_fused(const Geom &g, const LayerWeights &w, const uint16_t *x, int batch,
                              const EpilogueArgs &ep, uint16_t *y, void *, cudaStream_t s)
{
    return with_scheme(g, [&](auto sch) {
        simple_fused_kernel<decltype(sch)><<<g.out, kSimpleTokens, 0, s>>>(g, w, x, batch, ep, y);
        return cudaGetLastError();
    });
}

cudaError_t launch_glu_gemv(const Geom &g, const LayerWeights &gate, const LayerWeights &up, const uint16_t *x,
                            int batch, int act, uint16_t *y, void *, cudaStream_t s)
{
    return with_scheme(g, [&](auto sch) {
        simple_glu_kernel<decltype(sch)><<<g.out, kSimpleTokens, 0, s>>>(g, gate, up, x, batch, act, y);
        return cudaGetLastError();
    });
}

}  // namespace aqh
