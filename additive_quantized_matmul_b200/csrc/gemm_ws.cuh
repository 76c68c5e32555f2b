// Warp-specialised product kernel on the 5th-generation tensor cores, shared
// by the prefill product (gemm.cu), its fused forms (gemm_fused.cu) and the
// transposed product (input_grad.cu).
//
// Tile M = 128 rows x N = BN tokens (256 or 512), K = 64 per stage; the
// decoded W tile feeds BN tokens, so BN = 512 halves the decode work per
// MMA (the 1x16 decode, ~1024 random L2 gathers per stage, is slower than
// the four N = 256 MMAs of a stage).  Split-K over the contraction
// (blockIdx.z) fills the SMs when the tile grid is small.
//   warp 0     X producer: one lane issues BN/64 2-D TMA loads per stage (64
//              tokens x 64 features each, 128-byte swizzle, MN-major) that
//              complete on full_b[stage];
//   warp 1     MMA issuer: one lane waits for full_a/full_b, issues
//              tcgen05.mma (M 128, N 256, K 16; two per K step for BN = 512)
//              into a BN-column fp32 TMEM accumulator and commits to
//              empty[stage] (buffer free) and, after the last stage, to
//              acc_full;
//   warps 2-5  (and 6-9) decoders, then epilogue: thread t of a group owns
//              one code chunk (8 rows x one group) of each of its stages.
//              1x16: the 8 codewords go from the L2-resident codebook
//              straight into the swizzled A tile by 16-byte cp.async, as
//              many stages ahead as the ring is deep; 2x8: codewords come
//              from the codebooks in shared memory, summed with binary16
//              adds, and each thread fences its writes to the async proxy.
//              128 arrivals on full_a[stage].  The epilogue reads TMEM lanes
//              32*(warp%4).. with tcgen05.ld and hands each row's sums, 16
//              tokens at a time, to the operator.
//
// Pairs (512-token tiles of every operator but the plain product): two CTAs
// with a row tile each run as one for tcgen05 (cta_group::2, M 256).  Each
// holds its own W tile and half of X, so X comes from L2 and is written to
// shared memory once for both; the even CTA issues the MMAs, on barriers that
// both arrive on.  What bounds the main loop is the SM's shared memory (128
// bytes a clock): per stage the MMAs read 64 KiB of operands (96 KiB
// unpaired), TMA writes 32 (64), and the decode takes 1024 single 16-byte
// fills (1x16) or about 800 wavefronts of random codeword reads and tile
// writes (2x8).  Measured cycles a stage at 1.7 GHz, unpaired and paired:
// 1x16 2157 -> 1399, 2x8 1500 -> 1255; the MMAs alone take 1024.
//
// The operator (Op) says what the tile's rows are, where the weights come
// from and what becomes of the sums:
//  * rows of one layer (PlainOp, FusedOp): thread t decodes chunk (row tile
//    t/8, group t%8), A K-major;
//  * kGated: 64 rows of two layers, gate and up, interleaved so that each
//    TMEM lane quarter holds 16 rows of the gate and the same 16 of the up
//    projection: the pair of an output meets in one warp, and one decoded
//    tile still feeds BN tokens;
//  * kTransposed: the tile's rows are 128 input features, the contraction
//    runs over the layer's rows (of one or two layers, one after the other):
//    thread t decodes chunk (row tile t/16, group t%16) and its codewords
//    lie along M, so A is MN-major like B.  The row scale belongs to the
//    contraction index and is multiplied, divided by 2^E, into the weights (one
//    or two 8-bit codebooks, weight_exponent) or, before, into the other operand
//    (scale_rows in layer_ops.cuh): one rounding to binary16; 2^E is applied to
//    the fp32 sums.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <type_traits>

#include "epilogue.cuh"
#include "scheme.cuh"
#include "tc_common.cuh"

namespace aqk {

constexpr int kBM = 128;                    // tile rows (MMA M)
constexpr int kBK = 64;                     // contraction per stage
constexpr int kTileABytes = kBM * kBK * 2;  // 16 KiB

// Ring depth: 4 stages of (16 KiB A + 32 KiB B) for BN = 256, 3 when the
// codebooks take 16 KiB or more of the shared memory (two layers' 2x8, 8x8);
// 2 stages of (16 + 64 KiB) for BN = 512.  `BB`: bytes of 8-bit codebooks.
// `Pair`: a CTA pair, each CTA holding half of every X tile (32 KiB a stage).
template <class S, int BN, int BB, bool Pair>
constexpr int kWsStagesOf = Pair ? 4 : (BN == 512) ? 2 : (BB > 8192 || (S::K == 1 && S::B == 16)) ? 3 : 4;
// The W (decoded) tiles have a ring of their own, 5 deep (4 with the 32 KiB
// of 8x8 codebooks): with 512-token X tiles taking 64 KiB a stage, a shared
// ring would be 2 deep.  The 1x16 decoders (two groups of 128 threads, two
// of each group's stages in flight: about 4000 codeword reads per CTA) need
// the depth; at 256-token tiles 1x16 trades an X stage for two W stages
// (6 W, 3 X).  Pairs leave 96 KiB for W tiles and codebooks.
template <class S, int BN, int BB, bool Pair>
constexpr int kWsAStagesOf = (Pair && BB == 0)        ? 6
                             : (BN == 512)              ? ((BB > 16384) ? 4 : 5)
                             : (S::K == 1 && S::B == 16) ? 6
                                                         : kWsStagesOf<S, BN, BB, Pair>;
// Decoder groups of 4 warps taking alternate stages: one CTA per SM (the X
// tiles fill its shared memory), so the decode rate per SM is that of its
// decoders; with one or two codebooks two groups run (twice the 1x16
// codeword reads in flight; twice the shared-memory decode of 8-bit codes:
// at 512 tokens 20 % faster for both), eight 8-bit codebooks keep one (their
// registers).
template <class S>
constexpr int kWsGroupsOf = (S::K <= 2) ? 2 : 1;
template <class S>
constexpr int kWsThreadsOf = 64 + 128 * kWsGroupsOf<S>;  // X producer, MMA issuer, decoders

// Layers whose 8-bit codebooks a CTA keeps in shared memory.
template <class S, class Op>
constexpr int kWsBookBytes = S::kSmemBookBytes * Op::kLayers;

// Boxes of an operator's input in a tile.
template <class Op, int BN>
constexpr int kInBoxes = Op::kStaged ? BN / 64 * 4 : 0;

template <int N>
struct TensorMaps {
    CUtensorMap m[N];
};

struct GemmSplit {
    float *partials;  // a split cluster's slices, or null with one split
};

// Grid of the tail mode: CTAs [0, full) take whole tiles (tile = index), the
// others split the tiles from `full` on, `ks` CTAs of `per` stages each.
struct TailMap {
    int full;  // CTAs with a whole tile; 0: no tail mode (3-D grid)
    int ks;    // splits per tail tile
    int per;   // 64-feature stages per split
};

__device__ __forceinline__ uint4 round_h8(const float *v)
{
    return make_uint4(f2h2(v[0], v[1]), f2h2(v[2], v[3]), f2h2(v[4], v[5]), f2h2(v[6], v[7]));
}

__device__ __forceinline__ void widen_h8(uint4 p, float *v)
{
    float2 f;
    f = h2f2(p.x), v[0] = f.x, v[1] = f.y;
    f = h2f2(p.y), v[2] = f.x, v[3] = f.y;
    f = h2f2(p.z), v[4] = f.x, v[5] = f.y;
    f = h2f2(p.w), v[6] = f.x, v[7] = f.y;
}

// Where a tile's sums are written.
struct TileOut {
    int mt, n0, T;
    float factor;  // kTransposed: 2^E, or 1
};

// ---- operators ----------------------------------------------------------------
//
// PlainOp stores its rows straight from registers.  The others (kStaged) pass
// them through shared memory: `kRows` consecutive rows of the output per TMEM
// lane quarter, from row0(); of 16 accumulator columns (tokens gn ..) a lane
// turns its share into kPieces 16-byte pieces of its output row (two for 32
// rows: all 16 tokens; one for 16 rows: tokens 8 (lane / 16) ..), reading the
// matching pieces of its own input (residual or gradient) if it has one.
// io() are its arrays: 0 the input, 1 and 2 the outputs; their tensor maps
// follow the activations' in the kernel's parameters (T is a multiple of 8, or
// the rows of every array are padded to one).

// y = RN16(s (W x)); T % 8 == 0.
struct PlainOp {
    static constexpr bool kGated = false, kTransposed = false, kStaged = false;
    static constexpr bool kScaleWeights = false;
    static constexpr int kLayers = 1, kMaps = 1, kXMaps = 1, kAhead = 4;
    static constexpr bool kPairs = false;
    LayerWeights w[1];
    uint16_t *y;
};

// y = RN16(act(s (W x) + bias) + residual), or, with gy: grad_z = RN16(gy
// act'(z)) and the sums of gy act'(z) over each block of 16 tokens.
struct FusedOp {
    static constexpr bool kGated = false, kTransposed = false, kStaged = true;
    static constexpr bool kScaleWeights = false;
    static constexpr int kLayers = 1, kXMaps = 1, kRows = 32, kPieces = 2, kOutputs = 1, kAhead = 4;
    static constexpr int kMaps = kXMaps + 3;
    static constexpr bool kPairs = true;
    LayerWeights w[1];
    int act;
    const uint16_t *bias;  // or null
    const uint16_t *in;    // residual, or gy (grad); or null
    uint16_t *out;         // y, or grad_z
    bool grad;
    float *sums;           // grad: [blocks of 16 tokens][out], or null
    unsigned *top;         // grad: ws_top, takes the largest |s grad_z|; or null

    struct Row {
        float sc, b;
    };
    __host__ __device__ const uint16_t *io(int i) const
    {
        return i == 0 ? in : i == 1 ? out : nullptr;
    }
    __device__ __forceinline__ int row0(const TileOut &o) const { return o.mt * kBM + (int)((threadIdx.x >> 5) & 3) * 32; }
    __host__ __device__ int rows(const Geom &L) const { return L.out; }
    __device__ __forceinline__ Row row(const Geom &L, const TileOut &o) const
    {
        const int i = row0(o) + (int)(threadIdx.x & 31);
        return Row{(i < L.out && w[0].scales) ? half_bits_to_float(w[0].scales[i]) : 1.f,
                   (i < L.out && bias) ? half_bits_to_float(bias[i]) : 0.f};
    }
    template <class F>
    __device__ __forceinline__ void dispatch(F &&f) const
    {
        with_act_family(act, [&](auto family) {
            if (grad) f(family, std::true_type{});
            else f(family, std::false_type{});
        });
    }
    template <int Family, bool Grad>
    __device__ __forceinline__ void apply(const Geom &L, const TileOut &o, const ActParams &k, const Row &r, int gn,
                                          float (&v)[16], const uint4 (&x)[2], uint4 (&y0)[2], uint4 (&)[2],
                                          uint32_t (&m)[2]) const
    {
        float sum = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float a[8], e[8];
            widen_h8(x[h], e);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float z = fmaf(r.sc, v[8 * h + j], r.b);
                if constexpr (Grad) {
                    float slope;
                    act_value<Family>(k, z, slope);
                    a[j] = e[j] * slope;
                    if (gn + 8 * h + j < o.T) sum += a[j];
                } else {
                    a[j] = act_value<Family>(k, z) + e[j];  // no residual: e = -0 changes nothing
                }
            }
            y0[h] = round_h8(a);
            if constexpr (Grad)
                if (top) finite_absmax_h8(m[0], y0[h]);
        }
        if constexpr (Grad) {
            const int i = row0(o) + (int)(threadIdx.x & 31);
            if (sums && i < L.out) sums[(size_t)(gn >> 4) * L.out + i] = sum;
        }
    }
    __device__ __forceinline__ float largest(const Row &r, const uint32_t (&m)[2]) const { return scaled_top(m[0], r.sc); }
};

// Gated block: y = RN16(act(g) u), or, with gy, the gradients of g and u.
struct GatedOp {
    static constexpr bool kGated = true, kTransposed = false, kStaged = true;
    static constexpr bool kScaleWeights = false;
    static constexpr int kLayers = 2, kXMaps = 1, kRows = 16, kPieces = 1, kOutputs = 2, kAhead = 4;
    static constexpr int kMaps = kXMaps + 3;
    static constexpr bool kPairs = true;
    LayerWeights w[2];  // gate, up
    int act;
    const uint16_t *gy;      // or null: forward
    uint16_t *out0, *out1;   // y, -; or grad_gate, grad_up
    unsigned *top;           // gy: ws_top, takes the largest |s_g grad_gate|, |s_u grad_up|; or null

    struct Row {
        float sc;
    };
    __host__ __device__ const uint16_t *io(int i) const
    {
        return i == 0 ? gy : i == 1 ? out0 : out1;
    }
    __device__ __forceinline__ int row0(const TileOut &o) const
    {
        return o.mt * (kBM / 2) + (int)((threadIdx.x >> 5) & 3) * 16;
    }
    __host__ __device__ int rows(const Geom &L) const { return L.out; }
    __device__ __forceinline__ Row row(const Geom &L, const TileOut &o) const
    {
        // lanes 0-15: gate rows, 16-31: the same rows of up
        const int i = row0(o) + (int)(threadIdx.x & 15);
        const uint16_t *s = (threadIdx.x & 16) ? w[1].scales : w[0].scales;
        return Row{(i < L.out && s) ? half_bits_to_float(s[i]) : 1.f};
    }
    // Lane l < 16 (gate) gives its tokens 8-15 to lane l + 16 (up) for that
    // lane's tokens 0-7: each then has eight tokens of both projections.
    template <class F>
    __device__ __forceinline__ void dispatch(F &&f) const
    {
        with_act_family(act, [&](auto family) {
            if (gy) f(family, std::true_type{});
            else f(family, std::false_type{});
        });
    }
    template <int Family, bool Grad>
    __device__ __forceinline__ void apply(const Geom &, const TileOut &, const ActParams &k, const Row &r, int,
                                          float (&v)[16], const uint4 (&x)[1], uint4 (&y0)[1], uint4 (&y1)[1],
                                          uint32_t (&m)[2]) const
    {
        const bool hi = threadIdx.x & 16;
        float a[8], c[8], e[8];
        if constexpr (Grad) widen_h8(x[0], e);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float lo_v = r.sc * v[j], hi_v = r.sc * v[j + 8];
            const float got = __shfl_xor_sync(0xffffffffu, hi ? lo_v : hi_v, 16);
            const float g = hi ? got : lo_v, u = hi ? hi_v : got;  // gate, up
            if constexpr (Grad) {
                float slope;
                c[j] = e[j] * act_value<Family>(k, g, slope);
                a[j] = e[j] * u * slope;
            } else {
                a[j] = act_value<Family>(k, g) * u;
            }
        }
        y0[0] = round_h8(a);
        if constexpr (Grad) {
            y1[0] = round_h8(c);
            if (top) {
                finite_absmax_h8(m[0], y0[0]);
                finite_absmax_h8(m[1], y1[0]);
            }
        }
    }
    __device__ __forceinline__ float largest(const Row &r, const uint32_t (&m)[2]) const
    {
        const bool hi = threadIdx.x & 16;
        const float other = __shfl_xor_sync(0xffffffffu, r.sc, 16);
        return fmaxf(scaled_top(m[0], hi ? other : r.sc), scaled_top(m[1], hi ? r.sc : other));
    }
};

// gx = RN16(2^E sum over the layers of W^T (s gy / 2^E)).  ScaleW: the decoders
// scale the weights, which pass through registers anyway, with E from the largest
// scale and codebook entry.  Else the scales are in gy, with E from the largest
// product: 16-bit codebooks are too long to look through in a CTA, 1x16 weights go
// into shared memory by asynchronous copies (scaling them on the way through
// registers took 2207 cycles a stage against 1400), and 8x8 decoders have no time
// to spare (input gradient 11008 x 4096, 2048 tokens 892 -> 856 us; 2x8, which
// would need two passes over the gradients, 206 -> 175 with scaled weights).
template <bool ScaleW>
struct BackOp {
    static constexpr bool kGated = false, kTransposed = true, kStaged = true;
    static constexpr bool kScaleWeights = ScaleW;
    static constexpr int kLayers = 2, kXMaps = 2, kRows = 32, kPieces = 2, kOutputs = 1, kAhead = 4;
    static constexpr int kMaps = kXMaps + 3;
    static constexpr bool kPairs = true;
    LayerWeights w[2];
    int layers;  // 1 or 2
    uint16_t *gx;
    const float *factor;  // !ScaleW: 2^E, or null: 1
    unsigned *top;        // with factor: to be cleared
    static constexpr int act = AQ_ACT_NONE;

    struct Row {
        float sc;
    };
    __host__ __device__ const uint16_t *io(int i) const { return i == 1 ? gx : nullptr; }
    __device__ __forceinline__ int row0(const TileOut &o) const { return o.mt * kBM + (int)((threadIdx.x >> 5) & 3) * 32; }
    __host__ __device__ int rows(const Geom &L) const { return L.in; }
    __device__ __forceinline__ Row row(const Geom &, const TileOut &o) const { return Row{o.factor}; }
    template <class F>
    __device__ __forceinline__ void dispatch(F &&f) const
    {
        f(std::integral_constant<int, kActLinear>{}, std::false_type{});
    }
    template <int, bool>
    __device__ __forceinline__ void apply(const Geom &, const TileOut &, const ActParams &, const Row &r, int,
                                          float (&v)[16], const uint4 (&)[2], uint4 (&y0)[2], uint4 (&)[2],
                                          uint32_t (&)[2]) const
    {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= r.sc;
        y0[0] = round_h8(v);
        y0[1] = round_h8(v + 8);
    }
};

// Row tiles of the grid, and 64-deep stages of the whole contraction.
template <class Op>
__host__ __device__ __forceinline__ int ws_mtiles(const Geom &L)
{
    if (Op::kTransposed) return (L.in + kBM - 1) / kBM;
    constexpr int rows = Op::kGated ? kBM / 2 : kBM;
    return (L.out + rows - 1) / rows;
}
// stages of one layer's contraction (kTransposed: `layers` of them in a row)
template <class Op>
__host__ __device__ __forceinline__ int ws_layer_stages(const Geom &L)
{
    return ((Op::kTransposed ? L.out : L.in) + kBK - 1) / kBK;
}

// Sums of one block of 16 columns over the `ks` splits of a tile, in split
// order: split z's own from `v` (tensor memory), the others' from their
// slices, kAhead splits' loads in flight at a time.
template <int kAhead>
__device__ __forceinline__ void add_slices(float (&v)[16], const float4 *src, size_t slice, int ks, int z)
{
    float acc[16];
    for (int z0 = 0; z0 < ks; z0 += kAhead) {
        float4 t[kAhead][4];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (z0 + i < ks && z0 + i != z) t[i][j] = __ldcg(src + (size_t)(z0 + i) * slice + j * kBM);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (z0 + i >= ks) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 u = (z0 + i == z) ? make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3])
                                               : t[i][j];
                if (z0 + i == 0) {
                    acc[4 * j] = u.x, acc[4 * j + 1] = u.y, acc[4 * j + 2] = u.z, acc[4 * j + 3] = u.w;
                } else {
                    acc[4 * j] += u.x, acc[4 * j + 1] += u.y, acc[4 * j + 2] += u.z, acc[4 * j + 3] += u.w;
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = acc[j];
}

// The splits of a tile: their slices at this thread's row, and which of them
// this CTA is (ks = 1: the sums are whole).
template <int BN>
struct Splits {
    const float4 *slices;
    int ks, z;
    template <int kAhead>
    __device__ __forceinline__ void add(int c, float (&v)[16]) const
    {
        constexpr size_t kSlice = kBM * BN / 4;  // float4 per slice
        if (ks > 1) add_slices<kAhead>(v, slices + ((c / 16) * 4) * kBM, kSlice, ks, z);
    }
};

// A warp's share of the finish: accumulator columns [c, end) of its 32 TMEM
// lanes at `tq`, 64 at a time, every `step`, as blocks of 16.  The next
// block's columns are requested before a block is worked on.
template <class F>
__device__ __forceinline__ void accumulator_blocks(uint32_t tq, int c, int step, int end, F &&block)
{
    uint32_t acc[16];
    if (c < end) tmem_ld16_start(tq + (uint32_t)c, acc);
#pragma unroll 1
    while (c < end) {
        float v[16];
        tmem_ld16_wait(acc, v);
        const int next = ((c + 16) & 63) ? c + 16 : c + 16 - 64 + step;
        if (next < end) tmem_ld16_start(tq + (uint32_t)next, acc);
        block(c, v);
        c = next;
    }
}

// Rows straight from registers.
template <int BN>
__device__ __forceinline__ void finish_direct(const PlainOp &op, const Geom &L, const TileOut &o, uint32_t tq, int c,
                                              int step, int end, const Splits<BN> &splits)
{
    const int row = o.mt * kBM + (int)((threadIdx.x >> 5) & 3) * 32 + (int)(threadIdx.x & 31);
    const float sc = (row < L.out && op.w[0].scales) ? half_bits_to_float(op.w[0].scales[row]) : 1.f;
    end = min(end, o.T - o.n0);
#pragma unroll 1
    for (; c < end; c += step) {
        float v[16];
        tmem_ld16(tq + (uint32_t)c, v);
        splits.template add<PlainOp::kAhead>(c, v);
        if (row >= L.out) continue;
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= sc;
        uint4 *dst = reinterpret_cast<uint4 *>(op.y + (size_t)row * o.T + o.n0 + c);
        dst[0] = round_h8(v);
        if (o.n0 + c + 8 < o.T) dst[1] = round_h8(v + 8);  // T % 8 == 0
    }
}

// Rows through shared memory: 64 tokens x kRows rows per warp and step in the
// layout of a 128-byte-swizzled TMA box, in the ring that the MMAs no longer
// read.  The input's boxes come by TMA, all requested at once; a lane reads
// its pieces, writes its results over them, and the box leaves by TMA.  (One
// row per lane straight to memory would make 32 requests of 32 bytes an
// instruction: measured 18 to 40 thousand cycles a tile instead of 7 to 14.)
// Not inlined: its registers are its own, and the decoders' loop keeps theirs.
template <int Family, bool Grad, int BN, class Op>
__device__ __noinline__ void finish_staged(const Op &op, const Geom &L, const TileOut &o, const CUtensorMap *io,
                                           uint8_t *stage, uint64_t *in_bar, void *ws, uint32_t tq, int c, int step,
                                           int end, const Splits<BN> &splits)
{
    constexpr int R = Op::kRows, P = Op::kPieces;
    constexpr int kBox = R * 128;  // bytes of a box
    constexpr bool kTwo = Op::kOutputs > 1 && Grad;
    constexpr uint32_t kNegZero = 0x80008000u;  // the neutral addend of a missing residual
    const int lane = threadIdx.x & 31, q = (threadIdx.x >> 5) & 3;
    const int row0 = op.row0(o), nrows = op.rows(L);
    const typename Op::Row row = op.row(L, o);
    const ActParams k = act_params(op.act);
    end = min(end, o.T - o.n0);
    if (row0 >= nrows || c >= end) return;  // (a pair's second row tile may be empty)
    const int r_lane = R == 32 ? lane : lane & 15, p_lane = R == 32 ? 0 : lane >> 4;
    auto box = [&](int cb, int a) { return stage + ((size_t)a * (BN / 64) + cb / 64) * (4 * kBox) + q * kBox; };
    const uint16_t *in = op.io(0);
    uint32_t top[2] = {0u, 0u};  // Grad: largest finite results, per half
    if (in && lane == 0) {
        fence_proxy_async_smem();
        for (int cb = c; cb < end; cb += step) {
            uint64_t *bar = &in_bar[(cb / 64) * 4 + q];
            mbar_arrive_expect_tx(bar, kBox);
            tma_load_2d(smem_u32(box(cb, 0)), &io[0], o.n0 + cb, row0, bar);
        }
    }
    __syncwarp();
    accumulator_blocks(tq, c, step, end, [&](int cc, float (&v)[16]) {
        const int cb = cc & ~63, b = (cc & 63) / 16;
        uint8_t *b0 = box(cb, 0);
        if (in && b == 0) {
            if (!mbar_wait_ns(&in_bar[(cb / 64) * 4 + q], 0, kWaitNs)) record_status(ws, AQ_ERR_TIMEOUT);
            __syncwarp();
        }
        splits.template add<Op::kAhead>(cc, v);
        uint4 x[P], y0[P], y1[P];
        // piece i of the lane: 16-byte chunk 2 b + p_lane + i of its row
        uint32_t at[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            at[i] = sw128((uint32_t)r_lane, (uint32_t)(2 * b + p_lane + i));
            x[i] = in ? *reinterpret_cast<const uint4 *>(b0 + at[i]) : make_uint4(kNegZero, kNegZero, kNegZero, kNegZero);
        }
        op.template apply<Family, Grad>(L, o, k, row, o.n0 + cc, v, x, y0, y1, top);
        uint8_t *b1 = kTwo ? box(cb, 1) : nullptr;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            *reinterpret_cast<uint4 *>(b0 + at[i]) = y0[i];
            if (kTwo) *reinterpret_cast<uint4 *>(b1 + at[i]) = y1[i];
        }
        if (b == 3 || cc + 16 >= end) {  // the box is complete (or the tokens are)
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(&io[1], smem_u32(b0), o.n0 + cb, row0);
                if (kTwo) tma_store_2d(&io[2], smem_u32(b1), o.n0 + cb, row0);
                bulk_commit();
            }
        }
    });
    if constexpr (Grad)
        if (op.top) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(op.largest(row, top)));
            if (lane == 0) atomicMax(op.top, m);
        }
    bulk_wait_all();  // the boxes have been read and written
}

// ---- split contractions ---------------------------------------------------------
//
// A tile whose contraction is split over several CTAs is finished from their
// fp32 sums, added in split order (deterministic).  The scratch holds one
// slice of kBM x BN floats per split in the order tensor memory hands them
// out: float4 j of column block cb of tile row r at ((cb 4 + j) 128 + r), so
// a warp's 32 rows are 512 contiguous bytes for the writer and the reader
// alike (the finishing thread of a row is the writer's thread of that row).
// Two forms:
//  * a grid smaller than the GPU: the `ks` splits of a tile (2, 4 or 8) run
//    as one thread-block cluster along blockIdx.z (the split index is the
//    CTA's rank).  The cluster guarantees that they run at the same time, so
//    the finish is spread over all of them: CTA z owns the tile's columns
//    [z BN / ks, (z + 1) BN / ks), writes the other columns' sums from tensor
//    memory to its slice (L2), and after the cluster barrier adds, for its
//    own columns, every split's sums (its own straight from tensor memory).
//  * the tail of a grid larger than one wave: when the last wave would hold
//    few tiles, their contraction is split over `ks` CTAs each (a 1-D grid:
//    whole tiles first, then the tail tiles' splits), so the last wave fills
//    the SMs.  Every split writes all its columns, arrives on the tile's
//    counter (acq_rel), and the last to arrive finishes the tile and resets
//    the counter.

// This warp's columns c, c + step, ... of the accumulator, but for those in
// [own0, own1), to a slice.
template <int BN>
__device__ __forceinline__ void publish_sums(float4 *slice, uint32_t tq, int c, int step, int own0, int own1, int live,
                                             int r)
{
#pragma unroll 1
    for (; c < min(BN, live); c += step) {
        if (c >= own0 && c < own1) continue;  // warp-uniform
        float v[16];
        tmem_ld16(tq + (uint32_t)c, v);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            __stcg(slice + ((c / 16) * 4 + j) * kBM + r, make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
    }
}

// ---- kernel -------------------------------------------------------------------

// Barrier of the decoder threads alone (the CTA's other warps do not take part).
__device__ __forceinline__ void decoder_barrier(int threads)
{
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
}

template <class S, int BN, class Op, bool Pair>
__global__ void __launch_bounds__(kWsThreadsOf<S>, 1)
gemm_ws_kernel(const __grid_constant__ TensorMaps<Op::kMaps> maps, Geom L, const __grid_constant__ Op op, int T,
               void *ws, GemmSplit sp, int stages_per_split, int cluster_ks, TailMap tm)
{
    constexpr int BB = kWsBookBytes<S, Op>;
    constexpr int kWsStages = kWsStagesOf<S, BN, BB, Pair>;    // X ring
    constexpr int kWsAStages = kWsAStagesOf<S, BN, BB, Pair>;  // W ring
    constexpr int kWsTileB = kBK * BN * 2 / (Pair ? 2 : 1);    // 32 or 64 KiB
    constexpr int kN = BN < 256 ? BN : 256;  // N of one MMA instruction
    constexpr int NG = kWsGroupsOf<S>;       // decoder groups
    constexpr bool kTr = Op::kTransposed, kScaleW = Op::kScaleWeights;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint8_t *tileA = smem;                                   // [stages][16 KiB]
    uint8_t *tileB = smem + kWsAStages * kTileABytes;        // [X stages][32 or 64 KiB]
    uint4 *scb = reinterpret_cast<uint4 *>(tileB + kWsStages * kWsTileB);
    uint64_t *full_a = reinterpret_cast<uint64_t *>(reinterpret_cast<uint8_t *>(scb) + BB);
    uint64_t *full_b = full_a + kWsAStages;
    uint64_t *empty = full_b + kWsStages;       // X buffers free
    uint64_t *empty_a = empty + kWsStages;      // W buffers free
    uint64_t *peer_a = empty_a + kWsAStages;    // pair with asynchronous copies: the odd CTA's W buffer is full
    uint64_t *acc_full = peer_a + (Pair ? kWsAStages : 0);
    uint64_t *in_bar = acc_full + 1;            // kStaged: the input's boxes, one per 64 tokens and lane quarter
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(in_bar + kInBoxes<Op, BN>);
    uint32_t *abort_flag = tmem_slot + 1;
    uint32_t *last_flag = abort_flag + 1;       // the last split of a tail tile
    uint32_t *scale_max = last_flag + 1;        // kScaleW: largest |s| and |C| (binary16 bits)

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int layer_stages = ws_layer_stages<Op>(L);
    int all_stages = layer_stages;
    if constexpr (kTr) all_stages *= op.layers;
    // the CTA's tile and split: a 3-D grid (row tile, token tile, split), or
    // the tail mode's 1-D grid
    // (a pair takes two row tiles, 2 u and 2 u + 1, of which the last may be empty)
    const int half = Pair ? blockIdx.x & 1 : 0;
    int mt = blockIdx.x, nt = blockIdx.y, z = blockIdx.z, per = stages_per_split, tail_idx = -1;
    if (tm.ks > 0) {
        const int mtiles = Pair ? (ws_mtiles<Op>(L) + 1) / 2 : ws_mtiles<Op>(L);
        int tile = Pair ? blockIdx.x >> 1 : blockIdx.x;
        z = 0;
        per = all_stages;
        if (tile >= tm.full) {
            const int rr = tile - tm.full;
            tail_idx = rr / tm.ks;
            z = rr % tm.ks;
            tile = tm.full + tail_idx;
            per = tm.per;
            if (Pair) tail_idx = 2 * tail_idx + half;  // each CTA has slices and a counter of its own
        }
        mt = tile % mtiles;
        if (Pair) mt = 2 * mt + half;
        nt = tile / mtiles;
    }
    const int n0 = nt * BN;
    // this split's stages: global stages s0 .. s0 + nk - 1
    const int s0 = z * per;
    const int nk = max(0, min(all_stages, s0 + per) - s0);

    // 1x16: codewords go from L2 into the tile by cp.async, as many stages in
    // flight as the ring holds (the copies arrive on the stage's barrier
    // themselves, and the MMA issuer orders them before its reads); other
    // schemes decode in registers
    constexpr bool kAsyncWeights = S::K == 1 && S::B == 16;
    static_assert(!kScaleW || (S::kBooksInSmem && S::K <= 2), "see BackOp");
    if (S::B == 16 && tid == 0) prefetch_table_share(op.w[0].cb, (uint32_t)S::K * 65536u * 16u);
    if constexpr (S::B == 16 && Op::kLayers > 1)
        if (tid == 32) prefetch_table_share(op.w[1].cb, (uint32_t)S::K * 65536u * 16u);
    if constexpr (S::kBooksInSmem) {
        for (int i = tid; i < S::K * 256; i += kWsThreadsOf<S>) {
#pragma unroll
            for (int l = 0; l < Op::kLayers; ++l) scb[l * S::K * 256 + i] = op.w[l].cb[i];
        }
    }
    if (tid == 0) {
        for (int s = 0; s < kWsAStages; ++s) {
            // one arrival per decoder thread; pair: the leader's, one per warp
            // of both CTAs (asynchronous copies arrive at home, see peer_a)
            mbar_init(&full_a[s], Pair && !kAsyncWeights ? 8 : 128);
            mbar_init(&empty_a[s], 1);
            if (Pair && kAsyncWeights) mbar_init(&peer_a[s], 1);
        }
        for (int s = 0; s < kWsStages; ++s) {
            mbar_init(&full_b[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        for (int i = 0; i < kInBoxes<Op, BN>; ++i) mbar_init(&in_bar[i], 1);
        *abort_flag = 0;
        if constexpr (kScaleW) scale_max[0] = scale_max[1] = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        if constexpr (Pair) tmem_alloc_pair(tmem_slot, BN);
        else tmem_alloc(tmem_slot, BN);
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (Pair) cluster_sync_all();  // the leader's barriers, before anyone arrives on them
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t leader = Pair ? cluster_ctarank() & ~1u : 0;  // cluster rank
    const uint16_t pair_mask = (uint16_t)(3u << leader);
    volatile uint32_t *abort_v = abort_flag;
    // this thread's (Pair: warp's, by one lane) writes of a W stage are visible to the MMAs
    auto publish = [&](int s) {
        fence_proxy_async_smem();
        if constexpr (Pair) {
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_shared(&full_a[s % kWsAStages], leader));
        } else {
            mbar_arrive(&full_a[s % kWsAStages]);
        }
    };
    TileOut out{mt, n0, T, 1.f};
    // programmatic dependent launch: before the wait a thread reads weights
    // only (codes, codebooks); X, y, the scales and the workspace follow it
    grid_launch_dependents();

    if (warp == 0) {
        // ---------------- X producer ----------------
        if (lane == 0) {
            grid_dependency_wait();
            for (int s = 0; s < nk; ++s) {
                const int buf = s % kWsStages;
                if (s >= kWsStages && !mbar_wait_ns(&empty[buf], ((s / kWsStages) - 1) & 1, kWaitNs)) {
                    *abort_v = 1;
                    break;
                }
                if (*abort_v) break;
                // pair: both halves complete on the leader's barrier
                if (!Pair || half == 0) mbar_arrive_expect_tx(&full_b[buf], kWsTileB * (Pair ? 2 : 1));
                const uint32_t dst = smem_u32(tileB + buf * kWsTileB);
                int row = (s0 + s) * kBK;
                const CUtensorMap *map = &maps.m[0];
                if constexpr (Op::kXMaps > 1)
                    if (s0 + s >= layer_stages) {
                        map = &maps.m[1];
                        row -= layer_stages * kBK;
                    }
                if constexpr (Pair) {
                    // of each 256 tokens of an MMA this CTA holds 128
                    const uint32_t bar = map_shared(&full_b[buf], leader);
#pragma unroll
                    for (int q = 0; q < BN / 128; ++q)
                        tma_load_2d_pair(dst + q * (kBK * 128), map, n0 + 256 * (q >> 1) + 128 * half + 64 * (q & 1), row,
                                         bar);
                } else {
#pragma unroll
                    for (int q = 0; q < BN / 64; ++q)
                        tma_load_2d(dst + q * (kBK * 128), map, n0 + 64 * q, row, &full_b[buf]);
                }
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        // first, the tile of the operator's own input (residual, gradient)
        // into L2, where the epilogue will ask for it
        const uint16_t *in = nullptr;
        if constexpr (Op::kStaged) in = op.io(0);
        if (in) {
            grid_dependency_wait();
            const int rows = Op::kGated ? kBM / 2 : kBM;
            for (int i = lane; i < rows && mt * rows + i < L.out; i += 32) {
                const int pitch = (T + 7) & ~7;
                prefetch_l2_bulk(in + (size_t)(mt * rows + i) * pitch + n0, 2u * (uint32_t)min(BN, pitch - n0));
            }
            __syncwarp();
        }
        if (lane == 0 && half == 0) {  // pair: the leader
            const uint32_t idesc = make_idesc(Pair ? 2 * kBM : kBM, kN, true) | (kTr ? 1u << 15 : 0u);  // kTr: A MN-major
            int s = 0;
            for (; s < nk; ++s) {
                const int buf = s % kWsStages, abuf = s % kWsAStages;
                const uint32_t pa = (s / kWsAStages) & 1, pb = (s / kWsStages) & 1;
                if (!mbar_wait_ns(&full_a[abuf], pa, kWaitNs) || !mbar_wait_ns(&full_b[buf], pb, kWaitNs)) {
                    *abort_v = 1;
                    break;
                }
                if constexpr (Pair && kAsyncWeights)
                    if (!mbar_wait_ns(&peer_a[abuf], pa, kWaitNs)) *abort_v = 1;
                if (*abort_v) break;
                if constexpr (kAsyncWeights) fence_proxy_async_smem();  // the decoders' copies, before the MMAs
                tc_fence_after();
                const uint32_t a0 = smem_u32(tileA + abuf * kTileABytes);
                const uint32_t b0 = smem_u32(tileB + buf * kWsTileB);
#pragma unroll
                for (int ks = 0; ks < kBK / 16; ++ks) {
                    // kTr: two 64-feature blocks 8 KiB apart, +2 KiB per 16 rows of the contraction
                    const uint64_t ad = kTr ? smem_desc_sw128(a0 + ks * 2048, kBK * 128, 1024)
                                            : smem_desc_sw128(a0 + ks * 32, 16, 1024);
#pragma unroll
                    for (int h = 0; h < BN / kN; ++h) {
                        // tokens 256 h .. : four 64-token boxes further on (pair: two, of each CTA)
                        constexpr int kBoxes = kN / 64 / (Pair ? 2 : 1);
                        const uint64_t bd = smem_desc_sw128(b0 + h * kBoxes * (kBK * 128) + ks * 2048, kBK * 128, 1024);
                        const uint32_t acc = (s > 0 || ks > 0) ? 1u : 0u;
                        if constexpr (Pair) mma_f16_ss_pair(tmem + h * kN, ad, bd, idesc, acc);
                        else mma_f16_ss(tmem + h * kN, ad, bd, idesc, acc);
                    }
                }
                // X buffer free once these MMAs complete, and the W buffer
                if constexpr (Pair) {
                    mma_commit_pair(&empty[buf], pair_mask);
                    mma_commit_pair(&empty_a[abuf], pair_mask);
                } else {
                    mma_commit(&empty[buf]);
                    mma_commit(&empty_a[abuf]);
                }
            }
            // completes when every MMA issued above has
            if constexpr (Pair) mma_commit_pair(acc_full, pair_mask);
            else mma_commit(acc_full);
        }
        if constexpr (Pair && kAsyncWeights) {
            // the odd CTA's copies have landed: tell the leader
            if (lane == 0 && half == 1)
                for (int s = 0; s < nk; ++s) {
                    const int abuf = s % kWsAStages;
                    if (!mbar_wait_ns(&full_a[abuf], (s / kWsAStages) & 1, kWaitNs)) *abort_v = 1;
                    if (*abort_v) break;
                    fence_proxy_async_smem();
                    mbar_arrive_cluster(map_shared(&peer_a[abuf], leader));
                }
        }
    } else {
        // ---------------- decoders ----------------
        // group dg takes stages dg, dg + NG, dg + 2 NG, ... (its own stage k
        // is stage dg + NG k); every group runs the epilogue
        const int dg = (tid - 64) / 128;
        const int t = (tid - 64) % 128;
        const int nown = (nk - dg + NG - 1) / NG;
        // this thread's chunk of a stage: row tile and group, fixed but for
        // the index that walks the contraction
        const int rt_l = kTr ? t >> 4 : t >> 3, gi = kTr ? t & 15 : t & 7;
        const int set = Op::kGated ? (rt_l >> 1) & 1 : 0;  // gated: two row tiles of gate, two of up per lane quarter
        const int rt = Op::kGated ? mt * 8 + (rt_l >> 2) * 2 + (rt_l & 1) : mt * (kBM / 8) + rt_l;  // !kTr
        // layer, row tile and group of stage s (local)
        auto layer_of = [&](int s) { return kTr ? (s0 + s >= layer_stages ? 1 : 0) : set; };
        auto tile_of = [&](int s) {
            return kTr ? (s0 + s - (s0 + s >= layer_stages ? layer_stages : 0)) * 8 + rt_l : rt;
        };
        auto group_of = [&](int s) { return kTr ? mt * (kBM / 8) + gi : (s0 + s) * 8 + gi; };
        auto live_of = [&](int s) { return s < nk && tile_of(s) < L.rtiles && group_of(s) < L.G; };
        auto fetch = [&](int s) {
            return load_chunk<S>(op.w[Op::kLayers > 1 ? layer_of(s) : 0].packed,
                                 (size_t)tile_of(s) * L.gp + group_of(s), live_of(s));
        };
        // 16-byte chunk of row r of the thread's codes in the A tile
        auto slot_of = [&](int r) {
            return kTr ? (uint32_t)(gi >> 3) * (kBK * 128) + sw128(rt_l * 8 + r, gi & 7) : sw128(rt_l * 8 + r, gi);
        };
        // code chunks kCodeAhead stages ahead (register ring): a stage's
        // gathers never wait on an HBM round trip
        constexpr int kCodeAhead = 4;
        Chunk<S> code_ring[kCodeAhead];
#pragma unroll
        for (int q = 0; q < kCodeAhead; ++q) code_ring[q] = fetch(dg + NG * q);
        // kScaleW: the rows' scales, one per lane (rows of the warp's two
        // row tiles), as far ahead as the codes; divided by 2^E where used
        float inv = 1.f;
        uint16_t scale_ring[kCodeAhead];
        auto fetch_scale = [&](int s) -> uint16_t {
            const int l = layer_of(s), o = (tile_of(s) - (rt_l & 1)) * 8 + (lane & 15);
            if (s >= nk || o >= L.out) return (uint16_t)0;  // rows past the layer weigh nothing
            const uint16_t *sc = op.w[l].scales;
            return sc ? __ldg(sc + o) : (uint16_t)0x3c00;
        };
        if constexpr (kScaleW) {
            uint32_t c = 0;
            for (int i = tid - 64; i < op.layers * S::K * 256; i += 128 * NG) finite_absmax_h8(c, scb[i]);
            c = __reduce_max_sync(0xffffffffu, max(c & 0xffffu, c >> 16));
            if (lane == 0) atomicMax(scale_max + 1, c);
            grid_dependency_wait();  // the scales
#pragma unroll
            for (int q = 0; q < kCodeAhead; ++q) scale_ring[q] = fetch_scale(dg + NG * q);
            uint32_t m = 0;
            for (int l = 0; l < op.layers; ++l)
                m = max(m, op.w[l].scales ? finite_absmax_share(op.w[l].scales, L.out, tid - 64, 128 * NG) : 0x3c00u);
            m = __reduce_max_sync(0xffffffffu, m);
            if (lane == 0) atomicMax(scale_max, m);
            decoder_barrier(128 * NG);
            volatile uint32_t *largest = scale_max;
            const int e = weight_exponent(largest[0], largest[1], S::K);
            inv = ldexpf(1.f, -e);
            out.factor = ldexpf(1.f, e);
        }
        bool ok = true;
        // unrolled by the ring depth so every ring index is static
        for (int k0 = 0; ok && k0 < nown; k0 += kCodeAhead) {
#pragma unroll
            for (int u = 0; u < kCodeAhead; ++u) {
                const int k = k0 + u, s = dg + NG * k;  // own stage, stage
                if (k >= nown) break;
                {
                    const int buf = s % kWsAStages;
                    // the buffer is free once the MMAs of stage s - depth completed
                    if (s >= kWsAStages && !mbar_wait_ns(&empty_a[buf], ((s / kWsAStages) - 1) & 1, kWaitNs)) *abort_v = 1;
                    // a warp leaves together where its lanes act together
                    if ((kScaleW || Pair) ? __any_sync(0xffffffffu, *abort_v != 0) : *abort_v != 0) {
                        ok = false;
                        break;
                    }
                    const Chunk<S> code = code_ring[u];
                    const bool live = live_of(s);
                    uint8_t *A = tileA + buf * kTileABytes;
                    const uint4 *books = scb + (Op::kLayers > 1 ? layer_of(s) * S::K * 256 : 0);
                    const uint4 *cb = op.w[Op::kLayers > 1 ? layer_of(s) : 0].cb;
                    // kTr: a row past the layer is zero, whatever its padding code selects
                    auto real = [&](int r) { return live && (!kTr || tile_of(s) * 8 + r < L.out); };
                    if constexpr (kScaleW) {
                        const uint32_t mine = float_to_half_bits(half_bits_to_float(scale_ring[u]) * inv);
                        auto put = [&](int r, uint4 v) {
                            const uint32_t h = __shfl_sync(0xffffffffu, mine, (rt_l & 1) * 8 + r);
                            const __half2 h2 = __half2half2(__ushort_as_half((uint16_t)h));
                            uint32_t p[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const __half2 m = __hmul2(*reinterpret_cast<__half2 *>(&p[j]), h2);
                                p[j] = real(r) ? *reinterpret_cast<const uint32_t *>(&m) : 0u;
                            }
                            *reinterpret_cast<uint4 *>(A + slot_of(r)) = make_uint4(p[0], p[1], p[2], p[3]);
                        };
                        uint4 tt[8][S::K];
#pragma unroll
                        for (int r = 0; r < 8; ++r) gather_terms<S>(code, r, books, cb, tt[r]);
#pragma unroll
                        for (int r = 0; r < 8; ++r) put(r, sum_round_fast_h8<S::K>(tt[r]));
                    } else if constexpr (kAsyncWeights) {
                        const uint32_t a0 = smem_u32(A);
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            const bool in = real(r);
                            cp_async16(a0 + slot_of(r), in ? (const void *)(cb + code.code(r, 0)) : (const void *)cb,
                                       in ? 16u : 0u);
                        }
                    } else if constexpr (S::K <= 2) {
                        // all codeword reads before the first tile store (the
                        // books and the tile share one shared array)
                        uint4 tt[8][S::K];
#pragma unroll
                        for (int r = 0; r < 8; ++r) gather_terms<S>(code, r, books, cb, tt[r]);
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            *reinterpret_cast<uint4 *>(A + slot_of(r)) =
                                real(r) ? sum_round_fast_h8<S::K>(tt[r]) : make_uint4(0, 0, 0, 0);
                    } else {
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            uint4 tt[S::K];
                            gather_terms<S>(code, r, books, cb, tt);
                            *reinterpret_cast<uint4 *>(A + slot_of(r)) =
                                real(r) ? sum_round_fast_h8<S::K>(tt) : make_uint4(0, 0, 0, 0);
                        }
                    }
                }
                if constexpr (kAsyncWeights) cp_async_arrive(&full_a[s % kWsAStages]);
                else publish(s);
                // the next requests follow the fence, which would wait for them
                code_ring[u] = fetch(s + NG * kCodeAhead);
                if constexpr (kScaleW) scale_ring[u] = fetch_scale(s + NG * kCodeAhead);
            }
        }
        cp_async_wait<0>();
        grid_dependency_wait();  // y, the scales and the workspace
        // ---------------- epilogue ----------------
        const bool got = (*abort_v == 0) && mbar_wait_ns(acc_full, 0, kWaitNs);
        if (!got) *abort_v = 1;
        tc_fence_after();
    }
    grid_dependency_wait();  // every thread, before the workspace and y
    __syncthreads();
    if (*abort_v) {
        // something gave up: record it and drain what was issued (bounded)
        if (tid == 0) record_status(ws, AQ_ERR_TIMEOUT);
        if (tid == 32) mbar_wait_ns(acc_full, 0, kWaitNs);
        if (tid == 0 && half == 0)  // (pair: the leader's barriers cover both CTAs' copies)
            for (int s = max(0, nk - kWsStages); s < nk; ++s)
                mbar_wait_ns(&full_b[s % kWsStages], (s / kWsStages) & 1, kWaitNs);
    }
    if constexpr (kTr && !kScaleW)
        if (op.factor) {
            out.factor = __ldcg(op.factor);
            if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) *op.top = 0u;
        }
    // The decoder warps finish: warp & 3 is the TMEM lane quarter, the NG
    // warps of a quarter take alternate blocks of 64 columns (PlainOp: 16).
    // After a timeout no tensor memory is read and the output is incomplete,
    // which the status word reports; the barriers and counters are still served.
    bool finish = warp >= 2 && *abort_v == 0;
    const uint32_t tq = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int r = (warp & 3) * 32 + lane;
    constexpr size_t kSlice = kBM * BN / 4;  // float4 per slice
    constexpr int kCols = Op::kStaged ? 64 : 16;
    int c = kCols * ((warp - 2) / 4), end = BN, ks = 1;
    const float4 *slices = nullptr;
    unsigned *counter = nullptr;
    tc_fence_after();
    if (cluster_ks > 1) {
        ks = cluster_ks;
        const int cw = BN / ks;  // columns each split owns (a multiple of 16)
        float4 *mine = reinterpret_cast<float4 *>(sp.partials) + ((size_t)blockIdx.y * gridDim.x + blockIdx.x) * ks * kSlice;
        slices = mine;
        if (finish) {
            publish_sums<BN>(mine + (size_t)z * kSlice, tq, 16 * ((warp - 2) / 4), 16 * NG, z * cw, (z + 1) * cw, T - n0, r);
            fence_acq_rel_gpu();
        }
        cluster_sync_all();  // every split's sums are in L2 (every thread, also after a timeout)
        c += z * cw;
        end = (z + 1) * cw;
    } else if (tail_idx >= 0) {
        ks = tm.ks;
        float4 *mine = reinterpret_cast<float4 *>(reinterpret_cast<char *>(ws) + kWsData) + (size_t)tail_idx * ks * kSlice;
        slices = mine;
        counter = reinterpret_cast<unsigned *>(reinterpret_cast<char *>(ws) + kWsHeader) + tail_idx;
        if (finish) publish_sums<BN>(mine + (size_t)z * kSlice, tq, 16 * ((warp - 2) / 4), 16 * NG, 0, 0, T - n0, r);
        __syncthreads();
        if (tid == 0) {
            // the barrier orders the CTA's slice stores before this increment,
            // whose release publishes them; its acquire orders the last CTA's
            // reads after every split's
            const unsigned prev = atom_add_acq_rel_gpu(counter, 1u);
            *last_flag = (prev == (unsigned)ks - 1u) ? 1u : 0u;
        }
        __syncthreads();
        if (!*reinterpret_cast<volatile uint32_t *>(last_flag)) finish = false, counter = nullptr;
    }
    if (finish) {
        const Splits<BN> splits{slices + r, ks, z};
        if constexpr (Op::kStaged)
            op.dispatch([&](auto family, auto grad) {
                finish_staged<decltype(family)::value, decltype(grad)::value, BN>(
                    op, L, out, &maps.m[Op::kXMaps], smem, in_bar, ws, tq, c, kCols * NG, end, splits);
            });
        else
            finish_direct<BN>(op, L, out, tq, c, kCols * NG, end, splits);
    }
    if (counter && tid == 0) *counter = 0u;
    tc_fence_before();
    __syncthreads();
    if constexpr (Pair) {
        cluster_sync_all();  // neither CTA's shared or tensor memory is in use by the other
        if (warp == 0) tmem_dealloc_pair(tmem, BN);
    } else {
        if (warp == 0) tmem_dealloc(tmem, BN);
    }
}

}  // namespace aqk

namespace aqh {
using namespace aqk;

// Launch plan: token tile, split-K, workspace.
struct GemmPlan {
    int bn;           // tokens per CTA: 512 above 256 tokens, else 256
    int mtiles, ntiles;
    int ks;           // splits of the contraction (blockIdx.z)
    int per_split;    // 64-deep stages per split
    bool cluster;     // the splits form one cluster and finish on chip
    TailMap tail;     // ks > 0: the tail mode's 1-D grid
    bool pair;        // CTA pairs of two row tiles (mtiles counts pairs)
    size_t ws_bytes;  // status word + tile counters + fp32 partials
};

// `mtiles` row tiles, `nst` stages of the contraction; `max_bn` where the
// shared memory does not hold 512-token tiles; `pairs`: the operator may run
// as CTA pairs (and finishes 64 columns at a time).
inline GemmPlan plan_ws(int mtiles, int nst, int T, int max_bn = 512, bool pairs = false)
{
    GemmPlan p{};
    p.ws_bytes = kWsHeader;
    p.mtiles = mtiles;
    // 512-token tiles halve the decode work per MMA; when they would leave
    // more than half the SMs without a tile (and so need a deep split of
    // the contraction, whose partial sums cost a pass through L2),
    // 256-token tiles with fewer splits are faster (measured on Llama-2-7B
    // shapes at 512 tokens)
    // 512-token tiles halve the decode work per MMA; with few row tiles
    // (a 4096-row layer at 512 tokens) they need a split of the
    // contraction, which the cluster finish makes cheap
    p.bn = T >= 384 || (T > 256 && (long)p.mtiles * ((T + 511) / 512) * 2 >= kNumSMs) ? 512 : 256;
    p.bn = std::min(p.bn, max_bn);
    p.ntiles = (T + p.bn - 1) / p.bn;
    long tiles = (long)p.mtiles * p.ntiles, slots = kNumSMs;  // tiles and how many of them run at once
    // 512-token tiles run as CTA pairs where a split in two at most fills
    // the GPU (a cluster of a pair and four splits holds eight CTAs, of which
    // only 15 fit at once)
    if (pairs && p.bn == 512) {
        const long t2 = (long)((mtiles + 1) / 2) * p.ntiles;
        if (t2 * 4 > kNumSMs / 2) {
            p.pair = true;
            p.mtiles = (mtiles + 1) / 2;
            tiles = t2;
            slots = kNumSMs / 2;
        }
    }
    const size_t slice = (size_t)kBM * p.bn * sizeof(float) * (p.pair ? 2 : 1);  // fp32 sums of a tile
    // the decode is the bound: split the contraction until about one CTA
    // per SM works, keeping at least 8 stages per split
    int ks = tiles < slots ? (int)(slots / tiles) : 1;
    ks = std::max(1, std::min(ks, nst / 8));
    // the split runs as one thread-block cluster along z whose CTAs share
    // the finish: 2, 4 or 8 CTAs (the largest power of two not above ks).
    // With at least 8 stages per split (nst >= 8 kc) none of them is empty:
    // per = ceil(nst / kc) gives exactly kc non-empty splits
    if (ks >= 2) {
        // (staged operators own whole blocks of 64 columns per split, and take
        // 8 splits only where all their clusters run at once: 15 of 8 full-SM
        // CTAs fit; 18 clusters measured 2x the time of a split in 4)
        const int most = p.pair ? 2 : !pairs ? 8 : (p.bn < 512 || tiles > 15) ? 4 : 8;
        int kc = 2;
        while (kc * 2 <= std::min(ks, most)) kc *= 2;
        ks = kc;
    }
    p.per_split = (nst + ks - 1) / ks;
    p.ks = (nst + p.per_split - 1) / p.per_split;
    p.cluster = p.ks > 1;
    if (p.ks > 1) p.ws_bytes = kWsData + (size_t)p.ks * tiles * slice;
    // more tiles than one wave, the last wave at most half full: its tiles'
    // contraction is split so that it fills the SMs (Llama-2-7B MLP
    // rows at 2048 tokens: 344 tiles, 48 in the third wave, split 3 ways)
    if (p.ks == 1 && tiles > slots) {
        const long tail = tiles % slots;
        if (tail > 0 && tail * 2 <= slots && tail * (p.pair ? 2 : 1) <= kWsMaxCounters) {
            int kt = std::min((int)(slots / tail), std::min(nst / 8, 8));
            if (kt >= 2) {
                const int per = (nst + kt - 1) / kt;
                kt = (nst + per - 1) / per;  // no empty split
                p.tail = TailMap{(int)(tiles - tail), kt, per};
                p.ws_bytes = kWsData + (size_t)tail * kt * slice;
            }
        }
    }
    return p;
}

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
    return fn;
}

// Activations [rows][T] binary16, rows `pitch` elements apart (a multiple of
// 8): innermost dimension tokens, box 64 tokens x `height` rows.
inline bool token_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap *map, const uint16_t *x, int rows, int T,
                      int pitch, int height = kBK)
{
    cuuint64_t dims[2] = {(cuuint64_t)T, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)pitch * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)height};
    cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<uint16_t *>(x), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The maps of a staged operator's arrays, rows `pitch` elements apart.
template <class Op>
bool io_maps(PFN_cuTensorMapEncodeTiled_v12000 encode, TensorMaps<Op::kMaps> *maps, const Op &op, const Geom &g, int T,
             int pitch)
{
    for (int i = 0; i < 3; ++i)
        if (op.io(i) && !token_map(encode, &maps->m[Op::kXMaps + i], op.io(i), op.rows(g), T, pitch, Op::kRows))
            return false;
    return true;
}

template <class S, int BN, class Op, bool Pair>
constexpr int gemm_ws_smem_bytes()
{
    constexpr int BB = kWsBookBytes<S, Op>;
    constexpr int NA = kWsAStagesOf<S, BN, BB, Pair>, NB = kWsStagesOf<S, BN, BB, Pair>;
    return 1024 + NA * kTileABytes + NB * (kBK * BN * 2 / (Pair ? 2 : 1)) + BB + ((Pair ? 3 : 2) * NA + 2 * NB + 1 + kInBoxes<Op, BN>) * 8 + 32;
}

// 512-token tiles of two layers' 8x8 codebooks (64 KiB) do not fit.
template <class S, class Op>
constexpr int kWsMaxBN = kWsBookBytes<S, Op> > 32768 ? 256 : 512;

template <class Op>
int ws_max_bn(const Geom &g)
{
    int bn = 512;
    with_scheme(g, [&](auto sch) {
        bn = kWsMaxBN<decltype(sch), Op>;
        return cudaSuccess;
    });
    return bn;
}

template <class S, class Op>
cudaError_t launch_ws_scheme(const Geom &g, const GemmPlan &p, const TensorMaps<Op::kMaps> &maps, const Op &op, int T,
                      void *ws, cudaStream_t s, bool pdl)
{
    const long tiles = (long)p.mtiles * p.ntiles;
    const unsigned width = p.pair ? 2 : 1;  // CTAs per tile
    const dim3 grid = p.tail.ks > 0 ? dim3(width * (unsigned)(p.tail.full + (tiles - p.tail.full) * p.tail.ks), 1, 1)
                                    : dim3(width * p.mtiles, p.ntiles, p.ks);
    GemmSplit sp{nullptr};
    if (p.ks > 1) sp.partials = reinterpret_cast<float *>(reinterpret_cast<char *>(ws) + kWsData);
    auto launch = [&](auto bn, auto pair) {
        constexpr int BN = decltype(bn)::value;
        constexpr bool Pair = decltype(pair)::value;
        if constexpr (BN > kWsMaxBN<S, Op>) {
            return cudaErrorInvalidValue;
        } else {
            constexpr int smem = gemm_ws_smem_bytes<S, BN, Op, Pair>();
            static_assert(smem <= 227 * 1024, "shared memory of the warp-specialised GEMM");
            auto kern = gemm_ws_kernel<S, BN, Op, Pair>;
            cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = grid;
            cfg.blockDim = dim3(kWsThreadsOf<S>);
            cfg.dynamicSmemBytes = smem;
            cfg.stream = s;
            cudaLaunchAttribute attr[2];
            int na = 0;
            if (p.cluster || Pair) {
                attr[na].id = cudaLaunchAttributeClusterDimension;
                attr[na].val.clusterDim.x = width;
                attr[na].val.clusterDim.y = 1;
                attr[na].val.clusterDim.z = p.cluster ? p.ks : 1;
                ++na;
            }
            if (pdl) {
                attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
                attr[na].val.programmaticStreamSerializationAllowed = 1;
                ++na;
            }
            cfg.attrs = attr;
            cfg.numAttrs = na;
            e = cudaLaunchKernelEx(&cfg, kern, maps, g, op, T, ws, sp, p.per_split, p.cluster ? p.ks : 0, p.tail);
            if (e != cudaSuccess) return e;
            return cudaGetLastError();
        }
    };
    if constexpr (Op::kPairs)
        if (p.pair) return launch(std::integral_constant<int, 512>{}, std::true_type{});
    return p.bn == 512 ? launch(std::integral_constant<int, 512>{}, std::false_type{})
                       : launch(std::integral_constant<int, 256>{}, std::false_type{});
}

template <class Op>
cudaError_t launch_ws(const Geom &g, const GemmPlan &p, const TensorMaps<Op::kMaps> &maps, const Op &op, int T,
                      void *ws, cudaStream_t s, bool pdl)
{
    return with_scheme(g, [&](auto sch) { return launch_ws_scheme<decltype(sch)>(g, p, maps, op, T, ws, s, pdl); });
}

}  // namespace aqh
