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
//              straight into the swizzled A tile by 16-byte cp.async, a few
//              stages ahead; 2x8: codewords come from the codebooks in
//              shared memory, summed with binary16 adds.  Each thread fences
//              its writes to the async proxy and arrives on full_a[stage]
//              (128 arrivals).  The epilogue reads TMEM lanes 32*(warp%4)..
//              with tcgen05.ld and hands each row's sums, 16 tokens at a
//              time, to the operator.
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
//    contraction index and is multiplied into the weights (one rounding to
//    binary16 each, after division by the power of two 2^E just above the
//    largest scale, so that nothing overflows and uniformly small scales
//    lose no bits; 2^E is applied to the fp32 sums).
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
template <class S, int BN, int BB>
constexpr int kWsStagesOf = (BN == 512) ? 2 : (BB > 8192 || (S::K == 1 && S::B == 16)) ? 3 : 4;
// The W (decoded) tiles have a ring of their own, 5 deep (4 with the 32 KiB
// of 8x8 codebooks): with 512-token X tiles taking 64 KiB a stage, a shared
// ring would be 2 deep.  The 1x16 decoders (two groups of 128 threads, two
// of each group's stages in flight: about 4000 codeword reads per CTA) need
// the depth; at 256-token tiles 1x16 trades an X stage for two W stages
// (6 W, 3 X).
template <class S, int BN, int BB>
constexpr int kWsAStagesOf = (BN == 512) ? ((BB > 16384) ? 4 : 5)
                                         : ((S::K == 1 && S::B == 16) ? 6 : kWsStagesOf<S, BN, BB>);
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
constexpr int kWsLag = 2;                     // cp.async stages in flight per decoder (< ring depth)

// Layers whose 8-bit codebooks a CTA keeps in shared memory.
template <class S, class Op>
constexpr int kWsBookBytes = S::kSmemBookBytes * Op::kLayers;

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

// ---- rows of binary16 arrays, 16 tokens of R consecutive rows per warp --------
//
// R = 32: lane l has all 16 tokens of row l; R = 16: lane l has tokens
// 8 (l / 16) .. + 7 of row l % 16.  With T a multiple of 8 the lane reads and
// writes its 16-byte pieces directly.  Otherwise rows start at any even
// address: the block passes through a per-warp kilobyte of shared memory so
// that each access covers 32 consecutive bytes of a row (one row per lane
// would touch a sector for every 2-byte element).  `load` requests a block,
// `settle` later brings what arrived into the lane's own pieces.
template <int R>
struct RowBlock {
    static constexpr int kPieces = R / 16;  // 16-byte pieces per lane
    uint4 p[kPieces];
};

template <int R>
struct RowIO {
    int T, row0, row_end;  // tokens (row pitch), the warp's first row, one past the array's last
    uint8_t *scratch;      // 1 KiB per warp
    bool vec;              // T % 8 == 0

    __device__ __forceinline__ int lane() const { return threadIdx.x & 31; }
    __device__ __forceinline__ int row() const { return row0 + (R == 32 ? lane() : (lane() & 15)); }
    __device__ __forceinline__ int first() const { return R == 32 ? 0 : 8 * (lane() >> 4); }  // lane's first token

    // Tokens gn .. gn + 15 (zeros past T or the last row), not yet settled:
    // element lane + 32 i of the block in half-word i when T is ragged.
    __device__ __forceinline__ RowBlock<R> load(const uint16_t *base, int gn) const
    {
        RowBlock<R> b;
#pragma unroll
        for (int i = 0; i < b.kPieces; ++i) b.p[i] = make_uint4(0u, 0u, 0u, 0u);
        if (vec) {
            if (row() < row_end) {
                const uint4 *src = reinterpret_cast<const uint4 *>(base + (size_t)row() * T + gn + first());
#pragma unroll
                for (int i = 0; i < b.kPieces; ++i)
                    if (gn + first() + 8 * i < T) b.p[i] = __ldcg(src + i);
            }
        } else {
            uint32_t h[R / 2];
            const int r = row0 + (lane() >> 4), c = gn + (lane() & 15);  // rows r, r + 2, ...
            const uint16_t *src = base + (size_t)r * T + c;
#pragma unroll
            for (int i = 0; i < R / 2; ++i, src += 2 * (size_t)T)
                h[i] = (r + 2 * i < row_end && c < T) ? (uint32_t)__ldcg(src) : 0u;
#pragma unroll
            for (int i = 0; i < b.kPieces; ++i)
                b.p[i] = make_uint4(h[8 * i] | (h[8 * i + 1] << 16), h[8 * i + 2] | (h[8 * i + 3] << 16),
                                    h[8 * i + 4] | (h[8 * i + 5] << 16), h[8 * i + 6] | (h[8 * i + 7] << 16));
        }
        return b;
    }

    __device__ __forceinline__ RowBlock<R> settle(RowBlock<R> b) const
    {
        if (!vec) {
            uint16_t *sh = reinterpret_cast<uint16_t *>(scratch);
#pragma unroll
            for (int i = 0; i < R / 2; ++i)
                sh[lane() + 32 * i] = (uint16_t)(u4_at(b.p[i / 8], (i % 8) / 2) >> (16 * (i & 1)));
            __syncwarp();
            const uint4 *mine = reinterpret_cast<const uint4 *>(sh + (row() - row0) * 16 + first());
#pragma unroll
            for (int i = 0; i < b.kPieces; ++i) b.p[i] = mine[i];
            __syncwarp();
        }
        return b;
    }

    __device__ __forceinline__ void put(uint16_t *base, int gn, const RowBlock<R> &b) const
    {
        if (vec) {
            if (row() < row_end) {
                uint4 *dst = reinterpret_cast<uint4 *>(base + (size_t)row() * T + gn + first());
#pragma unroll
                for (int i = 0; i < b.kPieces; ++i)
                    if (gn + first() + 8 * i < T) dst[i] = b.p[i];
            }
        } else {
            uint16_t *sh = reinterpret_cast<uint16_t *>(scratch);
            uint4 *mine = reinterpret_cast<uint4 *>(sh + (row() - row0) * 16 + first());
#pragma unroll
            for (int i = 0; i < b.kPieces; ++i) mine[i] = b.p[i];
            __syncwarp();
            const int r = row0 + (lane() >> 4), c = gn + (lane() & 15);
            uint16_t *dst = base + (size_t)r * T + c;
#pragma unroll
            for (int i = 0; i < R / 2; ++i, dst += 2 * (size_t)T)
                if (r + 2 * i < row_end && c < T) *dst = sh[lane() + 32 * i];
            __syncwarp();
        }
    }

    // The same block into an array whose rows are `pitch` (T rounded up to 8) apart.
    __device__ __forceinline__ void put_padded(uint16_t *base, int pitch, int gn, const RowBlock<R> &b) const
    {
        if (row() < row_end) {
            uint4 *dst = reinterpret_cast<uint4 *>(base + (size_t)row() * pitch + gn + first());
#pragma unroll
            for (int i = 0; i < b.kPieces; ++i)
                if (gn + first() + 8 * i < pitch) dst[i] = b.p[i];
        }
    }
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

// Where a tile's sums are written: the tile, its tokens and the epilogue
// warp's scratch.
struct TileOut {
    int mt, n0, T;
    uint8_t *scratch;  // this warp's kilobyte of the (idle) W ring
    float factor;      // kTransposed: 2^E
};

// ---- operators ----------------------------------------------------------------

// y = RN16(s (W x)); T % 8 == 0.
struct PlainOp {
    static constexpr bool kGated = false, kTransposed = false;
    static constexpr int kLayers = 1, kMaps = 1, kRows = 32, kAhead = 4;
    LayerWeights w[1];
    uint16_t *y;

    struct Row {
        RowIO<32> io;
        float sc;
    };
    __device__ __forceinline__ Row row(const Geom &L, const TileOut &o) const
    {
        Row r;
        r.io = RowIO<32>{o.T, o.mt * kBM + (int)((threadIdx.x >> 5) & 3) * 32, L.out, o.scratch, true};
        const int i = r.io.row();
        r.sc = (i < L.out && w[0].scales) ? half_bits_to_float(w[0].scales[i]) : 1.f;
        return r;
    }
    __device__ __forceinline__ RowBlock<32> input(const Row &, int) const { return RowBlock<32>{}; }
    __device__ __forceinline__ void store(const Row &r, int gn, float (&v)[16], const RowBlock<32> &) const
    {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= r.sc;
        RowBlock<32> b;
        b.p[0] = round_h8(v);
        b.p[1] = round_h8(v + 8);
        r.io.put(y, gn, b);
    }
};

// y = RN16(act(s (W x) + bias) + residual), or, with gy: grad_z = RN16(gy
// act'(z)) and the sums of gy act'(z) over each block of 16 tokens.
struct FusedOp {
    static constexpr bool kGated = false, kTransposed = false;
    static constexpr int kLayers = 1, kMaps = 1, kRows = 32, kAhead = 2;
    LayerWeights w[1];
    int act;
    const uint16_t *bias;  // or null
    const uint16_t *in;    // residual, or gy (grad); or null
    uint16_t *out;         // y, or grad_z
    bool grad;
    uint16_t *padded;      // grad, ragged T: a second copy of grad_z, rows `pitch` apart
    int pitch;
    float *sums;           // grad: [blocks of 16 tokens][out], or null

    struct Row {
        RowIO<32> io;
        float sc, b;
    };
    __device__ __forceinline__ Row row(const Geom &L, const TileOut &o) const
    {
        Row r;
        r.io = RowIO<32>{o.T, o.mt * kBM + (int)((threadIdx.x >> 5) & 3) * 32, L.out, o.scratch, (o.T & 7) == 0};
        const int i = r.io.row();
        r.sc = (i < L.out && w[0].scales) ? half_bits_to_float(w[0].scales[i]) : 1.f;
        r.b = (i < L.out && bias) ? half_bits_to_float(bias[i]) : 0.f;
        return r;
    }
    __device__ __forceinline__ RowBlock<32> input(const Row &r, int gn) const
    {
        return in ? r.io.load(in, gn) : RowBlock<32>{};
    }
    __device__ __forceinline__ void store(const Row &r, int gn, float (&v)[16], const RowBlock<32> &raw) const
    {
        RowBlock<32> x{}, b;
        if (in) x = r.io.settle(raw);
        float sum = 0.f;
        // eight tokens at a time: sixteen activations in flight would not fit the registers
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            float a[8], e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = fmaf(r.sc, h ? v[j + 8] : v[j], r.b);
            widen_h8(h ? x.p[1] : x.p[0], e);
            if (!grad) {
                act_values(act, a);
                if (in) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) a[j] += e[j];
                }
            } else {
                float slope[8];
                act_values_slopes(act, a, slope);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    a[j] = e[j] * slope[j];
                    if (gn + 8 * h + j < r.io.T) sum += a[j];
                }
            }
            if (h) b.p[1] = round_h8(a);
            else b.p[0] = round_h8(a);
        }
        if (sums && r.io.row() < r.io.row_end) sums[(size_t)(gn >> 4) * r.io.row_end + r.io.row()] = sum;
        r.io.put(out, gn, b);
        if (padded) r.io.put_padded(padded, pitch, gn, b);
    }
};

// Gated block: y = RN16(act(g) u), or, with gy, the gradients of g and u.
struct GatedOp {
    static constexpr bool kGated = true, kTransposed = false;
    static constexpr int kLayers = 2, kMaps = 1, kRows = 16, kAhead = 4;
    LayerWeights w[2];  // gate, up
    int act;
    const uint16_t *gy;      // or null: forward
    uint16_t *out0, *out1;   // y, -; or grad_gate, grad_up
    uint16_t *padded0, *padded1;  // grad, ragged T: second copies, rows `pitch` apart
    int pitch;

    struct Row {
        RowIO<16> io;
        float sc;
    };
    __device__ __forceinline__ Row row(const Geom &L, const TileOut &o) const
    {
        // lanes 0-15: gate rows, 16-31: the same rows of up
        Row r;
        r.io = RowIO<16>{o.T, o.mt * (kBM / 2) + (int)((threadIdx.x >> 5) & 3) * 16, L.out, o.scratch, (o.T & 7) == 0};
        const uint16_t *s = (threadIdx.x & 16) ? w[1].scales : w[0].scales;
        r.sc = (r.io.row() < L.out && s) ? half_bits_to_float(s[r.io.row()]) : 1.f;
        return r;
    }
    __device__ __forceinline__ RowBlock<16> input(const Row &r, int gn) const
    {
        return gy ? r.io.load(gy, gn) : RowBlock<16>{};
    }
    // Lane l < 16 (gate) gives its tokens 8-15 to lane l + 16 (up) for that
    // lane's tokens 0-7: each then has eight tokens of both projections.
    __device__ __forceinline__ void store(const Row &r, int gn, float (&v)[16], const RowBlock<16> &raw) const
    {
        const bool hi = threadIdx.x & 16;
        float e[8], a[8], c[8];
        if (gy) widen_h8(r.io.settle(raw).p[0], e);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float lo_v = r.sc * v[j], hi_v = r.sc * v[j + 8];
            const float got = __shfl_xor_sync(0xffffffffu, hi ? lo_v : hi_v, 16);
            a[j] = hi ? got : lo_v;   // gate
            c[j] = hi ? hi_v : got;   // up
        }
        RowBlock<16> b;
        if (!gy) {
            act_values(act, a);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] *= c[j];
            b.p[0] = round_h8(a);
            r.io.put(out0, gn, b);
        } else {
            float slope[8];
            act_values_slopes(act, a, slope);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float u = c[j];
                c[j] = e[j] * a[j];
                a[j] = e[j] * u * slope[j];
            }
            b.p[0] = round_h8(a);
            r.io.put(out0, gn, b);
            if (padded0) r.io.put_padded(padded0, pitch, gn, b);
            b.p[0] = round_h8(c);
            r.io.put(out1, gn, b);
            if (padded1) r.io.put_padded(padded1, pitch, gn, b);
        }
    }
};

// gx = RN16(sum over the layers of W^T (s gy)).
struct BackOp {
    static constexpr bool kGated = false, kTransposed = true;
    static constexpr int kLayers = 2, kMaps = 2, kRows = 32, kAhead = 4;
    LayerWeights w[2];
    int layers;  // 1 or 2
    uint16_t *gx;

    struct Row {
        RowIO<32> io;
        float sc;
    };
    __device__ __forceinline__ Row row(const Geom &L, const TileOut &o) const
    {
        return Row{RowIO<32>{o.T, o.mt * kBM + (int)((threadIdx.x >> 5) & 3) * 32, L.in, o.scratch, (o.T & 7) == 0},
                   o.factor};
    }
    __device__ __forceinline__ RowBlock<32> input(const Row &, int) const { return RowBlock<32>{}; }
    __device__ __forceinline__ void store(const Row &r, int gn, float (&v)[16], const RowBlock<32> &) const
    {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= r.sc;
        RowBlock<32> b;
        b.p[0] = round_h8(v);
        b.p[1] = round_h8(v + 8);
        r.io.put(gx, gn, b);
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

// Runs the operator over this warp's blocks of 16 tokens: columns c, c +
// step, ... below `end`, the sums of a block from `sums(c, v)`.  The
// operator's own input of a block is requested two blocks ahead.
template <class Op, class F>
__device__ __forceinline__ void finish_blocks(const Op &op, const Geom &L, const TileOut &o, int c, int step, int end,
                                              F &&sums)
{
    const typename Op::Row row = op.row(L, o);
    end = min(end, o.T - o.n0);
    RowBlock<Op::kRows> in[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (c + i * step < end) in[i] = op.input(row, o.n0 + c + i * step);
#pragma unroll 1
    for (; c < end; c += 2 * step) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int ci = c + i * step;
            if (ci >= end) break;  // warp-uniform
            float v[16];
            sums(ci, v);
            const RowBlock<Op::kRows> x = in[i];
            if (ci + 2 * step < end) in[i] = op.input(row, o.n0 + ci + 2 * step);
            op.store(row, o.n0 + ci, v, x);
        }
    }
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

// Largest |v| (as the bits of a binary16; NaN above infinity) of this
// thread's share of v[0 .. n), `threads` threads in all.
__device__ __forceinline__ uint32_t absmax_share(const uint16_t *__restrict__ v, int n, int thread, int threads)
{
    uint32_t m = 0;
    // 16-byte pieces between the ragged ends (v has 2-byte alignment)
    const int head = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(v) & 15)) & 15) / 2);
    const int nv = (n - head) / 8;
    const uint4 *v4 = reinterpret_cast<const uint4 *>(v + head);
#pragma unroll 8
    for (int i = thread; i < nv; i += threads) {
        const uint4 q = __ldg(v4 + i);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, max(w[j] & 0x7fffu, (w[j] >> 16) & 0x7fffu));
    }
    if (thread < head) m = max(m, (uint32_t)v[thread] & 0x7fffu);
    if (head + nv * 8 + thread < n && thread < 8) m = max(m, (uint32_t)v[head + nv * 8 + thread] & 0x7fffu);
    return m;
}

// Barrier of the decoder threads alone (the CTA's other warps do not take part).
__device__ __forceinline__ void decoder_barrier(int threads)
{
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
}

template <class S, int BN, class Op>
__global__ void __launch_bounds__(kWsThreadsOf<S>, 1)
gemm_ws_kernel(const __grid_constant__ TensorMaps<Op::kMaps> maps, Geom L, const __grid_constant__ Op op, int T,
               void *ws, GemmSplit sp, int stages_per_split, int cluster_ks, TailMap tm)
{
    constexpr int BB = kWsBookBytes<S, Op>;
    constexpr int kWsStages = kWsStagesOf<S, BN, BB>;    // X ring
    constexpr int kWsAStages = kWsAStagesOf<S, BN, BB>;  // W ring
    constexpr int kWsTileB = kBK * BN * 2;   // 32 or 64 KiB
    constexpr int kN = BN < 256 ? BN : 256;  // N of one MMA instruction
    constexpr int NG = kWsGroupsOf<S>;       // decoder groups
    constexpr bool kTr = Op::kTransposed;
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
    uint64_t *acc_full = empty_a + kWsAStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_full + 1);
    uint32_t *abort_flag = tmem_slot + 1;
    uint32_t *scale_max = abort_flag + 1;       // kTransposed: largest |s| (binary16 bits)
    uint32_t *last_flag = scale_max + 1;        // the last split of a tail tile

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int layer_stages = ws_layer_stages<Op>(L);
    int all_stages = layer_stages;
    if constexpr (kTr) all_stages *= op.layers;
    // the CTA's tile and split: a 3-D grid (row tile, token tile, split), or
    // the tail mode's 1-D grid
    int mt = blockIdx.x, nt = blockIdx.y, z = blockIdx.z, per = stages_per_split, tail_idx = -1;
    if (tm.ks > 0) {
        const int mtiles = ws_mtiles<Op>(L);
        int tile = blockIdx.x;
        z = 0;
        per = all_stages;
        if (tile >= tm.full) {
            const int rr = tile - tm.full;
            tail_idx = rr / tm.ks;
            z = rr % tm.ks;
            tile = tm.full + tail_idx;
            per = tm.per;
        }
        mt = tile % mtiles;
        nt = tile / mtiles;
    }
    const int n0 = nt * BN;
    // this split's stages: global stages s0 .. s0 + nk - 1
    const int s0 = z * per;
    const int nk = max(0, min(all_stages, s0 + per) - s0);

    // 1x16: codewords go from L2 into the tile by cp.async, copies of kWsLag
    // stages in flight; other schemes, and the transposed product (whose
    // weights are scaled on the way), decode in registers
    constexpr bool kAsyncWeights = (S::K == 1 && S::B == 16) && !kTr;
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
            mbar_init(&full_a[s], 128);
            mbar_init(&empty_a[s], 1);
        }
        for (int s = 0; s < kWsStages; ++s) {
            mbar_init(&full_b[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        *abort_flag = 0;
        *scale_max = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(tmem_slot, BN);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    volatile uint32_t *abort_v = abort_flag;
    TileOut out{mt, n0, T, tileA + (warp >= 2 ? warp - 2 : 0) * 1024, 1.f};
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
                mbar_arrive_expect_tx(&full_b[buf], kWsTileB);
                const uint32_t dst = smem_u32(tileB + buf * kWsTileB);
                int row = (s0 + s) * kBK;
                const CUtensorMap *map = &maps.m[0];
                if constexpr (Op::kMaps > 1)
                    if (s0 + s >= layer_stages) {
                        map = &maps.m[1];
                        row -= layer_stages * kBK;
                    }
#pragma unroll
                for (int q = 0; q < BN / 64; ++q)
                    tma_load_2d(dst + q * (kBK * 128), map, n0 + 64 * q, row, &full_b[buf]);
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        if (lane == 0) {
            const uint32_t idesc = make_idesc(kBM, kN, true) | (kTr ? 1u << 15 : 0u);  // kTr: A MN-major
            int s = 0;
            for (; s < nk; ++s) {
                const int buf = s % kWsStages, abuf = s % kWsAStages;
                if (!mbar_wait_ns(&full_a[abuf], (s / kWsAStages) & 1, kWaitNs) ||
                    !mbar_wait_ns(&full_b[buf], (s / kWsStages) & 1, kWaitNs)) {
                    *abort_v = 1;
                    break;
                }
                if (*abort_v) break;
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
                        // tokens 256 h .. : four 64-token boxes further on
                        const uint64_t bd = smem_desc_sw128(b0 + h * (kN / 64) * (kBK * 128) + ks * 2048, kBK * 128, 1024);
                        mma_f16_ss(tmem + h * kN, ad, bd, idesc, (s > 0 || ks > 0) ? 1u : 0u);
                    }
                }
                mma_commit(&empty[buf]);     // X buffer free once these MMAs complete
                mma_commit(&empty_a[abuf]);  // and the W buffer
            }
            mma_commit(acc_full);  // completes when every MMA issued above has
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
        // kTransposed: the rows' scales divided by 2^E, one per lane (rows of
        // the warp's two row tiles), as far ahead as the codes
        float inv = 1.f;
        uint32_t scale_ring[kCodeAhead];
        auto fetch_scale = [&](int s) -> uint32_t {
            const int l = layer_of(s), o = (tile_of(s) - (rt_l & 1)) * 8 + (lane & 15);
            if (s >= nk || o >= L.out) return 0u;  // rows past the layer weigh nothing
            const uint16_t *sc = op.w[l].scales;
            return (uint32_t)float_to_half_bits(sc ? half_bits_to_float(__ldg(sc + o)) * inv : inv);
        };
        uint4 ahead[8];  // kTransposed, one 16-bit codebook: the next stage's codewords
        constexpr bool kGatherAhead = kTr && S::K == 1 && S::B == 16;
        if constexpr (kTr) {
            if constexpr (kGatherAhead) {
#pragma unroll
                for (int r = 0; r < 8; ++r) ahead[r] = ldg_nc_v4(op.w[layer_of(dg)].cb + code_ring[0].code(r, 0));
            }
            grid_dependency_wait();  // the scales
            uint32_t m = 0;
            for (int l = 0; l < op.layers; ++l)
                m = max(m, op.w[l].scales ? absmax_share(op.w[l].scales, L.out, tid - 64, 128 * NG) : 0x3c00u);
            m = __reduce_max_sync(0xffffffffu, m);
            if (lane == 0) atomicMax(scale_max, m);
            decoder_barrier(128 * NG);
            m = *reinterpret_cast<volatile uint32_t *>(scale_max);
            // 2^E just above the largest |s| (1 if all are zero; 2^16 covers
            // every finite value, infinities and NaN go through)
            int e = 0;
            if (m >= 0x7c00u) e = 16;
            else if (m) e = ilogbf(half_bits_to_float((uint16_t)m)) + 1;
            inv = ldexpf(1.f, -e);
            out.factor = ldexpf(1.f, e);
#pragma unroll
            for (int q = 0; q < kCodeAhead; ++q) scale_ring[q] = fetch_scale(dg + NG * q);
        }
        // copies of kLag stages stay in flight; a stage is published kLag
        // iterations after it is issued, so kLag must stay below the ring
        // depth (the decoder waits for the MMAs of stage s - depth first)
        // (with NG groups a lag of kLag own stages spans NG kLag stages of the ring)
        constexpr int kLag = !kAsyncWeights ? 0 : kWsLag;
        static_assert(NG * kLag < kWsAStages || !kAsyncWeights, "copy lag must leave the MMAs a stage of slack");
        bool ok = true;
        int published = 0;  // own stages below this have been arrived on full_a[]
        // unrolled by the ring depth so every ring index is static
        for (int k0 = 0; ok && k0 < nown + kLag; k0 += kCodeAhead) {
#pragma unroll
            for (int u = 0; u < kCodeAhead; ++u) {
                const int k = k0 + u, s = dg + NG * k;  // own stage, stage
                if (k >= nown + kLag) break;
                if (k < nown) {
                    const int buf = s % kWsAStages;
                    // the buffer is free once the MMAs of stage s - depth
                    // completed; before blocking on it, publish every stage
                    // this thread has issued (the MMAs may need them first)
                    if (s >= kWsAStages) {
                        const uint32_t par = ((s / kWsAStages) - 1) & 1;
                        if (!mbar_test_wait(&empty_a[buf], par)) {
                            if constexpr (kAsyncWeights) {
                                cp_async_wait<0>();
                                fence_proxy_async_smem();
                                for (; published < k; ++published)
                                    mbar_arrive(&full_a[(dg + NG * published) % kWsAStages]);
                            }
                            if (!mbar_wait_ns(&empty_a[buf], par, kWaitNs)) *abort_v = 1;
                        }
                    }
                    // a warp leaves together (the scales are exchanged between lanes)
                    if (kTr ? __any_sync(0xffffffffu, *abort_v != 0) : *abort_v != 0) {
                        ok = false;
                        break;
                    }
                    const Chunk<S> code = code_ring[u];
                    const bool live = live_of(s);
                    code_ring[u] = fetch(s + NG * kCodeAhead);
                    uint8_t *A = tileA + buf * kTileABytes;
                    const uint4 *books = scb + (Op::kLayers > 1 ? layer_of(s) * S::K * 256 : 0);
                    const uint4 *cb = op.w[Op::kLayers > 1 ? layer_of(s) : 0].cb;
                    if constexpr (kTr) {
                        const uint32_t mine = scale_ring[u];
                        scale_ring[u] = fetch_scale(s + NG * kCodeAhead);
                        const uint4 *cb_next = op.w[layer_of(s + NG)].cb;
                        const Chunk<S> code_next = code_ring[(u + 1) % kCodeAhead];
                        auto put = [&](int r, uint4 v) {
                            const uint32_t h = __shfl_sync(0xffffffffu, mine, (rt_l & 1) * 8 + r);
                            const __half2 h2 = __half2half2(__ushort_as_half((uint16_t)h));
                            uint32_t p[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const __half2 m = __hmul2(*reinterpret_cast<__half2 *>(&p[j]), h2);
                                // a row past the layer: zero, whatever its padding code selects
                                p[j] = (live && tile_of(s) * 8 + r < L.out) ? *reinterpret_cast<const uint32_t *>(&m) : 0u;
                            }
                            *reinterpret_cast<uint4 *>(A + slot_of(r)) = make_uint4(p[0], p[1], p[2], p[3]);
                        };
                        if constexpr (kGatherAhead) {
#pragma unroll
                            for (int r = 0; r < 8; ++r) {
                                const uint4 v = ahead[r];
                                ahead[r] = ldg_nc_v4(cb_next + code_next.code(r, 0));
                                put(r, v);
                            }
                        } else if constexpr (S::K <= 2) {
                            uint4 tt[8][S::K];
#pragma unroll
                            for (int r = 0; r < 8; ++r) gather_terms<S>(code, r, books, cb, tt[r]);
#pragma unroll
                            for (int r = 0; r < 8; ++r) put(r, sum_round_fast_h8<S::K>(tt[r]));
                        } else {
#pragma unroll
                            for (int r = 0; r < 8; ++r) {
                                uint4 tt[S::K];
                                gather_terms<S>(code, r, books, cb, tt);
                                put(r, sum_round_fast_h8<S::K>(tt));
                            }
                        }
                    } else if constexpr (kAsyncWeights) {
                        const uint32_t a0 = smem_u32(A);
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            cp_async16(a0 + slot_of(r), live ? (const void *)(cb + code.code(r, 0)) : (const void *)cb,
                                       live ? 16u : 0u);
                    } else if constexpr (S::K <= 2) {
                        // all codeword reads before the first tile store (the
                        // books and the tile share one shared array)
                        uint4 tt[8][S::K];
#pragma unroll
                        for (int r = 0; r < 8; ++r) gather_terms<S>(code, r, books, cb, tt[r]);
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            *reinterpret_cast<uint4 *>(A + slot_of(r)) =
                                live ? sum_round_fast_h8<S::K>(tt[r]) : make_uint4(0, 0, 0, 0);
                    } else {
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            uint4 tt[S::K];
                            gather_terms<S>(code, r, books, cb, tt);
                            *reinterpret_cast<uint4 *>(A + slot_of(r)) =
                                live ? sum_round_fast_h8<S::K>(tt) : make_uint4(0, 0, 0, 0);
                        }
                    }
                }
                if constexpr (kAsyncWeights) {
                    cp_async_commit();
                    const int j = k - kLag;  // own stage whose copies have landed
                    if (j >= published) {
                        cp_async_wait<kLag>();
                        fence_proxy_async_smem();
                        mbar_arrive(&full_a[(dg + NG * j) % kWsAStages]);
                        published = j + 1;
                    }
                } else {
                    fence_proxy_async_smem();
                    mbar_arrive(&full_a[s % kWsAStages]);
                }
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
        if (tid == 0)
            for (int s = max(0, nk - kWsStages); s < nk; ++s)
                mbar_wait_ns(&full_b[s % kWsStages], (s / kWsStages) & 1, kWaitNs);
    }
    // The decoder warps finish: warp & 3 is the TMEM lane quarter, the NG
    // warps of a quarter take alternate blocks of 16 columns.  After a
    // timeout no tensor memory is read and the output is incomplete, which
    // the status word reports; the barriers and counters are still served.
    bool finish = warp >= 2 && *abort_v == 0;
    const uint32_t tq = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int r = (warp & 3) * 32 + lane;
    constexpr size_t kSlice = kBM * BN / 4;  // float4 per slice
    int c = 16 * ((warp - 2) / 4), end = BN, ks = 1;
    const float4 *slices = nullptr;
    unsigned *counter = nullptr;
    tc_fence_after();
    if (cluster_ks > 1) {
        ks = cluster_ks;
        const int cw = BN / ks;  // columns each split owns (a multiple of 16)
        float4 *mine = reinterpret_cast<float4 *>(sp.partials) + ((size_t)blockIdx.y * gridDim.x + blockIdx.x) * ks * kSlice;
        slices = mine;
        if (finish) {
            publish_sums<BN>(mine + (size_t)z * kSlice, tq, c, 16 * NG, z * cw, (z + 1) * cw, T - n0, r);
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
        if (finish) publish_sums<BN>(mine + (size_t)z * kSlice, tq, c, 16 * NG, 0, 0, T - n0, r);
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
    if (finish)
        finish_blocks(op, L, out, c, 16 * NG, end, [&](int c0, float (&v)[16]) {
            tmem_ld16(tq + (uint32_t)c0, v);
            if (ks > 1) add_slices<Op::kAhead>(v, slices + ((c0 / 16) * 4) * kBM + r, kSlice, ks, z);
        });
    if (counter && tid == 0) *counter = 0u;
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, BN);
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
    size_t ws_bytes;  // status word + tile counters + fp32 partials
};

// `mtiles` row tiles, `nst` stages of the contraction; `max_bn` where the
// shared memory does not hold 512-token tiles.
inline GemmPlan plan_ws(int mtiles, int nst, int T, int max_bn = 512)
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
    const long tiles = (long)p.mtiles * p.ntiles;
    // the decode is the bound: split the contraction until about one CTA
    // per SM works, keeping at least 8 stages per split
    int ks = tiles < kNumSMs ? (int)(kNumSMs / tiles) : 1;
    ks = std::max(1, std::min(ks, nst / 8));
    // the split runs as one thread-block cluster along z whose CTAs share
    // the finish: 2, 4 or 8 CTAs (the largest power of two not above ks).
    // With at least 8 stages per split (nst >= 8 kc) none of them is empty:
    // per = ceil(nst / kc) gives exactly kc non-empty splits
    if (ks >= 2) {
        int kc = 2;
        while (kc * 2 <= std::min(ks, 8)) kc *= 2;
        ks = kc;
    }
    p.per_split = (nst + ks - 1) / ks;
    p.ks = (nst + p.per_split - 1) / p.per_split;
    p.cluster = p.ks > 1;
    if (p.ks > 1) p.ws_bytes = kWsData + (size_t)p.ks * tiles * kBM * p.bn * sizeof(float);
    // more tiles than one wave, the last wave at most half full: its tiles'
    // contraction is split so that it fills the SMs (Llama-2-7B MLP
    // rows at 2048 tokens: 344 tiles, 48 in the third wave, split 3 ways)
    if (p.ks == 1 && tiles > kNumSMs) {
        const long tail = tiles % kNumSMs;
        if (tail > 0 && tail * 2 <= kNumSMs && tail <= kWsMaxCounters) {
            int kt = std::min((int)(kNumSMs / tail), std::min(nst / 8, 8));
            if (kt >= 2) {
                const int per = (nst + kt - 1) / kt;
                kt = (nst + per - 1) / per;  // no empty split
                p.tail = TailMap{(int)(tiles - tail), kt, per};
                p.ws_bytes = kWsData + (size_t)tail * kt * kBM * p.bn * sizeof(float);
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
// 8): innermost dimension tokens, box 64 tokens x 64 rows.
inline bool token_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap *map, const uint16_t *x, int rows, int T,
                      int pitch)
{
    cuuint64_t dims[2] = {(cuuint64_t)T, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)pitch * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)kBK};
    cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<uint16_t *>(x), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class S, int BN, class Op>
constexpr int gemm_ws_smem_bytes()
{
    constexpr int BB = kWsBookBytes<S, Op>;
    return 1024 + kWsAStagesOf<S, BN, BB> * kTileABytes + kWsStagesOf<S, BN, BB> * (kBK * BN * 2) + BB +
           (2 * kWsAStagesOf<S, BN, BB> + 2 * kWsStagesOf<S, BN, BB> + 1) * 8 + 16;
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

template <class Op>
cudaError_t launch_ws(const Geom &g, const GemmPlan &p, const TensorMaps<Op::kMaps> &maps, const Op &op, int T,
                      void *ws, cudaStream_t s, bool pdl)
{
    const long tiles = (long)p.mtiles * p.ntiles;
    const dim3 grid = p.tail.ks > 0 ? dim3((unsigned)(p.tail.full + (tiles - p.tail.full) * p.tail.ks), 1, 1)
                                    : dim3(p.mtiles, p.ntiles, p.ks);
    GemmSplit sp{nullptr};
    if (p.ks > 1) sp.partials = reinterpret_cast<float *>(reinterpret_cast<char *>(ws) + kWsData);
    auto launch = [&](auto sch, auto bn) {
        using S = decltype(sch);
        constexpr int BN = decltype(bn)::value;
        if constexpr (BN > kWsMaxBN<S, Op>) {
            return cudaErrorInvalidValue;
        } else {
            constexpr int smem = gemm_ws_smem_bytes<S, BN, Op>();
            static_assert(smem <= 227 * 1024, "shared memory of the warp-specialised GEMM");
            auto kern = gemm_ws_kernel<S, BN, Op>;
            cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = grid;
            cfg.blockDim = dim3(kWsThreadsOf<S>);
            cfg.dynamicSmemBytes = smem;
            cfg.stream = s;
            cudaLaunchAttribute attr[2];
            int na = 0;
            if (p.cluster) {
                attr[na].id = cudaLaunchAttributeClusterDimension;
                attr[na].val.clusterDim.x = 1;
                attr[na].val.clusterDim.y = 1;
                attr[na].val.clusterDim.z = p.ks;
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
    return with_scheme(g, [&](auto sch) {
        return p.bn == 512 ? launch(sch, std::integral_constant<int, 512>{})
                           : launch(sch, std::integral_constant<int, 256>{});
    });
}

}  // namespace aqh
