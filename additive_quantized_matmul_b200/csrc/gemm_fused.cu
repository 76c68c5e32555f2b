// Prefill products with what stands around them: bias, activation and
// residual in the epilogue (aq_gemm_fused), the gated feed-forward block
// (aq_glu_gemm), and the backward passes of both (aq_gemm_fused_grad,
// aq_glu_grad), which compute the projections again and take the gradient in
// the epilogue, then multiply it back (input_grad.cu).
//
// All run on the warp-specialised kernel of gemm_ws.cuh, whose arrays have
// rows of 16-byte multiples (TMA).  For T not a multiple of 8 one launch
// first copies the inputs to rows of T rounded up to 8 in the workspace, and
// one last launch copies the results from there.  (Ragged rows read and
// written by the kernel itself cost 15 to 40 us of epilogue at 1001 and 2047
// tokens; the two copies cost 2 us each and the traffic.)
//
// The products are bound by the SM's shared memory and, when calls follow one
// another, by the power limit (see gemm_ws.cuh).  In series, 2048 tokens:
// 4096 x 11008 1x16 with residual 185 to 191 us (976 TFLOP/s, 70 % of the tensor
// rate measured over seconds), gated 2 x 11008 x 4096 2x8 335 to 345 us (1077,
// 78 %), backward of the gated block, 1x16, 808 to 850 us (895 counting the
// products computed again, 65 %).  Alone: 178, 323 and 748 us.
#include "gemm_ws.cuh"
#include "layer_ops.cuh"

namespace aqk {

// Rows of T elements from one pitch to another.  A warp takes 2 KiB of a row:
// the 16-byte aligned pieces of the destination, 32 consecutive ones an
// access, four in flight.  The source of a piece starts m bytes into an
// aligned piece of its own, m the same for the whole row, so a lane reads one
// aligned piece, gets the next from its neighbour and shifts; the up to seven
// elements at either end of a row go singly.  With scales (a whole launch's
// arrays are multiplied, by 2^-E alone where an array has none) each product
// is rounded once.  Bound by the latency of its round trips: two scaled arrays of
// 11008 rows and 2048 tokens (90 MB read, 90 MB written) 42 us with cold caches,
// which is why aligned ones have scale_rows_kernel.
constexpr int kCopyThreads = 256;
constexpr int kCopyPieces = 128;  // pieces of a row per warp

struct RowCopies {
    aqh::RowCopy job[aqh::kMaxRowCopies];
    int jobs;
    float *factor;  // with scales: receives 2^E
    unsigned *top;  // with scales: the largest product (bits of a float)
};

// Bytes m .. m + 15 of the 32 bytes (a, b); m even, the same in every lane.
__device__ __forceinline__ uint4 bytes_from(uint4 a, uint4 b, int m)
{
    uint32_t w[5];
    switch (m >> 2) {
    case 0: w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x; break;
    case 1: w[0] = a.y, w[1] = a.z, w[2] = a.w, w[3] = b.x, w[4] = b.y; break;
    case 2: w[0] = a.z, w[1] = a.w, w[2] = b.x, w[3] = b.y, w[4] = b.z; break;
    default: w[0] = a.w, w[1] = b.x, w[2] = b.y, w[3] = b.z, w[4] = b.w; break;
    }
    const int sh = 8 * (m & 2);
    return make_uint4(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh), __funnelshift_r(w[2], w[3], sh),
                      __funnelshift_r(w[3], w[4], sh));
}

// *top = the largest finite |scales[r] src[r][t]| over the jobs, all of as many
// rows (*top zero before).  A warp takes 4 KiB of a row at a time, its aligned
// pieces by 16 bytes, the up to seven elements at either end singly.  Bound by the
// latency of its round trips, two or three a warp: 11008 rows of 2047 tokens (45 MB)
// 18 us with cold caches, 2.5 TB/s; 4096 rows of 512 tokens 6 us.
constexpr int kMaxPieces = 256;  // pieces of a row per warp

__global__ void __launch_bounds__(kCopyThreads) scaled_max_kernel(const __grid_constant__ RowCopies jobs, int T)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, rows = jobs.job[0].rows;
    const unsigned shares = ((unsigned)T + 8 * kMaxPieces - 1) / (8 * kMaxPieces);
    const int step = gridDim.x * (kCopyThreads / 32);
    float m = 0.f;
    for (int j = 0; j < jobs.jobs; ++j) {
        const aqh::RowCopy &c = jobs.job[j];
        for (long i = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); i < (long)rows * shares; i += step) {
            const int r = shares == 1 ? (int)i : (int)(i / shares);
            const int t0 = shares == 1 ? 0 : (int)(i % shares) * (8 * kMaxPieces);
            const int n = min(8 * kMaxPieces, T - t0);
            const uint16_t *src = c.src + (size_t)r * c.src_pitch + t0;
            const int head = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(src) & 15)) & 15) / 2);
            const int pieces = (n - head) / 8;
            const uint4 *from = reinterpret_cast<const uint4 *>(src + head);
            uint32_t h = 0;
#pragma unroll
            for (int q = 0; q < kMaxPieces / 32; ++q)
                if (32 * q + lane < pieces) finite_absmax_h8(h, __ldg(from + 32 * q + lane));
            const int e = lane < 8 ? lane : head + 8 * pieces + lane - 8;
            if (lane < 8 ? lane < head : lane < 16 && e < n) finite_absmax_h2(h, src[e]);
            m = fmaxf(m, scaled_top(h, c.scales ? half_bits_to_float(__ldg(c.scales + r)) : 1.f));
        }
    }
    __shared__ uint32_t part[kCopyThreads / 32];
    const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
    if (lane == 0) part[threadIdx.x >> 5] = w;
    __syncthreads();
    if (threadIdx.x < 32) {
        const uint32_t all = __reduce_max_sync(0xffffffffu, lane < kCopyThreads / 32 ? part[lane] : 0u);
        if (lane == 0) atomicMax(jobs.top, all);
    }
}

// E of the largest product: 2^14 <= top / 2^E < 2^15, so that none overflows, nor
// loses bits that matter beside the largest one (2^-25 is 2^-39 of it).  |E| < 64.
__device__ __forceinline__ int scale_exponent(const RowCopies &jobs)
{
    const float m = __uint_as_float(__ldcg(jobs.top));
    return m > 0.f ? ilogbf(m) - 14 : 0;
}

__global__ void __launch_bounds__(kCopyThreads) copy_rows_kernel(const __grid_constant__ RowCopies jobs, int T)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const aqh::RowCopy &c = jobs.job[blockIdx.z];
    const int lane = threadIdx.x & 31;
    float inv = 1.f;
    if (jobs.factor) {  // some job has scales
        const int e = scale_exponent(jobs);
        inv = ldexpf(1.f, -e);
        if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) *jobs.factor = ldexpf(1.f, e);
    }
    // first byte past the source array: an aligned piece that passes it is read by elements
    const uintptr_t src_end = reinterpret_cast<uintptr_t>(c.src + (size_t)(c.rows - 1) * c.src_pitch + T);
    for (int r = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); r < c.rows; r += gridDim.x * (kCopyThreads / 32)) {
        uint16_t *dst = c.dst + (size_t)r * c.dst_pitch;
        const uint16_t *src = c.src + (size_t)r * c.src_pitch;
        const float sc = c.scales ? half_bits_to_float(__ldg(c.scales + r)) * inv : inv;
        const int head = min(T, (int)((16 - (reinterpret_cast<uintptr_t>(dst) & 15)) & 15) / 2);
        const int pieces = (T - head) / 8;
        const uintptr_t from = reinterpret_cast<uintptr_t>(src + head);
        const int m = (int)(from & 15);
        auto read = [&](int piece) {  // the aligned piece in which piece `piece`'s source starts
            const uintptr_t at = (from & ~(uintptr_t)15) + 16 * (size_t)piece;
            if (at + 16 <= src_end) return __ldg(reinterpret_cast<const uint4 *>(at));
            uint32_t w[4] = {0u, 0u, 0u, 0u};
            for (int j = 0; j < 8; ++j)
                if (at + 2 * j < src_end) w[j / 2] |= (uint32_t)*reinterpret_cast<const uint16_t *>(at + 2 * j) << (16 * (j & 1));
            return make_uint4(w[0], w[1], w[2], w[3]);
        };
        const int p0 = blockIdx.y * kCopyPieces;
        uint4 a[kCopyPieces / 32], b[kCopyPieces / 32];
#pragma unroll
        for (int i = 0; i < kCopyPieces / 32; ++i) {
            const int p = p0 + 32 * i + lane;
            if (p < pieces) a[i] = read(p);
            // the last lane's (or piece's) neighbour is not in the warp
            if (p < pieces && m && (lane == 31 || p == pieces - 1)) b[i] = read(p + 1);
        }
#pragma unroll
        for (int i = 0; i < kCopyPieces / 32; ++i) {
            const int p = p0 + 32 * i + lane;
            uint4 n;
            n.x = __shfl_down_sync(0xffffffffu, a[i].x, 1), n.y = __shfl_down_sync(0xffffffffu, a[i].y, 1);
            n.z = __shfl_down_sync(0xffffffffu, a[i].z, 1), n.w = __shfl_down_sync(0xffffffffu, a[i].w, 1);
            if (lane == 31 || p == pieces - 1) n = b[i];
            if (p < pieces) {
                uint4 v = bytes_from(a[i], n, m);
                if (jobs.factor) v = scale_round_h8(v, sc);
                *reinterpret_cast<uint4 *>(dst + head + 8 * (size_t)p) = v;
            }
        }
        if (blockIdx.y == 0) {
            const int tail = head + 8 * pieces;
            const int e = lane < 8 ? lane : tail + lane - 8;
            if (lane < 8 ? lane < head : lane < 16 && e < T)
                dst[e] = jobs.factor ? float_to_half_bits(sc * half_bits_to_float(src[e])) : src[e];
        }
    }
}

// The same for scaled rows of T = pitch, a multiple of 8: every piece is aligned
// in both arrays.  A warp takes 2 KiB of a row, the next row's share requested
// before this one's is multiplied; 48 registers leave room for five CTAs an SM
// (64 and four above).  Two arrays of 11008 rows and 2048 tokens (90 MB read, 90 MB
// written, of which 36 MB left L2 meanwhile) 27 us with cold caches.
__global__ void __launch_bounds__(kCopyThreads, 5) scale_rows_kernel(const __grid_constant__ RowCopies jobs, int T)
{
    constexpr int kN = kCopyPieces / 32;
    grid_dependency_wait();
    grid_launch_dependents();
    const aqh::RowCopy &c = jobs.job[blockIdx.z];
    const int lane = threadIdx.x & 31, pieces = T / 8, step = gridDim.x * (kCopyThreads / 32);
    const int p0 = blockIdx.y * kCopyPieces + lane;
    auto read = [&](int r, uint4 (&a)[kN]) {
        const uint4 *src = reinterpret_cast<const uint4 *>(c.src + (size_t)r * T);
#pragma unroll
        for (int i = 0; i < kN; ++i)
            if (p0 + 32 * i < pieces) a[i] = __ldg(src + p0 + 32 * i);
    };
    int r = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
    uint4 a[kN] = {}, b[kN] = {};
    if (r < c.rows) read(r, a);
    const int e = scale_exponent(jobs);
    const float inv = ldexpf(1.f, -e);
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) *jobs.factor = ldexpf(1.f, e);
    for (; r < c.rows; r += step) {
        if (r + step < c.rows) read(r + step, b);
        const float sc = c.scales ? half_bits_to_float(__ldg(c.scales + r)) * inv : inv;
        uint4 *dst = reinterpret_cast<uint4 *>(c.dst + (size_t)r * T);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            if (p0 + 32 * i < pieces) dst[p0 + 32 * i] = scale_round_h8(a[i], sc);
            a[i] = b[i];
        }
    }
}

// grad_bias[o] = sums[0][o] + sums[1][o] + ..., in that order within each of
// eight interleaved parts, the parts then in order: 32 rows per CTA, one
// warp per part.  The epilogue just before left the sums in L2 (4 bytes per row
// and 16 tokens), so this is one launch's latency.
__global__ void __launch_bounds__(256) bias_grad_kernel(const float *__restrict__ sums, int blocks, int out,
                                                        float *__restrict__ grad_bias)
{
    __shared__ float part[8][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, p = threadIdx.x >> 5, o = blockIdx.x * 32 + lane;
    float a = 0.f;
    if (o < out) {
#pragma unroll 4
        for (int b = p; b < blocks; b += 8) a += __ldcg(sums + (size_t)b * out + o);
    }
    part[p][lane] = a;
    __syncthreads();
    if (p == 0 && o < out) {
#pragma unroll
        for (int i = 1; i < 8; ++i) a += part[i][lane];
        grad_bias[o] = a;
    }
}

// Without an activation: grad_z = gy, grad_bias its row sums.  One warp per
// row; a lane adds its tokens (one in 32, or for T a multiple of 8, where rows
// are 16-byte aligned, eight in 256) in order, then the lanes in a tree.
// Bound by HBM, one read and one write of the array.
// 11008 rows, 2048 tokens: 18.4 us, 4.9 TB/s (75 % of the measured copy rate);
// by single elements, as ragged rows are, 23.8 us.
__global__ void __launch_bounds__(256) linear_grad_kernel(const uint16_t *__restrict__ gy, int out, int T,
                                                          uint16_t *__restrict__ grad_z, float *__restrict__ grad_bias)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    for (int o = blockIdx.x * 8 + (threadIdx.x >> 5); o < out; o += gridDim.x * 8) {
        const size_t row = (size_t)o * T;
        float a = 0.f;
        if (T % 8 == 0) {
            const uint4 *from = reinterpret_cast<const uint4 *>(gy + row);
            uint4 *to = reinterpret_cast<uint4 *>(grad_z + row);
#pragma unroll 4
            for (int p = lane; p < T / 8; p += 32) {
                const uint4 v = __ldg(from + p);
                to[p] = v;
                float f[8];
                widen_h8(v, f);
                a += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
            }
        } else {
#pragma unroll 8
            for (int t = lane; t < T; t += 32) {
                const uint16_t h = __ldg(gy + row + t);
                grad_z[row + t] = h;
                a += half_bits_to_float(h);
            }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) a += __shfl_xor_sync(0xffffffffu, a, d);
        if (lane == 0 && grad_bias) grad_bias[o] = a;
    }
}

}  // namespace aqk

namespace aqh {
using namespace aqk;

static RowCopies all_jobs(const RowCopy *jobs, int n)
{
    RowCopies all{};
    all.jobs = n;
    for (int i = 0; i < n; ++i) all.job[i] = jobs[i];
    return all;
}

// `per_sm` CTAs an SM over `arrays` arrays, or one per eight rows
static dim3 copy_grid(int rows, int T, int n, int arrays, int per_sm)
{
    const unsigned pieces = (unsigned)std::max(1, (T / 8 + kCopyPieces - 1) / kCopyPieces);
    const int share = (int)pieces * arrays;
    return dim3(std::max(1, std::min((rows + 7) / 8, per_sm * kNumSMs / share + 1)), pieces, n);
}

cudaError_t copy_rows(const RowCopy *jobs, int n, int T, cudaStream_t s)
{
    int rows = 0;
    for (int i = 0; i < n; ++i) rows = std::max(rows, jobs[i].rows);
    return launch_programmatic(copy_rows_kernel, copy_grid(rows, T, n, 1, 16), dim3(kCopyThreads), s, all_jobs(jobs, n), T);
}

cudaError_t scale_rows(const RowCopy *jobs, int n, int T, float *factor, unsigned *top, bool known, cudaStream_t s)
{
    const int rows = jobs[0].rows;
    RowCopies all = all_jobs(jobs, n);
    all.factor = factor;
    all.top = top;
    if (!known) {
        const long shares = ((long)T + 8 * kMaxPieces - 1) / (8 * kMaxPieces);
        const unsigned ctas = (unsigned)std::min<long>(4 * kNumSMs, (rows * shares + 7) / 8);
        const cudaError_t e = launch_programmatic(scaled_max_kernel, dim3(ctas), dim3(kCopyThreads), s, all, T);
        if (e != cudaSuccess) return e;
    }
    if (T % 8 == 0)
        return launch_programmatic(scale_rows_kernel, copy_grid(rows, T, n, n, 5), dim3(kCopyThreads), s, all, T);
    return launch_programmatic(copy_rows_kernel, copy_grid(rows, T, n, n, 4), dim3(kCopyThreads), s, all, T);
}

namespace {

// Workspace of an operator: the plan's part (of the product, and of the
// transposed product after it), then the sums of the bias gradient, with T
// ragged the padded arrays, and the scaled gradients.  An unsplit plan ends
// before the arrival counters, which are other calls' as well as its own: an
// array never starts among them.  A call takes some of the arrays that the
// sizes below take, in another order: the spare bytes of `size` cover the
// alignment.
struct Layout {
    GemmPlan p;
    size_t end;
    size_t take(size_t bytes)
    {
        const size_t at = align_up(std::max(end, kWsData));
        end = at + bytes;
        return at;
    }
    size_t size() const { return end > kWsData ? end + 128 : end; }
};

template <class Op>
Layout layout_of(const Geom &g, int T, bool back)
{
    Layout l;
    l.p = plan_ws(ws_mtiles<Op>(g), ws_layer_stages<Op>(g), T, ws_max_bn<Op>(g), Op::kPairs);
    l.end = back ? std::max(l.p.ws_bytes, back_plan_bytes(g, Op::kLayers, T)) : l.p.ws_bytes;
    return l;
}

template <class Op>
cudaError_t product(const Geom &g, const Layout &l, const uint16_t *x, int T, const Op &op, char *ws, cudaStream_t s)
{
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    TensorMaps<Op::kMaps> maps{};
    const int pitch = padded_tokens(T);
    if (!token_map(encode, &maps.m[0], x, g.in, T, pitch) || !io_maps(encode, &maps, op, g, T, pitch))
        return cudaErrorInvalidValue;
    return launch_ws(g, l.p, maps, op, T, ws, s, true);
}

// An operator's arrays where the kernels see them: the caller's own, or with
// T ragged their padded stand-ins in the workspace.
class Arrays {
public:
    Arrays(Layout &l, char *ws, int T) : l_(l), ws_(ws), T_(T), pad_(T % 8 != 0) {}
    const uint16_t *in(const uint16_t *a, int rows)
    {
        if (!pad_ || !a) return a;
        uint16_t *p = room(rows);
        in_[nin_++] = RowCopy{a, p, rows, T_, padded_tokens(T_), nullptr};
        return p;
    }
    uint16_t *out(uint16_t *a, int rows)
    {
        if (!pad_ || !a) return a;
        uint16_t *p = room(rows);
        out_[nout_++] = RowCopy{p, a, rows, padded_tokens(T_), T_, nullptr};
        return p;
    }
    cudaError_t before(cudaStream_t s) const { return nin_ ? copy_rows(in_, nin_, T_, s) : cudaSuccess; }
    cudaError_t after(cudaStream_t s) const { return nout_ ? copy_rows(out_, nout_, T_, s) : cudaSuccess; }

private:
    uint16_t *room(int rows) { return reinterpret_cast<uint16_t *>(ws_ + l_.take(padded_bytes(rows, T_))); }
    Layout &l_;
    char *ws_;
    int T_;
    bool pad_;
    RowCopy in_[kMaxRowCopies], out_[kMaxRowCopies];
    int nin_ = 0, nout_ = 0;
};

// Room for padded arrays of [in] and of [out] rows.
void take_padded(Layout &l, const Geom &g, int T, int in_arrays, int out_arrays)
{
    if (T % 8 == 0) return;
    for (int i = 0; i < in_arrays; ++i) l.take(padded_bytes(g.in, T));
    for (int i = 0; i < out_arrays; ++i) l.take(padded_bytes(g.out, T));
}

// The gradients that the transposed product reads: as they are, or copies
// multiplied by the layers' scales.
struct Scaled {
    const uint16_t *g[2];
    float *factor;  // or null
};

void take_scaled(Layout &l, const Geom &g, int T, int layers)
{
    if (back_scales_weights(g)) return;
    l.take(sizeof(float));
    for (int i = 0; i < layers; ++i) l.take(padded_bytes(g.out, T));
}

bool scaled_gradients(const Geom &g, const LayerWeights &w0, const LayerWeights &w1)
{
    return !back_scales_weights(g) && (w0.scales || w1.scales);
}

// `pitch`: of the gradients in memory (T where they are ragged and unpadded);
// `known`: ws_top holds the largest scaled one.
cudaError_t scale_gradients(const Geom &g, Layout &l, char *ws, int layers, const LayerWeights *w,
                            const uint16_t *const *grads, int T, int pitch, bool known, Scaled *out, cudaStream_t s)
{
    *out = Scaled{{grads[0], layers > 1 ? grads[1] : grads[0]}, nullptr};
    const bool scales = scaled_gradients(g, w[0], layers > 1 ? w[1] : w[0]);
    if (!scales && pitch == padded_tokens(T)) return cudaSuccess;
    if (scales) out->factor = reinterpret_cast<float *>(ws + l.take(sizeof(float)));
    RowCopy jobs[2];
    for (int i = 0; i < layers; ++i) {
        uint16_t *z = reinterpret_cast<uint16_t *>(ws + l.take(padded_bytes(g.out, T)));
        jobs[i] = RowCopy{grads[i], z, g.out, pitch, padded_tokens(T), w[i].scales};
        out->g[i] = z;
    }
    if (!scales) return copy_rows(jobs, layers, T, s);
    return scale_rows(jobs, layers, T, out->factor, ws_top(ws), known, s);
}

size_t bias_sums_bytes(const Geom &g, int T) { return (size_t)((T + 15) / 16) * g.out * sizeof(float); }

}  // namespace

size_t gemm_fused_workspace_bytes(const Geom &g, int T)
{
    Layout l = layout_of<FusedOp>(g, T, false);
    take_padded(l, g, T, 1, 2);
    return l.size();
}

cudaError_t launch_gemm_fused(const Geom &g, const LayerWeights &w, const uint16_t *x, int T, const EpilogueArgs &ep,
                              uint16_t *y, void *ws, cudaStream_t s)
{
    Layout l = layout_of<FusedOp>(g, T, false);
    char *base = reinterpret_cast<char *>(ws);
    Arrays a(l, base, T);
    const uint16_t *xk = a.in(x, g.in), *rk = a.in(ep.residual, g.out);
    const FusedOp op{{w}, ep.act, ep.bias, rk, a.out(y, g.out), false, nullptr, nullptr};
    cudaError_t e = a.before(s);
    if (e == cudaSuccess) e = product(g, l, xk, T, op, base, s);
    return e == cudaSuccess ? a.after(s) : e;
}

size_t glu_gemm_workspace_bytes(const Geom &g, int T)
{
    Layout l = layout_of<GatedOp>(g, T, false);
    take_padded(l, g, T, 1, 1);
    return l.size();
}

cudaError_t launch_glu_gemm(const Geom &g, const LayerWeights &gate, const LayerWeights &up, const uint16_t *x, int T,
                            int act, uint16_t *y, void *ws, cudaStream_t s)
{
    Layout l = layout_of<GatedOp>(g, T, false);
    char *base = reinterpret_cast<char *>(ws);
    Arrays a(l, base, T);
    const uint16_t *xk = a.in(x, g.in);
    const GatedOp op{{gate, up}, act, nullptr, a.out(y, g.out), nullptr, nullptr};
    cudaError_t e = a.before(s);
    if (e == cudaSuccess) e = product(g, l, xk, T, op, base, s);
    return e == cudaSuccess ? a.after(s) : e;
}

size_t gemm_fused_grad_workspace_bytes(const Geom &g, int T)
{
    Layout l = layout_of<FusedOp>(g, T, true);
    l.take(bias_sums_bytes(g, T));
    take_padded(l, g, T, 2, 2);
    take_scaled(l, g, T, 1);
    return l.size();
}

cudaError_t launch_gemm_fused_grad(const Geom &g, const LayerWeights &w, const uint16_t *x, const uint16_t *gy, int T,
                                   const EpilogueArgs &ep, uint16_t *grad_z, float *grad_bias, uint16_t *grad_x,
                                   void *ws, cudaStream_t s)
{
    if (ep.act == AQ_ACT_NONE) {  // z is not needed
        const cudaError_t e = launch_programmatic(linear_grad_kernel, dim3(std::min((g.out + 7) / 8, 8 * kNumSMs)),
                                                  dim3(256), s, gy, g.out, T, grad_z, grad_bias);
        return e == cudaSuccess && grad_x ? launch_input_grad(g, w, gy, T, grad_x, ws, s) : e;
    }
    Layout l = layout_of<FusedOp>(g, T, true);
    char *base = reinterpret_cast<char *>(ws);
    float *sums = reinterpret_cast<float *>(base + l.take(bias_sums_bytes(g, T)));
    Arrays a(l, base, T);
    const uint16_t *xk = a.in(x, g.in), *gk = a.in(gy, g.out);
    uint16_t *zk = a.out(grad_z, g.out), *gxk = a.out(grad_x, g.in);
    const FusedOp op{{w}, ep.act, ep.bias, gk, zk, true, grad_bias ? sums : nullptr,
                     grad_x && scaled_gradients(g, w, w) ? ws_top(ws) : nullptr};
    cudaError_t e = a.before(s);
    if (e == cudaSuccess) e = product(g, l, xk, T, op, base, s);
    if (e == cudaSuccess && grad_bias)
        e = launch_programmatic(bias_grad_kernel, dim3((g.out + 31) / 32), dim3(256), s, (const float *)sums,
                                (T + 15) / 16, g.out, grad_bias);
    if (e == cudaSuccess && grad_x) {
        Scaled z;
        e = scale_gradients(g, l, base, 1, &w, &zk, T, padded_tokens(T), true, &z, s);
        if (e == cudaSuccess) e = launch_back(g, 1, w, z.g[0], w, nullptr, T, z.factor, gxk, ws, s);
    }
    return e == cudaSuccess ? a.after(s) : e;
}

size_t glu_grad_workspace_bytes(const Geom &g, int T)
{
    Layout l = layout_of<GatedOp>(g, T, true);
    take_padded(l, g, T, 2, 3);
    take_scaled(l, g, T, 2);
    return l.size();
}

cudaError_t launch_glu_grad(const Geom &g, const LayerWeights &gate, const LayerWeights &up, const uint16_t *x,
                            const uint16_t *gy, int T, int act, uint16_t *grad_gate, uint16_t *grad_up,
                            uint16_t *grad_x, void *ws, cudaStream_t s)
{
    Layout l = layout_of<GatedOp>(g, T, true);
    char *base = reinterpret_cast<char *>(ws);
    Arrays a(l, base, T);
    const uint16_t *xk = a.in(x, g.in), *gk = a.in(gy, g.out);
    uint16_t *ggk = a.out(grad_gate, g.out), *guk = a.out(grad_up, g.out), *gxk = a.out(grad_x, g.in);
    const GatedOp op{{gate, up}, act, gk, ggk, guk, grad_x && scaled_gradients(g, gate, up) ? ws_top(ws) : nullptr};
    cudaError_t e = a.before(s);
    if (e == cudaSuccess) e = product(g, l, xk, T, op, base, s);
    if (e == cudaSuccess && grad_x) {
        const LayerWeights w[2] = {gate, up};
        const uint16_t *grads[2] = {ggk, guk};
        Scaled z;
        e = scale_gradients(g, l, base, 2, w, grads, T, padded_tokens(T), true, &z, s);
        if (e == cudaSuccess) e = launch_back(g, 2, gate, z.g[0], up, z.g[1], T, z.factor, gxk, ws, s);
    }
    return e == cudaSuccess ? a.after(s) : e;
}

size_t input_grad_workspace_bytes(const Geom &g, int T)
{
    Layout l;
    l.end = back_plan_bytes(g, 1, T);
    take_padded(l, g, T, 1, 1);
    take_scaled(l, g, T, 1);
    return l.size();
}

cudaError_t launch_input_grad(const Geom &g, const LayerWeights &w, const uint16_t *gy, int T, uint16_t *gx, void *ws,
                              cudaStream_t s)
{
    Layout l;
    l.end = back_plan_bytes(g, 1, T);
    char *base = reinterpret_cast<char *>(ws);
    Arrays a(l, base, T);
    uint16_t *gxk = a.out(gx, g.in);
    Scaled z;  // (the copy of ragged rows pads them, scaled or not)
    cudaError_t e = scale_gradients(g, l, base, 1, &w, &gy, T, T, false, &z, s);
    if (e == cudaSuccess) e = launch_back(g, 1, w, z.g[0], w, nullptr, T, z.factor, gxk, ws, s);
    return e == cudaSuccess ? a.after(s) : e;
}

}  // namespace aqh
