// Prefill product Y = diag(s) W X on the 5th-generation tensor cores (sm_100a):
// the launcher of aq_gemm, which runs on the warp-specialised kernel of
// gemm_ws.cuh (PlainOp) for T a multiple of 8, and the kernel for the others.
//
// W is decoded tile by tile from its codes (AQLM wiki entry, "Niveau
// intermédiaire": each group of 8 weights is sum_k C_k[i_k]) straight into
// shared memory in the 128-byte-swizzled K-major layout the tensor core
// reads; X tiles are staged MN-major (128-byte swizzle) next to it; one
// thread issues tcgen05.mma (kind::f16: binary16 operands, fp32 accumulator
// in tensor memory).  Tile: M = 128 rows of W, N = 128 tokens, K = 64 input
// features (8 code groups) per stage, two stages so that decoding stage
// k+1 overlaps the MMAs of stage k; X rows are read with plain loads, which
// TMA could not address.  The epilogue reads the accumulator with
// tcgen05.ld, applies the row scale and rounds to binary16.
//
// Every wait is bounded (wall-clock limit via %globaltimer): on give-up the
// kernel records AQ_ERR_TIMEOUT in the workspace status word, drains what
// it issued (again bounded), frees its tensor memory and returns.
#include "gemm_ws.cuh"

namespace aqk {

constexpr int kBN = 128;           // tokens per CTA (MMA N)
constexpr int kStages = 2;
constexpr int kGemmThreads = 128;  // 4 warps: decode, stage X, epilogue
constexpr int kTileBBytes = kBK * kBN * 2;  // 16 KiB
// ---- kernel -----------------------------------------------------------------

template <class S>
__global__ void __launch_bounds__(kGemmThreads, 1)
gemm_tc_kernel(Geom L, const uint8_t *__restrict__ packed, const uint4 *__restrict__ cb,
               const uint16_t *__restrict__ scales, const uint16_t *__restrict__ x, int T,
               uint16_t *__restrict__ y, void *ws)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
    uint8_t *smem = smem_raw + pad;
    uint8_t *tileA = smem;                                // [2][16 KiB]
    uint8_t *tileB = smem + kStages * kTileABytes;        // [2][16 KiB]
    uint4 *scb = reinterpret_cast<uint4 *>(tileB + kStages * kTileBBytes);  // B = 8 codebooks
    uint64_t *bars = reinterpret_cast<uint64_t *>(reinterpret_cast<uint8_t *>(scb) + S::kSmemBookBytes);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kStages);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int m0 = blockIdx.x * kBM;
    const int n0 = blockIdx.y * kBN;

    if constexpr (S::kBooksInSmem)
        for (int i = tid; i < S::K * 256; i += kGemmThreads) scb[i] = cb[i];
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(&bars[s], 1);
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(tmem_slot, kBN);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int nk = (L.in + kBK - 1) / kBK;
    const uint32_t idesc = make_idesc(kBM, kBN);
    const bool vec_x = (T % 8) == 0;
    bool ok = true;

    for (int kt = 0; kt < nk; ++kt) {
        const int st = kt & 1;
        if (kt >= kStages) {
            // the MMAs that read this stage were committed at kt - 2; the
            // outcome is made CTA-uniform before anyone leaves the loop
            const bool got = mbar_wait_ns(&bars[st], ((kt - kStages) / kStages) & 1, kWaitNs);
            if (!__syncthreads_and(got)) { ok = false; break; }
        }
        uint8_t *A = tileA + st * kTileABytes;
        uint8_t *Bt = tileB + st * kTileBBytes;

        // -- decode the W tile: thread -> (row tile rt_l = tid/8, group gi = tid%8)
        {
            const int rt_l = tid >> 3, gi = tid & 7;
            const int rt = (m0 >> 3) + rt_l;
            const int g = kt * 8 + gi;
            const bool live = (rt < L.rtiles) && (g < L.G);
            const Chunk<S> code = load_chunk<S>(packed, (size_t)rt * L.gp + g, live);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (live) {
                    uint4 t[S::K];
                    gather_terms<S>(code, r, scb, cb, t);
                    v = sum_round_fast_h8<S::K>(t);
                }
                const uint32_t row = rt_l * 8 + r;
                *reinterpret_cast<uint4 *>(A + sw128(row, gi)) = v;
            }
        }
        // -- stage the X tile: rows k (input features), 128 tokens as two
        //    64-token MN-major atoms columns of 64 rows x 128 bytes each.
        for (int i = tid; i < kBK * (kBN / 8); i += kGemmThreads) {
            const int k = i / (kBN / 8);
            const int c16 = i % (kBN / 8);      // 16-byte chunk along tokens
            const int nb = c16 >> 3, c = c16 & 7;
            const int gk = kt * kBK + k;
            const int gn = n0 + c16 * 8;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (gk < L.in) {
                const uint16_t *src = x + (size_t)gk * T + gn;
                if (vec_x && gn + 8 <= T) {
                    v = ldg_nc_v4(src);
                } else {
                    uint16_t h[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[j] = (gn + j < T) ? src[j] : (uint16_t)0;
                    v = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16),
                                   h[6] | (h[7] << 16));
                }
            }
            *reinterpret_cast<uint4 *>(Bt + nb * (kBK * 128) + sw128(k, c)) = v;
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after();
            const uint32_t a0 = smem_u32(A), b0 = smem_u32(Bt);
#pragma unroll
            for (int ks = 0; ks < kBK / 16; ++ks) {
                // A: K-major, +32 bytes per 16-element K step inside the swizzle row
                const uint64_t ad = smem_desc_sw128(a0 + ks * 32, 16, 1024);
                // B: MN-major, 64-token blocks 8 KiB apart (LBO), 8-row K groups
                // 1 KiB apart (SBO), +2 KiB per 16-row K step
                const uint64_t bd = smem_desc_sw128(b0 + ks * 2048, kBK * 128, 1024);
                mma_f16_ss(tmem, ad, bd, idesc, (kt > 0 || ks > 0) ? 1u : 0u);
            }
            mma_commit(&bars[st]);
        }
    }

    // Wait for the last commit (it covers every earlier MMA).
    if (ok && nk > 0) {
        const int last = nk - 1;
        ok = __syncthreads_and(mbar_wait_ns(&bars[last & 1], (last / kStages) & 1, kWaitNs));
    }
    if (!ok) {
        if (tid == 0) record_status(ws, AQ_ERR_TIMEOUT);
        // drain: give the issued MMAs one more bounded chance to finish
        if (nk > 0) mbar_wait_ns(&bars[(nk - 1) & 1], ((nk - 1) / kStages) & 1, kWaitNs);
    }
    tc_fence_after();

    if (ok) {
        // Epilogue: warp w owns TMEM lanes 32w..32w+31 = rows m0 + 32w + lane.
        const int row = m0 + warp * 32 + lane;
        const float sc = (row < L.out && scales) ? __half2float(__ushort_as_half(scales[row])) : 1.f;
        const uint32_t tbase = tmem + ((uint32_t)(warp * 32) << 16);
#pragma unroll 1
        for (int c0 = 0; c0 < kBN; c0 += 16) {
            float v[16];
            tmem_ld16(tbase + c0, v);
            if (row < L.out) {
                const int gn = n0 + c0;
                uint16_t *dst = y + (size_t)row * T + gn;
                if (vec_x && gn + 16 <= T) {
                    uint4 o0 = make_uint4(f2h2(sc * v[0], sc * v[1]), f2h2(sc * v[2], sc * v[3]),
                                          f2h2(sc * v[4], sc * v[5]), f2h2(sc * v[6], sc * v[7]));
                    uint4 o1 = make_uint4(f2h2(sc * v[8], sc * v[9]), f2h2(sc * v[10], sc * v[11]),
                                          f2h2(sc * v[12], sc * v[13]), f2h2(sc * v[14], sc * v[15]));
                    reinterpret_cast<uint4 *>(dst)[0] = o0;
                    reinterpret_cast<uint4 *>(dst)[1] = o1;
                } else {
                    for (int j = 0; j < 16; ++j)
                        if (gn + j < T) dst[j] = __half_as_ushort(__float2half_rn(sc * v[j]));
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, kBN);
}


// ---- self-test of the bounded wait -----------------------------------------

__global__ void selftest_wait_kernel(void *ws, int spin_limit)
{
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);  // expects one arrival that never comes
        fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        if (!mbar_wait_bounded(&bar, 0, (uint32_t)spin_limit)) record_status(ws, AQ_ERR_TIMEOUT);
    }
}

}  // namespace aqk

namespace aqh {
using namespace aqk;

static GemmPlan plan_gemm(const Geom &g, int T)
{
    return plan_ws(ws_mtiles<PlainOp>(g), ws_layer_stages<PlainOp>(g), T);
}

// T not a multiple of 8 takes the two-stage kernel, which splits nothing.
size_t gemm_workspace_bytes(const Geom &g, int T) { return T % 8 ? kWsHeader : plan_gemm(g, T).ws_bytes; }

template <class S>
static constexpr int gemm_smem_bytes()
{
    return 1024 /* alignment slack */ + kStages * (kTileABytes + kTileBBytes) + S::kSmemBookBytes +
           kStages * 8 + 16;
}

cudaError_t launch_gemm(const Geom &g, const void *packed, const uint16_t *cb,
                        const uint16_t *scales, const uint16_t *x, int T, uint16_t *y, void *ws,
                        cudaStream_t s, bool pdl)
{
    const uint8_t *pk = reinterpret_cast<const uint8_t *>(packed);
    const uint4 *c = reinterpret_cast<const uint4 *>(cb);
    PFN_cuTensorMapEncodeTiled_v12000 encode = T % 8 == 0 ? tensor_map_encoder() : nullptr;
    if (encode) {
        TensorMaps<1> maps;
        if (!token_map(encode, &maps.m[0], x, g.in, T, T)) return cudaErrorInvalidValue;
        return launch_ws(g, plan_gemm(g, T), maps, PlainOp{{{pk, c, scales}}, y}, T, ws, s, pdl);
    }
    // T not a multiple of 8: rows of X are not 16-byte aligned for TMA; the
    // two-stage kernel stages X with ordinary loads.
    const dim3 grid((g.out + kBM - 1) / kBM, (T + kBN - 1) / kBN);
    return with_scheme(g, [&](auto sch) {
        using S = decltype(sch);
        constexpr int smem = gemm_smem_bytes<S>();
        cudaError_t e = cudaFuncSetAttribute(gemm_tc_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        gemm_tc_kernel<S><<<grid, kGemmThreads, smem, s>>>(g, pk, c, scales, x, T, y, ws);
        return cudaGetLastError();
    });
}

cudaError_t launch_selftest_wait(void *ws, int spin_limit, cudaStream_t s)
{
    selftest_wait_kernel<<<1, 32, 0, s>>>(ws, spin_limit);
    return cudaGetLastError();
}

}  // namespace aqh
