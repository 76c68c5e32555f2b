// Launch plans of the decode-time products (gemv_kernels.cuh): which kernel,
// how the group sum is split, and the launch itself.  Shared by aq_gemv
// (gemv.cu) and its fused and gated forms (gemv_fused.cu).
#pragma once

#include "gemv_kernels.cuh"

namespace aqh {
using namespace aqk;

enum Path { kLut = 1, kTensor = 2, kCudaCores = 3, kRegFrag = 4 };

struct GemvPlan {
    Path path;
    int ks;          // splits of the group sum (grid.y; 1 for stream-K)
    int layers;      // grid.z: 2 for a gated block
    int len;         // tensor: stages per CTA
    bool stream_k;   // tensor: stream-K split (else per row tile)
    int rt_per_cta;  // row tiles per CTA (LUT path)
    int cc_smem;     // CUDA-core path: dynamic shared memory (x, then the split-K staging)
    int grid_x;
    int counters;    // arrival counters: LUT row ranges, tensor row tiles
    int slots;       // partial-sum slots per row range (0: no split-K)
    size_t ws_bytes;
};


// Depends on the shape and batch only, so the workspace size can be
// computed on a host without a GPU.
template <class S>
constexpr int tc_smem_bytes();

// CTAs of gemv_tc_kernel that fit on one SM (228 KiB of shared memory, 1 KiB
// reserved per CTA; 160 threads each, far below the thread limit).
inline int tc_resident_ctas(const Geom &g)
{
    int smem = 0;
    with_scheme(g, [&](auto sch) {
        smem = tc_smem_bytes<decltype(sch)>();
        return cudaSuccess;
    });
    return smem > 0 ? std::max(1, (228 * 1024) / (smem + 1024)) : 1;
}

// Shortest stream-K share: below 4 stages a CTA's fixed costs (prologue,
// pipeline fill and drain, split-K finish) dominate.
constexpr int kTcMinLen = 4;

// Cost of `ctas` CTAs of `len` stages each, `res` of them resident per SM,
// in tenths of the time in which an SM running two CTAs advances both by one
// stage; a model fitted to Llama-2 7B/70B shapes at batch 1..16:
//  * k >= 2 CTAs on an SM share its codeword-read throughput (k len / 2
//    periods); a CTA alone on its SM has half the reads in flight and runs
//    about 1.5x slower per stage;
//  * every wave of CTAs pays about three stages of prologue, pipeline fill
//    and drain and split-K finish;
//  * where the decoders start before the previous launch ends (1x16), fewer
//    than 32 free CTA slots keep the next launch from starting early in
//    them, which exposes the fill and drain (about 1.4 + 0.2 batch stages).
inline long tc_cost(long ctas, int len, int res, int batch, bool early)
{
    const long per_sm = (ctas + kNumSMs - 1) / kNumSMs;
    const long waves = (per_sm + res - 1) / res;
    const long k_last = per_sm - (waves - 1) * res;
    long cost = (waves - 1) * (5L * res * len + 30) + (k_last == 1 ? 15 : 5 * k_last) * (long)len + 30;
    const long last_wave = ctas - (waves - 1) * res * kNumSMs;
    if (early && (long)res * kNumSMs - last_wave < 32) cost += 14 + 2 * batch;
    return cost;
}

// Group splits of the table path: one per kLutGroups groups.
inline int lut_splits(const Geom &g)
{
    const int ng = g.K == 1 ? kLutGroups<1> : kLutGroups<2>;
    return (g.G + ng - 1) / ng;
}

// Row tiles per CTA of the table path: as many row ranges as put one CTA
// on each SM in one wave.
inline int lut_rt_per_cta(const Geom &g, int layers)
{
    const int ranges = std::max(1, std::min(g.rtiles, kNumSMs / (lut_splits(g) * layers)));
    return (g.rtiles + ranges - 1) / ranges;
}

// Partial-sum slots of a row range whose sum is split `ks` ways (a gated
// block always meets in its slots), and their workspace.
inline int split_slots(int ks, int layers) { return ks * layers > 1 ? ks * layers : 0; }
inline size_t slots_ws(const Geom &g, int batch, int slots)
{
    return slots > 0 ? kWsData + (size_t)slots * g.rows8 * batch * sizeof(float) : kWsHeader;
}

// Register-fragment path (1x16 from batch 3, 2x8 from batch 2): groups per
// CTA and group splits.  At most kRfMaxGroups groups per CTA, and few
// enough that two CTAs fit on an SM; about two CTAs per SM in all.
// Returns false when the layer's scheme does not take this path, or when
// the split's partial sums would not fit `cap`.
inline bool plan_rf(const Geom &g, int batch, size_t cap, int layers, GemvPlan &p)
{
    const bool k2 = (g.K == 2 && g.B == 8);
    if (!(k2 || (g.K == 1 && g.B == 16))) return false;
    if (batch < (k2 ? 2 : 3)) return false;
    const int nt = batch <= 8 ? 1 : 2;
    auto smem = [&](int gc) {
        return k2 ? (nt == 1 ? rf_smem_bytes<Scheme<2, 8>, 1>(gc) : rf_smem_bytes<Scheme<2, 8>, 2>(gc))
                  : (nt == 1 ? rf_smem_bytes<Scheme<1, 16>, 1>(gc) : rf_smem_bytes<Scheme<1, 16>, 2>(gc));
    };
    const int rows = k2 ? RfTraits<Scheme<2, 8>>::kRows : RfTraits<Scheme<1, 16>>::kRows;
    const int per_sm_slots = k2 ? RfTraits<Scheme<2, 8>>::kPerSM : RfTraits<Scheme<1, 16>>::kPerSM;
    int gc_max = kRfMaxGroups;  // as many groups as fit the CTAs an SM holds
    while (gc_max > 16 && smem(gc_max) > (per_sm_slots == 1 ? 220 : 113) * 1024) gc_max -= 16;
    const int nrb = (g.rtiles + rows / 8 - 1) / (rows / 8);
    auto ws_of = [&](int gcv) {
        return slots_ws(g, batch, split_slots((g.G + gcv - 1) / gcv, layers));
    };
    // the split (groups per CTA, a multiple of 4) whose busiest SM has the
    // least work: CTAs beyond the two slots of every SM form a second wave,
    // and an SM that runs two CTAs takes about twice as long as one with one
    int gc = std::min(gc_max, (g.G + 3) / 4 * 4);
    double best = 0;
    for (int ks = 1; ks <= (g.G + 3) / 4; ++ks) {
        const int gcv = (g.G + ks - 1) / ks;
        const int gc4 = (gcv + 3) / 4 * 4;
        if (gc4 > gc_max || (g.G + gc4 - 1) / gc4 != ks) continue;
        if (gc4 < std::min(32, (g.G + 3) / 4 * 4)) break;  // at least 8 sets per CTA: fixed costs dominate below
        if (ws_of(gc4) > cap || (ks * layers > 1 && nrb > kWsMaxCounters)) continue;
        const long ctas = (long)nrb * ks * layers;
        const long per_sm = (ctas + kNumSMs - 1) / kNumSMs;  // CTAs on the busiest SM
        double load = (double)per_sm * gc4 + (per_sm > per_sm_slots ? 1e9 : 0);  // groups it works through
        // a gated block has twice the CTAs, often more than fit at once: then
        // the waves count, each with a fixed cost of about 24 groups (1x16
        // 11008 x 4096 at batch 16: 5 splits in 3 waves of 104 groups, 62 us;
        // 2 splits in 2 waves of 256, 73 us; 8 splits 72 us)
        if (layers > 1) {
            const long slots = (long)per_sm_slots * kNumSMs;
            load = ctas <= slots ? (double)per_sm * (gc4 + 24) / per_sm_slots : (double)((ctas + slots - 1) / slots) * (gc4 + 24);
        }
        if (best == 0 || load < best) {
            best = load;
            gc = gc4;
        }
        if (ctas > (long)per_sm_slots * kNumSMs * (layers > 1 ? 8 : 1)) break;
    }
    const int ks = (g.G + gc - 1) / gc;
    if (ws_of(gc) > cap || (ks * layers > 1 && nrb > kWsMaxCounters)) return false;
    p.path = kRegFrag;
    p.len = gc;
    p.ks = ks;
    p.grid_x = nrb;
    p.counters = nrb;
    p.slots = split_slots(ks, layers);
    // shared memory: the kernel's own, or more, so that the last CTA of a
    // row block stages all its splits' partial sums in one pass (one L2
    // round trip), while the CTAs an SM holds still fit
    const size_t stage = (size_t)ks * layers * rows * batch * sizeof(float) + (k2 ? RfTraits<Scheme<2, 8>>::kBookBytes : 0);
    // (a gated 1x16 block keeps more of L1 for its two codebooks instead: 62
    // against 66 us at batch 16)
    const int cap_smem = (per_sm_slots == 1 ? 220 : layers > 1 ? 40 : 113) * 1024;
    p.cc_smem = std::max(smem(gc), (int)std::min<size_t>(stage, (size_t)cap_smem));
    return true;
}

// `cap`: largest workspace the caller can offer (the no-allocation entry
// point's scratch); the plan lengthens the CTAs' shares until its partial
// sums fit, down to one row tile per CTA (no partials).
inline GemvPlan plan_gemv(const Geom &g, int batch, size_t cap = ~(size_t)0, int layers = 1)
{
    GemvPlan p{};
    p.layers = layers;
    const int cc_ranges = (g.rtiles + kCcRowTiles - 1) / kCcRowTiles;
    // 1x16 at batch 1..kCcMaxBatch on the CUDA cores: as many group splits
    // as fill the resident CTA slots in one wave (at most kCcMaxSplits, else
    // too few rows for this path) and at most 1536 / batch groups per split
    // (their x in shared memory)
    const int cc_per_sm = batch == 1 ? kCcPerSMOf<1> : kCcPerSMOf<2>;
    const int cc_ks = std::max(1, std::min((cc_per_sm * kNumSMs) / (cc_ranges * layers), (g.G + 7) / 8));
    const size_t cc_ws = slots_ws(g, batch, split_slots(cc_ks, layers));
    if (batch <= kCcMaxBatch && g.K == 1 && g.B == 16 && cc_ks <= kCcMaxSplits &&
        (g.G + cc_ks - 1) / cc_ks * batch <= 1536 && cc_ws <= cap &&
        (cc_ks * layers == 1 || cc_ranges <= kWsMaxCounters)) {
        p.path = kCudaCores;
        p.grid_x = cc_ranges;
        p.len = (g.G + cc_ks - 1) / cc_ks;  // groups per split
        p.ks = (g.G + p.len - 1) / p.len;
        p.counters = p.grid_x;
        p.slots = split_slots(p.ks, layers);
        const int nvec = kCcRowTiles * 8 * batch / 4;  // float4 of one row range's partial sums
        p.cc_smem = std::max(p.len * 32 * batch, std::min(kCcStage, p.slots * nvec * 16));
    } else if (plan_rf(g, batch, cap, layers, p)) {
        // p is filled in
    } else if (batch == 1 && g.B == 8 && g.K <= 2 && slots_ws(g, 1, split_slots(lut_splits(g), layers)) <= cap) {
        p.path = kLut;
        p.ks = lut_splits(g);
        // one CTA per SM in one wave: every CTA builds its tables once, and
        // a CTA of the next launch fits beside it, so that it can start early
        p.rt_per_cta = lut_rt_per_cta(g, layers);
        p.grid_x = (g.rtiles + p.rt_per_cta - 1) / p.rt_per_cta;
        p.counters = p.grid_x;
        p.slots = split_slots(p.ks, layers);
    } else {
        // the tensor-core path, also for 8-bit codebooks at batch 1 when the
        // table path's partial sums would not fit `cap`
        p.path = kTensor;
        const int mtiles = (g.out + kTcBM - 1) / kTcBM;
        const int nst = (g.G + 7) / 8;
        const long units = (long)mtiles * nst;
        const int res = tc_resident_ctas(g);
        const long slots = (long)res * kNumSMs;
        const bool early = (g.K == 1 && g.B == 16);  // decoders that do not wait for the previous launch
        auto ws_of = [&](int nslots) { return slots_ws(g, batch, nslots); };
        // a split needs one arrival counter per row tile in the fixed area
        const bool may_split = mtiles <= kWsMaxCounters;
        // per row tile: ks splits of `per` stages (the last may be shorter)
        long best_pt = -1;
        p.stream_k = false;
        p.len = nst;
        p.ks = 1;
        for (int ks = 1; ks <= std::max(1, nst / kTcMinLen); ++ks) {
            const int per = (nst + ks - 1) / ks, kk = (nst + per - 1) / per;
            if (kk < ks) continue;  // same split as a smaller ks
            if (kk > 1 && (!may_split || ws_of(split_slots(kk, layers)) > cap)) break;
            const long c = tc_cost((long)mtiles * kk * layers, per, res, batch, early);
            if (best_pt < 0 || c < best_pt) {
                best_pt = c;
                p.len = per;
                p.ks = kk;
            }
        }
        // stream-K: from the share that fills every resident CTA slot in one
        // wave up to one CTA per SM; a row tile meets at most
        // ceil((nst - 1) / len) + 1 shares
        const int lmin = (int)std::min<long>(nst, std::max<long>(kTcMinLen, (units + slots - 1) / slots));
        const int lmax = (int)std::min<long>(nst, std::max<long>(lmin, (units + kNumSMs - 1) / kNumSMs));
        auto sk_slots = [&](int len) { return len >= nst ? 0 : (nst - 1 + len - 1) / len + 1; };
        long best_sk = -1;
        int sk_len = nst;
        for (int len = lmin; len <= lmax && may_split && layers == 1; ++len) {
            if (ws_of(sk_slots(len)) > cap) continue;
            const long c = tc_cost((units + len - 1) / len, len, res, batch, early);
            if (best_sk < 0 || c < best_sk) {
                best_sk = c;
                sk_len = len;
            }
        }
        // stream-K only on a clear predicted gain (the model favours it by
        // a few percent where the per-tile split measures faster: crossing
        // row tiles costs what the model does not see)
        if (best_sk >= 0 && (best_pt < 0 || best_sk * 100 < best_pt * (early ? 95 : 85))) {
            p.stream_k = true;
            p.len = sk_len;
            p.ks = 1;
            p.slots = sk_slots(sk_len);
            p.grid_x = (int)((units + sk_len - 1) / sk_len);
        } else {
            p.slots = split_slots(p.ks, layers);
            p.grid_x = mtiles;
        }
        p.counters = mtiles;
        p.rt_per_cta = kTcBM / 8;
    }
    p.ws_bytes = slots_ws(g, batch, p.slots);
    return p;
}

// ring of (A tile, B tile, x slot) + codebooks + barriers, TMEM slot, flag
template <class S>
constexpr int tc_smem_bytes()
{
    return 1024 + TcRing<S>::depth * kTcTileA + TcRing<S>::xring * (kTcTileB + kTcXSlot) +
           S::kSmemBookBytes * TcRing<S>::kReplicas + (2 * TcRing<S>::depth + TcRing<S>::xring + 1) * 8 + 16;
}

template <class Kern>
cudaError_t set_smem(Kern k, int bytes)
{
    return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// Launch with programmatic stream serialisation: the kernel's weight-only
// prologue may overlap the tail of the previous kernel on the stream; the
// kernel itself waits (griddepcontrol.wait) before touching x, y or the
// workspace.
// With `pdl` false the launch is an ordinary one: the kernel starts only
// after the previous work on the stream has completed (griddepcontrol.wait
// then returns at once).
template <class... KArgs, class... Args>
cudaError_t launch_pdl(bool pdl, void (*kern)(KArgs...), dim3 grid, dim3 block, int smem, cudaStream_t s,
                       Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

template <class Out>
cudaError_t launch_plan(const Geom &g, const GemvPlan &p, const Out &out, const uint16_t *x, int batch, void *ws,
                        cudaStream_t s, bool pdl)
{
    SplitK sk;
    char *base = reinterpret_cast<char *>(ws);
    sk.counters = reinterpret_cast<unsigned *>(base + kWsHeader);
    sk.partials = reinterpret_cast<float *>(base + kWsData);
    const dim3 grid(p.grid_x, p.ks, p.layers);
    cudaError_t e = cudaSuccess;
    if (p.path == kCudaCores) {
        auto cc = [&](auto kern) {
            cudaError_t r = set_smem(kern, p.cc_smem);
            if (r != cudaSuccess) return r;
            return launch_pdl(pdl, kern, grid, dim3(kCcThreads), p.cc_smem, s, g, out, x, sk, p.len,
                              p.cc_smem);
        };
        static_assert(kCcMaxBatch == 2, "one instantiation per batch on this path");
        e = batch == 1 ? cc(gemv_1x16_cc_kernel<1, Out>) : cc(gemv_1x16_cc_kernel<2, Out>);
    } else if (p.path == kRegFrag) {
        auto rf = [&](auto sch, auto ntc) {
            using S = decltype(sch);
            constexpr int NT = decltype(ntc)::value;
            cudaError_t r = set_smem(gemv_rf_kernel<S, NT, Out>, p.cc_smem);
            if (r != cudaSuccess) return r;
            return launch_pdl(pdl, gemv_rf_kernel<S, NT, Out>, grid, dim3(RfTraits<S>::kThreads), p.cc_smem, s, g, out, x,
                              batch, sk, p.len, p.cc_smem);
        };
        using One = std::integral_constant<int, 1>;
        using Two = std::integral_constant<int, 2>;
        if (g.K == 2)
            e = batch <= 8 ? rf(Scheme<2, 8>{}, One{}) : rf(Scheme<2, 8>{}, Two{});
        else
            e = batch <= 8 ? rf(Scheme<1, 16>{}, One{}) : rf(Scheme<1, 16>{}, Two{});
    } else if (p.path == kLut) {
        // The tables and the code rings.  The fused forms ask for enough to have
        // an SM to themselves: with room for a second CTA, launches in a row can
        // settle into a state where some SMs hold two CTAs of one launch and
        // others none (eager calls back to back, 11008 x 4096 at one token:
        // gated 13.2 or 20 us, with SiLU 8.6 or 12.3; alone 13.3 and 8.9)
        const int smem = Out::kFused || Out::kGated ? std::max(kLutSmem, 112 * 1024) : kLutSmem;
        auto lut = [&](auto sch) {
            using S = decltype(sch);
            if constexpr (S::B == 8 && S::K <= 2) {
                auto go = [&](auto kern) {
                    cudaError_t r = set_smem(kern, smem);
                    if (r != cudaSuccess) return r;
                    return launch_pdl(pdl, kern, grid, dim3(kLutThreads), smem, s, g, out, x, sk,
                                      p.rt_per_cta);
                };
                return p.slots > 8 ? go(gemv_lut_kernel<S, true, Out>) : go(gemv_lut_kernel<S, false, Out>);
            } else {
                return cudaErrorInvalidValue;
            }
        };
        e = with_scheme(g, lut);
    } else {
        e = with_scheme(g, [&](auto sch) {
            using S = decltype(sch);
            const int smem = tc_smem_bytes<S>();
            if constexpr (!Out::kGated)
                if (p.stream_k) {
                    cudaError_t r = set_smem(gemv_tc_kernel<S, true, Out>, smem);
                    if (r != cudaSuccess) return r;
                    return launch_pdl(pdl, gemv_tc_kernel<S, true, Out>, dim3(p.grid_x), dim3(kTcThreads), smem, s, g,
                                      out, x, batch, sk, ws, p.len);
                }
            cudaError_t r = set_smem(gemv_tc_kernel<S, false, Out>, smem);
            if (r != cudaSuccess) return r;
            return launch_pdl(pdl, gemv_tc_kernel<S, false, Out>, grid, dim3(kTcThreads), smem, s, g, out, x, batch, sk,
                              ws, p.len);
        });
    }
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace aqh
