// gdr_bwd.cuh -- the gated delta rule's backward pass on the tensor cores (sm_100a): the adjoint's chain and the
// gradients of q, k and the gates.
//
// With the forward's quantities of a chunk (gdr_tc.cuh; P, A' carry β_j, and k̂ = k / |k|), dO = dJ/dY, and dS the
// adjoint of the state that leaves the chunk:
//   dE  = Pᵀ dO + diag(β e^{G_end - G}) K̂ dSᵀ            seeds of the corrections
//   dV  = Tᵀ dE                                            the triangular system's adjoint; dV is v's gradient
//   dS <- e^{G_end} dS + dOᵀ diag(scale e^G) Q̂ - dVᵀ diag(e^G) K̂
// the forward's chain run backwards (ss_gdr_rev_kernel: the same division of work, TMEM lanes = rows v).  The rest is
// parallel over chunks (ss_gdr_grad_kernel), with S the entering state and dS the leaving one's adjoint, kept by the
// two chains:
//   M^P_ij = (dO_i·E_j) e^{G_i - G_j} β_j (j <= i),   M^A_ij = -(dV_i·E_j) e^{G_i - G_j} β_j (j < i)
//   dQ̂ = diag(e^G) dO S + M^P K̂,    dK̂ = -diag(e^G) dV S + diag(β e^{G_end - G}) E dS + M^Pᵀ Q̂ + M^A K̂ + M^Aᵀ K̂
// and for the gates, with <S, dS> of the state that leaves the chunk (every term of Y and of S that carries e^{G_i}
// is a term of dO_i·Y_i, and every e^{-G_i} one of dV_i·V_i, which is what makes the sums this short):
//   dlog α_t = <S, dS> + Σ_{i >= t} (dO_i·Y_i - dV_i·V_i) over the chunk,     dβ_j = dV_j·E_j / β_j
// A chunk's sum starts from its own <S, dS>, so rounding does not pile up over a long sequence.
//
// Precision: the chain as in the forward (fp32 operands as two bf16 terms; the sums for the gates in fp32).  dQ and
// dK leave as bf16, and their products read E, dV, S, dS, M rounded once to bf16.
#pragma once

#include "gdr_tc.cuh"

namespace selscan {
namespace gdr {

// ---------------------------------------------------------------------------------------- the adjoint's chain
// TMEM columns.  S: dS's terms, then its update; A: K dSᵀ, then dE's terms over it; R: Pᵀ dO in two halves (P's terms);
// V: Tᵀ dE in two halves, then the terms of -e^G dV over the first; O: the terms of scale e^G dO.
constexpr uint32_t kRevS = 0, kRevA = 128, kRevR = 192, kRevV = 320, kRevO = 448;
// Shared memory: two stages of [K 0][Q 0][K 1][Q 1][record]; then, once each, dO and V (swizzled blocks), E's image, and
// dV staged for its store.
constexpr uint32_t kRevStage = 4 * kTile + kRecBytes, kRevOffRec = 4 * kTile;
constexpr uint32_t kRevOffO = 2 * kRevStage, kRevOffV = kRevOffO + 2 * kTile, kRevOffE = kRevOffV + 2 * kTile;
constexpr uint32_t kRevOffOut = kRevOffE + 2 * kTile, kRevOffDot = kRevOffOut + 2 * kTile;
constexpr uint32_t kRevOffBar = kRevOffDot + 2 * 4 * kC * 4 + 2 * 16 * 4;
constexpr uint32_t kRevSmem = kRevOffBar + 256 + 1024;
static_assert(kRevStage % 1024 == 0 && kRevSmem <= 227 * 1024, "shared memory");

struct RevBars {
    uint64_t full[2], empty[2];      // K, Q and the record of a stage
    uint64_t o_full, o_free;         // dO landed; read (state warps, after its product)
    uint64_t ve_full, ve_free;       // V and E landed; read (state warps)
    uint64_t ks, e, ds;              // products done
    uint64_t s_ready[2], x_ready, w_ready;
    uint64_t out_full, out_free;     // dV and the sums staged (state warps); stored (1)
    uint64_t fin;
    uint32_t tmem;
};
static_assert(sizeof(RevBars) <= 256, "barrier region");

// Grid: one CTA per (b, h).  tm_o reads dO and tm_v V in swizzled blocks, tm_dv writes dV unswizzled.
template <int DK>
__global__ void __launch_bounds__(kThreads, 1)
ss_gdr_rev_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tm_q,
                  const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ CUtensorMap tm_dv) {
    constexpr int KB = DK / 64, KH = DK / kParts;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* gbase = smem_raw + (base - raw);
    RevBars* const bar = reinterpret_cast<RevBars*>(gbase + kRevOffBar);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const GdrParams& g = p.g;
    const int item = blockIdx.x, b = item / g.H, h = item % g.H, hk = h / (g.H / g.Hk);
    const int64_t len = gdr_len(g, b);
    const int nchunk = static_cast<int>((len + kC - 1) / kC);
    const bool ragged = len % kC != 0 && len < g.L;   // other tokens follow in the last chunk's tiles
    const uint64_t lim = p.wait_ns;
    const int64_t toks = p.nchunks * kC;

    if (tid == 0) {
        uint64_t* one[] = {bar->full, bar->full + 1, bar->empty, bar->empty + 1, &bar->o_full, &bar->ve_full, &bar->ks,
                           &bar->e,   &bar->ds,      &bar->out_free, &bar->fin};
        for (uint64_t* x : one) mbar_init(x, 1);
        uint64_t* all[] = {&bar->o_free, &bar->ve_free, bar->s_ready, bar->s_ready + 1, &bar->x_ready, &bar->w_ready,
                           &bar->out_full};
        for (uint64_t* x : all) mbar_init(x, kStateWarps);
        fence_mbar_init();
    }
    if (warp == 0) {
        tc::tmem_alloc(&bar->tmem, kTmemCols);
        tc::tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem;

    auto record = [&]() {
        if (p.status) atomicCAS(p.status, 0u, static_cast<uint32_t>(SS_ERR_TIMEOUT));
    };
    auto wait1 = [&](uint64_t* x, uint32_t parity) {
        if (mbar_wait_bounded(x, parity, lim)) return true;
        record();
        return false;
    };
    auto wait_warp = [&](uint64_t* x, uint32_t parity) {
        const bool got = __all_sync(0xffffffffu, mbar_wait_bounded(x, parity, lim));
        if (!got && lane == 0) record();
        return got;
    };
    auto arrive_warp = [&](uint64_t* x) {
        __syncwarp();
        if (lane == 0) mbar_arrive(x);
    };
    int issued = 0, o_issued = 0, ve_issued = 0;

    // Step n handles chunk nchunk - 1 - n.
    if (warp == kLoadWarp) {
        if (lane == 0) {
            for (int n = 0; n < nchunk; ++n) {
                const int c = nchunk - 1 - n, s = n & 1;
                if (n >= 2 && !wait1(&bar->empty[s], ((n >> 1) - 1) & 1)) break;
                const uint32_t st = base + s * kRevStage;
                uint64_t* f = &bar->full[s];
                mbar_arrive_expect_tx(f, 2 * KB * kTile + kRecBytes);
                for (int kb = 0; kb < KB; ++kb) {
                    tma_load_4d(st + (2 * kb) * kTile, &tm_k, 64 * kb, hk, c * kC, b, f);
                    tma_load_4d(st + (2 * kb + 1) * kTile, &tm_q, 64 * kb, hk, c * kC, b, f);
                }
                bulk_load(st + kRevOffRec, p.rec + (item * p.nchunks + c) * p.rec_bytes, kRecBytes, f);
                issued = n + 1;
                if (n >= 1 && !wait1(&bar->o_free, (n - 1) & 1)) break;
                mbar_arrive_expect_tx(&bar->o_full, kC * p.dv * 2);
                for (int vb = 0; vb < p.dv / 64; ++vb)
                    tma_load_4d(base + kRevOffO + vb * kTile, &tm_o, 64 * vb, h, c * kC, b, &bar->o_full);
                o_issued = n + 1;
                if (n >= 1 && !wait1(&bar->ve_free, (n - 1) & 1)) break;
                mbar_arrive_expect_tx(&bar->ve_full, kC * p.dv * 4);
                for (int vb = 0; vb < p.dv / 64; ++vb)
                    tma_load_4d(base + kRevOffV + vb * kTile, &tm_v, 64 * vb, h, c * kC, b, &bar->ve_full);
                bulk_load(base + kRevOffE, p.keep + (item * (p.nchunks + 1) + c) * kKeepBytes + kKeepE, kC * p.dv * 2,
                          &bar->ve_full);
                ve_issued = n + 1;
            }
        }
        __syncwarp();
    } else if (warp == kStoreWarp) {
        for (int n = 0; n < nchunk; ++n) {
            const int c = nchunk - 1 - n;
            if (!wait_warp(&bar->out_full, n & 1)) break;
            if (lane == 0) {   // rows behind a sequence's end are zero rows: dO is zero there
                tc::tma_store_4d(&tm_dv, base + kRevOffOut, 0, h, c * kC, b);
                tc::bulk_commit();
            }
            const float* q = reinterpret_cast<const float*>(gbase + kRevOffDot);
#pragma unroll
            for (int w = 0; w < 2; ++w) {   // dV·V, dV·E: the four lane groups, in order
                const float* d = q + w * 4 * kC;
                float* out = p.dots + (w + 1) * (static_cast<int64_t>(g.batch) * g.H * toks) + item * toks + static_cast<int64_t>(c) * kC;
                for (int i = lane; i < kC; i += 32) out[i] = (d[i] + d[kC + i]) + (d[2 * kC + i] + d[3 * kC + i]);
            }
            float a = q[8 * kC + (n & 1) * 16 + (lane & 15)];   // <S, dS>: the sixteen warps' sums
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
            if (lane == 0) {
                p.dots[3 * (static_cast<int64_t>(g.batch) * g.H * toks) + item * p.nchunks + c] = a;
                tc::bulk_wait_read0();
            }
            arrive_warp(&bar->out_free);
        }
        if (lane == 0) bulk_wait0();
        __syncwarp();
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            const uint32_t lbo = p.dv == 128 ? kTile : 0;   // d_v 64: the lanes 64.. repeat the rows 0..63
            for (int n = 0; n < nchunk; ++n) {
                const int s = n & 1;
                const uint32_t par = n & 1, st = base + s * kRevStage, pr = st + kRevOffRec;
                if (!wait1(&bar->full[s], (n >> 1) & 1)) break;
                if (!wait1(&bar->o_full, par)) break;
                if (n == 0 && !wait1(&bar->s_ready[0], 0)) break;   // the tiles' rows behind the end are zero by then
                tc_fence_after();
                // R = dOᵀ P, P's terms side by side (their columns were read before dE's terms were handed over)
#pragma unroll
                for (int j = 0; j < kC / 16; ++j)
                    umma(tmem + kRevR, sdesc(base + kRevOffO + 2048u * j, lbo, 1024), sdesc(pr + kRecP + 2048u * j, kTile, 1024),
                         idesc(2 * kC, true, true), j > 0);
                auto ks_step = [&](int ks) {
                    const uint64_t bd = sdesc(st + (ks >> 2) * 2 * kTile + (ks & 3) * 32, 16, 1024);
                    umma_ts(tmem + kRevA, tmem + kRevS + 16 * ks, bd, idesc(kC, false), ks > 0);
                    umma_ts(tmem + kRevA, tmem + kRevS + 16 * ks + 8, bd, idesc(kC, false), 1);
                };
                constexpr int kStep = KH / 16;
                if (!wait1(&bar->s_ready[0], par)) break;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < DK / 16; ks += kStep) ks_step(ks);
                if (!wait1(&bar->s_ready[1], par)) break;
                tc_fence_after();
                if (kStep == 2) {
#pragma unroll
                    for (int ks = 1; ks < DK / 16; ks += 2) ks_step(ks);
                }
                umma_commit(&bar->ks);
                if (!wait1(&bar->x_ready, par)) break;
                tc_fence_after();
                // Vᵀ = dEᵀ T
#pragma unroll
                for (int j = 0; j < kC / 16; ++j) {
                    const uint64_t bd = sdesc(pr + kRecT + 2048u * j, kTile, 1024);
                    umma_ts(tmem + kRevV, tmem + kRevA + 16 * j, bd, idesc(2 * kC, true), j > 0);
                    umma_ts(tmem + kRevV, tmem + kRevA + 16 * j + 8, bd, idesc(kC, true), 1);
                }
                umma_commit(&bar->e);
                // dS's update: (scale e^G dO)ᵀ Q, then (-e^G dV)ᵀ K, over the columns of dS's terms
#pragma unroll
                for (int j = 0; j < kC / 16; ++j) {
                    const uint64_t bd = sdesc(st + kTile + 2048u * j, 2 * kTile, 1024);
                    umma_ts(tmem + kRevS, tmem + kRevO + 16 * j, bd, idesc(DK, true), j > 0);
                    umma_ts(tmem + kRevS, tmem + kRevO + 16 * j + 8, bd, idesc(DK, true), 1);
                }
                if (!wait1(&bar->w_ready, par)) break;
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < kC / 16; ++j) {
                    const uint64_t bd = sdesc(st + 2048u * j, 2 * kTile, 1024);
                    umma_ts(tmem + kRevS, tmem + kRevV + 16 * j, bd, idesc(DK, true), 1);
                    umma_ts(tmem + kRevS, tmem + kRevV + 16 * j + 8, bd, idesc(DK, true), 1);
                }
                umma_commit(&bar->ds);
                umma_commit(&bar->empty[s]);
            }
        }
        __syncwarp();
    } else if (warp < kStateWarps) {
        const int v = (warp & 3) * 32 + lane, part = warp >> 2;
        const bool row_in = v < p.dv;
        const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const int64_t srow = (static_cast<int64_t>(item) * p.dv + v) * DK + part * KH;
        f32x2 S[KH / 2];   // dS
#pragma unroll
        for (int k = 0; k < KH; k += 4) {
            float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (p.dfinal && row_in) q = quad(p.dfinal + srow + k);
            S[k / 2] = pk2(q.x, q.y);
            S[k / 2 + 1] = pk2(q.z, q.w);
        }
#pragma unroll
        for (int k = 0; k < KH; k += 16) store_terms(tl + kRevS + part * KH + k, S + k / 2);
        tmem_wait_st();
        tc_fence_before();
        // a bf16 value of token kTok · part + e, row v, of a swizzled [64][d_v] tile
        auto val = [&](uint32_t off, int e) {
            const uint32_t t = kTok * part + e;
            const uint32_t a = chunk_addr(off + static_cast<uint32_t>(v >> 6) * kTile, t, (v & 63) >> 3) + 2 * (v & 7);
            return row_in ? __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(gbase + a)) : 0.0f;
        };
        float* const dots = reinterpret_cast<float*>(gbase + kRevOffDot);
        bool ok = true;
        for (int n = 0; n < nchunk; ++n) {
            const int c = nchunk - 1 - n, s = n & 1;
            const uint32_t par = n & 1, st = base + s * kRevStage;
            const Scal& sc = *reinterpret_cast<const Scal*>(gbase + s * kRevStage + kRevOffRec + kRecScal);
            if (n == 0) {
                if (ragged) {   // rows behind the end, whatever they hold, become zero rows
                    ok = wait_warp(&bar->full[0], 0) && wait_warp(&bar->o_full, 0) && wait_warp(&bar->ve_full, 0);
                    if (!ok) break;
                    const int n0 = static_cast<int>(len - static_cast<int64_t>(c) * kC);
                    for (int i = n0 * 8 + tid; i < kC * 8; i += 32 * kStateWarps) {
                        for (int kb = 0; kb < 2 * KB; ++kb) sts128(st + kb * kTile + 16 * i, make_uint4(0, 0, 0, 0));
                        for (int vb = 0; vb < p.dv / 64; ++vb) {
                            sts128(base + kRevOffO + vb * kTile + 16 * i, make_uint4(0, 0, 0, 0));
                            sts128(base + kRevOffV + vb * kTile + 16 * i, make_uint4(0, 0, 0, 0));
                        }
                    }
                    fence_proxy_async_smem();
                }
                arrive_warp(&bar->s_ready[0]);
                arrive_warp(&bar->s_ready[1]);
                // (the zero rows of other warps' share are visible behind the product's own barrier)
            }
            {   // keep dS, and <S, dS> of the state that leaves the chunk
                unsigned char* kp = p.keep + (item * (p.nchunks + 1) + c) * kKeepBytes;
                const unsigned char* sp = kp + kKeepBytes;
                float dot = 0.0f;
#pragma unroll
                for (int k = 0; k < KH; k += 16) {
                    const int key = part * KH + k;
                    keep_terms(kp + kKeepD, nullptr, v, key, S + k / 2);
#pragma unroll
                    for (int h2 = 0; h2 < 2; ++h2) {
                        const uint32_t o = chunk_addr(static_cast<uint32_t>(key >> 6) * 2 * kTile, v, ((key & 63) >> 3) + h2);
                        const uint4 hi = *reinterpret_cast<const uint4*>(sp + kKeepShi + o);
                        const uint4 lo = *reinterpret_cast<const uint4*>(sp + kKeepSlo + o);
                        const uint32_t hw[4] = {hi.x, hi.y, hi.z, hi.w}, lw[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const f32x2 d = S[k / 2 + 4 * h2 + e];
                            dot = fmaf(d.x, lo_f(hw[e]) + lo_f(lw[e]), dot);
                            dot = fmaf(d.y, hi_f(hw[e]) + hi_f(lw[e]), dot);
                        }
                    }
                }
                if (!row_in) dot = 0.0f;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                // (two buffers: the sums of step n - 1 may still wait for their store)
                if (lane == 0) dots[8 * kC + (n & 1) * 16 + warp] = dot;
            }
            ok = wait_warp(&bar->full[s], (n >> 1) & 1) && wait_warp(&bar->o_full, par);
            if (!ok) break;
            f32x2 x[8];
            if (!(n == 0 && ragged)) {   // scale e^G dO (in a ragged chunk once every warp's zero rows are written)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = pk2(val(kRevOffO, 2 * e), val(kRevOffO, 2 * e + 1));
                scale16(x, sc.qe + kTok * part);
                store_terms(tl + kRevO + kTok * part, x);
            }
            ok = wait_warp(&bar->ks, par);
            if (!ok) break;
            tc_fence_after();
            if (n == 0 && ragged) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = pk2(val(kRevOffO, 2 * e), val(kRevOffO, 2 * e + 1));
                scale16(x, sc.qe + kTok * part);
                store_terms(tl + kRevO + kTok * part, x);
            }
            {
                f32x2 w[8];
                tmem_ld16(tl + kRevA + kTok * part, x);
                scale16(x, sc.wk + kTok * part);
                tmem_ld16(tl + kRevR + kTok * part, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = add2(x[e], w[e]);
                tmem_ld16(tl + kRevR + kC + kTok * part, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = add2(x[e], w[e]);
            }
            store_terms(tl + kRevA + kTok * part, x);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar->x_ready);
                mbar_arrive(&bar->o_free);
            }
            ok = wait_warp(&bar->e, par);
            if (!ok) break;
            tc_fence_after();
            {
                f32x2 w[8];
                tmem_ld16x2(tl + kRevV + kTok * part, tl + kRevV + kC + kTok * part, x, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = add2(x[e], w[e]);
                    w[e] = x[e];
                }
                scale16(w, sc.ek + kTok * part);
                store_terms(tl + kRevV + kTok * part, w);
            }
            const float end = sc.end[0];
            tmem_wait_st();
            tc_fence_before();
            arrive_warp(&bar->w_ready);
            // dV, and its products with V and E, while dS is multiplied
            ok = wait_warp(&bar->ve_full, par) && (n == 0 || wait_warp(&bar->out_free, (n - 1) & 1));
            if (!ok) break;
            if (row_in) {
                __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(gbase + kRevOffOut) + kTok * part * p.dv + v;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    o[2 * e * p.dv] = __float2bfloat16_rn(x[e].x);
                    o[(2 * e + 1) * p.dv] = __float2bfloat16_rn(x[e].y);
                }
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                float d[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    d[e] = ((e & 1) ? x[e >> 1].y : x[e >> 1].x) * val(w == 0 ? kRevOffV : kRevOffE, e);
                if (!row_in) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) d[e] = 0.0f;
                }
                const float sum = lane_sums16(d, lane);
                if (!(lane & 1)) dots[(4 * w + (warp & 3)) * kC + kTok * part + (lane >> 1)] = sum;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar->ve_free);
                mbar_arrive(&bar->out_full);
            }
            ok = wait_warp(&bar->ds, par);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < KH; k += 16) {
                tmem_ld16(tl + kRevS + part * KH + k, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) S[k / 2 + e] = fma2(pk2(end, end), S[k / 2 + e], x[e]);
                store_terms(tl + kRevS + part * KH + k, S + k / 2);
                if (n + 1 < nchunk) {
                    tmem_wait_st();
                    tc_fence_before();
                    arrive_warp(&bar->s_ready[k / 16]);
                    if (KH == 16) arrive_warp(&bar->s_ready[1]);
                }
            }
            tmem_wait_st();
            tc_fence_before();
        }
        if (ok && p.dinit && row_in) {
#pragma unroll
            for (int k = 0; k < KH; k += 4)
                *reinterpret_cast<float4*>(p.dinit + srow + k) = make_float4(S[k / 2].x, S[k / 2].y, S[k / 2 + 1].x, S[k / 2 + 1].y);
        }
        tc_fence_before();
    }

    __syncthreads();
    if (warp == kLoadWarp && lane == 0) {
        for (int n = issued > 2 ? issued - 2 : 0; n < issued; ++n)
            mbar_wait_bounded(&bar->full[n & 1], (n >> 1) & 1, p.drain_ns);
        if (o_issued) mbar_wait_bounded(&bar->o_full, (o_issued - 1) & 1, p.drain_ns);
        if (ve_issued) mbar_wait_bounded(&bar->ve_full, (ve_issued - 1) & 1, p.drain_ns);
    }
    if (tid == 32 * kMmaWarp) {
        umma_commit(&bar->fin);
        mbar_wait_bounded(&bar->fin, 0, p.drain_ns);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------------------------ gradients of q and k
// One block per (b, key head, chunk); the value heads that share the key head one after the other, their sums in
// fp32 registers.  Per value head (M = 128 lanes, two 64-row operands on top of one another):
//   D1 [dO; dV] S              -> columns   0 .. 127 (K: d_v)
//   D3 [E; .] dS               ->         128 .. 255 (K: d_v; lanes 64.. are not read)
//   D2 [dO; dV] Eᵀ             ->         384 .. 447 (K: d_v), read into M^P, M^A (bf16, shared memory)
//   D4 [M^P; M^A] K            ->         256 .. 383 (K: 64 tokens)
//   D5 [M^P; M^A]ᵀ [Q; K]      ->         384 .. 511 (K: 128; lanes 64.. are not read)
//   dq~ = qe D1 + D4 (lanes 0..63),   dk~ = ek D1 + D4 (lanes 64..127) + wk D3 + D5 (lanes 0..63)
// (ek carries the minus of -e^G.)  Bound by latency: loads, two rounds of products, and the M's between them.
constexpr int kGradThreads = 256;
constexpr uint32_t kGK = 0;                       // [K 0][Q 0][K 1][Q 1]
constexpr uint32_t kGO = 4 * kTile;               // [dO 0][dV 0][dO 1][dV 1]
constexpr uint32_t kGE = 8 * kTile;               // [E 0][E 1] (an operand of 128 rows reads on into S: not used)
constexpr uint32_t kGS = 10 * kTile;              // S: two blocks of 128 rows
constexpr uint32_t kGD = 14 * kTile;              // dS
constexpr uint32_t kGM = 18 * kTile;              // [M^P][M^A], 64 rows of 64 each
constexpr uint32_t kGX = 20 * kTile;              // dk~'s other half, fp32 [64][DK + 4]
constexpr uint32_t kGScal = kGX + 64 * 132 * 4;   // Scal, Local (one copy from the record)
constexpr uint32_t kGBar = kGScal + 1024 + 2048;
constexpr uint32_t kGradSmem = kGBar + 128 + 1024;
static_assert(kGradSmem <= 227 * 1024, "shared memory");

struct GradBars {
    uint64_t qk, in, m1, m2;
    uint32_t tmem;
};

struct GradParams {
    Params p;
    __nv_bfloat16 *dq, *dk, *dv;
};

template <int DK>
__global__ void __launch_bounds__(kGradThreads, 1)
ss_gdr_grad_kernel(const __grid_constant__ GradParams gp, const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_o,
                   const __grid_constant__ CUtensorMap tm_dv) {
    constexpr int KB = DK / 64, CN = DK / 2;   // CN: columns of a thread
    const Params& p = gp.p;
    const GdrParams& g = p.g;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* gbase = smem_raw + (base - raw);
    GradBars* const bar = reinterpret_cast<GradBars*>(gbase + kGBar);
    const Scal& sc = *reinterpret_cast<const Scal*>(gbase + kGScal);
    const Local& lo = *reinterpret_cast<const Local*>(gbase + kGScal + 1024);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t c = blockIdx.x % p.nchunks, bk = blockIdx.x / p.nchunks;
    const int b = static_cast<int>(bk / g.Hk), hk = static_cast<int>(bk % g.Hk), rep = g.H / g.Hk;
    const int64_t t0 = c * kC, left = gdr_len(g, b) - t0;
    const int rows = static_cast<int>(g.L - t0 < kC ? g.L - t0 : kC);   // rows that exist
    const int valid = left < kC ? static_cast<int>(left) : kC;          // rows of the sequence
    if (valid <= 0) {   // behind the sequence's end every gradient is zero
        const uint4 z = make_uint4(0, 0, 0, 0);
        for (int i = tid; i < rows * (DK / 8); i += kGradThreads) {
            const int64_t o = ((static_cast<int64_t>(b) * g.L + t0 + i / (DK / 8)) * g.Hk + hk) * DK + 8 * (i % (DK / 8));
            *reinterpret_cast<uint4*>(gp.dq + o) = z;
            *reinterpret_cast<uint4*>(gp.dk + o) = z;
        }
        const int w = rep * p.dv / 8;   // the value heads of a key head are neighbours
        for (int i = tid; i < rows * w; i += kGradThreads)
            *reinterpret_cast<uint4*>(gp.dv + ((static_cast<int64_t>(b) * g.L + t0 + i / w) * g.H + hk * rep) * p.dv + 8 * (i % w)) = z;
        return;
    }
    if (tid == 0) {
        mbar_init(&bar->qk, 1);
        mbar_init(&bar->in, 1);
        mbar_init(&bar->m1, 1);
        mbar_init(&bar->m2, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tc::tmem_alloc(&bar->tmem, kTmemCols);
        tc::tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem;
    const int t = static_cast<int>(t0);
    if (tid == 0) {
        mbar_arrive_expect_tx(&bar->qk, 2 * KB * kTile);
        for (int kb = 0; kb < KB; ++kb) {
            tma_load_4d(base + kGK + (2 * kb) * kTile, &tm_k, 64 * kb, hk, t, b, &bar->qk);
            tma_load_4d(base + kGK + (2 * kb + 1) * kTile, &tm_q, 64 * kb, hk, t, b, &bar->qk);
        }
    }
    // thread: lane row r of TMEM (token r & 63; dq~ below 64, dk~ from 64 on), columns CN · half ..
    const int r = (warp & 3) * 32 + lane, half = warp >> 2, i = r & 63, rb = (r >> 5) & 1;
    const bool is_k = r >= 64;
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float acc[CN];   // dq~ or dk~ of this thread's row and columns
#pragma unroll
    for (int e = 0; e < CN; ++e) acc[e] = 0.0f;
    float* const xch = reinterpret_cast<float*>(gbase + kGX);
    bool bad = false;
    for (int j = 0; j < rep && !bad; ++j) {
        const int h = hk * rep + j;
        const int64_t item = static_cast<int64_t>(b) * g.H + h;
        const uint32_t par = j & 1;
        if (tid == 0) {
            const unsigned char* kp = p.keep + (item * (p.nchunks + 1) + c) * kKeepBytes;
            const uint32_t vb = p.dv / 64;
            mbar_arrive_expect_tx(&bar->in, vb * 3 * kTile + 2 * KB * 2 * kTile + 1024 + sizeof(Local));
            for (uint32_t w = 0; w < vb; ++w) {
                tma_load_4d(base + kGO + 2 * w * kTile, &tm_o, 64 * w, h, t, b, &bar->in);
                tma_load_4d(base + kGO + (2 * w + 1) * kTile, &tm_dv, 64 * w, h, t, b, &bar->in);
            }
            bulk_load(base + kGE, kp + kKeepE, vb * kTile, &bar->in);
            bulk_load(base + kGS, kp + kKeepShi, KB * 2 * kTile, &bar->in);
            bulk_load(base + kGD, kp + kKeepD, KB * 2 * kTile, &bar->in);
            bulk_load(base + kGScal, p.rec + (item * p.nchunks + c) * p.rec_bytes + kRecScal, 1024 + sizeof(Local), &bar->in);
        }
        bool got = mbar_wait_bounded(&bar->in, par, p.wait_ns);
        if (j == 0) {
            got = mbar_wait_bounded(&bar->qk, 0, p.wait_ns) && got;
        }
        if (valid < kC && got) {   // rows behind the sequence's end: K, Q (once) and dO become zero rows (dV has them)
            for (int w = valid * 8 + tid; w < kC * 8; w += kGradThreads) {
                for (int kb = 0; kb < 2 * KB && j == 0; ++kb) sts128(base + kGK + kb * kTile + 16 * w, make_uint4(0, 0, 0, 0));
                for (int vb = 0; vb < p.dv / 64; ++vb) sts128(base + kGO + 2 * vb * kTile + 16 * w, make_uint4(0, 0, 0, 0));
            }
            fence_proxy_async_smem();
        }
        bad = __syncthreads_or(!got) != 0;
        if (bad) break;
        if (tid == 0) {
            const int vs = p.dv / 16;
            for (int ks = 0; ks < vs; ++ks) {   // D2 first: the M's wait for it
                const uint32_t o = (ks >> 2) * 2 * kTile + (ks & 3) * 32, e = (ks >> 2) * kTile + (ks & 3) * 32;
                umma(tmem + 384, sdesc(base + kGO + o, 16, 1024), sdesc(base + kGE + e, 16, 1024), idesc(kC, false), ks > 0);
            }
            umma_commit(&bar->m1);
            for (int ks = 0; ks < vs; ++ks) {
                const uint32_t o = (ks >> 2) * 2 * kTile + (ks & 3) * 32, e = (ks >> 2) * kTile + (ks & 3) * 32;
                umma(tmem, sdesc(base + kGO + o, 16, 1024), sdesc(base + kGS + 2048u * ks, 2 * kTile, 1024), idesc(DK, true), ks > 0);
                umma(tmem + 128, sdesc(base + kGE + e, 16, 1024), sdesc(base + kGD + 2048u * ks, 2 * kTile, 1024), idesc(DK, true), ks > 0);
            }
        }
        got = mbar_wait_bounded(&bar->m1, par, p.wait_ns);
        bad = __syncthreads_or(!got) != 0;
        if (bad) break;
        tc_fence_after();
        {   // M^P (rows 0..63), M^A (64..127): one 32-column block per thread
            const uint32_t blk = base + kGM + (is_k ? kTile : 0);
            float v[32];
            const bool diag = half == rb;
            if (diag || half < rb) {
                tmem_ld32(tl + 384 + 32 * half, v);
                const float row = is_k ? -lo.rk[i] : lo.rq[i];
                if (diag) decay_diagonal(v, lo, 32 * rb, lo.gh[i], lo.gl[i], row, i & 31, !is_k);
                else decay_left(v, lo, lo.gh[i], lo.gl[i], row);
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = 0.0f;
            }
#pragma unroll
            for (int w = 0; w < 4; ++w)
                sts128(chunk_addr(blk, i, 4 * half + w),
                       make_uint4(pk(v[8 * w], v[8 * w + 1]), pk(v[8 * w + 2], v[8 * w + 3]), pk(v[8 * w + 4], v[8 * w + 5]),
                                  pk(v[8 * w + 6], v[8 * w + 7])));
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < kC / 16; ++ks)
                umma(tmem + 256, sdesc(base + kGM + 32u * ks, 16, 1024), sdesc(base + kGK + 2048u * ks, 2 * kTile, 1024),
                     idesc(DK, true), ks > 0);
#pragma unroll
            for (int ks = 0; ks < 2 * kC / 16; ++ks) {   // rows r of [M^P; M^A] with rows r of [Q; K]
                const uint32_t qk = base + kGK + (ks < 4 ? kTile : 0) + 2048u * (ks & 3);
                umma(tmem + 384, sdesc(base + kGM + 2048u * ks, 0, 1024), sdesc(qk, 2 * kTile, 1024), idesc(DK, true, true), ks > 0);
            }
            umma_commit(&bar->m2);
        }
        got = mbar_wait_bounded(&bar->m2, par, p.wait_ns);
        bad = __syncthreads_or(!got) != 0;
        if (bad) break;
        tc_fence_after();
        const float f1 = is_k ? sc.ek[i] : sc.qe[i], f3 = sc.wk[i];
#pragma unroll
        for (int e = 0; e < CN; e += 32) {
            float v[32], w[32];
            tmem_ld32(tl + CN * half + e, v);
            tmem_ld32(tl + 256 + CN * half + e, w);
#pragma unroll
            for (int x = 0; x < 32; ++x) acc[e + x] += fmaf(f1, v[x], w[x]);
            if (!is_k) {   // dk~'s terms that lie in the lanes below 64
                tmem_ld32(tl + 128 + CN * half + e, v);
                tmem_ld32(tl + 384 + CN * half + e, w);
#pragma unroll
                for (int x = 0; x < 32; x += 4)
                    *reinterpret_cast<float4*>(xch + i * 132 + CN * half + e + x) =
                        make_float4(fmaf(f3, v[x], w[x]), fmaf(f3, v[x + 1], w[x + 1]), fmaf(f3, v[x + 2], w[x + 2]),
                                    fmaf(f3, v[x + 3], w[x + 3]));
            }
        }
        tc_fence_before();
        __syncthreads();
        if (is_k) {
#pragma unroll
            for (int x = 0; x < CN; x += 4) {
                const float4 q = quad(xch + i * 132 + CN * half + x);
                acc[x] += q.x;
                acc[x + 1] += q.y;
                acc[x + 2] += q.z;
                acc[x + 3] += q.w;
            }
        }
        // (the next head's loads overwrite nothing that is still read: the barrier above, and xch is written two
        // barriers later)
    }
    if (!bad) {
        // the unit length's own derivative: d = d~ - x (x·d~) / |x|²; the row's two halves meet in shared memory
        const uint32_t own = base + kGK + (is_k ? 0 : kTile);   // this row of K or Q
        float x2 = 0.0f, xd = 0.0f;
        __syncthreads();
        if (g.l2norm) {
#pragma unroll
            for (int w = 0; w < CN / 8; ++w) {
                const int col = CN * half + 8 * w;
                const uint4 q = lds128(chunk_addr(own + (col >> 6) * 2 * kTile, i, (col & 63) >> 3));
                const uint32_t a[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x2 = fmaf(lo_f(a[e]), lo_f(a[e]), fmaf(hi_f(a[e]), hi_f(a[e]), x2));
                    xd = fmaf(lo_f(a[e]), acc[8 * w + 2 * e], fmaf(hi_f(a[e]), acc[8 * w + 2 * e + 1], xd));
                }
            }
            xch[2 * (128 * half + r)] = x2;
            xch[2 * (128 * half + r) + 1] = xd;
        }
        __syncthreads();
        if (g.l2norm) {
            x2 += xch[2 * (128 * (half ^ 1) + r)];
            xd += xch[2 * (128 * (half ^ 1) + r) + 1];
            const float f = -xd / (x2 + kGdrL2Eps);
#pragma unroll
            for (int w = 0; w < CN / 8; ++w) {
                const int col = CN * half + 8 * w;
                const uint4 q = lds128(chunk_addr(own + (col >> 6) * 2 * kTile, i, (col & 63) >> 3));
                const uint32_t a[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[8 * w + 2 * e] = fmaf(f, lo_f(a[e]), acc[8 * w + 2 * e]);
                    acc[8 * w + 2 * e + 1] = fmaf(f, hi_f(a[e]), acc[8 * w + 2 * e + 1]);
                }
            }
        }
        if (i < rows) {
            __nv_bfloat16* out = (is_k ? gp.dk : gp.dq) + ((static_cast<int64_t>(b) * g.L + t0 + i) * g.Hk + hk) * DK + CN * half;
#pragma unroll
            for (int w = 0; w < CN / 8; ++w) {
                const float* a = acc + 8 * w;
                const bool live = i < valid;
                *reinterpret_cast<uint4*>(out + 8 * w) =
                    live ? make_uint4(pk(a[0], a[1]), pk(a[2], a[3]), pk(a[4], a[5]), pk(a[6], a[7])) : make_uint4(0, 0, 0, 0);
            }
        }
    } else {
        if (tid == 0) {
            if (p.status) atomicCAS(p.status, 0u, static_cast<uint32_t>(SS_ERR_TIMEOUT));
            // what is in flight ends before the shared memory and the TMEM columns go
            mbar_wait_bounded(&bar->qk, 0, p.drain_ns);
            for (uint32_t q = 0; q < 2; ++q) mbar_wait_bounded(&bar->in, q, p.drain_ns);
            umma_commit(&bar->m2);
            for (uint32_t q = 0; q < 2; ++q) mbar_wait_bounded(&bar->m2, q, p.drain_ns);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------------------------ gradients of the gates
struct GateParams {
    Params p;
    __nv_bfloat16 *ddt, *dbeta;
    float* part;              // [items][2]: this item's share of dA and ddt_bias
};

// One block per (b, h); a warp per chunk, two tokens per lane, the suffix sum by shuffles.
__global__ void __launch_bounds__(256) ss_gdr_gate_kernel(const __grid_constant__ GateParams gt) {
    const Params& p = gt.p;
    const GdrParams& g = p.g;
    __shared__ double red[2][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t item = blockIdx.x, b = item / g.H, h = item % g.H;
    const int64_t len = gdr_len(g, static_cast<int>(b)), toks = p.nchunks * kC;
    const int64_t plane = static_cast<int64_t>(g.batch) * g.H * toks;
    const float A = g.A[h], bias = g.dt_bias ? g.dt_bias[h] : 0.0f;
    double sa = 0.0, sb = 0.0;
    for (int64_t c = warp; c < p.nchunks; c += 8) {
        const int64_t t = c * kC + 2 * lane;
        float r[2], ve[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const bool in = t + e < len;
            const float* d = p.dots + item * toks + t + e;
            r[e] = in ? d[0] - d[plane] : 0.0f;
            ve[e] = in ? d[2 * plane] : 0.0f;
        }
        float s = r[0] + r[1];   // suffix sums over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float v = __shfl_down_sync(0xffffffffu, s, o);
            if (lane + o < 32) s += v;
        }
        const float anchor = c * kC < len ? p.dots[3 * plane + item * p.nchunks + c] : 0.0f;
        const float dla[2] = {anchor + s, anchor + (s - r[0])};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (t + e >= g.L) continue;
            const int64_t o = (b * g.L + t + e) * g.H + h;
            float ddt = 0.0f, db = 0.0f;
            if (t + e < len) {
                const float pre = to_f32(static_cast<const __nv_bfloat16*>(g.dt)[o]) + bias;
                const float delta = g.softplus ? softplus_accurate(pre) : pre;
                // the decay of the first token meets a state of zero
                const float d = (t + e == 0 && !g.h_init) ? 0.0f : dla[e];
                ddt = d * A * (g.softplus ? 1.0f / (1.0f + expf(-pre)) : 1.0f);
                sa += static_cast<double>(d) * static_cast<double>(delta);
                sb += static_cast<double>(ddt);
                const float raw = to_f32(static_cast<const __nv_bfloat16*>(g.beta)[o]);
                if (g.sigmoid) {
                    db = ve[e] * (1.0f / (1.0f + expf(raw)));   // (dV·E / β) β (1 - β)
                } else {
                    db = ve[e] / (fabsf(raw) < 1e-20f ? 1e-20f : raw);
                }
            }
            gt.ddt[o] = __float2bfloat16_rn(ddt);
            gt.dbeta[o] = __float2bfloat16_rn(db);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sa += __shfl_xor_sync(0xffffffffu, sa, o);
        sb += __shfl_xor_sync(0xffffffffu, sb, o);
    }
    if (lane == 0) {
        red[0][warp] = sa;
        red[1][warp] = sb;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        double s = 0.0;
        for (int w = 0; w < 8; ++w) s += red[threadIdx.x][w];
        gt.part[2 * item + threadIdx.x] = static_cast<float>(s);
    }
}

// dA_h, ddt_bias_h: the batch entries' shares, in order.
__global__ void ss_gdr_head_kernel(const float* __restrict__ part, int batch, int H, float* dA, float* ddt_bias) {
    const int h = blockIdx.x * blockDim.x + threadIdx.x;
    if (h >= H) return;
    double a = 0.0, s = 0.0;
    for (int b = 0; b < batch; ++b) {
        const float* q = part + 2 * (static_cast<int64_t>(b) * H + h);
        a += q[0];
        s += q[1];
    }
    dA[h] = static_cast<float>(a);
    if (ddt_bias) ddt_bias[h] = static_cast<float>(s);
}

}  // namespace gdr
}  // namespace selscan
