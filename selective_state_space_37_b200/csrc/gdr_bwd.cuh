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
//   dQ̂ = [diag(e^G) dO S + M^P K̂]
//   dK̂ = [-diag(e^G) dV S + M^A K̂] + [diag(β e^{G_end - G}) E dS + M^Pᵀ Q̂ + M^Aᵀ K̂]
// For the gates: a token's decay stands in every path that crosses it, and log α's gradient is the sum of those paths:
//   dlog α_t = e^{G_end} <S, dS> + Σ_{i>=t} r_i + Σ_{j<t} c_j + Σ_{i>=t>j} W_ij,        dβ_j = dV_j·E_j / β_j
//   r_i = q̂_i·(diag(e^G) dO S)_i - k̂_i·(diag(e^G) dV S)_i           from the entering state to token i
//   c_j = k̂_j·(diag(β e^{G_end - G}) E dS)_j                       from token j to the leaving state
//   W_ij = M^P_ij (q̂_i·k̂_j) + M^A_ij (k̂_i·k̂_j)                   from token j to token i
// Every term holds the factor α_t, so that a head that forgets fast sums small terms.  A running sum of what ends less
// what begins at each token is the same number, but there the paths that do not cross a token (M^P's diagonal above
// all) come in and cancel only up to rounding: at Δ A = -29 what was left was ten times the gradient.
//
// Precision: what the adjoint's chain carries -- dS, dE, dV, dO's scaled rows -- and P enter as three bf16 terms, T as two
// (the first state's gradient is 2e-7 off on average; dS and dE as two and P as two: 1e-6 and 6e-7 more).  In the
// gradient kernel dV and M enter as two, E, S and dS as three, and <S, dS> is a sum of fp32 products: dA and ddt_bias are
// sums over all tokens of both signs, and come out in fp32 (all of them as two terms: 2e-6 to 3e-5 off).
#pragma once

#include "gdr_tc.cuh"

namespace selscan {
namespace gdr {

// ---------------------------------------------------------------------------------------- the adjoint's chain
// TMEM columns.  S: dS's terms, then its update; A: K dSᵀ, then dE's terms over it; R: Pᵀ dO in two halves (P's terms),
// then the third terms of scale e^G dO over the first half and dE's over the second; V: Tᵀ dE in two halves, then the
// terms of -e^G dV over the first and its third over the second, then the next dS's third terms over the first; O: the
// terms of scale e^G dO.
constexpr uint32_t kRevS = 0, kRevA = 128, kRevR = 192, kRevV = 320, kRevO = 448;
// Shared memory: two stages of [K 0][Q 0][K 1][Q 1][record]; dO (swizzled blocks) and P's third term; an image on its way
// out, dS in fp32 and then dVᵀ's terms.
constexpr uint32_t kRevStage = 4 * kTile + kRecBytes, kRevOffRec = 4 * kTile;
constexpr uint32_t kRevOffO = 2 * kRevStage, kRevOffP3 = kRevOffO + 2 * kTile, kRevOffImg = kRevOffP3 + kTile;
constexpr uint32_t kRevOffBar = kRevOffImg + 8 * kTile;
constexpr uint32_t kRevSmem = kRevOffBar + 256 + 1024;
static_assert(kRevStage % 1024 == 0 && kRevSmem <= 227 * 1024, "shared memory");

struct RevBars {
    uint64_t full[2], empty[2];      // K, Q and the record of a stage
    uint64_t o_full, o_free;         // dO and P's third term landed; read (state warps, behind their product)
    uint64_t img_full, img_free;     // dS's terms staged, then dV's (state warps); stored (1)
    uint64_t ks, e, ds;              // products done
    uint64_t s_ready[2], x_ready, w_ready;
    uint64_t fin;
    uint32_t tmem;
};
static_assert(sizeof(RevBars) <= 256, "barrier region");

// Grid: one CTA per (b, h).  dV of every chunk and the adjoints of the states between the chunks are kept, and leave by
// bulk copies from shared memory (16-byte stores from the threads' registers: 279 against 236 us).  8 x 2048 tokens, 12
// heads of 128 (96 CTAs of 32 chunks): 159 us, 5.0 us a chunk, tensor pipe 42 %: its hand-overs bound it, beside
// the 96 KB that a chunk keeps.
template <int DK>
__global__ void __launch_bounds__(kThreads, 1)
ss_gdr_rev_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tm_q,
                  const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_o) {
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
    if (tid == 0) {
        uint64_t* one[] = {bar->full, bar->full + 1, bar->empty, bar->empty + 1, &bar->o_full,
                           &bar->img_free, &bar->ks, &bar->e, &bar->ds, &bar->fin};
        for (uint64_t* x : one) mbar_init(x, 1);
        uint64_t* all[] = {bar->s_ready, bar->s_ready + 1, &bar->x_ready, &bar->w_ready, &bar->o_free,
                           &bar->img_full};
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
    int issued = 0, o_issued = 0;

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
                mbar_arrive_expect_tx(&bar->o_full, kC * p.dv * 2 + kTile);
                bulk_load(base + kRevOffP3, p.rec + (item * p.nchunks + c) * p.rec_bytes + kRecP3, kTile, &bar->o_full);
                for (int vb = 0; vb < p.dv / 64; ++vb)
                    tma_load_4d(base + kRevOffO + vb * kTile, &tm_o, 64 * vb, h, c * kC, b, &bar->o_full);
                o_issued = n + 1;
            }
        }
        __syncwarp();
    } else if (warp == kStoreWarp) {
        for (int n = 0; n < 2 * nchunk + 1; ++n) {   // dS of a state, dV of the chunk before it, and so on
            if (!wait_warp(&bar->img_full, n & 1)) break;
            if (lane == 0) {
                unsigned char* kp = p.keep + (item * (p.nchunks + 1) + nchunk - ((n + 1) >> 1)) * kKeepBytes;
                if (n & 1) {
                    bulk_store(kp + kKeepV, base + kRevOffImg, 4 * kTile);
                } else {
                    bulk_store(kp + kKeepD, base + kRevOffImg, 4 * KB * kTile);
                }
                tc::bulk_commit();
                tc::bulk_wait_read0();
            }
            arrive_warp(&bar->img_free);
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
                const uint32_t ot = base + kRevOffO;
                if (!wait1(&bar->o_full, par)) break;
                // the tiles' rows behind the end are zero by then; R's columns hold the third term of the last step's dO
                // until its update is done (the state warps take the update up meanwhile)
                if (n == 0 ? !wait1(&bar->s_ready[0], 0) : !wait1(&bar->ds, par ^ 1)) break;
                tc_fence_after();
                // R = dOᵀ P, P's terms side by side (their columns were read before dE's terms were handed over)
#pragma unroll
                for (int j = 0; j < kC / 16; ++j)
                    umma(tmem + kRevR, sdesc(ot + 2048u * j, lbo, 1024), sdesc(pr + kRecP + 2048u * j, kTile, 1024),
                         idesc(2 * kC, true, true), j > 0);
#pragma unroll
                for (int j = 0; j < kC / 16; ++j)
                    umma(tmem + kRevR, sdesc(ot + 2048u * j, lbo, 1024), sdesc(base + kRevOffP3 + 2048u * j, kTile, 1024),
                         idesc(kC, true, true), 1);
                constexpr int kStep = KH / 16;
                auto ks_steps = [&](int first) {   // small terms first, as in the forward
#pragma unroll
                    for (int w = 0; w < 3; ++w)
#pragma unroll
                        for (int ks = first; ks < DK / 16; ks += kStep)
                            umma_ts(tmem + kRevA, tmem + (w == 0 ? kRevV + 8 * ks : w == 1 ? kRevS + 16 * ks + 8 : kRevS + 16 * ks),
                                    sdesc(st + (ks >> 2) * 2 * kTile + (ks & 3) * 32, 16, 1024), idesc(kC, false), first + w + ks > 0);
                };
                if (!wait1(&bar->s_ready[0], par)) break;
                tc_fence_after();
                ks_steps(0);
                if (!wait1(&bar->s_ready[1], par)) break;
                tc_fence_after();
                if (kStep == 2) ks_steps(1);
                if (!(p.test_drop && blockIdx.x == 0 && n == 0)) umma_commit(&bar->ks);
                if (!wait1(&bar->x_ready, par)) break;
                tc_fence_after();
                // Vᵀ = dEᵀ T
#pragma unroll
                for (int w = 0; w < 3; ++w)
#pragma unroll
                    for (int j = 0; j < kC / 16; ++j)
                        umma_ts(tmem + kRevV, tmem + (w == 0 ? kRevR + kC : w == 1 ? kRevA + 8 : kRevA) + 16 * j,
                                sdesc(pr + kRecT + 2048u * j, kTile, 1024), idesc(2 * kC, true), w + j > 0);
                umma_commit(&bar->e);
                // dS's update: (scale e^G dO)ᵀ Q, then (-e^G dV)ᵀ K, over the columns of dS's terms
#pragma unroll
                for (int w = 0; w < 3; ++w)
#pragma unroll
                    for (int j = 0; j < kC / 16; ++j)
                        umma_ts(tmem + kRevS, tmem + (w == 0 ? kRevR : w == 1 ? kRevO + 8 : kRevO) + 16 * j,
                                sdesc(st + kTile + 2048u * j, 2 * kTile, 1024), idesc(DK, true), w + j > 0);
                if (!wait1(&bar->w_ready, par)) break;
                tc_fence_after();
#pragma unroll
                for (int w = 0; w < 3; ++w)
#pragma unroll
                    for (int j = 0; j < kC / 16; ++j)
                        umma_ts(tmem + kRevS, tmem + (w == 0 ? kRevV + kC : w == 1 ? kRevV + 8 : kRevV) + 16 * j,
                                sdesc(st + 2048u * j, 2 * kTile, 1024), idesc(DK, true), 1);
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
        for (int k = 0; k < KH; k += 16)
            store_terms3(tl + kRevS + part * KH + k, tl + kRevV + (part * KH + k) / 2, S + k / 2);
        tmem_wait_st();
        tc_fence_before();
        // a bf16 value of token kTok · part + e, row v, of a swizzled [64][d_v] tile
        auto val = [&](uint32_t off, int e) {
            const uint32_t t = kTok * part + e;
            const uint32_t a = chunk_addr(off + static_cast<uint32_t>(v >> 6) * kTile, t, (v & 63) >> 3) + 2 * (v & 7);
            return row_in ? __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(gbase + a)) : 0.0f;
        };
        auto keep_state = [&](int n) {   // dS, store 2 n
            if (n > 0 && !wait_warp(&bar->img_free, 1)) return false;
#pragma unroll
            for (int k = 0; k < KH; k += 16)
                stage_f32(base + kRevOffImg, v, part * KH + k, S + k / 2);
            fence_proxy_async_smem();
            arrive_warp(&bar->img_full);
            return true;
        };
        bool ok = true;
        for (int n = 0; n < nchunk; ++n) {
            const int c = nchunk - 1 - n, s = n & 1;
            const uint32_t par = n & 1, st = base + s * kRevStage;
            const Scal& sc = *reinterpret_cast<const Scal*>(gbase + s * kRevStage + kRevOffRec + kRecScal);
            if (n == 0) {
                if (ragged) {   // rows behind the end, whatever they hold, become zero rows
                    ok = wait_warp(&bar->full[0], 0) && wait_warp(&bar->o_full, 0);
                    if (!ok) break;
                    const int n0 = static_cast<int>(len - static_cast<int64_t>(c) * kC);
                    for (int i = n0 * 8 + tid; i < kC * 8; i += 32 * kStateWarps) {
                        for (int kb = 0; kb < 2 * KB; ++kb) sts128(st + kb * kTile + 16 * i, make_uint4(0, 0, 0, 0));
                        for (int vb = 0; vb < p.dv / 64; ++vb)
                            sts128(base + kRevOffO + vb * kTile + 16 * i, make_uint4(0, 0, 0, 0));
                    }
                    fence_proxy_async_smem();
                }
                arrive_warp(&bar->s_ready[0]);
                arrive_warp(&bar->s_ready[1]);
                // (the zero rows of other warps' share are visible behind the product's own barrier)
            }
            ok = keep_state(n);
            if (!ok) break;
            ok = wait_warp(&bar->full[s], (n >> 1) & 1) && wait_warp(&bar->o_full, par);
            const uint32_t ot = kRevOffO;
            if (!ok) break;
            f32x2 x[8];
            uint32_t third[8];           // of scale e^G dO, until R's columns are free
            auto scaled_do = [&]() {
                f32x2 q[8];
                uint32_t hi[8], lw[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) q[e] = pk2(val(ot, 2 * e), val(ot, 2 * e + 1));
                scale16(q, sc.qe + kTok * part);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    hi[e] = pk(q[e].x, q[e].y);
                    split2(fma2(pk2(lo_f(hi[e]), hi_f(hi[e])), pk2(-1.0f, -1.0f), q[e]), lw[e], third[e]);
                }
                tmem_st8(tl + kRevO + kTok * part, hi);
                tmem_st8(tl + kRevO + kTok * part + 8, lw);
            };
            // (in a ragged chunk once every warp's zero rows are written)
            if (!(n == 0 && ragged)) scaled_do();
            ok = wait_warp(&bar->ks, par);
            if (!ok) break;
            tc_fence_after();
            if (n == 0 && ragged) scaled_do();
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
            tmem_st8(tl + kRevR + kTok * part, third);
            store_terms3(tl + kRevA + kTok * part, tl + kRevR + kC + kTok * part, x);
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
                store_terms3(tl + kRevV + kTok * part, tl + kRevV + kC + kTok * part, w);
            }
            const float end = sc.end[0];
            tmem_wait_st();
            tc_fence_before();
            arrive_warp(&bar->w_ready);
            ok = wait_warp(&bar->img_free, 0);   // dV's terms, store 2 n + 1, while dS is multiplied
            if (!ok) break;
            stage_terms<false>(base + kRevOffImg, v, kTok * part, x);
            fence_proxy_async_smem();
            arrive_warp(&bar->img_full);
            ok = wait_warp(&bar->ds, par);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < KH; k += 16) {
                tmem_ld16(tl + kRevS + part * KH + k, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) S[k / 2 + e] = fma2(pk2(end, end), S[k / 2 + e], x[e]);
                store_terms3(tl + kRevS + part * KH + k, tl + kRevV + (part * KH + k) / 2, S + k / 2);
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
        if (ok) ok = keep_state(nchunk);
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
// fp32 registers.  Per value head (M = 128 lanes, two 64-row operands on top of one another; every operand but dO, K
// and Q in terms, S and dS made so here):
//   D2 [dO; dV] Eᵀ             -> columns 384 .. 447 (K: d_v), read into M^P, M^A (two bf16 terms, shared memory)
//   D0 [Q; K] Kᵀ               ->         448 .. 511 (K: d_k), for W
//   D1 [dO; dV] S              ->           0 .. 127 (K: d_v)
//   D4 [M^P; M^A] K            ->         256 .. 383 (K: 64 tokens)
//   D5 [M^P; M^A]ᵀ [Q; K]      ->         384 .. 511 (K: 128; lanes 64.. repeat the rows 0..63)
//   D3 E dS                    ->         128 .. 255 (K: d_v; likewise)
//   dq~ = qe D1 + D4 (lanes 0..63),   dk~ = ek D1 + D4 (lanes 64..127) + wk D3 + D5 (lanes 0..63)
// (ek carries the minus of -e^G), and of each token r, c and the sum of W that crosses it: a row's prefix sums over its
// columns, added over the rows by shuffles.  dV comes from the chain transposed and is turned in shared memory; dO has
// no lo terms, so the products with dV's write the lanes from 64 on alone; S and dS pass through one buffer, in fp32 and
// then as terms.  Bound by the latency of its stages, one block per SM (219 KB): 8 x 2048 tokens, 12 heads of 128 (a
// block per head and chunk) 450 us, 22 us a block, 2.1 TB/s, tensor pipe 22 %.  (S, dS and E as two terms, made by the
// chains: 342 us, and dA 5 times further off; 512 threads then 351 against 346 us.)
constexpr int kGradThreads = 256;
constexpr uint32_t kGK = 0;                       // [Q 0][K 0][Q 1][K 1]
constexpr uint32_t kG1 = 4 * kTile;               // [dO 0][dV hi 0][dO 1][dV hi 1]; then dS's third terms
constexpr uint32_t kG2 = 8 * kTile;               // [dV lo 0][dV lo 1]; then [M^P lo][M^A lo]
constexpr uint32_t kGE = 10 * kTile;              // Eᵀ hi, lo: 128 rows each
constexpr uint32_t kGS = 14 * kTile;              // S, then dS: fp32 (four 32-wide blocks of 128 rows), then the terms in
                                                  // place, [hi 0][lo 0][hi 1][lo 1]; then dk~'s other bracket, fp32 [64][132]
constexpr uint32_t kGM = 22 * kTile;              // dVᵀ hi, lo (128 rows each); E's third terms over lo; S's third terms;
                                                  // then [M^P hi][M^A hi], and E's third terms again
constexpr uint32_t kGScal = 26 * kTile;           // Scal, Local (one copy from the record)
constexpr uint32_t kGRed = kGScal + 1024 + sizeof(Local);   // row products of the two halves, [3][2][64]
constexpr uint32_t kGCross = kGRed + 3 * 2 * kC * 4;        // W's sums across each token, of [P, A][diagonal, left blocks]
constexpr uint32_t kGBar = kGCross + 4 * kC * 4;
constexpr uint32_t kGradSmem = kGBar + 128 + 1024;
constexpr int kGPitch = 132;
static_assert(kGradSmem <= 227 * 1024, "shared memory");

struct GradBars {
    uint64_t qk, in, e3, s, d, m2, m1, m5, m3, fin;
    uint32_t tmem;
};

struct GradParams {
    Params p;
    __nv_bfloat16 *dq, *dk, *dv;
};

// Four 8 x 8 bf16 blocks, each lane giving a row's address: loaded transposed, and stored.
__device__ __forceinline__ void turn8x4(uint32_t src, uint32_t dst) {
    uint32_t r0, r1, r2, r3;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(src)
                 : "memory");
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(r0), "r"(r1), "r"(r2),
                 "r"(r3)
                 : "memory");
}

// D[tmem] += A · B in the lanes from 64 on; the others keep what they hold.
__device__ __forceinline__ void umma_upper(uint32_t d, uint64_t a, uint64_t b, uint32_t id) {
    const uint32_t off = 0xffffffffu, on = 0u;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, 1, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%4, %4, %5, %5}, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(off), "r"(on)
        : "memory");
}

// 64 keys of a row of an fp32 image (two 32-wide blocks), and their terms: hi in the first block's place, lo in the
// second's -- a thread rewrites what it alone has read -- and the third in an image of its own.
__device__ __forceinline__ void read_row(uint32_t img, int r, f32x2 (&s)[32]) {
#pragma unroll
    for (int q = 0; q < 16; ++q) {
        const uint4 w = lds128(chunk_addr(img + (q >> 3) * 2 * kTile, r, q & 7));
        s[2 * q] = pk2(__uint_as_float(w.x), __uint_as_float(w.y));
        s[2 * q + 1] = pk2(__uint_as_float(w.z), __uint_as_float(w.w));
    }
}
__device__ __forceinline__ void write_terms(uint32_t img, uint32_t third, int r, const f32x2 (&s)[32]) {
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        uint32_t a[4], b[4], c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split3(s[4 * w + e], a[e], b[e], c[e]);
        sts128(chunk_addr(img, r, w), make_uint4(a[0], a[1], a[2], a[3]));
        sts128(chunk_addr(img + 2 * kTile, r, w), make_uint4(b[0], b[1], b[2], b[3]));
        sts128(chunk_addr(third, r, w), make_uint4(c[0], c[1], c[2], c[3]));
    }
}

template <int DK>
__global__ void __launch_bounds__(kGradThreads, 1)
ss_gdr_grad_kernel(const __grid_constant__ GradParams gp, const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_o) {
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
        uint64_t* all[] = {&bar->qk, &bar->in, &bar->e3, &bar->s, &bar->d, &bar->m2, &bar->m1, &bar->m5, &bar->m3, &bar->fin};
        for (uint64_t* x : all) mbar_init(x, 1);
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
    const int t = static_cast<int>(t0), vb = p.dv / 64, vs = p.dv / 16;
    // thread: lane row r of TMEM (token i; q's bracket below 64, k's first from 64 on), columns CN · half ..
    const int r = (warp & 3) * 32 + lane, half = warp >> 2, i = r & 63, rb = (r >> 5) & 1;
    const bool is_k = r >= 64;
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int64_t plane = static_cast<int64_t>(g.batch) * g.H * p.nchunks * kC;
    auto load_in = [&](int64_t item, int h) {   // dVᵀ, E, dO and the factors
        const unsigned char* kp = p.keep + (item * (p.nchunks + 1) + c) * kKeepBytes;
        mbar_arrive_expect_tx(&bar->in, 8 * kTile + vb * kTile + 1024 + sizeof(Local));
        bulk_load(base + kGM, kp + kKeepV, 4 * kTile, &bar->in);
        bulk_load(base + kGE, kp + kKeepE, 4 * kTile, &bar->in);
        for (int w = 0; w < vb; ++w) tma_load_4d(base + kG1 + 2 * w * kTile, &tm_o, 64 * w, h, t, b, &bar->in);
        bulk_load(base + kGScal, p.rec + (item * p.nchunks + c) * p.rec_bytes + kRecScal, 1024 + sizeof(Local), &bar->in);
    };
    auto load_e3 = [&](int64_t item, uint64_t* f, uint32_t with) {   // and `with` bytes that the caller loads
        mbar_arrive_expect_tx(f, 2 * kTile + with);
        bulk_load(base + kGM + 2 * kTile, p.keep + (item * (p.nchunks + 1) + c) * kKeepBytes + kKeepE3, 2 * kTile, f);
    };
    if (tid == 0) {
        mbar_arrive_expect_tx(&bar->qk, 2 * KB * kTile);
        for (int kb = 0; kb < KB; ++kb) {
            tma_load_4d(base + kGK + (2 * kb) * kTile, &tm_q, 64 * kb, hk, t, b, &bar->qk);
            tma_load_4d(base + kGK + (2 * kb + 1) * kTile, &tm_k, 64 * kb, hk, t, b, &bar->qk);
        }
    }
    // Σ over this thread's columns of its row of Q or K (own) times d
    auto row_product = [&](uint32_t own, const float (&d)[CN]) {
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int w = 0; w < CN / 8; ++w) {
            const int col = CN * half + 8 * w;
            const uint4 q = lds128(chunk_addr(own + (col >> 6) * 2 * kTile, i, (col & 63) >> 3));
            const uint32_t a[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s0 = fmaf(lo_f(a[e]), d[8 * w + 2 * e], s0);
                s1 = fmaf(hi_f(a[e]), d[8 * w + 2 * e + 1], s1);
            }
        }
        return s0 + s1;
    };
    float acc[CN];   // dq~ or dk~ of this thread's row and columns
#pragma unroll
    for (int e = 0; e < CN; ++e) acc[e] = 0.0f;
    float* const xch = reinterpret_cast<float*>(gbase + kGS);
    float* const red = reinterpret_cast<float*>(gbase + kGRed);
    float* const cross = reinterpret_cast<float*>(gbase + kGCross);
    const uint32_t own = base + kGK + (is_k ? kTile : 0);   // this row of K or Q
    bool bad = false;
    int stage = 0, e3s = 0;   // what thread 0 has in flight, for the wind-down
    for (int j = 0; j < rep; ++j) {
        const int h = hk * rep + j;
        const int64_t item = static_cast<int64_t>(b) * g.H + h;
        const uint32_t par = j & 1;
        auto wait_all = [&](uint64_t* x, uint32_t ph) {   // every thread; a uniform outcome
            const bool got = mbar_wait_bounded(x, ph, p.wait_ns);
            bad = __syncthreads_or(!got) != 0;
            return !bad;
        };
        if (tid == 0) {
            load_in(item, h);
            mbar_arrive_expect_tx(&bar->s, 4 * KB * kTile);
            bulk_load(base + kGS, p.keep + (item * (p.nchunks + 1) + c) * kKeepBytes + kKeepS, 4 * KB * kTile, &bar->s);
            stage = 4 * j + 2;
        }
        if (j == 0 && !wait_all(&bar->qk, 0)) break;
        if (!wait_all(&bar->in, par)) break;
        // dV's rows (its terms turned), and zero rows behind the sequence's end
        for (int w = warp; w < 4 * vb * 8; w += 8) {   // four 8-row groups of v by 8 tokens, hi then lo
            const int term = w / (2 * vb * 8), x = w % (2 * vb * 8), vg = (x >> 3) * 4, tc8 = x & 7;
            const int m = vg + (lane >> 3), l7 = lane & 7;
            turn8x4(chunk_addr(base + kGM + term * 2 * kTile, 8 * m + l7, tc8),
                    chunk_addr(base + (term ? kG2 + (m >> 3) * kTile : kG1 + (2 * (m >> 3) + 1) * kTile), 8 * tc8 + l7, m & 7));
        }
        if (valid < kC) {   // K, Q (once) and dO (dV has them)
            for (int w = valid * 8 + tid; w < kC * 8; w += kGradThreads) {
                for (int kb = 0; kb < 2 * KB && j == 0; ++kb) sts128(base + kGK + kb * kTile + 16 * w, make_uint4(0, 0, 0, 0));
                for (int x = 0; x < vb; ++x) sts128(base + kG1 + 2 * x * kTile + 16 * w, make_uint4(0, 0, 0, 0));
            }
        }
        fence_proxy_async_smem();
        __syncthreads();
        // 16 columns of [dO; dV hi], and of dV lo as the rows 64.. of an operand (whose others are not written out)
        auto a_hi = [&](int ks) { return sdesc(base + kG1 + (ks >> 2) * 2 * kTile + (ks & 3) * 32u, 16, 1024); };
        auto a_lo = [&](int ks) { return sdesc(base + kG2 - kTile + (ks >> 2) * kTile + (ks & 3) * 32u, 16, 1024); };
        if (tid == 0) {
            tc_fence_after();   // (behind the last head's reads of these columns)
            load_e3(item, &bar->e3, 0);
            e3s = j + 1;
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks) {
                const uint32_t off = base + kGK + (ks >> 2) * 2 * kTile + (ks & 3) * 32u;
                umma(tmem + 448, sdesc(off, 16, 1024), sdesc(off + kTile, 16, 1024), idesc(kC, false), ks > 0);
            }
            // (the accumulator is cut off, not rounded, after every product: here and below the small terms come first)
            for (int ks = 0; ks < vs; ++ks)
                umma(tmem + 384, a_hi(ks), sdesc(base + kGE + 2 * kTile + 2048u * ks, 0, 1024), idesc(kC, true), ks > 0);
            for (int ks = 0; ks < vs; ++ks) {
                umma_upper(tmem + 384, a_lo(ks), sdesc(base + kGE + 2 * kTile + 2048u * ks, 0, 1024), idesc(kC, true));
                umma_upper(tmem + 384, a_lo(ks), sdesc(base + kGE + 2048u * ks, 0, 1024), idesc(kC, true));
            }
        }
        // v's gradient: dV's hi terms are its values rounded to bf16
        for (int w = tid; w < rows * vb * 8; w += kGradThreads) {
            const int row = w / (vb * 8), q = w % (vb * 8);
            *reinterpret_cast<uint4*>(gp.dv + ((static_cast<int64_t>(b) * g.L + t0 + row) * g.H + h) * p.dv + 8 * q) =
                lds128(chunk_addr(base + kG1 + (2 * (q >> 3) + 1) * kTile, row, q & 7));
        }
        // <S, dS> of the entering state and the leaving one's adjoint: dS from memory, quad by quad in the order of S's
        // image, fetched ahead in two batches
        float4 ds[4 * KB];
        auto fetch_ds = [&](int w0) {
            const unsigned char* kp = p.keep + (item * (p.nchunks + 1) + c + 1) * kKeepBytes + kKeepD;
#pragma unroll
            for (int w = 0; w < 4 * KB; ++w)
                ds[w] = __ldg(reinterpret_cast<const float4*>(kp + 16u * (tid + kGradThreads * (w0 + w))));
        };
        fetch_ds(0);
        if (tid == 0 && mbar_wait_bounded(&bar->e3, par, p.wait_ns)) {   // (else the next wait runs out)
            for (int ks = 0; ks < vs; ++ks)
                umma(tmem + 384, a_hi(ks), sdesc(base + kGM + 2 * kTile + 2048u * ks, 0, 1024), idesc(kC, true), 1);
            for (int ks = 0; ks < vs; ++ks)
                umma(tmem + 384, a_hi(ks), sdesc(base + kGE + 2048u * ks, 0, 1024), idesc(kC, true), 1);
            umma_commit(&bar->m2);
        }
        __syncwarp();
        if (!wait_all(&bar->m2, par)) break;
        tc_fence_after();
        float v[32];   // M^P (rows 0..63), M^A (64..127): one 32-column block per thread
        {
            const bool diag = half == rb;
            if (diag || half < rb) {
                tmem_ld32(tl + 384 + 32 * half, v);
                const float row = is_k ? -lo.rk[i] : lo.rq[i];
                if (diag) {
                    if (is_k) p.dots[3 * plane + (item * p.nchunks + c) * kC + i] = pick32(v, i & 31);   // dV·E
                    decay_diagonal(v, lo, 32 * rb, lo.gh[i], lo.gl[i], row, i & 31, !is_k);
                } else {
                    decay_left(v, lo, lo.gh[i], lo.gl[i], row);
                }
                // W's sums across the tokens of these columns: each row's prefix sums, in the diagonal block up to its
                // own token, added over the warp's rows; lane t ends with column t
                float u[32];
                tmem_ld32(tl + 448 + 32 * half, u);
                float s = 0.0f;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float w = v[e] * u[e];
                    u[e] = diag && e > lane ? 0.0f : s;
                    s += w;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const bool up = lane & o;
#pragma unroll
                    for (int e = 0; e < o; ++e) {
                        const float give = up ? u[e] : u[e + o], keep = up ? u[e + o] : u[e];
                        u[e] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                    }
                }
                float* x = cross + (2 * is_k + (diag ? 0 : 1)) * kC;
                x[32 * half + lane] = u[0];
                if (!diag) {   // whole rows of the left block, across the tokens 32 .. their own
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const float w = __shfl_down_sync(0xffffffffu, s, o);
                        if (lane + o < 32) s += w;
                    }
                    x[32 + lane] = s;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = 0.0f;
            }
        }
        if (!wait_all(&bar->s, par)) break;
        {
            float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
            for (int batch = 0; batch < 2; ++batch) {
#pragma unroll
                for (int w = 0; w < 4 * KB; ++w) {
                    const uint32_t o = 16u * (tid + kGradThreads * (4 * KB * batch + w));
                    const uint4 x = lds128(base + kGS + o);
                    if (static_cast<int>((o >> 7) & 127) < p.dv) {
                        s0 = fmaf(__uint_as_float(x.x), ds[w].x, fmaf(__uint_as_float(x.y), ds[w].y, s0));
                        s1 = fmaf(__uint_as_float(x.z), ds[w].z, fmaf(__uint_as_float(x.w), ds[w].w, s1));
                    }
                }
                if (batch == 0) fetch_ds(4 * KB);
            }
            s0 += s1;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, o);
            if (lane == 0) red[warp] = s0;
        }
        // S's terms in its place; the third over dVᵀ and E's third, which D2 has read
        const int half64 = tid >> 7;   // 64 keys of row tid & 127
        const uint32_t sblk = base + kGS + half64 * 4 * kTile;
        {
            f32x2 s[32];
            if (half64 < KB) read_row(sblk, tid & 127, s);
            __syncthreads();   // (the products above read other rows)
            if (half64 < KB) write_terms(sblk, base + kGM + half64 * 2 * kTile, tid & 127, s);
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after();
            for (int ks = 0; ks < vs; ++ks) {
                umma(tmem, a_hi(ks), sdesc(base + kGM + 2048u * ks, 2 * kTile, 1024), idesc(DK, true), ks > 0);
                umma(tmem, a_hi(ks), sdesc(base + kGS + 2 * kTile + 2048u * ks, 4 * kTile, 1024), idesc(DK, true), 1);
                umma_upper(tmem, a_lo(ks), sdesc(base + kGS + 2 * kTile + 2048u * ks, 4 * kTile, 1024), idesc(DK, true));
                umma_upper(tmem, a_lo(ks), sdesc(base + kGS + 2048u * ks, 4 * kTile, 1024), idesc(DK, true));
            }
            for (int ks = 0; ks < vs; ++ks)
                umma(tmem, a_hi(ks), sdesc(base + kGS + 2048u * ks, 4 * kTile, 1024), idesc(DK, true), 1);
            umma_commit(&bar->m1);
        }
        if (!wait_all(&bar->m1, par)) break;   // S and dV's lo terms are read
        if (tid == 0) {
            float s = 0.0f;
            for (int w = 0; w < 8; ++w) s += red[w];
            p.dots[4 * plane + item * (p.nchunks + 1) + c] = s * sc.end[0];
        }
        if (tid == 0) {
            load_e3(item, &bar->d, 4 * KB * kTile);   // and the leaving state's dS
            bulk_load(base + kGS, p.keep + (item * (p.nchunks + 1) + c + 1) * kKeepBytes + kKeepD, 4 * KB * kTile, &bar->d);
            stage = 4 * j + 3;
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t hw[4], lw[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split2(pk2(v[8 * w + 2 * e], v[8 * w + 2 * e + 1]), hw[e], lw[e]);
            const uint32_t o = chunk_addr(is_k ? kTile : 0, i, 4 * half + w);
            sts128(base + kGM + o, make_uint4(hw[0], hw[1], hw[2], hw[3]));
            sts128(base + kG2 + o, make_uint4(lw[0], lw[1], lw[2], lw[3]));
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after();
#pragma unroll
            for (int w = 0; w < 2; ++w) {   // M's hi terms, then its lo terms
                const uint32_t mt = base + (w ? kG2 : kGM);
#pragma unroll
                for (int ks = 0; ks < kC / 16; ++ks)
                    umma(tmem + 256, sdesc(mt + 32u * ks, 16, 1024), sdesc(base + kGK + kTile + 2048u * ks, 2 * kTile, 1024),
                         idesc(DK, true), w + ks > 0);
#pragma unroll
                for (int ks = 0; ks < 2 * kC / 16; ++ks)   // rows r of [M^P; M^A] with rows r of [Q; K]
                    umma(tmem + 384, sdesc(mt + 2048u * ks, 0, 1024), sdesc(base + kGK + 2048u * ks, 2 * kTile, 1024),
                         idesc(DK, true, true), w + ks > 0);
            }
            umma_commit(&bar->m5);
        }
        if (!wait_all(&bar->d, par)) break;
        if (half64 < KB) {   // dS's terms, as S's
            f32x2 s[32];
            read_row(sblk, tid & 127, s);
            write_terms(sblk, base + kG1 + half64 * 2 * kTile, tid & 127, s);
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            for (int ks = 0; ks < vs; ++ks) {   // every pair of terms down to 2^-24
                const uint64_t dh = sdesc(base + kGS + 2048u * ks, 4 * kTile, 1024);
                const uint64_t dl = sdesc(base + kGS + 2 * kTile + 2048u * ks, 4 * kTile, 1024);
                const uint64_t e = sdesc(base + kGE + 2048u * ks, 0, 1024), el = sdesc(base + kGE + 2 * kTile + 2048u * ks, 0, 1024);
                umma(tmem + 128, e, sdesc(base + kG1 + 2048u * ks, 2 * kTile, 1024), idesc(DK, true, true), ks > 0);
                umma(tmem + 128, el, dl, idesc(DK, true, true), 1);
                umma(tmem + 128, sdesc(base + kGM + 2 * kTile + 2048u * ks, 0, 1024), dh, idesc(DK, true, true), 1);
                umma(tmem + 128, e, dl, idesc(DK, true, true), 1);
                umma(tmem + 128, el, dh, idesc(DK, true, true), 1);
            }
            for (int ks = 0; ks < vs; ++ks)
                umma(tmem + 128, sdesc(base + kGE + 2048u * ks, 0, 1024), sdesc(base + kGS + 2048u * ks, 4 * kTile, 1024),
                     idesc(DK, true, true), 1);
            umma_commit(&bar->m3);
        }
        if (!wait_all(&bar->m5, par)) break;
        tc_fence_after();
        const int64_t tok = (item * p.nchunks + c) * kC + i;
        float d[CN];
        {
            const float f1 = is_k ? sc.ek[i] : sc.qe[i];
#pragma unroll
            for (int e = 0; e < CN; e += 32) {
                float w[32];
                tmem_ld32(tl + CN * half + e, v);
                tmem_ld32(tl + 256 + CN * half + e, w);
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                    d[e + x] = f1 * v[x];
                    acc[e + x] += d[e + x] + w[x];
                }
            }
            red[(is_k ? 2 : 0) * kC + half * kC + i] = row_product(own, d);
        }
        if (!wait_all(&bar->m3, par)) break;   // (dS is read: its buffer takes dk~'s other bracket)
        tc_fence_after();
        if (!is_k) {
            const float f3 = sc.wk[i];
#pragma unroll
            for (int e = 0; e < CN; e += 32) {
                float w[32];
                tmem_ld32(tl + 128 + CN * half + e, v);
                tmem_ld32(tl + 384 + CN * half + e, w);
#pragma unroll
                for (int x = 0; x < 32; ++x) d[e + x] = f3 * v[x];
#pragma unroll
                for (int x = 0; x < 32; x += 4)
                    *reinterpret_cast<float4*>(xch + i * kGPitch + CN * half + e + x) =
                        make_float4(d[e + x] + w[x], d[e + x + 1] + w[x + 1], d[e + x + 2] + w[x + 2], d[e + x + 3] + w[x + 3]);
            }
            red[4 * kC + half * kC + i] = row_product(base + kGK + kTile, d);
        }
        tc_fence_before();
        __syncthreads();
        if (is_k) {
#pragma unroll
            for (int x = 0; x < CN; x += 4) {
                const float4 q = quad(xch + i * kGPitch + CN * half + x);
                acc[x] += q.x;
                acc[x + 1] += q.y;
                acc[x + 2] += q.z;
                acc[x + 3] += q.w;
            }
        } else if (half == 0) {   // r, c, W's sum across the token
            p.dots[tok] = (red[i] + red[kC + i]) + (red[2 * kC + i] + red[3 * kC + i]);
            p.dots[plane + tok] = red[4 * kC + i] + red[5 * kC + i];
            p.dots[2 * plane + tok] = (cross[i] + cross[kC + i]) + (cross[2 * kC + i] + cross[3 * kC + i]);
        }
        fence_proxy_async_smem();   // the exchange was written and read before the next head's loads land there
        __syncthreads();
    }
    if (!bad) {
        // the unit length's own derivative: d = d~ - x (x·d~) / |x|²; the row's two halves meet in shared memory
        float x2 = 0.0f, xd = 0.0f;
        if (g.l2norm) {
            xd = row_product(own, acc);
#pragma unroll
            for (int w = 0; w < CN / 8; ++w) {
                const int col = CN * half + 8 * w;
                const uint4 q = lds128(chunk_addr(own + (col >> 6) * 2 * kTile, i, (col & 63) >> 3));
                const uint32_t a[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) x2 = fmaf(lo_f(a[e]), lo_f(a[e]), fmaf(hi_f(a[e]), hi_f(a[e]), x2));
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
    } else if (tid == 0) {
        if (p.status) atomicCAS(p.status, 0u, static_cast<uint32_t>(SS_ERR_TIMEOUT));
        // what is in flight ends before the shared memory and the TMEM columns go
        const uint32_t ph = static_cast<uint32_t>((stage - 1) >> 2) & 1;
        mbar_wait_bounded(&bar->qk, 0, p.drain_ns);
        mbar_wait_bounded(&bar->in, ph, p.drain_ns);
        if (e3s) mbar_wait_bounded(&bar->e3, (e3s - 1) & 1, p.drain_ns);
        if ((stage & 3) >= 2) mbar_wait_bounded(&bar->s, ph, p.drain_ns);
        if ((stage & 3) == 3) mbar_wait_bounded(&bar->d, ph, p.drain_ns);
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

// ------------------------------------------------------------------------------------ gradients of the gates
struct GateParams {
    Params p;
    __nv_bfloat16 *ddt, *dbeta;
    float* part;              // [items][2]: this item's share of dA and ddt_bias
};

// One block per (b, h); a warp per chunk, two tokens per lane, the sums over tokens by shuffles.  96 items of 2048 tokens:
// 16 us.
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
        float r[2], cb[2], w[2], ve[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const bool in = t + e < len;
            const float* d = p.dots + item * toks + t + e;
            r[e] = in ? d[0] : 0.0f;
            cb[e] = in ? d[plane] : 0.0f;
            w[e] = in ? d[2 * plane] : 0.0f;
            ve[e] = in ? d[3 * plane] : 0.0f;
        }
        float ends = r[0] + r[1], begun = cb[0] + cb[1];   // sums from this lane on, and up to it
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_down_sync(0xffffffffu, ends, o), y = __shfl_up_sync(0xffffffffu, begun, o);
            if (lane + o < 32) ends += x;
            if (lane >= o) begun += y;
        }
        float after = __shfl_down_sync(0xffffffffu, ends, 1), before = __shfl_up_sync(0xffffffffu, begun, 1);
        if (lane == 31) after = 0.0f;
        if (lane == 0) before = 0.0f;
        const float whole = c * kC < len ? p.dots[4 * plane + item * (p.nchunks + 1) + c] : 0.0f;
        float dla[2] = {whole + (r[0] + (r[1] + after)) + before + w[0], whole + (r[1] + after) + (before + cb[0]) + w[1]};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (t + e >= g.L) continue;
            const int64_t o = (b * g.L + t + e) * g.H + h;
            float ddt = 0.0f, db = 0.0f;
            if (t + e < len) {
                const float pre = to_f32(static_cast<const __nv_bfloat16*>(g.dt)[o]) + bias;
                const float delta = g.softplus ? softplus_accurate(pre) : pre;
                // where α is zero in fp32 so is its gradient, which an infinite Δ would make NaN below
                if (delta * A < -104.0f) dla[e] = 0.0f;
                ddt = dla[e] * A * (g.softplus ? 1.0f / (1.0f + expf(-pre)) : 1.0f);
                sa += static_cast<double>(dla[e]) * static_cast<double>(delta);
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
