// gdr_tc.cuh -- the gated delta rule chunk by chunk on the fifth-generation tensor cores (sm_100a).
//
// Per (b, value head h), over a chunk of C = 64 tokens with G_i = Σ_{r<=i} Δ_r A (so α_i ... α_{j+1} = e^{G_i - G_j}),
// S the state that enters it (d_v x d_k), K, Q, V, E the chunk's rows:
//   e_i = v_i - e^{G_i} S k̂_i - Σ_{j<i} e^{G_i - G_j} (k̂_i·k̂_j) β_j e_j
// is one triangular system for all 64 corrections, so with A'_ij = e^{G_i - G_j} (k̂_i·k̂_j) β_j (j < i):
//   E = T (V - diag(e^G) K̂ Sᵀ),  T = (I + A')^-1
//   Y = diag(e^G) Q̂ Sᵀ + P diag(β) E,       P_ij = e^{G_i - G_j} q̂_i·k̂_j (j <= i)
//   S <- e^{G_end} S + (diag(β e^{G_end - G}) E)ᵀ K̂
// Every exponent is a difference G_i - G_j with j <= i, so nothing overflows; the differences are taken of 48-bit
// values (pairs of floats of a 64-bit prefix sum), so a long decay keeps its near differences.  T does not depend
// on S: it is computed chunks ahead, and what is left in the chain from chunk to chunk is three products and two
// element-wise steps.
//
// The products run transposed: the 128 TMEM lanes are the rows v of the state, and the columns are tokens or keys.
//   KS  [v, i] = S Kᵀ        A: S (TMEM),  B: K tile, K-major
//   E   [v, i] = X Tᵀ        A: X = (V - diag KS)ᵀ (TMEM),  B: T tile, K-major; T's zero blocks are left out
//   dS  [v, k] = W K         A: W = scaled E (TMEM),  B: K tile, MN-major
//   QS  [v, i] = S Qᵀ,  PV [v, i] = (β E) Pᵀ    off the chain, under the element-wise steps
// so that the state, the right hand side and the corrections go from registers to TMEM and never through shared
// memory, a thread owning one row v (two threads to a row, each with half its columns).
//
// Precision: q, k, v are bf16 values as given and unit lengths are factors of rows and columns, so they enter
// exactly.  fp32 operands -- S, X, T, W, P, β E -- enter as two bf16 terms, hi + lo (the product of two such pairs
// without lo·lo): 16 bits, an error near 2^-18 a product.  One term for P and β E would do for y's own rounding,
// but not where keys repeat: the corrections are then differences of values, and P (β E) cancels most of them.
// Accumulation is fp32, the state is kept in fp32 registers.
//
// Warps: 0..7 state (above); 8..11 prepare (per-token scalars, K Kᵀ and Q Kᵀ, the inverse T: up to two chunks ahead);
// 12 issues the chain's MMAs; 13 the TMA loads (three tiles of K, Q, V in flight).  They hand over through
// mbarriers.  Every wait is bounded: one that runs out records SS_ERR_TIMEOUT and the CTA winds down.
#pragma once

#include "../../include/selscan.h"
#include "gdr_rec.cuh"
#include "ssd_tc.cuh"

namespace selscan {
namespace gdr {

using tc::bulk_wait0;
using tc::chunk_addr;
using tc::hi_f;
using tc::lds128;
using tc::lo_f;
using tc::mbar_arrive;
using tc::pk;
using tc::sdesc;
using tc::sts128;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::tma_load_4d;
using tc::tmem_ld32;
using tc::umma;
using tc::umma_commit;

constexpr int kC = 64;                 // tokens of a chunk
constexpr int kStages = 3;             // K, Q tiles in flight (they are prepared ahead)
constexpr int kVStages = 2;            // V tiles in flight
constexpr int kStateWarps = 8, kPrepWarps = 4;
constexpr int kMmaWarp = kStateWarps + kPrepWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kLoadWarp + 1);

// TMEM columns.  S: the state's bf16 terms (hi and lo of each half of the keys, d_k columns in all); dS is
// accumulated over them once they have been read.
constexpr uint32_t kColS = 0, kColKS = 128, kColQS = 192, kColPV = 256, kColX = 320, kColVn = 384, kColGram = 448;
constexpr uint32_t kTmemCols = 512;

// Shared memory: byte offsets from a 1024-aligned base.
constexpr uint32_t kTile = 8192;                       // 64 rows of 128 bytes, 128-byte swizzle
constexpr uint32_t kStageBytes = 4 * kTile;            // [K 0][Q 0][K 1][Q 1]
constexpr uint32_t kOffV = kStages * kStageBytes;      // V [64][d_v], not swizzled
constexpr uint32_t kVBytes = 2 * kTile;
constexpr uint32_t kOffPrep = kOffV + kVStages * kVBytes;   // two buffers of [T hi][T lo][P hi][P lo]
constexpr uint32_t kPrepBytes = 4 * kTile;
constexpr uint32_t kOffA = kOffPrep + 2 * kPrepBytes;  // A', then T, fp32 [64][68]
constexpr int kPitchA = 68;
constexpr uint32_t kOffXs = kOffA + kC * kPitchA * 4;  // block products, fp32 [32][36]
constexpr int kPitchX = 36;
constexpr uint32_t kOffScal = kOffXs + 32 * kPitchX * 4;
// two buffers of per-token factors, then what only the prepare warps use
constexpr uint32_t kScalBytes = (4 * kC + 4) * 4;
constexpr uint32_t kOffLocal = kOffScal + 2 * kScalBytes;      // G hi, G lo, |k|^-1, β, 64-bit prefix
constexpr uint32_t kLocalBytes = 4 * kC * 4 + kC * 8;
constexpr uint32_t kOffBar = kOffLocal + kLocalBytes;
constexpr uint32_t kSmemBytes = kOffBar + 256 + 1024;
static_assert(kOffScal % 16 == 0 && kOffLocal % 16 == 0 && kOffBar % 16 == 0, "aligned regions");
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

struct alignas(16) Scal {   // one chunk's factors, as the state warps read them
    float ek[kC];      // e^{G_i} / |k_i|
    float be[kC];      // β_i
    float wk[kC];      // β_i e^{G_end - G_i} / |k_i|
    float qe[kC];      // scale e^{G_i} / |q_i|
    float end[4];      // e^{G_end}
};
static_assert(sizeof(Scal) == kScalBytes, "layout");

struct Params {
    GdrParams g;
    uint32_t* status;
    int dv;
    int test_drop;
    uint64_t wait_ns, drain_ns;
};

// kind::f16, bf16 x bf16 -> fp32, M = 128; bmn: B is MN-major.
__host__ __device__ constexpr uint32_t idesc(uint32_t n, bool bmn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (bmn ? 1u << 16 : 0u) | ((n >> 3) << 17) | (8u << 24);
}

// D[tmem] (+)= A[tmem] · B[smem descriptor]; issued by one thread.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
    const uint32_t z = 0;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8}, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(id), "r"(acc), "r"(z), "r"(z), "r"(z), "r"(z)
        : "memory");
}
// 16 columns of this thread's lane, written; complete after tmem_wait_st().
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 values as 16 words of bf16 pairs: hi, and lo = what hi leaves.
__device__ __forceinline__ void split32(const float (&v)[32], uint32_t (&hi)[16], uint32_t (&lo)[16]) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        hi[e] = pk(v[2 * e], v[2 * e + 1]);
        lo[e] = pk(v[2 * e] - lo_f(hi[e]), v[2 * e + 1] - hi_f(hi[e]));
    }
}

constexpr int kPrepBar = 1;   // named barrier of the 128 prepare threads
__device__ __forceinline__ void prep_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool prep_any(bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(pred ? 1u : 0u)
        : "memory");
    return r != 0;
}

struct Bars {
    uint64_t full[kStages];    // K and Q of a stage landed
    uint64_t v_full[kVStages], v_empty[kVStages];   // V landed; read (8 warps)
    uint64_t empty[kStages];   // the chunk's last MMA is done with the stage
    uint64_t prep_full[2];     // T, P and the factors of a buffer written (4 warps)
    uint64_t prep_empty[2];    // its last MMA done (1) and its factors read (8 warps)
    uint64_t gram;             // K Kᵀ and Q Kᵀ done
    uint64_t ks, e, ds, pv;    // the chain's products done
    uint64_t qs;               // S's terms read by KS and QS
    uint64_t s_ready;          // S's terms written (8 warps)
    uint64_t x_ready, w_ready; // X, W written (8 warps)
    uint64_t o_free;           // QS and PV read (8 warps)
    uint64_t fin[2];           // wind-down
    uint32_t tmem;
};
static_assert(sizeof(Bars) <= 256, "barrier region");

// Sum over four values' products of a 16-byte word of bf16 pairs with itself.
__device__ __forceinline__ float sq8(uint4 w, float s) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) s = fmaf(lo_f(a[e]), lo_f(a[e]), fmaf(hi_f(a[e]), hi_f(a[e]), s));
    return s;
}

// (I + A')^-1 of the strictly lower triangular A' in `a` ([64][kPitchA]), in place, by the 128 prepare threads:
// the four 16-blocks on the diagonal column by column, then T21 = -T22 A21 T11 of the 32-blocks and of the whole.
// fp32 throughout; about 75 000 multiply-adds.
__device__ __forceinline__ void invert64(float* a, float* xs, int pt) {
    const int pw = pt >> 5, lane = pt & 31;
    {
        float* d = a + 16 * pw * kPitchA + 16 * pw;
        const int j = lane & 15;
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
            for (int l = 0; l < i; l += 4) {
                const float4 r = *reinterpret_cast<const float4*>(d + i * kPitchA + l);
                s0 = fmaf(r.x, t[l], s0);
                if (l + 1 < i) s1 = fmaf(r.y, t[l + 1], s1);
                if (l + 2 < i) s0 = fmaf(r.z, t[l + 2], s0);
                if (l + 3 < i) s1 = fmaf(r.w, t[l + 3], s1);
            }
            t[i] = (i == j ? 1.0f : 0.0f) - (s0 + s1);
        }
        __syncwarp();
        if (lane < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) d[i * kPitchA + j] = t[i];
        }
    }
    prep_sync();
    {   // 16-blocks: threads 64 m .. 64 m + 63 on the 32-block m, four neighbouring columns each
        const int m = pt >> 6, r = (pt & 63) >> 2, c = (pt & 3) * 4;
        float* d = a + 32 * m * kPitchA + 32 * m;
        float* x = xs + m * 16 * kPitchX;
        auto product = [&](const float* p, int pp, const float* q, int pq) {
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
                const float4 u = *reinterpret_cast<const float4*>(p + r * pp + k);
                const float uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 w = *reinterpret_cast<const float4*>(q + (k + e) * pq + c);
                    s.x = fmaf(uu[e], w.x, s.x);
                    s.y = fmaf(uu[e], w.y, s.y);
                    s.z = fmaf(uu[e], w.z, s.z);
                    s.w = fmaf(uu[e], w.w, s.w);
                }
            }
            return s;
        };
        const float4 s = product(d + 16 * kPitchA, kPitchA, d, kPitchA);
        *reinterpret_cast<float4*>(x + r * kPitchX + c) = make_float4(-s.x, -s.y, -s.z, -s.w);
        prep_sync();
        const float4 t = product(d + 16 * kPitchA + 16, kPitchA, x, kPitchX);
        *reinterpret_cast<float4*>(d + (16 + r) * kPitchA + c) = t;
    }
    prep_sync();
    {   // 32-blocks: two rows of four columns each
        const int r = (pt >> 3) * 2, c = (pt & 7) * 4;
        auto product = [&](const float* p, int pp, const float* q, int pq, float4 (&s)[2]) {
            s[0] = s[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
                const float4 u = *reinterpret_cast<const float4*>(p + r * pp + k);
                const float4 v = *reinterpret_cast<const float4*>(p + (r + 1) * pp + k);
                const float uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 w = *reinterpret_cast<const float4*>(q + (k + e) * pq + c);
                    s[0] = make_float4(fmaf(uu[e], w.x, s[0].x), fmaf(uu[e], w.y, s[0].y), fmaf(uu[e], w.z, s[0].z),
                                       fmaf(uu[e], w.w, s[0].w));
                    s[1] = make_float4(fmaf(vv[e], w.x, s[1].x), fmaf(vv[e], w.y, s[1].y), fmaf(vv[e], w.z, s[1].z),
                                       fmaf(vv[e], w.w, s[1].w));
                }
            }
        };
        float4 s[2];
        product(a + 32 * kPitchA, kPitchA, a, kPitchA, s);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float4*>(xs + (r + i) * kPitchX + c) = make_float4(-s[i].x, -s[i].y, -s[i].z, -s[i].w);
        prep_sync();
        product(a + 32 * kPitchA + 32, kPitchA, xs, kPitchX, s);
#pragma unroll
        for (int i = 0; i < 2; ++i) *reinterpret_cast<float4*>(a + (32 + r + i) * kPitchA + c) = s[i];
    }
    prep_sync();
}

// Grid: one CTA per (b, h).
template <int DK>
__global__ void __launch_bounds__(kThreads, 1)
ss_gdr_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tm_q,
                 const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
    constexpr int KB = DK / 64;       // 64-wide blocks of a K or Q row
    constexpr int KH = DK / 2;        // keys of a state thread
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* gbase = smem_raw + (base - raw);
    Bars* const bar = reinterpret_cast<Bars*>(gbase + kOffBar);
    Scal* const scal = reinterpret_cast<Scal*>(gbase + kOffScal);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const GdrParams& g = p.g;
    const int item = blockIdx.x, b = item / g.H, h = item % g.H, hk = h / (g.H / g.Hk);
    const int64_t len = gdr_len(g, b);
    const int nchunk = static_cast<int>((len + kC - 1) / kC);
    const uint64_t lim = p.wait_ns;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bar->full[i], 1);
            mbar_init(&bar->empty[i], 1);
        }
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(&bar->v_full[i], 1);
            mbar_init(&bar->v_empty[i], kStateWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar->prep_full[i], kPrepWarps);
            mbar_init(&bar->prep_empty[i], 1 + kStateWarps);
            mbar_init(&bar->fin[i], 1);
        }
        uint64_t* one[] = {&bar->gram, &bar->ks, &bar->e, &bar->ds, &bar->pv, &bar->qs};
        for (uint64_t* x : one) mbar_init(x, 1);
        uint64_t* all[] = {&bar->s_ready, &bar->x_ready, &bar->w_ready, &bar->o_free};
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
    // one thread's wait; a whole warp's (uniform outcome)
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

    int issued = 0, v_issued = 0;   // loads of the load thread

    if (warp == kLoadWarp) {
        // ============================================================ loads (one thread)
        if (lane == 0) {
            tma_prefetch_desc(&tm_q);
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
            for (int c = 0; c < nchunk; ++c) {
                const int s = c % kStages;
                if (c >= kStages && !wait1(&bar->empty[s], ((c / kStages) - 1) & 1)) break;
                const uint32_t st = base + s * kStageBytes;
                mbar_arrive_expect_tx(&bar->full[s], 2 * KB * kTile);
                for (int kb = 0; kb < KB; ++kb) {
                    tma_load_4d(st + (2 * kb) * kTile, &tm_k, 64 * kb, hk, c * kC, b, &bar->full[s]);
                    tma_load_4d(st + (2 * kb + 1) * kTile, &tm_q, 64 * kb, hk, c * kC, b, &bar->full[s]);
                }
                issued = c + 1;
                const int vs = c % kVStages;
                if (c >= kVStages && !wait1(&bar->v_empty[vs], ((c / kVStages) - 1) & 1)) break;
                mbar_arrive_expect_tx(&bar->v_full[vs], kC * p.dv * 2);
                tma_load_4d(base + kOffV + vs * kVBytes, &tm_v, 0, h, c * kC, b, &bar->v_full[vs]);
                v_issued = c + 1;
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ============================================================ the chain's MMAs (one thread)
        if (lane == 0) {
            for (int c = 0; c < nchunk; ++c) {
                const int s = c % kStages, pb = c & 1;
                const uint32_t par = c & 1, st = base + s * kStageBytes;
                const uint32_t pr = base + kOffPrep + pb * kPrepBytes;
                if (!wait1(&bar->full[s], (c / kStages) & 1)) break;
                if (!wait1(&bar->prep_full[pb], (c >> 1) & 1)) break;   // the tile's rows behind the end are zero
                if (!wait1(&bar->s_ready, par)) break;
                tc_fence_after();
                // S's two terms of the 16 keys of step ks
                auto s_hi = [&](int ks) { return tmem + kColS + (ks * 16 / KH) * KH + (ks * 16 % KH) / 2; };
#pragma unroll
                for (int ks = 0; ks < DK / 16; ++ks) {
                    const uint64_t bd = sdesc(st + (ks >> 2) * 2 * kTile + (ks & 3) * 32, 16, 1024);
                    umma_ts(tmem + kColKS, s_hi(ks), bd, idesc(kC, false), ks > 0);
                    umma_ts(tmem + kColKS, s_hi(ks) + KH / 2, bd, idesc(kC, false), 1);
                }
                if (!(p.test_drop && blockIdx.x == 0 && c == 0)) umma_commit(&bar->ks);
                if (c > 0 && !wait1(&bar->o_free, (c - 1) & 1)) break;   // QS and PV of the last chunk read
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < DK / 16; ++ks) {
                    const uint64_t bd = sdesc(st + ((ks >> 2) * 2 + 1) * kTile + (ks & 3) * 32, 16, 1024);
                    umma_ts(tmem + kColQS, s_hi(ks), bd, idesc(kC, false), ks > 0);
                    umma_ts(tmem + kColQS, s_hi(ks) + KH / 2, bd, idesc(kC, false), 1);
                }
                umma_commit(&bar->qs);
                if (!wait1(&bar->x_ready, par)) break;
                tc_fence_after();
                // E = X Tᵀ: tokens 16 j .. 16 j + 15 reach the rows i >= 16 j of T alone
#pragma unroll
                for (int j = 0; j < kC / 16; ++j) {
                    const uint32_t n = kC - 16 * j, row = 2048u * j + 32u * j;
                    const uint32_t d = tmem + kColKS + 16 * j, x = tmem + kColX + 8 * j;
                    umma_ts(d, x, sdesc(pr + row, 16, 1024), idesc(n, false), j > 0);
                    umma_ts(d, x, sdesc(pr + kTile + row, 16, 1024), idesc(n, false), 1);
                    umma_ts(d, x + 32, sdesc(pr + row, 16, 1024), idesc(n, false), 1);
                }
                umma_commit(&bar->e);
                if (!wait1(&bar->w_ready, par) || !wait1(&bar->qs, par)) break;
                tc_fence_after();
                // dS = W K over the columns of S's terms
#pragma unroll
                for (int j = 0; j < kC / 16; ++j) {
                    const uint64_t bd = sdesc(st + 2048u * j, 2 * kTile, 1024);
                    umma_ts(tmem + kColS, tmem + kColX + 8 * j, bd, idesc(DK, true), j > 0);
                    umma_ts(tmem + kColS, tmem + kColX + 32 + 8 * j, bd, idesc(DK, true), 1);
                }
                umma_commit(&bar->ds);
#pragma unroll
                for (int j = 0; j < kC / 16; ++j) {
                    const uint32_t n = kC - 16 * j, row = 2 * kTile + 2048u * j + 32u * j;
                    const uint32_t d = tmem + kColPV + 16 * j, x = tmem + kColVn + 8 * j;
                    umma_ts(d, x, sdesc(pr + row, 16, 1024), idesc(n, false), j > 0);
                    umma_ts(d, x, sdesc(pr + kTile + row, 16, 1024), idesc(n, false), 1);
                    umma_ts(d, x + 32, sdesc(pr + row, 16, 1024), idesc(n, false), 1);
                }
                umma_commit(&bar->pv);
                umma_commit(&bar->empty[s]);
                umma_commit(&bar->prep_empty[pb]);
            }
        }
        __syncwarp();
    } else if (warp >= kStateWarps) {
        // ============================================================ prepare warps
        const int pt = tid - 32 * kStateWarps, i = pt & 63;
        const bool is_q = pt >= 64;
        float* const Gh = reinterpret_cast<float*>(gbase + kOffLocal);
        float *const Gl = Gh + kC, *const rk = Gl + kC, *const be = rk + kC;
        double* const Gd = reinterpret_cast<double*>(be + kC);
        float* const a = reinterpret_cast<float*>(gbase + kOffA);
        float* const xs = reinterpret_cast<float*>(gbase + kOffXs);
        const float Ah = g.A[h], bias = g.dt_bias ? g.dt_bias[h] : 0.0f;
        const __nv_bfloat16* dtp = static_cast<const __nv_bfloat16*>(g.dt);
        const __nv_bfloat16* bep = static_cast<const __nv_bfloat16*>(g.beta);
        float dt_n = 0.0f, be_n = 0.0f;
        auto fetch = [&](int c) {   // the raw gates of this thread's token
            const int64_t t = static_cast<int64_t>(c) * kC + i;
            if (!is_q && t < len) {
                const int64_t o = (static_cast<int64_t>(b) * g.L + t) * g.H + h;
                dt_n = to_f32(dtp[o]);
                be_n = to_f32(bep[o]);
            }
        };
        if (nchunk > 0) fetch(0);
        for (int c = 0; c < nchunk; ++c) {
            const int s = c % kStages, pb = c & 1;
            const uint32_t st = base + s * kStageBytes, pr = base + kOffPrep + pb * kPrepBytes;
            Scal& sc = scal[pb];
            const int valid = static_cast<int>(len - static_cast<int64_t>(c) * kC < kC ? len - static_cast<int64_t>(c) * kC : kC);
            bool got = mbar_wait_bounded(&bar->full[s], (c / kStages) & 1, lim);
            if (got && valid < kC) got = mbar_wait_bounded(&bar->v_full[c % kVStages], (c / kVStages) & 1, lim);
            if (got && c >= 2) got = mbar_wait_bounded(&bar->prep_empty[pb], ((c >> 1) - 1) & 1, lim);
            if (prep_any(!got)) {
                if (pt == 0) record();
                break;
            }
            // rows behind the end (another token's values, or anything) become zero rows
            if (i >= valid) {
                for (int kb = 0; kb < KB; ++kb)
                    for (int w = 0; w < 8; ++w)
                        sts128(st + (2 * kb + (is_q ? 1 : 0)) * kTile + i * 128 + w * 16, make_uint4(0, 0, 0, 0));
                if (!is_q)
                    for (int w = 0; w < p.dv / 8; ++w) 
                        sts128(base + kOffV + (c % kVStages) * kVBytes + i * p.dv * 2 + w * 16, make_uint4(0, 0, 0, 0));
                fence_proxy_async_smem();
            }
            float rn = 1.0f;   // 1 / |row i| of K, or of Q
            if (g.l2norm) {
                float q0 = 0.0f, q1 = 0.0f;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int w = 0; w < 8; w += 2) {
                        const uint32_t blk = st + (2 * kb + (is_q ? 1 : 0)) * kTile;
                        q0 = sq8(lds128(chunk_addr(blk, i, w)), q0);
                        q1 = sq8(lds128(chunk_addr(blk, i, w + 1)), q1);
                    }
                rn = 1.0f / sqrtf(q0 + q1 + kGdrL2Eps);
            }
            double G = 0.0;
            if (!is_q) {
                const bool in = i < valid;
                const float delta = in ? gdr_delta(dt_n, bias, g.softplus) : 0.0f;
                be[i] = in ? gdr_beta(be_n, g.sigmoid) : 0.0f;
                rk[i] = rn;
                if (c + 1 < nchunk) fetch(c + 1);
                G = static_cast<double>(delta) * static_cast<double>(Ah) * 1.4426950408889634074;   // log2 α
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double v = __shfl_up_sync(0xffffffffu, G, o);
                    if (lane >= o) G += v;
                }
                Gd[i] = G;
            }
            tc_fence_before();
            prep_sync();
            if (pt == 0) {   // [K; Q] Kᵀ: lanes 0..63 K's rows, 64..127 Q's
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < DK / 16; ++ks) {
                    const uint32_t off = (ks >> 2) * 2 * kTile + (ks & 3) * 32;
                    umma(tmem + kColGram, sdesc(st + off, 16, 1024), sdesc(st + off, 16, 1024), idesc(kC, false), ks > 0);
                }
                umma_commit(&bar->gram);
            }
            const double first = Gd[31], end = first + Gd[63];
            if (!is_q) {
                if (i >= 32) G += first;
                const float hi = static_cast<float>(G);
                Gh[i] = hi;
                Gl[i] = static_cast<float>(G - static_cast<double>(hi));
                sc.ek[i] = exp2f(hi) * rn;
                sc.be[i] = be[i];
                sc.wk[i] = be[i] * exp2f(static_cast<float>(end - G)) * rn;
                if (i == 0) sc.end[0] = exp2f(static_cast<float>(end));
            }
            if (prep_any(!mbar_wait_bounded(&bar->gram, c & 1, lim))) {
                if (pt == 0) record();
                break;
            }
            tc_fence_after();
            {
                const float gh = Gh[i], gl = Gl[i];
                const float row = is_q ? rn * g.scale : rn;
                if (is_q) sc.qe[i] = exp2f(gh) * row;
                const uint32_t src = tmem + kColGram + (static_cast<uint32_t>((warp & 3) * 32) << 16);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float v[32];
                    tmem_ld32(src + 32 * half, v);
#pragma unroll
                    for (int j4 = 0; j4 < 32; j4 += 4) {
                        const int j = 32 * half + j4;
                        const float4 h4 = *reinterpret_cast<const float4*>(Gh + j), l4 = *reinterpret_cast<const float4*>(Gl + j);
                        const float4 r4 = *reinterpret_cast<const float4*>(rk + j), b4 = *reinterpret_cast<const float4*>(be + j);
                        const float hh[4] = {h4.x, h4.y, h4.z, h4.w}, ll[4] = {l4.x, l4.y, l4.z, l4.w};
                        const float rr[4] = {r4.x, r4.y, r4.z, r4.w}, bb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float d = ex2_approx((gh - hh[e]) + (gl - ll[e]));
                            const float f = v[j4 + e] * row * rr[e] * d * (is_q ? 1.0f : bb[e]);
                            v[j4 + e] = (is_q ? j + e <= i : j + e < i) ? f : 0.0f;
                        }
                    }
                    if (is_q) {
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            uint32_t hw[4], lw[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float x0 = v[8 * w + 2 * e], x1 = v[8 * w + 2 * e + 1];
                                hw[e] = pk(x0, x1);
                                lw[e] = pk(x0 - lo_f(hw[e]), x1 - hi_f(hw[e]));
                            }
                            sts128(chunk_addr(pr + 2 * kTile, i, 4 * half + w), make_uint4(hw[0], hw[1], hw[2], hw[3]));
                            sts128(chunk_addr(pr + 3 * kTile, i, 4 * half + w), make_uint4(lw[0], lw[1], lw[2], lw[3]));
                        }
                    } else {
#pragma unroll
                        for (int w = 0; w < 8; ++w)
                            *reinterpret_cast<float4*>(a + i * kPitchA + 32 * half + 4 * w) =
                                make_float4(v[4 * w], v[4 * w + 1], v[4 * w + 2], v[4 * w + 3]);
                    }
                }
            }
            prep_sync();
            invert64(a, xs, pt);
            {   // T as two bf16 terms: half a row each
                const int r = pt >> 1, j0 = (pt & 1) * 32;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float4 u = *reinterpret_cast<const float4*>(a + r * kPitchA + j0 + 8 * w);
                    const float4 v = *reinterpret_cast<const float4*>(a + r * kPitchA + j0 + 8 * w + 4);
                    // what lies above the diagonal blocks was A's zero
                    const uint32_t h0 = pk(u.x, u.y), h1 = pk(u.z, u.w), h2 = pk(v.x, v.y), h3 = pk(v.z, v.w);
                    sts128(chunk_addr(pr, r, (pt & 1) * 4 + w), make_uint4(h0, h1, h2, h3));
                    sts128(chunk_addr(pr + kTile, r, (pt & 1) * 4 + w),
                           make_uint4(pk(u.x - lo_f(h0), u.y - hi_f(h0)), pk(u.z - lo_f(h1), u.w - hi_f(h1)),
                                      pk(v.x - lo_f(h2), v.y - hi_f(h2)), pk(v.z - lo_f(h3), v.w - hi_f(h3))));
                }
            }
            fence_proxy_async_smem();
            arrive_warp(&bar->prep_full[pb]);
        }
    } else {
        // ============================================================ state warps
        const int v = (warp & 3) * 32 + lane, half = warp >> 2;
        const bool row_in = v < p.dv;
        const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const int64_t srow = (static_cast<int64_t>(item) * p.dv + v) * DK + half * KH;
        float S[KH];
#pragma unroll
        for (int k = 0; k < KH; k += 4) {
            float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (g.h_init && row_in) q = *reinterpret_cast<const float4*>(g.h_init + srow + k);
            S[k] = q.x;
            S[k + 1] = q.y;
            S[k + 2] = q.z;
            S[k + 3] = q.w;
        }
        auto store_s = [&]() {   // S's two terms into this thread's d_k / 2 columns
#pragma unroll
            for (int k = 0; k < KH; k += 32) {
                float t[32];
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int e = 0; e < 32; ++e) t[e] = S[k + e];
                split32(t, hi, lo);
                tmem_st16(tl + kColS + half * KH + k / 2, hi);
                tmem_st16(tl + kColS + half * KH + KH / 2 + k / 2, lo);
            }
            tmem_wait_st();
            tc_fence_before();
        };
        store_s();
        arrive_warp(&bar->s_ready);
        bool ok = true;
        for (int c = 0; c < nchunk; ++c) {
            const int vs = c % kVStages, pb = c & 1;
            const uint32_t par = c & 1;
            const Scal& sc = scal[pb];
            const int64_t t0 = static_cast<int64_t>(c) * kC + half * 32;
            ok = wait_warp(&bar->v_full[vs], (c / kVStages) & 1) && wait_warp(&bar->prep_full[pb], (c >> 1) & 1) &&
                 wait_warp(&bar->ks, par);
            if (!ok) break;
            tc_fence_after();
            {   // X = V - diag(e^G / |k|) K Sᵀ of this thread's 32 tokens
                float x[32];
                tmem_ld32(tl + kColKS + 32 * half, x);
                const __nv_bfloat16* vt = reinterpret_cast<const __nv_bfloat16*>(gbase + kOffV + vs * kVBytes) +
                                          half * 32 * p.dv + v;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float vv = row_in ? __bfloat162float(vt[e * p.dv]) : 0.0f;
                    x[e] = fmaf(-sc.ek[32 * half + e], x[e], vv);
                }
                uint32_t hi[16], lo[16];
                split32(x, hi, lo);
                tmem_st16(tl + kColX + 16 * half, hi);
                tmem_st16(tl + kColX + 32 + 16 * half, lo);
                tmem_wait_st();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar->x_ready);
                mbar_arrive(&bar->v_empty[vs]);
            }
            ok = wait_warp(&bar->e, par);
            if (!ok) break;
            tc_fence_after();
            {
                float x[32], w[32];
                tmem_ld32(tl + kColKS + 32 * half, x);
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int e = 0; e < 32; ++e) w[e] = x[e] * sc.wk[32 * half + e];
                split32(w, hi, lo);
                tmem_st16(tl + kColX + 16 * half, hi);
                tmem_st16(tl + kColX + 32 + 16 * half, lo);
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] *= sc.be[32 * half + e];
                split32(x, hi, lo);
                tmem_st16(tl + kColVn + 16 * half, hi);
                tmem_st16(tl + kColVn + 32 + 16 * half, lo);
                tmem_wait_st();
                tc_fence_before();
            }
            arrive_warp(&bar->w_ready);
            ok = wait_warp(&bar->ds, par);
            if (!ok) break;
            tc_fence_after();
            const float end = sc.end[0];
#pragma unroll
            for (int k = 0; k < KH; k += 32) {
                float d[32];
                tmem_ld32(tl + kColS + half * KH + k, d);
#pragma unroll
                for (int e = 0; e < 32; ++e) S[k + e] = fmaf(end, S[k + e], d[e]);
            }
            store_s();
            arrive_warp(&bar->s_ready);
            // y, while the next chunk's K Sᵀ runs
            ok = wait_warp(&bar->pv, par);
            if (!ok) break;
            tc_fence_after();
            {
                float qs[32], pv[32];
                tmem_ld32(tl + kColQS + 32 * half, qs);
                tmem_ld32(tl + kColPV + 32 * half, pv);
                tc_fence_before();
                __nv_bfloat16* yp = static_cast<__nv_bfloat16*>(g.y) +
                                    ((static_cast<int64_t>(b) * g.L + t0) * g.H + h) * p.dv + v;
                const int64_t pitch = static_cast<int64_t>(g.H) * p.dv;
                const int n = row_in ? static_cast<int>(len - t0 < 32 ? len - t0 : 32) : 0;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (e < n) yp[e * pitch] = __float2bfloat16_rn(fmaf(sc.qe[32 * half + e], qs[e], pv[e]));
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar->o_free);
                mbar_arrive(&bar->prep_empty[pb]);
            }
        }
        if (ok && g.final_state && row_in) {
#pragma unroll
            for (int k = 0; k < KH; k += 4)
                *reinterpret_cast<float4*>(g.final_state + srow + k) = make_float4(S[k], S[k + 1], S[k + 2], S[k + 3]);
        }
    }

    // Wind-down: loads in flight land before the shared memory goes, MMAs end before the TMEM columns do.
    __syncthreads();
    if (warp == kLoadWarp && lane == 0) {
        for (int c = issued > kStages ? issued - kStages : 0; c < issued; ++c)
            mbar_wait_bounded(&bar->full[c % kStages], (c / kStages) & 1, p.drain_ns);
        for (int c = v_issued > kVStages ? v_issued - kVStages : 0; c < v_issued; ++c)
            mbar_wait_bounded(&bar->v_full[c % kVStages], (c / kVStages) & 1, p.drain_ns);
    }
    if (warp == kMmaWarp && lane == 0) {
        umma_commit(&bar->fin[0]);
        mbar_wait_bounded(&bar->fin[0], 0, p.drain_ns);
    }
    if (tid == 32 * kStateWarps) {
        umma_commit(&bar->fin[1]);
        mbar_wait_bounded(&bar->fin[1], 0, p.drain_ns);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace gdr
}  // namespace selscan
