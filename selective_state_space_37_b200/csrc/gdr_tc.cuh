// gdr_tc.cuh -- the gated delta rule chunk by chunk on the fifth-generation tensor cores (sm_100a).
//
// Per (b, value head h), over a chunk of C = 64 tokens with G_i = Σ_{r<=i} Δ_r A (so α_i ... α_{j+1} = e^{G_i - G_j}),
// S the state that enters it (d_v x d_k), K, Q, V, E the chunk's rows:
//   e_i = v_i - e^{G_i} S k̂_i - Σ_{j<i} e^{G_i - G_j} (k̂_i·k̂_j) β_j e_j
// is one triangular system for all 64 corrections, so with A'_ij = e^{G_i - G_j} (k̂_i·k̂_j) β_j (j < i):
//   E = T (V - diag(e^G) K̂ Sᵀ),  T = (I + A')^-1
//   Y = diag(e^G) Q̂ Sᵀ + P E,       P_ij = e^{G_i - G_j} (q̂_i·k̂_j) β_j (j <= i)
//   S <- e^{G_end} S + (diag(β e^{G_end - G}) E)ᵀ K̂
// Every exponent is a difference G_i - G_j with j <= i, so nothing overflows; the differences are taken of 48-bit
// values (pairs of floats of a 64-bit prefix sum), so a long decay keeps its near differences.
//
// Two kernels.  What does not depend on S -- T, P and the factors -- is prepared for every chunk at once
// (ss_gdr_prep_kernel, a block per chunk, five resident per SM) and left in the workspace, as the shared-memory
// image that the second kernel copies in.  ss_gdr_tc_kernel then walks the chunks of a (b, h) in order; in its chain
// from chunk to chunk remain three products and three element-wise steps.  With the preparation inside the second
// kernel (two groups of four warps, up to two chunks ahead) its latency, about 14 000 cycles a chunk beside the
// state's warps, set the pace: 8 700 cycles a chunk.
//
// Precision: q, k, v are bf16 values as given and unit lengths are factors of rows and columns, so they enter
// exactly.  fp32 operands enter as bf16 terms of 8 bits each: S, X and W as three, hi to third, 24 bits; T, P and E as
// two.  With two for S and X the state is 1.2e-6 off on average, with three 6e-7 (all of it T's; W with two alone: 2.4e-6).
// The backward pass's fp32 outputs are sums of both signs: its forward half takes T, and its adjoint P, as three.
// One term for P and E would do for y's own rounding, but not where keys repeat: the corrections are then differences
// of values, and P E cancels most of them.  Accumulation is fp32, the state is kept in fp32 registers.
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

constexpr int kC = 64;                  // tokens of a chunk
constexpr uint32_t kTile = 8192;        // 64 rows of 128 bytes, 128-byte swizzle
constexpr int kPitchX = 36;             // floats from row to row of the inverse's scratch

struct alignas(16) Scal {   // one chunk's factors
    float ek[kC];           // -e^{G_i} / |k_i|
    float wk[kC];           // β_i e^{G_end - G_i} / |k_i|
    float qe[kC];           // scale e^{G_i} / |q_i|
    float end[4];           // e^{G_end}
    float pad[60];
};
// One chunk's record in the workspace: T and P, each as two bf16 terms in the swizzled layout that the MMAs read, then
// the factors.
constexpr uint32_t kRecT = 0, kRecP = 2 * kTile, kRecScal = 4 * kTile;
constexpr uint32_t kRecBytes = kRecScal + sizeof(Scal);
static_assert(sizeof(Scal) == 1024 && kRecBytes % 16 == 0, "records are copied whole");

struct alignas(16) Local {  // what a chunk's decay factors are made of (the backward pass keeps it behind the record)
    float gh[kC], gl[kC];   // log2 of the decay from the chunk's start, as a pair
    float cb[kC];           // β_j / |k_j|
    float cf[kC];           // β_j / |k_j| e^{G_31 - G_j}, j < 32
    float rk[kC], rq[kC];   // 1 / |k_i|, scale / |q_i|
};
// For the backward pass also the third terms of T and P.
constexpr uint32_t kRecLocal = kRecBytes, kRecT3 = kRecLocal + 2048, kRecP3 = kRecT3 + kTile, kRecBwdBytes = kRecP3 + kTile;
static_assert(sizeof(Local) <= 2048, "record");

// What the backward pass keeps of a chunk, beside its record, as images of tiles with the swizzle of the MMAs.  Eᵀ as
// three bf16 terms, dVᵀ as two: [128 rows v][64 tokens] each; S, the state that enters the chunk, and dS, its adjoint, in
// fp32: [128 rows v][32 keys], d_k / 32 times.  (The state that leaves the last chunk has a place behind it.)
constexpr uint32_t kKeepE = 0, kKeepE3 = 4 * kTile, kKeepV = 6 * kTile, kKeepS = 10 * kTile, kKeepD = 18 * kTile;
constexpr uint32_t kKeepBytes = 26 * kTile;

struct Params {
    GdrParams g;
    unsigned char* rec;      // [items][nchunks] records
    int64_t nchunks;         // chunks of g.L tokens
    uint32_t rec_bytes;      // from record to record
    // time segments: items n_whole .. are cut into nseg segments of cseg chunks
    int n_whole, nseg, cseg;
    float* seg_in;           // [cut items][nseg - 1][d_v][d_k]: the states that enter the segments 1 ..
    float* seg_first;        // [cut items][d_v][d_k]: h_init, which the last segments may overwrite with the final state
                             // before the first ones have read it
    float* seg_loc;          // [cut items][nseg - 1][d_v][d_k]: a segment's end from a zero (segment 0: the entering) state
    float* seg_map;          // [cut items][nseg - 1][d_k][d_k]: its end from the unit matrix, without values
    // backward pass
    unsigned char* keep;     // [items][nchunks + 1]
    float* dots;             // [4][items][nchunks * 64] of each token, then [items][nchunks + 1]: e^{G_end} <S, dS> of a
                             // chunk's entering state and its leaving one's adjoint
    const float* dfinal;     // [batch, H, d_v, d_k] or null
    float* dinit;            // [batch, H, d_v, d_k] or null
    uint32_t* status;
    int dv;
    int test_drop;
    uint64_t wait_ns, drain_ns;
};

// kind::f16, bf16 x bf16 -> fp32, M = 128; bmn, amn: B, A is MN-major.
__host__ __device__ constexpr uint32_t idesc(uint32_t n, bool bmn, bool amn = false) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (amn ? 1u << 15 : 0u) | (bmn ? 1u << 16 : 0u) | ((n >> 3) << 17) | (8u << 24);
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
// 8 columns of this thread's lane, written; complete after tmem_wait_st().
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 16 columns of this thread's lane as pairs.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, f32x2 (&v)[8]) {
    float t[16];
    tc::tmem_ld16(taddr, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = pk2(t[2 * e], t[2 * e + 1]);
}

// Two such ranges, one wait.
__device__ __forceinline__ void tmem_ld16x2(uint32_t a0, uint32_t a1, f32x2 (&v)[8], f32x2 (&w)[8]) {
    float t[32];
    tc::tmem_ld16x2(a0, a1, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = pk2(t[2 * e], t[2 * e + 1]);
        w[e] = pk2(t[16 + 2 * e], t[17 + 2 * e]);
    }
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const f32x2 (&v)[8]) {
    uint32_t r[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r[2 * e] = __float_as_uint(v[4 * h + e].x);
            r[2 * e + 1] = __float_as_uint(v[4 * h + e].y);
        }
        tmem_st8(taddr + 8 * h, r);
    }
}

// A pair as a word of bf16 values, hi, and a word of what hi leaves, lo.
__device__ __forceinline__ void split2(f32x2 v, uint32_t& hi, uint32_t& lo) {
    hi = pk(v.x, v.y);
    const f32x2 r = fma2(pk2(lo_f(hi), hi_f(hi)), pk2(-1.0f, -1.0f), v);
    lo = pk(r.x, r.y);
}
// A pair as three words of bf16 values.
__device__ __forceinline__ void split3(f32x2 v, uint32_t& hi, uint32_t& lo, uint32_t& third) {
    hi = pk(v.x, v.y);
    split2(fma2(pk2(lo_f(hi), hi_f(hi)), pk2(-1.0f, -1.0f), v), lo, third);
}
// 16 values' terms into 16 columns: hi in the first 8, lo in the others.
__device__ __forceinline__ void store_terms(uint32_t taddr, const f32x2* v) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) split2(v[e], hi[e], lo[e]);
    tmem_st8(taddr, hi);
    tmem_st8(taddr + 8, lo);
}
// The same in three terms, the third in the first 8 columns of `third`.
__device__ __forceinline__ void store_terms3(uint32_t taddr, uint32_t third, const f32x2* v) {
    uint32_t hi[8], lo[8], th[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) split3(v[e], hi[e], lo[e], th[e]);
    tmem_st8(taddr, hi);
    tmem_st8(taddr + 8, lo);
    tmem_st8(third, th);
}
// v *= f, 16 consecutive factors of shared memory (16-byte aligned).
__device__ __forceinline__ void scale16(f32x2 (&v)[8], const float* f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float4 q = *reinterpret_cast<const float4*>(f + 4 * e);
        v[2 * e] = mul2(v[2 * e], pk2(q.x, q.y));
        v[2 * e + 1] = mul2(v[2 * e + 1], pk2(q.z, q.w));
    }
}


// The untiled bulk copies: shared memory to global memory, and back (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// Float offset of element (i, j) of the fp32 [64][64] matrix: 16-byte quads permuted within a row, so that the same
// quad of eight consecutive rows lies in eight different banks.
__device__ __forceinline__ int at(int i, int j) { return i * kC + ((((j >> 2) ^ (i & 7)) << 2) | (j & 3)); }

// acc += u · row of four (packed), u a scalar.
__device__ __forceinline__ void axpy4(f32x2 (&acc)[2], float u, float4 w) {
    acc[0] = fma2(pk2(u, u), pk2(w.x, w.y), acc[0]);
    acc[1] = fma2(pk2(u, u), pk2(w.z, w.w), acc[1]);
}
__device__ __forceinline__ float4 quad(const float* p) { return *reinterpret_cast<const float4*>(p); }

// (I + A')^-1 of the strictly lower triangular A' in `a`, in place, by 128 threads: the four 16-blocks on the
// diagonal row by row (x (I + A') = a unit row, from its last entry back: a subtracted row of A' per step, with no
// sum to wait for), then T21 = -T22 A21 T11 of the two 32-blocks and of the whole.  fp32 throughout.  The 32 x 32
// block above the diagonal is neither read nor written.
__device__ __forceinline__ void invert64(float* a, float* xs, int pt) {
    {
        const int o = 16 * (pt >> 5), i = pt & 15;
        float x[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = i == j ? 1.0f : 0.0f;
#pragma unroll
        for (int l = 15; l > 0; --l) {
#pragma unroll
            for (int j = 0; j < l; j += 4) {   // (A' is zero from its diagonal on)
                const float4 r = quad(a + at(o + l, o + j));
                f32x2 s[2] = {pk2(x[j], x[j + 1]), pk2(x[j + 2], x[j + 3])};
                axpy4(s, -x[l], r);
                x[j] = s[0].x;
                if (j + 1 < l) x[j + 1] = s[0].y;
                if (j + 2 < l) x[j + 2] = s[1].x;
                if (j + 3 < l) x[j + 3] = s[1].y;
            }
        }
        __syncwarp();
        if ((pt & 31) < 16) {
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                *reinterpret_cast<float4*>(a + at(o + i, o + j)) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
        }
    }
    __syncthreads();
    {   // 16-blocks: threads 64 m .. 64 m + 63 on the 32-block m, a quad of a row each
        const int m = pt >> 6, r = (pt & 63) >> 2, c = (pt & 3) * 4, o = 32 * m;
        float* x = xs + m * 16 * kPitchX + c;
        const float* ur = a + (o + 16 + r) * kC;
        const float* wc = a + o * kC;
        int oc[8];   // where this thread's quad of columns lies in the rows 0 .. 7 (mod 8)
#pragma unroll
        for (int e = 0; e < 8; ++e) oc[e] = (((o + c) >> 2) ^ e) << 2;
        const int r7 = r & 7;
        f32x2 s[2] = {pk2(0.0f, 0.0f), pk2(0.0f, 0.0f)};
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
            const float4 u = quad(ur + ((((o + k) >> 2) ^ r7) << 2));
            const float uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) axpy4(s, uu[e], quad(wc + (k + e) * kC + oc[(k + e) & 7]));
        }
        *reinterpret_cast<float4*>(x + r * kPitchX) = make_float4(-s[0].x, -s[0].y, -s[1].x, -s[1].y);
        __syncthreads();
        s[0] = s[1] = pk2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
            const float4 u = quad(ur + ((((o + 16 + k) >> 2) ^ r7) << 2));
            const float uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) axpy4(s, uu[e], quad(x + (k + e) * kPitchX));
        }
        *reinterpret_cast<float4*>(a + at(o + 16 + r, o + c)) = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
    }
    __syncthreads();
    {   // 32-blocks: a quad of two rows each
        const int r = (pt >> 3) * 2, c = (pt & 7) * 4, r7 = r & 7;   // (r even: row r + 1's permutation is r7 ^ 1)
        const float* ur = a + (32 + r) * kC;
        float* x = xs + c;
        int oc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) oc[e] = ((c >> 2) ^ e) << 2;
        f32x2 s[2] = {pk2(0.0f, 0.0f), pk2(0.0f, 0.0f)}, w[2] = {s[0], s[0]};
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
            const float4 u = quad(ur + (((k >> 2) ^ r7) << 2)), v = quad(ur + kC + (((k >> 2) ^ r7 ^ 1) << 2));
            const float uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 q = quad(a + (k + e) * kC + oc[(k + e) & 7]);
                axpy4(s, uu[e], q);
                axpy4(w, vv[e], q);
            }
        }
        *reinterpret_cast<float4*>(x + r * kPitchX) = make_float4(-s[0].x, -s[0].y, -s[1].x, -s[1].y);
        *reinterpret_cast<float4*>(x + (r + 1) * kPitchX) = make_float4(-w[0].x, -w[0].y, -w[1].x, -w[1].y);
        __syncthreads();
        s[0] = s[1] = w[0] = w[1] = pk2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
            const float4 u = quad(ur + (((8 + (k >> 2)) ^ r7) << 2)), v = quad(ur + kC + (((8 + (k >> 2)) ^ r7 ^ 1) << 2));
            const float uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 q = quad(x + (k + e) * kPitchX);
                axpy4(s, uu[e], q);
                axpy4(w, vv[e], q);
            }
        }
        *reinterpret_cast<float4*>(a + at(32 + r, c)) = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
        *reinterpret_cast<float4*>(a + at(33 + r, c)) = make_float4(w[0].x, w[0].y, w[1].x, w[1].y);
    }
    __syncthreads();
}

// v[i] for a runtime i < 32: a tree of selects on the bits of i.
__device__ __forceinline__ float pick32(const float (&v)[32], int i) {
    float a[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) a[e] = (i & 16) ? v[e + 16] : v[e];
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = (i & 8) ? a[e + 8] : a[e];
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = (i & 4) ? a[e + 4] : a[e];
#pragma unroll
    for (int e = 0; e < 2; ++e) a[e] = (i & 2) ? a[e + 2] : a[e];
    return (i & 1) ? a[1] : a[0];
}

// v_e *= row · cb_j e^{G_i - G_j}, j = j0 + e, for the 32 columns of row i's block on the diagonal; zero from the
// diagonal on (incl: above it).  `r` is i's place in the block.
__device__ __forceinline__ void decay_diagonal(float (&v)[32], const Local& lo, int j0, float gh, float gl, float row,
                                               int r, bool incl) {
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
        const float4 h4 = quad(lo.gh + j0 + e), l4 = quad(lo.gl + j0 + e), c4 = quad(lo.cb + j0 + e);
        const f32x2 hh[2] = {pk2(h4.x, h4.y), pk2(h4.z, h4.w)}, ll[2] = {pk2(l4.x, l4.y), pk2(l4.z, l4.w)};
        const f32x2 cc[2] = {pk2(c4.x, c4.y), pk2(c4.z, c4.w)};
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const f32x2 m1 = pk2(-1.0f, -1.0f);
            const f32x2 d = add2(fma2(hh[f], m1, pk2(gh, gh)), fma2(ll[f], m1, pk2(gl, gl)));
            const f32x2 w = mul2(mul2(pk2(v[e + 2 * f], v[e + 2 * f + 1]), cc[f]), pk2(row, row));
            const f32x2 x = mul2(w, pk2(ex2_approx(d.x), ex2_approx(d.y)));
            const int k = e + 2 * f - (incl ? 1 : 0);
            v[e + 2 * f] = k < r ? x.x : 0.0f;
            v[e + 2 * f + 1] = k + 1 < r ? x.y : 0.0f;
        }
    }
}
// The same for j < 32 <= i: both factors of e^{G_i - G_31} e^{G_31 - G_j} lie between the product and 1.
__device__ __forceinline__ void decay_left(float (&v)[32], const Local& lo, float gh, float gl, float row) {
    const float rf = row * exp2f((gh - lo.gh[31]) + (gl - lo.gl[31]));
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
        const float4 c4 = quad(lo.cf + e);
        const f32x2 r0 = mul2(mul2(pk2(v[e], v[e + 1]), pk2(c4.x, c4.y)), pk2(rf, rf));
        const f32x2 r1 = mul2(mul2(pk2(v[e + 2], v[e + 3]), pk2(c4.z, c4.w)), pk2(rf, rf));
        v[e] = r0.x;
        v[e + 1] = r0.y;
        v[e + 2] = r1.x;
        v[e + 3] = r1.y;
    }
}

// ------------------------------------------------------------------------------------------ preparation
constexpr int kPrepThreads = 128;

struct alignas(16) PrepSmem {
    double G[kC];           // prefix sums over 32 tokens
    uint64_t full, gram;
    uint32_t tmem, pad[3];
};
// Shared memory: [K 0][Q 0][K 1][Q 1], of which P's terms take the first two tiles once K and Q have been read, and T
// the others, first as fp32 [64][64] and then its terms; the factors; scratch.
constexpr uint32_t kPrepT = 2 * kTile, kPrepScal = 4 * kTile, kPrepLocal = kPrepScal + sizeof(Scal);
constexpr uint32_t kPrepState = kPrepLocal + 2048, kPrepXs = kPrepState + sizeof(PrepSmem);
constexpr uint32_t kPrepSmem = kPrepXs + 32 * kPitchX * 4 + 1024;
static_assert(kPrepXs % 16 == 0 && 5 * (kPrepSmem + 1024) <= 228 * 1024, "five resident blocks");

// Grid: one block per (item, chunk), a sequence's chunks together.  Bound by the latency of the triangular inverse
// (fp32, about 75 000 multiply-adds in a dozen dependent steps), which the five resident blocks hide for one another.
// 20480 chunks (4 x 8192 tokens, 40 heads of 128): 344-356 us, 2.5 us a chunk and SM, issue slots 40 % busy (four
// resident blocks: 366 us; the inverse's products on tf32 mma.sync: 395 against 366 us).  The third terms of T and P, for
// the backward pass alone, go from the registers to the record (3000 chunks: 68 against 51 us).
template <int DK>
__global__ void __launch_bounds__(kPrepThreads)
ss_gdr_prep_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_k) {
    constexpr int KB = DK / 64;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* gbase = smem_raw + (base - raw);
    Scal& sc = *reinterpret_cast<Scal*>(gbase + kPrepScal);
    Local& lo = *reinterpret_cast<Local*>(gbase + kPrepLocal);
    PrepSmem& ps = *reinterpret_cast<PrepSmem*>(gbase + kPrepState);
    float* const a = reinterpret_cast<float*>(gbase + kPrepT);
    float* const xs = reinterpret_cast<float*>(gbase + kPrepXs);

    const GdrParams& g = p.g;
    const int pt = threadIdx.x, lane = pt & 31, warp = pt >> 5, i = pt & 63, rb = warp & 1;   // row i, its 32-block
    const bool is_q = pt >= 64;
    const uint32_t nch = static_cast<uint32_t>(p.nchunks), H = static_cast<uint32_t>(g.H);   // (32-bit quotients)
    const int64_t item = blockIdx.x / nch, c = blockIdx.x % nch;
    const int b = static_cast<int>(blockIdx.x / nch / H), h = static_cast<int>(blockIdx.x / nch % H), hk = h / (g.H / g.Hk);
    const int64_t left = gdr_len(g, b) - c * kC;
    if (left <= 0) return;
    const int valid = left < kC ? static_cast<int>(left) : kC;

    if (pt == 0) {
        mbar_init(&ps.full, 1);
        mbar_init(&ps.gram, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(&ps.full, 2 * KB * kTile);
        for (int kb = 0; kb < KB; ++kb) {
            tma_load_4d(base + (2 * kb) * kTile, &tm_k, 64 * kb, hk, static_cast<int>(c) * kC, b, &ps.full);
            tma_load_4d(base + (2 * kb + 1) * kTile, &tm_q, 64 * kb, hk, static_cast<int>(c) * kC, b, &ps.full);
        }
    }
    if (warp == 0) {
        tc::tmem_alloc(&ps.tmem, kC);
        tc::tmem_relinquish();
    }
    float be = 0.0f;
    double G = 0.0;
    if (!is_q) {   // the gates, while K and Q come in
        const int64_t o = (static_cast<int64_t>(b) * g.L + c * kC + i) * g.H + h;
        float delta = 0.0f;
        if (i < valid) {
            delta = gdr_delta(to_f32(static_cast<const __nv_bfloat16*>(g.dt)[o]), g.dt_bias ? g.dt_bias[h] : 0.0f, g.softplus);
            be = gdr_beta(to_f32(static_cast<const __nv_bfloat16*>(g.beta)[o]), g.sigmoid);
            // β's gradient is a quotient by β; 1e-20 stands for a β of zero there, and changes nothing else
            if (p.keep && !g.sigmoid && fabsf(be) < 1e-20f) be = 1e-20f;
        }
        G = static_cast<double>(delta) * static_cast<double>(g.A[h]) * 1.4426950408889634074;   // log2 α
        if (G < -2048.0) G = -2048.0;   // α is zero in fp32 from -150 down; the floor keeps differences of infinities out
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const double v = __shfl_up_sync(0xffffffffu, G, s);
            if (lane >= s) G += v;
        }
        ps.G[i] = G;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ps.tmem;
    bool got = mbar_wait_bounded(&ps.full, 0, p.wait_ns);
    if (valid < kC) {   // rows behind the end, whatever they hold, become zero rows
        if (i >= valid && got) {
            for (int w = 0; w < 8 * KB; ++w)
                sts128(base + (2 * (w >> 3) + (is_q ? 1 : 0)) * kTile + i * 128 + (w & 7) * 16, make_uint4(0, 0, 0, 0));
            fence_proxy_async_smem();
        }
        __syncthreads();
    }
    const bool issued = got && pt == 0;
    if (issued) {   // [K; Q] Kᵀ: lanes 0..63 K's rows, 64..127 Q's
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) {
            const uint32_t off = (ks >> 2) * 2 * kTile + (ks & 3) * 32;
            umma(tmem, sdesc(base + off, 16, 1024), sdesc(base + off, 16, 1024), idesc(kC, false), ks > 0);
        }
        umma_commit(&ps.gram);
    }
    const double first = ps.G[31], end = first + ps.G[63];
    float rn = 1.0f;   // 1 / |row i| of K, or of Q
    if (!is_q) {
        if (i >= 32) G += first;
        const float hi = static_cast<float>(G);
        lo.gh[i] = hi;
        lo.gl[i] = static_cast<float>(G - static_cast<double>(hi));
        if (i == 0) sc.end[0] = exp2f(static_cast<float>(end));
    } else if (g.l2norm) {
        f32x2 q0 = pk2(0.0f, 0.0f), q1 = q0;
#pragma unroll
        for (int w = 0; w < 8 * KB; ++w) {
            const uint4 x = lds128(chunk_addr(base + (2 * (w >> 3) + 1) * kTile, i, w & 7));
            const f32x2 x0 = pk2(lo_f(x.x), hi_f(x.x)), x1 = pk2(lo_f(x.y), hi_f(x.y));
            const f32x2 x2 = pk2(lo_f(x.z), hi_f(x.z)), x3 = pk2(lo_f(x.w), hi_f(x.w));
            q0 = fma2(x0, x0, fma2(x2, x2, q0));
            q1 = fma2(x1, x1, fma2(x3, x3, q1));
        }
        rn = 1.0f / sqrtf((q0.x + q0.y) + (q1.x + q1.y) + kGdrL2Eps);
    }
    if (got) got = mbar_wait_bounded(&ps.gram, 0, p.wait_ns);
    const bool bad = __syncthreads_or(!got) != 0;
    if (bad) {
        if (pt == 0 && p.status) atomicCAS(p.status, 0u, static_cast<uint32_t>(SS_ERR_TIMEOUT));
    } else {
        tc_fence_after();
        const uint32_t src = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        float v[32];
        tmem_ld32(src + 32 * rb, v);   // the block on the diagonal
        if (!is_q) {                   // |k_i|² is K Kᵀ's own diagonal
            if (g.l2norm) rn = 1.0f / sqrtf(pick32(v, lane) + kGdrL2Eps);
            lo.rk[i] = rn;
            lo.cb[i] = be * rn;
            if (rb == 0) lo.cf[i] = be * rn * exp2f(static_cast<float>(first - G));
            sc.ek[i] = -exp2f(static_cast<float>(G)) * rn;
            sc.wk[i] = be * exp2f(static_cast<float>(end - G)) * rn;
        }
        __syncthreads();
        const float gh = lo.gh[i], gl = lo.gl[i];
        const float row = is_q ? rn * g.scale : rn;
        unsigned char* const rec = p.rec + (item * p.nchunks + c) * p.rec_bytes;
        // a third term's 8 values of row i, straight to the record (the backward pass's alone)
        auto put3 = [&](uint32_t image, int w, const uint32_t (&t)[4]) {
            *reinterpret_cast<uint4*>(rec + chunk_addr(image, i, w)) = make_uint4(t[0], t[1], t[2], t[3]);
        };
        if (is_q) {
            sc.qe[i] = exp2f(gh) * row;
            lo.rq[i] = row;
        }
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
            // first the block on the diagonal, then (rows 32..63) the block left of it; above the diagonal P is zero
            if (blk == 1) {
                if (rb == 0) {
                    if (is_q)
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            sts128(chunk_addr(base, i, 4 + w), make_uint4(0, 0, 0, 0));
                            sts128(chunk_addr(base + kTile, i, 4 + w), make_uint4(0, 0, 0, 0));
                            if (p.keep) put3(kRecP3, 4 + w, {0, 0, 0, 0});
                        }
                    break;
                }
                tmem_ld32(src, v);
            }
            const int j0 = blk == 0 ? 32 * rb : 0;
            if (blk == 0) decay_diagonal(v, lo, j0, gh, gl, row, lane, is_q);
            else decay_left(v, lo, gh, gl, row);
            if (is_q) {   // (K and Q have been read: by the MMAs, and by the lengths before the barriers above)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t hw[4], lw[4], tw[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) split3(pk2(v[8 * w + 2 * e], v[8 * w + 2 * e + 1]), hw[e], lw[e], tw[e]);
                    if (p.keep) put3(kRecP3, j0 / 8 + w, tw);
                    sts128(chunk_addr(base, i, j0 / 8 + w), make_uint4(hw[0], hw[1], hw[2], hw[3]));
                    sts128(chunk_addr(base + kTile, i, j0 / 8 + w), make_uint4(lw[0], lw[1], lw[2], lw[3]));
                }
            } else {
#pragma unroll
                for (int w = 0; w < 8; ++w)
                    *reinterpret_cast<float4*>(a + at(i, j0 + 4 * w)) =
                        make_float4(v[4 * w], v[4 * w + 1], v[4 * w + 2], v[4 * w + 3]);
            }
        }
        __syncthreads();
        invert64(a, xs, pt);
        {   // T as two bf16 terms in its own place: half a row each (row pt & 63), read by all first
            const int hf = pt >> 6;
            float4 u[8];
#pragma unroll
            for (int w = 0; w < 8; ++w)   // (the block above the diagonal holds nothing)
                u[w] = i >= 32 || hf == 0 ? quad(a + at(i, 32 * hf + 4 * w)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            __syncthreads();
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t hw[4], lw[4], tw[4];
                split3(pk2(u[2 * w].x, u[2 * w].y), hw[0], lw[0], tw[0]);
                split3(pk2(u[2 * w].z, u[2 * w].w), hw[1], lw[1], tw[1]);
                split3(pk2(u[2 * w + 1].x, u[2 * w + 1].y), hw[2], lw[2], tw[2]);
                split3(pk2(u[2 * w + 1].z, u[2 * w + 1].w), hw[3], lw[3], tw[3]);
                if (p.keep) put3(kRecT3, 4 * hf + w, tw);
                sts128(chunk_addr(base + kPrepT, i, 4 * hf + w), make_uint4(hw[0], hw[1], hw[2], hw[3]));
                sts128(chunk_addr(base + kPrepT + kTile, i, 4 * hf + w), make_uint4(lw[0], lw[1], lw[2], lw[3]));
            }
        }
        fence_proxy_async_smem();
        tc_fence_before();
    }
    __syncthreads();
    if (pt == 0) {
        if (!bad) {
            unsigned char* r = p.rec + (item * p.nchunks + c) * p.rec_bytes;
            bulk_store(r + kRecT, base + kPrepT, 2 * kTile);
            bulk_store(r + kRecP, base, 2 * kTile);
            bulk_store(r + kRecScal, base + kPrepScal, sizeof(Scal));
            if (p.keep) bulk_store(r + kRecLocal, base + kPrepLocal, sizeof(Local));
            tc::bulk_commit();
            bulk_wait0();
        } else {   // what is still in flight ends before the shared memory and the TMEM columns go
            mbar_wait_bounded(&ps.full, 0, p.drain_ns);
            if (issued) mbar_wait_bounded(&ps.gram, 0, p.drain_ns);
        }
    }
    __syncwarp();
    if (warp == 0) {
        tc_fence_after();
        tc::tmem_dealloc(tmem, kC);
    }
}

// ------------------------------------------------------------------------------------------------ chain
// The products run transposed: the 128 TMEM lanes are the rows v of the state, and the columns are tokens or keys.
//   KS, QS [v, i] = S Kᵀ, S Qᵀ      A: S (TMEM),  B: K and Q tiles in one, K-major
//   E   [v, i] = Vᵀ Tᵀ + X Tᵀ       A: V tile, MN-major; X = -KS diag(e^G / |k|) (TMEM),  B: T tile, K-major
//   dS  [v, k] = W K                A: W = E diag(β e^{G_end - G} / |k|) (TMEM),  B: K tile, MN-major
//   Yᵀ  [v, i] = QS diag(scale e^G / |q|) + E Pᵀ    off the chain, under the element-wise steps
// so that the state, the right hand side and the corrections go from registers to TMEM and never through shared
// memory, a thread owning one row v (four threads to a row, each with a quarter of the columns).  X is written over
// KS, E's terms over E, S's terms over dS, by the thread that read them, which is what makes it fit in TMEM.
// An MMA of 128 x N x 16 takes about 58 cycles for every N up to 128 (measured here; 100 where N changes from one to
// the next, as when the zero blocks of T and P are left out), so operands are put side by side to N = 128 where they
// share A: K with Q, T's two terms, P's two terms, and the reader adds the two halves of E and of Y.  The order of
// issue keeps the chain's products first: E's part from V follows KS, Y's follows dS, and S's terms are handed over
// in two halves, so that KS starts on the first.
//
// Warps: 0..15 state (above); 16 issues the MMAs; 17 the loads (two chunks in flight); 18 stores y.  They hand over
// through mbarriers.  Every wait is bounded: one that runs out records SS_ERR_TIMEOUT and the CTA winds down.
//
// Bound by that chain: 8 x 2048 tokens, 12 heads of 128 (96 CTAs of 32 chunks) 147 us, 4.5 us a chunk of which 1.8 us
// are products' time (tensor pipe 47 %); 160 items of 128 chunks with their segments 606 us.  (With S and X as two terms
// 121 and 520 us; 28 bytes of each thread's registers spill at the 96 that 19 warps leave.)  Half the state warps: 1738 us
// for what 1378 us then took.
constexpr int kParts = 4;              // threads to a row of the state
constexpr int kStateWarps = 4 * kParts;
constexpr int kMmaWarp = kStateWarps, kLoadWarp = kMmaWarp + 1, kStoreWarp = kMmaWarp + 2;
constexpr int kThreads = 32 * (kStoreWarp + 1);
constexpr int kTok = kC / kParts;      // tokens of a state thread
constexpr int kStages = 2;             // chunks in flight

// TMEM columns.  A: KS, then X's terms over it, then W's (W's third over QS); B: E in two halves, then its terms over the
// first, and the next state's third terms over the second; S: the state's terms (of each 16 keys, hi then lo), then X's
// third over them, then dS; Y: in two halves.
constexpr uint32_t kColS = 0, kColA = 128, kColQS = 192, kColB = 256, kColS3 = kColB + kC, kColY = 384;
constexpr uint32_t kTmemCols = 512;

// Shared memory: byte offsets from a 1024-aligned base.  A stage: [K 0][Q 0][K 1][Q 1][V 0][V 1][record]; then y
// [64][d_v] for its store.  Without y there is no Q and of the record only T (three terms, where it has them) and the
// factors, and what is kept is staged for its store: S's image, then E's three over it.
template <bool Y>
struct Smem {
    static constexpr uint32_t kPair = Y ? 2 * kTile : kTile;   // from K's first block of keys to its second
    static constexpr uint32_t kV = 2 * kPair, kRec = kV + 2 * kTile;
    static constexpr uint32_t kFactors = kRec + (Y ? kRecScal : 3 * kTile);
    static constexpr uint32_t kStage = kFactors + sizeof(Scal);
    static constexpr uint32_t kOut = kStages * kStage;
    static constexpr uint32_t kBar = kOut + (Y ? 2 : 8) * kTile;
    static constexpr uint32_t kBytes = kBar + 256 + 1024;
    static_assert(kStage % 1024 == 0 && kBytes <= 227 * 1024, "shared memory");
};

// 16 values' terms, two or three, to images in shared memory one behind another (128 rows of 128 bytes): the 16 columns
// from `col` < 64 on of row r.
template <bool THREE>
__device__ __forceinline__ void stage_terms(uint32_t img, int r, int col, const f32x2* v) {
    uint32_t t[3][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (THREE) split3(v[e], t[0][e], t[1][e], t[2][e]);
        else split2(v[e], t[0][e], t[1][e]);
    }
#pragma unroll
    for (int w = 0; w < (THREE ? 3 : 2); ++w)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            sts128(chunk_addr(img + w * 2 * kTile, r, (col >> 3) + h),
                   make_uint4(t[w][4 * h], t[w][4 * h + 1], t[w][4 * h + 2], t[w][4 * h + 3]));
}
// 16 values in fp32 to an image of 32-wide blocks of 128 rows.
__device__ __forceinline__ void stage_f32(uint32_t img, int r, int col, const f32x2* v) {
    const uint32_t blk = img + static_cast<uint32_t>(col >> 5) * 2 * kTile;
#pragma unroll
    for (int h = 0; h < 4; ++h)
        sts128(chunk_addr(blk, r, ((col & 31) >> 2) + h),
               make_uint4(__float_as_uint(v[2 * h].x), __float_as_uint(v[2 * h].y), __float_as_uint(v[2 * h + 1].x),
                          __float_as_uint(v[2 * h + 1].y)));
}

struct Bars {
    uint64_t full[kStages];    // K, Q, V and the record of a stage landed
    uint64_t empty[kStages];   // the chunk's last MMA is done with the stage
    uint64_t ks, e, ds, pv;    // the chain's products done
    uint64_t s_ready[2];       // S's terms written: of the first 16 keys of each thread, of the others (state warps)
    uint64_t x_ready, w_ready, e_ready;   // X's terms, W's, E's and Y's first part written (state warps)
    uint64_t y_full, y_free;   // y staged (state warps); stored (1).  Without y: a chunk's S, then its E
    uint64_t fin;              // wind-down
    uint32_t tmem;
};
static_assert(sizeof(Bars) <= 256, "barrier region");

// Y: CTAs 0 .. n_whole - 1 run the items 0 .. n_whole - 1 whole, the others a segment each, from the state that
// enters it.  Y false: there is no y, and with it no QS and no product with P.  With p.keep it is the backward pass's
// forward half, one CTA per item, and E and the entering state of every chunk are kept; else it is the state
// pass over the cut items' segments but the last.  A segment's end is S_in M + S_loc, row by row: S_loc is its end from
// a zero state, and M its end from the unit matrix without values, a run of its own (the segment 0 needs none).
template <int DK, bool Y>
__global__ void __launch_bounds__(kThreads, 1)
ss_gdr_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tm_q,
                 const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ CUtensorMap tm_y) {
    using M = Smem<Y>;
    constexpr int KB = DK / 64;       // 64-wide blocks of a K or Q row
    constexpr int KH = DK / kParts;   // keys of a state thread
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* gbase = smem_raw + (base - raw);
    Bars* const bar = reinterpret_cast<Bars*>(gbase + M::kBar);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const GdrParams& g = p.g;
    int item = blockIdx.x, sg = 0, nseg = 1;
    bool unit = false;                // a segment's map: from the unit matrix, without values
    if (!Y && !p.keep) {
        const int per = 2 * p.nseg - 3, x = item % per;
        item = p.n_whole + item / per;
        sg = x < p.nseg - 1 ? x : x - (p.nseg - 1) + 1;
        unit = x >= p.nseg - 1;
        nseg = p.nseg;
    } else if (Y && item >= p.n_whole) {
        const int x = item - p.n_whole;
        item = p.n_whole + x / p.nseg;
        sg = x % p.nseg;
        nseg = p.nseg;
    }
    const int b = item / g.H, h = item % g.H, hk = h / (g.H / g.Hk);
    const int rows = unit ? DK : p.dv;
    const int64_t len = gdr_len(g, b);
    const int64_t all = (len + kC - 1) / kC, c0 = static_cast<int64_t>(sg) * (nseg > 1 ? p.cseg : 0);
    const int nchunk = static_cast<int>(max(int64_t{0}, (nseg > 1 ? min(all - c0, static_cast<int64_t>(p.cseg)) : all)));
    const int cbase = static_cast<int>(c0);   // chunk c of this CTA is the sequence's cbase + c
    // the last chunk of a sequence that ends before the tensor does: other tokens follow in its tile
    const int ragged = (len % kC != 0 && len < g.L) ? static_cast<int>(all - 1 - c0) : -1;
    const uint64_t lim = p.wait_ns;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bar->full[i], 1);
            mbar_init(&bar->empty[i], 1);
        }
        uint64_t* one[] = {&bar->ks, &bar->e, &bar->ds, &bar->pv, &bar->y_free, &bar->fin};
        for (uint64_t* x : one) mbar_init(x, 1);
        uint64_t* all[] = {bar->s_ready, bar->s_ready + 1, &bar->x_ready, &bar->w_ready, &bar->e_ready, &bar->y_full};
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
    int issued = 0;   // loads of the load thread

    if (warp == kLoadWarp) {
        // ============================================================ loads (one thread)
        if (lane == 0) {
            tma_prefetch_desc(&tm_q);
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
            for (int c = 0; c < nchunk; ++c) {
                const int s = c % kStages;
                if (c >= kStages && !wait1(&bar->empty[s], ((c / kStages) - 1) & 1)) break;
                const uint32_t st = base + s * M::kStage;
                uint64_t* f = &bar->full[s];
                mbar_arrive_expect_tx(f, (Y ? 2 : 1) * KB * kTile + (unit ? 0 : kC * p.dv * 2) + (M::kStage - M::kRec) -
                                             (Y || p.keep ? 0 : kTile));
                const int t0 = (cbase + c) * kC;
                for (int kb = 0; kb < KB; ++kb) {
                    tma_load_4d(st + kb * M::kPair, &tm_k, 64 * kb, hk, t0, b, f);
                    if (Y) tma_load_4d(st + kb * M::kPair + kTile, &tm_q, 64 * kb, hk, t0, b, f);
                }
                for (int vb = 0; !unit && vb < p.dv / 64; ++vb)
                    tma_load_4d(st + M::kV + vb * kTile, &tm_v, 64 * vb, h, t0, b, f);
                const unsigned char* r = p.rec + (item * p.nchunks + cbase + c) * p.rec_bytes;
                if (Y) {
                    bulk_load(st + M::kRec, r, kRecBytes, f);
                } else {
                    bulk_load(st + M::kRec, r + kRecT, 2 * kTile, f);
                    if (p.keep) bulk_load(st + M::kRec + 2 * kTile, r + kRecT3, kTile, f);
                    bulk_load(st + M::kFactors, r + kRecScal, sizeof(Scal), f);
                }
                issued = c + 1;
            }
        }
        __syncwarp();
    } else if (warp == kStoreWarp) {
        // ============================================================ y, or what is kept
        for (int n = 0; !Y && p.keep && n < 2 * nchunk + 1; ++n) {   // S of chunk n / 2, then its E; at last the final state
            if (!wait_warp(&bar->y_full, n & 1)) break;
            if (lane == 0) {
                unsigned char* kp = p.keep + (item * (p.nchunks + 1) + (n >> 1)) * kKeepBytes;
                if (n & 1) bulk_store(kp + kKeepE, base + M::kOut, 6 * kTile);
                else bulk_store(kp + kKeepS, base + M::kOut, 4 * KB * kTile);
                tc::bulk_commit();
                tc::bulk_wait_read0();
            }
            arrive_warp(&bar->y_free);
        }
        for (int c = 0; Y && c < nchunk; ++c) {
            if (!wait_warp(&bar->y_full, c & 1)) break;
            if (c != ragged) {   // rows behind the tensor's end are clipped by the copy
                if (lane == 0) {
                    tc::tma_store_4d(&tm_y, base + M::kOut, 0, h, (cbase + c) * kC, b);
                    tc::bulk_commit();
                    tc::bulk_wait_read0();
                }
            } else {             // rows behind the sequence's end stay as they are
                const int64_t t0 = static_cast<int64_t>(cbase + c) * kC;
                const int quads = p.dv / 8, n = static_cast<int>(len - t0) * quads;
                __nv_bfloat16* y = static_cast<__nv_bfloat16*>(g.y);
                for (int i = lane; i < n; i += 32) {
                    const int r = i / quads, q = i % quads;
                    *reinterpret_cast<uint4*>(y + ((static_cast<int64_t>(b) * g.L + t0 + r) * g.H + h) * p.dv + 8 * q) =
                        lds128(base + M::kOut + (r * p.dv + 8 * q) * 2);
                }
            }
            arrive_warp(&bar->y_free);
        }
        if (lane == 0) bulk_wait0();
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ============================================================ MMAs (one thread)
        if (lane == 0) {
            const uint32_t vlbo = p.dv == 128 ? kTile : 0;   // d_v 64: the lanes 64.. repeat the rows 0..63
            for (int c = 0; c < nchunk; ++c) {
                const int s = c % kStages;
                const uint32_t par = c & 1, st = base + s * M::kStage, pr = st + M::kRec;
                if (!wait1(&bar->full[s], (c / kStages) & 1)) break;
                // KS and QS: S's terms of 16 keys in 16 columns, K and Q of a 64-key block side by side.  (The accumulator
                // is cut off, not rounded, after every product: of the keys at hand the small terms come first.)
                constexpr int kStep = KH / 16;   // (the rows behind a sequence's end are zeroed before s_ready)
                auto ks_steps = [&](int first) {
#pragma unroll
                    for (int w = 0; w < 3; ++w)
#pragma unroll
                        for (int ks = first; ks < DK / 16; ks += kStep)
                            umma_ts(tmem + kColA, tmem + (w == 0 ? kColS3 + 8 * ks : w == 1 ? kColS + 16 * ks + 8 : kColS + 16 * ks),
                                    sdesc(st + (ks >> 2) * M::kPair + (ks & 3) * 32, 16, 1024),
                                    idesc(Y ? 2 * kC : kC, false), first + w + ks > 0);
                };
                if (!wait1(&bar->s_ready[0], par)) break;
                tc_fence_after();
                ks_steps(0);
                if (!wait1(&bar->s_ready[1], par)) break;
                tc_fence_after();
                if (kStep == 2) ks_steps(1);
                if (!(p.test_drop && blockIdx.x == 0 && c == 0)) umma_commit(&bar->ks);
                // E = Vᵀ Tᵀ, T's terms side by side, once the last chunk's E and the state's third terms are read (X is
                // made meanwhile)
                if (!wait1(&bar->ks, par)) break;
                if (Y && c > 0 && !wait1(&bar->pv, (c - 1) & 1)) break;
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < (unit ? 0 : kC / 16); ++j)
                    umma(tmem + kColB, sdesc(st + M::kV + 2048u * j, vlbo, 1024), sdesc(pr + kRecT + 32u * j, 16, 1024),
                         idesc(2 * kC, false, true), j > 0);
                const bool t3 = !Y && p.keep;   // T's third term, into E's first half
                if (t3) {
#pragma unroll
                    for (int j = 0; j < kC / 16; ++j)
                        umma(tmem + kColB, sdesc(st + M::kV + 2048u * j, vlbo, 1024), sdesc(pr + 2 * kTile + 32u * j, 16, 1024),
                             idesc(kC, false, true), 1);
                }
                if (!wait1(&bar->x_ready, par)) break;
                tc_fence_after();
                // E += X Tᵀ
                if (t3) {
#pragma unroll
                    for (int j = 0; j < kC / 16; ++j)
                        umma_ts(tmem + kColB, tmem + kColA + 16 * j, sdesc(pr + 2 * kTile + 32u * j, 16, 1024), idesc(kC, false), 1);
                }
#pragma unroll
                for (int w = 0; w < 3; ++w)
#pragma unroll
                    for (int j = 0; j < kC / 16; ++j)
                        umma_ts(tmem + kColB, tmem + (w == 0 ? kColS + 8 * j : w == 1 ? kColA + 16 * j + 8 : kColA + 16 * j),
                                sdesc(pr + kRecT + 32u * j, 16, 1024), idesc(2 * kC, false), unit && w + j == 0 ? 0 : 1);
                umma_commit(&bar->e);
                if (!wait1(&bar->w_ready, par)) break;
                tc_fence_after();
                // dS = W K over the columns of S's terms, W's third terms (in QS's place) first
#pragma unroll
                for (int w = 0; w < 3; ++w)
#pragma unroll
                    for (int j = 0; j < kC / 16; ++j)
                        umma_ts(tmem + kColS, tmem + (w == 0 ? kColQS : w == 1 ? kColA + 8 : kColA) + 16 * j,
                                sdesc(st + 2048u * j, M::kPair, 1024), idesc(DK, true), w + j > 0);
                umma_commit(&bar->ds);
                if (Y) {   // Yᵀ += E Pᵀ
                    if (!wait1(&bar->e_ready, par)) break;
                    tc_fence_after();
#pragma unroll
                    for (int j = 0; j < kC / 16; ++j) {
                        const uint64_t bd = sdesc(pr + kRecP + 32u * j, 16, 1024);
                        umma_ts(tmem + kColY, tmem + kColB + 16 * j, bd, idesc(2 * kC, false), 1);
                        umma_ts(tmem + kColY, tmem + kColB + 16 * j + 8, bd, idesc(2 * kC, false), 1);
                    }
                    umma_commit(&bar->pv);
                }
                umma_commit(&bar->empty[s]);
            }
        }
        __syncwarp();
    } else {
        // ============================================================ state warps
        const int v = (warp & 3) * 32 + lane, part = warp >> 2;
        const bool row_in = v < rows;
        const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const int64_t srow = (static_cast<int64_t>(item) * p.dv + v) * DK + part * KH;
        // the entering state: the call's, a segment's, zero or the unit matrix; and where the leaving one goes
        const int64_t cut = static_cast<int64_t>(item - p.n_whole) * (p.nseg - 1);
        const int64_t first = (static_cast<int64_t>(item - p.n_whole) * p.dv + v) * DK + part * KH;
        const float* from = sg == 0 ? (!g.h_init ? nullptr : Y && nseg > 1 ? p.seg_first + first : g.h_init + srow)
                          : Y       ? p.seg_in + ((cut + sg - 1) * p.dv + v) * DK + part * KH : nullptr;
        float* to = nullptr;
        if (!Y && !p.keep) to = unit ? p.seg_map + ((cut + sg) * DK + v) * DK + part * KH : p.seg_loc + ((cut + sg) * p.dv + v) * DK + part * KH;
        else if (g.final_state && sg == nseg - 1) to = g.final_state + srow;
        f32x2 S[KH / 2];
#pragma unroll
        for (int k = 0; k < KH; k += 4) {
            float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (from && row_in) q = quad(from + k);
            if (!Y && nseg > 1 && from && row_in) *reinterpret_cast<float4*>(p.seg_first + first + k) = q;
            if (unit) {
                const int d = v - (part * KH + k);
                q = make_float4(d == 0, d == 1, d == 2, d == 3);
            }
            S[k / 2] = pk2(q.x, q.y);
            S[k / 2 + 1] = pk2(q.z, q.w);
        }
#pragma unroll
        for (int k = 0; k < KH; k += 16)
            store_terms3(tl + kColS + part * KH + k, tl + kColS3 + (part * KH + k) / 2, S + k / 2);
        tmem_wait_st();
        tc_fence_before();
        // the state that enters chunk c, and its E's terms (without y); the stores are one behind another
        auto keep_state = [&](int c) {
            if (c > 0 && !wait_warp(&bar->y_free, 1)) return false;   // chunk c - 1's E, store 2 c - 1
#pragma unroll
            for (int k = 0; k < KH; k += 16)
                stage_f32(base + M::kOut, v, part * KH + k, S + k / 2);
            fence_proxy_async_smem();
            arrive_warp(&bar->y_full);
            return true;
        };
        auto finish_y = [&](int c) {     // chunk c's y
            if (c > 0 && !wait_warp(&bar->y_free, (c - 1) & 1)) return false;
            if (!wait_warp(&bar->pv, c & 1)) return false;
            tc_fence_after();
            f32x2 x[8], w[8];
            tmem_ld16x2(tl + kColY + kTok * part, tl + kColY + kC + kTok * part, x, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = add2(x[e], w[e]);
            __nv_bfloat16* ys = reinterpret_cast<__nv_bfloat16*>(gbase + M::kOut) + kTok * part * p.dv + v;
            if (row_in) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ys[2 * e * p.dv] = __float2bfloat16_rn(x[e].x);
                    ys[(2 * e + 1) * p.dv] = __float2bfloat16_rn(x[e].y);
                }
            }
            fence_proxy_async_smem();
            arrive_warp(&bar->y_full);
            return true;
        };
        bool ok = true;
        for (int c = 0; c < nchunk; ++c) {
            const int s = c % kStages;
            const uint32_t par = c & 1, st = base + s * M::kStage;
            const Scal& sc = *reinterpret_cast<const Scal*>(gbase + s * M::kStage + M::kFactors);
            if (c == ragged) {   // rows of K and V behind the end, whatever they hold, become zero rows
                ok = wait_warp(&bar->full[s], (c / kStages) & 1);
                if (!ok) break;
                const int n0 = static_cast<int>(len - static_cast<int64_t>(cbase + c) * kC);
                for (int i = n0 * 8 + tid; i < kC * 8; i += 32 * kStateWarps) {
                    for (int kb = 0; kb < KB; ++kb) sts128(st + kb * M::kPair + 16 * i, make_uint4(0, 0, 0, 0));
                    for (int vb = 0; !unit && vb < p.dv / 64; ++vb) sts128(st + M::kV + vb * kTile + 16 * i, make_uint4(0, 0, 0, 0));
                }
                fence_proxy_async_smem();
            }
            if (c == 0 || c == ragged) {   // (else: handed over below)
                arrive_warp(&bar->s_ready[0]);
                arrive_warp(&bar->s_ready[1]);
            }
            if (!Y && p.keep) {
                ok = keep_state(c);
                if (!ok) break;
            }
            if (Y && c > 0) {   // the last chunk's y, while this one's K Sᵀ runs
                ok = finish_y(c - 1);
                if (!ok) break;
            }
            ok = wait_warp(&bar->full[s], (c / kStages) & 1) && wait_warp(&bar->ks, par);
            if (!ok) break;
            tc_fence_after();
            f32x2 x[8];
            tmem_ld16(tl + kColA + kTok * part, x);   // X, the factors' sign with it
            scale16(x, sc.ek + kTok * part);
            store_terms3(tl + kColA + kTok * part, tl + kColS + 8 * part, x);
            tmem_wait_st();
            tc_fence_before();
            arrive_warp(&bar->x_ready);
            if (Y) {   // y's part from the entering state, while E is multiplied
                const uint32_t zero[8] = {};
                tmem_ld16(tl + kColQS + kTok * part, x);
                scale16(x, sc.qe + kTok * part);
                tmem_st16(tl + kColY + kTok * part, x);
                tmem_st8(tl + kColY + kC + kTok * part, zero);
                tmem_st8(tl + kColY + kC + kTok * part + 8, zero);
            }
            ok = wait_warp(&bar->e, par);
            if (!ok) break;
            tc_fence_after();
            {
                f32x2 w[8];
                tmem_ld16x2(tl + kColB + kTok * part, tl + kColB + kC + kTok * part, x, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = add2(x[e], w[e]);
            }
            {
                f32x2 w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = x[e];
                scale16(w, sc.wk + kTok * part);
                store_terms3(tl + kColA + kTok * part, tl + kColQS + kTok * part, w);
            }
            const float end = sc.end[0];
            tmem_wait_st();
            tc_fence_before();
            arrive_warp(&bar->w_ready);
            if (Y) {
                store_terms(tl + kColB + kTok * part, x);
                tmem_wait_st();
                tc_fence_before();
                arrive_warp(&bar->e_ready);
            } else if (p.keep) {
                ok = wait_warp(&bar->y_free, 0);   // its S, store 2 c
                if (!ok) break;
                stage_terms<true>(base + M::kOut, v, kTok * part, x);
                fence_proxy_async_smem();
                arrive_warp(&bar->y_full);
            }
            ok = wait_warp(&bar->ds, par);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < KH; k += 16) {
                tmem_ld16(tl + kColS + part * KH + k, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) S[k / 2 + e] = fma2(pk2(end, end), S[k / 2 + e], x[e]);
                store_terms3(tl + kColS + part * KH + k, tl + kColS3 + (part * KH + k) / 2, S + k / 2);
                if (c + 1 != ragged && c + 1 < nchunk) {
                    tmem_wait_st();
                    tc_fence_before();
                    arrive_warp(&bar->s_ready[k / 16]);
                    if (KH == 16) arrive_warp(&bar->s_ready[1]);
                }
            }
            tmem_wait_st();
            tc_fence_before();
        }
        if (Y && ok && nchunk > 0) ok = finish_y(nchunk - 1);
        if (!Y && p.keep && ok) ok = keep_state(nchunk);
        if (ok && to && row_in) {
#pragma unroll
            for (int k = 0; k < KH; k += 4)
                *reinterpret_cast<float4*>(to + k) =
                    make_float4(S[k / 2].x, S[k / 2].y, S[k / 2 + 1].x, S[k / 2 + 1].y);
        }
        tc_fence_before();
    }

    // Wind-down: loads in flight land before the shared memory goes, MMAs end before the TMEM columns do.
    __syncthreads();
    if (warp == kLoadWarp && lane == 0) {
        for (int c = issued > kStages ? issued - kStages : 0; c < issued; ++c)
            mbar_wait_bounded(&bar->full[c % kStages], (c / kStages) & 1, p.drain_ns);
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

// The states that enter the segments 1 .. nseg - 1 of the cut items: S_in(1) is the end of segment 0, and
// S_in(s + 1) = S_in(s) M_s + S_loc(s), in fp32.  A chain over the segments, so the next map is copied to shared memory
// under the product with this one; a thread has two rows of four keys, a warp whole rows.  16 items of 9 segments, 128 x
// 128: 28 us, the maps' 64 KB per block and step from L2.
template <int DK>
struct FoldSmem {
    static constexpr int kRows = 8 * 2 * (128 / DK);   // rows of S per block of 256 threads
    alignas(128) float map[2][DK * DK];
    float row[kRows][DK];
    uint64_t full[2];
};
template <int DK>
__global__ void __launch_bounds__(256) ss_gdr_fold_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    FoldSmem<DK>& sm = *reinterpret_cast<FoldSmem<DK>*>(smem_raw);
    constexpr int Q = DK / 4;   // quads of a row
    const int64_t it = static_cast<int64_t>(blockIdx.x) * (p.nseg - 1);
    const int lane = threadIdx.x & 31, c = (lane % Q) * 4;
    const int r0 = ((threadIdx.x >> 5) * (32 / Q) + lane / Q) * 2;   // rows r0, r0 + 1 of the block
    const int64_t v0 = static_cast<int64_t>(blockIdx.y) * FoldSmem<DK>::kRows + r0;
    constexpr uint32_t bytes = DK * DK * sizeof(float);
    if (threadIdx.x == 0) {
        mbar_init(&sm.full[0], 1);
        mbar_init(&sm.full[1], 1);
        fence_mbar_init();
    }
    __syncthreads();
    auto fetch = [&](int seg) {
        if (threadIdx.x != 0 || seg >= p.nseg - 1) return;
        mbar_arrive_expect_tx(&sm.full[seg & 1], bytes);
        bulk_load(smem_u32(sm.map[seg & 1]), p.seg_map + (it + seg) * DK * DK, bytes, &sm.full[seg & 1]);
    };
    fetch(1);
    fetch(2);
    auto at_state = [&](float* base, int seg, int r) { return base + ((it + seg) * p.dv + v0 + r) * DK + c; };
    f32x2 s[2][2];
    auto load_loc = [&](int seg) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float4 q = quad(at_state(p.seg_loc, seg, r));
            s[r][0] = pk2(q.x, q.y);
            s[r][1] = pk2(q.z, q.w);
        }
    };
    auto store_in = [&](int seg) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
            *reinterpret_cast<float4*>(at_state(p.seg_in, seg, r)) = make_float4(s[r][0].x, s[r][0].y, s[r][1].x, s[r][1].y);
    };
    load_loc(0);
    store_in(0);
    for (int seg = 1; seg < p.nseg - 1; ++seg) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
            *reinterpret_cast<float4*>(&sm.row[r0 + r][c]) = make_float4(s[r][0].x, s[r][0].y, s[r][1].x, s[r][1].y);
        load_loc(seg);
        __syncwarp();   // (a row is one warp's)
        // (segments seg use buffer seg & 1 from 1 on: buffer 1 first, in its phase 0)
        const bool got = mbar_wait_bounded(&sm.full[seg & 1], ((seg - 1) >> 1) & 1, p.wait_ns);
        if (!got && threadIdx.x == 0 && p.status) atomicCAS(p.status, 0u, static_cast<uint32_t>(SS_ERR_TIMEOUT));
        const float* m = sm.map[seg & 1] + c;
#pragma unroll 4
        for (int k = 0; k < DK; k += 4) {
            const float4 a = quad(&sm.row[r0][k]), b = quad(&sm.row[r0 + 1][k]);
            const float aa[4] = {a.x, a.y, a.z, a.w}, bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 q = quad(m + (k + e) * DK);
                axpy4(s[0], aa[e], q);
                axpy4(s[1], bb[e], q);
            }
        }
        store_in(seg);
        __syncthreads();   // the map is read
        fetch(seg + 2);
    }
    // what is still in flight lands before the shared memory goes (after a wait that ran out)
    if (threadIdx.x == 0)
        for (int seg = max(1, p.nseg - 3); seg < p.nseg - 1; ++seg)
            mbar_wait_bounded(&sm.full[seg & 1], ((seg - 1) >> 1) & 1, p.drain_ns);
}

}  // namespace gdr
}  // namespace selscan
