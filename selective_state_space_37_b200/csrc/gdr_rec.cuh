// gdr_rec.cuh -- the gated delta rule token by token (sm_100a): the decode step, and sequences in fp32
// or too short for the chunked kernel.
//
// Per (b, value head h), with k̂, q̂ the (optionally unit-length) key and query, α = exp(Δ A_h):
//   e = v - α S k̂,   S <- α S + β e k̂ᵀ,   y = scale S q̂          (S is d_v x d_k, fp32)
// The rows of S do not meet: row r needs only S[r, :], k̂, q̂ and v_r.  Both products are therefore taken
// on the state that enters the token, in one pass over the registers that hold it:
//   y_r = scale (α S[r,:]·q̂ + (k̂·q̂) β e_r)
// Eight lanes share a row, each with the 16-byte quads l, l + 8, ... of it, so that a warp's accesses are
// whole 128-byte lines and a dot product ends after three shuffles.
// The decode step is bound by HBM (the fp32 state read and written: 8 d_k d_v bytes a head against 6 d_k d_v
// operations), so a thread first loads all its rows and then computes.
#pragma once

#include "common.cuh"

namespace selscan {

constexpr int kGdrRecThreads = 128;
constexpr int kGdrRecRows = kGdrRecThreads / 8;   // rows of S that a block holds per row of a thread
constexpr float kGdrL2Eps = 1e-6f;

struct GdrParams {
    const void* q;           // [batch, L, Hk, d_k]
    const void* k;
    const void* v;           // [batch, L, H, d_v]
    const void* dt;          // [batch, L, H]
    const void* beta;
    const float* dt_bias;    // [H] or null
    const float* A;          // [H]
    const float* h_init;     // [batch, H, d_v, d_k] or null
    const int32_t* seqlens;  // [batch] or null
    void* y;                 // [batch, L, H, d_v]
    float* final_state;      // [batch, H, d_v, d_k] or null
    int64_t L;
    int batch, H, Hk;
    float scale;
    int softplus, sigmoid, l2norm;
};

// Δ, and β, of one token in full precision (a few per token and head: their cost does not show).
__device__ __forceinline__ float gdr_delta(float raw, float bias, int softplus) {
    const float x = raw + bias;
    return softplus ? softplus_accurate(x) : x;
}
__device__ __forceinline__ float gdr_beta(float raw, int sigmoid) {
    return sigmoid ? 1.0f / (1.0f + expf(-raw)) : raw;
}
__device__ __forceinline__ int64_t gdr_len(const GdrParams& p, int b) {
    if (!p.seqlens) return p.L;
    const int64_t n = p.seqlens[b];
    return n < 0 ? 0 : (n > p.L ? p.L : n);
}

template <typename IO>
__device__ __forceinline__ float4 load4(const IO* p);
template <>
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <>
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}

__device__ __forceinline__ float sum8(float v) {   // over the eight lanes of a row
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    v += __shfl_xor_sync(0xffffffffu, v, 2);
    return v + __shfl_xor_sync(0xffffffffu, v, 4);
}

// Grid: x = (b, h) items times blocks of kGdrRecRows * R rows of S.  SEQ: more than one token; a step without the loop
// takes fewer registers, and more blocks are in flight (10240 heads of 128 x 128: 198 us, 6.8 TB/s, against 206 in bf16,
// 201 against 234 in fp32).  Bound by HBM there, by a token's latency in a sequence: the sums over a row's lanes
// run side by side (one after the other: 256 fp32 tokens of 12 items 185 against 172 us, of 768 items 1653 against 1375;
// with the next token loaded and made ready under this one 184 and 1963).
template <typename IO, int DK, int R, bool SEQ>
__global__ void __launch_bounds__(kGdrRecThreads) ss_gdr_rec_kernel(const GdrParams p, int dv, int row_blocks) {
    constexpr int M = DK / 32;   // float4 quads of a row per lane
    const int item = blockIdx.x / row_blocks, rb = blockIdx.x % row_blocks;
    const int b = item / p.H, h = item % p.H;
    const int hk = h / (p.H / p.Hk);
    const int l = threadIdx.x & 7, r0 = rb * kGdrRecRows * R + (threadIdx.x >> 3);
    const int64_t n = gdr_len(p, b);
    const int64_t srow = (static_cast<int64_t>(item) * dv + r0) * DK + 4 * l;
    float4 S[R][M];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int m = 0; m < M; ++m)
            S[r][m] = p.h_init ? *reinterpret_cast<const float4*>(p.h_init + srow + r * kGdrRecRows * DK + 32 * m)
                               : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
    for (int64_t t = 0; t < n; ++t) {
        const int64_t tok = static_cast<int64_t>(b) * p.L + t;
        const IO* kp = static_cast<const IO*>(p.k) + (tok * p.Hk + hk) * DK + 4 * l;
        const IO* qp = static_cast<const IO*>(p.q) + (tok * p.Hk + hk) * DK + 4 * l;
        const IO* vp = static_cast<const IO*>(p.v) + (tok * p.H + h) * dv + r0;
        float4 k[M], q[M];
#pragma unroll
        for (int m = 0; m < M; ++m) {
            k[m] = load4(kp + 32 * m);
            q[m] = load4(qp + 32 * m);
        }
        float v[R];
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] = to_f32(vp[r * kGdrRecRows]);
        const float dt = gdr_delta(to_f32(static_cast<const IO*>(p.dt)[tok * p.H + h]), bias, p.softplus);
        const float be = gdr_beta(to_f32(static_cast<const IO*>(p.beta)[tok * p.H + h]), p.sigmoid);
        const float al = expf(dt * A);
        // all sums side by side: the lengths enter as factors of the products, not of the vectors
        float kk = 0.0f, qq = 0.0f, kq = 0.0f, sk[R], sq[R];
#pragma unroll
        for (int m = 0; m < M; ++m) {
            kk = fmaf(k[m].x, k[m].x, fmaf(k[m].y, k[m].y, fmaf(k[m].z, k[m].z, fmaf(k[m].w, k[m].w, kk))));
            qq = fmaf(q[m].x, q[m].x, fmaf(q[m].y, q[m].y, fmaf(q[m].z, q[m].z, fmaf(q[m].w, q[m].w, qq))));
            kq = fmaf(k[m].x, q[m].x, fmaf(k[m].y, q[m].y, fmaf(k[m].z, q[m].z, fmaf(k[m].w, q[m].w, kq))));
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            sk[r] = sq[r] = 0.0f;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const float4 s = S[r][m];
                sk[r] = fmaf(s.x, k[m].x, fmaf(s.y, k[m].y, fmaf(s.z, k[m].z, fmaf(s.w, k[m].w, sk[r]))));
                sq[r] = fmaf(s.x, q[m].x, fmaf(s.y, q[m].y, fmaf(s.z, q[m].z, fmaf(s.w, q[m].w, sq[r]))));
            }
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            kk += __shfl_xor_sync(0xffffffffu, kk, o);
            qq += __shfl_xor_sync(0xffffffffu, qq, o);
            kq += __shfl_xor_sync(0xffffffffu, kq, o);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                sk[r] += __shfl_xor_sync(0xffffffffu, sk[r], o);
                sq[r] += __shfl_xor_sync(0xffffffffu, sq[r], o);
            }
        }
        const float rk = p.l2norm ? 1.0f / sqrtf(kk + kGdrL2Eps) : 1.0f;
        const float rq = p.scale * (p.l2norm ? 1.0f / sqrtf(qq + kGdrL2Eps) : 1.0f);
        IO* yp = static_cast<IO*>(p.y) + (tok * p.H + h) * dv + r0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float w = be * rk * fmaf(-al * rk, sk[r], v[r]);   // β e / |k|
            if (l == 0) yp[r * kGdrRecRows] = from_f32<IO>(rq * fmaf(al, sq[r], kq * w));
#pragma unroll
            for (int m = 0; m < M; ++m) {
                S[r][m].x = fmaf(w, k[m].x, al * S[r][m].x);
                S[r][m].y = fmaf(w, k[m].y, al * S[r][m].y);
                S[r][m].z = fmaf(w, k[m].z, al * S[r][m].z);
                S[r][m].w = fmaf(w, k[m].w, al * S[r][m].w);
            }
        }
        if (!SEQ) break;
    }
    if (p.final_state) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int m = 0; m < M; ++m)
                *reinterpret_cast<float4*>(p.final_state + srow + r * kGdrRecRows * DK + 32 * m) = S[r][m];
    }
}

}  // namespace selscan
