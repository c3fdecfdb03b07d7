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
// operations), so a thread first loads all its rows and then computes: 10240 heads of 128 x 128 in 206 us, 6.5 TB/s.
// A sequence is bound by a token's latency, 0.7 us at 12 items (no loads ahead: the tokens' vectors come from L1 and L2).
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

// Grid: x = (b, h) items times blocks of kGdrRecRows * R rows of S.
template <typename IO, int DK, int R>
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
        float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            kk = fmaf(k[m].x, k[m].x, fmaf(k[m].y, k[m].y, fmaf(k[m].z, k[m].z, fmaf(k[m].w, k[m].w, kk))));
            qq = fmaf(q[m].x, q[m].x, fmaf(q[m].y, q[m].y, fmaf(q[m].z, q[m].z, fmaf(q[m].w, q[m].w, qq))));
            kq = fmaf(k[m].x, q[m].x, fmaf(k[m].y, q[m].y, fmaf(k[m].z, q[m].z, fmaf(k[m].w, q[m].w, kq))));
        }
        kk = sum8(kk);
        qq = sum8(qq);
        kq = sum8(kq);
        // the lengths enter as factors of the products, not of the vectors
        const float rk = p.l2norm ? 1.0f / sqrtf(kk + kGdrL2Eps) : 1.0f;
        const float rq = p.scale * (p.l2norm ? 1.0f / sqrtf(qq + kGdrL2Eps) : 1.0f);
        float dk_[R], dq[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float a = 0.0f, c = 0.0f;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                a = fmaf(S[r][m].x, k[m].x, fmaf(S[r][m].y, k[m].y, fmaf(S[r][m].z, k[m].z, fmaf(S[r][m].w, k[m].w, a))));
                c = fmaf(S[r][m].x, q[m].x, fmaf(S[r][m].y, q[m].y, fmaf(S[r][m].z, q[m].z, fmaf(S[r][m].w, q[m].w, c))));
            }
            dk_[r] = a;
            dq[r] = c;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            dk_[r] = sum8(dk_[r]);
            dq[r] = sum8(dq[r]);
        }
        IO* yp = static_cast<IO*>(p.y) + (tok * p.H + h) * dv + r0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float w = be * rk * fmaf(-al * rk, dk_[r], v[r]);   // β e |k|^-1
            if (l == 0) yp[r * kGdrRecRows] = from_f32<IO>(rq * fmaf(al, dq[r], kq * w));
#pragma unroll
            for (int m = 0; m < M; ++m) {
                S[r][m].x = fmaf(w, k[m].x, al * S[r][m].x);
                S[r][m].y = fmaf(w, k[m].y, al * S[r][m].y);
                S[r][m].z = fmaf(w, k[m].z, al * S[r][m].z);
                S[r][m].w = fmaf(w, k[m].w, al * S[r][m].w);
            }
        }
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
