// gdr_rec_bwd.cuh -- the gated delta rule's backward pass token by token (sm_100a): fp32, and short bf16 sequences.
//
// With S_t the state behind token t, g = dJ/dy_t and dS the adjoint of S_t, in reverse over t:
//   dS += scale g q̂ᵀ,   dq̂ = scale S_tᵀ g,   s = dS k̂,   de = β s (v's gradient),   dβ = s·e
//   dk̂ = β dSᵀ e - (α S_t-1)ᵀ de,   dS -= de k̂ᵀ,   dlog α = <dS, α S_t-1>,   dS *= α
// As in the forward (gdr_rec.cuh) the rows of S and dS do not meet: a row's eight lanes hold both.  What runs over rows
// (dq̂, dk̂ and the gates) is added over the 16 rows of a block, left in the workspace per block, and added over the
// blocks, and over the value heads of a key head, by ss_gdr_rec_fold_kernel in a fixed order.
// S_t-1 cannot be had from S_t (α may be small): a forward run keeps e of every token and S before every kRecSeg-th;
// the reverse run repeats a segment's states from there, which needs no products, and holds them in shared memory,
// every thread its own values.
// Bound by a token's latency (loads, three sums over eight lanes, the sums over rows and one barrier): d_k = d_v = 128 in
// fp32, both runs together 2.3 us a token with 2 items, 6.7 us with 96 (768 blocks, three resident per SM).
#pragma once

#include "gdr_rec.cuh"

namespace selscan {

constexpr int kRecSeg = 8;   // tokens of a segment: 64 KB of states per block at d_k = 128, three resident blocks

struct GdrRecBwd {
    GdrParams g;
    const void* dy;
    const float* dfinal;     // or null
    float* dinit;            // or null
    void *dq, *dk, *dv, *ddt, *dbeta;
    float* keep_s;           // [items][ceil(L / kRecSeg)][d_v][d_k]
    float* keep_e;           // [items][L][d_v]
    float* sums;             // [items][d_v / 16][L][2 d_k + 4]: dq̂, dk̂, dβ, dlog α (two unused) of a block's rows
    float* part;             // [items][2]
};

// The forward run: e and the states that the reverse run starts its segments from.
template <typename IO, int DK>
__global__ void __launch_bounds__(kGdrRecThreads) ss_gdr_rec_keep_kernel(const GdrRecBwd p, int dv, int row_blocks) {
    constexpr int M = DK / 32;
    const GdrParams& g = p.g;
    const int item = blockIdx.x / row_blocks, rb = blockIdx.x % row_blocks;
    const int b = item / g.H, h = item % g.H, hk = h / (g.H / g.Hk);
    const int l = threadIdx.x & 7, row = rb * kGdrRecRows + (threadIdx.x >> 3);
    const int64_t n = gdr_len(g, b), segs = (g.L + kRecSeg - 1) / kRecSeg;
    float4 S[M];
#pragma unroll
    for (int m = 0; m < M; ++m)
        S[m] = g.h_init ? *reinterpret_cast<const float4*>(g.h_init + (static_cast<int64_t>(item) * dv + row) * DK + 4 * l + 32 * m)
                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float A = g.A[h], bias = g.dt_bias ? g.dt_bias[h] : 0.0f;
    for (int64_t t = 0; t < n; ++t) {
        if (t % kRecSeg == 0) {
            float* to = p.keep_s + ((item * segs + t / kRecSeg) * dv + row) * DK + 4 * l;
#pragma unroll
            for (int m = 0; m < M; ++m) *reinterpret_cast<float4*>(to + 32 * m) = S[m];
        }
        const int64_t tok = static_cast<int64_t>(b) * g.L + t;
        const IO* kp = static_cast<const IO*>(g.k) + (tok * g.Hk + hk) * DK + 4 * l;
        float4 k[M];
#pragma unroll
        for (int m = 0; m < M; ++m) k[m] = load4(kp + 32 * m);
        const float v = to_f32(static_cast<const IO*>(g.v)[(tok * g.H + h) * dv + row]);
        const float al = expf(gdr_delta(to_f32(static_cast<const IO*>(g.dt)[tok * g.H + h]), bias, g.softplus) * A);
        const float be = gdr_beta(to_f32(static_cast<const IO*>(g.beta)[tok * g.H + h]), g.sigmoid);
        float kk = 0.0f, a = 0.0f;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            kk = fmaf(k[m].x, k[m].x, fmaf(k[m].y, k[m].y, fmaf(k[m].z, k[m].z, fmaf(k[m].w, k[m].w, kk))));
            a = fmaf(S[m].x, k[m].x, fmaf(S[m].y, k[m].y, fmaf(S[m].z, k[m].z, fmaf(S[m].w, k[m].w, a))));
        }
        kk = sum8(kk);
        const float rk = g.l2norm ? 1.0f / sqrtf(kk + kGdrL2Eps) : 1.0f;
        const float e = fmaf(-al * rk, sum8(a), v), w = be * rk * e;
        if (l == 0) p.keep_e[(item * g.L + t) * dv + row] = e;
#pragma unroll
        for (int m = 0; m < M; ++m)
            S[m] = make_float4(fmaf(w, k[m].x, al * S[m].x), fmaf(w, k[m].y, al * S[m].y), fmaf(w, k[m].z, al * S[m].z),
                               fmaf(w, k[m].w, al * S[m].w));
    }
}

// The reverse run.  Grid as above.
template <typename IO, int DK>
__global__ void __launch_bounds__(kGdrRecThreads) ss_gdr_rec_rev_kernel(const GdrRecBwd p, int dv, int row_blocks) {
    constexpr int M = DK / 32, kWarps = kGdrRecThreads / 32, kSum = 2 * DK + 4;
    extern __shared__ float4 held[];                 // [kRecSeg][M][threads]: S before each token of the segment
    __shared__ float red[2][kWarps][kSum];           // a token's sums over each warp's rows, in two buffers
    __shared__ float4 gate[kWarps][kRecSeg];         // α, β, 1 / |k|, scale / |q|: every warp its own
    const GdrParams& g = p.g;
    const int item = blockIdx.x / row_blocks, rb = blockIdx.x % row_blocks;
    const int b = item / g.H, h = item % g.H, hk = h / (g.H / g.Hk);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = tid & 7, row = rb * kGdrRecRows + (tid >> 3);
    const int64_t n = gdr_len(g, b), segs = (g.L + kRecSeg - 1) / kRecSeg;
    const int64_t srow = (static_cast<int64_t>(item) * dv + row) * DK + 4 * l;
    float4 S[M], dS[M];
#pragma unroll
    for (int m = 0; m < M; ++m)
        dS[m] = p.dfinal ? *reinterpret_cast<const float4*>(p.dfinal + srow + 32 * m) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float A = g.A[h], bias = g.dt_bias ? g.dt_bias[h] : 0.0f;
    auto vec = [&](const void* base, int64_t tok, float4 (&x)[M]) {
        const IO* x0 = static_cast<const IO*>(base) + (tok * g.Hk + hk) * DK + 4 * l;
#pragma unroll
        for (int m = 0; m < M; ++m) x[m] = load4(x0 + 32 * m);
    };
    auto dot = [](const float4 (&x)[M], const float4 (&y)[M]) {
        float s = 0.0f;
#pragma unroll
        for (int m = 0; m < M; ++m)
            s = fmaf(x[m].x, y[m].x, fmaf(x[m].y, y[m].y, fmaf(x[m].z, y[m].z, fmaf(x[m].w, y[m].w, s))));
        return s;
    };
    auto axpy = [](float a, const float4& x, const float4& y) {
        return make_float4(fmaf(a, x.x, y.x), fmaf(a, x.y, y.y), fmaf(a, x.z, y.z), fmaf(a, x.w, y.w));
    };
    auto times = [](float a, const float4& x) { return make_float4(a * x.x, a * x.y, a * x.z, a * x.w); };
    // over the four rows of a warp: the lanes with the same l
    auto rows4 = [](float x) {
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        return x + __shfl_xor_sync(0xffffffffu, x, 16);
    };
    int buf = 0;
    for (int64_t sg = (n + kRecSeg - 1) / kRecSeg - 1; sg >= 0; --sg) {
        const int64_t t0 = sg * kRecSeg;
        const int cnt = static_cast<int>(n - t0 < kRecSeg ? n - t0 : kRecSeg);
        const float* from = p.keep_s + ((item * segs + sg) * dv + row) * DK + 4 * l;
#pragma unroll
        for (int m = 0; m < M; ++m) S[m] = *reinterpret_cast<const float4*>(from + 32 * m);
        for (int j = 0; j < cnt; ++j) {
            const int64_t tok = static_cast<int64_t>(b) * g.L + t0 + j;
            float4 k[M], q[M];
            vec(g.k, tok, k);
            vec(g.q, tok, q);
            const float al = expf(gdr_delta(to_f32(static_cast<const IO*>(g.dt)[tok * g.H + h]), bias, g.softplus) * A);
            const float be = gdr_beta(to_f32(static_cast<const IO*>(g.beta)[tok * g.H + h]), g.sigmoid);
            const float kk = sum8(dot(k, k)), qq = sum8(dot(q, q));
            const float rk = g.l2norm ? 1.0f / sqrtf(kk + kGdrL2Eps) : 1.0f;
            const float rq = g.scale * (g.l2norm ? 1.0f / sqrtf(qq + kGdrL2Eps) : 1.0f);
            if (lane == 0) gate[warp][j] = make_float4(al, be, rk, rq);
            const float w = be * rk * p.keep_e[(item * g.L + t0 + j) * dv + row];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                held[(j * M + m) * kGdrRecThreads + tid] = S[m];
                S[m] = axpy(w, k[m], times(al, S[m]));
            }
        }
        __syncwarp();
        for (int j = cnt - 1; j >= 0; --j) {
            const int64_t t = t0 + j, tok = static_cast<int64_t>(b) * g.L + t;
            float4 k[M], q[M];
            vec(g.k, tok, k);
            vec(g.q, tok, q);
            const float4 f = gate[warp][j];
            const float al = f.x, be = f.y, rk = f.z, rq = f.w;
            const float gy = to_f32(static_cast<const IO*>(p.dy)[(tok * g.H + h) * dv + row]);
            const float e = p.keep_e[(item * g.L + t) * dv + row];
            float* r = red[buf][warp];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                dS[m] = axpy(gy * rq, q[m], dS[m]);
                const float4 x = times(gy, S[m]);
                const float4 s = make_float4(rows4(x.x), rows4(x.y), rows4(x.z), rows4(x.w));
                if (lane < 8) *reinterpret_cast<float4*>(r + 4 * l + 32 * m) = s;
            }
            const float s = rk * sum8(dot(dS, k)), de = be * s;
            float dla = 0.0f;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                S[m] = held[(j * M + m) * kGdrRecThreads + tid];
                const float4 Sd = times(al, S[m]);
                const float4 x = axpy(-de, Sd, times(be * e, dS[m]));
                const float4 y = make_float4(rows4(x.x), rows4(x.y), rows4(x.z), rows4(x.w));
                if (lane < 8) *reinterpret_cast<float4*>(r + DK + 4 * l + 32 * m) = y;
                dS[m] = axpy(-de * rk, k[m], dS[m]);
                dla = fmaf(dS[m].x, Sd.x, fmaf(dS[m].y, Sd.y, fmaf(dS[m].z, Sd.z, fmaf(dS[m].w, Sd.w, dla))));
                dS[m] = times(al, dS[m]);
            }
            dla = rows4(sum8(dla));
            const float dbe = rows4(s * e);
            if (lane == 0) *reinterpret_cast<float4*>(r + 2 * DK) = make_float4(dbe, dla, 0.0f, 0.0f);
            if (l == 0) static_cast<IO*>(p.dv)[(tok * g.H + h) * dv + row] = from_f32<IO>(de);
            __syncthreads();   // (one per token: the next token writes the other buffer)
            float* to = p.sums + ((static_cast<int64_t>(item) * row_blocks + rb) * g.L + t) * kSum;
            for (int c = tid; c < kSum; c += kGdrRecThreads)
                to[c] = (red[buf][0][c] + red[buf][1][c]) + (red[buf][2][c] + red[buf][3][c]);
            buf ^= 1;
        }
        __syncwarp();   // the next segment writes gate
    }
    if (p.dinit) {
#pragma unroll
        for (int m = 0; m < M; ++m) *reinterpret_cast<float4*>(p.dinit + srow + 32 * m) = dS[m];
    }
    for (int64_t t = n; t < g.L; ++t)
        if (l == 0) static_cast<IO*>(p.dv)[((static_cast<int64_t>(b) * g.L + t) * g.H + h) * dv + row] = from_f32<IO>(0.0f);
}

// dq, dk of a token and key head per warp: the sums over blocks and value heads, then the lengths' derivative.
template <typename IO, int DK>
__global__ void __launch_bounds__(128) ss_gdr_rec_fold_kernel(const GdrRecBwd p, int row_blocks) {
    constexpr int N = DK / 32, kSum = 2 * DK + 4;
    const GdrParams& g = p.g;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);   // (b, t, key head)
    if (w >= static_cast<int64_t>(g.batch) * g.L * g.Hk) return;
    const int lane = threadIdx.x & 31, hk = static_cast<int>(w % g.Hk), rep = g.H / g.Hk;
    const int64_t tok = w / g.Hk, b = tok / g.L, t = tok % g.L;
    const bool live = t < gdr_len(g, static_cast<int>(b));
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const IO* x = static_cast<const IO*>(which ? g.k : g.q) + (tok * g.Hk + hk) * DK;
        IO* to = static_cast<IO*>(which ? p.dk : p.dq) + (tok * g.Hk + hk) * DK;
        float d[N], xv[N];
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = xv[i] = 0.0f;
        if (live) {
            for (int e = 0; e < rep * row_blocks; ++e) {   // (head by head, block by block)
                const int64_t item = b * g.H + hk * rep + e / row_blocks;
                const float* s = p.sums + ((item * row_blocks + e % row_blocks) * g.L + t) * kSum + which * DK;
#pragma unroll
                for (int i = 0; i < N; ++i) d[i] += s[lane + 32 * i];
            }
            float xx = 0.0f, xd = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (!which) d[i] *= g.scale;
                xv[i] = to_f32(x[lane + 32 * i]);
                xx = fmaf(xv[i], xv[i], xx);
                xd = fmaf(xv[i], d[i], xd);
            }
            if (g.l2norm) {   // x̂ = x / |x|:  dx = (dx̂ - x̂ (x̂·dx̂)) / |x|
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    xx += __shfl_xor_sync(0xffffffffu, xx, o);
                    xd += __shfl_xor_sync(0xffffffffu, xd, o);
                }
                const float r = 1.0f / sqrtf(xx + kGdrL2Eps);
#pragma unroll
                for (int i = 0; i < N; ++i) d[i] = r * fmaf(-xv[i] * r * r, xd, d[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) to[lane + 32 * i] = from_f32<IO>(d[i]);
    }
}

// The gates' gradients, a block per (b, h), and the item's shares of dA and ddt_bias.
template <typename IO>
__global__ void __launch_bounds__(256) ss_gdr_rec_gate_kernel(const GdrRecBwd p, int row_blocks, int dk) {
    __shared__ double red[2][8];
    const GdrParams& g = p.g;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sum = 2 * dk + 4;
    const int64_t item = blockIdx.x, b = item / g.H, h = item % g.H, n = gdr_len(g, static_cast<int>(b));
    const float A = g.A[h], bias = g.dt_bias ? g.dt_bias[h] : 0.0f;
    double sa = 0.0, sb = 0.0;
    for (int64_t t = threadIdx.x; t < g.L; t += 256) {
        const int64_t o = (b * g.L + t) * g.H + h;
        float ddt = 0.0f, db = 0.0f;
        if (t < n) {
            float dla = 0.0f;
            for (int r = 0; r < row_blocks; ++r) {
                const float2 s = *reinterpret_cast<const float2*>(p.sums + ((item * row_blocks + r) * g.L + t) * sum + 2 * dk);
                db += s.x;
                dla += s.y;
            }
            const float pre = to_f32(static_cast<const IO*>(g.dt)[o]) + bias;
            const float delta = g.softplus ? softplus_accurate(pre) : pre;
            ddt = dla * A * (g.softplus ? 1.0f / (1.0f + expf(-pre)) : 1.0f);
            sa += static_cast<double>(dla) * static_cast<double>(delta);
            sb += static_cast<double>(ddt);
            if (g.sigmoid) {
                const float raw = to_f32(static_cast<const IO*>(g.beta)[o]);
                db *= (1.0f / (1.0f + expf(-raw))) * (1.0f / (1.0f + expf(raw)));
            }
        }
        static_cast<IO*>(p.ddt)[o] = from_f32<IO>(ddt);
        static_cast<IO*>(p.dbeta)[o] = from_f32<IO>(db);
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
        p.part[2 * item + threadIdx.x] = static_cast<float>(s);
    }
}

}  // namespace selscan
