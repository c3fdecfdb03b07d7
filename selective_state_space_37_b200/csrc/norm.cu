// norm.cu -- layer norm over rows, forward and backward (sm_100a).
//
//   μ = Σ x / C,  r = 1 / sqrt(Σ (x - μ)² / C + eps),  x̂ = (x - μ) r,  y = x̂ w + b
//   dx = r (g - mean(g) - x̂ mean(g x̂)),  g = dy w;   dw = Σ_rows dy x̂,  db = Σ_rows dy
//
// Both are bound by HBM: x (and dy) read once, y (or dx) written once.  A row is
// therefore held in registers between its statistics and its output, by the
// threads of one block (or of one warp where a row is short): thread i holds the
// 16-byte vectors i, i + T, ... of the row, T chosen so that every thread has
// work.  The variance is Σ (x - μ)² over the held values, so a large mean costs
// no precision.  The backward pass keeps each thread's columns of dw and db in
// registers over all the rows that its block takes, writes one partial row per
// block, and a second small kernel adds the partials in a fixed order.
// Rows whose length is not a multiple of 16 bytes take single-element accesses in
// the same scheme; rows too long for the registers are read again from L2.
#include <type_traits>

#include "common.cuh"
#include "host.cuh"

using namespace selscan;

namespace {

constexpr int kWarpRows = 4;     // rows per block where one warp takes a row
constexpr int kHeld = 16;        // values of a row that a thread holds
constexpr int kMaxThreads = 512;

struct NormParams {
    const void* x;
    const void* dy;
    const float* weight;
    const float* bias;
    void* out;               // y, or dx
    float* mean;             // written by the forward, read by the backward
    float* rstd;
    float* part;             // [blocks][2][cols]: partial dw, db
    int64_t rows, cols;
    float eps;
};

template <typename IO>
struct VecOf {
    static constexpr int kN = 16 / sizeof(IO);
    static constexpr int kSlots = kHeld / kN;   // vectors that a thread holds
};

// Element e of this thread's vector s: in a row of 16-byte vectors, or (VEC false)
// element by element with neighbouring threads on neighbouring elements.
template <typename IO, bool VEC>
__device__ __forceinline__ int64_t col_of(int s, int e, int t, int T) {
    constexpr int N = VecOf<IO>::kN;
    return VEC ? (static_cast<int64_t>(s) * T + t) * N + e : (static_cast<int64_t>(s) * N + e) * T + t;
}

// This thread's vector s of a row as fp32 (zero behind the row's end).
template <typename IO, bool VEC>
__device__ __forceinline__ void load_vec(const IO* row, int64_t cols, int s, int t, int T,
                                         float (&v)[VecOf<IO>::kN]) {
    constexpr int N = VecOf<IO>::kN;
    if (VEC) {
        const int64_t c = col_of<IO, true>(s, 0, t, T);
        uint4 w = make_uint4(0, 0, 0, 0);
        if (c < cols) w = *reinterpret_cast<const uint4*>(row + c);
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (sizeof(IO) == 2) {
                v[2 * e] = __uint_as_float(a[e] << 16);
                v[2 * e + 1] = __uint_as_float(a[e] & 0xffff0000u);
            } else {
                v[e] = __uint_as_float(a[e]);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int64_t c = col_of<IO, false>(s, e, t, T);
            v[e] = c < cols ? to_f32(row[c]) : 0.0f;
        }
    }
}

template <typename IO, bool VEC>
__device__ __forceinline__ void store_vec(IO* row, int64_t cols, int s, int t, int T,
                                          const float (&v)[VecOf<IO>::kN]) {
    constexpr int N = VecOf<IO>::kN;
    if (VEC) {
        const int64_t c = col_of<IO, true>(s, 0, t, T);
        if (c >= cols) return;
        uint32_t a[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (sizeof(IO) == 2) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
                a[e] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                a[e] = __float_as_uint(v[e]);
            }
        }
        *reinterpret_cast<uint4*>(row + c) = make_uint4(a[0], a[1], a[2], a[3]);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int64_t c = col_of<IO, false>(s, e, t, T);
            if (c < cols) row[c] = from_f32<IO>(v[e]);
        }
    }
}

// The same, kept as it was loaded until it is used (so that the load's latency stays off the row it is fetched in).
template <typename IO>
struct RawVec {
    uint32_t w[4];
};
template <typename IO, bool VEC>
__device__ __forceinline__ void load_raw(const IO* row, int64_t cols, int s, int t, int T, RawVec<IO>& v) {
    constexpr int N = VecOf<IO>::kN;
    if (VEC) {
        const int64_t c = col_of<IO, true>(s, 0, t, T);
        uint4 w = make_uint4(0, 0, 0, 0);
        if (c < cols) w = *reinterpret_cast<const uint4*>(row + c);
        v.w[0] = w.x;
        v.w[1] = w.y;
        v.w[2] = w.z;
        v.w[3] = w.w;
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int64_t c = col_of<IO, false>(s, e, t, T);
            if (sizeof(IO) == 2) {
                const uint32_t b = c < cols ? reinterpret_cast<const unsigned short*>(row)[c] : 0u;
                v.w[e >> 1] = (e & 1) ? v.w[e >> 1] | (b << 16) : b;
            } else {
                v.w[e & 3] = c < cols ? reinterpret_cast<const uint32_t*>(row)[c] : 0u;
            }
        }
    }
}
template <typename IO>
__device__ __forceinline__ void unpack_row(const RawVec<IO>& v, float (&f)[VecOf<IO>::kN]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (sizeof(IO) == 2) {
            f[2 * e] = __uint_as_float(v.w[e] << 16);
            f[2 * e + 1] = __uint_as_float(v.w[e] & 0xffff0000u);
        } else {
            f[e] = __uint_as_float(v.w[e]);
        }
    }
}

// fp32 parameters at a vector's columns (`other` behind the row's end or without a parameter).
template <typename IO, bool VEC>
__device__ __forceinline__ void load_par(const float* par, float other, int64_t cols, int s, int t, int T,
                                         float (&v)[VecOf<IO>::kN]) {
    constexpr int N = VecOf<IO>::kN;
    const int64_t c0 = col_of<IO, true>(s, 0, t, T);
    if (VEC && par && c0 < cols) {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
            const float4 q = *reinterpret_cast<const float4*>(par + c0 + e);
            v[e] = q.x;
            v[e + 1] = q.y;
            v[e + 2] = q.z;
            v[e + 3] = q.w;
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int64_t c = col_of<IO, VEC>(s, e, t, T);
        v[e] = (par && c < cols) ? par[c] : other;
    }
}

// Sums of a and b over the threads of a row (a warp, or the whole block of at most 16 warps), in every thread, in a
// fixed order.  Behind the barrier every thread adds the warps' sums itself (a few wide reads: a second round of
// shuffles costs more).
struct RowSums {
    float4 buf[2][2][4];   // two buffers: the next sum may start before every warp has read this one
};
template <bool WARP>
__device__ __forceinline__ void row_sum2(float& a, float& b, RowSums& red, int& flip) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (WARP) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    float4 (&buf)[2][4] = red.buf[flip];
    flip ^= 1;
    if (lane == 0) {
        reinterpret_cast<float*>(buf[0])[warp] = a;
        reinterpret_cast<float*>(buf[1])[warp] = b;
    }
    if (threadIdx.x < 16 && threadIdx.x >= nw) {   // warps that are not there
        reinterpret_cast<float*>(buf[0])[threadIdx.x] = 0.0f;
        reinterpret_cast<float*>(buf[1])[threadIdx.x] = 0.0f;
    }
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (4 * q >= nw) break;
        const float4 x = buf[0][q], y = buf[1][q];
        a += (x.x + x.y) + (x.z + x.w);
        b += (y.x + y.y) + (y.z + y.w);
    }
}

// HELD: the row fits the block's registers (kHeld values per thread); otherwise `slots` vectors are read
// again for each use.  WARP: one warp per row.
template <typename IO, bool VEC, bool WARP, bool HELD>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : kMaxThreads) ss_norm_fwd_kernel(const NormParams p, int slots) {
    constexpr int N = VecOf<IO>::kN, kSlots = VecOf<IO>::kSlots;
    __shared__ RowSums red;
    int flip = 0;
    const int T = WARP ? 32 : blockDim.x, t = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t first = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = WARP ? static_cast<int64_t>(gridDim.x) * kWarpRows : gridDim.x;
    const int64_t C = p.cols;
    const float inv = 1.0f / static_cast<float>(C);
    float w[HELD ? kSlots : 1][N], b[HELD ? kSlots : 1][N];
    if (HELD) {
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            load_par<IO, VEC>(p.weight, 1.0f, C, s, t, T, w[s]);
            load_par<IO, VEC>(p.bias, 0.0f, C, s, t, T, b[s]);
        }
    }
    for (int64_t r = first; r < p.rows; r += step) {
        const IO* row = static_cast<const IO*>(p.x) + r * C;
        IO* out = static_cast<IO*>(p.out) + r * C;
        float v[HELD ? kSlots : 1][N];
        float sum = 0.0f, none = 0.0f;
        if (HELD) {
#pragma unroll
            for (int s = 0; s < kSlots; ++s) load_vec<IO, VEC>(row, C, s, t, T, v[s]);
#pragma unroll
            for (int s = 0; s < kSlots; ++s)
#pragma unroll
                for (int e = 0; e < N; ++e) sum += v[s][e];
        } else {
            for (int s = 0; s < slots; ++s) {
                load_vec<IO, VEC>(row, C, s, t, T, v[0]);
#pragma unroll
                for (int e = 0; e < N; ++e) sum += v[0][e];
            }
        }
        row_sum2<WARP>(sum, none, red, flip);
        const float mu = sum * inv;
        float sq = 0.0f;
        if (HELD) {
#pragma unroll
            for (int s = 0; s < kSlots; ++s)
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float d = col_of<IO, VEC>(s, e, t, T) < C ? v[s][e] - mu : 0.0f;
                    v[s][e] = d;
                    sq = fmaf(d, d, sq);
                }
        } else {
            for (int s = 0; s < slots; ++s) {
                load_vec<IO, VEC>(row, C, s, t, T, v[0]);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float d = col_of<IO, VEC>(s, e, t, T) < C ? v[0][e] - mu : 0.0f;
                    sq = fmaf(d, d, sq);
                }
            }
        }
        row_sum2<WARP>(sq, none, red, flip);
        const float rs = 1.0f / sqrtf(fmaf(sq, inv, p.eps));
        if (HELD) {
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
#pragma unroll
                for (int e = 0; e < N; ++e) v[s][e] = fmaf(v[s][e] * rs, w[s][e], b[s][e]);
                store_vec<IO, VEC>(out, C, s, t, T, v[s]);
            }
        } else {
            for (int s = 0; s < slots; ++s) {
                load_vec<IO, VEC>(row, C, s, t, T, v[0]);
                load_par<IO, VEC>(p.weight, 1.0f, C, s, t, T, w[0]);
                load_par<IO, VEC>(p.bias, 0.0f, C, s, t, T, b[0]);
#pragma unroll
                for (int e = 0; e < N; ++e) v[0][e] = fmaf((v[0][e] - mu) * rs, w[0][e], b[0][e]);
                store_vec<IO, VEC>(out, C, s, t, T, v[0]);
            }
        }
        if (t == 0) {
            if (p.mean) p.mean[r] = mu;
            if (p.rstd) p.rstd[r] = rs;
        }
    }
}

// Forward, rows of whole 16-byte vectors that a warp holds: NV vectors per lane, all loaded before the first is used,
// no barrier; the parameters lie in shared memory (their vectors' quads in planes, so that a warp's reads are
// consecutive), loaded once by a block that walks rows.  32768 x 2560 bf16: 60 us, 5.6 TB/s, bound by HBM's
// latency at 16 resident warps per SM (two blocks from NV = 9 on, three below).  In bf16 NV = 16 spills 372 bytes of
// registers and NV = 8 136 (32768 x 4096 111 us, 4.9 TB/s); rows of few vectors leave lanes idle (65536 x 256 17.6 us,
// x 64 14 us).
constexpr int kRowWarps = 8;
template <typename IO, int NV>
__global__ void __launch_bounds__(32 * kRowWarps, NV <= 8 ? 3 : 2) ss_norm_fwd_rows_kernel(const NormParams p) {
    constexpr int N = VecOf<IO>::kN, P = N / 4;   // quads of parameters per vector
    extern __shared__ float4 par[];               // [2][P][vecs]: weight, bias
    const int lane = threadIdx.x & 31;
    const int vecs = static_cast<int>(p.cols / N);
    for (int i = threadIdx.x; i < 2 * P * vecs; i += 32 * kRowWarps) {
        const int which = i / (P * vecs), q = (i / vecs) % P, v = i % vecs;
        const float* src = which ? p.bias : p.weight;
        const float other = which ? 0.0f : 1.0f;
        par[i] = src ? reinterpret_cast<const float4*>(src)[v * P + q] : make_float4(other, other, other, other);
    }
    __syncthreads();
    const float inv = 1.0f / static_cast<float>(p.cols);
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5); r < p.rows;
         r += static_cast<int64_t>(gridDim.x) * kRowWarps) {
        const uint4* row = reinterpret_cast<const uint4*>(static_cast<const IO*>(p.x) + r * p.cols);
        uint4* out = reinterpret_cast<uint4*>(static_cast<IO*>(p.out) + r * p.cols);
        uint4 raw[NV];
#pragma unroll
        for (int s = 0; s < NV; ++s) {
            const int v = lane + 32 * s;
            raw[s] = v < vecs ? __ldcs(row + v) : make_uint4(0, 0, 0, 0);
        }
        auto unpack = [](uint4 w, float (&f)[N]) {
            const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (sizeof(IO) == 2) {
                    f[2 * e] = __uint_as_float(a[e] << 16);
                    f[2 * e + 1] = __uint_as_float(a[e] & 0xffff0000u);
                } else {
                    f[e] = __uint_as_float(a[e]);
                }
            }
        };
        float f[N], sum = 0.0f, sq = 0.0f;
#pragma unroll
        for (int s = 0; s < NV; ++s) {
            unpack(raw[s], f);
            float t = 0.0f;
#pragma unroll
            for (int e = 0; e < N; ++e) t += f[e];
            sum += t;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float mu = sum * inv;
#pragma unroll
        for (int s = 0; s < NV; ++s) {
            unpack(raw[s], f);
            float t = 0.0f;
#pragma unroll
            for (int e = 0; e < N; ++e) t = fmaf(f[e] - mu, f[e] - mu, t);
            if (lane + 32 * s < vecs) sq += t;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
        const float rs = 1.0f / sqrtf(fmaf(sq, inv, p.eps));
#pragma unroll
        for (int s = 0; s < NV; ++s) {
            const int v = lane + 32 * s;
            if (v >= vecs) continue;
            unpack(raw[s], f);
#pragma unroll
            for (int q = 0; q < P; ++q) {
                const float4 w = par[q * vecs + v], b = par[(P + q) * vecs + v];
                f[4 * q] = fmaf((f[4 * q] - mu) * rs, w.x, b.x);
                f[4 * q + 1] = fmaf((f[4 * q + 1] - mu) * rs, w.y, b.y);
                f[4 * q + 2] = fmaf((f[4 * q + 2] - mu) * rs, w.z, b.z);
                f[4 * q + 3] = fmaf((f[4 * q + 3] - mu) * rs, w.w, b.w);
            }
            uint32_t a[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (sizeof(IO) == 2) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
                    a[e] = *reinterpret_cast<const uint32_t*>(&h);
                } else {
                    a[e] = __float_as_uint(f[e]);
                }
            }
            __stcs(out + v, make_uint4(a[0], a[1], a[2], a[3]));
        }
        if (lane == 0) {
            if (p.mean) p.mean[r] = mu;
            if (p.rstd) p.rstd[r] = rs;
        }
    }
}

// dx, and (HELD) this block's partial sums of dw and db.  Without HELD the column sums are a kernel of their own.
template <typename IO, bool VEC, bool WARP, bool HELD>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : kMaxThreads)
ss_norm_bwd_kernel(const NormParams p, int slots, int sums) {
    constexpr int N = VecOf<IO>::kN, kSlots = VecOf<IO>::kSlots;
    __shared__ RowSums red;
    int flip = 0;
    const int T = WARP ? 32 : blockDim.x, t = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t first = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = WARP ? static_cast<int64_t>(gridDim.x) * kWarpRows : gridDim.x;
    const int64_t C = p.cols;
    const float inv = 1.0f / static_cast<float>(C);
    constexpr int H = kHeld / 2;   // a thread's values as pairs
    float w[1][N];
    f32x2 w2[HELD ? H : 1], dw[HELD ? H : 1], db[HELD ? H : 1];
    if (HELD) {
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            load_par<IO, VEC>(p.weight, 1.0f, C, s, t, T, w[0]);
#pragma unroll
            for (int e = 0; e < N; e += 2) w2[(s * N + e) / 2] = pk2(w[0][e], w[0][e + 1]);
        }
#pragma unroll
        for (int e = 0; e < H; ++e) dw[e] = db[e] = pk2(0.0f, 0.0f);
    }
    struct {
        RawVec<IO> x[HELD ? kSlots : 1], g[HELD ? kSlots : 1];
        float mu, rs;
    } next;
    auto fetch_row = [&](int64_t r) {
#pragma unroll
        for (int s = 0; s < (HELD ? kSlots : 0); ++s) {
            load_raw<IO, VEC>(static_cast<const IO*>(p.x) + r * C, C, s, t, T, next.x[s]);
            load_raw<IO, VEC>(static_cast<const IO*>(p.dy) + r * C, C, s, t, T, next.g[s]);
        }
        next.mu = p.mean[r];
        next.rs = p.rstd[r];
    };
    if (HELD && first < p.rows) fetch_row(first);
    for (int64_t r = first; r < p.rows; r += step) {
        const IO* xrow = static_cast<const IO*>(p.x) + r * C;
        const IO* grow = static_cast<const IO*>(p.dy) + r * C;
        IO* out = static_cast<IO*>(p.out) + r * C;
        const float mu = HELD ? next.mu : p.mean[r], rs = HELD ? next.rs : p.rstd[r];
        float x[1][N], g[1][N];
        f32x2 xh[HELD ? H : 1], gw2[HELD ? H : 1];
        float c1 = 0.0f, c2 = 0.0f;
        if (HELD) {
            f32x2 s1 = pk2(0.0f, 0.0f), s2 = s1;
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
                unpack_row<IO>(next.x[s], x[0]);
                unpack_row<IO>(next.g[s], g[0]);
#pragma unroll
                for (int e = 0; e < N; e += 2) {   // behind the row's end g is zero, and with it every term
                    const int i = (s * N + e) / 2;
                    const f32x2 gg = pk2(g[0][e], g[0][e + 1]);
                    xh[i] = mul2(add2(pk2(x[0][e], x[0][e + 1]), pk2(-mu, -mu)), pk2(rs, rs));
                    dw[i] = fma2(gg, xh[i], dw[i]);
                    db[i] = add2(db[i], gg);
                    gw2[i] = mul2(gg, w2[i]);
                    s1 = add2(s1, gw2[i]);
                    s2 = fma2(gw2[i], xh[i], s2);
                }
            }
            c1 = s1.x + s1.y;
            c2 = s2.x + s2.y;
            if (r + step < p.rows) fetch_row(r + step);   // under this row's sums
        } else {
            for (int s = 0; s < slots; ++s) {
                load_vec<IO, VEC>(xrow, C, s, t, T, x[0]);
                load_vec<IO, VEC>(grow, C, s, t, T, g[0]);
                load_par<IO, VEC>(p.weight, 1.0f, C, s, t, T, w[0]);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float gw = g[0][e] * w[0][e];
                    c1 += gw;
                    c2 = fmaf(gw, (x[0][e] - mu) * rs, c2);
                }
            }
        }
        row_sum2<WARP>(c1, c2, red, flip);
        c1 *= inv;
        c2 *= inv;
        if (HELD) {
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    const int i = (s * N + e) / 2;
                    const f32x2 d = mul2(fma2(xh[i], pk2(-c2, -c2), add2(gw2[i], pk2(-c1, -c1))), pk2(rs, rs));
                    x[0][e] = d.x;
                    x[0][e + 1] = d.y;
                }
                store_vec<IO, VEC>(out, C, s, t, T, x[0]);
            }
        } else {
            for (int s = 0; s < slots; ++s) {
                load_vec<IO, VEC>(xrow, C, s, t, T, x[0]);
                load_vec<IO, VEC>(grow, C, s, t, T, g[0]);
                load_par<IO, VEC>(p.weight, 1.0f, C, s, t, T, w[0]);
#pragma unroll
                for (int e = 0; e < N; ++e) x[0][e] = rs * (g[0][e] * w[0][e] - c1 - (x[0][e] - mu) * rs * c2);
                store_vec<IO, VEC>(out, C, s, t, T, x[0]);
            }
        }
    }
    if (!HELD || !sums) return;
    const int64_t pr = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    float* pw = p.part + pr * 2 * C;
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int64_t c = col_of<IO, VEC>(s, e, t, T);
            if (c < C) {
                const f32x2 a = dw[(s * N + e) / 2], b = db[(s * N + e) / 2];
                pw[c] = (e & 1) ? a.y : a.x;
                pw[C + c] = (e & 1) ? b.y : b.x;
            }
        }
}

// Partial column sums of rows too long for the kernel above: block (i, j) adds the rows j, j + gridDim.y, ...
template <typename IO>
__global__ void __launch_bounds__(256) ss_norm_colsum_kernel(const NormParams p) {
    const int64_t C = p.cols, c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (c >= C) return;
    float dw = 0.0f, db = 0.0f;
    for (int64_t r = blockIdx.y; r < p.rows; r += gridDim.y) {
        const float g = to_f32(static_cast<const IO*>(p.dy)[r * C + c]);
        const float xh = (to_f32(static_cast<const IO*>(p.x)[r * C + c]) - p.mean[r]) * p.rstd[r];
        dw = fmaf(g, xh, dw);
        db += g;
    }
    float* pw = p.part + static_cast<int64_t>(blockIdx.y) * 2 * C;
    pw[c] = dw;
    pw[C + c] = db;
}

// dw, db = the sums of `n` partial rows, 32 columns of the 2 C per block, 32 threads per column (444 rows of 2 x 2560:
// 13 us with 8, whose chains of loads show).
constexpr int kFoldWays = 32;
__global__ void __launch_bounds__(32 * kFoldWays)
ss_norm_fold_kernel(const float* __restrict__ part, int n, int64_t C, float* dw, float* db) {
    __shared__ float acc[kFoldWays][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + x;
    float s = 0.0f;
    if (c < 2 * C) {
#pragma unroll 8
        for (int i = y; i < n; i += kFoldWays) s += part[static_cast<int64_t>(i) * 2 * C + c];
    }
    acc[y][x] = s;
    __syncthreads();
    s = acc[x][y];   // column y of the block, its 32 sums over a warp's lanes
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + y;
    if (x != 0 || col >= 2 * C) return;
    if (col < C) {
        if (dw) dw[col] = s;
    } else if (db) {
        db[col - C] = s;
    }
}

// How a row is spread: T threads with `slots` vectors each.
struct NormPlan {
    bool vec, warp, held;
    int T, slots;
    int64_t blocks, parts;   // backward: blocks, and partial rows
};

NormPlan norm_plan(int64_t rows, int64_t cols, bool bf16, bool bwd) {
    NormPlan pl{};
    const int64_t N = bf16 ? 8 : 4;
    pl.vec = cols % N == 0;
    const int64_t vecs = ceil_div(cols, N);
    const int64_t slots = kHeld / N;
    pl.warp = vecs <= 32 * slots;
    pl.held = vecs <= kMaxThreads * slots;
    if (pl.warp) {
        pl.T = 32;
    } else if (pl.held) {
        pl.T = static_cast<int>(ceil_div(ceil_div(vecs, slots), 32) * 32);
    } else {
        pl.T = kMaxThreads;
    }
    pl.slots = static_cast<int>(std::min<int64_t>(ceil_div(vecs, pl.T), INT32_MAX));
    const int64_t items = pl.warp ? ceil_div(rows, kWarpRows) : rows;
    const int threads = pl.warp ? 32 * kWarpRows : pl.T;
    const int64_t sms = sm_count_of_current_device();
    // forward: a block per row while there are few, else blocks that walk rows with the parameters in registers;
    // backward: as many blocks as are resident together at 128 registers a thread (32768 x 2560 bf16: 128 us with twice
    // as many, 120 us so; rows through a ring of bulk copies in shared memory instead of the next row in registers:
    // 117 us, not kept), and their partial rows are written and read once.  (Where a warp takes a row, fp32 and unaligned
    // rows take 146 and 168 registers: three of the four blocks per SM run first, then the fourth.)
    const int64_t resident = sms * std::max(1, (bwd ? 512 : 2048) / threads);
    pl.blocks = std::max<int64_t>(1, std::min(items, resident));
    if (bwd && !pl.held) {
        pl.parts = std::max<int64_t>(1, std::min<int64_t>(rows, 64));
    } else {
        pl.parts = pl.blocks * (pl.warp ? kWarpRows : 1);
    }
    return pl;
}

int check_norm(const ss_norm_dims* dims, uint32_t flags) {
    if (!dims || (flags & ~static_cast<uint32_t>(SS_BF16 | SS_SYNC_CHECK))) return SS_ERR_INVALID_ARG;
    if (dims->rows < 0 || dims->cols < 0 || (dims->cols == 0 && dims->rows > 0)) return SS_ERR_INVALID_ARG;
    if (dims->cols >= (int64_t(1) << 31) || double(dims->rows) * double(dims->cols) > 4.0e18) return SS_ERR_INVALID_ARG;
    return SS_OK;
}

size_t norm_ws(const ss_norm_dims* dims, bool bf16) {
    if (dims->cols == 0 || dims->rows == 0) return 256;
    const NormPlan pl = norm_plan(dims->rows, dims->cols, bf16, true);
    return std::max<size_t>(256, static_cast<size_t>(pl.parts) * 2 * static_cast<size_t>(dims->cols) * sizeof(float));
}

// The row kernel for rows of `vecs` whole vectors, with the least NV that holds them; false if none does.  It is taken
// where its blocks fill every SM (rows >= 8 per SM): fewer rows want a whole block each (row kernel / block kernel, us:
// 16 x 2560 bf16 4.6 / 2.4, 592 x 2560 4.7 / 4.6, 1184 x 2560 5.0 / 6.6, 1184 x 768 3.2 / 2.9, 4736 x 768 6.0 / 8.3,
// 1184 x 2048 fp32 5.1 / 5.3, 32768 x 2560 bf16 60 / 118).
template <typename IO, int NV, int... More>
bool launch_rows(const NormParams& p, int64_t vecs, cudaStream_t stream) {
    if (vecs <= 32 * NV) {
        const size_t smem = static_cast<size_t>(p.cols) * 8;   // two parameters of 4 bytes per column, at most 32 KB
        const int64_t blocks = ceil_div(p.rows, kRowWarps), most = 8 * sm_count_of_current_device();
        ss_norm_fwd_rows_kernel<IO, NV><<<static_cast<unsigned>(std::min(blocks, most)), 32 * kRowWarps, smem, stream>>>(p);
        return true;
    }
    if constexpr (sizeof...(More) > 0) return launch_rows<IO, More...>(p, vecs, stream);
    return false;
}

template <typename IO, bool VEC>
void launch_norm_fwd(const NormParams& p, const NormPlan& pl, cudaStream_t stream) {
    if (VEC && p.rows >= int64_t(kRowWarps) * sm_count_of_current_device() &&
        launch_rows<IO, 1, 2, 3, 4, 6, 8, 10, 12, 16>(p, p.cols / VecOf<IO>::kN, stream))
        return;
    const unsigned g = static_cast<unsigned>(pl.blocks), t = static_cast<unsigned>(pl.warp ? 32 * kWarpRows : pl.T);
    if (pl.warp) ss_norm_fwd_kernel<IO, VEC, true, true><<<g, t, 0, stream>>>(p, pl.slots);
    else if (pl.held) ss_norm_fwd_kernel<IO, VEC, false, true><<<g, t, 0, stream>>>(p, pl.slots);
    else ss_norm_fwd_kernel<IO, VEC, false, false><<<g, t, 0, stream>>>(p, pl.slots);
}

template <typename IO, bool VEC>
void launch_norm_bwd(const NormParams& p, const NormPlan& pl, int sums, cudaStream_t stream) {
    const unsigned g = static_cast<unsigned>(pl.blocks), t = static_cast<unsigned>(pl.warp ? 32 * kWarpRows : pl.T);
    if (!pl.held && sums) {   // before the pass that may overwrite dy
        const dim3 grid(static_cast<unsigned>(ceil_div(p.cols, 256)), static_cast<unsigned>(pl.parts));
        ss_norm_colsum_kernel<IO><<<grid, 256, 0, stream>>>(p);
    }
    if (pl.warp) ss_norm_bwd_kernel<IO, VEC, true, true><<<g, t, 0, stream>>>(p, pl.slots, sums);
    else if (pl.held) ss_norm_bwd_kernel<IO, VEC, false, true><<<g, t, 0, stream>>>(p, pl.slots, sums);
    else ss_norm_bwd_kernel<IO, VEC, false, false><<<g, t, 0, stream>>>(p, pl.slots, sums);
}

int finish(uint32_t flags, cudaStream_t stream) {
    if (cudaGetLastError() != cudaSuccess) return SS_ERR_CUDA;
    if ((flags & SS_SYNC_CHECK) && cudaStreamSynchronize(stream) != cudaSuccess) return SS_ERR_CUDA;
    return SS_OK;
}

}  // namespace

extern "C" {

int ss_norm_fwd(const void* x, const float* weight, const float* bias, void* y, float* mean, float* rstd, float eps,
                uint32_t flags, const ss_norm_dims* dims, const ss_launch* launch) {
    if (!launch) return SS_ERR_INVALID_ARG;
    const int rc = check_norm(dims, flags);
    if (rc != SS_OK) return rc;
    if (!(eps >= 0.0f)) return SS_ERR_INVALID_ARG;
    if (dims->rows == 0) return SS_OK;
    if (!x || !y) return SS_ERR_INVALID_ARG;
    const void* ptrs[] = {x, weight, bias, y, mean, rstd};
    for (const void* q : ptrs)
        if (!aligned16(q)) return SS_ERR_INVALID_ARG;
    const bool bf16 = flags & SS_BF16;
    cudaStream_t stream = static_cast<cudaStream_t>(launch->stream);
    const NormPlan pl = norm_plan(dims->rows, dims->cols, bf16, false);
    NormParams p{};
    p.x = x; p.weight = weight; p.bias = bias; p.out = y; p.mean = mean; p.rstd = rstd;
    p.rows = dims->rows; p.cols = dims->cols; p.eps = eps;
    if (bf16) {
        if (pl.vec) launch_norm_fwd<__nv_bfloat16, true>(p, pl, stream);
        else launch_norm_fwd<__nv_bfloat16, false>(p, pl, stream);
    } else {
        if (pl.vec) launch_norm_fwd<float, true>(p, pl, stream);
        else launch_norm_fwd<float, false>(p, pl, stream);
    }
    return finish(flags, stream);
}

size_t ss_norm_bwd_workspace_bytes(const ss_norm_dims* dims, uint32_t flags) {
    return check_norm(dims, flags) == SS_OK ? norm_ws(dims, flags & SS_BF16) : 0;
}

int ss_norm_bwd(const void* dy, const void* x, const float* mean, const float* rstd, const float* weight, void* dx,
                float* dweight, float* dbias, uint32_t flags, const ss_norm_dims* dims, const ss_launch* launch) {
    if (!launch) return SS_ERR_INVALID_ARG;
    const int rc = check_norm(dims, flags);
    if (rc != SS_OK) return rc;
    const void* ptrs[] = {dy, x, mean, rstd, weight, dx, dweight, dbias};
    for (const void* q : ptrs)
        if (!aligned16(q)) return SS_ERR_INVALID_ARG;
    const bool bf16 = flags & SS_BF16;
    cudaStream_t stream = static_cast<cudaStream_t>(launch->stream);
    const int64_t C = dims->cols;
    if (dims->rows == 0) {
        const size_t n = static_cast<size_t>(C) * sizeof(float);
        if ((dweight && n && cudaMemsetAsync(dweight, 0, n, stream) != cudaSuccess) ||
            (dbias && n && cudaMemsetAsync(dbias, 0, n, stream) != cudaSuccess))
            return SS_ERR_CUDA;
        return SS_OK;
    }
    if (!dy || !x || !mean || !rstd || !dx) return SS_ERR_INVALID_ARG;
    if (!launch->workspace || launch->workspace_bytes < norm_ws(dims, bf16) || !aligned16(launch->workspace))
        return SS_ERR_WORKSPACE;
    const NormPlan pl = norm_plan(dims->rows, C, bf16, true);
    NormParams p{};
    p.x = x; p.dy = dy; p.weight = weight; p.out = dx;
    p.mean = const_cast<float*>(mean); p.rstd = const_cast<float*>(rstd);
    p.part = static_cast<float*>(launch->workspace);
    p.rows = dims->rows; p.cols = C;
    const int sums = (dweight || dbias) ? 1 : 0;
    if (bf16) {
        if (pl.vec) launch_norm_bwd<__nv_bfloat16, true>(p, pl, sums, stream);
        else launch_norm_bwd<__nv_bfloat16, false>(p, pl, sums, stream);
    } else {
        if (pl.vec) launch_norm_bwd<float, true>(p, pl, sums, stream);
        else launch_norm_bwd<float, false>(p, pl, sums, stream);
    }
    if (sums)
        ss_norm_fold_kernel<<<static_cast<unsigned>(ceil_div(2 * C, 32)), 32 * kFoldWays, 0, stream>>>(
            p.part, static_cast<int>(pl.parts), C, dweight, dbias);
    return finish(flags, stream);
}

}  // extern "C"
