// gdr.cu -- the gated delta rule's entry points (ss_gdr_fwd, ss_gdr_step, ss_gdr_bwd): argument checks,
// workspace layout, choice of kernel and launches.
#include "common.cuh"
#include "gdr_bwd.cuh"
#include "gdr_rec.cuh"
#include "gdr_rec_bwd.cuh"
#include "gdr_tc.cuh"
#include "host.cuh"

using namespace selscan;

namespace {

constexpr uint32_t kGdrFlags = SS_BF16 | SS_DELTA_SOFTPLUS | SS_BETA_SIGMOID | SS_QK_L2NORM | SS_SYNC_CHECK |
                               SS_TEST_DROP_CARRY;

int check_gdr(const ss_gdr_dims* d, uint32_t flags) {
    if (!d || (flags & ~kGdrFlags)) return SS_ERR_INVALID_ARG;
    if (d->batch < 0 || d->seqlen < 0 || d->nheads < 0 || d->nheads_k < 0) return SS_ERR_INVALID_ARG;
    if ((d->d_k != 64 && d->d_k != 128) || (d->d_v != 64 && d->d_v != 128)) return SS_ERR_UNSUPPORTED;
    if (d->nheads > 0 && (d->nheads_k == 0 || d->nheads % d->nheads_k)) return SS_ERR_INVALID_ARG;
    const int64_t lim = int64_t(1) << 27;   // (b, head) items times the blocks that share one stay below 2^31
    if (double(d->batch) * double(d->nheads) * (double(d->seqlen) / 64.0 + 1.0) >= 2147483647.0) return SS_ERR_INVALID_ARG;
    if (d->batch >= lim || d->nheads >= lim || d->batch * d->nheads >= lim || d->seqlen >= (int64_t(1) << 31) - 256 ||
        double(d->batch) * double(d->seqlen) * double(d->nheads) * 128.0 > 2.0e18)
        return SS_ERR_INVALID_ARG;
    return SS_OK;
}

GdrParams gdr_params(const void* q, const void* k, const void* v, const void* dt, const float* dt_bias,
                     const float* A, const void* beta, float scale, uint32_t flags, const ss_gdr_dims* d, int64_t L) {
    GdrParams p{};
    p.q = q; p.k = k; p.v = v; p.dt = dt; p.beta = beta; p.dt_bias = dt_bias; p.A = A;
    p.L = L; p.batch = static_cast<int>(d->batch); p.H = static_cast<int>(d->nheads);
    p.Hk = static_cast<int>(d->nheads_k); p.scale = scale;
    p.softplus = (flags & SS_DELTA_SOFTPLUS) ? 1 : 0;
    p.sigmoid = (flags & SS_BETA_SIGMOID) ? 1 : 0;
    p.l2norm = (flags & SS_QK_L2NORM) ? 1 : 0;
    return p;
}

template <typename IO, int DK>
void launch_rec(const GdrParams& p, int dv, cudaStream_t stream) {
    // Four rows of the state per thread from 1.25 blocks per SM on, else one.  d_k = d_v = 128, four rows against one:
    // a decode step 2.7 / 2.2 us at 12 items, 4.0 / 3.9 at 96 (the border is at 93), 4.2 / 4.8 at 144, 198 / 224 at
    // 10240; 256 tokens in fp32 244 / 168 us at 12 items, 313 / 360 at 96, 1374 / 2269 at 768.
    const int64_t items = static_cast<int64_t>(p.batch) * p.H;
    const int big = dv / (kGdrRecRows * 4);
    const bool many = items * big * 4 >= 5 * sm_count_of_current_device();
    const int rb = many ? big : 4 * big;
    auto kern = p.L > 1 ? (many ? ss_gdr_rec_kernel<IO, DK, 4, true> : ss_gdr_rec_kernel<IO, DK, 1, true>)
                        : (many ? ss_gdr_rec_kernel<IO, DK, 4, false> : ss_gdr_rec_kernel<IO, DK, 1, false>);
    kern<<<static_cast<unsigned>(items * rb), kGdrRecThreads, 0, stream>>>(p, dv, rb);
}

int run_rec(const GdrParams& p, const ss_gdr_dims* d, uint32_t flags, cudaStream_t stream) {
    const int dv = static_cast<int>(d->d_v);
    if (flags & SS_BF16) {
        if (d->d_k == 128) launch_rec<__nv_bfloat16, 128>(p, dv, stream);
        else launch_rec<__nv_bfloat16, 64>(p, dv, stream);
    } else {
        if (d->d_k == 128) launch_rec<float, 128>(p, dv, stream);
        else launch_rec<float, 64>(p, dv, stream);
    }
    return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

// bf16 sequences of at least this many tokens run in chunks (token by token against in chunks, d_k = d_v = 128: at 8
// tokens 10 / 22 us with 12 items, 16 / 23 with 96, 84 / 134 with 1280; at 16 tokens 16 / 23, 27 / 23 and 154 / 133; at
// 24 tokens 22 / 22, 37 / 23 and 225 / 133: the two are even near 24, 13 and 14 tokens, and one border serves all).
constexpr int64_t kChunkedFrom = 16;

// 4-D map of a [batch, L, heads, d] bf16 tensor, boxes of `cols` x 64 tokens of one head.
bool head_map(CUtensorMap* m, const void* base, int64_t batch, int64_t L, int64_t heads, int64_t d, int64_t cols,
              CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(L),
                                static_cast<cuuint64_t>(batch)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(d * 2), static_cast<cuuint64_t>(heads * d * 2),
                                   static_cast<cuuint64_t>(L * heads * d * 2)};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(cols), 1, static_cast<cuuint32_t>(gdr::kC), 1};
    return make_map_bf16(m, base, 4, dims, strides, box, swizzle);
}

// Time segments.  Items 0 .. n_whole - 1 run whole, the others are cut into nseg segments of cseg chunks: a state pass
// (two runs for every segment but the first and the last), the fold, then every segment from its entering state.
constexpr int64_t kGdrMaxSeg = 16;
struct GdrPlan {
    int64_t n_whole, nseg, cseg;
};
// The plan with the least chunk-times on the busiest SM (one CTA per SM).  A chunk of the state pass takes 0.8 of one
// with y; the extra launches are charged 3 chunks and the fold one per segment.  Whole call, items whole / in segments:
// 16 items of 16 chunks 82 / 68 us in 4 (80 in 8), of 32 chunks 148 / 92 in 6 (102 in 4), of 512 chunks 2118 / 822 in 9;
// 12 items of 8 chunks 49 / 50 in 4 (runs whole); 160 items of 128 chunks 1392 / 1058, the last wave's 12 items in segments
// (all of them in 4: 1794).
GdrPlan gdr_plan(int64_t items, int64_t nchunks, int32_t chunk_len) {
    GdrPlan best{items, 1, nchunks};
    if (items == 0 || nchunks < 2 || items * 2 * kGdrMaxSeg >= (int64_t(1) << 31)) return best;   // (a launch's blocks)
    if (chunk_len > 0) {
        int64_t cs = std::max<int64_t>(1, ceil_div(chunk_len, gdr::kC));
        if (ceil_div(nchunks, cs) > kGdrMaxSeg) cs = ceil_div(nchunks, kGdrMaxSeg);
        const int64_t k = ceil_div(nchunks, cs);
        return k > 1 ? GdrPlan{0, k, cs} : best;
    }
    const int64_t sms = sm_count_of_current_device(), tail = items % sms;
    double cost = static_cast<double>(ceil_div(items, sms) * nchunks);
    for (int64_t k = 2; k <= std::min(kGdrMaxSeg, nchunks); ++k) {
        const int64_t cs = ceil_div(nchunks, k);
        if (ceil_div(nchunks, cs) != k) continue;
        for (const int64_t n : {items, tail}) {   // every item, or those of the last wave
            if (n == 0) continue;
            const double t = static_cast<double>((items - n) / sms * nchunks) +
                             0.8 * static_cast<double>(ceil_div(n * std::max<int64_t>(1, 2 * k - 3), sms) * cs) +
                             static_cast<double>(ceil_div(n * k, sms) * cs) + 3.0 + static_cast<double>(k);
            if (t < cost - 1e-9) {
                cost = t;
                best = GdrPlan{items - n, k, cs};
            }
        }
    }
    return best;
}

// Workspace: the status word's header, a record per (item, chunk), then the cut items' segment states.
struct GdrLayout {
    int64_t nchunks;
    GdrPlan plan;
    size_t rec, in, loc, map, first, total;
};
GdrLayout gdr_layout(const ss_gdr_dims* d, uint32_t flags, int32_t chunk_len) {
    GdrLayout w{};
    auto al = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    const int64_t items = d->batch * d->nheads;
    w.nchunks = ceil_div(d->seqlen, gdr::kC);
    w.plan = GdrPlan{items, 1, w.nchunks};
    w.rec = w.total = kHeaderBytes;
    if (!(flags & SS_BF16) || d->seqlen < kChunkedFrom) return w;
    w.plan = gdr_plan(items, w.nchunks, chunk_len);
    const size_t n = static_cast<size_t>((items - w.plan.n_whole) * (w.plan.nseg - 1));
    w.in = w.rec + al(static_cast<size_t>(items * w.nchunks) * gdr::kRecBytes);
    w.loc = w.in + al(n * static_cast<size_t>(d->d_v * d->d_k) * sizeof(float));
    w.map = w.loc + al(n * static_cast<size_t>(d->d_v * d->d_k) * sizeof(float));
    w.first = w.map + al(n * static_cast<size_t>(d->d_k * d->d_k) * sizeof(float));
    w.total = w.first;
    if (w.plan.nseg > 1)
        w.total += al(static_cast<size_t>((items - w.plan.n_whole) * d->d_v * d->d_k) * sizeof(float));
    return w;
}

struct Maps {
    CUtensorMap q, k, v, y;
};

template <int DK>
int launch_tc(const gdr::Params& p, const Maps& m, cudaStream_t stream) {
    auto prep = gdr::ss_gdr_prep_kernel<DK>;
    auto kern = gdr::ss_gdr_tc_kernel<DK, true>;
    auto state = gdr::ss_gdr_tc_kernel<DK, false>;
    auto fold = gdr::ss_gdr_fold_kernel<DK>;
    static std::atomic<bool> attr[4][kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || set_smem_limit(kern, gdr::Smem<true>::kBytes, attr[0], dev) != SS_OK ||
        set_smem_limit(prep, gdr::kPrepSmem, attr[1], dev) != SS_OK ||
        set_smem_limit(state, gdr::Smem<false>::kBytes, attr[2], dev) != SS_OK ||
        set_smem_limit(fold, sizeof(gdr::FoldSmem<DK>), attr[3], dev) != SS_OK)
        return SS_ERR_CUDA;
    const int64_t items = static_cast<int64_t>(p.g.batch) * p.g.H, cut = p.nseg > 1 ? items - p.n_whole : 0;
    prep<<<static_cast<unsigned>(items * p.nchunks), gdr::kPrepThreads, gdr::kPrepSmem, stream>>>(p, m.q, m.k);
    if (cut > 0) {
        state<<<static_cast<unsigned>(cut * (2 * p.nseg - 3)), gdr::kThreads, gdr::Smem<false>::kBytes, stream>>>(
            p, m.q, m.k, m.v, m.v);
        const dim3 grid(static_cast<unsigned>(cut), static_cast<unsigned>(p.dv / gdr::FoldSmem<DK>::kRows));
        fold<<<grid, 256, sizeof(gdr::FoldSmem<DK>), stream>>>(p);
    }
    kern<<<static_cast<unsigned>(items - cut + cut * p.nseg), gdr::kThreads, gdr::Smem<true>::kBytes, stream>>>(
        p, m.q, m.k, m.v, m.y);
    return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

int run_tc(const GdrParams& g, const ss_gdr_dims* d, uint32_t flags, const ss_launch* launch, cudaStream_t stream) {
    const GdrLayout w = gdr_layout(d, flags, launch->chunk_len);
    unsigned char* ws = static_cast<unsigned char*>(launch->workspace);
    gdr::Params p{};
    p.n_whole = static_cast<int>(w.plan.n_whole);
    p.nseg = static_cast<int>(w.plan.nseg);
    p.cseg = static_cast<int>(w.plan.cseg);
    p.seg_in = reinterpret_cast<float*>(ws + w.in);
    p.seg_loc = reinterpret_cast<float*>(ws + w.loc);
    p.seg_map = reinterpret_cast<float*>(ws + w.map);
    p.seg_first = reinterpret_cast<float*>(ws + w.first);
    p.g = g;
    p.status = static_cast<uint32_t*>(launch->workspace);
    p.rec = static_cast<unsigned char*>(launch->workspace) + w.rec;
    p.nchunks = w.nchunks;
    p.rec_bytes = gdr::kRecBytes;
    p.dv = static_cast<int>(d->d_v);
    p.test_drop = (flags & SS_TEST_DROP_CARRY) ? 1 : 0;
    p.wait_ns = launch->timeout_iters ? static_cast<uint64_t>(launch->timeout_iters) * 1000ull : kTmaWaitNs;
    p.drain_ns = kTmaWaitNs;
    Maps m;
    if (!head_map(&m.q, g.q, d->batch, d->seqlen, d->nheads_k, d->d_k, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !head_map(&m.k, g.k, d->batch, d->seqlen, d->nheads_k, d->d_k, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !head_map(&m.v, g.v, d->batch, d->seqlen, d->nheads, d->d_v, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !head_map(&m.y, g.y, d->batch, d->seqlen, d->nheads, d->d_v, d->d_v, CU_TENSOR_MAP_SWIZZLE_NONE))
        return SS_ERR_CUDA;
    return d->d_k == 128 ? launch_tc<128>(p, m, stream) : launch_tc<64>(p, m, stream);
}

// bf16 sequences of at least this many tokens run their backward pass in chunks (token by token against in chunks, d_k =
// d_v = 128: at 4 tokens 24 / 59 us with 2 items, 40 / 61 with 96, 354 / 447 with 1280; at 8 tokens 33 / 58, 62 / 61 and
// 648 / 448; at 16 tokens 50 / 58, 106 / 61 and 1245 / 451: the two are even near 19, 8 and 5 tokens, and one border
// serves all).
constexpr int64_t kBwdChunkedFrom = 8;

// The backward pass's workspace: header, records, what the chains keep, the tokens' sums, the items' shares.
// (Token by token: header, kept states and corrections, the blocks' sums, the items' shares.)
struct GdrBwdLayout {
    bool chunks;
    int64_t nchunks;
    size_t rec, keep, dots, part, total;
};
GdrBwdLayout gdr_bwd_layout(const ss_gdr_dims* d, uint32_t flags) {
    GdrBwdLayout w{};
    auto al = [](size_t x) { return (x + 1023) & ~static_cast<size_t>(1023); };
    w.nchunks = ceil_div(d->seqlen, gdr::kC);
    w.chunks = (flags & SS_BF16) && d->seqlen >= kBwdChunkedFrom;
    const size_t items = static_cast<size_t>(d->batch * d->nheads), n = static_cast<size_t>(w.nchunks);
    w.rec = 1024;
    if (!w.chunks) {
        const size_t L = static_cast<size_t>(d->seqlen), dv = static_cast<size_t>(d->d_v), dk = static_cast<size_t>(d->d_k);
        w.keep = w.rec + al(items * ((L + kRecSeg - 1) / kRecSeg) * dv * dk * sizeof(float));
        w.dots = w.keep + al(items * L * dv * sizeof(float));
        w.part = w.dots + al(items * (dv / kGdrRecRows) * L * (2 * dk + 4) * sizeof(float));
        w.total = w.part + al(items * 2 * sizeof(float));
        return w;
    }
    w.keep = w.rec + al(items * n * gdr::kRecBwdBytes);
    w.dots = w.keep + al(items * (n + 1) * gdr::kKeepBytes);
    w.part = w.dots + al((4 * items * n * gdr::kC + items * (n + 1)) * sizeof(float));
    w.total = w.part + al(items * 2 * sizeof(float));
    return w;
}

template <typename IO, int DK>
int launch_rec_bwd(const GdrRecBwd& p, int dv, float* dA, float* ddt_bias, cudaStream_t stream) {
    auto rev = ss_gdr_rec_rev_kernel<IO, DK>;
    constexpr size_t smem = static_cast<size_t>(kRecSeg) * DK / 8 * kGdrRecThreads * sizeof(float);
    static std::atomic<bool> attr[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || set_smem_limit(rev, smem, attr, dev) != SS_OK) return SS_ERR_CUDA;
    const int rb = dv / kGdrRecRows;
    const unsigned items = static_cast<unsigned>(p.g.batch) * static_cast<unsigned>(p.g.H), n = items * static_cast<unsigned>(rb);
    ss_gdr_rec_keep_kernel<IO, DK><<<n, kGdrRecThreads, 0, stream>>>(p, dv, rb);
    rev<<<n, kGdrRecThreads, smem, stream>>>(p, dv, rb);
    const int64_t warps = static_cast<int64_t>(p.g.batch) * p.g.L * p.g.Hk;
    ss_gdr_rec_fold_kernel<IO, DK><<<static_cast<unsigned>(ceil_div(warps, 4)), 128, 0, stream>>>(p, rb);
    ss_gdr_rec_gate_kernel<IO><<<items, 256, 0, stream>>>(p, rb, DK);
    gdr::ss_gdr_head_kernel<<<static_cast<unsigned>(ceil_div(p.g.H, 128)), 128, 0, stream>>>(p.part, p.g.batch, p.g.H, dA,
                                                                                        ddt_bias);
    return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

struct GdrGrads {
    __nv_bfloat16 *dq, *dk, *dv, *ddt, *dbeta;
    float *dA, *ddt_bias;
};

template <int DK>
int launch_bwd(const gdr::Params& p, const Maps& m, const CUtensorMap& mo, const GdrGrads& o, float* part,
               cudaStream_t stream) {
    auto prep = gdr::ss_gdr_prep_kernel<DK>;
    auto fwd = gdr::ss_gdr_tc_kernel<DK, false>;
    auto rev = gdr::ss_gdr_rev_kernel<DK>;
    auto grad = gdr::ss_gdr_grad_kernel<DK>;
    static std::atomic<bool> attr[4][kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || set_smem_limit(prep, gdr::kPrepSmem, attr[0], dev) != SS_OK ||
        set_smem_limit(fwd, gdr::Smem<false>::kBytes, attr[1], dev) != SS_OK ||
        set_smem_limit(rev, gdr::kRevSmem, attr[2], dev) != SS_OK ||
        set_smem_limit(grad, gdr::kGradSmem, attr[3], dev) != SS_OK)
        return SS_ERR_CUDA;
    const int64_t items = static_cast<int64_t>(p.g.batch) * p.g.H;
    const unsigned n = static_cast<unsigned>(items);
    prep<<<static_cast<unsigned>(items * p.nchunks), gdr::kPrepThreads, gdr::kPrepSmem, stream>>>(p, m.q, m.k);
    fwd<<<n, gdr::kThreads, gdr::Smem<false>::kBytes, stream>>>(p, m.q, m.k, m.v, m.v);
    rev<<<n, gdr::kThreads, gdr::kRevSmem, stream>>>(p, m.q, m.k, mo);
    gdr::GradParams gp{p, o.dq, o.dk, o.dv};
    const int64_t blocks = static_cast<int64_t>(p.g.batch) * p.g.Hk * p.nchunks;
    grad<<<static_cast<unsigned>(blocks), gdr::kGradThreads, gdr::kGradSmem, stream>>>(gp, m.q, m.k, mo);
    gdr::GateParams gt{p, o.ddt, o.dbeta, part};
    gdr::ss_gdr_gate_kernel<<<n, 256, 0, stream>>>(gt);
    gdr::ss_gdr_head_kernel<<<static_cast<unsigned>(ceil_div(p.g.H, 128)), 128, 0, stream>>>(part, p.g.batch, p.g.H, o.dA,
                                                                                        o.ddt_bias);
    return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t ss_gdr_fwd_workspace_bytes(const ss_gdr_dims* dims, uint32_t flags, int32_t chunk_len) {
    return check_gdr(dims, flags) == SS_OK ? gdr_layout(dims, flags, chunk_len).total : 0;
}

int ss_gdr_fwd(const void* q, const void* k, const void* v, const void* dt, const float* dt_bias, const float* A,
               const void* beta, const float* h_init, const int32_t* seqlens, void* y, float* final_state,
               float scale, uint32_t flags, const ss_gdr_dims* dims, const ss_launch* launch) {
    if (!launch) return SS_ERR_INVALID_ARG;
    int rc = check_gdr(dims, flags);
    if (rc != SS_OK) return rc;
    const int64_t L = dims->seqlen;
    if (dims->batch == 0 || dims->nheads == 0) return SS_OK;
    if (!A || (L > 0 && (!q || !k || !v || !dt || !beta || !y))) return SS_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, dt, dt_bias, A, beta, h_init, seqlens, y, final_state};
    for (const void* x : ptrs)
        if (!aligned16(x)) return SS_ERR_INVALID_ARG;
    if (!launch->workspace || launch->workspace_bytes < gdr_layout(dims, flags, launch->chunk_len).total ||
        !aligned16(launch->workspace))
        return SS_ERR_WORKSPACE;
    cudaStream_t stream = static_cast<cudaStream_t>(launch->stream);
    if (cudaMemsetAsync(launch->workspace, 0, sizeof(uint32_t), stream) != cudaSuccess) return SS_ERR_CUDA;
    GdrParams p = gdr_params(q, k, v, dt, dt_bias, A, beta, scale, flags, dims, L);
    p.h_init = h_init; p.seqlens = seqlens; p.y = y; p.final_state = final_state;
    rc = (flags & SS_BF16) && L >= kChunkedFrom ? run_tc(p, dims, flags, launch, stream)
                                                : run_rec(p, dims, flags, stream);
    if (rc != SS_OK) return rc;
    return (flags & SS_SYNC_CHECK) ? ss_check(launch) : SS_OK;
}

int ss_gdr_step(float* state, const void* q, const void* k, const void* v, const void* dt, const float* dt_bias,
                const float* A, const void* beta, void* y, float scale, uint32_t flags, const ss_gdr_dims* dims,
                const ss_launch* launch) {
    if (!launch || !dims) return SS_ERR_INVALID_ARG;
    ss_gdr_dims d = *dims;
    d.seqlen = 1;
    int rc = check_gdr(&d, flags);
    if (rc != SS_OK) return rc;
    if (d.batch == 0 || d.nheads == 0) return SS_OK;
    if (!state || !q || !k || !v || !dt || !A || !beta || !y) return SS_ERR_INVALID_ARG;
    const void* ptrs[] = {state, q, k, v, dt, dt_bias, A, beta, y};
    for (const void* x : ptrs)
        if (!aligned16(x)) return SS_ERR_INVALID_ARG;
    cudaStream_t stream = static_cast<cudaStream_t>(launch->stream);
    GdrParams p = gdr_params(q, k, v, dt, dt_bias, A, beta, scale, flags, &d, 1);
    p.h_init = state; p.final_state = state; p.y = y;
    rc = run_rec(p, &d, flags, stream);
    if (rc != SS_OK) return rc;
    if ((flags & SS_SYNC_CHECK) && cudaStreamSynchronize(stream) != cudaSuccess) return SS_ERR_CUDA;
    return SS_OK;
}

size_t ss_gdr_bwd_workspace_bytes(const ss_gdr_dims* dims, uint32_t flags) {
    return check_gdr(dims, flags) == SS_OK ? gdr_bwd_layout(dims, flags).total : 0;
}

int ss_gdr_bwd(const void* q, const void* k, const void* v, const void* dt, const float* dt_bias, const float* A,
               const void* beta, const float* h_init, const int32_t* seqlens, const void* dy, const float* dfinal_state,
               void* dq, void* dk, void* dv, void* ddt, void* dbeta, float* dA, float* ddt_bias, float* dh_init,
               float scale, uint32_t flags, const ss_gdr_dims* dims, const ss_launch* launch) {
    if (!launch) return SS_ERR_INVALID_ARG;
    int rc = check_gdr(dims, flags);
    if (rc != SS_OK) return rc;
    const int64_t L = dims->seqlen, items = dims->batch * dims->nheads;
    if (dims->nheads == 0) {   // no value head reads the key heads: their gradients are zero
        const double n = double(dims->batch) * double(L) * double(dims->nheads_k) * double(dims->d_k);
        if (n == 0.0) return SS_OK;
        if (n > 2.0e18 || !dq || !dk || !aligned16(dq) || !aligned16(dk)) return SS_ERR_INVALID_ARG;
        const size_t bytes = static_cast<size_t>(dims->batch * L * dims->nheads_k * dims->d_k) * ((flags & SS_BF16) ? 2 : 4);
        cudaStream_t stream = static_cast<cudaStream_t>(launch->stream);
        if (cudaMemsetAsync(dq, 0, bytes, stream) != cudaSuccess || cudaMemsetAsync(dk, 0, bytes, stream) != cudaSuccess)
            return SS_ERR_CUDA;
        return ((flags & SS_SYNC_CHECK) && cudaStreamSynchronize(stream) != cudaSuccess) ? SS_ERR_CUDA : SS_OK;
    }
    if (!A || !dA || (ddt_bias && !dt_bias)) return SS_ERR_INVALID_ARG;
    if (dims->batch > 0 && L > 0 &&
        (!q || !k || !v || !dt || !beta || !dy || !dq || !dk || !dv || !ddt || !dbeta))
        return SS_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, dt, dt_bias, A, beta, h_init, seqlens, dy, dfinal_state,
                          dq, dk, dv, ddt, dbeta, dA, ddt_bias, dh_init};
    for (const void* x : ptrs)
        if (!aligned16(x)) return SS_ERR_INVALID_ARG;
    if (!launch->workspace || launch->workspace_bytes < gdr_bwd_layout(dims, flags).total || !aligned16(launch->workspace))
        return SS_ERR_WORKSPACE;
    cudaStream_t stream = static_cast<cudaStream_t>(launch->stream);
    unsigned char* ws = static_cast<unsigned char*>(launch->workspace);
    if (cudaMemsetAsync(ws, 0, sizeof(uint32_t), stream) != cudaSuccess) return SS_ERR_CUDA;
    if (L == 0 || dims->batch == 0) {   // no token: the final state is the entering one
        const size_t n = static_cast<size_t>(dims->nheads) * sizeof(float);
        const size_t st = static_cast<size_t>(items * dims->d_k * dims->d_v) * sizeof(float);
        cudaError_t e = cudaMemsetAsync(dA, 0, n, stream);
        if (e == cudaSuccess && ddt_bias) e = cudaMemsetAsync(ddt_bias, 0, n, stream);
        if (e == cudaSuccess && dh_init && st && dh_init != dfinal_state)
            e = dfinal_state ? cudaMemcpyAsync(dh_init, dfinal_state, st, cudaMemcpyDeviceToDevice, stream)
                             : cudaMemsetAsync(dh_init, 0, st, stream);
        if (e != cudaSuccess) return SS_ERR_CUDA;
    } else if (const GdrBwdLayout w = gdr_bwd_layout(dims, flags); !w.chunks) {
        GdrRecBwd p{};
        p.g = gdr_params(q, k, v, dt, dt_bias, A, beta, scale, flags, dims, L);
        p.g.h_init = h_init;
        p.g.seqlens = seqlens;
        p.dy = dy; p.dfinal = dfinal_state; p.dinit = dh_init;
        p.dq = dq; p.dk = dk; p.dv = dv; p.ddt = ddt; p.dbeta = dbeta;
        p.keep_s = reinterpret_cast<float*>(ws + w.rec);
        p.keep_e = reinterpret_cast<float*>(ws + w.keep);
        p.sums = reinterpret_cast<float*>(ws + w.dots);
        p.part = reinterpret_cast<float*>(ws + w.part);
        const int d = static_cast<int>(dims->d_v);
        if (flags & SS_BF16)
            rc = dims->d_k == 128 ? launch_rec_bwd<__nv_bfloat16, 128>(p, d, dA, ddt_bias, stream)
                                  : launch_rec_bwd<__nv_bfloat16, 64>(p, d, dA, ddt_bias, stream);
        else
            rc = dims->d_k == 128 ? launch_rec_bwd<float, 128>(p, d, dA, ddt_bias, stream)
                                  : launch_rec_bwd<float, 64>(p, d, dA, ddt_bias, stream);
        if (rc != SS_OK) return rc;
    } else {
        gdr::Params p{};
        p.g = gdr_params(q, k, v, dt, dt_bias, A, beta, scale, flags, dims, L);
        p.g.h_init = h_init;
        p.g.seqlens = seqlens;
        p.rec = ws + w.rec;
        p.nchunks = w.nchunks;
        p.n_whole = static_cast<int>(items);
        p.nseg = 1;
        p.rec_bytes = gdr::kRecBwdBytes;
        p.keep = ws + w.keep;
        p.dots = reinterpret_cast<float*>(ws + w.dots);
        p.dfinal = dfinal_state;
        p.dinit = dh_init;
        p.status = reinterpret_cast<uint32_t*>(ws);
        p.dv = static_cast<int>(dims->d_v);
        p.test_drop = (flags & SS_TEST_DROP_CARRY) ? 1 : 0;
        p.wait_ns = launch->timeout_iters ? static_cast<uint64_t>(launch->timeout_iters) * 1000ull : kTmaWaitNs;
        p.drain_ns = kTmaWaitNs;
        Maps m;
        CUtensorMap mo;
        const int64_t B = dims->batch, H = dims->nheads, dvw = dims->d_v;
        if (!head_map(&m.q, q, B, L, dims->nheads_k, dims->d_k, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !head_map(&m.k, k, B, L, dims->nheads_k, dims->d_k, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !head_map(&m.v, v, B, L, H, dvw, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !head_map(&mo, dy, B, L, H, dvw, 64, CU_TENSOR_MAP_SWIZZLE_128B))
            return SS_ERR_CUDA;
        const GdrGrads o{static_cast<__nv_bfloat16*>(dq), static_cast<__nv_bfloat16*>(dk), static_cast<__nv_bfloat16*>(dv),
                         static_cast<__nv_bfloat16*>(ddt), static_cast<__nv_bfloat16*>(dbeta), dA, ddt_bias};
        float* part = reinterpret_cast<float*>(ws + w.part);
        rc = dims->d_k == 128 ? launch_bwd<128>(p, m, mo, o, part, stream)
                              : launch_bwd<64>(p, m, mo, o, part, stream);
        if (rc != SS_OK) return rc;
    }
    return (flags & SS_SYNC_CHECK) ? ss_check(launch) : SS_OK;
}

}  // extern "C"
