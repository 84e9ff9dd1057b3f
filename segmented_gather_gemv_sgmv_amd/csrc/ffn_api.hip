// ffn_api.hip -- C ABI of the gated feed-forward block (declared in
// include/sgmv.h): argument checks and kernel choice.
#include "proj_launch.hpp"

namespace {

using namespace sgmv;

int check_ffn(int R, int H, int I, int act, int dtype) {
    if (!known_dtype(dtype)) return SGMV_ERR_BAD_DTYPE;
    if (R < 0 || H < 1 || I < 1 || !known_act(act)) return SGMV_ERR_BAD_SHAPE;
    // A tile's 256 rows are reached by 32-bit byte offsets from its first.
    if (H > (1 << 20) || I > (1 << 20) || R > 0x7FFFFF00) return SGMV_ERR_UNSUPPORTED;
    return SGMV_OK;
}

// Takes an option's bit out of dtype.
bool take_option(int32_t& dtype, int option) {
    const bool has = dtype >= 0 && (dtype & option) != 0;
    if (has) dtype &= ~option;
    return has;
}

template <typename DT, int XR, int MT, int PD>
int run_rows(const RowsArgs& a, hipStream_t st) {
    launch(&rows_kernel<DT, PlainSrc<DT>, XR, MT, 1, PD, 1, true>,
           dim3((unsigned)ceil_div(a.N, 16), (unsigned)ceil_div(a.R, 16 * MT)),
           dim3(kRowsThreads), st, a);
    return launch_status();
}

template <typename DT>
int run_forward(const RowsArgs& a, hipStream_t st) {
    const FfnPath path = ffn_path(a.R, a.N, DT::kBytes, a.xvec && a.wvec);
    if (path == kFfnRows4) return run_rows<DT, 4, 1, 2>(a, st);
    if (path == kFfnRows16) return run_rows<DT, 16, 1, 2>(a, st);
    if (path == kFfnRows32) return run_rows<DT, 16, 2, 1>(a, st);
    if constexpr (DT::kBytes == 2) {
        using Src = PlainSrc<DT>;
        const bool wide = ffn_wide_strips(a.N);
        if (path == kFfnStrips32)
            return wide ? launch_strip<DT, Src, 2, 1, 2, 4, 2, 1, true>(a, st)
                        : launch_strip<DT, Src, 2, 1, 4, 2, 2, 1, true>(a, st);
        if (path == kFfnStrips64)
            return wide ? launch_strip<DT, Src, 4, 1, 2, 4, 2, 1, true>(a, st)
                        : launch_strip<DT, Src, 4, 1, 4, 2, 2, 1, true>(a, st);
    }
    TileArgs t{};
    t.a[0] = a.x;
    t.lda = a.K;
    t.b[0] = a.m[0].w;
    t.b[1] = a.m[1].w;
    t.ldb = a.K;
    t.out[0] = a.y;
    for (int q = 0; q < 2; ++q) {
        t.add[q] = a.add[q];
        t.save[q] = a.save[q];
    }
    t.save_f32 = a.save_f32;
    t.M = a.R;
    t.N = a.N;
    t.K = a.K;
    t.batches = 1;
    t.avec = a.xvec;
    t.bvec = a.wvec;
    t.yvec = a.N % 4 == 0 && aligned16(a.y) && aligned16(a.add[0]) && aligned16(a.add[1]) &&
             aligned16(a.save[0]) && aligned16(a.save[1]);
    t.act = a.act;
    return launch_tiles_any<DT, kAlongK, kAlongK, 1, true>(t, a.xvec && a.wvec, st);
}

// Where a backward pass keeps what: floats of dx's sums, then (full gradients) the
// second parts of dg and du.
struct GradPlan {
    SumPlan sum;            // dx: of dg Wg, du Wu and, with second parts, theirs
    int parts;              // of dg and du: 1 or 2
    size_t lo_at, lo_each;  // bytes
    size_t bytes;
};

GradPlan plan_gradients(long long R, long long H, long long I, int dtype, bool full, bool dx) {
    GradPlan p{};
    p.parts = full && dtype != SGMV_F32 ? 2 : 1;
    p.sum = plan_sum(R, H, I, 2 * p.parts, dtype);
    if (dx && p.sum.ranges > 1) p.lo_at = (size_t)p.sum.ranges * p.sum.stride * sizeof(float);
    p.bytes = p.lo_at;
    if (p.parts == 2) {
        p.lo_each = (size_t)ceil_div(R * I * elem_size(dtype), 256) * 256;
        p.bytes += 2 * p.lo_each;
    }
    return p;
}

struct GradArgs {
    void *dx, *dWg, *dWu, *dg, *du;
    const void *dh, *x, *Wg, *Wu, *g, *u;
    int R, H, I, act;
    char* workspace;
    GradPlan plan;
};

template <typename DT>
int run_backward(const GradArgs& b, hipStream_t st) {
    using T = typename DT::storage;
    constexpr int PK = PieceOps<DT>::kPK;
    const int parts = b.plan.parts;
    void* const lo[2] = {parts == 2 ? b.workspace + b.plan.lo_at : nullptr,
                         parts == 2 ? b.workspace + b.plan.lo_at + b.plan.lo_each : nullptr};
    if (b.R > 0) {
        const long long n = (long long)b.R * b.I;
        const int vec = aligned16(b.dg) && aligned16(b.du) && aligned16(b.dh) && aligned16(b.g) &&
                        aligned16(b.u);
        const long long blocks = std::min<long long>(ceil_div(n, 256 * DT::kVec), 4096);
        auto run = [&](auto kernel) {
            launch(kernel, dim3((unsigned)blocks), dim3(256), st, (T*)b.dg, (T*)b.du, (T*)lo[0],
                   (T*)lo[1], (const T*)b.dh, b.g, b.u, n, b.act, vec);
        };
        if constexpr (DT::kBytes == 2) {
            if (parts == 2) run(&gated_grad_kernel<DT, true>);
        }
        if (parts == 1) run(&gated_grad_kernel<DT, false>);
        int rc = launch_status();
        if (rc != SGMV_OK) return rc;
    }
    const bool hvec = b.H % PK == 0, ivec = b.I % PK == 0;
    const bool gvec = ivec && aligned16(b.dg) && aligned16(b.du);
    if (b.dx && b.R > 0) {
        // dx = dg Wg + du Wu: segments of K = I, the weights across K.
        const SumPlan& sum = b.plan.sum;
        TileArgs t{};
        const void* const a[4] = {b.dg, b.du, lo[0], lo[1]};
        for (int s = 0; s < 2 * parts; ++s) {
            t.a[s] = a[s];
            t.b[s] = s % 2 == 0 ? b.Wg : b.Wu;
        }
        t.lda = b.I;
        t.ldb = b.H;
        t.out[0] = b.dx;
        t.M = b.R;
        t.N = b.H;
        t.K = b.I;
        t.batches = sum.ranges;
        t.in_ranges = 1;
        t.range_steps = sum.range_steps;
        t.avec = gvec;
        t.bvec = hvec && aligned16(b.Wg) && aligned16(b.Wu);
        t.yvec = b.H % 4 == 0 && aligned16(b.dx);
        if (sum.ranges > 1) {
            t.partial = (float*)b.workspace;
            t.partial_stride = sum.stride;
        }
        const bool direct = t.avec && t.bvec;
        auto run = [&](auto segments) {
            constexpr int kSegs = decltype(segments)::value;
            return sum.ranges == 1
                ? launch_tiles_any<DT, kAlongK, kAcrossK, kSegs, false>(t, direct, st)
                : launch_kind<DT, kAlongK, kAcrossK, kSegs, false>(
                      sum.kind, t, TileRange{0, t.M, 0, t.N}, direct, st);
        };
        int rc = SGMV_OK;
        if (parts == 1) rc = run(std::integral_constant<int, 2>{});
        else if constexpr (DT::kBytes == 2) rc = run(std::integral_constant<int, 4>{});
        if (rc != SGMV_OK) return rc;
        if (sum.ranges > 1) {
            const long long n = (long long)b.R * b.H;
            launch(&join_kernel<DT>, dim3((unsigned)ceil_div(n, 1024)), dim3(256), st, (T*)b.dx,
                   (const float*)b.workspace, sum.ranges, sum.stride, n, (int)aligned16(b.dx));
            rc = launch_status();
            if (rc != SGMV_OK) return rc;
        }
    }
    if (b.dWg || b.dWu) {
        // dWg = dg^T x and dWu = du^T x, or one of them: K = rows, both operands across
        // K; second parts are a second segment of K.
        TileArgs t{};
        for (int q = 0; q < 2; ++q) {
            void* const out = q == 0 ? b.dWg : b.dWu;
            if (!out) continue;
            t.out[t.batches] = out;
            for (int p = 0; p < parts; ++p) {
                t.a[parts * t.batches + p] = p == 1 ? lo[q] : q == 0 ? b.dg : b.du;
                t.b[parts * t.batches + p] = b.x;
            }
            ++t.batches;
        }
        t.lda = b.I;
        t.ldb = b.H;
        t.M = b.I;
        t.N = b.H;
        t.K = b.R;
        t.avec = gvec;
        t.bvec = hvec && aligned16(b.x);
        t.yvec = b.H % 4 == 0 && aligned16(b.dWg) && aligned16(b.dWu);
        const bool direct = t.avec && t.bvec;
        if (parts == 1) return launch_tiles_any<DT, kAcrossK, kAcrossK, 1, false>(t, direct, st);
        if constexpr (DT::kBytes == 2)
            return launch_tiles_any<DT, kAcrossK, kAcrossK, 2, false>(t, direct, st);
    }
    return SGMV_OK;
}

}  // namespace

extern "C" {

int gated_ffn(void* h, void* g_saved, void* u_saved, const void* x, const void* Wg, const void* Wu,
              const void* gate_add, const void* up_add, int32_t num_rows, int32_t in_features,
              int32_t out_features, int32_t act, int32_t dtype, void* stream) {
    const bool full = take_option(dtype, SGMV_FULL_GRADIENTS);
    take_option(dtype, SGMV_ONE_WEIGHT);
    const int rc = check_ffn(num_rows, in_features, out_features, act, dtype);
    if (rc != SGMV_OK) return rc;
    if (num_rows == 0) return SGMV_OK;
    if (!h || !x || !Wg || !Wu) return SGMV_ERR_NULL_PTR;
    const int pk = piece_elems(dtype);
    RowsArgs a{};
    a.y = h;
    a.x = x;
    a.m[0].w = Wg;
    a.m[1].w = Wu;
    a.add[0] = gate_add;
    a.add[1] = up_add;
    a.save[0] = g_saved;
    a.save[1] = u_saved;
    a.save_f32 = full;
    a.R = num_rows;
    a.N = out_features;
    a.K = in_features;
    a.kblocks = (int)ceil_div(in_features, 16 * pk);
    a.act = act;
    a.xvec = in_features % pk == 0 && aligned16(x);
    a.wvec = in_features % pk == 0 && aligned16(Wg) && aligned16(Wu);
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == SGMV_F32) return run_forward<F32>(a, st);
    if (dtype == SGMV_F16) return run_forward<F16>(a, st);
    return run_forward<BF16>(a, st);
}

size_t gated_ffn_backward_workspace_bytes(int32_t num_rows, int32_t in_features,
                                          int32_t out_features, int32_t dtype) {
    const bool full = take_option(dtype, SGMV_FULL_GRADIENTS);
    take_option(dtype, SGMV_ONE_WEIGHT);
    if (check_ffn(num_rows, in_features, out_features, SGMV_ACT_SILU, dtype) != SGMV_OK || num_rows == 0)
        return 0;
    return plan_gradients(num_rows, in_features, out_features, dtype, full, true).bytes;
}

int gated_ffn_backward(void* dx, void* dWg, void* dWu, void* dg, void* du, const void* dh,
                       const void* x, const void* Wg, const void* Wu, const void* g, const void* u,
                       int32_t num_rows, int32_t in_features, int32_t out_features, int32_t act,
                       int32_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
    const bool full = take_option(dtype, SGMV_FULL_GRADIENTS);
    const bool one_weight = take_option(dtype, SGMV_ONE_WEIGHT);
    const int rc = check_ffn(num_rows, in_features, out_features, act, dtype);
    if (rc != SGMV_OK) return rc;
    if (!one_weight && (dWg == nullptr) != (dWu == nullptr)) return SGMV_ERR_NULL_PTR;
    if (num_rows > 0 &&
        (!dg || !du || !dh || !g || !u || (dx && (!Wg || !Wu)) || ((dWg || dWu) && !x)))
        return SGMV_ERR_NULL_PTR;
    GradPlan plan = plan_gradients(num_rows, in_features, out_features, dtype, full, dx != nullptr);
    if (num_rows == 0) plan.bytes = 0, plan.parts = 1;
    if (plan.bytes > 0 && (!workspace || workspace_bytes < plan.bytes || !aligned16(workspace)))
        return SGMV_ERR_WORKSPACE;
    const GradArgs b{dx, dWg, dWu, dg, du, dh, x, Wg, Wu, g, u, num_rows, in_features, out_features,
                     act, (char*)workspace, plan};
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == SGMV_F32) return run_backward<F32>(b, st);
    if (dtype == SGMV_F16) return run_backward<F16>(b, st);
    return run_backward<BF16>(b, st);
}

}  // extern "C"
