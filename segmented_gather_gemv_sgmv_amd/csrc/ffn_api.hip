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

struct GradArgs {
    void *dx, *dWg, *dWu, *dg, *du;
    const void *dh, *x, *Wg, *Wu, *g, *u;
    int R, H, I, act;
    float* workspace;  // of dx's sums, when they are taken in ranges
    SumPlan sum;
};

template <typename DT>
int run_backward(const GradArgs& b, hipStream_t st) {
    using T = typename DT::storage;
    constexpr int PK = PieceOps<DT>::kPK;
    if (b.R > 0) {
        const long long n = (long long)b.R * b.I;
        const int vec = aligned16(b.dg) && aligned16(b.du) && aligned16(b.dh) && aligned16(b.g) &&
                        aligned16(b.u);
        const long long blocks = std::min<long long>(ceil_div(n, 256 * DT::kVec), 4096);
        launch(&gated_grad_kernel<DT>, dim3((unsigned)blocks), dim3(256), st, (T*)b.dg, (T*)b.du,
               (const T*)b.dh, (const T*)b.g, (const T*)b.u, n, b.act, vec);
        int rc = launch_status();
        if (rc != SGMV_OK) return rc;
    }
    const bool hvec = b.H % PK == 0, ivec = b.I % PK == 0;
    const bool gvec = ivec && aligned16(b.dg) && aligned16(b.du);
    if (b.dx && b.R > 0) {
        // dx = dg Wg + du Wu: two segments of K = I, the weights across K.
        TileArgs t{};
        t.a[0] = b.dg;
        t.a[1] = b.du;
        t.lda = b.I;
        t.b[0] = b.Wg;
        t.b[1] = b.Wu;
        t.ldb = b.H;
        t.out[0] = b.dx;
        t.M = b.R;
        t.N = b.H;
        t.K = b.I;
        t.batches = b.sum.ranges;
        t.range_steps = b.sum.range_steps;
        t.avec = gvec;
        t.bvec = hvec && aligned16(b.Wg) && aligned16(b.Wu);
        t.yvec = b.H % 4 == 0 && aligned16(b.dx);
        const bool direct = t.avec && t.bvec;
        int rc;
        if (b.sum.ranges == 1) {
            rc = launch_tiles_any<DT, kAlongK, kAcrossK, 2, false>(t, direct, st);
        } else {
            t.partial = b.workspace;
            t.partial_stride = b.sum.stride;
            rc = launch_kind<DT, kAlongK, kAcrossK, 2, false>(
                b.sum.kind, t, TileRange{0, t.M, 0, t.N}, direct, st);
            if (rc != SGMV_OK) return rc;
            const long long n = (long long)b.R * b.H;
            launch(&join_kernel<DT>, dim3((unsigned)ceil_div(n, 1024)), dim3(256), st, (T*)b.dx,
                   (const float*)b.workspace, b.sum.ranges, b.sum.stride, n, (int)aligned16(b.dx));
            rc = launch_status();
        }
        if (rc != SGMV_OK) return rc;
    }
    if (b.dWg || b.dWu) {
        // dWg = dg^T x and dWu = du^T x, or one of them: K = rows, both operands across K.
        TileArgs t{};
        t.a[0] = b.dWg ? b.dg : b.du;
        t.a[1] = b.du;
        t.lda = b.I;
        t.b[0] = b.x;
        t.b[1] = b.x;
        t.ldb = b.H;
        t.out[0] = b.dWg ? b.dWg : b.dWu;
        t.out[1] = b.dWu;
        t.M = b.I;
        t.N = b.H;
        t.K = b.R;
        t.batches = b.dWg && b.dWu ? 2 : 1;
        t.avec = gvec;
        t.bvec = hvec && aligned16(b.x);
        t.yvec = b.H % 4 == 0 && aligned16(b.dWg) && aligned16(b.dWu);
        return launch_tiles_any<DT, kAcrossK, kAcrossK, 1, false>(t, t.avec && t.bvec, st);
    }
    return SGMV_OK;
}

}  // namespace

extern "C" {

int gated_ffn(void* h, void* g_saved, void* u_saved, const void* x, const void* Wg, const void* Wu,
              const void* gate_add, const void* up_add, int32_t num_rows, int32_t in_features,
              int32_t out_features, int32_t act, int32_t dtype, void* stream) {
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
    take_option(dtype, SGMV_ONE_WEIGHT);
    if (check_ffn(num_rows, in_features, out_features, SGMV_ACT_SILU, dtype) != SGMV_OK || num_rows == 0)
        return 0;
    const SumPlan p = plan_sum(num_rows, in_features, out_features, dtype);
    return p.ranges == 1 ? 0 : (size_t)(p.ranges * p.stride) * sizeof(float);
}

int gated_ffn_backward(void* dx, void* dWg, void* dWu, void* dg, void* du, const void* dh,
                       const void* x, const void* Wg, const void* Wu, const void* g, const void* u,
                       int32_t num_rows, int32_t in_features, int32_t out_features, int32_t act,
                       int32_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
    const bool one_weight = take_option(dtype, SGMV_ONE_WEIGHT);
    const int rc = check_ffn(num_rows, in_features, out_features, act, dtype);
    if (rc != SGMV_OK) return rc;
    if (!one_weight && (dWg == nullptr) != (dWu == nullptr)) return SGMV_ERR_NULL_PTR;
    if (num_rows > 0 &&
        (!dg || !du || !dh || !g || !u || (dx && (!Wg || !Wu)) || ((dWg || dWu) && !x)))
        return SGMV_ERR_NULL_PTR;
    const size_t need =
        dx ? gated_ffn_backward_workspace_bytes(num_rows, in_features, out_features, dtype) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
        return SGMV_ERR_WORKSPACE;
    const GradArgs b{dx, dWg, dWu, dg, du, dh, x, Wg, Wu, g, u, num_rows, in_features, out_features,
                     act, (float*)workspace,
                     plan_sum(num_rows, in_features, out_features, dtype)};
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == SGMV_F32) return run_backward<F32>(b, st);
    if (dtype == SGMV_F16) return run_backward<F16>(b, st);
    return run_backward<BF16>(b, st);
}

}  // extern "C"
