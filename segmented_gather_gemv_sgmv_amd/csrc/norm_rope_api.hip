// norm_rope_api.hip -- C ABI of the normed rotation (declared in include/sgmv.h):
// argument checks and the choice of kernel and grid.
#include "sgmv_host.hpp"
#include "norm_plan.hpp"
#include "norm_rope.hpp"

namespace {

using namespace sgmv;

template <typename DT, bool kVec, bool kGrad>
void launch_norm(const NormRopeArgs& a, int per_lane, dim3 grid, hipStream_t st) {
    const dim3 block(kNormThreads);
    auto go_lanes = [&](auto k, auto lanes) {
        constexpr int K = decltype(k)::value, kLanes = decltype(lanes)::value;
        if constexpr (kGrad) launch(&norm_rope_grad_kernel<DT, kVec, K>, grid, block, st, a);
        else launch(&norm_rope_kernel<DT, kVec, K, kLanes>, grid, block, st, a);
    };
    auto go = [&](auto k) { go_lanes(k, std::integral_constant<int, 0>{}); };
    if constexpr (kVec && !kGrad) {  // whole heads of 64, 128 or 256, and 512 of 16 bits
        const std::integral_constant<int, 1> k{};
        const int lanes = a.units == a.lanes && a.rot == a.D && !a.interleaved ? a.lanes : 0;
        if constexpr (DT::kBytes == 2)
            if (lanes == 4) return go_lanes(k, std::integral_constant<int, 4>{});
        if (lanes == 8) return go_lanes(k, std::integral_constant<int, 8>{});
        if (lanes == 16) return go_lanes(k, std::integral_constant<int, 16>{});
        if (lanes == 32) return go_lanes(k, std::integral_constant<int, 32>{});
    }
    // 16-byte pieces of a head of at most 1024 elements: 128 units (16 bits) or 256 (float32)
    if (per_lane == 1) go(std::integral_constant<int, 1>{});
    else if (per_lane == 2) go(std::integral_constant<int, 2>{});
    else if constexpr (kVec && DT::kBytes == 4) go(std::integral_constant<int, 4>{});
    else if constexpr (!kVec) {
        if (per_lane == 4) go(std::integral_constant<int, 4>{});
        else go(std::integral_constant<int, 16>{});
    }
}

template <bool kGrad>
void launch_norm(const NormRopeArgs& a, int32_t dtype, bool vec, int per_lane, dim3 grid, hipStream_t st) {
    auto go = [&](auto dt) {
        using DT = decltype(dt);
        if (vec) launch_norm<DT, true, kGrad>(a, per_lane, grid, st);
        else launch_norm<DT, false, kGrad>(a, per_lane, grid, st);
    };
    if (dtype == SGMV_F32) go(F32{});
    else if (dtype == SGMV_F16) go(F16{});
    else go(BF16{});
}

int check_sizes(int32_t position_bytes, int32_t num_rows, int32_t q_heads, int32_t k_heads,
                int32_t head_dim, int32_t rotary_dim, float eps, int32_t dtype) {
    if (dtype != SGMV_F32 && dtype != SGMV_F16 && dtype != SGMV_BF16) return SGMV_ERR_BAD_DTYPE;
    if (num_rows < 0 || q_heads < 0 || k_heads < 0 || head_dim < 1 || rotary_dim < 2 ||
        rotary_dim > head_dim || (rotary_dim & 1) || (position_bytes != 4 && position_bytes != 8) ||
        !(eps >= 0.f))
        return SGMV_ERR_BAD_SHAPE;
    if (head_dim > kNormMaxDim || (long long)q_heads + k_heads > 65536) return SGMV_ERR_UNSUPPORTED;
    return SGMV_OK;
}

// The fields that both directions share; `vec` says whether 16-byte pieces fit all of it.
bool fill(NormRopeArgs& a, const void* const* in, const void* const* weight, const void* positions,
          int32_t position_bytes, const double* inv_freq, float magnitude, float eps, int32_t num_rows,
          int32_t q_heads, int32_t k_heads, int32_t head_dim, int32_t rotary_dim, int32_t interleaved,
          int32_t dtype) {
    const int V = dtype == SGMV_F32 ? 4 : 8;
    a.heads[0] = q_heads;
    a.heads[1] = k_heads;
    bool vec = head_dim % V == 0 && (interleaved ? rotary_dim : rotary_dim / 2) % V == 0;
    for (int w = 0; w < 2; ++w) {
        a.in[w] = in[w];
        a.weight[w] = weight[w];
        if (a.heads[w]) vec = vec && aligned16(in[w]) && aligned16(weight[w]);
    }
    a.positions = positions;
    a.wide_positions = position_bytes == 8;
    a.freq = inv_freq;
    a.mag = magnitude;
    a.eps = eps;
    a.inv_D = 1.f / (float)head_dim;
    a.rows = num_rows;
    a.D = head_dim;
    a.rot = rotary_dim;
    a.interleaved = interleaved != 0;
    a.rows_per_block = norm_rows_per_block(num_rows, rotary_dim);
    a.blocks = (int)((num_rows - 1ll + a.rows_per_block) / a.rows_per_block);
    return vec;
}

}  // namespace

extern "C" int qk_norm_rope(void* q_out, void* k_out, const void* q, const void* k,
                            const void* q_weight, const void* k_weight, const void* positions,
                            int32_t position_bytes, const double* inv_freq, float magnitude,
                            float eps, int32_t num_rows, int32_t q_heads, int32_t k_heads,
                            int32_t head_dim, int32_t rotary_dim, const int64_t* strides,
                            int32_t interleaved, int32_t dtype, void* stream) {
    if (const int e = check_sizes(position_bytes, num_rows, q_heads, k_heads, head_dim, rotary_dim,
                                  eps, dtype))
        return e;
    const long long heads = (long long)q_heads + k_heads;
    if (num_rows == 0 || heads == 0) return SGMV_OK;
    if ((q_heads > 0 && (!q || !q_out)) || (k_heads > 0 && (!k || !k_out)) || !positions ||
        !inv_freq || !strides)
        return SGMV_ERR_NULL_PTR;
    NormRopeArgs a{};
    const void* in[2] = {q, k};
    const void* weight[2] = {q_weight, k_weight};
    bool vec = fill(a, in, weight, positions, position_bytes, inv_freq, magnitude, eps, num_rows,
                    q_heads, k_heads, head_dim, rotary_dim, interleaved, dtype);
    const int V = dtype == SGMV_F32 ? 4 : 8;
    a.out[0] = q_out;
    a.out[1] = k_out;
    for (int w = 0; w < 2; ++w) {
        a.in_row[w] = strides[4 * w];
        a.in_head[w] = strides[4 * w + 1];
        a.out_row[w] = strides[4 * w + 2];
        a.out_head[w] = strides[4 * w + 3];
        if (a.heads[w] == 0) continue;
        vec = vec && aligned16(a.out[w]);
        for (int s = 0; s < 4; ++s) vec = vec && strides[4 * w + s] % V == 0;
    }
    const NormShape s = norm_shape(head_dim, rotary_dim, interleaved != 0, vec ? V : 1);
    a.units = s.units;
    a.lanes = s.lanes;
    a.heads_per_group = norm_heads_per_group(a.blocks, heads, s.lanes);
    a.groups = (int)((heads + a.heads_per_group - 1) / a.heads_per_group);
    if (!grid_fits((long long)a.blocks * a.groups, kNormThreads)) return SGMV_ERR_UNSUPPORTED;
    launch_norm<false>(a, dtype, vec, s.per_lane, dim3((unsigned)(a.blocks * a.groups)),
                       (hipStream_t)stream);
    return launch_status();
}

extern "C" size_t qk_norm_rope_backward_workspace_bytes(int32_t num_rows, int32_t head_dim,
                                                        int32_t rotary_dim) {
    if (num_rows < 1 || head_dim < 1 || head_dim > kNormMaxDim || rotary_dim < 2 ||
        rotary_dim > head_dim)
        return 0;
    // either tensor's workgroups are fewer with a share of them than with all
    return (size_t)norm_grad_shape(num_rows, rotary_dim, kNormGradBlocks).workgroups * 2 * head_dim * sizeof(float);
}

extern "C" int qk_norm_rope_backward(void* dq, void* dk, void* dq_weight, void* dk_weight,
                                     const void* dq_out, const void* dk_out, const void* q,
                                     const void* k, const void* q_weight, const void* k_weight,
                                     const void* positions, int32_t position_bytes,
                                     const double* inv_freq, float magnitude, float eps,
                                     int32_t num_rows, int32_t q_heads, int32_t k_heads,
                                     int32_t head_dim, int32_t rotary_dim, const int64_t* strides,
                                     int32_t interleaved, int32_t dtype, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    if (const int e = check_sizes(position_bytes, num_rows, q_heads, k_heads, head_dim, rotary_dim,
                                  eps, dtype))
        return e;
    const bool sums = dq_weight || dk_weight;
    const bool empty = num_rows == 0 || (q_heads == 0 && k_heads == 0);
    if (!empty && ((q_heads > 0 && (!q || !dq_out)) || (k_heads > 0 && (!k || !dk_out)) ||
                   !positions || !inv_freq || !strides))
        return SGMV_ERR_NULL_PTR;
    const size_t need = qk_norm_rope_backward_workspace_bytes(num_rows, head_dim, rotary_dim);
    if (sums && !empty && (!workspace || workspace_bytes < need || !aligned16(workspace)))
        return SGMV_ERR_WORKSPACE;
    const hipStream_t st = (hipStream_t)stream;
    int n[2] = {0, 0};
    if (!empty) {
        NormRopeArgs a{};
        const void* in[2] = {q, k};
        const void* weight[2] = {q_weight, k_weight};
        bool vec = fill(a, in, weight, positions, position_bytes, inv_freq, magnitude, eps, num_rows,
                        q_heads, k_heads, head_dim, rotary_dim, interleaved, dtype);
        const int V = dtype == SGMV_F32 ? 4 : 8;
        a.out[0] = dq;
        a.out[1] = dk;
        a.grad[0] = dq_out;
        a.grad[1] = dk_out;
        for (int w = 0; w < 2; ++w) {
            a.in_row[w] = strides[6 * w];
            a.in_head[w] = strides[6 * w + 1];
            a.grad_row[w] = strides[6 * w + 2];
            a.grad_head[w] = strides[6 * w + 3];
            a.out_row[w] = strides[6 * w + 4];
            a.out_head[w] = strides[6 * w + 5];
            if (a.heads[w] == 0) continue;
            vec = vec && aligned16(a.out[w]) && aligned16(a.grad[w]);
            for (int s = 0; s < 6; ++s) vec = vec && strides[6 * w + s] % V == 0;
        }
        a.partial = (float*)workspace;
        a.sums[0] = dq_weight != nullptr;
        a.sums[1] = dk_weight != nullptr;
        const NormShape s = norm_shape(head_dim, rotary_dim, interleaved != 0, vec ? V : 1);
        a.units = s.units;
        a.lanes = s.lanes;
        for (int w = 0; w < 2; ++w) {
            if (a.heads[w] == 0) continue;
            const NormGradShape shape = norm_grad_shape(num_rows, rotary_dim, norm_grad_share(q_heads, k_heads, w));
            a.grad_rows[w] = shape.block_rows;
            n[w] = shape.workgroups;
        }
        a.split = n[0];
        launch_norm<true>(a, dtype, vec, s.per_lane, dim3((unsigned)(n[0] + n[1])), st);
    }
    if (sums) {
        const dim3 grid((unsigned)((head_dim + 15) / 16), 2), block(1024);
        const float* p = (const float*)workspace;
        if (dtype == SGMV_F32) launch(&norm_join_kernel<F32>, grid, block, st, p, dq_weight, dk_weight, n[0], n[1], head_dim);
        else if (dtype == SGMV_F16) launch(&norm_join_kernel<F16>, grid, block, st, p, dq_weight, dk_weight, n[0], n[1], head_dim);
        else launch(&norm_join_kernel<BF16>, grid, block, st, p, dq_weight, dk_weight, n[0], n[1], head_dim);
    }
    return launch_status();
}
