// rope_api.hip -- C ABI of the rotary positions (declared in include/sgmv.h):
// argument checks and the choice of kernel and grid.
#include "sgmv_host.hpp"
#include "proj_plan.hpp"
#include "rope.hpp"

namespace {

using namespace sgmv;

template <typename DT, bool kVec>
void launch_rope(const RopeArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)((long long)a.rows * a.groups)), block(kRopeThreads);
    const int each = rope_units_per_thread(a.heads_per_group, a.units);
    if (each <= 1) launch(&rope_kernel<DT, kVec, 1>, grid, block, st, a);
    else if (each == 2) launch(&rope_kernel<DT, kVec, 2>, grid, block, st, a);
    else launch(&rope_kernel<DT, kVec, kRopeUnitsMost>, grid, block, st, a);
}

template <typename DT>
void launch_rope(const RopeArgs& a, bool vec, hipStream_t st) {
    if (vec) launch_rope<DT, true>(a, st);
    else launch_rope<DT, false>(a, st);
}

}  // namespace

extern "C" int rope(void* q_out, void* k_out, const void* q, const void* k,
                    const void* positions, int32_t position_bytes, const double* inv_freq,
                    float magnitude, int32_t num_rows, int32_t q_heads, int32_t k_heads, int32_t head_dim,
                    int32_t rotary_dim, const int64_t* strides, int32_t interleaved,
                    int32_t inverse, int32_t dtype, void* stream) {
    if (dtype != SGMV_F32 && dtype != SGMV_F16 && dtype != SGMV_BF16) return SGMV_ERR_BAD_DTYPE;
    if (num_rows < 0 || q_heads < 0 || k_heads < 0 || head_dim < 1 || rotary_dim < 2 ||
        rotary_dim > head_dim || (rotary_dim & 1) || (position_bytes != 4 && position_bytes != 8))
        return SGMV_ERR_BAD_SHAPE;
    if (head_dim > kRopeMaxDim) return SGMV_ERR_UNSUPPORTED;
    const long long heads = (long long)q_heads + k_heads;
    if (num_rows == 0 || heads == 0) return SGMV_OK;
    if ((q_heads > 0 && (!q || !q_out)) || (k_heads > 0 && (!k || !k_out)) || !positions ||
        !inv_freq || !strides)
        return SGMV_ERR_NULL_PTR;
    RopeArgs a{};
    a.out[0] = q_out;
    a.out[1] = k_out;
    a.in[0] = q;
    a.in[1] = k;
    for (int w = 0; w < 2; ++w) {
        a.in_row[w] = strides[4 * w];
        a.in_head[w] = strides[4 * w + 1];
        a.out_row[w] = strides[4 * w + 2];
        a.out_head[w] = strides[4 * w + 3];
    }
    a.positions = positions;
    a.wide_positions = position_bytes == 8;
    a.freq = inv_freq;
    a.mag = magnitude;
    a.sign = inverse ? -1.f : 1.f;
    a.rows = num_rows;
    a.heads[0] = q_heads;
    a.heads[1] = k_heads;
    a.D = head_dim;
    a.rot = rotary_dim;
    a.interleaved = interleaved != 0;

    const int V = dtype == SGMV_F32 ? 4 : 8;
    bool vec = head_dim % V == 0 && (interleaved ? rotary_dim : rotary_dim / 2) % V == 0;
    for (int w = 0; w < 2; ++w) {
        if (a.heads[w] == 0) continue;
        vec = vec && aligned16(a.in[w]) && aligned16(a.out[w]);
        for (int s = 0; s < 4; ++s) vec = vec && strides[4 * w + s] % V == 0;
    }
    const RopeGrid g = rope_grid(num_rows, heads, head_dim, rotary_dim, interleaved != 0, vec ? V : 1);
    a.units = g.units;
    a.units_magic = (uint32_t)(((1ull << 32) + a.units - 1) / a.units);
    a.heads_per_group = g.heads_per_group;
    a.groups = g.groups;
    if ((long long)num_rows * a.groups > 0x7FFFFFFFll) return SGMV_ERR_UNSUPPORTED;
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == SGMV_F32) launch_rope<F32>(a, vec, st);
    else if (dtype == SGMV_F16) launch_rope<F16>(a, vec, st);
    else launch_rope<BF16>(a, vec, st);
    return launch_status();
}
