// q4_api.hip -- C ABI of the 4-bit projections (declared in include/sgmv.h):
// the one-time packing of a weight, argument checks and kernel choice.
#include "q4_run.hpp"

namespace sgmv {

// One thread per packed dword: the eight codes of lane `lane` of tile
// (nt, kb), step s -- output feature 16 nt + lane % 16, K from 128 kb + 32 s
// + 8 (lane / 16) on -- and, in the first threads, the pairs of scale and
// biased zero point 16 + z (exact in every type) that go with the tiles
// (ProjWeight).  Codes past N or K are 0.
template <typename DT>
__global__ __launch_bounds__(256) void q4_pack_kernel(
    uint32_t* __restrict__ tiles, typename DT::storage* __restrict__ meta,
    const uint8_t* __restrict__ codes, const typename DT::storage* __restrict__ scales,
    const uint8_t* __restrict__ zeros, int N, int K, int kblocks, int groups, int group,
    int flushes, long long dwords, long long metas) {
    const long long t = (long long)blockIdx.x * 256 + threadIdx.x;
    if (t < dwords) {
        const int s = (int)(t & 3), lane = (int)(t >> 2) & 63;
        const long long tile = t >> 8;
        const long long nt = tile / kblocks;
        const int kb = (int)(tile - nt * kblocks);
        const long long n = nt * 16 + (lane & 15);
        const int k0 = kb * 128 + s * 32 + (lane >> 4) * 8;
        const long long ld = (K + 1) / 2;
        uint32_t w = 0;
        if (n < N) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int k = k0 + e;
                if (k >= K) break;
                const uint32_t q = (codes[n * ld + (k >> 1)] >> (4 * (k & 1))) & 15u;
                w |= q << (4 * (e >> 1) + 16 * (e & 1));
            }
        }
        tiles[t] = w;
    }
    if (t < metas) {  // [N / 16][kblocks][16][flushes]
        const long long cell = t / (16 * flushes);
        const int in_cell = (int)(t - cell * 16 * flushes);
        const long long nt = cell / kblocks;
        const int kb = (int)(cell - nt * kblocks);
        const long long n = nt * 16 + in_cell / flushes;
        const int k = kb * 128 + in_cell % flushes * (128 / flushes);
        const bool in = n < N && k < K;
        const long long at = n * groups + k / group;
        const int z = in && zeros ? zeros[at] & 15 : 8;
        meta[2 * t] = in ? scales[at] : DT::from_float(0.f);
        meta[2 * t + 1] = DT::from_float(kCodeBias + (float)z);
    }
}

}  // namespace sgmv

namespace {

using namespace sgmv;

int check_q4(int N, int K, int group, int dtype) {
    if (!known_dtype(dtype)) return SGMV_ERR_BAD_DTYPE;
    if (N < 1 || K < 1 || group < 32 || group % 32 != 0) return SGMV_ERR_BAD_SHAPE;
    if (K > (1 << 20) || N > 0x7FFFFF00 || group > (1 << 21)) return SGMV_ERR_UNSUPPORTED;
    return SGMV_OK;
}

struct Q4Geometry {
    long long ntiles;
    int kblocks, groups;
    int flushes;  // scale pairs per feature and tile of 128 K
};
Q4Geometry geometry(int N, int K, int group) {
    Q4Geometry q;
    q.ntiles = ceil_div(N, 16);
    q.kblocks = (int)ceil_div(K, 128);
    q.groups = (int)ceil_div(K, group);
    q.flushes = group % 128 == 0 || group >= K ? 1 : group % 64 == 0 ? 2 : 4;
    return q;
}

template <bool kGated>
int run_q4_dtype(const RowsArgs& a, int group, int dtype, hipStream_t st) {
    const int flushes = geometry(a.N, a.K, group).flushes;
    if (dtype == SGMV_F32) return run_q4<F32, kGated>(a, flushes, st);
    if (dtype == SGMV_F16) return run_q4<F16, kGated>(a, flushes, st);
    return run_q4<BF16, kGated>(a, flushes, st);
}

RowsArgs rows_args(void* y, const void* x, int R, int N, int K, int dtype) {
    RowsArgs a{};
    a.y = y;
    a.x = x;
    a.R = R;
    a.N = N;
    a.K = K;
    a.kblocks = (int)ceil_div(K, 128);
    a.xvec = aligned16(x) && K % piece_elems(dtype) == 0;
    return a;
}

}  // namespace

extern "C" {

size_t q4_tiles_bytes(int32_t out_features, int32_t in_features) {
    if (out_features < 1 || in_features < 1) return 0;
    return (size_t)ceil_div(out_features, 16) * (size_t)ceil_div(in_features, 128) * 1024u;
}

size_t q4_meta_bytes(int32_t out_features, int32_t in_features, int32_t group_size,
                     int32_t dtype) {
    if (out_features < 1 || in_features < 1 || group_size < 32 || group_size % 32 != 0 ||
        !known_dtype(dtype))
        return 0;
    const Q4Geometry q = geometry(out_features, in_features, group_size);
    return (size_t)q.ntiles * (size_t)q.kblocks * 16u * (size_t)q.flushes * 2u *
           (size_t)elem_size(dtype);
}

int q4_pack(void* tiles, void* meta, const uint8_t* codes, const void* scales,
            const uint8_t* zeros, int32_t out_features, int32_t in_features, int32_t group_size,
            int32_t dtype, void* stream) {
    const int rc = check_q4(out_features, in_features, group_size, dtype);
    if (rc != SGMV_OK) return rc;
    if (!tiles || !meta || !codes || !scales) return SGMV_ERR_NULL_PTR;
    const Q4Geometry q = geometry(out_features, in_features, group_size);
    const long long dwords = q.ntiles * q.kblocks * 256, metas = q.ntiles * q.kblocks * 16 * q.flushes;
    const long long blocks = ceil_div(std::max(dwords, metas), 256);
    if (blocks > 0x7FFFFFFFll) return SGMV_ERR_UNSUPPORTED;
    auto run = [&](auto dt) {
        using DT = decltype(dt);
        using T = typename DT::storage;
        launch(&q4_pack_kernel<DT>, dim3((unsigned)blocks), dim3(256), (hipStream_t)stream,
               (uint32_t*)tiles, (T*)meta, codes, (const T*)scales, zeros,
               (int)out_features, (int)in_features, q.kblocks, q.groups, (int)group_size,
               q.flushes, dwords, metas);
    };
    if (dtype == SGMV_F32) run(F32{});
    else if (dtype == SGMV_F16) run(F16{});
    else run(BF16{});
    return launch_status();
}

int q4_linear(void* y, const void* x, const sgmv_q4_weight* w, const void* bias, int32_t num_rows,
              int32_t out_features, int32_t in_features, int32_t group_size, int32_t dtype,
              void* stream) {
    const int rc = check_q4(out_features, in_features, group_size, dtype);
    if (rc != SGMV_OK) return rc;
    if (num_rows < 0) return SGMV_ERR_BAD_SHAPE;
    if (num_rows == 0) return SGMV_OK;
    if (!y || !x || !w || !w->tiles || !w->meta) return SGMV_ERR_NULL_PTR;
    if (!aligned16(w->tiles) || !aligned16(w->meta)) return SGMV_ERR_UNSUPPORTED;
    RowsArgs a = rows_args(y, x, num_rows, out_features, in_features, dtype);
    a.m[0] = ProjWeight{w->tiles, w->meta};
    a.add[0] = bias;
    return run_q4_dtype<false>(a, group_size, dtype, (hipStream_t)stream);
}

int q4_gated_ffn(void* h, const void* x, const sgmv_q4_weight* gate, const sgmv_q4_weight* up,
                 const void* gate_add, const void* up_add, int32_t num_rows, int32_t out_features,
                 int32_t in_features, int32_t group_size, int32_t act, int32_t dtype, void* stream) {
    const int rc = check_q4(out_features, in_features, group_size, dtype);
    if (rc != SGMV_OK) return rc;
    if (num_rows < 0 || !known_act(act)) return SGMV_ERR_BAD_SHAPE;
    if (num_rows == 0) return SGMV_OK;
    if (!h || !x || !gate || !up || !gate->tiles || !gate->meta || !up->tiles || !up->meta)
        return SGMV_ERR_NULL_PTR;
    if (!aligned16(gate->tiles) || !aligned16(gate->meta) || !aligned16(up->tiles) ||
        !aligned16(up->meta))
        return SGMV_ERR_UNSUPPORTED;
    RowsArgs a = rows_args(h, x, num_rows, out_features, in_features, dtype);
    a.m[0] = ProjWeight{gate->tiles, gate->meta};
    a.m[1] = ProjWeight{up->tiles, up->meta};
    a.add[0] = gate_add;
    a.add[1] = up_add;
    a.act = act;
    return run_q4_dtype<true>(a, group_size, dtype, (hipStream_t)stream);
}

}  // extern "C"
