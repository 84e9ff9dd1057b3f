// q4_api.hip -- C ABI of the 4-bit projections (declared in include/sgmv.h):
// the one-time packing of a weight, argument checks and kernel choice.
#include "proj_launch.hpp"

namespace sgmv {

// One thread per packed dword: the eight codes of lane `lane` of tile
// (nt, kb), step s -- output feature 16 nt + lane % 16, K from 128 kb + 32 s
// + 8 (lane / 16) on -- and, in the first grid rows, the scales and zero
// points gathered per n-tile.  Codes past N or K are 0.
template <typename DT>
__global__ __launch_bounds__(256) void q4_pack_kernel(
    uint32_t* __restrict__ tiles, typename DT::storage* __restrict__ pscales,
    uint8_t* __restrict__ pzeros, const uint8_t* __restrict__ codes,
    const typename DT::storage* __restrict__ scales, const uint8_t* __restrict__ zeros, int N, int K,
    int kblocks, int groups, long long dwords, long long metas) {
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
    if (t < metas) {  // [N / 16][groups][16]
        const long long row = t >> 4;
        const long long nt = row / groups;
        const int g = (int)(row - nt * groups);
        const long long n = nt * 16 + (t & 15);
        typename DT::storage sc = 0;
        if (n < N) sc = scales[n * groups + g];
        pscales[t] = sc;
        if (pzeros) pzeros[t] = n < N ? (uint8_t)(zeros[n * groups + g] & 15u) : (uint8_t)0;
    }
}

}  // namespace sgmv

namespace {

using namespace sgmv;

// Rows up to which the rows kernel is taken (16-bit types; float32 has no
// other): beyond, re-reading and unpacking the weight once per 64 rows costs
// more than the tiles' fill and drain.
constexpr int kQ4RowsMax = 256;

int check_q4(int N, int K, int group, int dtype) {
    if (!known_dtype(dtype)) return SGMV_ERR_BAD_DTYPE;
    if (N < 1 || K < 1 || group < 32 || group % 32 != 0) return SGMV_ERR_BAD_SHAPE;
    if (K > (1 << 20) || N > 0x7FFFFF00 || group > (1 << 21)) return SGMV_ERR_UNSUPPORTED;
    return SGMV_OK;
}

struct Q4Geometry {
    int kblocks, groups, group_steps;
    uint32_t magic;
    long long ntiles;
};
Q4Geometry geometry(int N, int K, int group) {
    Q4Geometry q;
    q.kblocks = (int)ceil_div(K, 128);
    // A group longer than the row is the row.
    const int g = (int)std::min<long long>(group, ceil_div(K, 32) * 32);
    q.groups = (int)ceil_div(K, g);
    q.group_steps = g / 32;
    q.magic = (uint32_t)(((1ull << 32) + q.group_steps - 1) / q.group_steps);
    q.ntiles = ceil_div(N, 16);
    return q;
}

template <typename DT, int MT, int FL, bool kGated>
int run_rows(const RowsArgs& a, hipStream_t st) {
    const long long gx = ceil_div(a.N, 16), gy = ceil_div(a.R, 16 * MT);
    if (gy > 65535) return SGMV_ERR_UNSUPPORTED;
    launch(&rows_kernel<DT, Q4Src<DT>, MT, 1, FL, kGated>, dim3((unsigned)gx, (unsigned)gy),
           dim3(kRowsThreads), st, a);
    return launch_status();
}

template <typename DT, bool kGated>
int run_rows_any(const RowsArgs& a, hipStream_t st) {
    auto with_rows = [&](auto fl) {
        constexpr int FL = decltype(fl)::value;
        if (a.R <= 16) return run_rows<DT, 1, FL, kGated>(a, st);
        if (a.R <= 32) return run_rows<DT, 2, FL, kGated>(a, st);
        return run_rows<DT, 4, FL, kGated>(a, st);
    };
    if (a.group_steps % 4 == 0) return with_rows(std::integral_constant<int, 4>{});
    if (a.group_steps % 2 == 0) return with_rows(std::integral_constant<int, 2>{});
    return with_rows(std::integral_constant<int, 1>{});
}

template <typename DT, bool kGated>
int run_q4(const RowsArgs& a, hipStream_t st) {
    if constexpr (DT::kBytes == 2) {
        if (a.R > kQ4RowsMax) {
            TileArgs t{};
            t.a[0] = a.x;
            t.lda = a.K;
            t.q[0] = a.m[0];
            t.q[1] = a.m[1];
            t.out[0] = a.y;
            t.add[0] = a.add[0];
            t.add[1] = a.add[1];
            t.M = a.R;
            t.N = a.N;
            t.K = a.K;
            t.batches = 1;
            t.avec = a.xvec;
            t.yvec = a.yvec;
            t.kblocks = a.kblocks;
            t.group_steps = a.group_steps;
            t.group_magic = a.group_magic;
            t.groups = a.groups;
            t.act = a.act;
            return launch_tiles_any<DT, kAlongK, kCodes, 1, kGated>(t, a.xvec != 0, st);
        }
    }
    return run_rows_any<DT, kGated>(a, st);
}

template <bool kGated>
int run_q4_dtype(const RowsArgs& a, int dtype, hipStream_t st) {
    if (dtype == SGMV_F32) return run_q4<F32, kGated>(a, st);
    if (dtype == SGMV_F16) return run_q4<F16, kGated>(a, st);
    return run_q4<BF16, kGated>(a, st);
}

void fill_common(RowsArgs& a, void* y, const void* x, int R, int N, int K, int group, int dtype) {
    const Q4Geometry q = geometry(N, K, group);
    a.y = y;
    a.x = x;
    a.R = R;
    a.N = N;
    a.K = K;
    a.kblocks = q.kblocks;
    a.group_steps = q.group_steps;
    a.group_magic = q.magic;
    a.groups = q.groups;
    a.xvec = aligned16(x) && K % piece_elems(dtype) == 0;
    a.yvec = aligned16(y) && N % 4 == 0;
}

}  // namespace

extern "C" {

size_t q4_tiles_bytes(int32_t out_features, int32_t in_features) {
    if (out_features < 1 || in_features < 1) return 0;
    return (size_t)ceil_div(out_features, 16) * (size_t)ceil_div(in_features, 128) * 1024u;
}

size_t q4_groups_padded(int32_t out_features, int32_t in_features, int32_t group_size) {
    if (out_features < 1 || in_features < 1 || group_size < 32 || group_size % 32 != 0) return 0;
    return (size_t)ceil_div(out_features, 16) * 16u * (size_t)ceil_div(in_features, group_size);
}

int q4_pack(void* tiles, void* packed_scales, uint8_t* packed_zeros, const uint8_t* codes,
            const void* scales, const uint8_t* zeros, int32_t out_features, int32_t in_features,
            int32_t group_size, int32_t dtype, void* stream) {
    const int rc = check_q4(out_features, in_features, group_size, dtype);
    if (rc != SGMV_OK) return rc;
    if (!tiles || !packed_scales || !codes || !scales || (zeros && !packed_zeros))
        return SGMV_ERR_NULL_PTR;
    if (!zeros) packed_zeros = nullptr;
    const Q4Geometry q = geometry(out_features, in_features, group_size);
    const long long dwords = q.ntiles * q.kblocks * 256, metas = q.ntiles * 16 * q.groups;
    const long long blocks = ceil_div(std::max(dwords, metas), 256);
    if (blocks > 0x7FFFFFFFll) return SGMV_ERR_UNSUPPORTED;
    auto run = [&](auto dt) {
        using DT = decltype(dt);
        using T = typename DT::storage;
        launch(&q4_pack_kernel<DT>, dim3((unsigned)blocks), dim3(256), (hipStream_t)stream,
               (uint32_t*)tiles, (T*)packed_scales, packed_zeros, codes, (const T*)scales, zeros,
               (int)out_features, (int)in_features, q.kblocks, q.groups, dwords, metas);
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
    if (!y || !x || !w || !w->tiles || !w->scales) return SGMV_ERR_NULL_PTR;
    if (!aligned16(w->tiles) || !aligned16(w->scales)) return SGMV_ERR_UNSUPPORTED;
    RowsArgs a{};
    fill_common(a, y, x, num_rows, out_features, in_features, group_size, dtype);
    a.m[0] = ProjWeight{w->tiles, w->scales, w->zeros};
    a.add[0] = bias;
    a.yvec = a.yvec && aligned16(bias);
    return run_q4_dtype<false>(a, dtype, (hipStream_t)stream);
}

int q4_gated_ffn(void* h, const void* x, const sgmv_q4_weight* gate, const sgmv_q4_weight* up,
                 const void* gate_add, const void* up_add, int32_t num_rows, int32_t out_features,
                 int32_t in_features, int32_t group_size, int32_t act, int32_t dtype, void* stream) {
    const int rc = check_q4(out_features, in_features, group_size, dtype);
    if (rc != SGMV_OK) return rc;
    if (num_rows < 0 || !known_act(act)) return SGMV_ERR_BAD_SHAPE;
    if (num_rows == 0) return SGMV_OK;
    if (!h || !x || !gate || !up || !gate->tiles || !gate->scales || !up->tiles || !up->scales)
        return SGMV_ERR_NULL_PTR;
    if (!aligned16(gate->tiles) || !aligned16(gate->scales) || !aligned16(up->tiles) ||
        !aligned16(up->scales))
        return SGMV_ERR_UNSUPPORTED;
    RowsArgs a{};
    fill_common(a, h, x, num_rows, out_features, in_features, group_size, dtype);
    a.m[0] = ProjWeight{gate->tiles, gate->scales, gate->zeros};
    a.m[1] = ProjWeight{up->tiles, up->scales, up->zeros};
    a.add[0] = gate_add;
    a.add[1] = up_add;
    a.act = act;
    a.yvec = a.yvec && aligned16(gate_add) && aligned16(up_add);
    return run_q4_dtype<true>(a, dtype, (hipStream_t)stream);
}

}  // extern "C"
