// kv_api.hip -- C ABI of the quantized K / V cache (declared in include/sgmv.h):
// argument checks and the choice of kernel and grid.
#include "kv_api.hpp"
#include "kv_cache.hpp"
#include "sgmv_host.hpp"

namespace {

using namespace sgmv;

// Rows of a workgroup: 64 leave whole 16-token lines between ragged ends; fewer where these
// would leave CUs without work.
int kv_row_tile(int rows, int heads) { return (rows + 63ll) / 64 * heads * 2 >= 512 ? 64 : 16; }

template <bool kWrite, typename DT, int BITS, int P>
void launch_kv(const KvArgs& a, hipStream_t st) {
    const int rt = kv_row_tile(a.rows, a.heads);
    const dim3 grid((unsigned)((a.rows - 1ll + rt) / rt), (unsigned)a.heads, 2), block(kKvThreads);
    if constexpr (kWrite) {
        if (rt == 64) launch(&kv_write_kernel<DT, BITS, P, 64>, grid, block, st, a);
        else launch(&kv_write_kernel<DT, BITS, P, 16>, grid, block, st, a);
    } else {
        if (rt == 64) launch(&kv_read_kernel<DT, BITS, P, 64>, grid, block, st, a);
        else launch(&kv_read_kernel<DT, BITS, P, 16>, grid, block, st, a);
    }
}

template <bool kWrite, typename DT, int BITS>
void launch_kv(const KvArgs& a, hipStream_t st) {
    const int p = kv_padded(a.D);
    if (p == 64) launch_kv<kWrite, DT, BITS, 64>(a, st);
    else if (p == 96) launch_kv<kWrite, DT, BITS, 96>(a, st);
    else if (p == 128) launch_kv<kWrite, DT, BITS, 128>(a, st);
    else if (p == 192) launch_kv<kWrite, DT, BITS, 192>(a, st);
    else launch_kv<kWrite, DT, BITS, 256>(a, st);
}

template <bool kWrite, typename DT>
void launch_kv(const KvArgs& a, int kind, hipStream_t st) {
    if (kind == SGMV_KV_FP8) launch_kv<kWrite, DT, 8>(a, st);
    else launch_kv<kWrite, DT, 4>(a, st);
}

// kv_write and kv_read: `k` and `v` are in or out.
template <bool kWrite>
int run_kv(const sgmv_kv_cache* cache, const void* k, const void* v, const void* slots,
           int32_t slot_bytes, int32_t num_rows, const int64_t* strides, int32_t dtype, void* stream) {
    if (dtype != SGMV_F32 && dtype != SGMV_F16 && dtype != SGMV_BF16) return SGMV_ERR_BAD_DTYPE;
    if (num_rows < 0 || (slot_bytes != 4 && slot_bytes != 8)) return SGMV_ERR_BAD_SHAPE;
    if (const int e = kv_check(cache)) return e;
    const int rt = kv_row_tile(num_rows, cache->kv_heads);
    if (!grid_fits((num_rows - 1ll + rt) / rt, kKvThreads)) return SGMV_ERR_UNSUPPORTED;
    if (num_rows == 0) return SGMV_OK;
    if (!k || !v || !slots || !strides) return SGMV_ERR_NULL_PTR;
    KvArgs a{};
    a.codes[0] = (uint8_t*)cache->k;
    a.codes[1] = (uint8_t*)cache->v;
    a.scales[0] = (uint8_t*)cache->k_scales;
    a.scales[1] = (uint8_t*)cache->v_scales;
    const void* x[2] = {k, v};
    const int V = dtype == SGMV_F32 ? 4 : 8;
    a.vec = 1;
    for (int w = 0; w < 2; ++w) {
        a.in[w] = x[w];
        a.out[w] = const_cast<void*>(x[w]);
        a.row[w] = strides[2 * w];
        a.head[w] = strides[2 * w + 1];
        a.vec = a.vec && aligned16(x[w]) && a.row[w] % V == 0 && a.head[w] % V == 0;
    }
    a.slots = slots;
    a.wide_slots = slot_bytes == 8;
    a.num_slots = (long long)cache->num_pages * cache->page_size;
    a.page_size = cache->page_size;
    a.rows = num_rows;
    a.heads = cache->kv_heads;
    a.D = cache->head_dim;
    kv_exponents(cache->kind, dtype, &a.lo, &a.hi);
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == SGMV_F32) launch_kv<kWrite, F32>(a, cache->kind, st);
    else if (dtype == SGMV_F16) launch_kv<kWrite, F16>(a, cache->kind, st);
    else launch_kv<kWrite, BF16>(a, cache->kind, st);
    return launch_status();
}

bool bad_sizes(int32_t num_pages, int32_t page_size, int32_t kv_heads, int32_t head_dim, int32_t kind) {
    return kv_check_sizes(num_pages, page_size, kv_heads, head_dim, kind) != SGMV_OK;
}

}  // namespace

extern "C" size_t kv_codes_bytes(int32_t num_pages, int32_t page_size, int32_t kv_heads,
                                 int32_t head_dim, int32_t kind) {
    if (bad_sizes(num_pages, page_size, kv_heads, head_dim, kind)) return 0;
    return (size_t)num_pages * page_size * kv_heads * kv_code_bytes(head_dim, kind);
}

extern "C" size_t kv_scales_bytes(int32_t num_pages, int32_t page_size, int32_t kv_heads,
                                  int32_t head_dim, int32_t kind) {
    if (bad_sizes(num_pages, page_size, kv_heads, head_dim, kind)) return 0;
    return (size_t)num_pages * page_size * kv_heads * kv_groups(head_dim, kind);
}

extern "C" int kv_write(const sgmv_kv_cache* cache, const void* k, const void* v, const void* slots,
                        int32_t slot_bytes, int32_t num_rows, const int64_t* strides, int32_t dtype,
                        void* stream) {
    return run_kv<true>(cache, k, v, slots, slot_bytes, num_rows, strides, dtype, stream);
}

extern "C" int kv_read(void* k, void* v, const sgmv_kv_cache* cache, const void* slots,
                       int32_t slot_bytes, int32_t num_rows, const int64_t* strides, int32_t dtype,
                       void* stream) {
    return run_kv<false>(cache, k, v, slots, slot_bytes, num_rows, strides, dtype, stream);
}
