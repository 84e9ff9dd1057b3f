// attn_api.hip -- C ABI of attention over the quantized cache (declared in include/sgmv.h):
// argument checks, the plan, and the choice of kernel.
#include "attn_plan.hpp"
#include "attn_run.hpp"
#include "kv_api.hpp"

namespace {

using namespace sgmv;

// What a plan and its calls share; checks all of it.
struct Shape {
    AttnSizes sizes;
    PlanLayout at;
    int padded;
};

int check_shape(const sgmv_kv_cache* cache, int32_t num_rows, int32_t num_seqs, int32_t num_prefixes,
                int32_t q_heads, int32_t dtype, Shape* s) {
    if (dtype != SGMV_F32 && dtype != SGMV_F16 && dtype != SGMV_BF16) return SGMV_ERR_BAD_DTYPE;
    if (!cache) return SGMV_ERR_NULL_PTR;
    if (const int e = kv_check_sizes(cache->num_pages, cache->page_size, cache->kv_heads, cache->head_dim,
                                     cache->kind))
        return e;
    if (num_rows < 0 || num_seqs < 0 || num_prefixes < 0 || q_heads < 1 || q_heads % cache->kv_heads)
        return SGMV_ERR_BAD_SHAPE;
    s->padded = kv_padded(cache->head_dim);
    s->sizes = attn_sizes(num_rows, num_seqs, num_prefixes, q_heads, cache->kv_heads, s->padded, dtype);
    // Slots and (row, head) pairs are counted in 31 bits; both kernels have to be launchable.
    const long long pairs = (long long)num_rows * q_heads;
    if (s->sizes.slots > 0x7FFFFFFFll || pairs > 0x7FFFFFFFll || s->sizes.plan_ints > 0x7FFFFFFFull ||
        !grid_fits(s->sizes.items, kAttnThreads) || !grid_fits(pairs + 256, attn_join_lanes(s->padded)))
        return SGMV_ERR_UNSUPPORTED;
    s->at = plan_layout(num_rows, num_seqs, num_prefixes, s->sizes.items);
    return SGMV_OK;
}

// Tokens of a page table's row are counted in 31 bits, and its 16-token blocks are divided by
// those of a page with one multiplication (exact while their product stays below 2^32).
bool table_fits(const sgmv_kv_cache* cache, int32_t width) {
    const long long per = cache->page_size / kKvBlock, blocks = (long long)width * per;
    return blocks * kKvBlock <= 0x7FFFFFC0ll && blocks * per < (1ll << 32);
}

// Scores are taken times scale log2(e), which has to be finite.
constexpr float kScaleMost = 2e38f;

size_t part_bytes(const Shape& s) { return (size_t)s.sizes.slots * s.padded * sizeof(float); }

}  // namespace

extern "C" size_t prefix_plan_bytes(const sgmv_kv_cache* cache, int32_t num_rows, int32_t num_seqs,
                                    int32_t num_prefixes, int32_t q_heads, int32_t dtype) {
    Shape s;
    if (check_shape(cache, num_rows, num_seqs, num_prefixes, q_heads, dtype, &s)) return 0;
    return s.sizes.plan_ints * sizeof(int);
}

extern "C" size_t prefix_attention_workspace_bytes(const sgmv_kv_cache* cache, int32_t num_rows,
                                                   int32_t num_seqs, int32_t num_prefixes,
                                                   int32_t q_heads, int32_t dtype) {
    Shape s;
    if (check_shape(cache, num_rows, num_seqs, num_prefixes, q_heads, dtype, &s)) return 0;
    return part_bytes(s) + (size_t)s.sizes.slots * sizeof(float2);
}

extern "C" int prefix_plan(void* plan, size_t plan_bytes, const sgmv_kv_cache* cache,
                           const int32_t* lengths, const int32_t* row_indptr, int32_t pages_per_seq,
                           const int32_t* prefix_lengths, const int32_t* prefix_indptr,
                           int32_t pages_per_prefix, int32_t num_rows, int32_t num_seqs,
                           int32_t num_prefixes, int32_t q_heads, int32_t dtype, void* stream) {
    Shape s;
    if (const int e = check_shape(cache, num_rows, num_seqs, num_prefixes, q_heads, dtype, &s)) return e;
    if (pages_per_seq < 0 || pages_per_prefix < 0 || (!row_indptr && num_rows < num_seqs) ||
        (num_prefixes > 1 && !prefix_indptr))
        return SGMV_ERR_BAD_SHAPE;
    if (!table_fits(cache, pages_per_seq) || !table_fits(cache, pages_per_prefix)) return SGMV_ERR_UNSUPPORTED;
    if (num_rows == 0 || num_seqs == 0) return SGMV_OK;
    if (!plan || !lengths || (num_prefixes > 0 && !prefix_lengths)) return SGMV_ERR_NULL_PTR;
    if (plan_bytes < s.sizes.plan_ints * sizeof(int)) return SGMV_ERR_WORKSPACE;
    PlanArgs a{};
    a.plan = (int*)plan;
    a.at = s.at;
    a.lengths = lengths;
    a.row_indptr = row_indptr;
    a.prefix_lengths = prefix_lengths;
    a.prefix_indptr = prefix_indptr;
    a.rows = num_rows;
    a.seqs = num_seqs;
    a.prefixes = num_prefixes;
    a.kv_heads = cache->kv_heads;
    a.rep = q_heads / cache->kv_heads;
    a.own_tokens = (long long)pages_per_seq * cache->page_size;
    a.prefix_tokens = (long long)pages_per_prefix * cache->page_size;
    a.items = s.sizes.items;
    a.slots = s.sizes.slots;
    a.tiles = attn_tiles(s.padded, dtype);
    launch(&attn_plan_kernel, dim3(1), dim3(kPlanThreads), (hipStream_t)stream, a);
    return launch_status();
}

extern "C" int prefix_attention(void* o, float* lse, const void* q, const sgmv_kv_cache* cache,
                                const void* plan, const int32_t* pages, int32_t pages_per_seq,
                                const int32_t* prefix_pages, int32_t pages_per_prefix,
                                int32_t num_rows, int32_t num_seqs, int32_t num_prefixes,
                                int32_t q_heads, float scale, const int64_t* strides, int32_t dtype,
                                void* workspace, size_t workspace_bytes, void* stream) {
    Shape s;
    if (const int e = check_shape(cache, num_rows, num_seqs, num_prefixes, q_heads, dtype, &s)) return e;
    if (pages_per_seq < 0 || pages_per_prefix < 0 || !(scale > 0.f) || !(scale <= kScaleMost))
        return SGMV_ERR_BAD_SHAPE;
    if (!table_fits(cache, pages_per_seq) || !table_fits(cache, pages_per_prefix) ||
        (long long)cache->num_pages * (cache->page_size / kKvBlock) * cache->kv_heads >= 0xFFFFFFFFll)
        return SGMV_ERR_UNSUPPORTED;  // blocks over all heads are counted in 32 bits
    if (num_rows == 0 || num_seqs == 0) return SGMV_OK;
    if (const int e = kv_check(cache)) return e;
    if (!o || !q || !plan || !strides || (pages_per_seq > 0 && !pages) ||
        (num_prefixes > 0 && pages_per_prefix > 0 && !prefix_pages))
        return SGMV_ERR_NULL_PTR;
    const size_t parts = part_bytes(s);
    if (!workspace || !aligned16(workspace) || workspace_bytes < parts + (size_t)s.sizes.slots * sizeof(float2))
        return SGMV_ERR_WORKSPACE;
    AttnArgs a{};
    a.q = q;
    a.o = o;
    a.lse = lse;
    a.q_row = strides[0];
    a.q_head = strides[1];
    a.o_row = strides[2];
    a.o_head = strides[3];
    a.k = (const uint8_t*)cache->k;
    a.v = (const uint8_t*)cache->v;
    a.k_scales = (const uint8_t*)cache->k_scales;
    a.v_scales = (const uint8_t*)cache->v_scales;
    a.num_pages = cache->num_pages;
    a.blocks_per_page = cache->page_size / kKvBlock;
    a.page_one = a.blocks_per_page == 1 ? ~0u : 0u;
    a.page_magic = a.page_one ? 0u : (uint32_t)(((1ull << 32) + a.blocks_per_page - 1) / a.blocks_per_page);
    a.own_pages = pages;
    a.prefix_pages = prefix_pages;
    a.own_width = pages_per_seq;
    a.prefix_width = pages_per_prefix;
    a.plan = (const int*)plan;
    a.at = s.at;
    a.part_o = (float*)workspace;
    a.part_ml = (float2*)((char*)workspace + parts);
    a.rows = num_rows;
    a.seqs = num_seqs;
    a.prefixes = num_prefixes;
    a.q_heads = q_heads;
    a.kv_heads = cache->kv_heads;
    a.rep = q_heads / cache->kv_heads;
    a.D = cache->head_dim;
    a.c = scale * 1.4426950408889634f;
    const int V = dtype == SGMV_F32 ? 4 : 8;
    a.vec = aligned16(q) && strides[0] % V == 0 && strides[1] % V == 0;
    const uintptr_t four = dtype == SGMV_F32 ? 16 : 8;
    a.o_vec = (uintptr_t)o % four == 0 && strides[2] % 4 == 0 && strides[3] % 4 == 0;
    const hipStream_t st = (hipStream_t)stream;
    const int items = (int)s.sizes.items;
    if (dtype == SGMV_F32) run_attn_f32(a, cache->kind, items, st);
    else if (dtype == SGMV_F16) run_attn_f16(a, cache->kind, items, st);
    else run_attn_bf16(a, cache->kind, items, st);
    return launch_status();
}
