// api_selected.cu -- the C ABI of serving with selected pages: host-side checks and
// launches (include/pagedkv.h, "Serving with selected pages").
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <initializer_list>

#include "pool_impl.hpp"
#include "selected.cuh"

namespace {

inline bool aligned(const void* p, uintptr_t n) {
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

inline pkv_status cuda_status(cudaError_t e) { return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA; }

struct Range {
    const void* p;
    size_t bytes;
};

inline bool overlaps(const Range& a, const Range& b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.bytes && y < x + a.bytes;
}

// Some output overlaps an input or another output.
bool any_alias(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Range& i : ins)
            if (overlaps(*o, i)) return true;
        for (auto x = o + 1; x != outs.end(); ++x)
            if (overlaps(*o, *x)) return true;
    }
    return false;
}

// n rows of `bytes` bytes, `stride` bytes apart.
struct Rows {
    const void* p;
    size_t bytes, stride;
};

inline Range span(const Rows& r, size_t n) {
    return {r.p, n && r.p ? (n - 1) * r.stride + r.bytes : 0};
}

// Whether any of n rows of a meets any of b's: rows of one stride may interleave.
bool rows_meet(const Rows& a, const Rows& b, size_t n) {
    if (!overlaps(span(a, n), span(b, n))) return false;
    if (n == 1 || a.stride != b.stride) return true;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    const size_t s = a.stride;
    const size_t d = x >= y ? (x - y) % s : (s - (y - x) % s) % s;  // a's start behind b's
    return !(d >= b.bytes && s - d >= a.bytes);
}

pkv_status check_shapes(int batch, int n_q_heads, int n_kv_heads, int head_dim, int page_size,
                        int num_pages, int table_stride, pkv_dtype dtype) {
    if (batch < 0 || n_q_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0 || page_size <= 0)
        return PKV_ERR_INVALID_ARG;
    if (n_q_heads % n_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (page_size % 16 != 0 || page_size > 256) return PKV_ERR_UNSUPPORTED;
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
    if (num_pages <= 0 || table_stride <= 0) return PKV_ERR_INVALID_ARG;
    return PKV_OK;
}

inline size_t pool_bytes(const pkv_pool* p) {
    return (size_t)p->num_pages * p->n_kv_heads * p->page_size * p->head_dim * 2;
}

struct SelectLayout {
    size_t scores, stats, total;
};

SelectLayout select_layout(int batch, int n_kv_heads, int table_stride) {
    SelectLayout w;
    const size_t units = (size_t)batch * n_kv_heads;
    w.scores = align256(units * table_stride * 8);  // the 64-bit scores come first
    w.stats = w.scores + align256(units * table_stride * 4);
    w.total = w.stats + units * ((table_stride + pkv::kSelectTile - 1) / pkv::kSelectTile) * 16;
    return w;
}

// Limits of the selection's grids and of the shared memory that holds a head's queries.
pkv_status check_select(int batch, int n_kv_heads, int table_stride) {
    if (batch < 0 || n_kv_heads <= 0 || table_stride <= 0) return PKV_ERR_INVALID_ARG;
    if (batch > 65535 || table_stride > pkv::kMaxSelectPages) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

bool positive(double x) { return x > 0.0 && isfinite(x); }

}  // namespace

extern "C" {

pkv_status paged_tables_build(const int32_t* cached_lens, const int32_t* new_lens, int batch,
                              const int32_t* free_pages, int n_free_pages,
                              const int32_t* free_begin, int32_t* free_end, int page_size,
                              int num_pages, int32_t* page_table, int table_stride,
                              int32_t* context_lens, int32_t* query_starts, int n_tokens,
                              int32_t* positions, int32_t* seq_ids, int64_t* slots,
                              uint32_t* dev_status, pkv_stream stream) {
    if (batch < 0 || n_free_pages < 0 || page_size <= 0 || num_pages <= 0 || table_stride <= 0 ||
        n_tokens < 0)
        return PKV_ERR_INVALID_ARG;
    if (page_size % 16 != 0 || page_size > 256 || batch > pkv::kMaxTableBatch)
        return PKV_ERR_UNSUPPORTED;
    if (!free_end || !query_starts || (n_free_pages && !free_pages)) return PKV_ERR_INVALID_ARG;
    if (batch && (!cached_lens || !new_lens || !page_table || !context_lens))
        return PKV_ERR_INVALID_ARG;
    if (n_tokens && (!positions || !seq_ids || !slots)) return PKV_ERR_INVALID_ARG;
    for (const void* p : {(const void*)cached_lens, (const void*)new_lens, (const void*)free_pages,
                          (const void*)free_begin, (const void*)free_end, (const void*)page_table,
                          (const void*)context_lens, (const void*)query_starts,
                          (const void*)positions, (const void*)seq_ids, (const void*)dev_status})
        if (!aligned(p, 4)) return PKV_ERR_INVALID_ARG;
    if (!aligned(slots, 8)) return PKV_ERR_INVALID_ARG;
    const size_t B = batch, N = n_tokens;
    if (any_alias({{page_table, B * table_stride * 4},
                   {context_lens, B * 4},
                   {query_starts, (B + 1) * 4},
                   {positions, N * 4},
                   {seq_ids, N * 4},
                   {slots, N * 8},
                   {free_end, 4},
                   {dev_status, 4}},
                  {{cached_lens, B * 4},
                   {new_lens, B * 4},
                   {free_pages, (size_t)n_free_pages * 4},
                   {free_begin, 4}}))
        return PKV_ERR_ALIAS;
    pkv::TablesArgs a = {};
    a.cached = cached_lens;
    a.fresh = new_lens;
    a.batch = batch;
    a.free_pages = free_pages;
    a.n_free = n_free_pages;
    a.free_begin = free_begin;
    a.free_end = free_end;
    a.page_size = page_size;
    a.num_pages = num_pages;
    a.table = page_table;
    a.table_stride = table_stride;
    a.lens = context_lens;
    a.starts = query_starts;
    a.n_tokens = n_tokens;
    a.positions = positions;
    a.seq_ids = seq_ids;
    a.slots = slots;
    a.status = dev_status;
    return cuda_status(pkv::launch_tables(a, reinterpret_cast<cudaStream_t>(stream)));
}

pkv_status pkv_rope_init(pkv_rope* out, int rotary_dim, double theta, int interleaved,
                         double magnitude, pkv_rope_scaling scaling, double factor,
                         double low_turns, double high_turns, double original_context) {
    if (!out || rotary_dim <= 0 || rotary_dim > 128 || rotary_dim % 16 != 0)
        return PKV_ERR_INVALID_ARG;
    if (!positive(theta) || !positive(magnitude) || !isfinite((float)magnitude))
        return PKV_ERR_INVALID_ARG;
    if (scaling != PKV_ROPE_NONE && scaling != PKV_ROPE_LINEAR && scaling != PKV_ROPE_TURNS &&
        scaling != PKV_ROPE_INDEX)
        return PKV_ERR_INVALID_ARG;
    if (scaling != PKV_ROPE_NONE && !positive(factor)) return PKV_ERR_INVALID_ARG;
    const bool by_turns = scaling == PKV_ROPE_TURNS || scaling == PKV_ROPE_INDEX;
    if (by_turns && (!positive(low_turns) || !positive(high_turns) || !(low_turns < high_turns) ||
                     !positive(original_context)))
        return PKV_ERR_INVALID_ARG;
    if (scaling == PKV_ROPE_INDEX && theta == 1.0) return PKV_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925;
    double first = 0.0, last = 0.0;
    if (scaling == PKV_ROPE_INDEX) {
        const double per = rotary_dim / (2.0 * log(theta));
        first = fmax(floor(per * log(original_context / (two_pi * high_turns))), 0.0);
        last = fmin(ceil(per * log(original_context / (two_pi * low_turns))), rotary_dim - 1.0);
        last = fmax(last, first + 0.001);  // a step, where both ends meet
    }
    memset(out, 0, sizeof(*out));
    out->rotary_dim = rotary_dim;
    out->interleaved = interleaved != 0;
    out->magnitude = (float)magnitude;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = pow(theta, -2.0 * i / rotary_dim);
        if (scaling == PKV_ROPE_LINEAR) {
            f /= factor;
        } else if (by_turns) {
            const double g = scaling == PKV_ROPE_TURNS
                                 ? (original_context * f / two_pi - low_turns) /
                                       (high_turns - low_turns)
                                 : 1.0 - (i - first) / (last - first);
            const double keep = fmin(fmax(g, 0.0), 1.0);
            f = keep * f + (1.0 - keep) * f / factor;
        }
        double turns = f / two_pi;
        turns -= floor(turns);
        if (!(turns >= 0.0 && turns < 1.0)) turns = 0.0;  // beyond double's range
        out->turns[i] = (uint64_t)ldexp(turns, 64);
    }
    return PKV_OK;
}

pkv_status kv_append_tokens(const pkv_pool* pool, const void* k_new, int64_t k_stride,
                            const void* v_new, int64_t v_stride, const int64_t* slots,
                            int n_tokens, const void* q, int64_t q_stride, int n_q_heads,
                            const int32_t* positions, const pkv_rope* rope,
                            const void* q_norm_weight, const void* k_norm_weight, float norm_eps,
                            void* q_out, int64_t q_out_stride, uint32_t* dev_status,
                            pkv_stream stream) {
    if (!pool || n_tokens < 0 || n_q_heads < 0) return PKV_ERR_INVALID_ARG;
    if (pool->dtype == PKV_E4M3) return PKV_ERR_UNSUPPORTED;  // kv8_append
    const int D = pool->head_dim;
    if (!rope && (q || q_out || positions || q_norm_weight || k_norm_weight || n_q_heads))
        return PKV_ERR_INVALID_ARG;
    if (rope) {
        if (rope->rotary_dim <= 0 || rope->rotary_dim % 16 != 0 || rope->reserved != 0 ||
            !isfinite(rope->magnitude))
            return PKV_ERR_INVALID_ARG;
        if (rope->rotary_dim > D) return PKV_ERR_UNSUPPORTED;
        // (an empty tensor may have no address)
        if (n_tokens > 0 && ((n_q_heads > 0) != (q != nullptr) || !q != !q_out ||
                             (!q && q_norm_weight)))
            return PKV_ERR_INVALID_ARG;
        if ((q_norm_weight || k_norm_weight) && !(norm_eps >= 0.f && isfinite(norm_eps)))
            return PKV_ERR_INVALID_ARG;
    }
    if ((int64_t)n_q_heads + 2 * (int64_t)pool->n_kv_heads > pkv::kMaxAppendRows)
        return PKV_ERR_UNSUPPORTED;
    if (n_tokens == 0) return PKV_OK;
    if (!k_new || !v_new || !slots || (rope && !positions)) return PKV_ERR_INVALID_ARG;
    const int64_t kv_row = (int64_t)pool->n_kv_heads * D, q_row = (int64_t)n_q_heads * D;
    auto bad_stride = [](int64_t s, int64_t row) {
        return s < row || s % 8 != 0 || s > (int64_t(1) << 30);
    };
    if (bad_stride(k_stride, kv_row) || bad_stride(v_stride, kv_row) ||
        (q && (bad_stride(q_stride, q_row) || bad_stride(q_out_stride, q_row))))
        return PKV_ERR_INVALID_ARG;
    for (const void* p : {k_new, v_new, q, (const void*)q_out, q_norm_weight, k_norm_weight,
                          (const void*)pool->k, (const void*)pool->v})
        if (!aligned(p, 16)) return PKV_ERR_INVALID_ARG;
    if (!aligned(slots, 8) || !aligned(positions, 4) || !aligned(dev_status, 4))
        return PKV_ERR_INVALID_ARG;

    const size_t n = n_tokens;
    const Rows k{k_new, (size_t)kv_row * 2, (size_t)k_stride * 2};
    const Rows v{v_new, (size_t)kv_row * 2, (size_t)v_stride * 2};
    const Rows qi{q, (size_t)q_row * 2, (size_t)q_stride * 2};
    const Rows qo{q_out, (size_t)q_row * 2, (size_t)q_out_stride * 2};
    const Range kp{pool->k, pool_bytes(pool)}, vp{pool->v, pool_bytes(pool)};
    const Range small[5] = {{slots, n * 8}, {positions, n * 4}, {q_norm_weight, (size_t)D * 2},
                            {k_norm_weight, (size_t)D * 2}, {dev_status, 4}};
    if (overlaps(kp, vp)) return PKV_ERR_ALIAS;
    for (const Range& pl : {kp, vp}) {
        for (const Rows& r : {k, v, qi, qo})
            if (overlaps(pl, span(r, n))) return PKV_ERR_ALIAS;
        for (const Range& s : small)
            if (overlaps(pl, s)) return PKV_ERR_ALIAS;
    }
    if (q) {
        const bool in_place = q == q_out && q_stride == q_out_stride;
        if ((!in_place && rows_meet(qo, qi, n)) || rows_meet(qo, k, n) || rows_meet(qo, v, n))
            return PKV_ERR_ALIAS;
        for (const Range& s : small)
            if (overlaps(span(qo, n), s)) return PKV_ERR_ALIAS;
    }
    pkv::AppendTokensArgs a = {};
    a.q = q;
    a.k = k_new;
    a.v = v_new;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out_stride = q_out_stride;
    a.slots = slots;
    a.positions = rope ? positions : nullptr;
    a.n_tokens = n_tokens;
    a.n_q_heads = n_q_heads;
    a.n_kv_heads = pool->n_kv_heads;
    a.page_size = pool->page_size;
    a.n_slots = (long long)pool->num_pages * pool->page_size;
    a.k_pool = pool->k;
    a.v_pool = pool->v;
    a.q_out = q_out;
    a.q_norm = q_norm_weight;
    a.k_norm = k_norm_weight;
    a.eps = norm_eps;
    a.status = dev_status;
    if (rope) a.rope = *rope;
    return cuda_status(pkv::launch_append_tokens(a, pool->dtype == PKV_BF16, D,
                                                 reinterpret_cast<cudaStream_t>(stream)));
}

pkv_status kv_page_bounds(const pkv_pool* pool, const int64_t* slots, int n_tokens, void* bounds,
                          uint32_t* dev_status, pkv_stream stream) {
    if (!pool || n_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (pool->dtype == PKV_E4M3 || pool->n_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
    if (n_tokens == 0) return PKV_OK;
    if (!slots || !bounds) return PKV_ERR_INVALID_ARG;
    if (!aligned(slots, 8) || !aligned(bounds, 16) || !aligned(pool->k, 16) ||
        !aligned(dev_status, 4))
        return PKV_ERR_INVALID_ARG;
    const size_t bytes = (size_t)pool->num_pages * pool->n_kv_heads * 2 * pool->head_dim * 2;
    if (any_alias({{bounds, bytes}, {dev_status, 4}},
                  {{pool->k, pool_bytes(pool)}, {pool->v, pool_bytes(pool)},
                   {slots, (size_t)n_tokens * 8}}))
        return PKV_ERR_ALIAS;
    pkv::BoundsArgs a = {};
    a.k_pool = pool->k;
    a.slots = slots;
    a.n_tokens = n_tokens;
    a.n_kv_heads = pool->n_kv_heads;
    a.page_size = pool->page_size;
    a.n_slots = (long long)pool->num_pages * pool->page_size;
    a.bounds = bounds;
    a.status = dev_status;
    return cuda_status(pkv::launch_page_bounds(a, pool->dtype == PKV_BF16, pool->head_dim,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

pkv_status paged_select_workspace_size(int batch, int n_kv_heads, int table_stride,
                                       size_t* bytes) {
    if (!bytes) return PKV_ERR_INVALID_ARG;
    *bytes = 0;
    const pkv_status st = check_select(batch, n_kv_heads, table_stride);
    if (st == PKV_OK) *bytes = select_layout(batch, n_kv_heads, table_stride).total;
    return st;
}

pkv_status paged_select_pages(const void* q, const void* bounds, const int32_t* page_table,
                              int table_stride, const int32_t* context_lens, int batch,
                              int n_q_heads, int n_kv_heads, int head_dim, int page_size,
                              int num_pages, pkv_dtype dtype, int keep_first, int keep_last,
                              int max_pages, int32_t* selected, void* workspace, size_t ws_bytes,
                              uint32_t* dev_status, pkv_stream stream) {
    pkv_status st = check_shapes(batch, n_q_heads, n_kv_heads, head_dim, page_size, num_pages,
                                 table_stride, dtype);
    if (st != PKV_OK) return st;
    if (max_pages <= 0 || keep_first < 0 || keep_last < 0 ||
        (long long)keep_first + keep_last > max_pages)
        return PKV_ERR_INVALID_ARG;
    if ((st = check_select(batch, n_kv_heads, table_stride)) != PKV_OK) return st;
    if (n_q_heads / n_kv_heads > pkv::kMaxSelectGroup) return PKV_ERR_UNSUPPORTED;
    if (batch == 0) return PKV_OK;
    if (!q || !bounds || !page_table || !context_lens || !selected) return PKV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(bounds, 16) || !aligned(page_table, 4) ||
        !aligned(context_lens, 4) || !aligned(selected, 4) || !aligned(dev_status, 4))
        return PKV_ERR_INVALID_ARG;
    const SelectLayout w = select_layout(batch, n_kv_heads, table_stride);
    if (!workspace || !aligned(workspace, 256) || ws_bytes < w.total) return PKV_ERR_WORKSPACE;
    const size_t units = (size_t)batch * n_kv_heads;
    if (any_alias({{selected, units * max_pages * 4}, {workspace, w.total}, {dev_status, 4}},
                  {{q, (size_t)batch * n_q_heads * head_dim * 2},
                   {bounds, (size_t)num_pages * n_kv_heads * 2 * head_dim * 2},
                   {page_table, (size_t)batch * table_stride * 4},
                   {context_lens, (size_t)batch * 4}}))
        return PKV_ERR_ALIAS;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    pkv::SelectArgs a = {};
    a.q = q;
    a.bounds = bounds;
    a.table = page_table;
    a.table_stride = table_stride;
    a.lens = context_lens;
    a.batch = batch;
    a.n_q_heads = n_q_heads;
    a.n_kv_heads = n_kv_heads;
    a.page_size = page_size;
    a.num_pages = num_pages;
    a.keep_first = keep_first;
    a.keep_last = keep_last;
    a.max_pages = max_pages;
    a.selected = selected;
    a.keys64 = reinterpret_cast<unsigned long long*>(ws);
    a.scores = reinterpret_cast<float*>(ws + w.scores);
    a.stats = reinterpret_cast<uint4*>(ws + w.stats);
    a.status = dev_status;
    return cuda_status(pkv::launch_select(a, dtype == PKV_BF16, head_dim,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

pkv_status paged_decode_attention_selected(const void* q, const void* k_pool, const void* v_pool,
                                           const int32_t* page_table, int table_stride,
                                           const int32_t* context_lens, const int32_t* selected,
                                           int max_pages, int batch, int n_q_heads,
                                           int n_kv_heads, int head_dim, int page_size,
                                           int num_pages, pkv_dtype dtype, float scale, void* out,
                                           uint32_t* dev_status, pkv_stream stream) {
    pkv_status st = check_shapes(batch, n_q_heads, n_kv_heads, head_dim, page_size, num_pages,
                                 table_stride, dtype);
    if (st != PKV_OK) return st;
    if (max_pages <= 0 || !isfinite(scale)) return PKV_ERR_INVALID_ARG;
    const long long pool_rows = (long long)num_pages * n_kv_heads * page_size;
    if (pool_rows > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;  // 32-bit tensor row coordinate
    const int group = n_q_heads / n_kv_heads, head_blocks = (group + 15) / 16;
    // (eight CTAs of a unit at most)
    if ((long long)batch * n_kv_heads * head_blocks > 0x7fffffffLL / 8 ||
        (long long)max_pages * (page_size / 16) > 0x7fffffffLL)
        return PKV_ERR_UNSUPPORTED;
    if (batch == 0) return PKV_OK;
    if (!q || !k_pool || !v_pool || !page_table || !context_lens || !selected || !out)
        return PKV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(out, 16) ||
        !aligned(page_table, 4) || !aligned(context_lens, 4) || !aligned(selected, 4) ||
        !aligned(dev_status, 4))
        return PKV_ERR_INVALID_ARG;
    const size_t qo = (size_t)batch * n_q_heads * head_dim * 2;
    const size_t pool = (size_t)pool_rows * head_dim * 2;
    if (any_alias({{out, qo}, {dev_status, 4}},
                  {{q, qo},
                   {k_pool, pool},
                   {v_pool, pool},
                   {page_table, (size_t)batch * table_stride * 4},
                   {context_lens, (size_t)batch * 4},
                   {selected, (size_t)batch * n_kv_heads * max_pages * 4}}))
        return PKV_ERR_ALIAS;
    CUtensorMap km, vm;
    try {  // the maps are kept in a std::map
        st = pkv::pool_rows_map(k_pool, pool_rows, head_dim, dtype, &km);
        if (st == PKV_OK) st = pkv::pool_rows_map(v_pool, pool_rows, head_dim, dtype, &vm);
    } catch (...) {
        st = PKV_ERR_CUDA;
    }
    if (st != PKV_OK) return st;
    pkv::SelectedParams p = {};
    p.q = q;
    p.table = page_table;
    p.table_stride = table_stride;
    p.lens = context_lens;
    p.selected = selected;
    p.max_pages = max_pages;
    p.batch = batch;
    p.n_q_heads = n_q_heads;
    p.n_kv_heads = n_kv_heads;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.group = group;
    p.head_blocks = head_blocks;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.out = out;
    p.status = dev_status;
    return cuda_status(pkv::launch_selected(p, dtype == PKV_BF16, head_dim, km, vm,
                                            reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
