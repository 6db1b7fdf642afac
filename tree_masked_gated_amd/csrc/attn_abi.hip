// attn_abi.hip -- the C ABI of the softmax-attention calls: argument checks, kernel
// selection, launches.  Every check runs on the host before anything is enqueued.
#include <math.h>
#include <stdint.h>

#include "attn_common.hpp"
#include "attn_verify.hpp"

namespace {

using namespace gdn;

bool misaligned(const void* p, uintptr_t to = 16) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Heads up to which the kernels' 32-bit piece counts (a row's pieces, times four rows or times a
// path of 1024) do not overflow, and 16-byte pieces of a page.
constexpr int kMaxHeadsQ = 1 << 20, kMaxHeadsKv = 1 << 13;
constexpr int64_t kMaxPagePieces = 1 << 30;

int check_dims(const gdn_attn_dims* d) {
    if (!d) return GDN_ERR_NULL;
    if (d->io_dtype != GDN_F32 && d->io_dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (d->batch < 0 || d->n_nodes < 1 || d->n_nodes > kMaxNodes) return GDN_ERR_DIMS;
    if (d->h_kv < 1 || d->h_q < 1 || d->h_q % d->h_kv != 0) return GDN_ERR_DIMS;
    if (d->h_q > kMaxHeadsQ || d->h_kv > kMaxHeadsKv) return GDN_ERR_DIMS;
    if (d->d < 8 || d->d > kMaxHead || d->d % 8 != 0) return GDN_ERR_DIMS;
    if ((int64_t)d->n_nodes * (d->h_q / d->h_kv) > 65536) return GDN_ERR_DIMS;
    return GDN_OK;
}

int elem(int io) { return io == GDN_F32 ? 4 : 2; }

// Strides: not negative, whole 16-byte pieces.
int check_strides(std::initializer_list<int64_t> strides, int io) {
    for (int64_t s : strides) {
        if (s < 0) return GDN_ERR_DIMS;
        if (s % (16 / elem(io)) != 0) return GDN_ERR_ALIGN;
    }
    return GDN_OK;
}

int check_rows(std::initializer_list<const gdn_attn_rows*> rows, int io) {
    for (const gdn_attn_rows* r : rows)
        if (!r || !r->data) return GDN_ERR_NULL;
    for (const gdn_attn_rows* r : rows) {
        if (misaligned(r->data)) return GDN_ERR_ALIGN;
        int rc = check_strides({r->row, r->head}, io);
        if (rc) return rc;
    }
    return GDN_OK;
}

int check_cache(const gdn_paged_cache* c) {
    if (!c || !c->k || !c->v) return GDN_ERR_NULL;
    if (c->io_dtype != GDN_F32 && c->io_dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (c->n_layers < 1 || c->n_pages < 1 || c->page_rows < 1 || c->page_rows > 65536 || c->h_kv < 1)
        return GDN_ERR_DIMS;
    if (c->d < 8 || c->d > kMaxHead || c->d % 8 != 0) return GDN_ERR_DIMS;
    if ((int64_t)c->page_rows * c->h_kv > kMaxPagePieces / (c->d * elem(c->io_dtype) / 16)) return GDN_ERR_DIMS;
    if (misaligned(c->k) || misaligned(c->v)) return GDN_ERR_ALIGN;
    return check_strides({c->k_layer, c->k_page, c->k_row, c->k_head, c->v_layer, c->v_page, c->v_row, c->v_head},
                         c->io_dtype);
}

// The cache against the dims of a call on one of its layers; a table without columns is never read.
int check_layer(const gdn_attn_dims* d, const gdn_paged_cache* c, int32_t layer, const int32_t* table,
                int32_t width) {
    int rc = check_cache(c);
    if (rc) return rc;
    if (c->io_dtype != d->io_dtype) return GDN_ERR_DTYPE;
    if (c->h_kv != d->h_kv || c->d != d->d || layer < 0 || layer >= c->n_layers || width < 0 || width > (1 << 20))
        return GDN_ERR_DIMS;
    if (!table && width > 0) return GDN_ERR_NULL;
    return misaligned(table) ? GDN_ERR_ALIGN : GDN_OK;
}

int check_offsets(const int32_t* offsets) { return misaligned(offsets, 4) ? GDN_ERR_ALIGN : GDN_OK; }

Rows rows_of(const gdn_attn_rows* r) { return Rows{(char*)r->data, r->row, r->head}; }

Pool key_pool(const gdn_paged_cache* c, int32_t layer) {
    return Pool{(char*)c->k + layer * c->k_layer * elem(c->io_dtype), c->k_page, c->k_row, c->k_head};
}
Pool value_pool(const gdn_paged_cache* c, int32_t layer) {
    return Pool{(char*)c->v + layer * c->v_layer * elem(c->io_dtype), c->v_page, c->v_row, c->v_head};
}

int check_pages(const gdn_page_dims* d) {
    if (!d) return GDN_ERR_NULL;
    if (d->n_pages < 1 || d->n_pages > (1 << 30) || d->page_rows < 1 || d->page_rows > 65536 || d->n_slots < 1 ||
        d->n_slots > 4096 || d->width < 1 || d->width > (1 << 20))
        return GDN_ERR_DIMS;
    return GDN_OK;
}

int check_ints(std::initializer_list<const int32_t*> ps) {
    for (const int32_t* p : ps)
        if (!p) return GDN_ERR_NULL;
    for (const int32_t* p : ps)
        if (misaligned(p)) return GDN_ERR_ALIGN;
    return GDN_OK;
}

int status_of(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH; }

}  // namespace

namespace gdn {

size_t attn_workspace(int B, int N, int Hq, int Hk, int d, int io) {
    const int g = Hq / Hk;
    if (io == GDN_F32)
        return d <= 64    ? attn_bytes_f32_64(B, N, g, Hk)
               : d <= 128 ? attn_bytes_f32_128(B, N, g, Hk)
                          : attn_bytes_f32_256(B, N, g, Hk);
    return d <= 64    ? attn_bytes_bf16_64(B, N, g, Hk)
           : d <= 128 ? attn_bytes_bf16_128(B, N, g, Hk)
                      : attn_bytes_bf16_256(B, N, g, Hk);
}

hipError_t launch_attn(const AttnArgs& a, int io, hipStream_t stream) {
    if (io == GDN_F32)
        return a.d <= 64    ? attn_launch_f32_64(a, stream)
               : a.d <= 128 ? attn_launch_f32_128(a, stream)
                            : attn_launch_f32_256(a, stream);
    return a.d <= 64    ? attn_launch_bf16_64(a, stream)
           : a.d <= 128 ? attn_launch_bf16_128(a, stream)
                        : attn_launch_bf16_256(a, stream);
}

}  // namespace gdn

extern "C" {

int gdn_attn_rope(const gdn_attn_dims* dims, const gdn_rope_dims* rope, const int32_t* offsets,
                  int64_t n_rows, const gdn_attn_rows* q, const gdn_attn_rows* k, const double* freq,
                  const int32_t* ctx, const int32_t* depth, const gdn_attn_rows* q_out,
                  const gdn_attn_rows* k_out, hipStream_t stream) {
    int rc = check_dims(dims);
    if (rc) return rc;
    if (!rope) return GDN_ERR_NULL;
    if (rope->rot < 2 || rope->rot > dims->d || rope->rot % 2 != 0 || !isfinite(rope->amp) ||
        (rope->layout != GDN_ROPE_HALF && rope->layout != GDN_ROPE_INTERLEAVED))
        return GDN_ERR_DIMS;
    if (n_rows < 0 || n_rows > 0x7fffffffLL) return GDN_ERR_DIMS;
    if (dims->batch == 0 || n_rows == 0) return GDN_OK;
    rc = check_rows({q, k, q_out, k_out}, dims->io_dtype);
    if (rc) return rc;
    if (!freq) return GDN_ERR_NULL;
    rc = check_ints({ctx, depth});
    if (rc) return rc;
    if (misaligned(freq)) return GDN_ERR_ALIGN;
    rc = check_offsets(offsets);
    if (rc) return rc;
    RopeArgs a{dims->batch, dims->n_nodes, dims->h_q, dims->h_kv, dims->d, rope->rot, rope->layout, rope->amp,
               n_rows, offsets, rows_of(q), rows_of(k), rows_of(q_out), rows_of(k_out), freq, ctx, depth};
    return status_of(launch_rope(a, dims->io_dtype, stream));
}

int gdn_attn_workspace_bytes(const gdn_attn_dims* dims, size_t* bytes) {
    int rc = check_dims(dims);
    if (rc) return rc;
    if (!bytes) return GDN_ERR_NULL;
    *bytes = dims->batch == 0 ? 0
                              : attn_workspace(dims->batch, dims->n_nodes, dims->h_q, dims->h_kv, dims->d,
                                               dims->io_dtype);
    return GDN_OK;
}

int gdn_attn_verify(const gdn_attn_dims* dims, const int32_t* offsets, const gdn_paged_cache* cache,
                    int32_t layer, const int32_t* table, int32_t width, const int32_t* ctx,
                    const gdn_attn_rows* q, const gdn_attn_rows* k, const gdn_attn_rows* v,
                    const uint32_t* anc_mask, const int32_t* tree_status, const gdn_attn_rows* o,
                    void* workspace, hipStream_t stream) {
    int rc = check_dims(dims);
    if (rc) return rc;
    if (!(dims->scale > 0.0f) || !isfinite(dims->scale)) return GDN_ERR_DIMS;
    if (dims->batch == 0) return GDN_OK;
    rc = check_layer(dims, cache, layer, table, width);
    if (rc) return rc;
    rc = check_rows({q, k, v, o}, dims->io_dtype);
    if (rc) return rc;
    rc = check_ints({ctx, (const int32_t*)anc_mask, tree_status});
    if (rc) return rc;
    if (!workspace) return GDN_ERR_NULL;
    if (misaligned(workspace)) return GDN_ERR_ALIGN;
    rc = check_offsets(offsets);
    if (rc) return rc;
    const int group = dims->h_q / dims->h_kv, es = elem(dims->io_dtype);
    auto rows_bytes = [es](const gdn_attn_rows* r) { return Rows{(char*)r->data, r->row * es, r->head * es}; };
    auto pool_bytes = [es](Pool p) { return Pool{p.p, p.page * es / 16, p.row * es / 16, p.head * es}; };
    for (int64_t x : {cache->k_page, cache->v_page, cache->k_row, cache->v_row})
        if (x / (16 / es) > 0xffffffffLL) return GDN_ERR_DIMS;
    AttnArgs a{dims->batch, dims->n_nodes, dims->h_q, dims->h_kv, group, dims->d, cache->n_pages, width,
               (dims->n_nodes + 31) / 32, dims->scale, fast_div(cache->page_rows), fast_div(group), offsets,
               pool_bytes(key_pool(cache, layer)), pool_bytes(value_pool(cache, layer)), rows_bytes(q), rows_bytes(k),
               rows_bytes(v), rows_bytes(o), table, ctx, anc_mask, tree_status, (char*)workspace};
    return status_of(launch_attn(a, dims->io_dtype, stream));
}

int gdn_attn_commit(const gdn_attn_dims* dims, const int32_t* offsets, const gdn_paged_cache* cache,
                    int32_t layer, const int32_t* table, int32_t width, const int32_t* ctx,
                    const gdn_attn_rows* k, const gdn_attn_rows* v, const int32_t* path,
                    const int32_t* path_len, int32_t* new_len, hipStream_t stream) {
    int rc = check_dims(dims);
    if (rc) return rc;
    if (dims->batch == 0) return GDN_OK;
    rc = check_layer(dims, cache, layer, table, width);
    if (rc) return rc;
    rc = check_rows({k, v}, dims->io_dtype);
    if (rc) return rc;
    rc = check_ints({ctx, path, path_len, new_len});
    if (rc) return rc;
    rc = check_offsets(offsets);
    if (rc) return rc;
    if (new_len == ctx || new_len == path_len) return GDN_ERR_ALIAS;
    AppendArgs a{dims->batch, dims->n_nodes, dims->h_kv, dims->d, cache->n_pages, width,
                 fast_div(cache->page_rows), offsets, key_pool(cache, layer), value_pool(cache, layer), rows_of(k),
                 rows_of(v), table, ctx, path, path_len, new_len};
    return status_of(launch_append(a, dims->io_dtype, stream));
}

int gdn_pages_fork(const gdn_page_dims* dims, int32_t n, const int32_t* src_seq, const int32_t* dst_seq,
                   int32_t* ref, int32_t* table, int32_t* held, int32_t* length, int32_t* status,
                   hipStream_t stream) {
    int rc = check_pages(dims);
    if (rc) return rc;
    if (n < 0) return GDN_ERR_DIMS;
    if (n == 0) return GDN_OK;
    rc = check_ints({src_seq, dst_seq, ref, table, held, length, status});
    if (rc) return rc;
    PageArgs a{dims->n_pages, dims->page_rows, dims->n_slots, dims->width, ref, table, held, length};
    return status_of(launch_pages_fork(a, n, src_seq, dst_seq, status, stream));
}

int gdn_pages_reserve(const gdn_page_dims* dims, const int32_t* need, int32_t* ref, int32_t* table,
                      int32_t* held, const int32_t* length, int32_t* src, int32_t* dst, int32_t* count,
                      int32_t* status, hipStream_t stream) {
    int rc = check_pages(dims);
    if (rc) return rc;
    rc = check_ints({need, ref, table, held, length, src, dst, count, status});
    if (rc) return rc;
    PageArgs a{dims->n_pages, dims->page_rows, dims->n_slots, dims->width, ref, table, held,
               const_cast<int32_t*>(length)};
    return status_of(launch_pages_reserve(a, need, src, dst, count, status, stream));
}

int gdn_pages_copy(const gdn_paged_cache* cache, int32_t n, const int32_t* src, const int32_t* dst,
                   const int32_t* count, hipStream_t stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    if (n < 0) return GDN_ERR_DIMS;
    if (n == 0) return GDN_OK;
    rc = check_ints({src, dst, count});
    if (rc) return rc;
    CopyArgs a{n, cache->n_pages, cache->n_layers, cache->page_rows, cache->h_kv, cache->d, key_pool(cache, 0),
               value_pool(cache, 0), cache->k_layer, cache->v_layer, src, dst, count};
    return status_of(launch_pages_copy(a, cache->io_dtype, stream));
}

int gdn_pages_free(const gdn_page_dims* dims, const int32_t* drop, int32_t* ref, int32_t* table,
                   int32_t* held, int32_t* length, hipStream_t stream) {
    int rc = check_pages(dims);
    if (rc) return rc;
    rc = check_ints({drop, ref, table, held, length});
    if (rc) return rc;
    PageArgs a{dims->n_pages, dims->page_rows, dims->n_slots, dims->width, ref, table, held, length};
    return status_of(launch_pages_free(a, drop, stream));
}

int gdn_pages_compact(const gdn_page_dims* dims, int32_t n, int32_t* ref, int32_t* table,
                      const int32_t* held, int32_t* src, int32_t* dst, int32_t* count, int32_t* remap,
                      hipStream_t stream) {
    int rc = check_pages(dims);
    if (rc) return rc;
    if (n < 1) return GDN_ERR_DIMS;
    rc = check_ints({ref, table, held, src, dst, count, remap});
    if (rc) return rc;
    PageArgs a{dims->n_pages, dims->page_rows, dims->n_slots, dims->width, ref, table,
               const_cast<int32_t*>(held), nullptr};
    return status_of(launch_pages_compact(a, n, src, dst, count, remap, stream));
}

}  // extern "C"
