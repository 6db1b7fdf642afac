// rule_abi.hip -- the C ABI of the gated delta rule over whole sequences: argument checks, the
// workspace's layout, kernel selection.  Every check runs on the host before anything is enqueued.
#include <stdint.h>

#include "rule_common.hpp"

namespace {

using namespace gdn;

bool misaligned(const void* p, uintptr_t to = 16) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

constexpr int kMaxRuleBatch = 1 << 20, kMaxRuleHeads = 1 << 15;
constexpr int64_t kMaxGrid = 0x7fffffff;

int check_dims(const gdn_rule_dims* d) {
    if (!d) return GDN_ERR_NULL;
    if (d->io_dtype != GDN_F32 && d->io_dtype != GDN_BF16) return GDN_ERR_DTYPE;
    if (d->batch < 0 || d->batch > kMaxRuleBatch) return GDN_ERR_DIMS;
    if (d->h_k < 1 || d->h_v < 1 || d->h_v > kMaxRuleHeads || d->h_v % d->h_k != 0) return GDN_ERR_DIMS;
    if (d->d_k < 1 || d->d_k > kMaxHead || d->d_v < 1 || d->d_v > kMaxHead) return GDN_ERR_DIMS;
    return GDN_OK;
}

int padded_dk(const gdn_rule_dims* d) { return d->d_k <= 64 ? 64 : d->d_k <= 128 ? 128 : 256; }
int padded_dv(const gdn_rule_dims* d) { return (d->d_v + 31) / 32 * 32; }
int64_t chunk_slots(const gdn_rule_dims* d, int64_t rows) { return rows / kC + d->batch; }

// Sizes whose grids would pass what a launch takes, besides check_dims.
int check_sizes(const gdn_rule_dims* d, int64_t rows) {
    if (rows < 0 || rows > 0x7fffffffLL) return GDN_ERR_DIMS;
    if ((int64_t)d->batch * d->h_v * (padded_dv(d) / 16) > kMaxGrid / 512) return GDN_ERR_DIMS;
    return chunk_slots(d, rows) * 1024 > kMaxGrid ? GDN_ERR_DIMS : GDN_OK;
}

int check_rows(std::initializer_list<const gdn_attn_rows*> rows) {
    for (const gdn_attn_rows* r : rows)
        if (!r || !r->data) return GDN_ERR_NULL;
    for (const gdn_attn_rows* r : rows)
        if (r->row < 0 || r->head < 0) return GDN_ERR_DIMS;
    return GDN_OK;
}
int check_rows_at(std::initializer_list<const gdn_attn_rows*> rows, int io) {
    for (const gdn_attn_rows* r : rows)
        if (misaligned(r->data, io == GDN_F32 ? 4 : 2)) return GDN_ERR_ALIGN;
    return GDN_OK;
}

int check_floats(std::initializer_list<const void*> need, std::initializer_list<const void*> may) {
    for (const void* p : need)
        if (!p) return GDN_ERR_NULL;
    for (const void* p : need)
        if (misaligned(p)) return GDN_ERR_ALIGN;
    for (const void* p : may)
        if (misaligned(p)) return GDN_ERR_ALIGN;
    return GDN_OK;
}

// An output that is one of the inputs.
int check_alias(std::initializer_list<const void*> outs, std::initializer_list<const void*> ins) {
    for (const void* o : outs) {
        if (!o) continue;
        for (const void* i : ins)
            if (o == i) return GDN_ERR_ALIAS;   // o is not NULL here
        int same = 0;
        for (const void* p : outs) same += o == p;
        if (same > 1) return GDN_ERR_ALIAS;
    }
    return GDN_OK;
}

Rows rows_of(const gdn_attn_rows* r) { return Rows{(char*)r->data, r->row, r->head}; }

// Rows that can be read eight elements at a time, 16 bytes each.
int vectors(const gdn_attn_rows* r, int d, int io) {
    const int step = io == GDN_F32 ? 4 : 8;
    return d % 8 == 0 && r->row % step == 0 && r->head % step == 0 && !misaligned(r->data);
}

// Places the workspace's arrays from `at`; returns the bytes.
size_t place(RuleArgs& a, int io, int dkp, bool back, char* at) {
    const size_t planes = io == GDN_F32 ? 3 : 1, round = io == GDN_F32 ? 3 : 2, slots = a.n_slots;
    const size_t keys = slots * a.Hk, vals = slots * a.Hv;
    const size_t tile = planes * kC * dkp * 2, tri = (size_t)kTriFrags * kFrag;
    size_t used = 0;
    auto take = [&](auto& p, size_t bytes) {
        p = reinterpret_cast<std::remove_reference_t<decltype(p)>>(at + used);
        used += (bytes + 255) / 256 * 256;
    };
    take(a.kf, keys * tile);
    take(a.kt, keys * tile);
    take(a.tm, vals * kSum * tri);
    take(a.coef, vals * 3 * kC * sizeof(float));
    if (!back) {
        take(a.qf, keys * tile);
        take(a.ym, vals * round * tri);
        return used;
    }
    take(a.qt, keys * tile);
    take(a.tt, vals * kSum * tri);
    take(a.yt, vals * kSum * tri);
    take(a.gram, keys * 10 * 2 * 256 * sizeof(float));
    take(a.gam, vals * kC * sizeof(double));
    take(a.ht, vals * dkp * a.dvp * sizeof(float));
    take(a.dht, vals * dkp * a.dvp * sizeof(float));
    take(a.w, vals * kC * a.dvp * sizeof(float));
    take(a.dr, vals * kC * a.dvp * sizeof(float));
    const size_t slices = a.dvp / 16;
    take(a.pb, vals * slices * kC * sizeof(float));
    take(a.pe, vals * slices * kC * sizeof(float));
    take(a.pa, vals * slices * (dkp / 32) * 4 * sizeof(float));
    take(a.hs, vals * (dkp / 16) * kC * sizeof(float));
    take(a.zs, vals * 320 * sizeof(float));
    return used;
}

RuleArgs sizes_of(const gdn_rule_dims* d, int64_t rows) {
    RuleArgs a{};
    a.B = d->batch;
    a.Hk = d->h_k;
    a.Hv = d->h_v;
    a.group = d->h_v / d->h_k;
    a.dk = d->d_k;
    a.dv = d->d_v;
    a.dvp = padded_dv(d);
    a.T = rows;
    a.n_slots = (int)chunk_slots(d, rows);
    return a;
}

int status_of(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH; }

template <int IO>
hipError_t forward(const RuleArgs& a, int dkp, hipStream_t s) {
    return dkp == 64    ? rule_forward_launch<IO, 64>(a, s)
           : dkp == 128 ? rule_forward_launch<IO, 128>(a, s)
                        : rule_forward_launch<IO, 256>(a, s);
}
template <int IO>
hipError_t backward(const RuleArgs& a, int dkp, hipStream_t s) {
    return dkp == 64    ? rule_backward_launch<IO, 64>(a, s)
           : dkp == 128 ? rule_backward_launch<IO, 128>(a, s)
                        : rule_backward_launch<IO, 256>(a, s);
}

}  // namespace

extern "C" {

int gdn_rule_workspace_bytes(const gdn_rule_dims* dims, int64_t n_rows, int32_t backward_, size_t* bytes) {
    int rc = check_dims(dims);
    if (!rc) rc = check_sizes(dims, n_rows);
    if (rc) return rc;
    if (!bytes) return GDN_ERR_NULL;
    RuleArgs a = sizes_of(dims, n_rows);
    *bytes = place(a, dims->io_dtype, padded_dk(dims), backward_ != 0, nullptr);
    return GDN_OK;
}

int gdn_rule_forward(const gdn_rule_dims* dims, const int32_t* offsets, int64_t n_rows, const float* S0,
                     const gdn_attn_rows* q, const gdn_attn_rows* k, const gdn_attn_rows* v, const float* beta,
                     const float* g, const gdn_attn_rows* o, float* S_out, void* workspace, hipStream_t stream) {
    int rc = check_dims(dims);
    if (!rc) rc = check_sizes(dims, n_rows);
    if (rc) return rc;
    if (dims->batch == 0) return GDN_OK;
    const int io = dims->io_dtype;
    rc = check_floats({workspace}, {S0, S_out});
    if (!rc) rc = !offsets ? GDN_ERR_NULL : misaligned(offsets, 4) ? GDN_ERR_ALIGN : GDN_OK;
    if (!rc && n_rows > 0) {                         // tensors without rows may have no memory
        rc = check_rows({q, k, v, o});
        if (!rc) rc = check_floats({beta, g}, {});
        if (!rc) rc = check_rows_at({q, k, v, o}, io);
        if (!rc) rc = check_alias({o->data, S_out}, {q->data, k->data, v->data, beta, g});
        if (!rc) rc = check_alias({o->data}, {S0});
    }
    if (rc) return rc;
    RuleArgs a = sizes_of(dims, n_rows);
    a.offsets = offsets;
    if (n_rows > 0) {
        a.q = rows_of(q), a.k = rows_of(k), a.v = rows_of(v), a.o = rows_of(o);
        a.vq = vectors(q, a.dk, io), a.vk = vectors(k, a.dk, io), a.vo = vectors(o, 8, io);
    }
    a.beta = beta, a.g = g, a.S0 = S0, a.S_out = S_out;
    const int dkp = padded_dk(dims);
    place(a, io, dkp, false, (char*)workspace);
    return status_of(io == GDN_F32 ? forward<GDN_F32>(a, dkp, stream) : forward<GDN_BF16>(a, dkp, stream));
}

int gdn_rule_backward(const gdn_rule_dims* dims, const int32_t* offsets, int64_t n_rows, const float* S0,
                      const gdn_attn_rows* q, const gdn_attn_rows* k, const gdn_attn_rows* v, const float* beta,
                      const float* g, const gdn_attn_rows* d_o, const float* dS_out, const gdn_attn_rows* dq,
                      const gdn_attn_rows* dk, const gdn_attn_rows* dv, float* dbeta, float* dlog_g, float* dS0,
                      void* workspace, hipStream_t stream) {
    int rc = check_dims(dims);
    if (!rc) rc = check_sizes(dims, n_rows);
    if (rc) return rc;
    if (dims->batch == 0) return GDN_OK;
    const int io = dims->io_dtype;
    rc = check_floats({workspace}, {S0, dS_out, dS0});
    if (!rc) rc = !offsets ? GDN_ERR_NULL : misaligned(offsets, 4) ? GDN_ERR_ALIGN : GDN_OK;
    if (!rc && dS0 && dS0 == S0) rc = GDN_ERR_ALIAS;
    if (!rc && n_rows > 0) {
        rc = check_rows({q, k, v, d_o, dq, dk, dv});
        if (!rc) rc = check_floats({beta, g, dbeta, dlog_g}, {});
        if (!rc) rc = check_rows_at({q, k, v, d_o, dq, dk, dv}, io);
        if (!rc)
            rc = check_alias({dq->data, dk->data, dv->data, dbeta, dlog_g, dS0},
                             {q->data, k->data, v->data, d_o->data, beta, g});
        if (!rc) rc = check_alias({dq->data, dk->data, dv->data, dbeta, dlog_g}, {S0, dS_out});
    }
    if (rc) return rc;
    RuleArgs a = sizes_of(dims, n_rows);
    a.offsets = offsets;
    if (n_rows > 0) {
        a.q = rows_of(q), a.k = rows_of(k), a.v = rows_of(v), a.d_o = rows_of(d_o);
        a.dq = rows_of(dq), a.dk_out = rows_of(dk), a.dv_out = rows_of(dv);
        a.vq = vectors(q, a.dk, io), a.vk = vectors(k, a.dk, io), a.vdo = vectors(d_o, a.dv, io);
    }
    a.beta = beta, a.g = g, a.S0 = S0, a.dS_out = dS_out, a.dS0 = dS0, a.dbeta = dbeta, a.dlog_g = dlog_g;
    const int dkp = padded_dk(dims);
    place(a, io, dkp, true, (char*)workspace);
    return status_of(io == GDN_F32 ? backward<GDN_F32>(a, dkp, stream) : backward<GDN_BF16>(a, dkp, stream));
}

int gdn_rule_step(const gdn_rule_dims* dims, const int32_t* slot, int32_t n_slots, const gdn_attn_rows* q,
                  const gdn_attn_rows* k, const gdn_attn_rows* v, const float* beta, const float* g, float* state,
                  const gdn_attn_rows* o, hipStream_t stream) {
    int rc = check_dims(dims);
    if (rc) return rc;
    if (dims->batch > 65535 || n_slots < 0 || (!slot && n_slots < dims->batch)) return GDN_ERR_DIMS;
    if (dims->batch == 0) return GDN_OK;
    const int io = dims->io_dtype;
    rc = check_rows({q, k, v, o});
    if (!rc) rc = check_floats({beta, g, state}, {});
    if (!rc) rc = misaligned(slot, 4) ? GDN_ERR_ALIGN : GDN_OK;
    if (!rc) rc = check_rows_at({q, k, v, o}, io);
    if (!rc) rc = check_alias({o->data, state}, {q->data, k->data, v->data, beta, g});
    if (rc) return rc;
    RuleStepArgs a{dims->batch, dims->h_k, dims->h_v, dims->h_v / dims->h_k, dims->d_k, dims->d_v, n_slots, slot,
                   rows_of(q), rows_of(k), rows_of(v), rows_of(o), beta, g, state};
    return status_of(launch_rule_step(a, io, stream));
}

}  // extern "C"
