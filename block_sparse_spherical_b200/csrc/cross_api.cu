// C ABI of cross attention, its backward and shared-prefix attention (declared
// in include/bsa.h): argument validation, workspace layout and dispatch. No
// allocation, no synchronisation, no state beyond the driver's entry point for
// tensor maps and a note of the devices on which a kernel has been set up.
#include <math.h>

#include "bsa_testing.h"
#include "cross.cuh"

namespace {

using bsa::DenseProblem;
using bsa::KeySet;

constexpr int64_t kMaxRows = 0x7fffff00LL;   // row coordinates are int32, tiles round up

bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

bsa_status make_dense(int32_t batch, int32_t heads, int32_t kv_heads, int32_t n_q, int32_t head_dim, int32_t dtype,
                      float scale, DenseProblem *p) {
    if (batch < 1 || heads < 1 || kv_heads < 1 || n_q < 1 || head_dim < 1 || heads % kv_heads != 0)
        return BSA_ERR_INVALID_ARG;
    if (dtype != BSA_F32 && dtype != BSA_BF16) return BSA_ERR_INVALID_ARG;
    if (!(scale >= 0.0f) || isinf(scale)) return BSA_ERR_INVALID_ARG;
    if (dtype != BSA_BF16 || (head_dim != 64 && head_dim != 128)) return BSA_ERR_UNSUPPORTED;
    p->batch = batch;
    p->heads = heads;
    p->kv_heads = kv_heads;
    p->n_q = n_q;
    p->d = head_dim;
    p->rows = (int64_t)(heads / kv_heads) * n_q;
    p->scale = scale > 0.0f ? scale : 1.0f / sqrtf((float)head_dim);
    // slabs are a TMA coordinate; rows of a slab too
    if (p->rows > kMaxRows || (int64_t)batch * kv_heads > kMaxRows) return BSA_ERR_UNSUPPORTED;
    return BSA_OK;
}

bsa_status make_cross(const bsa_cross_config *c, DenseProblem *p) {
    if (!c || c->n_k < 1) return BSA_ERR_INVALID_ARG;
    const bsa_status st = make_dense(c->batch, c->heads, c->kv_heads, c->n_q, c->head_dim, c->dtype, c->scale, p);
    return st != BSA_OK ? st : (c->n_k > kMaxRows ? BSA_ERR_UNSUPPORTED : BSA_OK);
}

bsa_status make_prefix(const bsa_prefix_config *c, DenseProblem *p) {
    if (!c || c->n_prefix < 1 || c->n_own < 1 || c->groups < 1) return BSA_ERR_INVALID_ARG;
    if (c->batch < 1 || c->batch % c->groups != 0) return BSA_ERR_INVALID_ARG;
    const bsa_status st = make_dense(c->batch, c->heads, c->kv_heads, c->n_q, c->head_dim, c->dtype, c->scale, p);
    return st != BSA_OK ? st : (c->n_prefix > kMaxRows || c->n_own > kMaxRows ? BSA_ERR_UNSUPPORTED : BSA_OK);
}

bsa_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return BSA_OK;
    return e == cudaErrorNotSupported ? BSA_ERR_UNSUPPORTED : BSA_ERR_CUDA;
}

bsa_status check_workspace(const void *workspace, size_t have, size_t need) {
    if (need == 0) return BSA_OK;
    if (!workspace || have < need) return BSA_ERR_WORKSPACE;
    return aligned(workspace, 256) ? BSA_OK : BSA_ERR_ALIGNMENT;
}

// The memory of a call's arguments. Whatever a kernel writes may meet nothing else of the call: tiles are read and
// rows written in no fixed order.
struct Extent {
    const void *at;         // null: not given
    size_t bytes;
};
template <size_t N, size_t M> bool apart(const Extent (&written)[N], const Extent (&read)[M]) {
    auto meet = [](const Extent &a, const Extent &b) {
        const uintptr_t x = (uintptr_t)a.at, y = (uintptr_t)b.at;
        return x && y && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
    };
    for (size_t i = 0; i < N; ++i) {
        for (size_t j = i + 1; j < N; ++j)
            if (meet(written[i], written[j])) return false;
        for (const Extent &r : read)
            if (meet(written[i], r)) return false;
    }
    return true;
}
// Bytes of the query rows' tensors and of a set's keys.
size_t q_bytes(const DenseProblem &p) { return (size_t)(p.batch * p.kv_heads * p.rows * p.d) * 2; }
size_t set_bytes(const DenseProblem &p, const KeySet &s) { return (size_t)(s.sets * p.kv_heads * s.n * p.d) * 2; }
size_t len_bytes(const KeySet &s) { return (size_t)s.sets * 4; }

KeySet cross_set(const bsa_cross_config *c, const void *k, const void *v, const int32_t *len) {
    return KeySet{k, v, len, c->n_k, c->batch, 1};
}
void prefix_sets(const bsa_prefix_config *c, const void *kp, const void *vp, const int32_t *plen, const void *ko,
                 const void *vo, const int32_t *olen, KeySet *sets) {
    sets[0] = KeySet{kp, vp, plen, c->n_prefix, c->groups, c->batch / c->groups};
    sets[1] = KeySet{ko, vo, olen, c->n_own, c->batch, 1};
}
// With or without lengths alike: a pass without lengths needs at least what one with lengths does.
size_t fwd_bytes(const DenseProblem &p, const KeySet *sets, int nsets) {
    size_t floats = 0;
    for (int k = 0; k < nsets; ++k) {
        KeySet full = sets[k];
        full.len = nullptr;
        floats += bsa::fwd_layout_of(bsa::make_fwd_plan(p, full), p.d, nsets == 2).total;
    }
    return floats * sizeof(float);
}
size_t bwd_bytes(const DenseProblem &p, KeySet s) {
    s.len = nullptr;
    return bsa::dense_bwd_floats(p, s) * sizeof(float);
}

// The calls; `withhold`: a test hook (cross.cuh), -1 for the library's own.
bsa_status cross_forward(const bsa_cross_config *cfg, const void *q, const void *k, const void *v,
                         const int32_t *key_len, void *out, float *lse, void *out_low, void *workspace,
                         size_t workspace_bytes, uint32_t *status_word, cudaStream_t stream, int64_t withhold) {
    DenseProblem p;
    const bsa_status st = make_cross(cfg, &p);
    if (st != BSA_OK) return st;
    p.withhold = withhold;
    if (!q || !k || !v || !out) return BSA_ERR_INVALID_ARG;
    for (const void *x : {q, k, v})
        if (x == out || x == out_low) return BSA_ERR_INVALID_ARG;
    if (out_low == out) return BSA_ERR_INVALID_ARG;
    const KeySet s = cross_set(cfg, k, v, key_len);
    const size_t need = fwd_bytes(p, &s, 1);
    const bsa_status ws = check_workspace(workspace, workspace_bytes, need);
    if (ws != BSA_OK) return ws;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(out_low, 16) || !aligned(key_len, 4) || !aligned(status_word, 4))
        return BSA_ERR_ALIGNMENT;
    const size_t rows = q_bytes(p), keys = set_bytes(p, s);
    if (!apart({{out, rows}, {out_low, rows}, {lse, rows / p.d * 2}, {workspace, need}, {status_word, 4}},
               {{q, rows}, {k, keys}, {v, keys}, {key_len, len_bytes(s)}}))
        return BSA_ERR_INVALID_ARG;
    return from_cuda(bsa::launch_dense_fwd(p, q, &s, 1, out, out_low, lse, static_cast<float *>(workspace), status_word, stream));
}

bsa_status cross_backward(const bsa_cross_config *cfg, const void *q, const void *k, const void *v,
                          const int32_t *key_len, const void *out, const float *lse, const void *out_low,
                          const void *dout, void *dq, void *dk, void *dv, void *workspace, size_t workspace_bytes,
                          uint32_t *status_word, cudaStream_t stream, int64_t withhold) {
    DenseProblem p;
    const bsa_status st = make_cross(cfg, &p);
    if (st != BSA_OK) return st;
    p.withhold = withhold;
    const void *in[] = {q, k, v, out, dout, lse};
    void *grads[] = {dq, dk, dv};
    for (const void *x : in)
        if (!x) return BSA_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i) {
        if (!grads[i] || grads[i] == grads[(i + 1) % 3]) return BSA_ERR_INVALID_ARG;
        for (const void *x : in)
            if (x == grads[i]) return BSA_ERR_INVALID_ARG;
        if (grads[i] == out_low) return BSA_ERR_INVALID_ARG;
    }
    const KeySet s = cross_set(cfg, k, v, key_len);
    const size_t need = bwd_bytes(p, s);
    const bsa_status ws = check_workspace(workspace, workspace_bytes, need);
    if (ws != BSA_OK) return ws;
    for (int i = 0; i < 5; ++i)
        if (!aligned(in[i], 16)) return BSA_ERR_ALIGNMENT;
    if (!aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(out_low, 16) || !aligned(lse, 4) || !aligned(key_len, 4) ||
        !aligned(status_word, 4))
        return BSA_ERR_ALIGNMENT;
    const size_t rows = q_bytes(p), keys = set_bytes(p, s);
    if (!apart({{dq, rows}, {dk, keys}, {dv, keys}, {workspace, need}, {status_word, 4}},
               {{q, rows}, {k, keys}, {v, keys}, {key_len, len_bytes(s)}, {out, rows}, {lse, rows / p.d * 2}, {out_low, rows}, {dout, rows}}))
        return BSA_ERR_INVALID_ARG;
    return from_cuda(bsa::launch_dense_bwd(p, q, s, out, out_low, lse, dout, dq, dk, dv, static_cast<float *>(workspace), status_word,
                                           stream));
}

bsa_status prefix_forward(const bsa_prefix_config *cfg, const void *q, const void *k_prefix, const void *v_prefix,
                          const int32_t *prefix_len, const void *k_own, const void *v_own, const int32_t *own_len,
                          void *out, void *workspace, size_t workspace_bytes, uint32_t *status_word,
                          cudaStream_t stream, int64_t withhold) {
    DenseProblem p;
    const bsa_status st = make_prefix(cfg, &p);
    if (st != BSA_OK) return st;
    p.withhold = withhold;
    const void *in[] = {q, k_prefix, v_prefix, k_own, v_own};
    for (const void *x : in)
        if (!x || x == out) return BSA_ERR_INVALID_ARG;
    if (!out) return BSA_ERR_INVALID_ARG;
    KeySet sets[2];
    prefix_sets(cfg, k_prefix, v_prefix, prefix_len, k_own, v_own, own_len, sets);
    const size_t need = fwd_bytes(p, sets, 2);
    const bsa_status ws = check_workspace(workspace, workspace_bytes, need);
    if (ws != BSA_OK) return ws;
    for (const void *x : in)
        if (!aligned(x, 16)) return BSA_ERR_ALIGNMENT;
    if (!aligned(out, 16) || !aligned(prefix_len, 4) || !aligned(own_len, 4) || !aligned(status_word, 4))
        return BSA_ERR_ALIGNMENT;
    const size_t rows = q_bytes(p), shared = set_bytes(p, sets[0]), own = set_bytes(p, sets[1]);
    if (!apart({{out, rows}, {workspace, need}, {status_word, 4}},
               {{q, rows}, {k_prefix, shared}, {v_prefix, shared}, {prefix_len, len_bytes(sets[0])}, {k_own, own}, {v_own, own},
                {own_len, len_bytes(sets[1])}}))
        return BSA_ERR_INVALID_ARG;
    return from_cuda(
        bsa::launch_dense_fwd(p, q, sets, 2, out, nullptr, nullptr, static_cast<float *>(workspace), status_word, stream));
}

}  // namespace

extern "C" {

bsa_status bsa_cross_workspace_size(const bsa_cross_config *cfg, size_t *bytes) {
    DenseProblem p;
    const bsa_status st = make_cross(cfg, &p);
    if (st != BSA_OK) return st;
    if (!bytes) return BSA_ERR_INVALID_ARG;
    const KeySet s = cross_set(cfg, nullptr, nullptr, nullptr);
    *bytes = fwd_bytes(p, &s, 1);
    return BSA_OK;
}

bsa_status bsa_cross_attention(const bsa_cross_config *cfg, const void *q, const void *k, const void *v,
                               const int32_t *key_len, void *out, float *lse, void *out_low, void *workspace,
                               size_t workspace_bytes, uint32_t *status_word, cudaStream_t stream) {
    return cross_forward(cfg, q, k, v, key_len, out, lse, out_low, workspace, workspace_bytes, status_word, stream, -1);
}

bsa_status bsa_cross_backward_workspace_size(const bsa_cross_config *cfg, size_t *bytes) {
    DenseProblem p;
    const bsa_status st = make_cross(cfg, &p);
    if (st != BSA_OK) return st;
    if (!bytes) return BSA_ERR_INVALID_ARG;
    *bytes = bwd_bytes(p, cross_set(cfg, nullptr, nullptr, nullptr));
    return BSA_OK;
}

bsa_status bsa_cross_attention_backward(const bsa_cross_config *cfg, const void *q, const void *k, const void *v,
                                        const int32_t *key_len, const void *out, const float *lse, const void *out_low,
                                        const void *dout, void *dq, void *dk, void *dv, void *workspace,
                                        size_t workspace_bytes, uint32_t *status_word, cudaStream_t stream) {
    return cross_backward(cfg, q, k, v, key_len, out, lse, out_low, dout, dq, dk, dv, workspace, workspace_bytes, status_word, stream, -1);
}

bsa_status bsa_prefix_workspace_size(const bsa_prefix_config *cfg, size_t *bytes) {
    DenseProblem p;
    const bsa_status st = make_prefix(cfg, &p);
    if (st != BSA_OK) return st;
    if (!bytes) return BSA_ERR_INVALID_ARG;
    KeySet sets[2];
    prefix_sets(cfg, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, sets);
    *bytes = fwd_bytes(p, sets, 2);
    return BSA_OK;
}

bsa_status bsa_prefix_attention(const bsa_prefix_config *cfg, const void *q, const void *k_prefix, const void *v_prefix,
                                const int32_t *prefix_len, const void *k_own, const void *v_own, const int32_t *own_len,
                                void *out, void *workspace, size_t workspace_bytes, uint32_t *status_word,
                                cudaStream_t stream) {
    return prefix_forward(cfg, q, k_prefix, v_prefix, prefix_len, k_own, v_own, own_len, out, workspace, workspace_bytes, status_word, stream, -1);
}

// Test hooks (include/bsa_testing.h): the same with a copy withheld, so that bounded waits expire on purpose.

bsa_status bsa_testing_cross_attention_withhold(const bsa_cross_config *cfg, const void *q, const void *k, const void *v,
                                                const int32_t *key_len, void *out, float *lse, void *out_low,
                                                void *workspace, size_t workspace_bytes, uint32_t *status_word,
                                                cudaStream_t stream, int64_t withhold) {
    if (!status_word || withhold < 0) return BSA_ERR_INVALID_ARG;
    return cross_forward(cfg, q, k, v, key_len, out, lse, out_low, workspace, workspace_bytes, status_word, stream, withhold);
}

bsa_status bsa_testing_cross_attention_backward_withhold(const bsa_cross_config *cfg, const void *q, const void *k,
                                                         const void *v, const int32_t *key_len, const void *out,
                                                         const float *lse, const void *out_low, const void *dout,
                                                         void *dq, void *dk, void *dv, void *workspace,
                                                         size_t workspace_bytes, uint32_t *status_word,
                                                         cudaStream_t stream, int64_t withhold) {
    if (!status_word || withhold < 0) return BSA_ERR_INVALID_ARG;
    return cross_backward(cfg, q, k, v, key_len, out, lse, out_low, dout, dq, dk, dv, workspace, workspace_bytes, status_word, stream, withhold);
}

bsa_status bsa_testing_prefix_attention_withhold(const bsa_prefix_config *cfg, const void *q, const void *k_prefix,
                                                 const void *v_prefix, const int32_t *prefix_len, const void *k_own,
                                                 const void *v_own, const int32_t *own_len, void *out, void *workspace,
                                                 size_t workspace_bytes, uint32_t *status_word, cudaStream_t stream,
                                                 int64_t withhold) {
    if (!status_word || withhold < 0) return BSA_ERR_INVALID_ARG;
    return prefix_forward(cfg, q, k_prefix, v_prefix, prefix_len, k_own, v_own, own_len, out, workspace, workspace_bytes, status_word, stream, withhold);
}

}  // extern "C"
