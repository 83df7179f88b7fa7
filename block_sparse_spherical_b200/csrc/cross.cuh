// Shared declarations of the dense attention over states of another length
// (cross attention, its backward, and attention over a shared prefix).
#pragma once

#include "bsa_internal.cuh"

namespace bsa {

// One set of keys for the rows of a forward pass. The rows of a slab are
// (member, head of the key head's group, query) with `rows` = (heads /
// kv_heads)·n_q rows a member, which [B][H][n_q][d] keeps contiguous; the
// members of one set share its keys.
struct KeySet {
    const void *k, *v;      // [sets][kv_heads][n][d] bf16
    const int32_t *len;     // [sets], nullable
    int64_t n;              // keys of a set
    int64_t sets;           // batch / members
    int64_t members;        // batch entries that share a set
};

struct DenseProblem {
    int64_t batch, heads, kv_heads, n_q, d;
    int64_t rows;           // (heads / kv_heads) * n_q: rows of a batch entry and key head
    float scale;
};

// Launchers (return cudaGetLastError()). s1.k may be null: one set of keys.
cudaError_t launch_dense_fwd(const DenseProblem &p, const void *q, const KeySet &s0, const KeySet &s1, void *out,
                             float *lse, uint32_t *status, cudaStream_t stream);
cudaError_t launch_dense_bwd(const DenseProblem &p, const void *q, const KeySet &s, const void *out, const float *lse,
                             const void *dout, void *dq, void *dk, void *dv, uint32_t *status, cudaStream_t stream);

}  // namespace bsa
