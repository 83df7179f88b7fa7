// Gradients of dense attention over states of another length on the CUDA cores,
// the plain way: one warp a query row (dq) or a key row (dk, dv), lane j holding
// the j-th of 32 keys (rows) for the scores and d/32 channels for the sums.
#include <math_constants.h>

#include "cross.cuh"

namespace bsa {
namespace {

constexpr int kWarps = 4;

template <int D>
__device__ __forceinline__ float dot_row(const float *a, const __nv_bfloat16 *b) {
    float s = 0.f;
    for (int c = 0; c < D; c += 2) {
        const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(b + c));
        s = fmaf(a[c], x.x, s);
        s = fmaf(a[c + 1], x.y, s);
    }
    return s;
}

// dq of one row: dq = s Σ_j p_j (dp_j - D) k_j
template <int D>
__global__ void dq_kernel(DenseProblem p, const __nv_bfloat16 *q, KeySet s, const __nv_bfloat16 *out, const float *lse,
                          const __nv_bfloat16 *dout, __nv_bfloat16 *dq, uint32_t *status) {
    __shared__ float qs[kWarps][D], os[kWarps][D];
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t row = (int64_t)blockIdx.x * kWarps + w;
    if (row >= p.batch * p.kv_heads * p.rows) return;
    const int64_t slab = row / p.rows, b = slab / p.kv_heads;
    float dt = 0.f, acc[D / 32];
    for (int e = 0; e < D / 32; ++e) {
        const int c = lane + 32 * e;
        acc[e] = 0.f;
        qs[w][c] = __bfloat162float(q[row * D + c]) * p.scale;
        os[w][c] = __bfloat162float(dout[row * D + c]);
        dt = fmaf(os[w][c], __bfloat162float(out[row * D + c]), dt);
    }
    for (int i = 16; i; i >>= 1) dt += __shfl_xor_sync(~0u, dt, i);
    __syncwarp();
    const int len = set_len(s.len, b, s.n, status);
    const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(s.k) + slab * s.n * D;
    const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(s.v) + slab * s.n * D;
    const float ls = lse[row];
    for (int j0 = 0; j0 < len; j0 += 32) {
        const int j = j0 + lane;
        float ds = 0.f;
        if (j < len) {
            const float x = dot_row<D>(qs[w], k + (int64_t)j * D), dp = dot_row<D>(os[w], v + (int64_t)j * D);
            ds = expf(x - ls) * (dp - dt);
        }
        const int cnt = min(32, len - j0);
        for (int jj = 0; jj < cnt; ++jj) {
            const float dj = __shfl_sync(~0u, ds, jj);
            for (int e = 0; e < D / 32; ++e)
                acc[e] = fmaf(dj, __bfloat162float(k[(int64_t)(j0 + jj) * D + lane + 32 * e]), acc[e]);
        }
    }
    for (int e = 0; e < D / 32; ++e) dq[row * D + lane + 32 * e] = __float2bfloat16_rn(acc[e] * p.scale);
}

// dk, dv of one key: dv = Σ_i p_i do_i, dk = s Σ_i p_i (dp_i - D_i) q_i
template <int D>
__global__ void dkv_kernel(DenseProblem p, const __nv_bfloat16 *q, KeySet s, const __nv_bfloat16 *out,
                           const float *lse, const __nv_bfloat16 *dout, __nv_bfloat16 *dk, __nv_bfloat16 *dv,
                           uint32_t *status) {
    __shared__ float ks[kWarps][D], vs[kWarps][D];
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t row = (int64_t)blockIdx.x * kWarps + w;
    if (row >= p.batch * p.kv_heads * s.n) return;
    const int64_t slab = row / s.n, b = slab / p.kv_heads;
    const int len = set_len(s.len, b, s.n, status);
    float ak[D / 32], av[D / 32];
    for (int e = 0; e < D / 32; ++e) ak[e] = av[e] = 0.f;
    if (row % s.n < len) {
        for (int c = lane; c < D; c += 32) {
            ks[w][c] = __bfloat162float(static_cast<const __nv_bfloat16 *>(s.k)[row * D + c]) * p.scale;
            vs[w][c] = __bfloat162float(static_cast<const __nv_bfloat16 *>(s.v)[row * D + c]);
        }
        __syncwarp();
        const int64_t r0 = slab * p.rows;
        for (int64_t i0 = 0; i0 < p.rows; i0 += 32) {
            const int64_t i = i0 + lane;
            float pr = 0.f, ds = 0.f;
            if (i < p.rows) {
                const __nv_bfloat16 *qi = q + (r0 + i) * D, *oi = dout + (r0 + i) * D, *yi = out + (r0 + i) * D;
                float dt = 0.f;
                for (int c = 0; c < D; ++c) dt = fmaf(__bfloat162float(oi[c]), __bfloat162float(yi[c]), dt);
                pr = expf(dot_row<D>(ks[w], qi) - lse[r0 + i]);
                ds = pr * (dot_row<D>(vs[w], oi) - dt);
            }
            const int cnt = (int)min((int64_t)32, p.rows - i0);
            for (int ii = 0; ii < cnt; ++ii) {
                const float pi = __shfl_sync(~0u, pr, ii), di = __shfl_sync(~0u, ds, ii);
                for (int e = 0; e < D / 32; ++e) {
                    const int64_t at = (r0 + i0 + ii) * D + lane + 32 * e;
                    av[e] = fmaf(pi, __bfloat162float(dout[at]), av[e]);
                    ak[e] = fmaf(di, __bfloat162float(q[at]), ak[e]);
                }
            }
        }
    }
    for (int e = 0; e < D / 32; ++e) {
        dk[row * D + lane + 32 * e] = __float2bfloat16_rn(ak[e] * p.scale);
        dv[row * D + lane + 32 * e] = __float2bfloat16_rn(av[e]);
    }
}

using bf = __nv_bfloat16;
unsigned ctas(int64_t rows) { return (unsigned)((rows + kWarps - 1) / kWarps); }

}  // namespace

cudaError_t launch_dense_bwd(const DenseProblem &p, const void *q, const KeySet &s, const void *out, const float *lse,
                             const void *dout, void *dq, void *dk, void *dv, uint32_t *status, cudaStream_t stream) {
    const int64_t rows = p.batch * p.kv_heads * p.rows, keys = p.batch * p.kv_heads * s.n;
    auto kq = p.d == 64 ? dq_kernel<64> : dq_kernel<128>;
    kq<<<ctas(rows), 32 * kWarps, 0, stream>>>(p, static_cast<const bf *>(q), s, static_cast<const bf *>(out), lse,
                                               static_cast<const bf *>(dout), static_cast<bf *>(dq), status);
    auto kk = p.d == 64 ? dkv_kernel<64> : dkv_kernel<128>;
    kk<<<ctas(keys), 32 * kWarps, 0, stream>>>(p, static_cast<const bf *>(q), s, static_cast<const bf *>(out), lse,
                                               static_cast<const bf *>(dout), static_cast<bf *>(dk),
                                               static_cast<bf *>(dv), status);
    return cudaGetLastError();
}

}  // namespace bsa
