// Backward of dense softmax attention to states of another length on the sm_100a
// tensor cores (bf16, head_dim D = 64 or 128, fp32 accumulation).
//
// With the forward's row log-sum-exp and D_i = dout_i·out_i (a row pass ahead):
//   s_ij = q_i·k_j,  p_ij = exp(c s_ij - lse_i),  dp_ij = dout_i·v_j,
//   ds_ij = p_ij (dp_ij - D_i),
//   dv_j = Σ_i p_ij dout_i,  dk_j = c Σ_i ds_ij q_i,  dq_i = c Σ_j ds_ij k_j.
// Two passes, each with its sums in tensor memory, so that no gradient is reduced
// through atomics and all are the same from call to call; the second recomputes s
// and dp (7 products a pair of tiles where one pass would need 5 and an fp32
// reduction of dq through L2 in an order that changes).
//
// Key-major (dk, dv): a unit is a tile of 128 keys, a step 64 query rows.
//   Sᵀ = K·Qᵀ, dPᵀ = V·dOᵀ (M = 128 keys, N = 64) into tensor memory; a thread owns a key:
//   Pᵀ and dSᵀ as bf16 pairs back into tensor memory, the A operands of
//   dV += Pᵀ·dO and dK += dSᵀ·Q, so nothing passes through shared memory.
//   Two groups of 128 threads take alternate steps; one warp issues Sᵀ and dPᵀ, another
//   dV and dK (one thread alone does not issue such small MMAs fast enough).
// Query-major (dq): a unit is two tiles of 128 query rows, one a pipeline; a step 64 keys.
//   S = Q·Kᵀ, dP = dO·Vᵀ, dS into tensor memory, dQ += dS·K. The pipelines share K and V.
//
// Both deal their steps to the CTAs in equal shares; a unit cut between CTAs leaves fp32
// parts, which a last kernel adds in the order of the CTAs.
//
// Keys behind a length: their p and ds are set to 0 (whatever K and V hold); the copy
// warp of the query-major pass zeroes those rows of K, since 0·NaN is NaN. Query rows
// behind the last are filled with zeros by the copy and have lse = +inf, so p = 0.
//
// Every wait on an mbarrier is bounded (2 s), as in the forward.
#include <math_constants.h>

#include "cross.cuh"
#include "cross_tc.cuh"

namespace bsa {
namespace {

using namespace tc;

constexpr int NTHREADS = 384;
constexpr int kCtrlRegs = 72, kSoftRegs = 216;
constexpr int kRegsNeeded = 128 * kCtrlRegs + 256 * kSoftRegs;
static_assert(kRegsNeeded <= 65536, "register split");
constexpr int kSub = 64;                    // query rows (key-major) or keys (query-major) of a step
constexpr int kStat = 2 * kSub;             // floats of a query tile's statistics: lse·log2 e, then D

struct BwdParams {
    FwdPlan plan;           // key-major: s.fixed query tiles a unit; query-major: as a forward's
    const float *stat;      // [slabs][query tiles of 64][2][64]
    int64_t qtiles;         // query tiles of 64 rows a slab
    __nv_bfloat16 *dq, *dk, *dv;
    float *part;            // key-major [2 ctas][128][2][D] (dv, dk), query-major [2 ctas][256][D]
    float scale, scale_log2;
    uint32_t *status;
};
struct BwdMaps {
    CUtensorMap q, o, k, v; // boxes of 128 rows for the side that is a unit, 64 for the other
};

// ---------------------------------------------------------------- statistics

// Per query row lse·log2 e (+inf for rows without keys or behind the last: p = 0) and D = dout·out;
// and zeros for the gradients of keys behind a length. D/8 lanes a row, 16 bytes each.
template <int D>
__global__ void __launch_bounds__(256) bwd_stat_kernel(const __grid_constant__ BwdParams p, const __nv_bfloat16 *out,
                                                       const float *lse, const __nv_bfloat16 *dout, float *stat,
                                                       int64_t slabs) {
    constexpr int L = D / 8;
    const int sub = threadIdx.x % L;
    const int64_t rows = p.qtiles * kSub, step = (int64_t)gridDim.x * blockDim.x / L;
    const int64_t n_all = (slabs * rows + 31) / 32 * 32;     // whole warps stay together for the shuffles
    for (int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / L; i < n_all; i += step) {
        const int64_t slab = i / rows, r = i - slab * rows;
        const bool there = slab < slabs && r < p.plan.rows;
        float d = 0.f, x = CUDART_INF_F;
        if (there) {
            const int64_t at = slab * p.plan.rows + r;
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(out + at * D) + sub);
            const uint4 b = __ldg(reinterpret_cast<const uint4 *>(dout + at * D) + sub);
            const uint32_t ua[4] = {a.x, a.y, a.z, a.w}, ub[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                d = fmaf(__uint_as_float(ua[e] << 16), __uint_as_float(ub[e] << 16), d);
                d = fmaf(__uint_as_float(ua[e] & 0xffff0000u), __uint_as_float(ub[e] & 0xffff0000u), d);
            }
            x = __ldg(lse + at) * 1.4426950408889634f;
            if (x == -CUDART_INF_F) x = CUDART_INF_F;
        }
#pragma unroll
        for (int o = L / 2; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        if (sub == 0 && slab < slabs) {
            float *s = stat + (slab * p.qtiles + r / kSub) * kStat + r % kSub;
            s[0] = x;
            s[kSub] = x == CUDART_INF_F ? 0.f : d;
        }
    }
    const FwdSet &s = p.plan.s;
    if (!s.len) return;
    for (int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / L; i < slabs * s.n; i += step) {
        const int64_t slab = i / s.n;
        if (i - slab * s.n < set_len(s.len, slab / p.plan.kv_heads, s.n, nullptr)) continue;
        reinterpret_cast<uint4 *>(p.dk + i * D)[sub] = make_uint4(0u, 0u, 0u, 0u);
        reinterpret_cast<uint4 *>(p.dv + i * D)[sub] = make_uint4(0u, 0u, 0u, 0u);
    }
}

// ---------------------------------------------------------------- key-major: dk, dv

template <int D> struct KeyCfg {
    static constexpr int HALVES = D / 64;
    static constexpr int UNIT = kTile * D * 2;         // bytes of a K or V tile
    static constexpr int STEP = kSub * D * 2;          // bytes of a Q or dO tile
    static constexpr int STAGES = D == 64 ? 7 : 3;
};
template <int D> struct alignas(1024) KeyShared {
    uint8_t k[2][KeyCfg<D>::UNIT], v[2][KeyCfg<D>::UNIT];
    uint8_t q[KeyCfg<D>::STAGES][KeyCfg<D>::STEP], o[KeyCfg<D>::STAGES][KeyCfg<D>::STEP];
    float stat[KeyCfg<D>::STAGES][kStat];
    uint64_t kv_full[2], kv_empty[2], st_full[KeyCfg<D>::STAGES], st_empty[KeyCfg<D>::STAGES];
    uint64_t s_full[2], s_free[2], p_full[2], g_done[2], acc_full, acc_free, drain[2];
    int64_t first, last;
    StepAt at;
    uint32_t tmem_base;
    int abort_flag;
};
struct KeyChunk {
    int64_t slab;
    int tile, t0, nt, slot, valid;   // key tile, its query tiles [t0, t0 + nt), valid keys
};
struct KeyWalk {
    int64_t z, uu, left;
    int t;
};
template <int D> __device__ __forceinline__ KeyWalk key_begin(const BwdParams &p, const KeyShared<D> &sh) {
    KeyWalk w;
    if (p.plan.stream) {
        w.z = sh.at.z;
        w.uu = sh.at.uu;
        w.t = sh.at.t;
        w.left = sh.last - sh.first;
    } else {
        w.left = blockIdx.x;
    }
    return w;
}
__device__ __forceinline__ bool key_next(const BwdParams &p, KeyWalk &w, KeyChunk &c, uint32_t *status) {
    const FwdSet &s = p.plan.s;
    const int64_t hk_n = p.plan.kv_heads;
    int64_t hk;
    int len;
    if (p.plan.stream) {
        if (w.left <= 0) return false;
        if (w.t == s.fixed) {
            w.t = 0;
            if (++w.uu == hk_n * set_steps(s, w.z)) {
                w.uu = 0;
                if (++w.z == s.sets) return false;
            }
        }
        len = set_len(s.len, w.z, s.n, status);
        const int kt = max(1, (len + kTile - 1) / kTile);
        hk = w.uu / kt;
        c.tile = (int)(w.uu - hk * kt);
        c.slab = w.z * hk_n + hk;
        c.t0 = w.t;
        c.nt = (int)min((int64_t)(s.fixed - w.t), w.left);
        c.slot = c.nt == s.fixed ? -1 : (w.t > 0 ? 0 : 1);
        w.t += c.nt;
        w.left -= c.nt;
    } else {
        const int64_t kt = (s.n + kTile - 1) / kTile, u = w.left;
        if (u >= s.sets * hk_n * kt) return false;
        c.slab = u / kt;
        c.tile = (int)(u - c.slab * kt);
        len = set_len(s.len, c.slab / hk_n, s.n, status);
        c.t0 = 0;
        c.nt = s.fixed;
        c.slot = -1;
        w.left += gridDim.x;
    }
    c.valid = len - c.tile * kTile;
    if (c.valid <= 0) c.nt = 0;             // no key of this tile counts: its gradients are zeroed elsewhere
    return true;
}

template <int D>
__device__ void key_copy_role(const BwdParams &p, const BwdMaps &maps, KeyShared<D> &sh, int lane) {
    using C = KeyCfg<D>;
    volatile int *abort_flag = &sh.abort_flag;
    const bool leader = elect_one();    // issues; the whole warp runs the loop
    auto wait_w = [&](uint64_t *b, uint32_t par) -> bool {
        return __all_sync(0xffffffffu, wait_soon(b, par, abort_flag, p.status));
    };
    uint32_t u = 0, g = 0;
    bool ok = true;
    KeyChunk c;
    KeyWalk w = key_begin<D>(p, sh);
    while (ok && key_next(p, w, c, leader ? p.status : nullptr)) {
        if (c.nt <= 0) continue;
        const int kb = u & 1;
        if (!(ok = wait_w(&sh.kv_empty[kb], ((u >> 1) & 1) ^ 1))) break;
        if (leader) {
            mbar_expect_tx(&sh.kv_full[kb], 2 * C::UNIT);
            for (int h = 0; h < C::HALVES; ++h) {
                tma_load_3d(sh.k[kb] + h * (kTile * 128), &maps.k, &sh.kv_full[kb], 64 * h, c.tile * kTile, (int)c.slab);
                tma_load_3d(sh.v[kb] + h * (kTile * 128), &maps.v, &sh.kv_full[kb], 64 * h, c.tile * kTile, (int)c.slab);
            }
        }
        __syncwarp();
        ++u;
        for (int t = 0; t < c.nt; ++t, ++g) {
            const int st = g % C::STAGES;
            if (!(ok = wait_w(&sh.st_empty[st], ((g / C::STAGES) & 1) ^ 1))) break;
            if (leader) {
                uint64_t *bar = &sh.st_full[st];
                const int row = (c.t0 + t) * kSub;
                mbar_expect_tx(bar, 2 * C::STEP + kStat * 4);
                for (int h = 0; h < C::HALVES; ++h) {
                    tma_load_3d(sh.q[st] + h * (kSub * 128), &maps.q, bar, 64 * h, row, (int)c.slab);
                    tma_load_3d(sh.o[st] + h * (kSub * 128), &maps.o, bar, 64 * h, row, (int)c.slab);
                }
                bulk_load(sh.stat[st], p.stat + (c.slab * p.qtiles + c.t0 + t) * kStat, kStat * 4, bar);
            }
            __syncwarp();
        }
    }
    if (!ok) {
        for (uint32_t i = g > (uint32_t)C::STAGES ? g - C::STAGES : 0; i < g; ++i)
            drain_bar(&sh.st_full[i % C::STAGES], (i / C::STAGES) & 1);
        for (uint32_t i = u > 2 ? u - 2 : 0; i < u; ++i) drain_bar(&sh.kv_full[i & 1], (i >> 1) & 1);
    }
}

// Tensor memory, key-major: stage b: Sᵀ cols 128b.., dPᵀ cols 128b+64..; D = 64: Pᵀ and dSᵀ of stage b
// at cols 256+64b and 288+64b, dV 384, dK 448; D = 128: Pᵀ and dSᵀ in place, dV 256, dK 384.
template <int D> __device__ __forceinline__ uint32_t key_p(int b) { return D == 64 ? 256u + 64u * b : 128u * b; }
template <int D> __device__ __forceinline__ uint32_t key_ds(int b) { return D == 64 ? 288u + 64u * b : 128u * b + 64u; }
template <int D> constexpr uint32_t kColDv = D == 64 ? 384u : 256u;
template <int D> constexpr uint32_t kColDk = D == 64 ? 448u : 384u;

// Sᵀ and dPᵀ of every step.
template <int D>
__device__ void key_score_role(const BwdParams &p, KeyShared<D> &sh, uint32_t tmem, int lane) {
    using C = KeyCfg<D>;
    volatile int *abort_flag = &sh.abort_flag;
    const bool leader = elect_one();    // issues; the whole warp runs the loop
    auto wait_w = [&](uint64_t *b, uint32_t par) -> bool {
        return __all_sync(0xffffffffu, wait_soon(b, par, abort_flag, p.status));
    };
    const uint64_t dk0 = desc_kmajor_sw128(sh.k[0]), dv0 = desc_kmajor_sw128(sh.v[0]);
    const uint64_t dq0 = desc_kmajor_sw128(sh.q[0]), do0 = desc_kmajor_sw128(sh.o[0]);
    uint32_t u = 0, g = 0;
    bool ok = true;
    KeyChunk c;
    KeyWalk w = key_begin<D>(p, sh);
    while (ok && key_next(p, w, c, nullptr)) {
        if (c.nt <= 0) continue;
        const int kb = u & 1;
        if (!(ok = wait_w(&sh.kv_full[kb], (u >> 1) & 1))) break;
        ++u;
        for (int t = 0; t < c.nt; ++t, ++g) {
            const int st = g % C::STAGES, b = g & 1;
            // the stage's columns are free: read (D = 64), or read as Pᵀ and dSᵀ by the gradients' MMAs
            if (g >= 2 && !(ok = wait_w(D == 64 ? &sh.s_free[b] : &sh.g_done[b], ((g >> 1) & 1) ^ 1))) break;
            if (!(ok = wait_w(&sh.st_full[st], (g / C::STAGES) & 1))) break;
            fence_after();
            if (leader) {
                const uint64_t dk = dk0 + (uint64_t)kb * (C::UNIT >> 4), dv = dv0 + (uint64_t)kb * (C::UNIT >> 4);
                const uint64_t dq = dq0 + (uint64_t)st * (C::STEP >> 4), dO = do0 + (uint64_t)st * (C::STEP >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t a = (kk / 4) * ((kTile * 128) >> 4) + 2 * (kk % 4);
                    const uint64_t o = (kk / 4) * ((kSub * 128) >> 4) + 2 * (kk % 4);
                    mma_bf16(tmem + 128u * b, dk + a, dq + o, idesc_of(kSub, false), kk > 0);
                }
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t a = (kk / 4) * ((kTile * 128) >> 4) + 2 * (kk % 4);
                    const uint64_t o = (kk / 4) * ((kSub * 128) >> 4) + 2 * (kk % 4);
                    mma_bf16(tmem + 128u * b + 64u, dv + a, dO + o, idesc_of(kSub, false), kk > 0);
                }
                commit(&sh.s_full[b]);
                commit(&sh.st_empty[st]);
                if (t + 1 == c.nt) commit(&sh.kv_empty[kb]);
            }
            __syncwarp();
        }
    }
    if (leader) commit(&sh.drain[0]);
    __syncwarp();
    drain_bar(&sh.drain[0], 0);
}

// dV += Pᵀ·dO and dK += dSᵀ·Q of every step.
template <int D>
__device__ void key_grad_role(const BwdParams &p, KeyShared<D> &sh, uint32_t tmem, int lane) {
    using C = KeyCfg<D>;
    volatile int *abort_flag = &sh.abort_flag;
    const bool leader = elect_one();    // issues; the whole warp runs the loop
    auto wait_w = [&](uint64_t *b, uint32_t par) -> bool {
        return __all_sync(0xffffffffu, wait_soon(b, par, abort_flag, p.status));
    };
    const uint64_t dq0 = desc_mnmajor_sw128(sh.q[0], kSub * 128), do0 = desc_mnmajor_sw128(sh.o[0], kSub * 128);
    uint32_t u = 0, g = 0;
    bool ok = true;
    KeyChunk c;
    KeyWalk w = key_begin<D>(p, sh);
    while (ok && key_next(p, w, c, nullptr)) {
        if (c.nt <= 0) continue;
        if (u > 0 && !(ok = wait_w(&sh.acc_free, (u - 1) & 1))) break;
        ++u;
        for (int t = 0; t < c.nt; ++t, ++g) {
            const int st = g % C::STAGES, b = g & 1;
            if (!(ok = wait_w(&sh.p_full[b], (g >> 1) & 1))) break;
            fence_after();
            if (leader) {
                const uint64_t dq = dq0 + (uint64_t)st * (C::STEP >> 4), dO = do0 + (uint64_t)st * (C::STEP >> 4);
#pragma unroll
                for (int kk = 0; kk < kSub / 16; ++kk)
                    mma_ts(tmem + kColDv<D>, tmem + key_p<D>(b) + 8u * kk, dO + 128 * kk, idesc_of(D, true), t > 0 || kk > 0);
#pragma unroll
                for (int kk = 0; kk < kSub / 16; ++kk)
                    mma_ts(tmem + kColDk<D>, tmem + key_ds<D>(b) + 8u * kk, dq + 128 * kk, idesc_of(D, true), t > 0 || kk > 0);
                commit(&sh.g_done[b]);
                commit(&sh.st_empty[st]);
                if (t + 1 == c.nt) commit(&sh.acc_full);
            }
            __syncwarp();
        }
    }
    if (leader) commit(&sh.drain[1]);
    __syncwarp();
    drain_bar(&sh.drain[1], 0);
}

// 32 columns of a gradient row: bf16 to dst16, or fp32 to dst32 (dst16 null).
__device__ __forceinline__ void grad32(__nv_bfloat16 *dst16, float *dst32, const float *x, float f) {
    if (dst16) {
        uint4 *d4 = reinterpret_cast<uint4 *>(dst16);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            d4[c] = make_uint4(pack_bf16x2(x[8 * c] * f, x[8 * c + 1] * f), pack_bf16x2(x[8 * c + 2] * f, x[8 * c + 3] * f),
                               pack_bf16x2(x[8 * c + 4] * f, x[8 * c + 5] * f), pack_bf16x2(x[8 * c + 6] * f, x[8 * c + 7] * f));
    } else {
        float4 *d4 = reinterpret_cast<float4 *>(dst32);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            d4[c] = make_float4(x[4 * c] * f, x[4 * c + 1] * f, x[4 * c + 2] * f, x[4 * c + 3] * f);
    }
}

template <int D>
__device__ void key_softmax_role(const BwdParams &p, KeyShared<D> &sh, uint32_t tmem, int grp, int wq, int lane) {
    using C = KeyCfg<D>;
    volatile int *abort_flag = &sh.abort_flag;
    auto wait_all = [&](uint64_t *b, uint32_t par) -> bool {
        return __all_sync(0xffffffffu, wait_soon(b, par, abort_flag, p.status));
    };
    const uint32_t tw = tmem + ((uint32_t)(32 * wq) << 16);
    const int row = 32 * wq + lane;          // this thread's key of the tile
    const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
    uint32_t u = 0, g = 0;
    bool ok = true;
    KeyChunk c;
    KeyWalk w = key_begin<D>(p, sh);
    while (ok && key_next(p, w, c, nullptr)) {
        if (c.nt <= 0) continue;
        const bool counts = row < c.valid;
        for (int t = 0; t < c.nt; ++t, ++g) {
            if ((int)(g & 1) != grp) continue;
            const int st = g % C::STAGES;
            if (!(ok = wait_all(&sh.s_full[grp], (g >> 1) & 1))) break;
            fence_after();
            // statistics arrive with the step's tiles, whose barrier the MMA warp waited for; this
            // thread's own wait on it makes the copied values visible to it
            if (!(ok = wait_all(&sh.st_full[st], (g / C::STAGES) & 1))) break;
            const float4 *ls4 = reinterpret_cast<const float4 *>(sh.stat[st]);
            const float4 *dd4 = reinterpret_cast<const float4 *>(sh.stat[st] + kSub);
            uint32_t pp[32], ds[32];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float s[32], d[32];
                tmem_ld32(tw + 128u * grp + 32u * h, s);
                tmem_ld32(tw + 128u * grp + 64u + 32u * h, d);
                tmem_wait_ld();
                float2 x[16];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float4 l4 = ls4[8 * h + e];
                    x[2 * e] = __ffma2_rn(make_float2(s[4 * e], s[4 * e + 1]), sl2, make_float2(-l4.x, -l4.y));
                    x[2 * e + 1] = __ffma2_rn(make_float2(s[4 * e + 2], s[4 * e + 3]), sl2, make_float2(-l4.z, -l4.w));
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = make_float2(ex2(x[e].x), ex2(x[e].y));
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float4 d4 = dd4[8 * h + e];
                    const float2 a = __fmul2_rn(x[2 * e], __fadd2_rn(make_float2(d[4 * e], d[4 * e + 1]), make_float2(-d4.x, -d4.y)));
                    const float2 b = __fmul2_rn(x[2 * e + 1], __fadd2_rn(make_float2(d[4 * e + 2], d[4 * e + 3]), make_float2(-d4.z, -d4.w)));
                    ds[16 * h + 2 * e] = pack_bf16x2(a.x, a.y);
                    ds[16 * h + 2 * e + 1] = pack_bf16x2(b.x, b.y);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) pp[16 * h + e] = pack_bf16x2(x[e].x, x[e].y);
            }
            if constexpr (D == 64) {
                fence_before();
                warp_arrive(&sh.s_free[grp], lane);
            }
            if (!counts) {
#pragma unroll
                for (int e = 0; e < 32; ++e) pp[e] = ds[e] = 0u;
            }
            // the buffers' last readers, the gradients' MMAs two steps ago (D = 128: done before this Sᵀ began)
            if (D == 64 && g >= 2 && !(ok = wait_all(&sh.g_done[grp], ((g >> 1) & 1) ^ 1))) break;
            fence_after();
            tmem_st32(tw + key_p<D>(grp), reinterpret_cast<const float *>(pp));
            tmem_st32(tw + key_ds<D>(grp), reinterpret_cast<const float *>(ds));
            tmem_wait_st();
            fence_before();
            warp_arrive(&sh.p_full[grp], lane);
        }
        if (!ok || !(ok = wait_all(&sh.acc_full, u & 1))) break;
        ++u;
        fence_after();
        // group 0 stores dv, group 1 dk
        const uint32_t col = grp ? kColDk<D> : kColDv<D>;
        const int64_t at = c.slab * p.plan.s.n + (int64_t)c.tile * kTile + row;
        __nv_bfloat16 *d16 = c.slot >= 0 ? nullptr : (grp ? p.dk : p.dv) + at * D;
        float *d32 = p.part + (((2 * (int64_t)blockIdx.x + max(c.slot, 0)) * kTile + row) * 2 + grp) * D;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
            float x[32];
            tmem_ld32(tw + col + 32u * cc, x);
            tmem_wait_ld();
            if (counts) grad32(d16 ? d16 + 32 * cc : nullptr, d32 + 32 * cc, x, grp ? p.scale : 1.f);
        }
        fence_before();
        warp_arrive(&sh.acc_free, lane);
    }
}

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1) bwd_key_kernel(const __grid_constant__ BwdMaps maps,
                                                              const __grid_constant__ BwdParams p) {
    extern __shared__ uint8_t smem_raw[];
    KeyShared<D> &sh = *reinterpret_cast<KeyShared<D> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        sh.abort_flag = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.kv_full[i], 1);
            mbar_init(&sh.kv_empty[i], 1);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_free[i], 4);
            mbar_init(&sh.p_full[i], 4);
            mbar_init(&sh.g_done[i], 1);
            mbar_init(&sh.drain[i], 1);
        }
        for (int i = 0; i < KeyCfg<D>::STAGES; ++i) {
            mbar_init(&sh.st_full[i], 1);
            mbar_init(&sh.st_empty[i], 2);
        }
        mbar_init(&sh.acc_full, 1);
        mbar_init(&sh.acc_free, 8);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem_base))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == 3 && p.plan.stream) {
        const int64_t total = total_steps(p.plan, lane);
        const int64_t first = cta_first(blockIdx.x, total, p.plan.ctas), last = cta_first(blockIdx.x + 1, total, p.plan.ctas);
        StepAt at{};
        if (first < last) at = step_at(p.plan, first, lane);
        if (lane == 0) {
            sh.first = first;
            sh.last = last;
            sh.at = at;
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem_base;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtrlRegs));
        if (warp == 0) key_copy_role<D>(p, maps, sh, lane);
        else if (warp == 1) key_score_role<D>(p, sh, tmem, lane);
        else if (warp == 2) key_grad_role<D>(p, sh, tmem, lane);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        key_softmax_role<D>(p, sh, tmem, (warp - 4) >> 2, warp & 3, lane);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ---------------------------------------------------------------- query-major: dq

template <int D> struct QryCfg {
    static constexpr int HALVES = D / 64;
    static constexpr int UNIT = kTile * D * 2;         // bytes of a Q or dO tile
    static constexpr int STEP = kSub * D * 2;          // bytes of a K or V tile
    static constexpr int STAGES = D == 64 ? 8 : 3;
};
template <int D> struct alignas(1024) QryShared {
    uint8_t q[2][QryCfg<D>::UNIT], o[2][QryCfg<D>::UNIT];
    uint8_t k[QryCfg<D>::STAGES][QryCfg<D>::STEP], v[QryCfg<D>::STAGES][QryCfg<D>::STEP];
    uint64_t q_full[2], q_empty[2], st_full[QryCfg<D>::STAGES], st_empty[QryCfg<D>::STAGES], tail;
    uint64_t s_full[2], s_free[2], p_full[2], acc_full[2], drain[2];
    int64_t first, last;
    StepAt at;
    uint32_t tmem_base;
    int abort_flag;
};
struct QryChunk {
    int64_t slab, pair;
    int k0, nt, len, slot;   // first key, steps of 64 keys, the set's keys
};
struct QryWalk {
    int64_t z, uu, left;
    int t, steps;
};
template <int D> __device__ __forceinline__ QryWalk qry_begin(const BwdParams &p, const QryShared<D> &sh) {
    QryWalk w;
    if (p.plan.stream) {
        w.z = sh.at.z;
        w.uu = sh.at.uu;
        w.t = sh.at.t;
        w.steps = sh.at.steps;
        w.left = sh.last - sh.first;
    } else {
        w.left = blockIdx.x;
    }
    return w;
}
__device__ __forceinline__ bool qry_next(const BwdParams &p, QryWalk &w, QryChunk &c, uint32_t *status) {
    const FwdSet &s = p.plan.s;
    int64_t z, uu;
    int t0, n;
    if (p.plan.stream) {
        if (w.left <= 0) return false;
        if (w.t == w.steps) {
            w.t = 0;
            if (++w.uu == s.upz) {
                w.uu = 0;
                if (++w.z == s.sets) return false;
                w.steps = set_steps(s, w.z);
            }
        }
        z = w.z;
        uu = w.uu;
        t0 = w.t;
        n = (int)min((int64_t)(w.steps - w.t), w.left);
        c.slot = n == w.steps ? -1 : (w.t > 0 ? 0 : 1);
        w.t += n;
        w.left -= n;
    } else {
        if (w.left >= s.sets * s.upz) return false;
        z = w.left / s.upz;
        uu = w.left - z * s.upz;
        t0 = 0;
        n = 0x7fffff;
        c.slot = -1;
        w.left += gridDim.x;
    }
    const int64_t hk = uu / s.pairs;
    c.pair = uu - hk * s.pairs;
    c.slab = z * p.plan.kv_heads + hk;
    c.len = set_len(s.len, z, s.n, status);
    c.k0 = t0 * kTile;
    const int64_t end = min((int64_t)c.len, ((int64_t)t0 + n) * kTile);
    c.nt = (int)max((int64_t)0, (end - c.k0 + kSub - 1) / kSub);
    return true;
}

template <int D>
__device__ void qry_copy_role(const BwdParams &p, const BwdMaps &maps, QryShared<D> &sh, int lane) {
    using C = QryCfg<D>;
    volatile int *abort_flag = &sh.abort_flag;
    const bool leader = elect_one();    // issues; the whole warp runs the loop
    auto wait_w = [&](uint64_t *b, uint32_t par) -> bool {
        return __all_sync(0xffffffffu, wait_soon(b, par, abort_flag, p.status));
    };
    const FwdSet &s = p.plan.s;
    uint32_t nq[2] = {0, 0}, g = 0, ntail = 0;
    bool ok = true;
    QryChunk c;
    QryWalk w = qry_begin<D>(p, sh);
    while (ok && qry_next(p, w, c, leader ? p.status : nullptr)) {
        if (c.nt <= 0) continue;
        for (int pl = 0; pl < 2 && ok; ++pl) {
            const int64_t t = 2 * c.pair + pl;
            if (t >= s.tiles) continue;
            if (!(ok = wait_w(&sh.q_empty[pl], (nq[pl] & 1) ^ 1))) break;
            if (leader) {
                mbar_expect_tx(&sh.q_full[pl], 2 * C::UNIT);
                for (int h = 0; h < C::HALVES; ++h) {
                    tma_load_3d(sh.q[pl] + h * (kTile * 128), &maps.q, &sh.q_full[pl], 64 * h, (int)(t * kTile), (int)c.slab);
                    tma_load_3d(sh.o[pl] + h * (kTile * 128), &maps.o, &sh.q_full[pl], 64 * h, (int)(t * kTile), (int)c.slab);
                }
            }
            __syncwarp();
            ++nq[pl];
        }
        for (int t = 0; t < c.nt && ok; ++t) {
            const int st = g % C::STAGES;
            if (!(ok = wait_w(&sh.st_empty[st], ((g / C::STAGES) & 1) ^ 1))) break;
            const int row = c.k0 + t * kSub;
            // rows of K behind the length that are in the buffer: zeroed (0·NaN is NaN)
            const int z0 = c.len - row, z1 = (int)min((int64_t)kSub, s.n - row);
            const bool zero = z0 < z1;
            uint64_t *bar = zero ? &sh.tail : &sh.st_full[st];
            if (leader) {
                mbar_expect_tx(bar, 2 * C::STEP);
                for (int h = 0; h < C::HALVES; ++h) {
                    tma_load_3d(sh.k[st] + h * (kSub * 128), &maps.k, bar, 64 * h, row, (int)c.slab);
                    tma_load_3d(sh.v[st] + h * (kSub * 128), &maps.v, bar, 64 * h, row, (int)c.slab);
                }
            }
            __syncwarp();
            ++g;
            if (zero) {
                ok = wait_w(&sh.tail, ntail & 1);
                if (!ok) drain_bar(&sh.tail, ntail & 1);
                ++ntail;
                if (ok) {
                    for (int h = 0; h < C::HALVES; ++h) {
                        uint4 *rows = reinterpret_cast<uint4 *>(sh.k[st] + h * (kSub * 128));
                        for (int i = z0 * 8 + lane; i < z1 * 8; i += 32) rows[i] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async();
                }
                __syncwarp();
                if (leader) mbar_arrive(&sh.st_full[st]);
            }
        }
    }
    if (!ok) {
        for (uint32_t i = g > (uint32_t)C::STAGES ? g - C::STAGES : 0; i < g; ++i)
            drain_bar(&sh.st_full[i % C::STAGES], (i / C::STAGES) & 1);
        for (int pl = 0; pl < 2; ++pl)
            if (nq[pl]) drain_bar(&sh.q_full[pl], (nq[pl] - 1) & 1);
    }
}

// Tensor memory, query-major, pipeline base 256·pl: D = 64: S of even and odd steps at 0 and 64, dP 128,
// dQ 192; D = 128: S 0, dP 64, dQ 128. dS takes the place of its step's S.
template <int D> __device__ __forceinline__ uint32_t qry_s(uint32_t g) { return D == 64 ? 64u * (g & 1) : 0u; }
template <int D> constexpr uint32_t kColDp = D == 64 ? 128u : 64u;
template <int D> constexpr uint32_t kColDq = D == 64 ? 192u : 128u;

template <int D>
__device__ void qry_mma_role(const BwdParams &p, QryShared<D> &sh, uint32_t tmem, int pl, int lane) {
    using C = QryCfg<D>;
    volatile int *abort_flag = &sh.abort_flag;
    const bool leader = elect_one();    // issues; the whole warp runs the loop
    auto wait_w = [&](uint64_t *b, uint32_t par) -> bool {
        return __all_sync(0xffffffffu, wait_soon(b, par, abort_flag, p.status));
    };
    const uint32_t tp = tmem + 256u * pl;
    const uint64_t dq = desc_kmajor_sw128(sh.q[pl]), dO = desc_kmajor_sw128(sh.o[pl]);
    const uint64_t dk0 = desc_kmajor_sw128(sh.k[0]), dv0 = desc_kmajor_sw128(sh.v[0]);
    const uint64_t dkm0 = desc_mnmajor_sw128(sh.k[0], kSub * 128);
    uint32_t pos = 0, g = 0, nq = 0;       // step of the CTA, this pipeline's steps and units
    bool ok = true;
    auto issue_s = [&](uint32_t at, uint32_t gs, bool last) -> bool {
        const int st = at % C::STAGES;
        if (!wait_w(&sh.st_full[st], (at / C::STAGES) & 1)) return false;
        fence_after();
        if (leader) {
            const uint64_t dk = dk0 + (uint64_t)st * (C::STEP >> 4), dv = dv0 + (uint64_t)st * (C::STEP >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t a = (kk / 4) * ((kTile * 128) >> 4) + 2 * (kk % 4);
                const uint64_t b = (kk / 4) * ((kSub * 128) >> 4) + 2 * (kk % 4);
                mma_bf16(tp + qry_s<D>(gs), dq + a, dk + b, idesc_of(kSub, false), kk > 0);
            }
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t a = (kk / 4) * ((kTile * 128) >> 4) + 2 * (kk % 4);
                const uint64_t b = (kk / 4) * ((kSub * 128) >> 4) + 2 * (kk % 4);
                mma_bf16(tp + kColDp<D>, dO + a, dv + b, idesc_of(kSub, false), kk > 0);
            }
            commit(&sh.s_full[pl]);
            if (last) commit(&sh.q_empty[pl]);
        }
        __syncwarp();
        return true;
    };
    auto issue_dq = [&](uint32_t at, bool first, bool last) -> bool {
        const int st = at % C::STAGES;
        if (!wait_w(&sh.p_full[pl], g & 1)) return false;
        fence_after();
        if (leader) {
            const uint64_t dkm = dkm0 + (uint64_t)st * (C::STEP >> 4);
#pragma unroll
            for (int kk = 0; kk < kSub / 16; ++kk)
                mma_ts(tp + kColDq<D>, tp + qry_s<D>(g) + 8u * kk, dkm + 128 * kk, idesc_of(D, true), !first || kk > 0);
            commit(&sh.st_empty[st]);
            if (last) commit(&sh.acc_full[pl]);
        }
        __syncwarp();
        ++g;
        return true;
    };
    QryChunk c;
    QryWalk w = qry_begin<D>(p, sh);
    while (ok && qry_next(p, w, c, nullptr)) {
        if (c.nt <= 0) continue;
        if (2 * c.pair + pl >= p.plan.s.tiles) {
            for (int t = 0; t < c.nt && ok; ++t) {     // released once there
                const int st = (pos + t) % C::STAGES;
                ok = wait_w(&sh.st_full[st], ((pos + t) / C::STAGES) & 1);
                if (ok && leader) mbar_arrive(&sh.st_empty[st]);
                __syncwarp();
            }
        } else {
            if (!(ok = wait_w(&sh.q_full[pl], nq & 1))) break;
            ++nq;
            if (D == 64) {
                ok = issue_s(pos, g, c.nt == 1);
                for (int t = 0; t < c.nt && ok; ++t) {
                    if (t + 1 < c.nt)
                        ok = wait_w(&sh.s_free[pl], g & 1) && issue_s(pos + t + 1, g + 1, t + 2 == c.nt);
                    ok = ok && issue_dq(pos + t, t == 0, t + 1 == c.nt);
                }
            } else {
                for (int t = 0; t < c.nt && ok; ++t)
                    ok = issue_s(pos + t, g, t + 1 == c.nt) && issue_dq(pos + t, t == 0, t + 1 == c.nt);
            }
        }
        pos += c.nt;
    }
    if (leader) commit(&sh.drain[pl]);
    __syncwarp();
    drain_bar(&sh.drain[pl], 0);
}

template <int D>
__device__ void qry_softmax_role(const BwdParams &p, QryShared<D> &sh, uint32_t tmem, int pl, int wq, int lane) {
    volatile int *abort_flag = &sh.abort_flag;
    auto wait_all = [&](uint64_t *b, uint32_t par) -> bool {
        return __all_sync(0xffffffffu, wait_soon(b, par, abort_flag, p.status));
    };
    const uint32_t tw = tmem + 256u * pl + ((uint32_t)(32 * wq) << 16);
    const int i = 32 * wq + lane;            // this thread's row of the tile
    const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
    const FwdSet &s = p.plan.s;
    uint32_t g = 0, nu = 0;
    bool ok = true;
    QryChunk c;
    QryWalk w = qry_begin<D>(p, sh);
    while (ok && qry_next(p, w, c, nullptr)) {
        const int64_t tile = 2 * c.pair + pl, r = tile * kTile + i;
        if (tile >= s.tiles) continue;
        const bool there = r < p.plan.rows;
        float lse = CUDART_INF_F, dt = 0.f;
        if (there && c.nt > 0) {
            const float *st = p.stat + (c.slab * p.qtiles + r / kSub) * kStat + r % kSub;
            lse = __ldg(st);
            dt = __ldg(st + kSub);
        }
        const float2 nl2 = make_float2(-lse, -lse), nd2 = make_float2(-dt, -dt);
        for (int t = 0; t < c.nt; ++t, ++g) {
            if (!(ok = wait_all(&sh.s_full[pl], g & 1))) break;
            fence_after();
            const int valid = c.len - c.k0 - t * kSub;
            uint32_t ds[32];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x[32], d[32];
                tmem_ld32(tw + qry_s<D>(g) + 32u * h, x);
                tmem_ld32(tw + kColDp<D> + 32u * h, d);
                tmem_wait_ld();
                float2 e2[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) e2[e] = __ffma2_rn(make_float2(x[2 * e], x[2 * e + 1]), sl2, nl2);
#pragma unroll
                for (int e = 0; e < 16; ++e) e2[e] = make_float2(ex2(e2[e].x), ex2(e2[e].y));
#pragma unroll
                for (int e = 0; e < 16; ++e) e2[e] = __fmul2_rn(e2[e], __fadd2_rn(make_float2(d[2 * e], d[2 * e + 1]), nd2));
                if (valid < kSub) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        if (32 * h + 2 * e >= valid) e2[e].x = 0.f;
                        if (32 * h + 2 * e + 1 >= valid) e2[e].y = 0.f;
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) ds[16 * h + e] = pack_bf16x2(e2[e].x, e2[e].y);
            }
            fence_before();
            if constexpr (D == 64) warp_arrive(&sh.s_free[pl], lane);
            tmem_st32(tw + qry_s<D>(g), reinterpret_cast<const float *>(ds));
            tmem_wait_st();
            fence_before();
            warp_arrive(&sh.p_full[pl], lane);
        }
        if (!ok) break;
        if (c.nt > 0) {
            if (!(ok = wait_all(&sh.acc_full[pl], nu & 1))) break;
            ++nu;
        }
        fence_after();
        __nv_bfloat16 *d16 = c.slot >= 0 ? nullptr : p.dq + (c.slab * p.plan.rows + r) * D;
        float *d32 = p.part + ((2 * (int64_t)blockIdx.x + max(c.slot, 0)) * (2 * kTile) + kTile * pl + i) * D;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
            float x[32];
            if (c.nt > 0) {
                tmem_ld32(tw + kColDq<D> + 32u * cc, x);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = 0.f;
            }
            if (there) grad32(d16 ? d16 + 32 * cc : nullptr, d32 + 32 * cc, x, p.scale);
        }
        fence_before();
    }
}

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1) bwd_qry_kernel(const __grid_constant__ BwdMaps maps,
                                                              const __grid_constant__ BwdParams p) {
    extern __shared__ uint8_t smem_raw[];
    QryShared<D> &sh = *reinterpret_cast<QryShared<D> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        sh.abort_flag = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_empty[i], 1);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_free[i], 4);
            mbar_init(&sh.p_full[i], 4);
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.drain[i], 1);
        }
        for (int i = 0; i < QryCfg<D>::STAGES; ++i) {
            mbar_init(&sh.st_full[i], 1);
            mbar_init(&sh.st_empty[i], 2);
        }
        mbar_init(&sh.tail, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem_base))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == 3 && p.plan.stream) {
        const int64_t total = total_steps(p.plan, lane);
        const int64_t first = cta_first(blockIdx.x, total, p.plan.ctas), last = cta_first(blockIdx.x + 1, total, p.plan.ctas);
        StepAt at{};
        if (first < last) at = step_at(p.plan, first, lane);
        if (lane == 0) {
            sh.first = first;
            sh.last = last;
            sh.at = at;
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem_base;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtrlRegs));
        if (warp == 0) qry_copy_role<D>(p, maps, sh, lane);
        else if (warp < 3) qry_mma_role<D>(p, sh, tmem, warp - 1, lane);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        qry_softmax_role<D>(p, sh, tmem, (warp - 4) >> 2, warp & 3, lane);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ---------------------------------------------------------------- parts added

// A block adds 8 rows of the unit in which CTA c begins, if it is the first CTA to begin inside that
// unit: the sum of the parts in the order of their CTAs, one warp a row (key-major: of dv and of dk).
template <int D, bool KEY>
__device__ __forceinline__ void add_parts(const BwdParams &p, int c, int rowblock, int warp, int lane) {
    const int64_t total = total_steps(p.plan, lane), x = cta_first(c, total, p.plan.ctas);
    if (x >= total) return;
    const StepAt at = step_at(p.plan, x, lane);
    if (at.t == 0) return;
    const int64_t a = x - at.t;
    if (cta_of(a, total, p.plan.ctas) != c - 1) return;
    const int cb = cta_of(a + at.steps - 1, total, p.plan.ctas);
    const FwdSet &s = p.plan.s;
    constexpr int ROWS = KEY ? kTile : 2 * kTile, W = KEY ? 2 * D : D, E = W / 32;   // floats a row, a lane
    const int i = 8 * rowblock + warp;
    int64_t row;
    if (KEY) {
        const int len = set_len(s.len, at.z, s.n, nullptr), kt = max(1, (len + kTile - 1) / kTile);
        const int64_t hk = at.uu / kt, key = (at.uu - hk * kt) * kTile + i;
        if (key >= len) return;
        row = (at.z * p.plan.kv_heads + hk) * s.n + key;
    } else {
        const int64_t hk = at.uu / s.pairs, r = (at.uu - hk * s.pairs) * (2 * kTile) + i;
        if (r >= p.plan.rows) return;
        row = (at.z * p.plan.kv_heads + hk) * p.plan.rows + r;
    }
    float sum[E];
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] = 0.f;
    for (int k = c - 1; k <= cb; ++k) {
        const float2 *src = reinterpret_cast<const float2 *>(p.part + ((2 * (int64_t)k + (k == c - 1)) * ROWS + i) * W);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            const float2 y = src[32 * e + lane];
            sum[2 * e] += y.x;
            sum[2 * e + 1] += y.y;
        }
    }
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
        const int col = 2 * (32 * e + lane);           // of [dv | dk] or of dq
        __nv_bfloat16 *dst = KEY ? (col < D ? p.dv + row * D + col : p.dk + row * D + col - D) : p.dq + row * D + col;
        *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(sum[2 * e], sum[2 * e + 1]);
    }
}
// Blocks [0, key blocks): dk and dv; the rest: dq.
template <int D>
__global__ void __launch_bounds__(256) bwd_join_kernel(const __grid_constant__ BwdParams key, const __grid_constant__ BwdParams qry,
                                                       int key_blocks) {
    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    int b = blockIdx.x;
    if (b < key_blocks) {
        add_parts<D, true>(key, b / (kTile / 8) + 1, b % (kTile / 8), warp, lane);
    } else {
        b -= key_blocks;
        add_parts<D, false>(qry, b / (2 * kTile / 8) + 1, b % (2 * kTile / 8), warp, lane);
    }
}

// ---------------------------------------------------------------- host

struct BwdPlans {
    FwdPlan key, qry;
    int64_t qtiles;
    size_t stat, key_part, qry_part, total;
};

BwdPlans make_plans(const DenseProblem &p, const KeySet &ks) {
    BwdPlans r;
    r.qry = make_fwd_plan(p, ks);
    FwdSet &q = r.qry.s;
    q.few = 0;
    q.bb = 0;
    q.tpm = (int32_t)((p.rows + kTile - 1) / kTile);
    r.qtiles = (p.rows + kSub - 1) / kSub;
    r.key = r.qry;
    FwdSet &s = r.key.s;
    s.fixed = (int32_t)r.qtiles;
    s.upz = p.kv_heads * r.qtiles;
    const int64_t kt = (ks.n + kTile - 1) / kTile, units = ks.sets * p.kv_heads * kt;
    r.key.stream = (!ks.len || ks.sets <= 1024) && r.qtiles > 4 && units < 16 * kCtas;
    const int64_t want = r.key.stream ? (units * r.qtiles + 3) / 4 : units;
    r.key.ctas = (int32_t)(want < kCtas ? want : kCtas);
    size_t o = 0;
    auto take = [&](size_t floats) { const size_t at = o; o += (floats + 63) / 64 * 64; return at; };
    r.stat = take((size_t)p.batch * p.kv_heads * r.qtiles * kStat);
    r.key_part = take(r.key.stream ? (size_t)r.key.ctas * 4 * kTile * p.d : 0);
    r.qry_part = take(r.qry.stream ? (size_t)r.qry.ctas * 4 * kTile * p.d : 0);
    r.total = o;
    return r;
}

bool row_map(CUtensorMap *m, const void *base, int64_t d, int64_t rows, int64_t slabs, int box) {
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)slabs};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)rows * d * 2};
    const cuuint32_t b[3] = {64, (cuuint32_t)box, 1};
    return make_map(m, base, 3, dims, strides, b);
}

template <int D>
cudaError_t launch(const DenseProblem &pb, const void *q, const KeySet &ks, const void *out, const float *lse,
                   const void *dout, const BwdPlans &plans, BwdParams key, float *stat, float *qry_part,
                   cudaStream_t stream) {
    const int64_t slabs = pb.batch * pb.kv_heads;
    BwdMaps mk, mq;
    if (!row_map(&mk.q, q, D, pb.rows, slabs, kSub) || !row_map(&mk.o, dout, D, pb.rows, slabs, kSub) ||
        !row_map(&mk.k, ks.k, D, ks.n, slabs, kTile) || !row_map(&mk.v, ks.v, D, ks.n, slabs, kTile) ||
        !row_map(&mq.q, q, D, pb.rows, slabs, kTile) || !row_map(&mq.o, dout, D, pb.rows, slabs, kTile) ||
        !row_map(&mq.k, ks.k, D, ks.n, slabs, kSub) || !row_map(&mq.v, ks.v, D, ks.n, slabs, kSub))
        return cudaErrorInvalidValue;
    BwdParams qry = key;
    qry.plan = plans.qry;
    qry.part = qry_part;
    const size_t ksm = sizeof(KeyShared<D>) + 1024, qsm = sizeof(QryShared<D>) + 1024;
    static_assert(sizeof(KeyShared<D>) + 1024 <= 232448 && sizeof(QryShared<D>) + 1024 <= 232448, "shared memory");
    cudaError_t e = kernel_ready<bwd_key_kernel<D>>(ksm, NTHREADS, kRegsNeeded);
    if (e == cudaSuccess) e = kernel_ready<bwd_qry_kernel<D>>(qsm, NTHREADS, kRegsNeeded);
    if (e != cudaSuccess) return e;
    const int64_t stat_blocks = (slabs * plans.qtiles * kSub + 256 / (D / 8) - 1) / (256 / (D / 8));
    bwd_stat_kernel<D><<<(unsigned)(stat_blocks < 8 * kCtas ? stat_blocks : 8 * kCtas), 256, 0, stream>>>(
        key, static_cast<const __nv_bfloat16 *>(out), lse, static_cast<const __nv_bfloat16 *>(dout), stat, slabs);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    bwd_key_kernel<D><<<key.plan.ctas, NTHREADS, ksm, stream>>>(mk, key);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    bwd_qry_kernel<D><<<qry.plan.ctas, NTHREADS, qsm, stream>>>(mq, qry);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int kb = key.plan.stream ? (key.plan.ctas - 1) * (kTile / 8) : 0;
    const int qb = qry.plan.stream ? (qry.plan.ctas - 1) * (2 * kTile / 8) : 0;
    if (kb + qb > 0) bwd_join_kernel<D><<<kb + qb, 256, 0, stream>>>(key, qry, kb);
    return cudaGetLastError();
}

}  // namespace

size_t dense_bwd_floats(const DenseProblem &p, const KeySet &s) { return make_plans(p, s).total; }

cudaError_t launch_dense_bwd(const DenseProblem &pb, const void *q, const KeySet &ks, const void *out, const float *lse,
                             const void *dout, void *dq, void *dk, void *dv, float *ws, uint32_t *status,
                             cudaStream_t stream) {
    const BwdPlans plans = make_plans(pb, ks);
    BwdParams p{};
    p.plan = plans.key;
    p.stat = ws + plans.stat;
    p.qtiles = plans.qtiles;
    p.dq = static_cast<__nv_bfloat16 *>(dq);
    p.dk = static_cast<__nv_bfloat16 *>(dk);
    p.dv = static_cast<__nv_bfloat16 *>(dv);
    p.part = ws + plans.key_part;
    p.scale = pb.scale;
    p.scale_log2 = pb.scale * 1.4426950408889634f;
    p.status = status;
    float *stat = ws + plans.stat, *qp = ws + plans.qry_part;
    return pb.d == 64 ? launch<64>(pb, q, ks, out, lse, dout, plans, p, stat, qp, stream)
                      : launch<128>(pb, q, ks, out, lse, dout, plans, p, stat, qp, stream);
}

}  // namespace bsa
