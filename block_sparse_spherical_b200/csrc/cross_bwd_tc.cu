// Backward of dense softmax attention to states of another length on the sm_100a
// tensor cores (bf16, head_dim D = 64 or 128, fp32 accumulation).
//
// With the forward's row log-sum-exp and D_i = dout_i·(out_i + out_low_i) (a row pass ahead):
//   s_ij = q_i·k_j,  p_ij = exp(c s_ij - lse_i),  dp_ij = dout_i·v_j,
//   ds_ij = p_ij (dp_ij - D_i),
//   dv_j = Σ_i p_ij dout_i,  dk_j = c Σ_i ds_ij q_i,  dq_i = c Σ_j ds_ij k_j.
// Two passes of one kernel, each with its sums in tensor memory, so that no gradient is
// reduced through atomics and all are the same from call to call; the second recomputes
// s and dp (8 products a pair of tiles, two of them dq's, where one pass would need 5 and
// an fp32 reduction of dq through L2 in an order that changes).
//
// A unit is a tile of 128 rows of one side, with operands A0 and A1, a step a tile of 128 of
// the other, with B0 and B1:
//   KEY  (dk, dv): unit = keys, A0 = K, A1 = V; step = query rows, B0 = Q, B1 = dO;
//   !KEY (dq):     unit = query rows, A0 = Q, A1 = dO; step = keys, B0 = K, B1 = V.
// S = A0·B0ᵀ and dP = A1·B1ᵀ (tcgen05.mma, M = N = 128) go to tensor memory, where thread
// (w, row) of 512 takes its unit row's columns 32w..32w+31; P (KEY only) and dS return there as
// bf16 pairs and are the A operands of acc0 += P·B1 (dv) and acc1 += dS·B0 (dk, dq), so
// nothing passes through shared memory. S and dP have barriers of their own, and so have P and
// dS: exponentials run while dP is formed, P·B1 while dS is computed, and S of the next step
// as soon as this one's is read (where P has columns of its own) or its P used up (KEY,
// D = 128, where tensor memory holds no more; see kParts).
//
// Roundings: P and dS are bf16 as operands, as out and the gradients are (each off by half a step, a mean
// of 1.66e-3 in bf16). For dq, dS is given as two bf16 terms, its rounding and what that leaves off: with one, dq
// was off by 2.5e-3 of its norm from 64 bits, with two it is 1.7e-3, which is its own rounding. That costs
// the dq pass a product more (12288 x 12288, 8 heads, D = 64: 652 us, with one term 565). dk
// and dv (2.4e-3) have no columns of tensor memory left for it. D's own error would be common to
// a row's dS: from out alone, which is rounded, it took dq and dk to 2.8e-3 at 64 keys.
//
// What bounds it (here and below: GPU time of calls on the same inputs): 12288 x 12288, 8 heads, D = 64: both passes
// 1,250 to 1,390 us, with the data and the clock (launched alone, at the slower end: dk and dv 718, dq 650), the row
// pass 10, the parts' sum 7; 10 n² d flops a head are 773 GFLOP for the 8 heads, 0.56 to 0.62 PFLOP/s. D = 128,
// 4 heads: 977 us, 0.79 PFLOP/s. Tensor pipe and exponential unit are each 46 % busy (D = 128: 60 % and 30 %). At
// D = 64 a step of 128 x 128 needs 1,024 clocks of the exponential unit and about as many of the tensor cores; what
// it takes (2,400) is the chain S, exponentials, P, dP, dS, product, of which only parts overlap in the tensor
// memory there is.
//
// One persistent CTA per SM, 640 threads: warp 0 finds the units, hands them out and copies their tiles,
// warp 1 issues S and dP, warp 2 P·B1 (KEY), warp 3 dS·B0 (one thread issues a tcgen05 instruction
// about every 60 clocks: one warp for all of them, or steps of 64 columns with twice the instructions,
// and their issue sets the pace), warps 4-19 the softmax (with eight warps, two a scheduler, a step's
// chain of waits, loads and stores took 1,900 clocks beside the exponentials).
//
// Tensor memory: S 0..127, dP 128..255. KEY, D = 64: P 256, dS 320 (64 columns each), dv 384, dk 448.
// KEY, D = 128: P and dS in the place of the thread's own S and dP columns, dv 256, dk 384.
// !KEY: dS 256, dq 320, dS's second term 448.
//
// The steps of all units are dealt to the CTAs in equal shares; a unit cut between CTAs leaves fp32
// parts, which a last kernel adds in the order of the CTAs.
//
// Keys behind a length: their p and ds are set to 0 (whatever K and V hold); the copy
// warp of the dq pass zeroes those rows of K, since 0·NaN is NaN. Query rows behind the
// last are filled with zeros by the copy and have lse = +inf, and their p is set to 0 too: the score of
// an infinite key is 0·inf there.
//
// Every wait on an mbarrier is bounded (2 s), as in the forward.
#include <math_constants.h>

#include "cross.cuh"
#include "cross_tc.cuh"

namespace bsa {
namespace {

using namespace tc;

constexpr int kSoftWarps = 16;              // of the softmax: thread (w, row) has columns 32w.. of a step
constexpr int NTHREADS = 128 + 32 * kSoftWarps;
constexpr int kCtrlRegs = 56, kSoftRegs = 104;
constexpr int kRegsNeeded = 128 * kCtrlRegs + 32 * kSoftWarps * kSoftRegs;
static_assert(kRegsNeeded <= 65536 / NTHREADS / 8 * 8 * NTHREADS, "register split");
constexpr int kStat = 2 * kTile;            // floats of a query tile's statistics: -lse·log2 e, then -D

struct BwdParams {
    FwdPlan plan;           // KEY: s.fixed query tiles a unit; !KEY: units are query tiles, steps key tiles
    const float *stat;      // [slabs][query tiles][2][128]
    int64_t qtiles;         // query tiles a slab
    __nv_bfloat16 *dq, *dk, *dv;
    float *part;            // KEY [2 ctas][128][2][D] (dv, dk), !KEY [2 ctas][128][D]
    Cut *cuts;              // [ctas], stream only
    int cta0;               // first block of this pass in the launch
    float scale, scale_log2;
    uint32_t *status;
    int64_t withhold;       // test hook
};
__device__ __forceinline__ int this_cta(const BwdParams &p) { return (int)blockIdx.x - p.cta0; }
struct BwdMaps {
    CUtensorMap a0, a1, b0, b1;
};

// ---------------------------------------------------------------- statistics

// Per query row -lse·log2 e (-inf for rows without keys or behind the last: p = 0) and -D = -dout·out
// (negated, since a packed add or fma has no negated operand);
// and zeros for the gradients of keys behind a length. D/8 lanes a row, 16 bytes each.
template <int D>
__global__ void __launch_bounds__(256) bwd_stat_kernel(const __grid_constant__ BwdParams p, const __nv_bfloat16 *out,
                                                       const __nv_bfloat16 *low, const float *lse,
                                                       const __nv_bfloat16 *dout, float *stat,
                                                       int64_t slabs) {
    constexpr int L = D / 8;
    const int sub = threadIdx.x % L;
    const int64_t rows = p.qtiles * kTile, step = (int64_t)gridDim.x * blockDim.x / L;
    const int64_t n_all = (slabs * rows + 31) / 32 * 32;     // whole warps stay together for the shuffles
    for (int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / L; i < n_all; i += step) {
        const int64_t slab = i / rows, r = i - slab * rows;
        const bool there = slab < slabs && r < p.plan.rows;
        float d = 0.f, x = CUDART_INF_F;
        if (there) {
            const int64_t at = slab * p.plan.rows + r;
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(out + at * D) + sub);
            const uint4 b = __ldg(reinterpret_cast<const uint4 *>(dout + at * D) + sub);
            const uint4 c = low ? __ldg(reinterpret_cast<const uint4 *>(low + at * D) + sub) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t ua[4] = {a.x, a.y, a.z, a.w}, ub[4] = {b.x, b.y, b.z, b.w}, uc[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                d = fmaf(__uint_as_float(ua[e] << 16) + __uint_as_float(uc[e] << 16), __uint_as_float(ub[e] << 16), d);
                d = fmaf(__uint_as_float(ua[e] & 0xffff0000u) + __uint_as_float(uc[e] & 0xffff0000u),
                         __uint_as_float(ub[e] & 0xffff0000u), d);
            }
            x = __ldg(lse + at) * 1.4426950408889634f;
            if (x == -CUDART_INF_F) x = CUDART_INF_F;
        }
#pragma unroll
        for (int o = L / 2; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        if (sub == 0 && slab < slabs) {
            float *s = stat + (slab * p.qtiles + r / kTile) * kStat + r % kTile;
            s[0] = -x;
            s[kTile] = x == CUDART_INF_F ? 0.f : -d;
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

// ---------------------------------------------------------------- one kernel, two passes

template <int D> struct Cfg {
    static constexpr int HALVES = D / 64;              // 128-byte column groups of a row
    static constexpr int TILE = kTile * D * 2;         // bytes of a 128-row tile
    static constexpr int UB = D == 64 ? 2 : 1;         // buffers of a unit's two tiles
    static constexpr int STAGES = D == 64 ? 4 : 2;     // of a step's two tiles
};
// What a CTA does next: steps [t0, t0 + nt) of a unit; nt 0: nothing to add, -1: nothing more.
struct Chunk {
    int nt, t0, tile, slot; // slot -1: the whole unit
    int rows, cols;         // rows of the unit that count; columns (keys, or query rows) from step t0 on that count
    int64_t slab;
};
constexpr int kChunks = 4;
template <bool KEY> constexpr int kReaders = (KEY ? 3 : 2) + kSoftWarps;   // warps that read a chunk: MMA, softmax
template <int D> struct alignas(1024) Shared {
    uint8_t a0[Cfg<D>::UB][Cfg<D>::TILE], a1[Cfg<D>::UB][Cfg<D>::TILE];
    uint8_t b0[Cfg<D>::STAGES][Cfg<D>::TILE], b1[Cfg<D>::STAGES][Cfg<D>::TILE];
    float stat[Cfg<D>::STAGES][kStat];
    uint64_t u_full[2], u_empty[2], st_full[4], st_empty[4], tail;
    uint64_t s_full[2], dp_full[2], s_free[2], p_full[2], ds_full[2], v_done[2], k_done[2];    // of each part of a step
    uint64_t acc_full, acc_free, drain[3];
    uint64_t ch_full[kChunks], ch_empty[kChunks];
    Chunk ch[kChunks];
    uint32_t tmem_base;
    int abort_flag;
};

struct Walk {
    int t, steps;
    int64_t z, uu, left, at, total;
};
template <bool KEY> __device__ __forceinline__ int64_t units_of(const FwdPlan &p, int64_t z) {
    return KEY ? p.kv_heads * set_steps(p.s, z) : p.s.upz;
}
__device__ __forceinline__ Walk walk_begin(const BwdParams &p, int lane) {
    Walk w{};
    if (p.plan.stream) {
        if (lane == 0) p.cuts[this_cta(p)].last = -1;  // until one is noted
        w.total = total_steps(p.plan, lane);
        w.at = cta_first(this_cta(p), w.total, p.plan.ctas);
        w.left = cta_first(this_cta(p) + 1, w.total, p.plan.ctas) - w.at;
        if (w.left > 0) {
            const StepAt at = step_at(p.plan, w.at, lane);
            w.t = at.t;
            w.steps = at.steps;
            w.z = at.z;
            w.uu = at.uu;
        }
    } else {
        w.left = this_cta(p);
    }
    return w;
}
template <bool KEY> __device__ __forceinline__ bool walk_next(const BwdParams &p, Walk &w, Chunk &c, bool lead) {
    const FwdSet &s = p.plan.s;
    const int64_t hk_n = p.plan.kv_heads;
    int64_t z, uu;
    int n;
    if (p.plan.stream) {
        if (w.left <= 0) return false;
        if (w.t == w.steps) {
            w.t = 0;
            if (++w.uu == units_of<KEY>(p.plan, w.z)) {
                w.uu = 0;
                ++w.z;
                if (!KEY) w.steps = set_steps(s, w.z);
            }
        }
        z = w.z;
        uu = w.uu;
        c.t0 = w.t;
        n = (int)min((int64_t)(w.steps - w.t), w.left);
        c.slot = n == w.steps ? -1 : (w.t > 0 ? 0 : 1);
    } else {
        const int64_t per = KEY ? hk_n * ((s.n + kTile - 1) / kTile) : s.upz;
        if (w.left >= s.sets * per) return false;
        z = quotient(w.left, per);
        uu = w.left - z * per;
        c.t0 = 0;
        n = KEY ? s.fixed : 0x7fffffff;
        c.slot = -1;
    }
    const int len = set_len(s.len, z, s.n, lead ? p.status : nullptr);
    const int64_t tiles = KEY ? (p.plan.stream ? set_steps(s, z) : (s.n + kTile - 1) / kTile) : s.tiles;
    const int64_t hk = quotient(uu, tiles);
    c.tile = (int)(uu - hk * tiles);
    c.slab = z * hk_n + hk;
    if (p.plan.stream) {
        if (lead && w.t == 0 && c.slot == 1)
            p.cuts[this_cta(p)] = Cut{(int)z, (int)hk, c.tile, cta_of(w.at + w.steps - 1, w.total, p.plan.ctas)};
        w.t += n;
        w.at += n;
        w.left -= n;
    } else {
        w.left += p.plan.ctas;
    }
    if (KEY) {
        c.rows = len - c.tile * kTile;
        c.cols = (int)(p.plan.rows - (int64_t)c.t0 * kTile);
        c.nt = c.rows > 0 ? n : 0;                     // no key counts: its gradients are zeroed elsewhere
    } else {
        c.rows = (int)min((int64_t)kTile, p.plan.rows - (int64_t)c.tile * kTile);
        c.cols = len - c.t0 * kTile;
        c.nt = min(n, (len + kTile - 1) / kTile - c.t0);
    }
    return true;
}
// The i-th chunk, or null at the end (and after a wait that expired: `ok` false).
template <int D>
__device__ __forceinline__ const Chunk *chunk_at(const BwdParams &p, Shared<D> &sh, uint32_t i, bool &ok) {
    const int at = i % kChunks;
    ok = __all_sync(0xffffffffu, wait_soon(&sh.ch_full[at], (i / kChunks) & 1, &sh.abort_flag, p.status));
    return ok && sh.ch[at].nt >= 0 ? &sh.ch[at] : nullptr;
}
template <int D> __device__ __forceinline__ void chunk_done(Shared<D> &sh, uint32_t i, int lane) {
    warp_arrive(&sh.ch_empty[i % kChunks], lane);
}

// The CTA's chunks, and the copies of their tiles.
template <int D, bool KEY>
__device__ void copy_role(const BwdParams &p, const BwdMaps &maps, Shared<D> &sh, int lane) {
    using C = Cfg<D>;
    volatile int *abort_flag = &sh.abort_flag;
    const bool leader = elect_one();    // issues; the whole warp runs the loop
    auto wait_w = [&](uint64_t *b, uint32_t par) -> bool {
        return __all_sync(0xffffffffu, wait_soon(b, par, abort_flag, p.status));
    };
    auto load = [&](uint8_t *dst, const CUtensorMap *map, uint64_t *bar, int row, int slab) {
        for (int h = 0; h < C::HALVES; ++h) tma_load_3d(dst + h * (kTile * 128), map, bar, 64 * h, row, slab);
    };
    uint32_t u = 0, g = 0, ntail = 0;
    bool ok = true, more = true;
    Walk walk = walk_begin(p, lane);
    for (uint32_t i = 0; ok; ++i) {
        const int at = i % kChunks;
        if (!(ok = wait_w(&sh.ch_empty[at], ((i / kChunks) & 1) ^ 1))) break;
        Chunk c{};
        more = walk_next<KEY>(p, walk, c, lane == 0);
        if (!more) c.nt = -1;
        if (lane == 0) {
            sh.ch[at] = c;
            mbar_arrive(&sh.ch_full[at]);
        }
        __syncwarp();
        if (!more) break;
        if (c.nt == 0) continue;
        const int ub = u % C::UB;
        if (!(ok = wait_w(&sh.u_empty[ub], ((u / C::UB) & 1) ^ 1))) break;
        if (leader) {
            mbar_expect_tx(&sh.u_full[ub], 2 * C::TILE);
            load(sh.a0[ub], &maps.a0, &sh.u_full[ub], c.tile * kTile, (int)c.slab);
            load(sh.a1[ub], &maps.a1, &sh.u_full[ub], c.tile * kTile, (int)c.slab);
        }
        __syncwarp();
        ++u;
        for (int t = 0; t < c.nt; ++t) {
            const int st = g % C::STAGES;
            if (!(ok = wait_w(&sh.st_empty[st], ((g / C::STAGES) & 1) ^ 1))) break;
            const int row = (c.t0 + t) * kTile;
            // !KEY: rows of K behind the length that are in the buffer (behind it the copy fills zeros)
            const int z0 = c.cols - t * kTile, z1 = KEY ? 0 : (int)min((int64_t)kTile, p.plan.s.n - row);
            const bool zero = !KEY && z0 < z1;
            uint64_t *bar = zero ? &sh.tail : &sh.st_full[st];
            if (leader && !((int64_t)g == p.withhold && this_cta(p) == 0)) {
                mbar_expect_tx(bar, 2 * C::TILE + (KEY ? kStat * 4 : 0));
                load(sh.b0[st], &maps.b0, bar, row, (int)c.slab);
                load(sh.b1[st], &maps.b1, bar, row, (int)c.slab);
                if (KEY) bulk_load(sh.stat[st], p.stat + (c.slab * p.qtiles + c.t0 + t) * kStat, kStat * 4, bar);
            }
            __syncwarp();
            ++g;
            if (zero) {
                ok = wait_w(&sh.tail, ntail & 1);
                if (!ok) drain_bar(&sh.tail, ntail & 1);
                ++ntail;
                if (ok) {
                    for (int h = 0; h < C::HALVES; ++h) {
                        uint4 *rows = reinterpret_cast<uint4 *>(sh.b0[st] + h * (kTile * 128));
                        for (int e = z0 * 8 + lane; e < z1 * 8; e += 32) rows[e] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async();
                }
                __syncwarp();
                if (leader) mbar_arrive(&sh.st_full[st]);
                if (!ok) break;
            }
        }
    }
    if (!ok) {                              // let the copies in flight land before the CTA exits
        for (uint32_t i = g > (uint32_t)C::STAGES ? g - C::STAGES : 0; i < g; ++i)
            drain_bar(&sh.st_full[i % C::STAGES], (i / C::STAGES) & 1);
        for (uint32_t i = u > (uint32_t)C::UB ? u - C::UB : 0; i < u; ++i)
            drain_bar(&sh.u_full[i % C::UB], (i / C::UB) & 1);
    }
}

constexpr uint32_t kColS = 0, kColDp = 128;
// P and dS take the place of S and dP
template <int D, bool KEY> constexpr bool kInPlace = KEY && D == 128;
// Then a step's columns are handed over in two halves with barriers of their own: one half's softmax runs
// beside the products that the other's columns have to wait for (three entries of 4004 rows and up to 2345
// keys, dk and dv: 70 us, in one piece 76.5). Elsewhere S and dP of the next step are formed ahead, and
// twice as many products of half the width cost more than the halves gain (12288 x 12288, 8 heads,
// D = 64: 735 us, in one piece 718).
template <int D, bool KEY> constexpr int kParts = kInPlace<D, KEY> ? 2 : 1;
template <int D, bool KEY> constexpr int kWide = kTile / kParts<D, KEY>;    // columns of a part
// P and dS of columns 32w..32w+31 of a step
template <int D, bool KEY> __device__ __forceinline__ uint32_t col_p(int w) { return kInPlace<D, KEY> ? 32u * w : 256u + 16u * w; }
template <int D, bool KEY> __device__ __forceinline__ uint32_t col_ds(int w) {
    return kInPlace<D, KEY> ? 128u + 32u * w : (KEY ? 320u : 256u) + 16u * w;
}
constexpr uint32_t kDsLow = 192;            // !KEY: from a column of dS to that of what its rounding leaves off
template <int D, bool KEY> constexpr uint32_t kColV = D == 64 ? 384u : 256u;
template <int D, bool KEY> constexpr uint32_t kColK = !KEY ? 320u : (D == 64 ? 448u : 384u);

// S and dP of every step.
template <int D, bool KEY>
__device__ void score_role(const BwdParams &p, Shared<D> &sh, uint32_t tmem, int lane) {
    using C = Cfg<D>;
    volatile int *abort_flag = &sh.abort_flag;
    const bool leader = elect_one();
    auto wait_w = [&](uint64_t *b, uint32_t par) -> bool {
        return __all_sync(0xffffffffu, wait_soon(b, par, abort_flag, p.status));
    };
    const uint64_t a0 = desc_kmajor_sw128(sh.a0[0]), a1 = desc_kmajor_sw128(sh.a1[0]);
    const uint64_t b0 = desc_kmajor_sw128(sh.b0[0]), b1 = desc_kmajor_sw128(sh.b1[0]);
    constexpr int PARTS = kParts<D, KEY>, WIDE = kWide<D, KEY>;
    // part h of a step's columns
    auto product = [&](uint32_t col, uint64_t a, uint64_t b, int h) __attribute__((always_inline)) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = (kk / 4) * ((kTile * 128) >> 4) + 2 * (kk % 4);
            mma_bf16(tmem + col + WIDE * h, a + off, b + off + h * ((WIDE * 128) >> 4), idesc_of(WIDE, false), kk > 0);
        }
    };
    uint32_t u = 0, g = 0;
    bool ok = true;
    const Chunk *cp;
    for (uint32_t i = 0; ok && (cp = chunk_at<D>(p, sh, i, ok)); ++i) {
        const int nt = uniform(cp->nt);
        chunk_done<D>(sh, i, lane);
        if (nt == 0) continue;
        const int ub = u % C::UB;
        if (!(ok = wait_w(&sh.u_full[ub], (u / C::UB) & 1))) break;
        ++u;
        for (int t = 0; t < nt; ++t, ++g) {
            const int st = g % C::STAGES;
            if (!(ok = wait_w(&sh.st_full[st], (g / C::STAGES) & 1))) break;
            for (int h = 0; h < PARTS; ++h) {
                // the columns of S are free: read by the softmax, or (P in their place) by P·B1
                if (g > 0 && !(ok = wait_w(kInPlace<D, KEY> ? &sh.v_done[h] : &sh.s_free[h], (g - 1) & 1))) break;
                fence_after();
                if (leader) {
                    product(kColS, a0 + (uint64_t)(ub * (C::TILE >> 4)), b0 + (uint64_t)(st * (C::TILE >> 4)), h);
                    commit(&sh.s_full[h]);
                }
                __syncwarp();
            }
            for (int h = 0; h < PARTS && ok; ++h) {
                // those of dP: read, as dS of the step before is written, or (dS in their place) used up
                if (g > 0 && !(ok = wait_w(kInPlace<D, KEY> ? &sh.k_done[h] : &sh.ds_full[h], (g - 1) & 1))) break;
                fence_after();
                if (leader) {
                    product(kColDp, a1 + (uint64_t)(ub * (C::TILE >> 4)), b1 + (uint64_t)(st * (C::TILE >> 4)), h);
                    commit(&sh.dp_full[h]);
                    if (h == PARTS - 1) {
                        commit(&sh.st_empty[st]);
                        if (t + 1 == nt) commit(&sh.u_empty[ub]);
                    }
                }
                __syncwarp();
            }
            if (!ok) break;
        }
    }
    // every MMA this warp issued must be complete before TMEM is freed
    if (leader) commit(&sh.drain[0]);
    __syncwarp();
    drain_bar(&sh.drain[0], 0);
}

// acc0 += P·B1 (V) or acc1 += dS·B0 of every step.
template <int D, bool KEY, bool V>
__device__ void grad_role(const BwdParams &p, Shared<D> &sh, uint32_t tmem, int lane) {
    using C = Cfg<D>;
    constexpr int PARTS = kParts<D, KEY>, WIDE = kWide<D, KEY>;
    constexpr uint32_t A_STEP = kInPlace<D, KEY> ? 32 : 16;    // columns of P and dS from w to w + 1
    volatile int *abort_flag = &sh.abort_flag;
    const bool leader = elect_one();
    auto wait_w = [&](uint64_t *b, uint32_t par) -> bool {
        return __all_sync(0xffffffffu, wait_soon(b, par, abort_flag, p.status));
    };
    const uint64_t b0 = desc_mnmajor_sw128(V ? sh.b1[0] : sh.b0[0], kTile * 128);
    const uint32_t acc = tmem + (V ? kColV<D, KEY> : kColK<D, KEY>), from = tmem + (V ? col_p<D, KEY>(0) : col_ds<D, KEY>(0));
    uint32_t u = 0, g = 0;
    bool ok = true;
    const Chunk *cp;
    for (uint32_t i = 0; ok && (cp = chunk_at<D>(p, sh, i, ok)); ++i) {
        const int nt = uniform(cp->nt);
        chunk_done<D>(sh, i, lane);
        if (nt == 0) continue;
        if (u > 0 && !(ok = wait_w(&sh.acc_free, (u - 1) & 1))) break;
        ++u;
        for (int t = 0; t < nt; ++t, ++g) {
            const int st = g % C::STAGES;
            for (int h = 0; h < PARTS; ++h) {
                if (!(ok = wait_w(V ? &sh.p_full[h] : &sh.ds_full[h], g & 1))) break;
                fence_after();
                if (leader) {
                    const uint64_t b = b0 + (uint64_t)(st * (C::TILE >> 4)) + 8 * WIDE * h;
                    const uint32_t a = from + WIDE / 32 * A_STEP * h;
#pragma unroll
                    for (int kk = 0; kk < WIDE / 16; ++kk)    // blocks of 16 columns of the step
                        mma_ts(acc, a + A_STEP * (kk >> 1) + 8u * (kk & 1), b + 128 * kk, idesc_of(D, true), t > 0 || h > 0 || kk > 0);
                    if constexpr (!KEY) {
#pragma unroll
                        for (int kk = 0; kk < WIDE / 16; ++kk)
                            mma_ts(acc, a + kDsLow + 8u * kk, b + 128 * kk, idesc_of(D, true), 1u);
                    }
                    commit(V ? &sh.v_done[h] : &sh.k_done[h]);
                    if (h == PARTS - 1) {
                        commit(&sh.st_empty[st]);
                        if (t + 1 == nt) commit(&sh.acc_full);
                    }
                }
                __syncwarp();
            }
            if (!ok) break;
        }
    }
    if (leader) commit(&sh.drain[V ? 1 : 2]);
    __syncwarp();
    drain_bar(&sh.drain[V ? 1 : 2], 0);
}

template <int D, bool KEY>
__device__ void softmax_role(const BwdParams &p, Shared<D> &sh, uint32_t tmem, int w, int wq, int lane) {
    using C = Cfg<D>;
    constexpr bool IN_PLACE = kInPlace<D, KEY>;
    volatile int *abort_flag = &sh.abort_flag;
    auto wait_all = [&](uint64_t *b, uint32_t par) -> bool {
        return __all_sync(0xffffffffu, wait_soon(b, par, abort_flag, p.status));
    };
    const uint32_t tw = tmem + ((uint32_t)(32 * wq) << 16);
    const int row = 32 * wq + lane;          // this thread's row of the unit
    const int part = w / (kWide<D, KEY> / 32);   // its part of a step
    const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
    uint32_t u = 0, g = 0;
    bool ok = true;
    const Chunk *cp;
    for (uint32_t i = 0; ok && (cp = chunk_at<D>(p, sh, i, ok)); ++i) {
        const int nt = uniform(cp->nt), cols = uniform(cp->cols);
        const bool counts = row < cp->rows;
        float lse = -CUDART_INF_F, dt = 0.f;       // negated
        if (!KEY && counts && nt > 0) {
            const float *st = p.stat + (cp->slab * p.qtiles + cp->tile) * kStat + row;
            lse = __ldg(st);
            dt = __ldg(st + kTile);
        }
        for (int t = 0; t < nt; ++t, ++g) {
            const int st = g % C::STAGES;
            if (!(ok = wait_all(&sh.s_full[part], g & 1))) break;
            // KEY: the statistics arrived with the step's tiles; this thread's own wait on their barrier (long
            // complete) makes the copied values visible to it
            if (KEY && !(ok = wait_all(&sh.st_full[st], (g / C::STAGES) & 1))) break;
            fence_after();
            float x[32];
            tmem_ld32(tw + kColS + 32u * w, x);
            tmem_wait_ld_of(x);
            if constexpr (!IN_PLACE) {
                fence_before();
                warp_arrive(&sh.s_free[part], lane);
            }
            // p = 2^(c·log2 e·s - lse·log2 e), in place, 16 at a time
            const float4 *ls4 = reinterpret_cast<const float4 *>(sh.stat[st] + 32 * w);
            const float4 *dd4 = reinterpret_cast<const float4 *>(sh.stat[st] + kTile + 32 * w);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float2 e2[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 l4 = KEY ? ls4[4 * h + e] : make_float4(lse, lse, lse, lse);
                    const int c = 16 * h + 4 * e;
                    e2[2 * e] = __ffma2_rn(make_float2(x[c], x[c + 1]), sl2, make_float2(l4.x, l4.y));
                    e2[2 * e + 1] = __ffma2_rn(make_float2(x[c + 2], x[c + 3]), sl2, make_float2(l4.z, l4.w));
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    e2[e] = make_float2(ex2(e2[e].x), ex2(e2[e].y));
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[16 * h + 2 * e] = e2[e].x;
                    x[16 * h + 2 * e + 1] = e2[e].y;
                }
            }
            // this thread's columns that count (KEY: read anew in each step, 1,645 us for a training step of 12288 x 12288,
            // 8 heads, D = 64; with a register for it over the loop 1,656, without this mask 1,635)
            const int valid = (KEY ? *(volatile const int *)&cp->cols : cols) - t * kTile - 32 * w;
            if (KEY && !counts) {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = 0.f;
            }
            if (valid < 32) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (e >= valid) x[e] = 0.f;
            }
            // the columns that P and dS take are free: the gradients' products of the step before have read them
            // (in place: before this S and this dP began)
            if (KEY && !IN_PLACE && g > 0 && !(ok = wait_all(&sh.v_done[part], (g - 1) & 1))) break;
            if constexpr (KEY) {
                fence_after();
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) pk[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
                tmem_st16w(tw + col_p<D, KEY>(w), pk);
                tmem_wait_st();
                fence_before();
                warp_arrive(&sh.p_full[part], lane);
            }
            if (!(ok = wait_all(&sh.dp_full[part], g & 1))) break;
            fence_after();
            float d[32];
            uint32_t ds[16], low[16];
            tmem_ld32(tw + kColDp + 32u * w, d);
            tmem_wait_ld_of(d);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float4 d4 = KEY ? dd4[e] : make_float4(dt, dt, dt, dt);
                const int c = 4 * e;
                const float2 a = __fmul2_rn(make_float2(x[c], x[c + 1]),
                                            __fadd2_rn(make_float2(d[c], d[c + 1]), make_float2(d4.x, d4.y)));
                const float2 b = __fmul2_rn(make_float2(x[c + 2], x[c + 3]),
                                            __fadd2_rn(make_float2(d[c + 2], d[c + 3]), make_float2(d4.z, d4.w)));
                ds[2 * e] = pack_bf16x2(a.x, a.y);
                ds[2 * e + 1] = pack_bf16x2(b.x, b.y);
                if (!KEY) {
                    low[2 * e] = rest_bf16x2(a.x, a.y, ds[2 * e]);
                    low[2 * e + 1] = rest_bf16x2(b.x, b.y, ds[2 * e + 1]);
                }
            }
            // what does not count is 0 whatever dP holds there (0·NaN)
            if (KEY ? !counts : valid < 32) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint32_t keep = KEY || 2 * e >= valid ? 0u : (2 * e + 1 >= valid ? 0xffffu : 0xffffffffu);
                    ds[e] &= keep;
                    if (!KEY) low[e] &= keep;
                }
            }
            if (!IN_PLACE && g > 0 && !(ok = wait_all(&sh.k_done[part], (g - 1) & 1))) break;
            fence_after();
            tmem_st16w(tw + col_ds<D, KEY>(w), ds);
            if (!KEY) tmem_st16w(tw + col_ds<D, KEY>(w) + kDsLow, low);
            tmem_wait_st();
            fence_before();
            warp_arrive(&sh.ds_full[part], lane);
        }
        if (!ok) break;
        if (nt > 0) {
            if (!(ok = wait_all(&sh.acc_full, u & 1))) break;
            ++u;
            fence_after();
        }
        // KEY: w = 0, 1 store dv's columns, 2, 3 dk's (nothing where no key counts); !KEY: dq's, D / 4 each
        // (D = 64: w = 0, 1)
        const int grad = KEY ? w >> 1 : 1, piece = KEY ? w & 1 : w, wide = KEY ? D / 2 : 32;
        const uint32_t col = grad == 0 ? kColV<D, KEY> : kColK<D, KEY>;
        const int64_t at = cp->slab * (KEY ? p.plan.s.n : p.plan.rows) + (int64_t)cp->tile * kTile + row;
        const int slot = cp->slot;
        __nv_bfloat16 *d16 = (!KEY ? p.dq : grad == 0 ? p.dv : p.dk) + at * D;
        float *d32 = p.part + ((2 * (int64_t)this_cta(p) + max(slot, 0)) * kTile + row) * (KEY ? 2 * D : D) + (KEY ? grad * D : 0);
        const int c0 = piece * wide;
        if (nt > 0 && c0 < D) {
            // staged in the unit's own tiles, which no product reads any more
            const int ub = (u + C::UB - 1) % C::UB;
            uint8_t *stage = (4 * w + wq < 8 ? sh.a0[ub] : sh.a1[ub]) + 2048 * ((4 * w + wq) & 7);
            write_rows(stage, tw + col + c0, wide, grad == 0 ? 1.f : p.scale, false, slot < 0,
                       slot < 0 ? static_cast<void *>(d16 + c0) : d32 + c0, nullptr, counts, lane);
        } else if (!KEY && c0 < D && counts) {         // no keys: zeros (and the unit has no tiles here)
            for (int e = 0; e < 4; ++e) reinterpret_cast<uint4 *>(d16 + c0)[e] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_before();
        if (nt > 0) {
            // the staged rows are read, and the copies may overwrite them (another proxy)
            fence_proxy_async();
            warp_arrive(&sh.u_empty[(u + C::UB - 1) % C::UB], lane);
            warp_arrive(&sh.acc_free, lane);
        }
        chunk_done<D>(sh, i, lane);
    }
}

template <int D, bool KEY> __device__ __forceinline__ void bwd_cta(const BwdMaps &maps, const BwdParams &p) {
    extern __shared__ uint8_t smem_raw[];
    Shared<D> &sh = *reinterpret_cast<Shared<D> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        sh.abort_flag = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.u_full[i], 1);
            mbar_init(&sh.u_empty[i], 1 + kSoftWarps);     // the scores' products, and the epilogue
        }
        for (int i = 0; i < 3; ++i) mbar_init(&sh.drain[i], 1);
        for (int i = 0; i < Cfg<D>::STAGES; ++i) {
            mbar_init(&sh.st_full[i], 1);
            mbar_init(&sh.st_empty[i], KEY ? 3 : 2);     // the MMA warps
        }
        for (int i = 0; i < kChunks; ++i) {
            mbar_init(&sh.ch_full[i], 1);
            mbar_init(&sh.ch_empty[i], kReaders<KEY>);
        }
        mbar_init(&sh.tail, 1);
        constexpr int WARPS = kSoftWarps / kParts<D, KEY>;      // softmax warps of a part
        for (int h = 0; h < kParts<D, KEY>; ++h) {
            mbar_init(&sh.s_full[h], 1);
            mbar_init(&sh.dp_full[h], 1);
            mbar_init(&sh.s_free[h], WARPS);
            mbar_init(&sh.p_full[h], WARPS);
            mbar_init(&sh.ds_full[h], WARPS);
            mbar_init(&sh.v_done[h], 1);
            mbar_init(&sh.k_done[h], 1);
        }
        mbar_init(&sh.acc_full, KEY ? 2 : 1);
        mbar_init(&sh.acc_free, kSoftWarps);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane == 0) {
        prefetch_map(&maps.a0);
        prefetch_map(&maps.a1);
        prefetch_map(&maps.b0);
        prefetch_map(&maps.b1);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem_base))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem_base;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtrlRegs));
        if (warp == 0) copy_role<D, KEY>(p, maps, sh, lane);
        else if (warp == 1) score_role<D, KEY>(p, sh, tmem, lane);
        else if (warp == 3) grad_role<D, KEY, false>(p, sh, tmem, lane);
        else if (KEY) grad_role<D, KEY, true>(p, sh, tmem, lane);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        softmax_role<D, KEY>(p, sh, tmem, (warp - 4) >> 2, warp & 3, lane);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// Both passes in one launch, dk's and dv's CTAs first: few units of either run beside one another, and of
// many the dq pass begins on each SM as the other ends there (768 rows, 200 keys, 2 heads, D = 64: 14 us, in two
// launches 23).
template <int D>
__global__ void __launch_bounds__(NTHREADS, 1) bwd_kernel(const __grid_constant__ BwdMaps maps_key, const __grid_constant__ BwdParams key,
                                                          const __grid_constant__ BwdMaps maps_qry, const __grid_constant__ BwdParams qry) {
    if ((int)blockIdx.x < qry.cta0) bwd_cta<D, true>(maps_key, key);
    else bwd_cta<D, false>(maps_qry, qry);
}

// ---------------------------------------------------------------- parts added

// The unit that CTA ca began and left: the sum of its parts in the order of their CTAs. A warp has
// kRows rows (KEY: of dv and of dk beside one another), all of whose parts of a CTA load together.
constexpr int kJoinRows = 4;
template <int D, bool KEY> __device__ __forceinline__ void add_parts(const BwdParams &p, int ca, int i0, int lane) {
    const Cut cut = p.cuts[ca];
    if (cut.last < ca || cut.last >= p.plan.ctas) return;
    const FwdSet &s = p.plan.s;
    constexpr int W = KEY ? 2 * D : D, E = W / 64;     // floats of a row; pairs of them a lane
    const int64_t all = KEY ? s.n : p.plan.rows;
    const int count = KEY ? set_len(s.len, cut.z, s.n, nullptr) : (int)all;
    const int64_t base = ((int64_t)cut.z * p.plan.kv_heads + cut.hk) * all;
    float2 sum[kJoinRows][E];
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r)
#pragma unroll
        for (int e = 0; e < E; ++e) sum[r][e] = make_float2(0.f, 0.f);
    for (int c = ca; c <= cut.last; ++c) {
        const float2 *src = reinterpret_cast<const float2 *>(p.part + ((2 * (int64_t)c + (c == ca)) * kTile + i0) * W);
#pragma unroll
        for (int r = 0; r < kJoinRows; ++r) {
            if (cut.tile * kTile + i0 + r >= count) continue;      // a row that does not count was not written
#pragma unroll
            for (int e = 0; e < E; ++e) sum[r][e] = __fadd2_rn(sum[r][e], __ldg(src + r * (W / 2) + 32 * e + lane));
        }
    }
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) {
        const int64_t row = cut.tile * kTile + i0 + r;
        if (row >= count) continue;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int col = 2 * (32 * e + lane);                   // of [dv | dk] or of dq
            __nv_bfloat16 *dst = !KEY ? p.dq + (base + row) * D + col
                                      : (col < D ? p.dv + (base + row) * D + col : p.dk + (base + row) * D + col - D);
            *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(sum[r][e].x, sum[r][e].y);
        }
    }
}
// Blocks [0, key_blocks): dk and dv; the rest: dq. kTile / (8 kJoinRows) blocks a CTA's cut.
template <int D>
__global__ void __launch_bounds__(256) bwd_join_kernel(const __grid_constant__ BwdParams key, const __grid_constant__ BwdParams qry,
                                                       int key_blocks) {
    constexpr int PER = kTile / (8 * kJoinRows);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.x;
    if (b < key_blocks) add_parts<D, true>(key, b / PER, (b % PER * 8 + warp) * kJoinRows, lane);
    else add_parts<D, false>(qry, (b - key_blocks) / PER, ((b - key_blocks) % PER * 8 + warp) * kJoinRows, lane);
}

// ---------------------------------------------------------------- host

struct BwdPlans {
    FwdPlan key, qry;
    int64_t qtiles;
    size_t stat, key_part, qry_part, key_cuts, qry_cuts, total;
};

BwdPlans make_plans(const DenseProblem &p, const KeySet &ks) {
    BwdPlans r{};
    const bool scan = !ks.len || ks.sets <= 1024;
    r.qtiles = (p.rows + kTile - 1) / kTile;
    const int64_t kt = (ks.n + kTile - 1) / kTile;
    FwdPlan f{};
    f.rows = p.rows;
    f.kv_heads = p.kv_heads;
    f.batch = p.batch;
    f.s.len = ks.len;
    f.s.n = ks.n;
    f.s.sets = ks.sets;
    f.s.members = 1;
    f.s.tpm = (int32_t)r.qtiles;
    f.s.tiles = f.s.pairs = r.qtiles;
    f.s.upz = p.kv_heads * r.qtiles;
    r.qry = r.key = f;
    r.key.s.fixed = (int32_t)r.qtiles;      // upz: the steps of a set for each of its key tiles
    deal(r.qry, ks.sets * f.s.upz, kt, scan);
    deal(r.key, ks.sets * p.kv_heads * kt, r.qtiles, scan);
    size_t o = 0;
    auto take = [&](size_t floats) { const size_t at = o; o += (floats + 63) / 64 * 64; return at; };
    r.stat = take((size_t)p.batch * p.kv_heads * r.qtiles * kStat);
    if (r.key.stream) {
        r.key_part = take((size_t)r.key.ctas * 4 * kTile * p.d);
        r.key_cuts = take((size_t)r.key.ctas * 4);
    }
    if (r.qry.stream) {
        r.qry_part = take((size_t)r.qry.ctas * 2 * kTile * p.d);
        r.qry_cuts = take((size_t)r.qry.ctas * 4);
    }
    r.total = o;
    return r;
}

bool row_map(CUtensorMap *m, const void *base, int64_t d, int64_t rows, int64_t slabs) {
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)slabs};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)rows * d * 2};
    const cuuint32_t b[3] = {64, kTile, 1};
    return make_map(m, base, 3, dims, strides, b);
}

template <int D>
cudaError_t launch(const DenseProblem &pb, const void *q, const KeySet &ks, const void *out, const void *low,
                   const float *lse, const void *dout, const BwdPlans &plans, const BwdParams &key, const BwdParams &qry, float *stat,
                   cudaStream_t stream) {
    const int64_t slabs = pb.batch * pb.kv_heads;
    BwdMaps mk, mq;
    if (!row_map(&mk.a0, ks.k, D, ks.n, slabs) || !row_map(&mk.a1, ks.v, D, ks.n, slabs) ||
        !row_map(&mk.b0, q, D, pb.rows, slabs) || !row_map(&mk.b1, dout, D, pb.rows, slabs))
        return cudaErrorInvalidValue;
    mq.a0 = mk.b0;
    mq.a1 = mk.b1;
    mq.b0 = mk.a0;
    mq.b1 = mk.a1;
    const size_t smem = sizeof(Shared<D>) + 1024;
    static_assert(sizeof(Shared<D>) + 1024 <= 232448, "shared memory");
    cudaError_t e = kernel_ready<bwd_kernel<D>>(smem, NTHREADS, kRegsNeeded);
    if (e != cudaSuccess) return e;
    const int64_t rows_a_block = 256 / (D / 8), stat_blocks = (slabs * plans.qtiles * kTile + rows_a_block - 1) / rows_a_block;
    bwd_stat_kernel<D><<<(unsigned)(stat_blocks < 8 * kCtas ? stat_blocks : 8 * kCtas), 256, 0, stream>>>(
        key, static_cast<const __nv_bfloat16 *>(out), static_cast<const __nv_bfloat16 *>(low), lse, static_cast<const __nv_bfloat16 *>(dout), stat, slabs);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    bwd_kernel<D><<<key.plan.ctas + qry.plan.ctas, NTHREADS, smem, stream>>>(mk, key, mq, qry);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    constexpr int PER = kTile / (8 * kJoinRows);
    const int kb = key.cuts ? key.plan.ctas * PER : 0, qb = qry.cuts ? qry.plan.ctas * PER : 0;
    if (kb + qb > 0) bwd_join_kernel<D><<<kb + qb, 256, 0, stream>>>(key, qry, kb);
    return cudaGetLastError();
}

}  // namespace

size_t dense_bwd_floats(const DenseProblem &p, const KeySet &s) { return make_plans(p, s).total; }

cudaError_t launch_dense_bwd(const DenseProblem &pb, const void *q, const KeySet &ks, const void *out, const void *low,
                             const float *lse, const void *dout, void *dq, void *dk, void *dv, float *ws, uint32_t *status,
                             cudaStream_t stream) {
    const BwdPlans plans = make_plans(pb, ks);
    BwdParams key{};
    key.plan = plans.key;
    key.stat = ws + plans.stat;
    key.qtiles = plans.qtiles;
    key.dq = static_cast<__nv_bfloat16 *>(dq);
    key.dk = static_cast<__nv_bfloat16 *>(dk);
    key.dv = static_cast<__nv_bfloat16 *>(dv);
    key.part = ws + plans.key_part;
    key.cuts = plans.key.stream ? reinterpret_cast<Cut *>(ws + plans.key_cuts) : nullptr;
    key.scale = pb.scale;
    key.scale_log2 = pb.scale * 1.4426950408889634f;
    key.status = status;
    key.withhold = pb.withhold;
    BwdParams qry = key;
    qry.plan = plans.qry;
    qry.cta0 = plans.key.ctas;
    qry.part = ws + plans.qry_part;
    qry.cuts = plans.qry.stream ? reinterpret_cast<Cut *>(ws + plans.qry_cuts) : nullptr;
    float *stat = ws + plans.stat;
    return pb.d == 64 ? launch<64>(pb, q, ks, out, low, lse, dout, plans, key, qry, stat, stream)
                      : launch<128>(pb, q, ks, out, low, lse, dout, plans, key, qry, stat, stream);
}

}  // namespace bsa
