// Dense softmax attention of query rows to states of another length on the
// sm_100a tensor cores (bf16, head_dim D = 64 or 128, fp32 accumulation).
//
// Row i of a batch entry and key head (the query rows of all heads that share
// the key head, which lie one behind the other) against keys j < len:
//   s_ij = q_i·k_j (·s log2 e),  m_i = max_j s_ij (lazily: it may lag by up to 2^8),
//   p_ij = 2^(s_ij - m_i),  l_i = Σ_j p_ij,  o_i = Σ_j p_ij v_j / l_i.
// A step is one tile of 128 keys: S = Q·Kᵀ (tcgen05.mma, M = N = 128) into tensor
// memory, softmax numerators by 128 threads (a thread owns a row), P as bf16 pairs
// back into tensor memory, O += P·V with P as the A operand from there.
//
// Organisation: one persistent CTA per SM, 384 threads, two pipelines:
//   warp 0       copies (TMA, 128-byte swizzle): Q of a unit, then K and V tiles
//                through one ring that both pipelines read
//   warps 1, 2   the MMA warp of pipeline 0 and of pipeline 1
//   warp 3       finds the CTA's first unit
//   warps 4-7, 8-11  softmax and epilogue of pipeline 0 and of pipeline 1
// Many rows: the pipelines hold two tiles of 128 rows of one unit and both take
// every key tile, so K and V are read once for 256 rows, and one pipeline's
// products run beside the other's softmax. Few rows (at most 32: a decoding step's
// query heads, or an ensemble's members together): both hold the same rows, four
// times over in the four 32-lane quarters of tensor memory, and take alternate key
// tiles; warp w of a pipeline does the softmax of its tile's keys 32w..32w+31 only
// (P is zero elsewhere in its lanes). So the exponentials of a tile are spread over
// all threads although there are few rows, and the eight partial rows are merged by
// their maxima and sums at the unit's end.
//
// Tensor memory (512 columns): D = 64: S0 S1 (128 each), P0 P1 (64 each), O0 O1 (64
// each); S of the next step is formed while this one's softmax runs. D = 128: S0 S1,
// O0 O1 (128 each); P takes the first 64 columns of its S, and S of the next step
// follows P·V in the issue order of its pipeline.
//
// Keys behind a length: scores are replaced before the maximum (whatever K holds),
// and the copy warp zeroes those rows of V in shared memory, since 0·NaN is NaN.
//
// Every wait on an mbarrier is bounded (2 s), as in the block-sparse kernel.
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
constexpr float kRescaleLog2 = 8.0f;
constexpr float kLn2 = 0.69314718055994531f;

template <int D> struct Cfg {
    static constexpr int HALVES = D / 64;              // 128-byte column groups of a row
    static constexpr int TILE = kTile * D * 2;         // bytes of a 128-row tile
    static constexpr int STAGES = D == 64 ? 9 : 4;     // ring of K and V tiles
    static constexpr int MROWS = D == 64 ? 16 : 4;     // rows merged at a time (few rows)
    static constexpr int MSTRIDE = D + 4;              // floats, padded against bank conflicts
};

template <int D> struct alignas(1024) Shared {
    uint8_t q[2][Cfg<D>::TILE];
    uint8_t kv[Cfg<D>::STAGES][Cfg<D>::TILE];
    float merge[8][Cfg<D>::MROWS][Cfg<D>::MSTRIDE];
    float ml[2][8][32];                                // few rows: (m, l) of each partial row
    uint64_t q_full[2], q_empty[2], kv_full[Cfg<D>::STAGES], kv_empty[Cfg<D>::STAGES], tail;
    uint64_t s_full[2], s_free[2], p_full[2], o_done[2], merge_bar, drain[2];
    int64_t first, last;                               // stream: the CTA's steps
    StepAt at;
    uint32_t tmem_base;
    int abort_flag;
};

struct FwdParams {
    FwdPlan plan;
    __nv_bfloat16 *out;     // [rows of all][D]
    float *lse;             // nullable
    float *part_o, *part_lse, *whole_o, *whole_lse;
    int64_t all_rows;       // batch * kv_heads * rows
    float scale_log2;
    uint32_t *status;       // nullable
};

struct Maps {
    CUtensorMap q[2], k[2], v[2];
};

// What a CTA does next: key tiles [t0, t0 + nt) of a unit. slot -1: the whole unit.
struct Chunk {
    int set, t0, nt, len, slot;
    int64_t z, hk, pair;
};
struct Walk {
    int set, t, steps;
    int64_t z, uu, left;    // stream: steps left; whole: the unit's index
};
template <int D> __device__ __forceinline__ Walk walk_begin(const FwdParams &p, const Shared<D> &sh) {
    Walk w;
    if (p.plan.stream) {
        w.set = sh.at.set;
        w.t = sh.at.t;
        w.steps = sh.at.steps;
        w.z = sh.at.z;
        w.uu = sh.at.uu;
        w.left = sh.last - sh.first;
    } else {
        w.left = blockIdx.x;
    }
    return w;
}
__device__ __forceinline__ bool walk_next(const FwdParams &p, Walk &w, Chunk &c, uint32_t *status) {
    int steps;
    if (p.plan.stream) {
        if (w.left <= 0) return false;
        const FwdSet *s = &p.plan.s[w.set];
        if (w.t == w.steps) {                          // the next unit
            w.t = 0;
            if (++w.uu == s->upz) {
                w.uu = 0;
                if (++w.z == s->sets) {
                    w.z = 0;
                    if (++w.set == p.plan.nsets) return false;
                    s = &p.plan.s[w.set];
                }
                w.steps = set_steps(*s, w.z);
            }
        }
        c.set = w.set;
        c.z = w.z;
        c.hk = w.uu / s->pairs;
        c.pair = w.uu - c.hk * s->pairs;
        c.t0 = w.t;
        steps = (int)min((int64_t)(w.steps - w.t), w.left);
        c.slot = steps == w.steps ? -1 : (w.t > 0 ? 0 : 1);
        w.t += steps;
        w.left -= steps;
    } else {
        int64_t u = w.left;
        c.set = 0;
        const int64_t n0 = p.plan.s[0].sets * p.plan.s[0].upz;
        if (u >= n0) {
            u -= n0;
            c.set = 1;
            if (p.plan.nsets == 1 || u >= p.plan.s[1].sets * p.plan.s[1].upz) return false;
        }
        const FwdSet &s = p.plan.s[c.set];
        c.z = u / s.upz;
        u -= c.z * s.upz;
        c.hk = u / s.pairs;
        c.pair = u - c.hk * s.pairs;
        c.t0 = 0;
        c.slot = -1;
        steps = 0x7fffffff;
        w.left += gridDim.x;
    }
    const FwdSet &s = p.plan.s[c.set];
    c.len = set_len(s.len, c.z, s.n, status);
    const int tiles = (c.len + kTile - 1) / kTile;
    c.nt = min(steps, tiles - c.t0);                   // 0 for a set without keys
    return true;
}

// Tiles in flight through the ring, in the order in which both pipelines take them: many rows and
// D = 64: K0 K1 V0 K2 V1 ... (S of the next step goes before this one's P·V), else K0 V0 K1 V1 ...
template <int D> __device__ __forceinline__ bool looks_ahead(bool few) { return D == 64 && !few; }

template <int D>
__device__ void copy_role(const FwdParams &p, const Maps &maps, Shared<D> &sh, int lane) {
    using C = Cfg<D>;
    volatile int *abort_flag = &sh.abort_flag;
    const bool leader = lane == 0;
    auto wait_w = [&](uint64_t *b, uint32_t par) -> bool {
        return __all_sync(0xffffffffu, wait_fast(b, par, abort_flag, p.status));
    };
    uint32_t pos = 0, nq[2] = {0, 0}, ntail = 0;
    bool ok = true;
    Chunk c;
    Walk w = walk_begin<D>(p, sh);
    while (ok && walk_next(p, w, c, leader ? p.status : nullptr)) {
        if (c.nt <= 0) continue;
        const FwdSet &s = p.plan.s[c.set];
        for (int pl = 0; pl < 2 && ok; ++pl) {
            const int64_t t = s.few ? 0 : 2 * c.pair + pl;
            if (t >= s.tiles) continue;
            if (!(ok = wait_w(&sh.q_empty[pl], (nq[pl] & 1) ^ 1))) break;
            if (leader) {
                const int64_t member = c.z * s.members + (s.bb ? t * s.bb : t / s.tpm);
                const int row = s.bb ? 0 : (int)(t % s.tpm) * kTile;
                const int box = (s.bb ? s.bb * (int)p.plan.rows : kTile) * 128;   // bytes of a copied box
                const int reps = s.few ? 4 : 1;
                mbar_expect_tx(&sh.q_full[pl], (uint32_t)(box * reps * C::HALVES));
                for (int h = 0; h < C::HALVES; ++h)
                    for (int r = 0; r < reps; ++r)
                        tma_load_4d(sh.q[pl] + h * (kTile * 128) + r * (32 * 128), &maps.q[c.set], &sh.q_full[pl],
                                    64 * h, row, (int)c.hk, (int)member);
            }
            __syncwarp();
            ++nq[pl];
        }
        const int slab = (int)(c.z * p.plan.kv_heads + c.hk);
        // one tile of K or V into the next stage of the ring
        auto put = [&](const CUtensorMap *map, int t, bool is_v) -> bool {
            const int st = pos % C::STAGES;
            if (!wait_w(&sh.kv_empty[st], ((pos / C::STAGES) & 1) ^ 1)) return false;
            const int row = (c.t0 + t) * kTile;
            // rows behind the length that are in the buffer (behind the buffer the copy fills zeros)
            const int z0 = c.len - row, z1 = (int)min((int64_t)kTile, s.n - row);
            const bool zero = is_v && z0 < z1;
            uint64_t *bar = zero ? &sh.tail : &sh.kv_full[st];
            if (leader) {
                mbar_expect_tx(bar, C::TILE);
                for (int h = 0; h < C::HALVES; ++h)
                    tma_load_3d(sh.kv[st] + h * (kTile * 128), map, bar, 64 * h, row, slab);
            }
            __syncwarp();
            ++pos;
            if (zero) {
                const bool there = wait_w(&sh.tail, ntail & 1);
                ++ntail;
                if (!there) {
                    drain_bar(&sh.tail, (ntail - 1) & 1);
                    if (leader) mbar_arrive(&sh.kv_full[st]);
                    return false;
                }
                for (int h = 0; h < C::HALVES; ++h) {
                    uint4 *rows = reinterpret_cast<uint4 *>(sh.kv[st] + h * (kTile * 128));
                    for (int i = z0 * 8 + lane; i < z1 * 8; i += 32) rows[i] = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async();
                __syncwarp();
                if (leader) mbar_arrive(&sh.kv_full[st]);
            }
            return true;
        };
        if (!ok) break;
        if (looks_ahead<D>(s.few)) {
            if (!(ok = put(&maps.k[c.set], 0, false))) break;
            for (int t = 0; t < c.nt && ok; ++t) {
                if (t + 1 < c.nt && !(ok = put(&maps.k[c.set], t + 1, false))) break;
                ok = put(&maps.v[c.set], t, true);
            }
        } else {
            for (int t = 0; t < c.nt && ok; ++t)
                ok = put(&maps.k[c.set], t, false) && put(&maps.v[c.set], t, true);
        }
    }
    if (!ok) {                              // let the copies in flight land before the CTA exits
        for (uint32_t i = pos > (uint32_t)C::STAGES ? pos - C::STAGES : 0; i < pos; ++i)
            drain_bar(&sh.kv_full[i % C::STAGES], (i / C::STAGES) & 1);
        for (int pl = 0; pl < 2; ++pl)
            if (nq[pl]) drain_bar(&sh.q_full[pl], (nq[pl] - 1) & 1);
    }
}

template <int D> __device__ __forceinline__ uint32_t col_s(int pl) { return 128u * pl; }
template <int D> __device__ __forceinline__ uint32_t col_p(int pl) { return D == 64 ? 256u + 64u * pl : 128u * pl; }
template <int D> __device__ __forceinline__ uint32_t col_o(int pl) { return D == 64 ? 384u + 64u * pl : 256u + 128u * pl; }

template <int D>
__device__ void mma_role(const FwdParams &p, Shared<D> &sh, uint32_t tmem, int pl, int lane) {
    using C = Cfg<D>;
    volatile int *abort_flag = &sh.abort_flag;
    const bool leader = lane == 0;
    const uint32_t tS = tmem + col_s<D>(pl), tP = tmem + col_p<D>(pl), tO = tmem + col_o<D>(pl);
    const uint64_t dq = desc_kmajor_sw128(sh.q[pl]);
    const uint64_t dk0 = desc_kmajor_sw128(sh.kv[0]), dv0 = desc_mnmajor_sw128(sh.kv[0], kTile * 128);
    uint32_t pos = 0, g = 0, nq = 0;       // ring position, this pipeline's steps and units
    bool ok = true;
    auto wait_w = [&](uint64_t *b, uint32_t par) -> bool {
        return __all_sync(0xffffffffu, wait_fast(b, par, abort_flag, p.status));
    };
    // a tile that only the other pipeline takes: released once it is there
    auto skip = [&](uint32_t at) -> bool {
        const int st = at % C::STAGES;
        if (!wait_w(&sh.kv_full[st], (at / C::STAGES) & 1)) return false;
        if (leader) mbar_arrive(&sh.kv_empty[st]);
        __syncwarp();
        return true;
    };
    auto issue_s = [&](uint32_t at, bool last) -> bool {
        const int st = at % C::STAGES;
        if (!wait_w(&sh.kv_full[st], (at / C::STAGES) & 1)) return false;
        fence_after();
        if (leader) {
            const uint64_t dk = dk0 + (uint64_t)st * (C::TILE >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = (kk / 4) * ((kTile * 128) >> 4) + 2 * (kk % 4);
                mma_bf16(tS, dq + off, dk + off, idesc_of(128, false), kk > 0);
            }
            commit(&sh.s_full[pl]);
            commit(&sh.kv_empty[st]);
            if (last) commit(&sh.q_empty[pl]);
        }
        __syncwarp();
        return true;
    };
    auto issue_pv = [&](uint32_t at, bool first) -> bool {
        const int st = at % C::STAGES;
        if (!wait_w(&sh.p_full[pl], g & 1) || !wait_w(&sh.kv_full[st], (at / C::STAGES) & 1)) return false;
        fence_after();
        if (leader) {
            const uint64_t dv = dv0 + (uint64_t)st * (C::TILE >> 4);
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
                mma_ts(tO, tP + 8u * kk, dv + 128 * kk, idesc_of(D, true), (first && kk == 0) ? 0u : 1u);
            commit(&sh.o_done[pl]);
            commit(&sh.kv_empty[st]);
        }
        __syncwarp();
        ++g;
        return true;
    };
    Chunk c;
    Walk w = walk_begin<D>(p, sh);
    while (ok && walk_next(p, w, c, nullptr)) {
        if (c.nt <= 0) continue;
        const FwdSet &s = p.plan.s[c.set];
        const bool active = s.few || 2 * c.pair + pl < s.tiles;
        if (active && !(ok = wait_w(&sh.q_full[pl], nq & 1))) break;
        if (active) ++nq;
        if (!active) {
            for (int i = 0; i < 2 * c.nt && ok; ++i) ok = skip(pos + i);
        } else if (s.few) {                 // alternate tiles; S of this pipeline's next tile after its P·V
            // a pipeline without a tile of its own (one step) leaves Q unused
            const int mine = (c.nt - pl + 1) / 2;
            if (mine == 0 && leader) mbar_arrive(&sh.q_empty[pl]);
            __syncwarp();
            for (int t = 0; t < c.nt && ok; ++t) {
                if ((t & 1) == pl)
                    ok = issue_s(pos + 2 * t, t + 2 >= c.nt) && issue_pv(pos + 2 * t + 1, t == pl);
                else
                    ok = skip(pos + 2 * t) && skip(pos + 2 * t + 1);
            }
        } else if (looks_ahead<D>(false)) {
            ok = issue_s(pos, c.nt == 1);
            for (int t = 0; t < c.nt && ok; ++t) {
                if (t + 1 < c.nt)
                    ok = wait_w(&sh.s_free[pl], g & 1) && issue_s(pos + 2 * t + 1, t + 2 == c.nt);
                ok = ok && issue_pv(pos + (t + 1 < c.nt ? 2 * t + 2 : 2 * t + 1), t == 0);
            }
        } else {
            for (int t = 0; t < c.nt && ok; ++t)
                ok = issue_s(pos + 2 * t, t + 1 == c.nt) && issue_pv(pos + 2 * t + 1, t == 0);
        }
        pos += 2 * c.nt;
    }
    // every MMA this warp issued must be complete before TMEM is freed
    if (leader) commit(&sh.drain[pl]);
    __syncwarp();
    drain_bar(&sh.drain[pl], 0);
}

__device__ __forceinline__ float max32(const float *s) {
    float a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = fmaxf(fmax3(s[4 * i], s[4 * i + 1], s[4 * i + 2]), s[4 * i + 3]);
    return fmax3(fmax3(a[0], a[1], a[2]), fmax3(a[3], a[4], a[5]), fmaxf(a[6], a[7]));
}

// 32 scores of a row to bf16 pairs of 2^(s·sl2 - m), and their sum onto acc.
__device__ __forceinline__ void numerators32(const float *s, float sl2, float neg_m, uint32_t *pk, float2 &acc) {
    const float2 sc2 = make_float2(sl2, sl2), nm2 = make_float2(neg_m, neg_m);
    float2 x[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) x[c] = __ffma2_rn(make_float2(s[2 * c], s[2 * c + 1]), sc2, nm2);
#pragma unroll
    for (int c = 0; c < 16; ++c) x[c] = make_float2(ex2(x[c].x), ex2(x[c].y));
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        pk[c] = pack_bf16x2(x[c].x, x[c].y);
        acc = __fadd2_rn(acc, x[c]);
    }
}

// 32 columns of a finished row: bf16 to out or fp32 to a workspace row (dst16 null), times f.
__device__ __forceinline__ void store32(__nv_bfloat16 *dst16, float *dst32, const float *x, float f) {
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

// Where row i (of the unit's 256) of a chunk goes: out and lse, a part, or a whole row of a set.
struct RowOut {
    __nv_bfloat16 *o16;
    float *o32, *lse;
    float lse_unit;         // lse is kept in log2 units in the workspace, given out in natural ones
    bool valid;
};
template <int D>
__device__ __forceinline__ RowOut row_out(const FwdParams &p, const Chunk &c, int64_t tile, int i_tile, int i_unit) {
    RowOut r;
    const int64_t row = plan_row(p.plan, p.plan.s[c.set], c.z, c.hk, tile, i_tile);
    r.valid = row >= 0;
    r.o16 = nullptr;
    r.o32 = r.lse = nullptr;
    r.lse_unit = 1.f;
    if (!r.valid) return r;
    if (c.slot >= 0) {
        const int64_t at = (2 * (int64_t)blockIdx.x + c.slot) * (2 * kTile) + i_unit;
        r.o32 = p.part_o + at * D;
        r.lse = p.part_lse + at;
    } else if (p.whole_o) {
        const int64_t at = c.set * p.all_rows + row;
        r.o32 = p.whole_o + at * D;
        r.lse = p.whole_lse + at;
    } else {
        r.o16 = p.out + row * D;
        r.lse = p.lse ? p.lse + row : nullptr;
        r.lse_unit = kLn2;
    }
    return r;
}

template <int D>
__device__ void softmax_role(const FwdParams &p, Shared<D> &sh, uint32_t tmem, int pl, int wq, int lane) {
    using C = Cfg<D>;
    const unsigned FULL = 0xffffffffu;
    volatile int *abort_flag = &sh.abort_flag;
    const uint32_t wl = (uint32_t)(32 * wq) << 16;
    const uint32_t tS = tmem + col_s<D>(pl) + wl, tP = tmem + col_p<D>(pl) + wl, tO = tmem + col_o<D>(pl) + wl;
    const float sl2 = p.scale_log2;
    uint32_t g = 0, nmerge = 0;
    bool ok = true;
    auto wait_all = [&](uint64_t *b, uint32_t par) -> bool {
        return __all_sync(FULL, wait_fast(b, par, abort_flag, p.status));
    };
    // running maximum m (lazy) and sum l of this thread's row; O is rescaled when m grows by 2^8
    auto new_max = [&](float mx, float &m, float &l, bool started) {
        const bool first = m == -CUDART_INF_F;
        const bool need = !first && mx > m + kRescaleLog2;
        if (__any_sync(FULL, need) && started) {
            const float alpha = need ? ex2(m - mx) : 1.f;
            fence_after();
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
                float o[32];
                tmem_ld32(tO + 32 * cc, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= alpha;
                tmem_st32(tO + 32 * cc, o);
            }
            tmem_wait_st();
            l *= alpha;
        }
        if (first || need) m = mx;
    };
    Chunk c;
    Walk w = walk_begin<D>(p, sh);
    while (ok && walk_next(p, w, c, nullptr)) {
        const FwdSet &s = p.plan.s[c.set];
        float m = -CUDART_INF_F, l = 0.f;
        if (!s.few) {
            const int64_t tile = 2 * c.pair + pl;
            if (tile >= s.tiles) continue;
            for (int t = 0; t < c.nt; ++t, ++g) {
                if (!(ok = wait_all(&sh.s_full[pl], g & 1))) break;
                fence_after();
                float x[128];
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) tmem_ld32(tS + 32 * cc, x + 32 * cc);
                tmem_wait_ld();
                if constexpr (D == 64) {
                    fence_before();
                    mbar_arrive(&sh.s_free[pl]);
                }
                const int valid = c.len - (c.t0 + t) * kTile;
                if (valid < kTile) {
#pragma unroll
                    for (int e = 0; e < 128; ++e) x[e] = e < valid ? x[e] : -CUDART_INF_F;
                }
                const float mx = sl2 * fmaxf(fmaxf(max32(x), max32(x + 32)), fmaxf(max32(x + 64), max32(x + 96)));
                // P·V of the step before has read P and written O
                if (t > 0 && !(ok = wait_all(&sh.o_done[pl], (g - 1) & 1))) break;
                new_max(mx, m, l, t > 0);
                const float neg_m = m == -CUDART_INF_F ? 0.f : -m;
                float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) {
                    uint32_t pk[16];
                    numerators32(x + 32 * cc, sl2, neg_m, pk, acc);
                    tmem_st16w(tP + 16 * cc, pk);
                }
                l += acc.x + acc.y;
                tmem_wait_st();
                fence_before();
                mbar_arrive(&sh.p_full[pl]);
            }
            if (!ok || (c.nt > 0 && !(ok = wait_all(&sh.o_done[pl], (g - 1) & 1)))) break;
            fence_after();
            const RowOut r = row_out<D>(p, c, tile, 32 * wq + lane, kTile * pl + 32 * wq + lane);
            const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
                float o[32];
                if (c.nt > 0) {
                    tmem_ld32(tO + 32 * cc, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
                if (l == 0.f) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
                if (r.valid) store32(r.o16 ? r.o16 + 32 * cc : nullptr, r.o32 + 32 * cc, o, inv);
            }
            if (r.valid && r.lse) *r.lse = l == 0.f ? -CUDART_INF_F : (m + __log2f(l)) * r.lse_unit;
            fence_before();
            continue;
        }
        // few rows: this warp's keys are 32·wq .. +31 of each of its pipeline's tiles
        const int nrows = (int)(s.members * p.plan.rows);
        bool any = false;
        for (int t = pl; t < c.nt; t += 2, ++g) {
            if (!(ok = wait_all(&sh.s_full[pl], g & 1))) break;
            fence_after();
            float x[32];
            tmem_ld32(tS + 32 * wq, x);
            tmem_wait_ld();
            if constexpr (D == 64) {
                fence_before();
                mbar_arrive(&sh.s_free[pl]);
            }
            const int valid = c.len - (c.t0 + t) * kTile - 32 * wq;
            if (valid < 32) {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = e < valid ? x[e] : -CUDART_INF_F;
            }
            const float mx = sl2 * max32(x);
            if (any && !(ok = wait_all(&sh.o_done[pl], (g - 1) & 1))) break;
            new_max(mx, m, l, any);
            any = true;
            float2 acc = make_float2(0.f, 0.f);
            uint32_t pk[16], zero[16];
            numerators32(x, sl2, m == -CUDART_INF_F ? 0.f : -m, pk, acc);
#pragma unroll
            for (int e = 0; e < 16; ++e) zero[e] = 0u;
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
                if (cc == wq) tmem_st16w(tP + 16 * cc, pk);
                else tmem_st16w(tP + 16 * cc, zero);
            }
            l += acc.x + acc.y;
            tmem_wait_st();
            fence_before();
            mbar_arrive(&sh.p_full[pl]);
        }
        if (!ok || (any && !(ok = wait_all(&sh.o_done[pl], (g - 1) & 1)))) break;
        fence_after();
        // merge the eight partial rows: weights 2^(m - M) / L, then sums through shared memory. A row
        // that is not one of the unit's (lane >= nrows) holds whatever it holds and is not stored.
        const int idx = 4 * pl + wq;
        sh.ml[0][idx][lane] = m;
        sh.ml[1][idx][lane] = l;
        mbar_arrive(&sh.merge_bar);
        if (!(ok = wait_all(&sh.merge_bar, nmerge++ & 1))) break;
        float M = -CUDART_INF_F, L = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) M = fmaxf(M, sh.ml[0][i][lane]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float li = sh.ml[1][i][lane];
            L += li == 0.f ? 0.f : li * ex2(sh.ml[0][i][lane] - M);
        }
        const float f = l == 0.f ? 0.f : ex2(m - M) / L;
        for (int r0 = 0; r0 < nrows; r0 += C::MROWS) {
            const bool mine = lane >= r0 && lane < r0 + C::MROWS;
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
                float o[32];
                if (any) {
                    tmem_ld32(tO + 32 * cc, o);
                    tmem_wait_ld();
                }
                if (mine) {
                    float4 *dst = reinterpret_cast<float4 *>(&sh.merge[idx][lane - r0][32 * cc]);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[e] = l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                          : make_float4(o[4 * e] * f, o[4 * e + 1] * f, o[4 * e + 2] * f, o[4 * e + 3] * f);
                }
                __syncwarp();
            }
            mbar_arrive(&sh.merge_bar);
            if (!(ok = wait_all(&sh.merge_bar, nmerge++ & 1))) break;
            {   // MROWS·D/4 groups of four columns (128 or 256): one a thread
                const int at = 128 * pl + 32 * wq + lane, i = at / (D / 4), col = 4 * (at % (D / 4));
                if (i < C::MROWS && r0 + i < nrows) {
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float4 z = *reinterpret_cast<const float4 *>(&sh.merge[k][i][col]);
                        y.x += z.x;
                        y.y += z.y;
                        y.z += z.z;
                        y.w += z.w;
                    }
                    const RowOut r = row_out<D>(p, c, 0, r0 + i, r0 + i);
                    if (r.valid) {
                        if (r.o16)
                            *reinterpret_cast<uint2 *>(r.o16 + col) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
                        else
                            *reinterpret_cast<float4 *>(r.o32 + col) = y;
                    }
                }
            }
            mbar_arrive(&sh.merge_bar);    // the buffer is free again
            if (!(ok = wait_all(&sh.merge_bar, nmerge++ & 1))) break;
        }
        if (!ok) break;
        if (idx == 0 && lane < nrows) {
            const RowOut r = row_out<D>(p, c, 0, lane, lane);
            if (r.valid && r.lse) *r.lse = L == 0.f ? -CUDART_INF_F : (M + __log2f(L)) * r.lse_unit;
        }
        fence_before();
    }
}

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1) dense_fwd_kernel(const __grid_constant__ Maps maps,
                                                                const __grid_constant__ FwdParams p) {
    extern __shared__ uint8_t smem_raw[];
    Shared<D> &sh = *reinterpret_cast<Shared<D> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        sh.abort_flag = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_empty[i], 1);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_free[i], 128);
            mbar_init(&sh.p_full[i], 128);
            mbar_init(&sh.o_done[i], 1);
            mbar_init(&sh.drain[i], 1);
        }
        for (int i = 0; i < Cfg<D>::STAGES; ++i) {
            mbar_init(&sh.kv_full[i], 1);
            mbar_init(&sh.kv_empty[i], 2);
        }
        mbar_init(&sh.tail, 1);
        mbar_init(&sh.merge_bar, 256);
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
        if (warp == 0) copy_role<D>(p, maps, sh, lane);
        else if (warp < 3) mma_role<D>(p, sh, tmem, warp - 1, lane);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        softmax_role<D>(p, sh, tmem, (warp - 4) >> 2, warp & 3, lane);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ---------------------------------------------------------------- join

// The parts of one unit's row, weighted by 2^(lse - max): o = Σ w_p o_p / Σ w_p. One warp a row;
// lane holds columns lane·D/32.. of the sum. Parts come in the order of their CTAs.
template <int D> struct Joined {
    float o[D / 32], m, l;
};
template <int D> __device__ __forceinline__ void join_add(Joined<D> &j, const float *o, float lse, int lane) {
    if (lse == -CUDART_INF_F) return;
    const float mn = fmaxf(j.m, lse);
    const float a = j.m == -CUDART_INF_F ? 0.f : exp2f(j.m - mn), b = exp2f(lse - mn);
    float x[D / 32];
    if constexpr (D == 64) {
        const float2 y = *reinterpret_cast<const float2 *>(o + 2 * lane);
        x[0] = y.x, x[1] = y.y;
    } else {
        const float4 y = *reinterpret_cast<const float4 *>(o + 4 * lane);
        x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
    }
#pragma unroll
    for (int e = 0; e < D / 32; ++e) j.o[e] = j.o[e] * a + x[e] * b;
    j.l = j.l * a + b;
    j.m = mn;
}
template <int D> __device__ __forceinline__ void join_store(const FwdParams &p, const Joined<D> &j, int64_t row, int lane) {
    const float inv = j.l == 0.f ? 0.f : 1.f / j.l;
    uint32_t u[D / 64];
#pragma unroll
    for (int e = 0; e < D / 64; ++e) u[e] = pack_bf16x2(j.o[2 * e] * inv, j.o[2 * e + 1] * inv);
    if constexpr (D == 64) reinterpret_cast<uint32_t *>(p.out + row * D)[lane] = u[0];
    else reinterpret_cast<uint2 *>(p.out + row * D)[lane] = make_uint2(u[0], u[1]);
    if (p.lse && lane == 0) p.lse[row] = j.l == 0.f ? -CUDART_INF_F : (j.m + __log2f(j.l)) * kLn2;
}
template <int D> __device__ __forceinline__ void join_begin(Joined<D> &j) {
    j.m = -CUDART_INF_F;
    j.l = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) j.o[e] = 0.f;
}
// All parts of row i (of the unit's 256), begun by CTA ca and ended by CTA cb. With fewer steps than
// CTAs some of those in between have none.
template <int D>
__device__ __forceinline__ void join_parts(const FwdParams &p, Joined<D> &j, int ca, int cb, int i, int64_t total,
                                           int lane) {
    for (int c = ca; c <= cb; ++c) {
        if (total < p.plan.ctas && cta_first(c, total, p.plan.ctas) == cta_first(c + 1, total, p.plan.ctas)) continue;
        const int64_t at = (2 * (int64_t)c + (c == ca)) * (2 * kTile) + i;
        join_add<D>(j, p.part_o + at * D, p.part_lse[at], lane);
    }
}

// One set: a block joins 8 rows of the unit in which CTA blockIdx.x + 1 begins, if it is the first
// CTA to begin inside that unit. The other units' rows were finished by the one CTA that had them.
template <int D> __global__ void __launch_bounds__(256) join_one_kernel(const __grid_constant__ FwdParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x + 1;
    const int64_t total = total_steps(p.plan, lane), x = cta_first(c, total, p.plan.ctas);
    if (x >= total) return;
    const StepAt at = step_at(p.plan, x, lane);
    if (at.t == 0) return;
    const int64_t a = x - at.t;
    if (cta_of(a, total, p.plan.ctas) != c - 1) return;
    const FwdSet &s = p.plan.s[0];
    const int i = 8 * blockIdx.y + warp;
    const int64_t hk = at.uu / s.pairs, pair = at.uu - hk * s.pairs;
    const int64_t row = s.few ? plan_row(p.plan, s, at.z, hk, 0, i)
                              : (2 * pair + i / kTile < s.tiles ? plan_row(p.plan, s, at.z, hk, 2 * pair + i / kTile, i % kTile) : -1);
    if (row < 0) return;
    Joined<D> j;
    join_begin<D>(j);
    join_parts<D>(p, j, c - 1, cta_of(a + at.steps - 1, total, p.plan.ctas), i, total, lane);
    join_store<D>(p, j, row, lane);
}

// Two sets: a warp joins one row's parts of both.
template <int D> __global__ void __launch_bounds__(256) join_two_kernel(const __grid_constant__ FwdParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 8 + warp;
    if (row >= p.all_rows) return;
    const int64_t slab = row / p.plan.rows, r = row - slab * p.plan.rows, b = slab / p.plan.kv_heads;
    const int64_t hk = slab - b * p.plan.kv_heads;
    const int64_t total = p.plan.stream ? total_steps(p.plan, lane) : 0;
    int64_t base = 0;
    Joined<D> j;
    join_begin<D>(j);
    for (int k = 0; k < 2; ++k) {
        const FwdSet &s = p.plan.s[k];
        const int64_t z = b / s.members, member = b - z * s.members;
        int64_t t, i;
        if (s.bb) {
            t = member / s.bb;
            i = (member - t * s.bb) * p.plan.rows + r;
        } else {
            t = member * s.tpm + r / kTile;
            i = r % kTile;
        }
        bool whole = true;
        if (p.plan.stream) {
            const int steps = set_steps(s, z);
            const int64_t a = base + steps_before(s, z, lane) + (hk * s.pairs + t / 2) * steps;
            const int ca = cta_of(a, total, p.plan.ctas), cb = cta_of(a + steps - 1, total, p.plan.ctas);
            whole = ca == cb;
            if (!whole) join_parts<D>(p, j, ca, cb, (int)(s.few ? i : i + kTile * (t & 1)), total, lane);
            base += steps_before(s, s.sets, lane);
        }
        if (whole) {
            const int64_t at = k * p.all_rows + row;
            join_add<D>(j, p.whole_o + at * D, p.whole_lse[at], lane);
        }
    }
    join_store<D>(p, j, row, lane);
}

// ---------------------------------------------------------------- host

template <int D>
cudaError_t launch(const DenseProblem &pb, const void *q, const KeySet *sets, FwdParams &p, cudaStream_t stream) {
    Maps maps;
    for (int k = 0; k < 2; ++k) {
        const KeySet &ks = sets[k < p.plan.nsets ? k : 0];
        const FwdSet &s = p.plan.s[k < p.plan.nsets ? k : 0];
        const cuuint64_t qd[4] = {(cuuint64_t)D, (cuuint64_t)pb.rows, (cuuint64_t)pb.kv_heads, (cuuint64_t)pb.batch};
        const cuuint64_t qs[3] = {(cuuint64_t)D * 2, (cuuint64_t)pb.rows * D * 2, (cuuint64_t)pb.kv_heads * pb.rows * D * 2};
        const cuuint32_t qb[4] = {64, s.bb ? (cuuint32_t)pb.rows : (cuuint32_t)kTile, 1, s.bb ? (cuuint32_t)s.bb : 1u};
        const cuuint64_t kd[3] = {(cuuint64_t)D, (cuuint64_t)ks.n, (cuuint64_t)(ks.sets * pb.kv_heads)};
        const cuuint64_t kst[2] = {(cuuint64_t)D * 2, (cuuint64_t)ks.n * D * 2};
        const cuuint32_t kb[3] = {64, kTile, 1};
        if (!make_map(&maps.q[k], q, 4, qd, qs, qb) || !make_map(&maps.k[k], ks.k, 3, kd, kst, kb) ||
            !make_map(&maps.v[k], ks.v, 3, kd, kst, kb))
            return cudaErrorInvalidValue;
    }
    auto kern = dense_fwd_kernel<D>;
    const size_t smem = sizeof(Shared<D>) + 1024;
    static_assert(sizeof(Shared<D>) + 1024 <= 232448, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    // setmaxnreg.inc would wait forever for registers that the CTA was not launched with
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    if (fa.numRegs * NTHREADS < kRegsNeeded || fa.maxThreadsPerBlock < NTHREADS) return cudaErrorInvalidConfiguration;
    kern<<<p.plan.ctas, NTHREADS, smem, stream>>>(maps, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (p.plan.nsets == 2)
        join_two_kernel<D><<<(unsigned)((p.all_rows + 7) / 8), 256, 0, stream>>>(p);
    else if (p.plan.stream && p.plan.ctas > 1)
        join_one_kernel<D><<<dim3(p.plan.ctas - 1, p.plan.s[0].few ? kFewRows / 8 : 2 * kTile / 8), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

FwdPlan make_fwd_plan(const DenseProblem &p, const KeySet *sets, int nsets) {
    FwdPlan r{};
    r.nsets = nsets;
    r.rows = p.rows;
    r.kv_heads = p.kv_heads;
    r.batch = p.batch;
    int64_t units = 0, steps = 0, most = 0;
    bool scan = true;
    for (int k = 0; k < nsets; ++k) {
        const KeySet &ks = sets[k];
        FwdSet &s = r.s[k];
        s.len = ks.len;
        s.n = ks.n;
        s.sets = ks.sets;
        s.members = ks.members;
        s.few = p.rows <= kFewRows && ks.members * p.rows <= kFewRows;
        if (p.rows <= kTile) {
            const int64_t fit = kTile / p.rows;
            s.bb = (int32_t)(ks.members < fit ? ks.members : fit);
            s.tpm = 0;
            s.tiles = (ks.members + s.bb - 1) / s.bb;
        } else {
            s.bb = 0;
            s.tpm = (int32_t)((p.rows + kTile - 1) / kTile);
            s.tiles = ks.members * s.tpm;
        }
        s.pairs = (s.tiles + 1) / 2;
        s.upz = p.kv_heads * s.pairs;
        const int64_t t = (ks.n + kTile - 1) / kTile;
        units += s.sets * s.upz;
        steps += s.sets * s.upz * t;
        most = t > most ? t : most;
        scan = scan && (!ks.len || ks.sets <= 1024);
    }
    // Units of a few steps each, or very many of them, go whole to the CTAs: cutting would save less
    // than the join costs.
    r.stream = scan && most > 4 && units < 16 * kCtas;
    const int64_t want = r.stream ? (steps + 1) / 2 : units;
    r.ctas = (int32_t)(want < kCtas ? want : kCtas);
    return r;
}

FwdLayout fwd_layout_of(const FwdPlan &plan, int64_t d) {
    FwdLayout L{};
    size_t o = 0;
    auto take = [&](size_t floats) { const size_t at = o; o += (floats + 63) / 64 * 64; return at; };
    const size_t all = (size_t)plan.batch * plan.kv_heads * plan.rows;
    if (plan.stream && plan.ctas > 1) {
        L.part_o = take((size_t)plan.ctas * 4 * kTile * d);
        L.part_lse = take((size_t)plan.ctas * 4 * kTile);
    }
    if (plan.nsets == 2) {
        L.whole_o = take(2 * all * d);
        L.whole_lse = take(2 * all);
    }
    L.total = o;
    return L;
}

cudaError_t launch_dense_fwd(const DenseProblem &pb, const void *q, const KeySet *sets, int nsets, void *out, float *lse,
                             float *ws, uint32_t *status, cudaStream_t stream) {
    FwdParams p{};
    p.plan = make_fwd_plan(pb, sets, nsets);
    const FwdLayout L = fwd_layout_of(p.plan, pb.d);
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    p.part_o = ws + L.part_o;
    p.part_lse = ws + L.part_lse;
    p.whole_o = nsets == 2 ? ws + L.whole_o : nullptr;
    p.whole_lse = nsets == 2 ? ws + L.whole_lse : nullptr;
    p.all_rows = pb.batch * pb.kv_heads * pb.rows;
    p.scale_log2 = pb.scale * 1.4426950408889634f;
    p.status = status;
    return pb.d == 64 ? launch<64>(pb, q, sets, p, stream) : launch<128>(pb, q, sets, p, stream);
}

}  // namespace bsa
