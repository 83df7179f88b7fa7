// Dense softmax attention of query rows to states of another length on the
// sm_100a tensor cores (bf16, head_dim D = 64 or 128, fp32 accumulation).
//
// Row i of a batch entry and key head (the query rows of all heads that share
// the key head, which lie one behind the other) against keys j < len:
//   s_ij = q_i·k_j (·s log2 e),  m_i = max_j s_ij (lazily: it may lag by up to 2^8),
//   p_ij = 2^(s_ij - m_i),  l_i = Σ_j p_ij,  o_i = Σ_j p_ij v_j / l_i.
// A step is one tile of 128 keys: S = Q·Kᵀ (tcgen05.mma, M = N = 128) into tensor
// memory, softmax numerators by the threads of its rows, P as bf16 pairs back into
// tensor memory, O += P·V with P as the A operand from there.
//
// Organisation: one persistent CTA per SM, two pipelines:
//   warp 0       copies (TMA, 128-byte swizzle): Q of a unit, then K and V tiles
//                through one ring that both pipelines read
//   warps 1, 2   the MMA warp of pipeline 0 and of pipeline 1
//   warp 3       finds the CTA's units and hands them out
//   warps 4..    softmax and epilogue of pipeline 0, then of pipeline 1: four warps
//                each, or eight (many rows, D = 64)
// Many rows: the pipelines hold two tiles of 128 rows of one unit and both take
// every key tile, so K and V are read once for 256 rows.
//   D = 64 (640 threads, two for a row, each with half of a tile's keys): a step is a key tile. S of the next
//   one is formed as soon as this one's is read, and P has columns of its own; a thread keeps P in
//   registers until the P·V before it has read those (waiting for that ahead of the exponentials put
//   P·V's whole chain, from the arrival of P to its completion about 1,000 clocks, into every step:
//   2.09 us for 256 rows and 128 keys, where the exponentials alone need 1.08).
//   D = 128 (384 threads, one for a row): tensor memory has no columns left for that. A step is half a key
//   tile, S has two buffers, P(u) takes the place of S(u): the MMA warp issues S(0) S(1) PV(0)
//   S(2) PV(1) ..., so that the products of one step run beside the softmax of the other.
// Few rows (at most 32: a decoding step's query heads, or an ensemble's members
// together): both pipelines hold the same rows, four times over in the four 32-lane
// quarters of tensor memory, and take alternate key tiles; warp w of a pipeline does
// the softmax of its tile's keys 32w..32w+31 only (P is zero elsewhere in its lanes).
// So the exponentials of a tile are spread over four warps although there are few
// rows, and the eight partial rows are merged by their maxima and sums at the end.
//
// Tensor memory (512 columns): D = 64: S0 S1 (128 each), P0 P1 (64 each), O0 O1 (64 each). D = 128: S0
// S1, O0 O1 (128 each), many rows: S in two buffers of 64, P in the first 32 columns of its buffer; few
// rows: P in the first 64 columns of its S, and S of the next tile follows P·V.
//
// Keys behind a length: scores are replaced before the maximum (whatever K holds),
// and the copy warp zeroes those rows of V in shared memory, since 0·NaN is NaN.
//
// Roundings: the weights are bf16 as an operand (V's type; their sums are taken before that, in fp32), out
// is bf16: each half a step, together 2.3e-3 of out's norm from 64 bits, where rounding out alone gives
// 1.7e-3. out_low carries what rounding out leaves off to the backward's row sums.
//
// What it takes (here and below: GPU time of calls on the same inputs in a graph; "a call": of the Python layer, on
// three sets of inputs in turn) and what bounds it:
//   12288 rows a head, 8 heads, on 29040 keys, D = 64: 920 to 955 us, 0.77 to 0.79 PFLOP/s (a call 1,005); 12288
//   on 12288: 400 to 450. The exponential unit alone needs 634 us of the first (16 a clock and SM) and is 64 %
//   busy, the tensor pipe 37 %, instructions issue in 65 % of all cycles: a step of 256 rows and 128 keys takes
//   1.55 us, the rest being issue and the chain S, maximum, exponentials, P, P·V of each pipeline where the
//   other does not cover it.
//   D = 128, 4 heads, 12288 on 12288: 281 us, 1.10 PFLOP/s; 8 heads on 29040 keys 1,365 us, 1.07. Tensor pipe and
//   exponential unit are both 53 % busy: the chain again, with half-tile steps in the tensor memory there is.
//   Few rows: 24 entries of one row, 16 heads on 4 key heads, D = 128, 29040 keys: 212 us for 1.43 GB of keys and
//   values, 6.75 TB/s, of which L2 holds some from call to call; a call 244 us, 5.85 TB/s.
//
// Every wait on an mbarrier is bounded (2 s), as in the block-sparse kernel.
#include <math_constants.h>

#include <type_traits>

#include "cross.cuh"
#include "cross_tc.cuh"

namespace bsa {
namespace {

using namespace tc;

// Threads of a row: two where tensor memory has room for P beside S (half of a tile's keys each).
template <int D, bool FEW> struct Threads {
    static constexpr int SPLIT = !FEW && D == 64 ? 2 : 1;
    static constexpr int SOFT_WARPS = 4 * SPLIT;       // a pipeline
    static constexpr int ALL = 128 + 64 * SOFT_WARPS;
    // register split: the control warpgroup drops to CTRL registers a thread, the softmax warps rise to SOFT
    static constexpr int CTRL = SPLIT == 2 ? 56 : 72, SOFT = SPLIT == 2 ? 104 : 216;
    static constexpr int REGS = 128 * CTRL + 64 * SOFT_WARPS * SOFT;
    static constexpr int READERS = 3 + 2 * SOFT_WARPS; // warps that read a chunk: copy, 2 MMA, softmax
    static_assert(REGS <= 65536 / ALL / 8 * 8 * ALL, "register split");
};
constexpr int kSub = 64;                    // keys of a step when there are many rows
// Of 16 pairs of exponentials, how many take the polynomial on the FMA pipe. D = 64 is bound by the
// exponentials and what goes out beside them (12288 x 29040, 8 heads: none 980 us, 1 of 16 974, 2 of 16
// 922, 4 of 16 940), D = 128 by the chain of its products (a step of 256 rows and 128 keys: none 2.33 us,
// 4 of 16 2.44).
template <int D> constexpr int kPoly = D == 64 ? 2 : 0;
constexpr float kRescaleLog2 = 8.0f;
constexpr float kLn2 = 0.69314718055994531f;

template <int D> struct Cfg {
    static constexpr int HALVES = D / 64;              // 128-byte column groups of a row
    static constexpr int TILE = kTile * D * 2;         // bytes of a 128-row tile
    static constexpr int STAGES = D == 64 ? 9 : 4;     // ring of K and V tiles
    static constexpr int MROWS = D == 64 ? 16 : 4;     // rows merged at a time (few rows)
    static constexpr int MSTRIDE = D + 4;              // floats, padded against bank conflicts
};

// What a CTA does next: key tiles [t0, t0 + nt) of a unit; nt 0: a set without keys, -1: nothing more.
// Warp 3 finds the chunks and hands them to the other warps through shared memory.
struct Chunk {
    int nt, t0, rel;        // rel: the set's keys from key tile t0 on
    int slot;               // -1: the whole unit
    int alone;              // many rows: the second pipeline has no tile
    int rows[2];            // tiles of one member's rows: how many, from row row0 on
    int64_t row0[2];
    int64_t z, hk, pair;
};
struct Walk {
    int t, steps;
    int64_t z, uu, left;    // stream: steps left; whole: the unit's index
    int64_t at, total;      // stream: the next step, all steps
};
constexpr int kChunks = 4;

template <int D> struct alignas(1024) Shared {
    uint8_t q[2][Cfg<D>::TILE];
    uint8_t kv[Cfg<D>::STAGES][Cfg<D>::TILE];
    float merge[8][Cfg<D>::MROWS][Cfg<D>::MSTRIDE];
    float ml[2][8][32];                                // few rows: (m, l) of each partial row
    float ls[2][2][2][kTile];                          // two threads a row: [chunk % 2][pipeline][half] sums
    uint64_t q_full[2], q_empty[2], kv_full[Cfg<D>::STAGES], kv_empty[Cfg<D>::STAGES], tail;
    uint64_t s_full[2][2], p_full[2][2], o_done[2][2];  // [pipeline][step % 2]
    uint64_t s_free[2], l_bar[2], merge_bar, drain[2];
    uint64_t ch_full[kChunks], ch_empty[kChunks];
    Chunk ch[kChunks];
    uint32_t tmem_base;
    int abort_flag;
};

struct FwdParams {
    FwdPlan plan;
    __nv_bfloat16 *out, *low;   // [rows of all][D]; low: what rounding out leaves off, nullable
    float *lse;             // nullable
    const __nv_bfloat16 *v; // few rows: for infinite values
    float *part_o, *part_lse, *whole_o, *whole_lse;     // whole: null for a single set
    Cut *cuts;              // [ctas]: single set
    int2 *spans;            // [units]: two sets: first and last CTA of a unit
    int64_t all_rows;       // batch * kv_heads * rows
    int cta0;               // first block of this pass in its launch
    float scale_log2;
    uint32_t *status;       // nullable
    int64_t withhold;       // test hook
};

__device__ __forceinline__ int this_cta(const FwdParams &p) { return (int)blockIdx.x - p.cta0; }

struct Maps {
    CUtensorMap q, k, v;
};

// Warp-wide (the scan of the sets' lengths).
__device__ __forceinline__ Walk walk_begin(const FwdParams &p, int lane) {
    Walk w{};
    if (p.plan.stream) {
        if (lane == 0 && p.cuts) p.cuts[this_cta(p)].last = -1;   // until one is noted
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
// The next chunk; a unit that begins here is noted for the join (by lane 0).
__device__ __forceinline__ bool walk_next(const FwdParams &p, Walk &w, Chunk &c, bool lead) {
    const FwdSet &s = p.plan.s;
    int steps;
    if (p.plan.stream) {
        if (w.left <= 0) return false;
        if (w.t == w.steps) {                          // the next unit
            w.t = 0;
            if (++w.uu == s.upz) {
                w.uu = 0;
                ++w.z;
                w.steps = set_steps(s, w.z);
            }
        }
        c.z = w.z;
        c.hk = quotient(w.uu, s.pairs);
        c.pair = w.uu - c.hk * s.pairs;
        c.t0 = w.t;
        steps = (int)min((int64_t)(w.steps - w.t), w.left);
        c.slot = steps == w.steps ? -1 : (w.t > 0 ? 0 : 1);
        if (lead && w.t == 0) {
            const int last = c.slot < 0 ? this_cta(p) : cta_of(w.at + w.steps - 1, w.total, p.plan.ctas);
            if (p.spans) p.spans[w.z * s.upz + w.uu] = make_int2(this_cta(p), last);
            else if (c.slot == 1) p.cuts[this_cta(p)] = Cut{(int)c.z, (int)c.hk, (int)c.pair, last};
        }
        w.t += steps;
        w.at += steps;
        w.left -= steps;
    } else {
        int64_t u = w.left;
        if (u >= s.sets * s.upz) return false;
        if (lead && p.spans) p.spans[u] = make_int2(0, 0);
        c.z = quotient(u, s.upz);
        u -= c.z * s.upz;
        c.hk = quotient(u, s.pairs);
        c.pair = u - c.hk * s.pairs;
        c.t0 = 0;
        c.slot = -1;
        steps = 0x7fffffff;
        w.left += p.plan.ctas;
    }
    const int len = set_len(s.len, c.z, s.n, lead ? p.status : nullptr), tiles = (len + kTile - 1) / kTile;
    c.nt = min(steps, tiles - c.t0);                   // 0 for a set without keys
    c.rel = len - c.t0 * kTile;
    c.alone = 2 * c.pair + 1 >= s.tiles;
    if (!s.bb) {
#pragma unroll
        for (int pl = 0; pl < 2; ++pl) {
            const int64_t t = 2 * c.pair + pl, member = quotient(t, s.tpm), r = (t - member * s.tpm) * kTile;
            c.rows[pl] = t < s.tiles ? (int)min((int64_t)kTile, p.plan.rows - r) : 0;
            c.row0[pl] = ((c.z * s.members + member) * p.plan.kv_heads + c.hk) * p.plan.rows + r;
        }
    }
    return true;
}

// Warp 3: the CTA's chunks, a few ahead of the warps that work on them.
template <int D> __device__ void chunk_role(const FwdParams &p, Shared<D> &sh, int lane) {
    Walk w = walk_begin(p, lane);
    for (uint32_t i = 0;; ++i) {
        const int at = i % kChunks;
        if (!__all_sync(0xffffffffu, wait_soon(&sh.ch_empty[at], ((i / kChunks) & 1) ^ 1, &sh.abort_flag, p.status))) return;
        Chunk c{};
        const bool more = walk_next(p, w, c, lane == 0);
        if (!more) c.nt = -1;
        if (lane == 0) {
            sh.ch[at] = c;
            mbar_arrive(&sh.ch_full[at]);
        }
        __syncwarp();
        if (!more) return;
    }
}
// The i-th chunk, or null at the end (and after a wait that expired: `ok` false).
template <int D>
__device__ __forceinline__ const Chunk *chunk_at(const FwdParams &p, Shared<D> &sh, uint32_t i, bool &ok) {
    const int at = i % kChunks;
    ok = __all_sync(0xffffffffu, wait_soon(&sh.ch_full[at], (i / kChunks) & 1, &sh.abort_flag, p.status));
    return ok && sh.ch[at].nt >= 0 ? &sh.ch[at] : nullptr;
}
template <int D> __device__ __forceinline__ void chunk_done(Shared<D> &sh, uint32_t i, int lane) {
    warp_arrive(&sh.ch_empty[i % kChunks], lane);
}

template <int D, bool FEW>
__device__ void copy_role(const FwdParams &p, const Maps &maps, Shared<D> &sh, int lane) {
    using C = Cfg<D>;
    volatile int *abort_flag = &sh.abort_flag;
    const bool leader = elect_one();    // issues; the whole warp runs the loop
    auto wait_w = [&](uint64_t *b, uint32_t par) -> bool {
        return __all_sync(0xffffffffu, wait_soon(b, par, abort_flag, p.status));
    };
    uint32_t pos = 0, nq[2] = {0, 0}, ntail = 0;
    bool ok = true;
    const Chunk *cp;
    for (uint32_t i = 0; ok && (cp = chunk_at<D>(p, sh, i, ok)); ++i) {
        const Chunk c = *cp;
        chunk_done<D>(sh, i, lane);
        if (c.nt == 0) continue;
        const FwdSet &s = p.plan.s;
        for (int pl = 0; pl < 2 && ok; ++pl) {
            const int64_t t = FEW ? 0 : 2 * c.pair + pl;
            if (t >= s.tiles) continue;
            if (!(ok = wait_w(&sh.q_empty[pl], (nq[pl] & 1) ^ 1))) break;
            if (leader) {
                const int64_t member = c.z * s.members + (s.bb ? t * s.bb : t / s.tpm);
                const int row = s.bb ? 0 : (int)(t % s.tpm) * kTile;
                const int box = (s.bb ? s.bb * (int)p.plan.rows : kTile) * 128;   // bytes of a copied box
                const int reps = FEW ? 4 : 1;
                mbar_expect_tx(&sh.q_full[pl], (uint32_t)(box * reps * C::HALVES));
                for (int h = 0; h < C::HALVES; ++h)
                    for (int r = 0; r < reps; ++r)
                        tma_load_4d(sh.q[pl] + h * (kTile * 128) + r * (32 * 128), &maps.q, &sh.q_full[pl],
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
            const int z0 = c.rel - t * kTile, z1 = (int)min((int64_t)kTile, s.n - row);
            const bool zero = is_v && z0 < z1;
            uint64_t *bar = zero ? &sh.tail : &sh.kv_full[st];
            if (leader && !((int64_t)pos == p.withhold && this_cta(p) == 0)) {
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
        for (int t = 0; t < c.nt && ok; ++t) ok = put(&maps.k, t, false) && put(&maps.v, t, true);
    }
    if (!ok) {                              // let the copies in flight land before the CTA exits
        for (uint32_t i = pos > (uint32_t)C::STAGES ? pos - C::STAGES : 0; i < pos; ++i)
            drain_bar(&sh.kv_full[i % C::STAGES], (i / C::STAGES) & 1);
        for (int pl = 0; pl < 2; ++pl)
            if (nq[pl]) drain_bar(&sh.q_full[pl], (nq[pl] - 1) & 1);
    }
}

__device__ __forceinline__ uint32_t col_s(int pl) { return 128u * pl; }
template <int D> __device__ __forceinline__ uint32_t col_o(int pl) { return D == 64 ? 384u + 64u * pl : 256u + 128u * pl; }
template <int D> __device__ __forceinline__ uint32_t col_p(int pl) { return D == 64 ? 256u + 64u * pl : 128u * pl; }
// Steps of a whole key tile (else of half a tile, with two buffers of S).
template <int D, bool FEW> constexpr bool kWhole = FEW || D == 64;

// Steps of 64 keys of a chunk.
__device__ __forceinline__ int sub_steps(int nt, int rel) { return (min(rel, nt * kTile) + kSub - 1) / kSub; }

template <int D, bool FEW>
__device__ void mma_role(const FwdParams &p, Shared<D> &sh, uint32_t tmem, int pl, int lane) {
    using C = Cfg<D>;
    constexpr bool WHOLE = kWhole<D, FEW>;
    constexpr int KEYS = WHOLE ? kTile : kSub;         // keys of a step
    volatile int *abort_flag = &sh.abort_flag;
    const bool leader = elect_one();    // issues; the whole warp runs the loop
    const uint32_t tS = tmem + col_s(pl), tP = tmem + col_p<D>(pl), tO = tmem + col_o<D>(pl);
    const uint64_t dq = desc_kmajor_sw128(sh.q[pl]);
    const uint64_t dk0 = desc_kmajor_sw128(sh.kv[0]), dv0 = desc_mnmajor_sw128(sh.kv[0], kTile * 128);
    uint32_t pos = 0, g = 0, nq = 0;       // ring position, this pipeline's steps and units
    bool ok = true;
    auto wait_w = [&](uint64_t *b, uint32_t par) -> bool {
        return __all_sync(0xffffffffu, wait_soon(b, par, abort_flag, p.status));
    };
    auto there = [&](uint32_t at) -> bool { return wait_w(&sh.kv_full[at % C::STAGES], (at / C::STAGES) & 1); };
    // A tile that only the other pipeline uses. Its arrival is waited for and its stages are given back all the
    // same: a pipeline that let a stage's turn pass could take the one before for the one it waits for (a
    // barrier tells two turns apart, not three), and did where a tile came in late.
    auto skip = [&](int t) -> bool {
        for (uint32_t at = pos + 2 * t; at < pos + 2 * t + 2; ++at) {
            if (!there(at)) return false;
            if (leader) mbar_arrive(&sh.kv_empty[at % C::STAGES]);
            __syncwarp();
        }
        return true;
    };
    // S(gs) = Q·Kᵀ of KEYS keys from key `from` of the tile at ring position `at`, which is there
    auto issue_s = [&](uint32_t gs, uint32_t at, int from, bool done, bool last) {
        const int st = at % C::STAGES, b = gs & 1;
        fence_after();
        if (leader) {
            const uint64_t dk = dk0 + (uint64_t)(st * (C::TILE >> 4) + from * 8);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = (kk / 4) * ((kTile * 128) >> 4) + 2 * (kk % 4);
                mma_bf16(tS + (WHOLE ? 0u : 64u * b), dq + off, dk + off, idesc_of(KEYS, false), kk > 0);
            }
            commit(&sh.s_full[pl][b]);
            if (done) commit(&sh.kv_empty[st]);
            if (last) commit(&sh.q_empty[pl]);
        }
        __syncwarp();
    };
    // O += P·V of step g once P is written; the tile at `at` is there
    auto issue_pv = [&](uint32_t at, int from, bool done, bool first) -> bool {
        const int st = at % C::STAGES, b = g & 1;
        if (!wait_w(&sh.p_full[pl][b], (g >> 1) & 1)) return false;
        fence_after();
        if (leader) {
            const uint64_t dv = dv0 + (uint64_t)(st * (C::TILE >> 4) + from * 8);
#pragma unroll
            for (int kk = 0; kk < KEYS / 16; ++kk)
                mma_ts(tO, tP + (WHOLE ? 0u : 64u * b) + 8u * kk, dv + 128 * kk, idesc_of(D, true), (first && kk == 0) ? 0u : 1u);
            commit(&sh.o_done[pl][b]);
            if (done) commit(&sh.kv_empty[st]);
        }
        __syncwarp();
        ++g;
        return true;
    };
    const Chunk *cp;
    for (uint32_t i = 0; ok && (cp = chunk_at<D>(p, sh, i, ok)); ++i) {
        // uniform over the warp, for the compiler too: the MMAs' descriptors then need no vector registers
        const int nt = uniform(cp->nt), rel = uniform(cp->rel);
        const bool idle = !FEW && pl == 1 && uniform(cp->alone);   // no tile of rows here
        chunk_done<D>(sh, i, lane);
        if (idle) {
            for (int t = 0; t < nt && ok; ++t) ok = skip(t);
        } else if (nt > 0) {
            if (!(ok = wait_w(&sh.q_full[pl], nq & 1))) break;
            ++nq;
            if constexpr (WHOLE) {
                constexpr int by = FEW ? 2 : 1;        // few rows: every other tile
                const int first = FEW ? pl : 0;
                if (FEW && first > 0 && !(ok = skip(0))) break;
                if (first >= nt) {                     // one tile: this pipeline's Q stays unused
                    if (leader) mbar_arrive(&sh.q_empty[pl]);
                    __syncwarp();
                } else {
                    if (!(ok = there(pos + 2 * first))) break;
                    issue_s(g, pos + 2 * first, 0, true, first + by >= nt);
                    for (int t = first; t < nt && ok; t += by) {
                        const bool more = t + by < nt;
                        const uint32_t kn = pos + 2 * (t + by), v = pos + 2 * t + 1;
                        if (FEW && D == 64 && t + 1 < nt && !(ok = skip(t + 1))) break;
                        if constexpr (D == 64) {       // P has columns of its own: S as soon as the last one is read
                            if (more) {
                                if (!(ok = there(kn) && wait_w(&sh.s_free[pl], g & 1))) break;
                                issue_s(g + 1, kn, 0, true, t + 2 * by >= nt);
                            }
                            ok = there(v) && issue_pv(v, 0, true, t == first);
                        } else {
                            ok = there(v) && issue_pv(v, 0, true, t == first) && (t + 1 >= nt || skip(t + 1)) && (!more || there(kn));
                            if (ok && more) issue_s(g, kn, 0, true, t + 2 * by >= nt);
                        }
                    }
                }
            } else {
                const int n = sub_steps(nt, rel);
                if (!(ok = there(pos))) break;
                const uint32_t g0 = g;
                auto s_step = [&](int u) {
                    issue_s(g0 + u, pos + 2 * (u >> 1), kSub * (u & 1), (u & 1) || u + 1 == n, u + 1 == n);
                };
                s_step(0);
                if (n > 1) s_step(1);
                for (int u = 0; u < n && ok; ++u) {
                    const uint32_t v = pos + 2 * (u >> 1) + 1;
                    ok = ((u & 1) || there(v)) && (u + 2 >= n || (u & 1) || there(pos + u + 2)) &&
                         issue_pv(v, kSub * (u & 1), (u & 1) || u + 1 == n, u == 0);
                    if (ok && u + 2 < n) s_step(u + 2);
                }
            }
        }
        pos += 2 * nt;
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

__device__ __forceinline__ float sum4(const float2 *a) {
    const float2 t = __fadd2_rn(__fadd2_rn(a[0], a[1]), __fadd2_rn(a[2], a[3]));
    return t.x + t.y;
}
// PAIRS pairs of a row's scores to bf16 pairs of 2^(s·sl2 - m), and their sums onto acc (four chains).
// In rotation: exponentials of pair c, the exponent of pair c + AHEAD, packing and sum of pair
// c - AHEAD, so that the other work goes out between the exponentials, of which the exp unit takes
// one instruction in eight clocks (issued in a row they fill its queue, and a warp that waits there
// issues nothing else). POLY of 16 pairs take the polynomial on the FMA pipe instead.
template <int POLY, int PAIRS>
__device__ __forceinline__ void numerators(const float *s, float sl2, float neg_m, uint32_t *pk, float2 *acc) {
    constexpr int AHEAD = 4;
    const float2 sc2 = make_float2(sl2, sl2), nm2 = make_float2(neg_m, neg_m);
    float2 x[2 * AHEAD + 1];
    auto at = [](int c) { return c % (2 * AHEAD + 1); };
#pragma unroll
    for (int c = 0; c < AHEAD && c < PAIRS; ++c) x[at(c)] = __ffma2_rn(make_float2(s[2 * c], s[2 * c + 1]), sc2, nm2);
#pragma unroll
    for (int c = 0; c < PAIRS + AHEAD; ++c) {
        if (c < PAIRS) {
            float2 &y = x[at(c)];
            if (c * POLY % 16 < POLY) {
                y = exp2_fma2(y);
            } else {
                asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(y.x));
                asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(y.y));
            }
        }
        if (c >= AHEAD) {
            const float2 y = x[at(c - AHEAD)];
            asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pk[c - AHEAD]) : "f"(y.y), "f"(y.x));
            acc[c & 3] = __fadd2_rn(acc[c & 3], y);
        }
        if (c + AHEAD < PAIRS) x[at(c + AHEAD)] = __ffma2_rn(make_float2(s[2 * (c + AHEAD)], s[2 * (c + AHEAD) + 1]), sc2, nm2);
    }
}

// Where row i of tile pl of a chunk's unit goes: out and lse, a part, or a whole row of a set.
struct RowOut {
    __nv_bfloat16 *o16, *low;
    float *o32, *lse;
    float lse_unit;         // lse is kept in log2 units in the workspace, given out in natural ones
    bool valid, bf16;       // bf16: o16, for all rows of the chunk
};
template <int D>
__device__ __forceinline__ RowOut row_out(const FwdParams &p, const Chunk &c, int pl, int i) {
    RowOut r;
    const int64_t row = p.plan.s.bb ? plan_row(p.plan, c.z, c.hk, 2 * c.pair + pl, i) : i < c.rows[pl] ? c.row0[pl] + i : -1;
    r.valid = row >= 0;
    r.o16 = r.low = nullptr;
    r.o32 = r.lse = nullptr;
    r.lse_unit = 1.f;
    r.bf16 = c.slot < 0 && !p.whole_o;
    if (!r.valid) return r;
    if (c.slot >= 0) {
        const int64_t at = (2 * (int64_t)this_cta(p) + c.slot) * (2 * kTile) + kTile * pl + i;
        r.o32 = p.part_o + at * D;
        r.lse = p.part_lse + at;
    } else if (p.whole_o) {
        const int64_t at = row;
        r.o32 = p.whole_o + at * D;
        r.lse = p.whole_lse + at;
    } else {
        r.o16 = p.out + row * D;
        r.low = p.low ? p.low + row * D : nullptr;
        r.lse = p.lse ? p.lse + row : nullptr;
        r.lse_unit = kLn2;
    }
    return r;
}

// A warp's rows j0..j1-1 (lane j knows row j's places) of a set without keys: zeros and lse = -inf (of a set among two
// lse alone is read). Many such units may follow one another on a CTA, each counted as one step: with
// the stores of other units they held up a forward (4 x 4004 rows of an empty entry among three) to 70 us, so 49.
template <int D> __device__ __forceinline__ void zero_rows(const RowOut &r, int j0, int j1, int lane) {
    constexpr int LANES = D / 8;                       // of a row
    auto fill = [&](__nv_bfloat16 *mine) {
#pragma unroll 2
        for (int j = j0; j < j1; j += 32 / LANES) {
            char *to = reinterpret_cast<char *>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), j + lane / LANES));
            if (to) *reinterpret_cast<uint4 *>(to + 16 * (lane % LANES)) = make_uint4(0u, 0u, 0u, 0u);
        }
    };
    fill(r.o16);
    fill(r.low);
    if (j0 == 0 && r.valid && r.lse) *r.lse = -CUDART_INF_F;
}
// The end of a unit of many rows: a warp's 32 rows, columns [c0, c0 + COLS) of o at taddr, and lse (with c0 = 0).
template <int D, int COLS>
__device__ __forceinline__ void end_rows(const FwdParams &p, const Chunk &c, int pl, int wq, int c0, uint32_t taddr, float m, float l,
                                      uint8_t *stage, int lane) {
    const RowOut r = row_out<D>(p, c, pl, 32 * wq + lane);
    if (c.nt <= 0) {                                   // a set without keys: half of the rows each
        zero_rows<D>(r, 32 * c0 / D, 32 * (c0 + COLS) / D, lane);
        return;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    write_rows(stage, taddr, COLS, inv, l == 0.f, r.bf16, r.bf16 ? static_cast<void *>(r.o16 + c0) : r.o32 + c0,
               r.low ? r.low + c0 : nullptr, r.valid, lane);
    if (c0 == 0 && r.valid && r.lse) *r.lse = l == 0.f ? -CUDART_INF_F : (m + __log2f(l)) * r.lse_unit;
}

// Few rows: four columns of a row's o that came out NaN although its weights did not. Every lane quarter's product
// takes all keys of a tile, with a weight of 0 for those of the other quarters, and 0 times an infinite value is
// NaN. A weight itself is above 0 however far its score lies below the others, so what such a column should
// hold is the sum of its infinite (and NaN) values, from another look at all of them. y stays where there is
// none. (v: the four columns of the chunk's first key. Only calls with infinite values come here. Eight loads are in
// flight: 32 rows, D = 128, on 40 million keys, 270,000 a CTA, take 149 ms instead of 2.9, within the 2 s that
// the other warps wait.)
template <int D> __device__ __noinline__ float4 infinite_values(const __nv_bfloat16 *v, int keys, float4 y) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [](float &to, uint32_t bits) {          // bits: a bf16 value in the upper half
        if ((bits & 0x7f800000u) == 0x7f800000u) to += __uint_as_float(bits);
    };
#pragma unroll 8
    for (int j = 0; j < keys; ++j) {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(v + (int64_t)j * D));
        add(a.x, u.x << 16), add(a.y, u.x & 0xffff0000u), add(a.z, u.y << 16), add(a.w, u.y & 0xffff0000u);
    }
    auto pick = [](float y, float a) { return y != y && a != 0.f ? a : y; };
    return make_float4(pick(y.x, a.x), pick(y.y, a.y), pick(y.z, a.z), pick(y.w, a.w));
}

template <int D, bool FEW>
__device__ void softmax_role(const FwdParams &p, Shared<D> &sh, uint32_t tmem, int pl, int hh, int wq, int lane) {
    using C = Cfg<D>;
    constexpr int SPLIT = Threads<D, FEW>::SPLIT;      // threads of a row; hh: which of them this is
    constexpr int WIDE = kTile / SPLIT, COLS = D / SPLIT;   // this thread's keys of a tile, columns of O
    const unsigned FULL = 0xffffffffu;
    volatile int *abort_flag = &sh.abort_flag;
    const uint32_t wl = (uint32_t)(32 * wq) << 16;
    const uint32_t tS = tmem + col_s(pl) + wl, tO = tmem + col_o<D>(pl) + wl, tP = tmem + col_p<D>(pl) + wl;
    const float sl2 = p.scale_log2;
    uint32_t g = 0, nmerge = 0, nl = 0;
    bool ok = true;
    auto wait_all = [&](uint64_t *b, uint32_t par) -> bool {
        return __all_sync(FULL, wait_soon(b, par, abort_flag, p.status));
    };
    // the P·V of the step before this one is complete
    auto wait_o = [&]() -> bool { return wait_all(&sh.o_done[pl][(g - 1) & 1], ((g - 1) >> 1) & 1); };
    // running maximum m (lazy) and sum l of this thread's row; when m grows by 2^8, O is rescaled, once
    // the P·V of the step before (`started`) is complete
    auto new_max = [&](float mx, float &m, float &l, bool started) -> bool {
        const bool first = m == -CUDART_INF_F;
        const bool need = !first && mx > m + kRescaleLog2;
        if (__any_sync(FULL, need) && started) {
            if (!wait_o()) return false;
            const float alpha = need ? ex2(m - mx) : 1.f;
            fence_after();
#pragma unroll 1
            for (int cc = COLS * hh; cc < COLS * (hh + 1); cc += 16) {
                uint32_t o[16];
                tmem_ld16_now(tO + cc, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st16w(tO + cc, o);
            }
            tmem_wait_st();
            l *= alpha;
        }
        if (first || need) m = mx;
        return true;
    };
    const Chunk *cp;
    for (uint32_t i = 0; ok && (cp = chunk_at<D>(p, sh, i, ok)); ++i) {
        const int nt = uniform(cp->nt), rel = uniform(cp->rel);
        float m = -CUDART_INF_F, l = 0.f;
        if constexpr (!FEW) {
            if (pl == 1 && cp->alone) {
                chunk_done<D>(sh, i, lane);
                continue;
            }
            const int n = nt <= 0 ? 0 : (D == 64 ? nt : sub_steps(nt, rel));
            if constexpr (D == 64) {
                // one wait a step: for the next S, which its thread issued behind the P·V that has to be done with
                // P's columns before this step's P goes there
                ok = n == 0 || wait_all(&sh.s_full[pl][g & 1], (g >> 1) & 1);
                for (int t = 0; t < n && ok; ++t, ++g) {
                    fence_after();
                    // both threads of a row need the maximum of the whole row: reading the other half costs
                    // less than an exchange. Keys behind the length count as -inf.
                    float x[WIDE], mx = -CUDART_INF_F;
                    const int valid = rel - t * kTile;
#pragma unroll
                    for (int h = SPLIT - 1; h >= 0; --h) {
                        const int half = hh ^ h;       // its own half last
#pragma unroll
                        for (int cc = 0; cc < WIDE; cc += 32) tmem_ld32(tS + WIDE * half + cc, x + cc);
                        tmem_wait_ld_of(x);
                        if (valid < kTile) {
#pragma unroll
                            for (int e = 0; e < WIDE; ++e) x[e] = WIDE * half + e < valid ? x[e] : -CUDART_INF_F;
                        }
#pragma unroll
                        for (int cc = 0; cc < WIDE; cc += 32) mx = fmaxf(mx, max32(x + cc));
                    }
                    fence_before();
                    warp_arrive(&sh.s_free[pl], lane);
                    if (!(ok = new_max(sl2 * mx, m, l, t > 0))) break;
                    const float neg_m = m == -CUDART_INF_F ? 0.f : -m;
                    float2 acc[4] = {};
                    uint32_t pk[WIDE / 2];
                    numerators<kPoly<D>, WIDE / 2>(x, sl2, neg_m, pk, acc);
                    l += sum4(acc);
                    if (t + 1 < n) ok = wait_all(&sh.s_full[pl][(g + 1) & 1], ((g + 1) >> 1) & 1);
                    else if (t > 0) ok = wait_o();
                    if (!ok) break;
                    fence_after();
#pragma unroll
                    for (int cc = 0; cc < WIDE / 2; cc += 32)
                        tmem_st32(tP + WIDE / 2 * hh + cc, reinterpret_cast<const float *>(pk + cc));
                    tmem_wait_st();
                    fence_before();
                    warp_arrive(&sh.p_full[pl][g & 1], lane);
                }
            } else {
                for (int u = 0; u < n; ++u, ++g) {
                    const uint32_t tSu = tS + 64u * (g & 1);
                    if (!(ok = wait_all(&sh.s_full[pl][g & 1], (g >> 1) & 1))) break;
                    fence_after();
                    float x[kSub];
                    tmem_ld32(tSu, x);
                    tmem_ld32(tSu + 32, x + 32);
                    tmem_wait_ld_of(x);
                    const int valid = rel - u * kSub;      // keys behind the length count as -inf
                    if (valid < kSub) {
#pragma unroll
                        for (int e = 0; e < kSub; ++e) x[e] = e < valid ? x[e] : -CUDART_INF_F;
                    }
                    if (!(ok = new_max(sl2 * fmaxf(max32(x), max32(x + 32)), m, l, u > 0))) break;
                    const float neg_m = m == -CUDART_INF_F ? 0.f : -m;
                    float2 acc[4] = {};
                    uint32_t pk[kSub / 2];
                    numerators<kPoly<D>, kSub / 2>(x, sl2, neg_m, pk, acc);
                    tmem_st32(tSu, reinterpret_cast<const float *>(pk));
                    l += sum4(acc);
                    tmem_wait_st();
                    fence_before();
                    warp_arrive(&sh.p_full[pl][g & 1], lane);
                }
            }
            if (!ok || (n > 0 && !(ok = wait_o()))) break;
            fence_after();
            if constexpr (SPLIT == 2) {                    // the row's sum is both threads'
                float *ls = &sh.ls[nl & 1][pl][0][32 * wq + lane];
                ls[kTile * hh] = l;
                warp_arrive(&sh.l_bar[pl], lane);
                if (!(ok = wait_all(&sh.l_bar[pl], nl & 1))) break;
                ++nl;
                l = ls[0] + ls[kTile];
            }
            uint8_t *stage = reinterpret_cast<uint8_t *>(sh.merge) + 2048 * (4 * (SPLIT * pl + hh) + wq);
            end_rows<D, COLS>(p, *cp, pl, wq, COLS * hh, tO + COLS * hh, m, l, stage, lane);
            fence_before();
            chunk_done<D>(sh, i, lane);
        } else {
        // few rows: this warp's keys are 32·wq .. +31 of each of its pipeline's tiles
        const int nrows = (int)(p.plan.s.members * p.plan.rows);
        bool any = false;
        for (int t = pl; t < nt; t += 2, ++g) {
            if (!(ok = wait_all(&sh.s_full[pl][g & 1], (g >> 1) & 1))) break;
            fence_after();
            float x[32];
            tmem_ld32(tS + 32 * wq, x);
            tmem_wait_ld_of(x);
            fence_before();
            warp_arrive(&sh.s_free[pl], lane);
            const int valid = rel - t * kTile - 32 * wq;
            if (valid < 32) {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = e < valid ? x[e] : -CUDART_INF_F;
            }
            const float mx = sl2 * max32(x);
            if (!(ok = new_max(mx, m, l, any))) break;
            float2 acc[4] = {};
            uint32_t pk[16], zero[16];
            numerators<0, 16>(x, sl2, m == -CUDART_INF_F ? 0.f : -m, pk, acc);
            if (D == 64 && any && !(ok = wait_o())) break;   // P is read
            any = true;
            fence_after();
#pragma unroll
            for (int e = 0; e < 16; ++e) zero[e] = 0u;
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
                if (cc == wq) tmem_st16w(tP + 16 * cc, pk);
                else tmem_st16w(tP + 16 * cc, zero);
            }
            l += sum4(acc);
            tmem_wait_st();
            fence_before();
            warp_arrive(&sh.p_full[pl][g & 1], lane);
        }
        if (!ok || (any && !(ok = wait_o()))) break;
        fence_after();
        // merge the eight partial rows: weights 2^(m - M) / L, then sums through shared memory. A row
        // that is not one of the unit's (lane >= nrows) holds whatever it holds and is not stored.
        const int idx = 4 * pl + wq;
        sh.ml[0][idx][lane] = m;
        sh.ml[1][idx][lane] = l;
        warp_arrive(&sh.merge_bar, lane);
        if (!(ok = wait_all(&sh.merge_bar, nmerge++ & 1))) break;
        float M = -CUDART_INF_F, L = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) M = fmaxf(M, sh.ml[0][k][lane]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float lk = sh.ml[1][k][lane];
            L += lk == 0.f ? 0.f : lk * ex2(sh.ml[0][k][lane] - M);
        }
        const float f = l == 0.f ? 0.f : ex2(m - M) / L;
        for (int r0 = 0; r0 < nrows; r0 += C::MROWS) {
            const bool mine = lane >= r0 && lane < r0 + C::MROWS;
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
                float o[32];
                if (any) {
                    tmem_ld32(tO + 32 * cc, o);
                    tmem_wait_ld_of(o);
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
            warp_arrive(&sh.merge_bar, lane);
            if (!(ok = wait_all(&sh.merge_bar, nmerge++ & 1))) break;
            {   // MROWS·D/4 groups of four columns (128 or 256): one a thread
                const int at = 128 * pl + 32 * wq + lane, mr = at / (D / 4), col = 4 * (at % (D / 4));
                const float row_l = __shfl_sync(FULL, L, (r0 + mr) & 31);
                if (mr < C::MROWS && r0 + mr < nrows) {
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float4 z = *reinterpret_cast<const float4 *>(&sh.merge[k][mr][col]);
                        y.x += z.x;
                        y.y += z.y;
                        y.z += z.z;
                        y.w += z.w;
                    }
                    const RowOut r = row_out<D>(p, *cp, 0, r0 + mr);
                    if (r.valid) {
                        if (row_l == row_l && (y.x != y.x || y.y != y.y || y.z != y.z || y.w != y.w)) {
                            const int64_t key = (cp->z * p.plan.kv_heads + cp->hk) * p.plan.s.n + (int64_t)cp->t0 * kTile;
                            y = infinite_values<D>(p.v + key * D + col, min(rel, nt * kTile), y);
                        }
                        if (r.o16) {
                            const uint2 u = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
                            *reinterpret_cast<uint2 *>(r.o16 + col) = u;
                            if (r.low)
                                *reinterpret_cast<uint2 *>(r.low + col) =
                                    make_uint2(rest_bf16x2(y.x, y.y, u.x), rest_bf16x2(y.z, y.w, u.y));
                        } else {
                            *reinterpret_cast<float4 *>(r.o32 + col) = y;
                        }
                    }
                }
            }
            if (r0 + C::MROWS >= nrows) break;   // (the next chunk's first barrier comes before its first write)
            warp_arrive(&sh.merge_bar, lane);    // the buffer is free again
            if (!(ok = wait_all(&sh.merge_bar, nmerge++ & 1))) break;
        }
        if (!ok) break;
        if (idx == 0 && lane < nrows) {
            const RowOut r = row_out<D>(p, *cp, 0, lane);
            if (r.valid && r.lse) *r.lse = L == 0.f ? -CUDART_INF_F : (M + __log2f(L)) * r.lse_unit;
        }
        fence_before();
        chunk_done<D>(sh, i, lane);
        }
    }
}

// One CTA of a pass. L: the threads and registers of the launch (a few-rows pass may share one of more
// threads; the warps beyond its own idle).
template <int D, bool FEW, typename L> __device__ __forceinline__ void fwd_cta(const Maps &maps, const FwdParams &p) {
    using T = Threads<D, FEW>;
    extern __shared__ uint8_t smem_raw[];
    Shared<D> &sh = *reinterpret_cast<Shared<D> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        sh.abort_flag = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_empty[i], 1);
            mbar_init(&sh.s_free[i], T::SOFT_WARPS);
            mbar_init(&sh.l_bar[i], T::SOFT_WARPS);
            for (int b = 0; b < 2; ++b) {
                mbar_init(&sh.s_full[i][b], 1);
                mbar_init(&sh.p_full[i][b], T::SOFT_WARPS);
                mbar_init(&sh.o_done[i][b], 1);
            }
            mbar_init(&sh.drain[i], 1);
        }
        for (int i = 0; i < Cfg<D>::STAGES; ++i) {
            mbar_init(&sh.kv_full[i], 1);
            mbar_init(&sh.kv_empty[i], 2);
        }
        for (int i = 0; i < kChunks; ++i) {
            mbar_init(&sh.ch_full[i], 1);
            mbar_init(&sh.ch_empty[i], T::READERS);
        }
        mbar_init(&sh.tail, 1);
        mbar_init(&sh.merge_bar, 8);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane == 0) {
        prefetch_map(&maps.q);
        prefetch_map(&maps.k);
        prefetch_map(&maps.v);
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
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::CTRL));
        if (warp == 0) copy_role<D, FEW>(p, maps, sh, lane);
        else if (warp < 3) mma_role<D, FEW>(p, sh, tmem, warp - 1, lane);
        else chunk_role<D>(p, sh, lane);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::SOFT));
        if (warp < 4 + 2 * T::SOFT_WARPS) softmax_role<D, FEW>(p, sh, tmem, (warp - 4) / T::SOFT_WARPS, (warp >> 2) % T::SPLIT, warp & 3, lane);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <int D, bool FEW>
__global__ void __launch_bounds__((Threads<D, FEW>::ALL), 1) dense_fwd_kernel(const __grid_constant__ Maps maps,
                                                                const __grid_constant__ FwdParams p) {
    fwd_cta<D, FEW, Threads<D, FEW>>(maps, p);
}
// Two sets in one launch, the first set's CTAs first: the second's begin on each SM as the first's end there
// (four members of 3 rows on 777 shared and 77 own keys: 15 us, in two launches 23).
template <int D, bool FEW0, bool FEW1>
__global__ void __launch_bounds__((Threads<D, FEW0>::ALL), 1)
dense_fwd_pair_kernel(const __grid_constant__ Maps maps0, const __grid_constant__ FwdParams p0, const __grid_constant__ Maps maps1,
                      const __grid_constant__ FwdParams p1) {
    using L = Threads<D, FEW0>;
    static_assert(L::ALL >= Threads<D, FEW1>::ALL, "threads of the launch");
    if ((int)blockIdx.x < p1.cta0) fwd_cta<D, FEW0, L>(maps0, p0);
    else fwd_cta<D, FEW1, L>(maps1, p1);
}

// ---------------------------------------------------------------- join

// Rows of several parts, one after the other: o = Σ w_p o_p / Σ w_p with w_p = 2^(lse_p - max). A warp
// has a row, lane l its columns l·D/32..; a part's lse is read by one lane, 32 parts at a time, so
// that all weights are known before the parts' rows, whose loads then do not wait for one another.
template <int D> struct Joined {
    float o[D / 32], m, l;
};
template <int D> __device__ __forceinline__ void join_begin(Joined<D> &j) {
    j.m = -CUDART_INF_F;
    j.l = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) j.o[e] = 0.f;
}
// `count` parts; part k's row is number row_of(k) of o and lse.
template <int D, typename F>
__device__ __forceinline__ void join_add(Joined<D> &j, const float *o, const float *lse, int count, F row_of, int lane) {
    for (int k0 = 0; k0 < count; k0 += 32) {
        const int k = k0 + lane, n = min(32, count - k0);
        const float mine = k < count ? __ldg(lse + row_of(k)) : -CUDART_INF_F;
        float mx = mine;
        for (int i = 16; i; i >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
        const float mn = fmaxf(j.m, mx);
        if (mn == -CUDART_INF_F) {                     // no keys in any part so far, or NaN, which a maximum passes over
            if (__any_sync(0xffffffffu, mine != mine)) j.l = CUDART_NAN_F;
            continue;
        }
        const float a = ex2(j.m - mn), wt = ex2(mine - mn);
        float sum = wt;
        for (int i = 16; i; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
        j.l = j.l * a + sum;
        j.m = mn;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) j.o[e] *= a;
        for (int i0 = 0; i0 < n; i0 += 8) {            // eight rows' loads together
            using V = typename std::conditional<D == 64, float2, float4>::type;
            V y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i0 + i < n) y[i] = __ldg(reinterpret_cast<const V *>(o + row_of(k0 + i0 + i) * D) + lane);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float w = i0 + i < n ? __shfl_sync(0xffffffffu, wt, i0 + i) : 0.f;
                if (w == 0.f) continue;                // its row may never have been written
                j.o[0] = fmaf(y[i].x, w, j.o[0]), j.o[1] = fmaf(y[i].y, w, j.o[1]);
                if constexpr (D == 128) j.o[2] = fmaf(y[i].z, w, j.o[2]), j.o[3] = fmaf(y[i].w, w, j.o[3]);
            }
        }
    }
}
template <int D>
__device__ __forceinline__ void join_store(const Joined<D> &j, const FwdParams &p, int64_t row, int lane) {
    using V = typename std::conditional<D == 64, uint32_t, uint2>::type;
    const float inv = j.l == 0.f ? 0.f : 1.f / j.l;
    uint32_t u[D / 64], low[D / 64];
#pragma unroll
    for (int e = 0; e < D / 64; ++e) {
        const float a = j.o[2 * e] * inv, b = j.o[2 * e + 1] * inv;
        u[e] = pack_bf16x2(a, b);
        low[e] = rest_bf16x2(a, b, u[e]);
    }
    auto put = [&](__nv_bfloat16 *to, const uint32_t *w) {
        if constexpr (D == 64) reinterpret_cast<V *>(to + row * D)[lane] = w[0];
        else reinterpret_cast<V *>(to + row * D)[lane] = make_uint2(w[0], w[1]);
    };
    put(p.out, u);
    if (p.low) put(p.low, low);
    if (p.lse && lane == 0) p.lse[row] = j.l == 0.f ? -CUDART_INF_F : (j.m + __log2f(j.l)) * kLn2;
}
// Row i (of a unit's 256) of the parts that CTA ca begins: number of the k-th part's row.
struct PartRow {
    int ca, i;
    __device__ int64_t operator()(int k) const { return (2 * ((int64_t)ca + k) + (k == 0)) * (2 * kTile) + i; }
};

// A single set: block (c, y) joins rows of the unit that CTA c begins and leaves, if there is one; the
// other units' rows were finished by the one CTA that had them. Units of many rows are cut into two
// or three parts as a rule: then a warp has four rows, and all their parts' loads go out together.
constexpr int kJoinRows = 4, kJoinParts = 4;
template <int D> __global__ void __launch_bounds__(256) join_cut_kernel(const __grid_constant__ FwdParams p, int each) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ca = blockIdx.x;
    const Cut cut = p.cuts[ca];
    if (cut.last < ca || cut.last >= p.plan.ctas) return;
    const int count = cut.last - ca + 1, i0 = (8 * blockIdx.y + warp) * each;
    auto row_at = [&](int i) -> int64_t {
        const int64_t t = 2 * (int64_t)cut.tile + i / kTile;
        return t < p.plan.s.tiles ? plan_row(p.plan, cut.z, cut.hk, t, i % kTile) : -1;
    };
    const int64_t mine = lane < each ? row_at(i0 + lane) : -1;     // the warp's rows, one a lane
    if (each == kJoinRows && count <= kJoinParts) {
        using V = typename std::conditional<D == 64, float2, float4>::type;
        V y[kJoinRows][kJoinParts];
        float ls[kJoinRows][kJoinParts];
#pragma unroll
        for (int r = 0; r < kJoinRows; ++r) {
            const bool there = __shfl_sync(0xffffffffu, mine, r) >= 0;
#pragma unroll
            for (int k = 0; k < kJoinParts; ++k) {
                ls[r][k] = -CUDART_INF_F;
                if (there && k < count) {
                    const int64_t at = PartRow{ca, i0 + r}(k);
                    ls[r][k] = __ldg(p.part_lse + at);
                    y[r][k] = __ldg(reinterpret_cast<const V *>(p.part_o + at * D) + lane);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < kJoinRows; ++r) {
            const int64_t row = __shfl_sync(0xffffffffu, mine, r);
            if (row < 0) continue;
            Joined<D> j;
            join_begin<D>(j);
            j.m = fmaxf(fmaxf(ls[r][0], ls[r][1]), fmaxf(ls[r][2], ls[r][3]));
#pragma unroll
            for (int k = 0; k < kJoinParts; ++k) {
                if (ls[r][k] == -CUDART_INF_F) continue;
                const float w = ex2(ls[r][k] - j.m);
                j.l += w;
                j.o[0] = fmaf(y[r][k].x, w, j.o[0]), j.o[1] = fmaf(y[r][k].y, w, j.o[1]);
                if constexpr (D == 128) j.o[2] = fmaf(y[r][k].z, w, j.o[2]), j.o[3] = fmaf(y[r][k].w, w, j.o[3]);
            }
            join_store<D>(j, p, row, lane);
        }
        return;
    }
    for (int i = i0; i < i0 + each; ++i) {
        const int64_t row = __shfl_sync(0xffffffffu, mine, i - i0);
        if (row < 0) continue;
        Joined<D> j;
        join_begin<D>(j);
        join_add<D>(j, p.part_o, p.part_lse, count, PartRow{ca, i}, lane);
        join_store<D>(j, p, row, lane);
    }
}

// Two sets: a warp joins its ROWS rows' parts of both. Where no unit is cut into more than four, all their loads
// go out together; else one row follows the other. So a warp has one row while one wave of blocks holds them
// (384 rows of 37 + 1 parts, D = 128: 7.1 us, two rows a warp 10.9), two where there are more (49152
// rows, D = 64: 19.0 us, one row a warp 24.1). Four blocks an SM need 64 registers a thread, which
// two rows of D = 128 do not fit.
template <int D, int ROWS>
__global__ void __launch_bounds__(256, D == 64 || ROWS == 1 ? 4 : 2) join_sets_kernel(const __grid_constant__ FwdParams p0, const __grid_constant__ FwdParams p1) {
    using V = typename std::conditional<D == 64, float2, float4>::type;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row0 = ((int64_t)blockIdx.x * 8 + warp) * ROWS;
    // lane 2r + k: where row r's parts of set k are: parts from CTA ca on at row i of a unit, or one whole row
    int count = 0, ca = 0, at = 0;
    if (lane < 2 * ROWS && row0 + (lane >> 1) < p0.all_rows) {
        const FwdParams &p = lane & 1 ? p1 : p0;
        const FwdSet &s = p.plan.s;
        const int64_t row = row0 + (lane >> 1);
        // 32-bit divisions where they do: rows of a slab, members and tiles of a set are far below 2^31
        const uint32_t rows = (uint32_t)p.plan.rows, heads = (uint32_t)p.plan.kv_heads;
        const uint32_t slab = (uint32_t)quotient(row, rows), r = (uint32_t)(row - (int64_t)slab * rows);
        const uint32_t b = slab / heads, hk = slab - b * heads;
        const uint32_t z = b / (uint32_t)s.members, member = b - z * (uint32_t)s.members;
        uint32_t t, i;
        if (s.bb) {
            t = member / (uint32_t)s.bb;
            i = (member - t * s.bb) * rows + r;
        } else {
            t = member * s.tpm + r / kTile;
            i = r % kTile;
        }
        const int2 span = p.spans[z * s.upz + hk * s.pairs + t / 2];
        // (after an expired wait a span may be missing; what it holds then must not lead out of the parts, of
        // which a set whose units are whole has none)
        if (span.x >= 0 && span.y >= span.x && span.y < p.plan.ctas && (p.plan.stream || span.y == span.x)) {
            count = span.y - span.x + 1;
            ca = span.x;
            at = (int)(i + kTile * (t & 1));
        }
    }
    const int most = __reduce_max_sync(0xffffffffu, count);
    if (most <= kJoinParts) {
        V y[ROWS][2][kJoinParts];
        float ls[ROWS][2][kJoinParts];
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const FwdParams &p = k ? p1 : p0;
                const int n = __shfl_sync(0xffffffffu, count, 2 * r + k), c = __shfl_sync(0xffffffffu, ca, 2 * r + k);
                const PartRow part{c, __shfl_sync(0xffffffffu, at, 2 * r + k)};
#pragma unroll
                for (int j = 0; j < kJoinParts; ++j) {
                    ls[r][k][j] = -CUDART_INF_F;
                    if (j < n) {
                        const int64_t from = n == 1 ? row0 + r : part(j);
                        ls[r][k][j] = __ldg((n == 1 ? p.whole_lse : p.part_lse) + from);
                        y[r][k][j] = __ldg(reinterpret_cast<const V *>((n == 1 ? p.whole_o : p.part_o) + from * D) + lane);
                    }
                }
            }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (row0 + r >= p0.all_rows) continue;
            Joined<D> j;
            join_begin<D>(j);
#pragma unroll
            for (int k = 0; k < 2 * kJoinParts; ++k) j.m = fmaxf(j.m, ls[r][k / kJoinParts][k % kJoinParts]);
#pragma unroll
            for (int k = 0; k < 2 * kJoinParts; ++k) {
                const float l = ls[r][k / kJoinParts][k % kJoinParts];
                if (l == -CUDART_INF_F) continue;
                const V v = y[r][k / kJoinParts][k % kJoinParts];
                const float w = ex2(l - j.m);
                j.l += w;
                j.o[0] = fmaf(v.x, w, j.o[0]), j.o[1] = fmaf(v.y, w, j.o[1]);
                if constexpr (D == 128) j.o[2] = fmaf(v.z, w, j.o[2]), j.o[3] = fmaf(v.w, w, j.o[3]);
            }
            join_store<D>(j, p0, row0 + r, lane);
        }
        return;
    }
    for (int r = 0; r < ROWS; ++r) {
        const int64_t row = row0 + r;
        if (row >= p0.all_rows) return;
        Joined<D> j;
        join_begin<D>(j);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const FwdParams &p = k ? p1 : p0;
            const int n = __shfl_sync(0xffffffffu, count, 2 * r + k), c = __shfl_sync(0xffffffffu, ca, 2 * r + k);
            const int i = __shfl_sync(0xffffffffu, at, 2 * r + k);
            if (n == 1) join_add<D>(j, p.whole_o, p.whole_lse, 1, [row](int) { return row; }, lane);
            else join_add<D>(j, p.part_o, p.part_lse, n, PartRow{c, i}, lane);
        }
        join_store<D>(j, p0, row, lane);
    }
}

// ---------------------------------------------------------------- host

bool make_maps(Maps &maps, const DenseProblem &pb, const void *q, const KeySet &ks, const FwdSet &s) {
    const cuuint64_t d = pb.d, rows = pb.rows, heads = pb.kv_heads, n = ks.n;
    const cuuint64_t qd[4] = {d, rows, heads, (cuuint64_t)pb.batch}, qs[3] = {d * 2, rows * d * 2, heads * rows * d * 2};
    const cuuint32_t qb[4] = {64, s.bb ? (cuuint32_t)rows : (cuuint32_t)kTile, 1, s.bb ? (cuuint32_t)s.bb : 1u};
    const cuuint64_t kd[3] = {d, n, (cuuint64_t)ks.sets * heads}, kst[2] = {d * 2, n * d * 2};
    const cuuint32_t kb[3] = {64, kTile, 1};
    return make_map(&maps.q, q, 4, qd, qs, qb) && make_map(&maps.k, ks.k, 3, kd, kst, kb) &&
           make_map(&maps.v, ks.v, 3, kd, kst, kb);
}
template <int D> constexpr size_t kSmem = sizeof(Shared<D>) + 1024;
static_assert(kSmem<64> <= 232448 && kSmem<128> <= 232448, "shared memory");
static_assert(sizeof(Shared<64>::merge) >= 2048 * 2 * Threads<64, false>::SOFT_WARPS &&
                  sizeof(Shared<128>::merge) >= 2048 * 2 * Threads<128, false>::SOFT_WARPS, "staging of the epilogue");

template <int D, bool FEW> cudaError_t launch_one(const Maps &maps, const FwdParams &p, cudaStream_t stream) {
    using T = Threads<D, FEW>;
    const cudaError_t e = kernel_ready<dense_fwd_kernel<D, FEW>>(kSmem<D>, T::ALL, T::REGS);
    if (e != cudaSuccess) return e;
    dense_fwd_kernel<D, FEW><<<p.plan.ctas, T::ALL, kSmem<D>, stream>>>(maps, p);
    return cudaGetLastError();
}
template <int D, bool FEW0, bool FEW1>
cudaError_t launch_pair(const Maps *maps, FwdParams *p, cudaStream_t stream) {
    using T = Threads<D, FEW0>;
    const cudaError_t e = kernel_ready<dense_fwd_pair_kernel<D, FEW0, FEW1>>(kSmem<D>, T::ALL, T::REGS);
    if (e != cudaSuccess) return e;
    p[1].cta0 = p[0].plan.ctas;
    dense_fwd_pair_kernel<D, FEW0, FEW1><<<p[0].plan.ctas + p[1].plan.ctas, T::ALL, kSmem<D>, stream>>>(maps[0], p[0], maps[1], p[1]);
    return cudaGetLastError();
}
template <int D> cudaError_t run(const DenseProblem &pb, const void *q, const KeySet *sets, int nsets, FwdParams *p, cudaStream_t stream) {
    Maps maps[2];
    for (int k = 0; k < nsets; ++k)
        if (!make_maps(maps[k], pb, q, sets[k], p[k].plan.s)) return cudaErrorInvalidValue;
    cudaError_t e;
    if (nsets == 1) {
        e = p[0].plan.s.few ? launch_one<D, true>(maps[0], p[0], stream) : launch_one<D, false>(maps[0], p[0], stream);
        if (e != cudaSuccess || !p[0].cuts) return e;
        const int each = p[0].plan.s.few ? 1 : kJoinRows, rows = p[0].plan.s.few ? kFewRows : 2 * kTile;
        join_cut_kernel<D><<<dim3(p[0].plan.ctas, rows / (8 * each)), 256, 0, stream>>>(p[0], each);
        return cudaGetLastError();
    }
    // the rows of a set are those of its members together: at least as many in the first set
    const bool few0 = p[0].plan.s.few, few1 = p[1].plan.s.few;
    if (few0 && !few1) return cudaErrorInvalidValue;
    // Short passes share the SMs by their steps (and one for each unit's end: 24 members' rows on 12288 shared
    // and 40 own keys, D = 128: 27 us, one after the other 31); of long ones the second follows the first on
    // each SM, which needs no guess of what a step of either costs.
    int64_t work[2];
    for (int k = 0; k < 2; ++k) {
        const FwdSet &s = p[k].plan.s;
        work[k] = s.sets * s.upz * ((s.n + kTile - 1) / kTile + 1);
    }
    if (p[0].plan.ctas + p[1].plan.ctas > kCtas && work[0] + work[1] < 16 * kCtas) {
        const int64_t share = kCtas * work[0] / (work[0] + work[1]), c0 = share < 1 ? 1 : (share > kCtas - 1 ? kCtas - 1 : share);
        if (p[0].plan.ctas > c0) p[0].plan.ctas = (int32_t)c0;
        if (p[1].plan.ctas > kCtas - c0) p[1].plan.ctas = (int32_t)(kCtas - c0);
    }
    e = few0   ? launch_pair<D, true, true>(maps, p, stream)
        : few1 ? launch_pair<D, false, true>(maps, p, stream)
               : launch_pair<D, false, false>(maps, p, stream);
    if (e != cudaSuccess) return e;
    if (p[0].all_rows <= 8 * 4 * kCtas)
        join_sets_kernel<D, 1><<<(unsigned)((p[0].all_rows + 7) / 8), 256, 0, stream>>>(p[0], p[1]);
    else
        join_sets_kernel<D, 2><<<(unsigned)((p[0].all_rows + 15) / 16), 256, 0, stream>>>(p[0], p[1]);
    return cudaGetLastError();
}

}  // namespace

FwdPlan make_fwd_plan(const DenseProblem &p, const KeySet &ks) {
    FwdPlan r{};
    r.rows = p.rows;
    r.kv_heads = p.kv_heads;
    r.batch = p.batch;
    FwdSet &s = r.s;
    s.len = ks.len;
    s.n = ks.n;
    s.sets = ks.sets;
    s.members = ks.members;
    s.few = p.rows <= kFewRows && ks.members * p.rows <= kFewRows;
    if (p.rows <= kTile) {
        const int64_t fit = kTile / p.rows;
        s.bb = (int32_t)(ks.members < fit ? ks.members : fit);
        s.tiles = (ks.members + s.bb - 1) / s.bb;
    } else {
        s.tpm = (int32_t)((p.rows + kTile - 1) / kTile);
        s.tiles = ks.members * s.tpm;
    }
    s.pairs = (s.tiles + 1) / 2;
    s.upz = p.kv_heads * s.pairs;
    const int64_t t = (ks.n + kTile - 1) / kTile, units = s.sets * s.upz;
    deal(r, units, t, !ks.len || ks.sets <= 1024);
    return r;
}

FwdLayout fwd_layout_of(const FwdPlan &plan, int64_t d, bool two_sets) {
    FwdLayout L{};
    size_t o = 0;
    auto take = [&](size_t floats) { const size_t at = o; o += (floats + 63) / 64 * 64; return at; };
    const size_t all = (size_t)plan.batch * plan.kv_heads * plan.rows;
    if (plan.stream) {
        L.part_o = take((size_t)plan.ctas * 4 * kTile * d);
        L.part_lse = take((size_t)plan.ctas * 4 * kTile);
        L.cuts = take((size_t)plan.ctas * 4);
    }
    if (two_sets) {
        L.whole_o = take(all * d);
        L.whole_lse = take(all);
        L.spans = take((size_t)plan.s.sets * plan.s.upz * 2);
    }
    L.total = o;
    return L;
}

cudaError_t launch_dense_fwd(const DenseProblem &pb, const void *q, const KeySet *sets, int nsets, void *out, void *low, float *lse,
                             float *ws, uint32_t *status, cudaStream_t stream) {
    FwdParams p[2] = {};
    for (int k = 0; k < nsets; ++k) {
        FwdParams &x = p[k];
        x.plan = make_fwd_plan(pb, sets[k]);
        const FwdLayout L = fwd_layout_of(x.plan, pb.d, nsets == 2);
        x.out = static_cast<__nv_bfloat16 *>(out);
        x.low = static_cast<__nv_bfloat16 *>(low);
        x.lse = lse;
        x.v = static_cast<const __nv_bfloat16 *>(sets[k].v);
        x.part_o = ws + L.part_o;
        x.part_lse = ws + L.part_lse;
        if (nsets == 2) {
            x.whole_o = ws + L.whole_o;
            x.whole_lse = ws + L.whole_lse;
            x.spans = reinterpret_cast<int2 *>(ws + L.spans);
        } else if (x.plan.stream) {
            x.cuts = reinterpret_cast<Cut *>(ws + L.cuts);
        }
        x.all_rows = pb.batch * pb.kv_heads * pb.rows;
        x.scale_log2 = pb.scale * 1.4426950408889634f;
        x.status = status;
        x.withhold = pb.withhold;
        ws += L.total;
    }
    return pb.d == 64 ? run<64>(pb, q, sets, nsets, p, stream) : run<128>(pb, q, sets, nsets, p, stream);
}

}  // namespace bsa
