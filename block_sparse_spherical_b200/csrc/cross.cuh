// Shared declarations of the dense attention over states of another length
// (cross attention, its backward, and attention over a shared prefix): the
// problem, how a forward's work is cut into units and handed to CTAs, and the
// launchers.
#pragma once

#include "bsa_internal.cuh"

namespace bsa {

struct DenseProblem {
    int64_t batch, heads, kv_heads, n_q, d;
    int64_t rows;           // (heads / kv_heads) * n_q: rows of a batch entry and key head
    float scale;
    int64_t withhold = -1;  // test hook: the copy of this number in the order of a CTA (key and value tiles; backward:
                            // steps) is not issued by the first CTA of each pass; -1: off
};

// One set of keys for the rows of a forward pass. The rows of a batch entry
// ("member") and key head are its `rows` = (heads / kv_heads)·n_q query rows,
// which [B][H][n_q][d] keeps contiguous; the members of one set share its keys.
struct KeySet {
    const void *k, *v;      // [sets][kv_heads][n][d] bf16
    const int32_t *len;     // [sets], nullable
    int64_t n;              // keys of a set
    int64_t sets;           // batch / members
    int64_t members;        // batch entries that share a set
};

constexpr int kTile = 128;          // query rows and keys of a tile
constexpr int kFewRows = 32;        // at most so many rows a set and key head: the "few rows" form
constexpr int kCtas = 148;          // SMs of a B200: the work is cut for one CTA each

// How the rows of one KeySet are cut. A unit is up to two tiles of 128 rows of
// one set and key head (all its rows in the few-rows form); its steps are the
// key tiles of the set's length, at least one.
struct FwdSet {
    const int32_t *len;
    int64_t n, sets, members;
    int32_t few;            // all rows of a set and key head fit kFewRows
    int32_t bb;             // members in a tile when rows <= 128, else 0 (a tile holds 128 rows of one member)
    int32_t tpm;            // bb == 0: tiles a member
    int64_t tiles, pairs;   // tiles and units of a set and key head
    int64_t upz;            // units of a set: kv_heads * pairs
    int32_t fixed;          // > 0 (key-major backward): a unit is a key tile and has so many steps, its
                            // query tiles; upz is then kv_heads * fixed, so that a set has upz steps a key tile
};

// A pass over one KeySet. `stream`: the steps of all units, end to end, are dealt to `ctas` CTAs in
// equal shares, so that a CTA begins and ends inside a unit; the parts of such a unit are joined
// afterwards. Otherwise CTA c takes the whole units c, c + ctas, ...
struct FwdPlan {
    FwdSet s;
    int32_t stream, ctas;
    int64_t rows, kv_heads, batch;
};

// Row i of tile t of set z, key head hk: its index in [B][kv_heads][rows], or -1. (32-bit divisions: a
// tile number of rows that fit a GPU is far below 2^31.)
__host__ __device__ inline int64_t plan_row(const FwdPlan &p, int64_t z, int64_t hk, int64_t t, int i) {
    const FwdSet &s = p.s;
    const uint32_t rows = (uint32_t)p.rows;
    uint32_t member, r;
    if (s.bb) {
        const uint32_t mi = (uint32_t)i / rows;
        if (mi >= (uint32_t)s.bb) return -1;
        member = (uint32_t)t * s.bb + mi;
        r = i - mi * rows;
    } else {
        member = (uint32_t)t / (uint32_t)s.tpm;
        r = ((uint32_t)t - member * s.tpm) * kTile + i;
    }
    if (member >= (uint32_t)s.members || r >= rows) return -1;
    return ((z * s.members + member) * p.kv_heads + hk) * p.rows + r;
}

// A unit that is cut, as its first CTA c leaves it for the join: its parts are that CTA's slot 1 and
// slot 0 of the CTAs up to `last`. last < 0: CTA c leaves none.
struct Cut {
    int32_t z, hk, tile, last;      // tile: pair of tiles (key-major backward: key tile)
};

// Workspace of a forward pass over a set, in floats. Parts: two slots a CTA (slot 1: a unit that the CTA
// begins and leaves unfinished, slot 0: one that it takes over) of 256 rows each, the normalised o
// and the row's log2-sum-exp. With two sets also: whole, the same of units that one CTA finished, by
// row, and of every unit its first and last CTA.
struct FwdLayout {
    size_t part_o, part_lse, cuts, whole_o, whole_lse, spans, total;
};
// How `units` of `steps` each go to the CTAs: p.stream and p.ctas. Cutting units gives every CTA the same
// number of steps, but its parts are written in fp32 (up to 256 rows a CTA, 38 MB at D = 128) and
// joined by a kernel: together 8 to 12 us, about six steps of 1.5 to 2.3 us (few rows: four of 1.0 to
// 1.3 us). So it is done where whole units would leave the busiest CTA with more steps than that.
// Measured at 96 units of up to 7 steps (six padded entries of 333 x 3 rows, D = 128): cut 33 us, whole
// units 24. `scan`: the lengths are few enough for a warp to add up at each CTA's start.
inline void deal(FwdPlan &p, int64_t units, int64_t steps, bool scan) {
    const int64_t rounds = (units + kCtas - 1) / kCtas, share = (units * steps + kCtas - 1) / kCtas;
    p.stream = scan && rounds * steps > (share > 2 ? share : 2) + (p.s.few ? 4 : 6);
    const int64_t want = p.stream ? (units * steps + 1) / 2 : units;
    p.ctas = (int32_t)(want < kCtas ? want : kCtas);
}
FwdPlan make_fwd_plan(const DenseProblem &p, const KeySet &set);
FwdLayout fwd_layout_of(const FwdPlan &plan, int64_t d, bool two_sets);

// Launchers (return cudaGetLastError()).
cudaError_t launch_dense_fwd(const DenseProblem &p, const void *q, const KeySet *sets, int nsets, void *out, void *low, float *lse,
                             float *workspace, uint32_t *status, cudaStream_t stream);
size_t dense_bwd_floats(const DenseProblem &p, const KeySet &s);   // workspace of a backward pass
cudaError_t launch_dense_bwd(const DenseProblem &p, const void *q, const KeySet &s, const void *out, const void *low,
                             const float *lse, const void *dout, void *dq, void *dk, void *dv, float *workspace, uint32_t *status,
                             cudaStream_t stream);

#ifdef __CUDACC__
// a / b of non-negative numbers: by the 32-bit division, a third of the 64-bit one's time, where it does.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// Keys of set z, clamped to the buffer; a length outside it is flagged in *status (nullable).
__device__ __forceinline__ int set_len(const int32_t *len, int64_t z, int64_t n, uint32_t *status) {
    if (!len) return (int)n;
    const int x = __ldg(len + z);
    if (x >= 0 && x <= n) return x;
    if (status) atomicOr(status, kStatusBadIndex);
    return x < 0 ? 0 : (int)n;
}
__device__ __forceinline__ int set_steps(const FwdSet &s, int64_t z) {
    return max(1, (set_len(s.len, z, s.n, nullptr) + kTile - 1) / kTile);
}
// Warp-wide: the sum over sets z < z1 of their units' steps.
__device__ __forceinline__ int64_t steps_before(const FwdSet &s, int64_t z1, int lane) {
    if (!s.len) return z1 * s.upz * set_steps(s, 0);
    int64_t sum = 0;
    for (int64_t z = lane; z < z1; z += 32) sum += set_steps(s, z);
    for (int i = 16; i; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
    return sum * s.upz;
}
// Of `total` steps dealt to min(ctas, total) CTAs: the first of CTA c, and the CTA that has step x.
__device__ __forceinline__ int64_t cta_first(int64_t c, int64_t total, int ctas) {
    const int64_t n = min((int64_t)ctas, total);
    return quotient(min(c, n) * total, n);
}
__device__ __forceinline__ int cta_of(int64_t x, int64_t total, int ctas) {
    const int64_t n = min((int64_t)ctas, total);
    return (int)quotient((x + 1) * n + total - 1, total) - 1;
}
// Warp-wide: the unit and step at which step x of the whole pass lies.
struct StepAt {
    int t, steps;           // step within the unit, steps of the unit
    int64_t z, uu;          // set, unit of the set
};
__device__ __forceinline__ StepAt step_at(const FwdPlan &p, int64_t x, int lane) {
    StepAt r;
    const FwdSet &s = p.s;
    if (!s.len) {
        r.steps = set_steps(s, 0);
        r.z = quotient(x, s.upz * r.steps);
        x -= r.z * s.upz * r.steps;
    } else {
        for (int64_t z0 = 0;; z0 += 32) {              // 32 sets at a time: an inclusive scan of their steps
            const int64_t z = z0 + lane;
            const int st = z < s.sets ? set_steps(s, z) : 0;
            int64_t inc = st * s.upz;
            for (int i = 1; i < 32; i <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, inc, i);
                if (lane >= i) inc += y;
            }
            const unsigned after = __ballot_sync(0xffffffffu, x < inc);
            if (after) {
                const int l = __ffs(after) - 1;
                const int64_t end = __shfl_sync(0xffffffffu, inc, l);
                r.steps = __shfl_sync(0xffffffffu, st, l);
                r.z = z0 + l;
                x -= end - r.steps * s.upz;
                break;
            }
            x -= __shfl_sync(0xffffffffu, inc, 31);
            if (z0 + 32 >= s.sets) {                   // not reached for x below the total
                r.z = s.sets - 1;
                r.steps = 1;
                x = 0;
                break;
            }
        }
    }
    if (s.fixed) r.steps = s.fixed;
    r.uu = quotient(x, r.steps);
    r.t = (int)(x - r.uu * r.steps);
    return r;
}
__device__ __forceinline__ int64_t total_steps(const FwdPlan &p, int lane) { return steps_before(p.s, p.s.sets, lane); }
#endif

}  // namespace bsa
