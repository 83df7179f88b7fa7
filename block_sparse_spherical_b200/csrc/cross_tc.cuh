// Tensor-core glue of the dense attention kernels: TMA copies of 3-d and 4-d boxes,
// tcgen05.mma with an operand in tensor memory, instruction descriptors, and the
// host side of their tensor maps.
#pragma once

#include <atomic>

#include "tc_common.cuh"

namespace bsa {
namespace tc {

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2,
                                            int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// A value that is the same in all lanes, known to be so by the compiler too (all lanes take part).
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Contiguous bytes (16-byte aligned, a multiple of 16) of global memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// Waits for this thread's loads from tensor memory. The loaded values pass through the wait, so that
// nothing that uses them can be moved ahead of it.
__device__ __forceinline__ void tmem_wait_ld_of(float (&x)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]), "+f"(x[8]),
          "+f"(x[9]), "+f"(x[10]), "+f"(x[11]), "+f"(x[12]), "+f"(x[13]), "+f"(x[14]), "+f"(x[15]), "+f"(x[16]),
          "+f"(x[17]), "+f"(x[18]), "+f"(x[19]), "+f"(x[20]), "+f"(x[21]), "+f"(x[22]), "+f"(x[23]), "+f"(x[24]),
          "+f"(x[25]), "+f"(x[26]), "+f"(x[27]), "+f"(x[28]), "+f"(x[29]), "+f"(x[30]), "+f"(x[31])
        :
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld_of(float (&x)[64]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]), "+f"(x[8]),
          "+f"(x[9]), "+f"(x[10]), "+f"(x[11]), "+f"(x[12]), "+f"(x[13]), "+f"(x[14]), "+f"(x[15]), "+f"(x[16]),
          "+f"(x[17]), "+f"(x[18]), "+f"(x[19]), "+f"(x[20]), "+f"(x[21]), "+f"(x[22]), "+f"(x[23]), "+f"(x[24]),
          "+f"(x[25]), "+f"(x[26]), "+f"(x[27]), "+f"(x[28]), "+f"(x[29]), "+f"(x[30]), "+f"(x[31]), "+f"(x[32]),
          "+f"(x[33]), "+f"(x[34]), "+f"(x[35]), "+f"(x[36]), "+f"(x[37]), "+f"(x[38]), "+f"(x[39]), "+f"(x[40]),
          "+f"(x[41]), "+f"(x[42]), "+f"(x[43]), "+f"(x[44]), "+f"(x[45]), "+f"(x[46]), "+f"(x[47]), "+f"(x[48]),
          "+f"(x[49]), "+f"(x[50]), "+f"(x[51]), "+f"(x[52]), "+f"(x[53]), "+f"(x[54]), "+f"(x[55]), "+f"(x[56]),
          "+f"(x[57]), "+f"(x[58]), "+f"(x[59]), "+f"(x[60]), "+f"(x[61]), "+f"(x[62]), "+f"(x[63])
        :
        : "memory");
}
// Bounded wait (2 s, as wait_bar) that does not read the global timer, which costs more than most waits
// last, before it has been suspended a few times.
__device__ __forceinline__ bool wait_soon(uint64_t *b, uint32_t parity, volatile int *abort_flag, uint32_t *status) {
    if (mbar_try_wait(b, parity)) return true;
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
        if (mbar_try_wait_sleep(b, parity, kSleepNs)) return true;
    return wait_bar(b, parity, abort_flag, status);
}
// One arrival for a whole warp, after all its lanes (32 arrivals at one address would queue up).
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// D (TMEM) (+)= A·B with A (K-major bf16 pairs, the lanes of D) read from tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor: D f32, A and B bf16, M = 128, N = n, A K-major, B K- or MN-major.
constexpr uint32_t idesc_of(int n, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// 2^x of two values on the FMA pipe, x < 127 (here at most 8, by which a running maximum may lag): x = n + f with
// n = round(x), f in [-1/2, 1/2]; 2^f by the degree-3 minimax polynomial that the block-sparse kernel's route
// uses too (relative error 7.5e-5, a twentieth of a bf16 rounding's mean), times 2^n. Below -126.5 n is -127, whose
// exponent bits are those of 0: exactly 0, also for -inf, as the exponential unit gives. NaN gives NaN.
__device__ __forceinline__ float2 exp2_fma2(float2 x) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(x.x) : "f"(-127.f));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(x.y) : "f"(-127.f));
    const float2 t = __fadd2_rn(x, make_float2(0x1.8p23f, 0x1.8p23f));           // low bits: n
    const float2 n = __fadd2_rn(t, make_float2(-0x1.8p23f, -0x1.8p23f));
    const float2 f = __ffma2_rn(n, make_float2(-1.f, -1.f), x);                 // x - n, exact
    float2 p = __ffma2_rn(f, make_float2(0x1.c3f76p-5f, 0x1.c3f76p-5f), make_float2(0x1.f0de1ap-3f, 0x1.f0de1ap-3f));
    p = __ffma2_rn(p, f, make_float2(0x1.62f31ap-1f, 0x1.62f31ap-1f));
    p = __ffma2_rn(p, f, make_float2(0x1.fff692p-1f, 0x1.fff692p-1f));
    return __fmul2_rn(p, make_float2(__uint_as_float((__float_as_uint(t.x) << 23) + 0x3f800000u),
                                     __uint_as_float((__float_as_uint(t.y) << 23) + 0x3f800000u)));
}
// 32 lanes x 16 columns: thread t of the warp gets TMEM lane (base + t), once the load is complete.
__device__ __forceinline__ void tmem_ld16_now(uint32_t taddr, uint32_t *u) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(taddr)
        : "memory");
}
// 32 lanes x 16 columns: thread t of the warp writes TMEM lane (base + t).
__device__ __forceinline__ void tmem_st16w(uint32_t taddr, const uint32_t *u) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]),
        "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
        : "memory");
}

// 64 bytes of each of a warp's 32 rows to global memory: lane l brings its row's 16 words and its address.
// Through 2 KB of shared memory (16-byte pieces exchanged so that neither side meets bank conflicts), so
// that four lanes write one row's 64 bytes together: with each lane writing its own row, every store
// touches 32 lines, and an epilogue of 128 rows of 128 floats took 10,000 clocks.
__device__ __forceinline__ void store_rows(uint8_t *stage, const uint32_t (&w)[16], void *dst, bool valid, int lane) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4 *>(stage + 64 * lane + 16 * (c ^ ((lane >> 1) & 3))) =
            make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    __syncwarp();
    const unsigned rows = __ballot_sync(0xffffffffu, valid);
    const int c = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2);
        const uint4 v = *reinterpret_cast<const uint4 *>(stage + 64 * r + 16 * (c ^ ((r >> 1) & 3)));
        char *to = reinterpret_cast<char *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), r));
        if ((rows >> r) & 1u) *reinterpret_cast<uint4 *>(to + 16 * c) = v;
    }
    __syncwarp();
}
// What rounding two values to bf16 (w) leaves off, as bf16.
__device__ __forceinline__ uint32_t rest_bf16x2(float a, float b, uint32_t w) {
    const float2 r = __ffma2_rn(make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)),
                                make_float2(-1.f, -1.f), make_float2(a, b));
    return pack_bf16x2(r.x, r.y);
}
// `cols` accumulator columns (a multiple of 32) of a warp's 32 rows, times f, to global memory: as bf16 (and
// what that rounding leaves off to `low`, if it is not null), or as fp32 parts. dst, low: lane l's row.
// zero: the row is zeros whatever the accumulator holds. Not inlined: an epilogue's registers would
// otherwise spill what the loop around it keeps.
static __device__ __noinline__ void write_rows(uint8_t *stage, uint32_t taddr, int cols, float f, bool zero, bool bf16, void *dst,
                                        void *low, bool valid, int lane) {
#pragma unroll 1
    for (int cc = 0; cc < cols; cc += 32) {
        float o[32];
        tmem_ld32(taddr + cc, o);
        tmem_wait_ld_of(o);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            const float2 y = __fmul2_rn(make_float2(o[e], o[e + 1]), make_float2(f, f));
            o[e] = y.x, o[e + 1] = y.y;
        }
        if (__any_sync(0xffffffffu, zero)) {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = zero ? 0.f : o[e];
        }
        uint32_t w[16];
        if (bf16) {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(o[2 * e], o[2 * e + 1]);
            store_rows(stage, w, static_cast<char *>(dst) + 2 * cc, valid, lane);
            if (__any_sync(0xffffffffu, low != nullptr)) {
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = rest_bf16x2(o[2 * e], o[2 * e + 1], w[e]);
                store_rows(stage, w, static_cast<char *>(low) + 2 * cc, valid && low, lane);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[16 * h + e]);
                store_rows(stage, w, static_cast<char *>(dst) + 4 * (cc + 16 * h), valid, lane);
            }
        }
    }
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// ---- host

inline bool make_map(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
              const cuuint32_t *box) {
    auto fn = encode_tiled_fn();
    if (!fn) return false;
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Sets a kernel up for its dynamic shared memory, once a device: later calls on the same device cost a
// look at a bit. Also refuses a kernel whose register split (setmaxnreg.inc would wait forever for
// registers that a CTA was not launched with) does not fit what it was compiled to.
template <auto KERNEL>
inline cudaError_t kernel_ready(size_t smem, int threads, int regs_needed) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, KERNEL)) != cudaSuccess) return e;
    if (fa.numRegs * threads < regs_needed || fa.maxThreadsPerBlock < threads) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

}  // namespace tc
}  // namespace bsa
