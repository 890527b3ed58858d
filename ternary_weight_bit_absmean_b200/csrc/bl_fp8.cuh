// bl_fp8.cuh -- building blocks of the 8-bit floating-point product kernels: the
// tcgen05 kind::f8f6f4 MMA, packed fp32 arithmetic, small asynchronous copies, and the
// description of one block-scaled product shared by the kernels.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "bl_device.cuh"
#include "bl_wait.cuh"

namespace bl {

// D[tmem] (+)= A[smem] * B[smem]^T on 8-bit floats, fp32 accumulation, issued by one thread.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor: kind::f8f6f4, A and B e4m3, K-major, D fp32, shape M x N.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4)                                 // D format: F32 (A and B formats 0: e4m3)
           | (static_cast<uint32_t>(N >> 3) << 17)   // N / 8
           | (static_cast<uint32_t>(M >> 4) << 24);  // M / 16
}

// The same over a CTA pair: M rows of A and N rows of B, half of each in either CTA's shared
// memory at the same offsets.  Issued by one thread of the even CTA.
__device__ __forceinline__ void tc_mma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Wait for every tcgen05.ld of this warp; the registers it fills are named so that no use of
// them can move ahead of the wait.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// Two fp32 values in one 64-bit register pair, for the packed multiply and fma.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Copy 4 bytes global -> shared without a register; and have this thread arrive on `bar`
// when all of its copies so far have landed (one of the barrier's expected arrivals).
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// True in one lane of a converged warp.  Instructions with warp-uniform operands (MMAs, commits,
// TMA loads) are cheap to issue under it; under a test of the lane number they are not.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// How the products' warps give a wait up.  The lanes of a warp poll a barrier and the abort flag on
// their own (wait_on), so some can see a phase complete while others give up, and what follows a wait
// (elect.sync, tcgen05.ld, __syncwarp) wants the warp whole.  So giving up ends no loop: the lane goes
// along to the end with its `ok` false; loads and MMAs are issued where the elected lane's waits all
// succeeded, and results stored where every lane's did.  (4096 x 4096 x 1536 34.1 us, its gradients 38
// and 40; with a vote and a way out after every wait instead 35.4, 40 and 43.)

// One product of the library in the kernels' terms:
//   out[q, p] = sum_g sq[g, q] sp(g, p) sum_{c in group g} Qm[q, c] Pm[p, c]
// Qm is the left operand of the public entry points (tokens, or rows of W for the weight
// gradient), Pm the right one; both hold e4m3 codes with the contraction index c
// innermost and groups of 128 of it.  sq has one scale per row of Qm; sp one per row
// (p_shift 0) or one per 128 rows (p_shift 7): sp[(p >> p_shift) * sp_p + g * sp_g].
struct Fp8Product {
    const uint8_t* q;
    const uint8_t* p;
    int64_t Q, P, C;
    const float* sq;
    const float* sp;
    int64_t sp_p, sp_g;
    int p_shift;
    void* out;      // [Q, P]
    int out_bf16;
    int32_t* err;
};

// 2-D tensor map over rows of `inner` bytes that start every `pitch` bytes, 128-byte
// swizzle, zero fill outside; encoded anew by every call (k_fp8_gemm.cu).
bool encode_tmap_u8_pitch(CUtensorMap* map, const void* ptr, uint64_t inner, uint64_t outer, uint64_t pitch,
                          uint32_t box_inner, uint32_t box_outer);

// The kernel on pairs of SMs (k_fp8_gemm2.cu), with tiles of 256 x tile_p.
cudaError_t launch_fp8_product_pair(const Fp8Product& d, int tile_p, int sms, cudaStream_t stream);

}  // namespace bl
