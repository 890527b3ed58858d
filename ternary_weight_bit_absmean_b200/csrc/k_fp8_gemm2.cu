// k_fp8_gemm2.cu -- the block-scaled e4m3 product of k_fp8_gemm.cu for many rows on both
// sides, on pairs of SMs (tcgen05.mma.cta_group::2 kind::f8f6f4).
//
//   out[q, p] = sum_g sq[g, q] sp(g, p) S_g[q, p],   S_g[q, p] = sum_{c in group g} Qm[q, c] Pm[p, c]
//
// A cluster of two CTAs computes a 256 x 256 tile; each CTA holds 128 rows of Qm and 128 rows
// of Pm per group of 128 (32 KB), and the accumulator of CTA r the products of its 128 rows of
// Qm with all 256 of Pm, one row per TMEM lane.  Per group the pair issues four MMAs (K = 32)
// into one of two 256-column accumulators; eight epilogue warps per CTA read the other one,
// scale it and add it to fp32 sums in registers (a thread owns one row and 128 columns).
// What a tile needs per group and SM: 512 cycles of the tensor pipe, 128 KB read from tensor
// memory, 32768 fp32 multiply-adds (256 cycles of the fp32 pipe; twice that when both sides
// are scaled by row), 64 KB through shared memory.  The tensor pipe is meant to be the bound.
//
// Roles per CTA (12 warps): warp 0 lane 0 issues the TMA loads (signalled on the even CTA's
// barrier), warp 1 lane 0 of the even CTA the MMAs, warp 2 copies scales into a ring of eight
// groups, warps 4-11 run the epilogue.  The register file is split by setmaxnreg: the first
// four warps give up what the epilogue's sums need.  All waits are bounded as in the
// ternary kernels; no load uses multicast.
#include <cuda_bf16.h>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "bl_device.cuh"
#include "bl_fp8.cuh"
#include "bl_internal.h"

namespace bl {

bool encode_tmap_u8_pitch(CUtensorMap* map, const void* ptr, uint64_t inner, uint64_t outer, uint64_t pitch,
                          uint32_t box_inner, uint32_t box_outer);

namespace {

constexpr int kHalf = 128;  // rows of Qm and of Pm per CTA
constexpr int kTile = 2 * kHalf;
constexpr int kG = 128;
constexpr int kThreads = 384;
constexpr int kWarpTma = 0, kWarpMma = 1, kWarpScale = 2, kWarpEpi = 4, kEpiWarps = 8;
constexpr int kOpBytes = kHalf * kG;  // one operand's half per stage: 16 KB
constexpr int kStages = 6;
constexpr int kSlots = 8;             // scale ring
constexpr int kSlotFloats = kHalf + kTile;
constexpr int kBars = 2 * kStages + 4 + 2 * kSlots + 1;
constexpr int kSmemBytes = 1024 + kStages * 2 * kOpBytes + kSlots * kSlotFloats * 4 + 8 * kBars + 16;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
// 128 threads give up registers for the 256 of the epilogue: 128 * 56 + 256 * 224 is
// the 384 * 168 that the block is launched with
constexpr int kRegsLaunch = 168, kRegsSmall = 56, kRegsEpi = 224;
static_assert(128 * kRegsSmall + 256 * kRegsEpi <= kThreads * kRegsLaunch, "register split");
constexpr unsigned long long kDrainNs = 200000000ull;

struct Args {
    Fp8Product d;
    int groups;
    int tiles_q, tiles_p, num_tiles;
};

// Tiles in panels of kPanel tiles along q, p running inside a panel: the tiles in flight share
// few rows of either operand, so both stay in L2.
constexpr int kPanel = 8;
__device__ __forceinline__ void tile_origin(const Args& a, int tile, int64_t& q0, int64_t& p0) {
    const int panel = tile / (kPanel * a.tiles_p);
    const int rest = tile - panel * kPanel * a.tiles_p;
    const int left = a.tiles_q - panel * kPanel;
    const int high = left < kPanel ? left : kPanel;
    q0 = static_cast<int64_t>(panel * kPanel + rest % high) * kTile;
    p0 = static_cast<int64_t>(rest / high) * kTile;
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
    const unsigned long long t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (globaltimer_ns() - t0 > kDrainNs) return;
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float2 v) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&p);
}

// 128 sums of one row -> out[q, p .. p + 127], 16-byte stores when the row allows them.
__device__ __forceinline__ void store_row(const Fp8Product& d, int64_t q, int64_t p, const uint64_t (&acc)[64]) {
    if (q >= d.Q) return;
    const int64_t off = q * d.P + p;
    if (p + 128 <= d.P && d.P % 8 == 0) {
        if (d.out_bf16) {
            uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(d.out) + off);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                o[j] = make_uint4(pack_bf16(unpack_f32x2(acc[4 * j])), pack_bf16(unpack_f32x2(acc[4 * j + 1])),
                                  pack_bf16(unpack_f32x2(acc[4 * j + 2])), pack_bf16(unpack_f32x2(acc[4 * j + 3])));
        } else {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(d.out) + off);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const float2 a = unpack_f32x2(acc[2 * j]), b = unpack_f32x2(acc[2 * j + 1]);
                o[j] = make_float4(a.x, a.y, b.x, b.y);
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 128; ++j) {
        if (p + j >= d.P) break;
        const float2 two = unpack_f32x2(acc[j / 2]);
        const float y = j % 2 == 0 ? two.x : two.y;
        if (d.out_bf16)
            static_cast<__nv_bfloat16*>(d.out)[off + j] = __float2bfloat16_rn(y);
        else
            static_cast<float*>(d.out)[off + j] = y;
    }
}

// ROWS: Pm is scaled by row (p_shift 0), else by blocks of 128 rows.
template <bool ROWS>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm2_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_p,
                     const Args a) {
    constexpr int ST = kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t sQ = base;
    const uint32_t sP = sQ + ST * kOpBytes;
    const uint32_t sScale = sP + ST * kOpBytes;
    const uint32_t sBar = sScale + kSlots * kSlotFloats * 4;
    auto full = [&](int s) { return sBar + 8u * s; };               // even CTA: both CTAs' loads
    auto empty = [&](int s) { return sBar + 8u * (ST + s); };       // local: stage read by the MMAs
    auto tfull = [&](int b) { return sBar + 8u * (2 * ST + b); };   // local: accumulator holds a group
    auto tempty = [&](int b) { return sBar + 8u * (2 * ST + 2 + b); };  // even CTA: read by both CTAs
    auto sfull = [&](int s) { return sBar + 8u * (2 * ST + 4 + s); };
    auto sempty = [&](int s) { return sBar + 8u * (2 * ST + 4 + kSlots + s); };
    const uint32_t drain_bar = sBar + 8u * (kBars - 1);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (sBar - base) + 8 * kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const float* scales = reinterpret_cast<const float*>(gbase + (sScale - base));

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull(b), 1);
            mbar_init(tempty(b), 2 * kEpiWarps);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(sfull(s), 32);
            mbar_init(sempty(s), kEpiWarps);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        mbar_fence_init();
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_p);
    }
    pdl_wait_then_release();
    if (warp == kWarpMma) {
        tmem_alloc_pair(smem_u32(tmem_slot), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers exist before either signals the other
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp < kWarpEpi) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsSmall));
        if (warp == kWarpTma && lane == 0) {
            // ------------------------------------------------------------ producer --
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            bool ok = true;
            for (int tile = first; ok && tile < a.num_tiles; tile += step) {
                int64_t q0, p0;
                tile_origin(a, tile, q0, p0);
                const int qr = static_cast<int>(q0) + kHalf * static_cast<int>(rank);
                const int pr = static_cast<int>(p0) + kHalf * static_cast<int>(rank);
                for (int g = 0; g < a.groups; ++g) {
                    if (!mbar_wait_cluster_bounded(empty(stage), phase ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (leader) mbar_arrive_expect_tx(full(stage), 4 * kOpBytes);
                    const uint32_t bar = mapa_shared(full(stage), 0);
                    tma_load_2d_pair(sQ + stage * kOpBytes, &tmap_q, bar, g * kG, qr);
                    tma_load_2d_pair(sP + stage * kOpBytes, &tmap_p, bar, g * kG, pr);
                    ++issued;
                    if (++stage == ST) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok && leader) {
                // both CTAs' loads are counted on this CTA's barriers
                for (int s = 0; s < ST; ++s) {
                    const long long fills = (issued - s + ST - 1) / ST;
                    if (fills > 0) drain_wait(full(s), static_cast<uint32_t>((fills - 1) & 1));
                }
            }
        } else if (warp == kWarpMma && lane == 0 && leader) {
            // ---------------------------------------------------------- MMA issuer --
            constexpr uint32_t idesc = idesc_e4m3(kTile, kTile);
            int stage = 0, buf = 0;
            uint32_t phase = 0, bphase = 0;
            bool ok = true;
            for (int tile = first; ok && tile < a.num_tiles; tile += step) {
                for (int g = 0; g < a.groups; ++g) {
                    if (!mbar_wait_cluster_bounded(tempty(buf), bphase ^ 1u, abort_flag) ||
                        !mbar_wait_cluster_bounded(full(stage), phase, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t qa = sQ + stage * kOpBytes, pa = sP + stage * kOpBytes;
#pragma unroll
                    for (int kk = 0; kk < kG / 32; ++kk)
                        tc_mma_f8_pair(tmem_base + static_cast<uint32_t>(buf * kTile), smem_desc_sw128(qa + kk * 32),
                                       smem_desc_sw128(pa + kk * 32), idesc, kk != 0 ? 1u : 0u);
                    tc_commit_pair_multicast(empty(stage), 0x3);
                    tc_commit_pair_multicast(tfull(buf), 0x3);
                    if (++stage == ST) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++buf == 2) {
                        buf = 0;
                        bphase ^= 1u;
                    }
                }
            }
            if (!ok) {
                tc_commit_pair_multicast(drain_bar, 0x1);
                drain_wait(drain_bar, 0);
            }
        } else if (warp == kWarpScale) {
            // -------------------------------------------------------------- scales --
            // rows past an edge take the last row's scale; they are not stored
            int slot = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int tile = first; ok && tile < a.num_tiles; tile += step) {
                int64_t q0, p0;
                tile_origin(a, tile, q0, p0);
                q0 += kHalf * static_cast<int>(rank);
                for (int g = 0; g < a.groups; ++g) {
                    if (!mbar_wait_bounded(sempty(slot), phase ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = sScale + static_cast<uint32_t>(slot * kSlotFloats * 4);
#pragma unroll
                    for (int c = 0; c < kHalf; c += 32) {
                        const int64_t q = q0 + c + lane < a.d.Q ? q0 + c + lane : a.d.Q - 1;
                        cp_async4(dst + 4u * (c + lane), a.d.sq + g * a.d.Q + q);
                    }
#pragma unroll
                    for (int c = 0; c < (ROWS ? kTile : 32); c += 32) {
                        // by blocks: two of them, copied by lanes 0 and 1
                        if (!ROWS && lane > 1) break;
                        const int64_t row = p0 + (ROWS ? c + lane : kHalf * lane);
                        const int64_t p = row < a.d.P ? row : a.d.P - 1;
                        cp_async4(dst + 4u * (kHalf + c + lane), a.d.sp + (p >> a.d.p_shift) * a.d.sp_p + g * a.d.sp_g);
                    }
                    cp_async_arrive(sfull(slot));
                    if (++slot == kSlots) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            }
            cp_async_wait_all();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
        // ------------------------------------------------------------ epilogue --
        const int quarter = warp & 3, half = (warp - kWarpEpi) >> 2;
        const int r = 32 * quarter + lane;
        const uint32_t t_addr = tmem_base + (static_cast<uint32_t>(32 * quarter) << 16) + 128u * half;
        int slot = 0, buf = 0;
        uint32_t sphase = 0, bphase = 0;
        bool ok = true;
        for (int tile = first; tile < a.num_tiles; tile += step) {
            int64_t q0, p0;
            tile_origin(a, tile, q0, p0);
            uint64_t acc[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[j] = 0;
            for (int g = 0; g < a.groups; ++g) {
                if (!mbar_wait_bounded(sfull(slot), sphase, abort_flag) ||
                    !mbar_wait_cluster_bounded(tfull(buf), bphase, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float* sc = scales + slot * kSlotFloats;
                const float fq = sc[r] * (ROWS ? 1.0f : sc[kHalf + half]);
                const uint64_t f2 = pack_f32x2(fq, fq);
                const uint32_t addr = t_addr + static_cast<uint32_t>(buf * kTile);
                uint32_t v[2][32];
                tmem_ld_32x32b_x32(addr, v[0]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tmem_ld_wait_for(v[c & 1]);
                    if (c < 3) {
                        tmem_ld_32x32b_x32(addr + 32u * (c + 1), v[(c + 1) & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(mapa_shared(tempty(buf), 0));
                    }
                    const float4* sp4 = reinterpret_cast<const float4*>(sc + kHalf + 128 * half + 32 * c);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t* w = &v[c & 1][4 * j];
                        uint64_t lo = f2, hi = f2;
                        if constexpr (ROWS) {
                            const float4 s4 = sp4[j];
                            lo = mul_f32x2(f2, pack_f32x2(s4.x, s4.y));
                            hi = mul_f32x2(f2, pack_f32x2(s4.z, s4.w));
                        }
                        uint64_t* o = &acc[16 * c + 2 * j];
                        o[0] = fma_f32x2(pack_f32x2(__uint_as_float(w[0]), __uint_as_float(w[1])), lo, o[0]);
                        o[1] = fma_f32x2(pack_f32x2(__uint_as_float(w[2]), __uint_as_float(w[3])), hi, o[1]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(sempty(slot));
                if (++slot == kSlots) {
                    slot = 0;
                    sphase ^= 1u;
                }
                if (++buf == 2) {
                    buf = 0;
                    bphase ^= 1u;
                }
            }
            if (!ok) break;
            store_row(a.d, q0 + kHalf * static_cast<int>(rank) + r, p0 + 128 * half, acc);
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // no CTA leaves while its peer may still signal its barriers
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
    if (threadIdx.x == 0 && *abort_flag && a.d.err != nullptr) atomicOr(a.d.err, kErrBitTimeout);
}

template <bool ROWS>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tp, const Args& a, int pairs, cudaStream_t stream) {
    static PerContextOnce attr;
    cudaError_t e = attr.run([] {
        return cudaFuncSetAttribute(fp8_gemm2_kernel<ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(fp8_gemm2_kernel<ROWS>, dim3(static_cast<unsigned>(2 * pairs)), dim3(kThreads), kSmemBytes,
                      stream, dim3(2, 1, 1), tq, tp, a);
}

}  // namespace

cudaError_t launch_fp8_product_pair(const Fp8Product& d, cudaStream_t stream) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t tiles_q = (d.Q + kTile - 1) / kTile, tiles_p = (d.P + kTile - 1) / kTile;
    // tile numbers are 32-bit, with room for one more step of the grid
    if (tiles_q * tiles_p >= (int64_t(1) << 30)) return cudaErrorInvalidValue;
    CUtensorMap tq, tp;
    const uint64_t pitch = static_cast<uint64_t>(fp8_row_bytes(d.C));
    if (!encode_tmap_u8_pitch(&tq, d.q, static_cast<uint64_t>(d.C), static_cast<uint64_t>(d.Q), pitch, kG, kHalf) ||
        !encode_tmap_u8_pitch(&tp, d.p, static_cast<uint64_t>(d.C), static_cast<uint64_t>(d.P), pitch, kG, kHalf))
        return cudaErrorInvalidValue;
    const Args a{d, static_cast<int>((d.C + kG - 1) / kG), static_cast<int>(tiles_q), static_cast<int>(tiles_p),
                 static_cast<int>(tiles_q * tiles_p)};
    const int pairs = a.num_tiles < sms / 2 ? a.num_tiles : sms / 2;
    return d.p_shift == 0 ? launch<true>(tq, tp, a, pairs, stream) : launch<false>(tq, tp, a, pairs, stream);
}

}  // namespace bl
