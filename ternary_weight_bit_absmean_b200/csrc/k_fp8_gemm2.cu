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
// are scaled by row), 64 KB through shared memory.
//
// Roles per CTA (12 warps): warp 0 issues the TMA loads (signalled on the even CTA's barrier),
// warp 1 of the even CTA the MMAs, warp 2 copies scales into a ring of eight groups, warps
// 4-11 run the epilogue.  Loads and MMAs are issued by an elected lane of a warp whose lanes
// all run the loop: issued from a branch of one lane, four MMAs and two commits took 590
// cycles against 230, more than the tensor pipe needs for them.  The register file is split
// by setmaxnreg.  All waits are bounded as in the ternary kernels; a pair that gives up (see
// bl_fp8.cuh) lets its roles run out and waits for its loads and MMAs in flight.  No load uses
// multicast.
//
// Measured (bf16 output): 8192 x 8640 x 3200 in 222 us on a cool GPU, 2.04 PFLOP/s, and up to 245
// where the power limit has lowered the clock (260 a call in a loop of calls); with the epilogue
// taken out, loads and MMAs alone run at 3.05 PFLOP/s.  What is left is the hand-over of the two
// accumulators (an accumulator is busy for its MMAs, the commit, the readers' 430 cycles and
// their signal back: about 1660 cycles for two groups on an idle GPU) and the clock, which
// the power limit lowers.
#include <cuda_bf16.h>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "bl_device.cuh"
#include "bl_fp8.cuh"
#include "bl_internal.h"

namespace bl {

namespace {

constexpr int kHalf = 128;  // rows of Qm per CTA
constexpr int kTileQ = 2 * kHalf;
constexpr int kG = 128;
constexpr int kThreads = 384;
constexpr int kWarpTma = 0, kWarpMma = 1, kWarpScale = 2, kWarpEpi = 4, kEpiWarps = 8;
constexpr int kSlots = 8;             // scale ring
constexpr int kTurnBytes = 4096;      // of an epilogue warp: 32 rows x 128 bytes of output

// TP: columns of a tile (rows of Pm), 256 or 128.
template <int TP>
struct Cfg {
    static constexpr int kCols = TP / (kEpiWarps / 4);  // columns of an epilogue thread
    static constexpr int kQBytes = kHalf * kG, kPBytes = TP / 2 * kG;  // of a stage, per CTA
    static constexpr int kStages = TP == 256 ? 5 : 7;
    static constexpr int kBufs = 512 / TP;              // accumulators
    static constexpr int kSlotFloats = kHalf + TP;
    static constexpr int kBars = 2 * kStages + 2 * kBufs + 2 * kSlots + 1;
    static constexpr int kSmemBytes = 1024 + kStages * (kQBytes + kPBytes) + kEpiWarps * kTurnBytes +
                                      kSlots * kSlotFloats * 4 + 8 * kBars + 16;  // and three words
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};
// the first four warps give up registers for the epilogue's sums: 128 * 56 + 256 * 224 is the
// 384 * 168 that the block is launched with
constexpr int kRegsLaunch = 168, kRegsSmall = 56, kRegsEpi = 224;
static_assert(128 * kRegsSmall + 256 * kRegsEpi <= kThreads * kRegsLaunch, "register split");

struct Args {
    Fp8Product d;
    int groups;
    int tiles_q, tiles_p, num_tiles;
    unsigned long long wait_ns;  // limit of every wait (2 s outside the bounded-wait test)
    int stall_after;             // the producers stop after this many loads (< 0: never)
};

// Tiles in panels of kPanel tiles along q, p running inside a panel: the tiles in flight share
// few rows of either operand, so both stay in L2.
constexpr int kPanel = 8;
__device__ __forceinline__ void tile_origin(const Args& a, int tp, int tile, int64_t& q0, int64_t& p0) {
    const int panel = tile / (kPanel * a.tiles_p);
    const int rest = tile - panel * kPanel * a.tiles_p;
    const int left = a.tiles_q - panel * kPanel;
    const int high = left < kPanel ? left : kPanel;
    q0 = static_cast<int64_t>(panel * kPanel + rest % high) * kTileQ;
    p0 = static_cast<int64_t>(rest / high) * tp;
}

// Shared variables of another CTA of the cluster, and a barrier's bytes of a load that never came.
__device__ __forceinline__ void st_shared_cluster(uint32_t addr, int v) {
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ int ld_shared_cluster(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ void add_scaled2(const uint32_t* v, uint64_t scale, float* acc) {
    const float2 r = unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(v[0]), __uint_as_float(v[1])), scale,
                                            pack_f32x2(acc[0], acc[1])));
    acc[0] = r.x;
    acc[1] = r.y;
}

// The sums of a warp's 32 rows (one per lane) x kCols columns -> out.
// A row's sums sit in one thread, so storing them from there would write 32 scattered pieces
// per instruction; they are turned in shared memory (128 bytes of every row at a time, 16-byte
// chunks swizzled so that neither side has bank conflicts) and leave as whole 128-byte lines.
template <typename T, int kCols>
__device__ __forceinline__ void store_rows(const Fp8Product& d, int64_t q, int64_t p, const float (&acc)[kCols],
                                           uint8_t* turn, int lane) {
    constexpr int kPer = 128 / static_cast<int>(sizeof(T));  // columns per round: 32 or 64
    const bool wide = (d.P * static_cast<int64_t>(sizeof(T))) % 16 == 0;
    T* out = static_cast<T*>(d.out);
#pragma unroll
    for (int c0 = 0; c0 < kCols; c0 += kPer) {
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint4 w;
            if constexpr (sizeof(T) == 2) {
                const float* s = &acc[c0 + 8 * c];
                w = make_uint4(pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]), pack_bf16(s[4], s[5]),
                               pack_bf16(s[6], s[7]));
            } else {
                const float* s = &acc[c0 + 4 * c];
                w = make_uint4(__float_as_uint(s[0]), __float_as_uint(s[1]), __float_as_uint(s[2]),
                               __float_as_uint(s[3]));
            }
            *reinterpret_cast<uint4*>(turn + 128 * lane + ((c ^ (lane & 7)) << 4)) = w;
        }
        __syncwarp();
        if (wide) {
            const int64_t pc = p + c0 + (lane & 7) * (16 / static_cast<int>(sizeof(T)));
            const int64_t left = pc < d.P ? d.Q - q : 0;  // rows to store
            T* o = out + q * d.P + pc;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 4 * i + (lane >> 3);
                const uint4 w = *reinterpret_cast<const uint4*>(turn + 128 * r + (((lane & 7) ^ (r & 7)) << 4));
                if (r < left) *reinterpret_cast<uint4*>(o + r * d.P) = w;
            }
        } else {
            // rows of `out` start anywhere: a lane stores four bytes of a row, in one piece where
            // they are aligned
            constexpr int kPair = 4 / static_cast<int>(sizeof(T));
            const int64_t pc = p + c0 + lane * kPair, room = d.P - pc;
            const int n = d.Q - q < 32 ? static_cast<int>(d.Q - q) : 32;
            T* o = out + q * d.P + pc;
            if (room > 0) {
#pragma unroll 4
                for (int r = 0; r < n; ++r, o += d.P) {
                    const uint32_t w =
                        *reinterpret_cast<const uint32_t*>(turn + 128 * r + (((lane >> 2) ^ (r & 7)) << 4) + 4 * (lane & 3));
                    if (room >= kPair && (reinterpret_cast<uintptr_t>(o) & 3u) == 0) {
                        *reinterpret_cast<uint32_t*>(o) = w;
                    } else {
                        uint16_t* h = reinterpret_cast<uint16_t*>(o);  // only bf16 comes here
                        h[0] = static_cast<uint16_t>(w);
                        if (room > 1) h[1] = static_cast<uint16_t>(w >> 16);
                    }
                }
            }
        }
    }
}

// ROWS: Pm is scaled by row (p_shift 0), else by blocks of 128 rows.
template <bool ROWS, int TP>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm2_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_p,
                     const Args a) {
    using C = Cfg<TP>;
    constexpr int ST = C::kStages, NB = C::kBufs, kCols = C::kCols;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t sQ = base;
    const uint32_t sP = sQ + ST * C::kQBytes;
    const uint32_t sTurn = sP + ST * C::kPBytes;
    const uint32_t sScale = sTurn + kEpiWarps * kTurnBytes;
    const uint32_t sBar = sScale + kSlots * C::kSlotFloats * 4;
    auto full = [&](int s) { return sBar + 8u * s; };               // even CTA: both CTAs' loads
    auto empty = [&](int s) { return sBar + 8u * (ST + s); };       // local: stage read by the MMAs
    auto tfull = [&](int b) { return sBar + 8u * (2 * ST + b); };   // local: accumulator holds a group
    auto tempty = [&](int b) { return sBar + 8u * (2 * ST + NB + b); };  // even CTA: read by both CTAs
    auto sfull = [&](int s) { return sBar + 8u * (2 * ST + 2 * NB + s); };
    auto sempty = [&](int s) { return sBar + 8u * (2 * ST + 2 * NB + kSlots + s); };
    const uint32_t drain_bar = sBar + 8u * (C::kBars - 1);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (sBar - base) + 8 * C::kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* issued_loads = reinterpret_cast<volatile int*>(tmem_slot + 2);  // by this CTA's producer
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
        for (int b = 0; b < NB; ++b) {
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
        if (warp == kWarpTma) {
            // ------------------------------------------------------------ producer --
            int stage = 0;
            uint32_t phase = 0;
            int issued = 0;
            bool ok = true;
            for (int tile = first; tile < a.num_tiles; tile += step) {
                int64_t q0, p0;
                tile_origin(a, TP, tile, q0, p0);
                const int qr = static_cast<int>(q0) + kHalf * static_cast<int>(rank);
                const int pr = static_cast<int>(p0) + TP / 2 * static_cast<int>(rank);
                for (int g = 0; g < a.groups; ++g) {
                    ok &= wait_on(empty(stage), phase ^ 1u, abort_flag, a.wait_ns);
                    if (ok && issued == a.stall_after) {  // the bounded-wait test: stop issuing
                        stall_until_abort(abort_flag, 4 * a.wait_ns);
                        ok = false;
                    }
                    issued += ok;
                    if (elect_one() && ok) {
                        if (leader) mbar_arrive_expect_tx(full(stage), 2 * (C::kQBytes + C::kPBytes));
                        const uint32_t bar = mapa_shared(full(stage), 0);
                        tma_load_2d_pair(sQ + stage * C::kQBytes, &tmap_q, bar, g * kG, qr);
                        tma_load_2d_pair(sP + stage * C::kPBytes, &tmap_p, bar, g * kG, pr);
                    }
                    __syncwarp();
                    if (++stage == ST) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (elect_one()) *issued_loads = issued;
            __syncwarp();
        } else if (warp == kWarpScale) {
            // -------------------------------------------------------------- scales --
            // rows past an edge take the last row's scale; they are not stored
            int slot = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int tile = first; ok && tile < a.num_tiles; tile += step) {
                int64_t q0, p0;
                tile_origin(a, TP, tile, q0, p0);
                q0 += kHalf * static_cast<int>(rank);
                for (int g = 0; g < a.groups; ++g) {
                    if (!wait_on(sempty(slot), phase ^ 1u, abort_flag, a.wait_ns)) {
                        ok = false;  // a lane alone may leave: nothing here wants the warp whole
                        break;
                    }
                    const uint32_t dst = sScale + static_cast<uint32_t>(slot * C::kSlotFloats * 4 + 4 * lane);
                    const float* sq = a.d.sq + g * a.d.Q;
#pragma unroll
                    for (int c = 0; c < kHalf / 32; ++c) {
                        const int64_t q = q0 + 32 * c + lane;
                        cp_async4(dst + 128u * c, sq + (q < a.d.Q ? q : a.d.Q - 1));
                    }
                    const float* sp = a.d.sp + g * a.d.sp_g;
#pragma unroll
                    for (int c = 0; c < (ROWS ? TP / 32 : 1); ++c) {
                        // by blocks: one for each 128 columns, copied by the first lanes
                        if (!ROWS && lane >= TP / 128) break;
                        const int64_t row = p0 + (ROWS ? 32 * c + lane : 128 * lane);
                        const int64_t p = row < a.d.P ? row : a.d.P - 1;
                        cp_async4(dst + 4u * kHalf + 128u * c, sp + (p >> a.d.p_shift) * a.d.sp_p);
                    }
                    cp_async_arrive(sfull(slot));
                    if (++slot == kSlots) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            }
            cp_async_wait_all();
        } else if (warp == kWarpMma && leader) {
            // ---------------------------------------------------------- MMA issuer --
            constexpr uint32_t idesc = idesc_e4m3(kTileQ, TP);
            int stage = 0, buf = 0;
            uint32_t phase = 0, bphase = 0;
            bool ok = true;
            for (int tile = first; tile < a.num_tiles; tile += step) {
                for (int g = 0; g < a.groups; ++g) {
                    ok &= wait_on(full(stage), phase, abort_flag, a.wait_ns);
                    ok &= wait_on(tempty(buf), bphase ^ 1u, abort_flag, a.wait_ns);
                    tc_fence_after();
                    if (elect_one() && ok) {
                        const uint32_t qa = sQ + stage * C::kQBytes, pa = sP + stage * C::kPBytes;
#pragma unroll
                        for (int kk = 0; kk < kG / 32; ++kk)
                            tc_mma_f8_pair(tmem_base + static_cast<uint32_t>(buf * TP),
                                           smem_desc_sw128(qa + kk * 32), smem_desc_sw128(pa + kk * 32), idesc,
                                           kk != 0 ? 1u : 0u);
                        // the accumulator's readers are the ones being waited for
                        tc_commit_pair_multicast(tfull(buf), 0x3);
                        tc_commit_pair_multicast(empty(stage), 0x3);
                    }
                    __syncwarp();
                    if (++stage == ST) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++buf == NB) {
                        buf = 0;
                        bphase ^= 1u;
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
        // ------------------------------------------------------------ epilogue --
        // a thread: one row (its TMEM lane), kCols columns; sums by blocks use plain multiply-adds,
        // which measured faster there than packed ones (8192^3: 586 against 650 us without stores)
        const int quarter = warp & 3, block = (warp - kWarpEpi) >> 2;
        const int r = 32 * quarter + lane;
        const uint32_t t_addr =
            tmem_base + (static_cast<uint32_t>(32 * quarter) << 16) + static_cast<uint32_t>(kCols * block);
        uint8_t* turn = gbase + (sTurn - base) + (warp - kWarpEpi) * kTurnBytes;
        int slot = 0, buf = 0;
        uint32_t sphase = 0, bphase = 0;
        bool ok = true;
        for (int tile = first; tile < a.num_tiles; tile += step) {
            float acc[kCols];
#pragma unroll
            for (int j = 0; j < kCols; ++j) acc[j] = 0.0f;
            for (int g = 0; g < a.groups; ++g) {
                ok &= wait_on(sfull(slot), sphase, abort_flag, a.wait_ns);
                const float* sc = scales + slot * C::kSlotFloats;
                const float fq = sc[r] * (ROWS ? 1.0f : sc[kHalf + block * kCols / 128]);
                ok &= wait_on(tfull(buf), bphase, abort_flag, a.wait_ns);
                __syncwarp();  // the lanes' polls may have ended at different times
                tc_fence_after();
                const uint32_t addr = t_addr + static_cast<uint32_t>(buf * TP);
                // the next 32 columns are on their way while these are scaled
                uint32_t v2[2][32];
                tmem_ld_32x32b_x32(addr, v2[0]);
#pragma unroll
                for (int c = 0; c < kCols / 32; ++c) {
                    uint32_t(&v)[32] = v2[c & 1];
                    tmem_ld_wait_for(v);
                    if (c + 1 < kCols / 32) {
                        tmem_ld_32x32b_x32(addr + 32u * (c + 1), v2[(c + 1) & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(mapa_shared(tempty(buf), 0));
                    }
                    float* o = &acc[32 * c];
                    if constexpr (ROWS) {
                        // two scales per sum: packed arithmetic halves the instructions
                        const float4* sp4 = reinterpret_cast<const float4*>(sc + kHalf + kCols * block + 32 * c);
                        const uint64_t f2 = pack_f32x2(fq, fq);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float4 s4 = sp4[j];
                            add_scaled2(v + 4 * j, mul_f32x2(f2, pack_f32x2(s4.x, s4.y)), o + 4 * j);
                            add_scaled2(v + 4 * j + 2, mul_f32x2(f2, pack_f32x2(s4.z, s4.w)), o + 4 * j + 2);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = fmaf(__uint_as_float(v[j]), fq, o[j]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(sempty(slot));
                if (++slot == kSlots) {
                    slot = 0;
                    sphase ^= 1u;
                }
                if (++buf == NB) {
                    buf = 0;
                    bphase ^= 1u;
                }
            }
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            int64_t q0, p0;
            tile_origin(a, TP, tile, q0, p0);
            q0 += kHalf * static_cast<int>(rank) + 32 * quarter;
            p0 += kCols * block;
            if (a.d.out_bf16)
                store_rows<__nv_bfloat16, kCols>(a.d, q0, p0, acc, turn, lane);
            else
                store_rows<float, kCols>(a.d, q0, p0, acc, turn, lane);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) st_shared_cluster(mapa_shared(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u), 1);
    cluster_sync_all();  // no CTA leaves while its peer may still signal its barriers
    if (*abort_flag) {
        // A role of either CTA gave up, and every role of both has ended, with loads and MMAs possibly
        // in flight.  Both CTAs' loads are counted on the even one's barriers, which expect both: a
        // stage that only one of them has filled (neither is ahead by more than one round of a stage,
        // which takes the MMAs of the round before) is made up for.
        if (leader && warp == kWarpTma) {
            const int mine = *issued_loads;
            const int peer = ld_shared_cluster(mapa_shared(smem_u32(const_cast<int*>(issued_loads)), 1));
            for (int s = 0; s < ST; ++s) {
                const int fills = fills_of(mine, ST, s), other = fills_of(peer, ST, s);
                if (lane == 0 && fills > other) mbar_complete_tx(full(s), C::kQBytes + C::kPBytes);
                if (lane == 0 && fills < other) mbar_arrive_expect_tx(full(s), C::kQBytes + C::kPBytes);
                __syncwarp();
                const int rounds = fills > other ? fills : other;
                if (rounds > 0) drain_wait(full(s), static_cast<uint32_t>((rounds - 1) & 1));
            }
        } else if (leader && warp == kWarpMma) {
            if (elect_one()) tc_commit_pair_multicast(drain_bar, 0x1);
            __syncwarp();
            drain_wait(drain_bar, 0);
        }
        __syncthreads();
        cluster_sync_all();
    }
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
    if (threadIdx.x == 0 && *abort_flag && a.d.err != nullptr) atomicOr(a.d.err, kErrBitTimeout);
}

template <bool ROWS, int TP>
cudaError_t launch(const Fp8Product& d, int sms, cudaStream_t stream) {
    using C = Cfg<TP>;
    const int64_t tiles_q = (d.Q + kTileQ - 1) / kTileQ, tiles_p = (d.P + TP - 1) / TP;
    // tile numbers are 32-bit, with room for one more step of the grid
    if (tiles_q * tiles_p >= (int64_t(1) << 30)) return cudaErrorInvalidValue;
    CUtensorMap tq, tp;
    const uint64_t pitch = static_cast<uint64_t>(fp8_row_bytes(d.C));
    if (!encode_tmap_u8_pitch(&tq, d.q, static_cast<uint64_t>(d.C), static_cast<uint64_t>(d.Q), pitch, kG, kHalf) ||
        !encode_tmap_u8_pitch(&tp, d.p, static_cast<uint64_t>(d.C), static_cast<uint64_t>(d.P), pitch, kG, TP / 2))
        return cudaErrorInvalidValue;
    static PerContextOnce attr;
    cudaError_t e = attr.run([] {
        // the split of the registers takes all that the block is launched with
        cudaFuncAttributes f;
        const cudaError_t e = cudaFuncGetAttributes(&f, fp8_gemm2_kernel<ROWS, TP>);
        if (e != cudaSuccess) return e;
        if (f.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
        return cudaFuncSetAttribute(fp8_gemm2_kernel<ROWS, TP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    C::kSmemBytes);
    });
    if (e != cudaSuccess) return e;
    const WaitTest wt = wait_test();
    const Args a{d, static_cast<int>((d.C + kG - 1) / kG), static_cast<int>(tiles_q), static_cast<int>(tiles_p),
                 static_cast<int>(tiles_q * tiles_p), wt.wait_ns, wt.stall_after};
    const int pairs = a.num_tiles < sms / 2 ? a.num_tiles : sms / 2;
    return launch_pdl(fp8_gemm2_kernel<ROWS, TP>, dim3(static_cast<unsigned>(2 * pairs)), dim3(kThreads),
                      C::kSmemBytes, stream, dim3(2, 1, 1), tq, tp, a);
}

}  // namespace

cudaError_t launch_fp8_product_pair(const Fp8Product& d, int tile_p, int sms, cudaStream_t stream) {
    if (tile_p == 256)
        return d.p_shift == 0 ? launch<true, 256>(d, sms, stream) : launch<false, 256>(d, sms, stream);
    return d.p_shift == 0 ? launch<true, 128>(d, sms, stream) : launch<false, 128>(d, sms, stream);
}

}  // namespace bl
