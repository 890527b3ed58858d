// k_fp8_gemm.cu -- the product of e4m3 matrices with one scale for each block of 128
// (tcgen05.mma kind::f8f6f4, fp32 accumulators in tensor memory), for single tokens up to
// middling batches.  It serves layers left unternarised next to the BitLinear ones, and
// both gradients of such a layer.
//
//   out[q, p] = sum_g sq[g, q] sp(g, p) S_g[q, p],   S_g[q, p] = sum_{c in group g} Qm[q, c] Pm[p, c]
//
// The scales change every 128 elements of the contraction, so the tensor cores sum one
// group (four MMAs of K = 32) into a fresh accumulator, and the epilogue warps read it
// back, multiply by the two scales and add it to fp32 sums in registers, while the tensor
// cores work on the next group in another accumulator.  Products of e4m3 values are exact
// in fp32.
//
// Tile: 128 rows of Pm (MMA M, TMEM lanes) x BQ rows of Qm (MMA N): with one token the
// 128-row weight tiles are what is streamed, and the outputs of a warp are 32 neighbours
// of an output row.  Per group of 128:
//   warp 0             TMA: 128 x 128 bytes of Pm, BQ x 128 bytes of Qm (128-byte swizzle);
//   warp 1             MMA issuer;
//   warp 2             scales: 4-byte asynchronous copies into a ring of eight groups;
//   warps 4 ..         epilogue: a thread owns one row of Pm (its TMEM lane) and a range of
//                      the BQ columns.
// With few tiles the groups are split over the blocks of a cluster, which add their
// partial sums through distributed shared memory in a fixed order.  All waits are bounded
// as in the ternary kernels; a block that gives up (see bl_fp8.cuh) lets its roles run out,
// waits for its loads and MMAs in flight, sets BL_ERRBIT_TIMEOUT and still takes part in the
// cluster barriers.
#include <algorithm>
#include <cmath>
#include <cuda_bf16.h>
#include <cstdint>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "bl_device.cuh"
#include "bl_fp8.cuh"
#include "bl_internal.h"

namespace bl {

bool encode_tmap_u8_pitch(CUtensorMap* map, const void* ptr, uint64_t inner, uint64_t outer, uint64_t pitch,
                          uint32_t box_inner, uint32_t box_outer) {
    struct Encode {
        PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
        Encode() {
            void* p = nullptr;
            cudaDriverEntryPointQueryResult q;
            if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                    cudaSuccess &&
                q == cudaDriverEntryPointSuccess)
                fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        }
    };
    static const Encode encode;  // looked up once (thread-safe static initialisation)
    if (encode.fn == nullptr) return false;
    const cuuint64_t dims[2] = {inner, outer};
    const cuuint64_t strides[1] = {pitch};
    const cuuint32_t box[2] = {box_inner, box_outer};
    const cuuint32_t estr[2] = {1, 1};
    return encode.fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

constexpr int kRows = 128;  // rows of Pm per tile
constexpr int kG = 128;     // contraction elements (bytes) per group and stage
constexpr int kWarpTma = 0, kWarpMma = 1, kWarpScale = 2, kWarpEpi = 4;
constexpr int kScaleSlots = 8;
constexpr int kMaxCluster = 8;

template <int BQ>
struct Cfg {
    static constexpr int kEpiWarps = BQ >= 128 ? 8 : 4;
    static constexpr int kThreads = 32 * (kWarpEpi + kEpiWarps);
    static constexpr int kCols = BQ / (kEpiWarps / 4);  // columns of an epilogue thread
    static constexpr int kQBytes = BQ * kG;
    static constexpr int kPBytes = kRows * kG;
    static constexpr int kStageBytes = kQBytes + kPBytes;
    // tiles of up to 64 rows of Qm leave room for a second block on the SM, whose loads run
    // on while this one starts, reduces and stores
    static constexpr int kStages = BQ >= 128 ? 6 : BQ == 64 ? 4 : 5;
    static constexpr int kBufs = BQ >= 128 ? 2 : 4;  // TMEM accumulators
    static constexpr int kTmemCols = BQ * kBufs;
    static constexpr int kSlotFloats = BQ + kRows;
    static constexpr int kScaleBytes = kScaleSlots * kSlotFloats * 4;
    static constexpr int kBars = 2 * kStages + 2 * kBufs + 2 * kScaleSlots + 1;
    static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kScaleBytes + 8 * kBars + 16;
    static_assert(BQ * kRows * 4 <= kStages * kStageBytes, "partial sums alias the stages");
    static_assert(kTmemCols >= 32 && kTmemCols <= (BQ >= 128 ? 512 : 256), "tensor memory of the resident blocks");
    static_assert(kSmemBytes <= (BQ >= 128 ? 227 : 113) * 1024, "shared memory of the resident blocks");
};

struct Args {
    Fp8Product d;
    int groups;            // of the contraction
    int groups_per_split;  // of a block of the cluster (the last takes the rest)
    int tiles_q;
    unsigned long long wait_ns;  // limit of every wait (2 s outside the bounded-wait test)
    int stall_after;             // the producers stop after this many loads (< 0: never)
};

__device__ __forceinline__ float4 ld_shared_cluster_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// out[q, p .. p + 3].
__device__ __forceinline__ void store_four(const Fp8Product& d, int64_t q, int64_t p, float4 v) {
    if (p >= d.P) return;
    const int64_t at = q * d.P + p;
    if (d.P % 4 == 0) {
        if (d.out_bf16) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(d.out) + at) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
        } else {
            *reinterpret_cast<float4*>(static_cast<float*>(d.out) + at) = v;
        }
        return;
    }
    const float y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (p + i >= d.P) break;
        if (d.out_bf16)
            static_cast<__nv_bfloat16*>(d.out)[at + i] = __float2bfloat16_rn(y[i]);
        else
            static_cast<float*>(d.out)[at + i] = y[i];
    }
}

// grid: x = (tile, block of the cluster), tiles ordered with the Qm tiles of one Pm tile
// next to each other (they read the same Pm rows, from L2 after the first).
template <int BQ>
__global__ void __launch_bounds__(Cfg<BQ>::kThreads, BQ >= 128 ? 1 : 2)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_p,
                    const Args a, const int nsplit) {
    using C = Cfg<BQ>;
    constexpr int ST = C::kStages, NB = C::kBufs;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t sP = base;
    const uint32_t sQ = sP + ST * C::kPBytes;
    const uint32_t sScale = sQ + ST * C::kQBytes;
    const uint32_t sBar = sScale + C::kScaleBytes;
    auto full = [&](int s) { return sBar + 8u * s; };                 // stage landed
    auto empty = [&](int s) { return sBar + 8u * (ST + s); };         // stage read by the MMAs
    auto tfull = [&](int b) { return sBar + 8u * (2 * ST + b); };     // accumulator holds a group
    auto tempty = [&](int b) { return sBar + 8u * (2 * ST + NB + b); };  // accumulator read
    auto sfull = [&](int s) { return sBar + 8u * (2 * ST + 2 * NB + s); };
    auto sempty = [&](int s) { return sBar + 8u * (2 * ST + 2 * NB + kScaleSlots + s); };
    const uint32_t drain_bar = sBar + 8u * (C::kBars - 1);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (sBar - base) + 8 * C::kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    float* scales = reinterpret_cast<float*>(gbase + (sScale - base));
    float* red = reinterpret_cast<float*>(gbase);  // [BQ][128] partial sums, after the main loop

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x % nsplit;
    const int tile = blockIdx.x / nsplit;
    const int64_t p0 = static_cast<int64_t>(tile / a.tiles_q) * kRows;
    const int64_t q0 = static_cast<int64_t>(tile % a.tiles_q) * BQ;
    const int g0 = split * a.groups_per_split;
    const int ng = (split + 1 == nsplit ? a.groups : g0 + a.groups_per_split) - g0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < NB; ++b) {
            mbar_init(tfull(b), 1);
            mbar_init(tempty(b), C::kEpiWarps);
        }
        for (int s = 0; s < kScaleSlots; ++s) {
            mbar_init(sfull(s), 32);
            mbar_init(sempty(s), C::kEpiWarps);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        mbar_fence_init();
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_p);
    }
    pdl_wait_then_release();
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    int issued = 0;  // loads, by the producer's elected lane
    if (warp == kWarpTma) {
        // ---------------------------------------------------------------- producer --
        bool ok = true;
        for (int i = 0; i < ng; ++i) {
            const int stage = i % ST;
            ok &= wait_on(empty(stage), static_cast<uint32_t>(((i / ST) & 1) ^ 1), abort_flag, a.wait_ns);
            if (ok && i == a.stall_after) {  // the bounded-wait test: stop issuing
                stall_until_abort(abort_flag, 4 * a.wait_ns);
                ok = false;
            }
            if (elect_one() && ok) {
                mbar_arrive_expect_tx(full(stage), C::kStageBytes);
                tma_load_2d(sP + stage * C::kPBytes, &tmap_p, full(stage), (g0 + i) * kG, static_cast<int>(p0));
                tma_load_2d(sQ + stage * C::kQBytes, &tmap_q, full(stage), (g0 + i) * kG, static_cast<int>(q0));
                issued = i + 1;
            }
            __syncwarp();
        }
    } else if (warp == kWarpMma) {
        // -------------------------------------------------------------- MMA issuer --
        constexpr uint32_t idesc = idesc_e4m3(kRows, BQ);
        bool ok = true;
        for (int i = 0; i < ng; ++i) {
            const int stage = i % ST, buf = i % NB;
            ok &= wait_on(full(stage), static_cast<uint32_t>((i / ST) & 1), abort_flag, a.wait_ns);
            ok &= wait_on(tempty(buf), static_cast<uint32_t>(((i / NB) & 1) ^ 1), abort_flag, a.wait_ns);
            tc_fence_after();
            if (elect_one() && ok) {
                const uint32_t pa = sP + stage * C::kPBytes, qa = sQ + stage * C::kQBytes;
#pragma unroll
                for (int kk = 0; kk < kG / 32; ++kk)
                    tc_mma_f8(tmem_base + static_cast<uint32_t>(buf * BQ), smem_desc_sw128(pa + 32 * kk),
                              smem_desc_sw128(qa + 32 * kk), idesc, kk != 0 ? 1u : 0u);
                tc_commit(tfull(buf));
                tc_commit(empty(stage));
            }
            __syncwarp();
        }
    } else if (warp == kWarpScale) {
        // -------------------------------------------------------------- scales --
        // rows past an edge take the last row's scale; they are not stored
        for (int i = 0; i < ng; ++i) {
            const int slot = i % kScaleSlots;
            if (!wait_on(sempty(slot), static_cast<uint32_t>(((i / kScaleSlots) & 1) ^ 1), abort_flag, a.wait_ns))
                break;  // a lane alone may: nothing here wants the warp whole
            const uint32_t dst = sScale + static_cast<uint32_t>(slot * C::kSlotFloats * 4);
            const int64_t g = g0 + i;
#pragma unroll
            for (int c = 0; c < BQ; c += 32) {
                const int j = c + lane;
                const int64_t q = q0 + j < a.d.Q ? q0 + j : a.d.Q - 1;
                if (BQ >= 32 || j < BQ) cp_async4(dst + 4u * j, a.d.sq + g * a.d.Q + q);
            }
#pragma unroll
            for (int c = 0; c < kRows; c += 32) {
                const int j = c + lane;
                const int64_t p = p0 + j < a.d.P ? p0 + j : a.d.P - 1;
                cp_async4(dst + 4u * (BQ + j), a.d.sp + (p >> a.d.p_shift) * a.d.sp_p + g * a.d.sp_g);
            }
            cp_async_arrive(sfull(slot));
        }
        cp_async_wait_all();
    } else if (warp >= kWarpEpi) {
        // ------------------------------------------------------------ epilogue --
        const int quarter = warp & 3, c_begin = ((warp - kWarpEpi) >> 2) * C::kCols;
        const int r = 32 * quarter + lane;
        const uint32_t lane_addr = static_cast<uint32_t>(32 * quarter) << 16;
        uint64_t acc[C::kCols / 2];
#pragma unroll
        for (int j = 0; j < C::kCols / 2; ++j) acc[j] = 0;
        bool ok = true;
        for (int i = 0; i < ng; ++i) {
            const int slot = i % kScaleSlots, buf = i % NB;
            ok &= wait_on(sfull(slot), static_cast<uint32_t>((i / kScaleSlots) & 1), abort_flag, a.wait_ns);
            ok &= wait_on(tfull(buf), static_cast<uint32_t>((i / NB) & 1), abort_flag, a.wait_ns);
            __syncwarp();  // the lanes' polls may have ended at different times
            tc_fence_after();
            const float* sc = scales + slot * C::kSlotFloats;
            const uint64_t sp2 = pack_f32x2(sc[BQ + r], sc[BQ + r]);
            constexpr int kW = C::kCols < 32 ? C::kCols : 32;  // columns read at a time
#pragma unroll
            for (int c = 0; c < C::kCols; c += kW) {
                uint32_t v[kW];
                const uint32_t addr = tmem_base + lane_addr + static_cast<uint32_t>(buf * BQ + c_begin + c);
                if constexpr (kW == 32)
                    tmem_ld_32x32b_x32(addr, v);
                else
                    tmem_ld_32x32b_x16(addr, v);
                tmem_ld_wait_for(v);
                if (c + kW == C::kCols) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(tempty(buf));
                }
#pragma unroll
                for (int j = 0; j < kW / 4; ++j) {
                    const float4 s4 = *reinterpret_cast<const float4*>(sc + c_begin + c + 4 * j);
                    uint64_t* o = &acc[c / 2 + 2 * j];
                    o[0] = fma_f32x2(pack_f32x2(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1])),
                                     mul_f32x2(sp2, pack_f32x2(s4.x, s4.y)), o[0]);
                    o[1] = fma_f32x2(pack_f32x2(__uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3])),
                                     mul_f32x2(sp2, pack_f32x2(s4.z, s4.w)), o[1]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(sempty(slot));
        }
        if (__all_sync(0xFFFFFFFFu, ok)) {
            float y[C::kCols];
#pragma unroll
            for (int j = 0; j < C::kCols / 2; ++j) {
                const float2 two = unpack_f32x2(acc[j]);
                y[2 * j] = two.x;
                y[2 * j + 1] = two.y;
            }
            if (nsplit > 1) {
                // every stage of this block has been read (its last group is in the sums), so the
                // partial sums may take the stages' place
#pragma unroll
                for (int j = 0; j < C::kCols; ++j) red[(c_begin + j) * kRows + r] = y[j];
            } else if (p0 + r < a.d.P) {
                const int64_t left = a.d.Q - q0 - c_begin, at = (q0 + c_begin) * a.d.P + p0 + r;
                const int n = left < C::kCols ? static_cast<int>(left) : C::kCols;
                if (a.d.out_bf16) {
                    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.d.out) + at;
#pragma unroll
                    for (int j = 0; j < C::kCols; ++j)
                        if (j < n) o[j * a.d.P] = __float2bfloat16_rn(y[j]);
                } else {
                    float* o = static_cast<float*>(a.d.out) + at;
#pragma unroll
                    for (int j = 0; j < C::kCols; ++j)
                        if (j < n) o[j * a.d.P] = y[j];
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // a role gave up: all have ended, with loads and MMAs possibly in flight
        if (warp == kWarpTma && elect_one()) {
            for (int s = 0; s < ST; ++s) {
                const int fills = fills_of(issued, ST, s);
                if (fills > 0) drain_wait(full(s), static_cast<uint32_t>((fills - 1) & 1));
            }
        } else if (warp == kWarpMma) {
            if (elect_one()) tc_commit(drain_bar);
            __syncwarp();
            drain_wait(drain_bar, 0);
        }
        __syncthreads();
    }
    if (nsplit > 1) {
        // every block's partial sums are in its shared memory: the blocks share out the columns,
        // and a thread adds four neighbouring rows of Pm over the blocks, in their order, with
        // all of its loads from the other blocks on their way together
        cluster_sync_all();
        const int share = (BQ + nsplit - 1) / nsplit;
        const int64_t left = a.d.Q - q0;
        int end = split * share + share;
        if (end > BQ) end = BQ;
        if (end > left) end = static_cast<int>(left);
        const uint32_t red_addr = smem_u32(red);
        for (int u = split * share * (kRows / 4) + static_cast<int>(threadIdx.x); u < end * (kRows / 4);
             u += C::kThreads) {
            float4 v[kMaxCluster];
#pragma unroll
            for (int b = 0; b < kMaxCluster; ++b)
                if (b < nsplit) v[b] = ld_shared_cluster_v4(mapa_shared(red_addr + 16u * u, b));
            float4 sum = v[0];
#pragma unroll
            for (int b = 1; b < kMaxCluster; ++b)
                if (b < nsplit) sum.x += v[b].x, sum.y += v[b].y, sum.z += v[b].z, sum.w += v[b].w;
            store_four(a.d, q0 + u / (kRows / 4), p0 + u % (kRows / 4) * 4, sum);
        }
        // no block leaves while another may still read its shared memory
        cluster_sync_all();
    }
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::kTmemCols);
    }
    if (threadIdx.x == 0 && *abort_flag && a.d.err != nullptr) atomicOr(a.d.err, kErrBitTimeout);
}

int sm_count() {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

template <int BQ>
cudaError_t launch_bq(const Fp8Product& d, int split, cudaStream_t stream) {
    using C = Cfg<BQ>;
    const int64_t tiles_p = (d.P + kRows - 1) / kRows, tiles_q = (d.Q + BQ - 1) / BQ;
    const int groups = static_cast<int>((d.C + kG - 1) / kG);
    const int per = (groups + split - 1) / split;
    split = (groups + per - 1) / per;  // every block has at least one group
    if (tiles_p * tiles_q * split >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    CUtensorMap tq, tp;
    if (!encode_tmap_u8_pitch(&tq, d.q, static_cast<uint64_t>(d.C), static_cast<uint64_t>(d.Q),
                              static_cast<uint64_t>(fp8_row_bytes(d.C)), kG, BQ) ||
        !encode_tmap_u8_pitch(&tp, d.p, static_cast<uint64_t>(d.C), static_cast<uint64_t>(d.P),
                              static_cast<uint64_t>(fp8_row_bytes(d.C)), kG, kRows))
        return cudaErrorInvalidValue;
    static PerContextOnce attr;
    cudaError_t e = attr.run([] {
        return cudaFuncSetAttribute(fp8_gemm_kernel<BQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    });
    if (e != cudaSuccess) return e;
    const WaitTest wt = wait_test();
    const Args a{d, groups, per, static_cast<int>(tiles_q), wt.wait_ns, wt.stall_after};
    return launch_pdl(fp8_gemm_kernel<BQ>, dim3(static_cast<unsigned>(tiles_p * tiles_q * split)), dim3(C::kThreads),
                      C::kSmemBytes, stream, split > 1 ? dim3(static_cast<unsigned>(split), 1, 1) : dim3(kNoCluster),
                      tq, tp, a, split);
}

}  // namespace

// Which kernel runs a product: the one with the least expected time, in microseconds.  The rates
// come from timing both sides of every choice on rows 1 .. 2048 of six weight shapes (512 x 256
// to 28672 x 2048): a block takes `group` per group of 128 as long as neither HBM (6.9 TB/s) nor
// the L2 (9 TB/s into the SMs) limits all of them together, after a fixed time for launch, first
// loads and stores, more when partial sums are joined over a cluster.
namespace {

double time_small(const Fp8Product& d, int bq, int split, int sms) {
    const double groups = static_cast<double>((d.C + kG - 1) / kG);
    const double tiles = static_cast<double>((d.P + kRows - 1) / kRows) * static_cast<double>((d.Q + bq - 1) / bq);
    const double per = std::ceil(groups / split);
    split = static_cast<int>(std::ceil(groups / per));
    const int occupancy = bq >= 128 ? 1 : 2;
    // a cluster's blocks share a GPC, whose SMs larger clusters fill less well
    const double fill = split == 1 ? 1.0 : split <= 4 ? 0.92 : split <= 6 ? 0.845 : 0.757;
    const double waves = std::ceil(tiles * split / std::floor(sms * fill * occupancy));
    const double group = bq <= 32 ? 0.255 : bq == 64 ? 0.30 : 0.32;
    const double fixed = split > 1 ? (bq == 16 ? 3.7 : bq == 32 ? 5.0 : bq == 64 ? 5.7 : 7.0)
                                   : (bq == 16 ? 2.5 : bq == 32 ? 3.2 : bq == 64 ? 4.5 : 5.2);
    // reads of Pm; fewer than one and a half blocks per SM draw about 12% less
    const double hbm = static_cast<double>(d.P) * static_cast<double>(d.C) / (tiles * split < 1.5 * sms ? 6.2e6 : 6.9e6);
    const double l2 = tiles * groups * (bq + kRows) * kG / 9.0e6;
    return fixed + std::max(waves * per * group, std::max(hbm, l2)) + (waves - 1) * (occupancy == 2 ? 2.2 : 5.0);
}

double time_pair(const Fp8Product& d, int tp, int sms) {
    const double groups = static_cast<double>((d.C + kG - 1) / kG);
    const double tiles = static_cast<double>((d.P + tp - 1) / tp) * static_cast<double>((d.Q + 255) / 256);
    const double rounds = std::ceil(tiles / (sms / 2));
    const bool rows = d.p_shift == 0;  // both sides scaled by row: twice the arithmetic per sum
    const double group = tp == 256 ? (rows ? 0.65 : 0.47) : 0.345;
    return (tp == 256 ? 5.8 : 4.5) + rounds * (groups * group + (tp == 256 ? 1.1 : 0.3));
}

}  // namespace

cudaError_t launch_fp8_product(const Fp8Product& d, cudaStream_t stream) {
    const int sms = sm_count();
    const int64_t groups = (d.C + kG - 1) / kG;
    const int bq = d.Q <= 16 ? 16 : d.Q <= 32 ? 32 : d.Q <= 64 ? 64 : 128;
    int split = 1;
    double best = time_small(d, bq, 1, sms);
    for (int s = 2; s <= kMaxCluster && s <= groups; ++s) {
        const double t = time_small(d, bq, s, sms);
        if (t < best) best = t, split = s;
    }
    int tile_p = 0;
    if (d.Q > 64)
        for (int tp = 128; tp <= 256; tp += 128) {
            const double t = time_pair(d, tp, sms);
            if (t < best) best = t, tile_p = tp;
        }
    if (tile_p != 0) return launch_fp8_product_pair(d, tile_p, sms, stream);
    switch (bq) {
        case 16: return launch_bq<16>(d, split, stream);
        case 32: return launch_bq<32>(d, split, stream);
        case 64: return launch_bq<64>(d, split, stream);
        default: return launch_bq<128>(d, split, stream);
    }
}

}  // namespace bl
