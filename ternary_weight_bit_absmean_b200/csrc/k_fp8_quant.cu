// k_fp8_quant.cu -- e4m3 codes with one fp32 scale for each block of 128, the operands of
// the 8-bit floating-point product (k_fp8_gemm.cu) for layers that are left unternarised
// ("1.58 bits: what BitNet promised and what it required": not every matrix of a b1.58
// model is ternary; "1-bit & Ternary LLMs", block "BitNet (Oct 2023)": absmax scaling to
// the largest code, no zero point).
//
//   a = max |x| over the block (a NaN stays one),  m = max(a, eps)
//   d = m / 448,   code = e4m3(x * (448 / m))      (IEEE fp32 quotients and product, then
//                                                   one rounding to nearest even)
// A block is 128 elements of a row (activations), 128 elements of a column (the same
// activations as the operand of a product over tokens, codes transposed), or 128 x 128
// (weights, codes in either or both orientations).  A block that holds an infinity or a
// NaN reads back as NaN: its scale or its codes are NaN.
//
// Bound by memory: every element is read once and leaves as one byte per orientation.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "bl_device.cuh"
#include "bl_internal.h"

namespace bl {
namespace {

constexpr int kG = 128;         // elements of a group, rows and columns of a block
constexpr float kTop = 448.0f;  // largest finite e4m3 value

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// max |v| over the warp, NaN if any lane holds one.
__device__ __forceinline__ float warp_absmax(float v) {
    float r;
    asm volatile("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

struct Scale {
    float d, ratio;  // what a code stands for, and its inverse
};
__device__ __forceinline__ Scale scale_of(float absmax, float eps) {
    const float m = max_nan(absmax, eps);
    return Scale{__fdiv_rn(m, kTop), __fdiv_rn(kTop, m)};
}

// Four codes, the first in the lowest byte.
__device__ __forceinline__ uint32_t codes4(const float (&v)[4], float ratio) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v[0], ratio), __fmul_rn(v[1], ratio)),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v[2], ratio), __fmul_rn(v[3], ratio)),
                                                 __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// The first n of four codes; the others (the padding behind a row's end) are zero whatever
// the block's scale.
__device__ __forceinline__ uint32_t keep(uint32_t codes, int64_t n) {
    return n >= 4 ? codes : n <= 0 ? 0u : codes & ((1u << (8 * static_cast<int>(n))) - 1u);
}

// Elements k .. k+3 of a row of K, zeros past its end.  VEC: K % 4 == 0 (k is), so the four
// are there or not together and lie on their own alignment.
template <bool VEC>
__device__ __forceinline__ void load4(const float* row, int64_t k, int64_t K, float (&v)[4]) {
    if constexpr (VEC) {
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (k < K) a = __ldg(reinterpret_cast<const float4*>(row + k));
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = k + i < K ? __ldg(row + k + i) : 0.0f;
    }
}
template <bool VEC>
__device__ __forceinline__ void load4(const __nv_bfloat16* row, int64_t k, int64_t K, float (&v)[4]) {
    if constexpr (VEC) {
        uint2 a = make_uint2(0u, 0u);
        if (k < K) a = __ldg(reinterpret_cast<const uint2*>(row + k));
        v[0] = __uint_as_float(a.x << 16), v[1] = __uint_as_float(a.x & 0xFFFF0000u);
        v[2] = __uint_as_float(a.y << 16), v[3] = __uint_as_float(a.y & 0xFFFF0000u);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = k + i < K ? __bfloat162float(row[k + i]) : 0.0f;
    }
}

__device__ __forceinline__ float absmax4(const float (&v)[4]) {
    return max_nan(max_nan(fabsf(v[0]), fabsf(v[1])), max_nan(fabsf(v[2]), fabsf(v[3])));
}

// ------------------------------------------------------------------ rows alone --
// One warp per group of 128, four elements a lane (a warp's load is the whole group:
// 256 or 512 neighbouring bytes, its store 128); four groups in flight per warp.
constexpr int kU = 4;
constexpr int kRowWarps = 8;

template <typename T, bool VEC>
__global__ void __launch_bounds__(32 * kRowWarps)
    fp8_quant_rows_kernel(const T* __restrict__ X, int64_t M, int64_t K, int64_t pitch, float eps,
                          uint8_t* __restrict__ q, float* __restrict__ s, int warps_per_row) {
    pdl_wait_then_release();
    const int lane = threadIdx.x;
    const int rows = kRowWarps / warps_per_row;
    const int64_t m = static_cast<int64_t>(blockIdx.x) * rows + threadIdx.y / warps_per_row;
    if (m >= M) return;
    const int64_t G = (K + kG - 1) / kG;
    const T* row = X + m * K;
    for (int64_t g0 = (static_cast<int64_t>(blockIdx.y) * warps_per_row + threadIdx.y % warps_per_row) * kU; g0 < G;
         g0 += static_cast<int64_t>(gridDim.y) * warps_per_row * kU) {
        float v[kU][4];
#pragma unroll
        for (int u = 0; u < kU; ++u) load4<VEC>(row, (g0 + u) * kG + 4 * lane, K, v[u]);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t g = g0 + u;
            if (g >= G) break;
            const Scale sc = scale_of(warp_absmax(absmax4(v[u])), eps);
            const int64_t k = g * kG + 4 * lane;
            if (k < pitch) *reinterpret_cast<uint32_t*>(q + m * pitch + k) = keep(codes4(v[u], sc.ratio), K - k);
            if (lane == 0) s[g * M + m] = sc.d;
        }
    }
}

// ----------------------------------------------------------- 128 x 128 tiles --
// 16 warps hold a tile in registers: warp w rows 8 w .. 8 w + 7, lane l columns 4 l .. 4 l + 3
// (a load is a whole row of the tile).  Row groups are reduced inside a warp, column groups
// and blocks over the warps through shared memory.  Transposed codes are turned in shared
// memory (a thread's eight rows of a column are eight neighbouring bytes there) and leave
// as 16-byte pieces of 128-byte runs.
constexpr int kTileWarps = 16;
constexpr int kTPitch = kG + 16;  // bytes of a column's codes in shared memory

struct TileArgs {
    int64_t M, K, tiles_k;
    int64_t pitch, pitch_t;
    float eps;
    uint8_t* q;    // [M, pitch] or NULL
    uint8_t* qt;   // [K, pitch_t] or NULL
    float* s;      // rows: [groups of K, M]; blocks: [row blocks, column blocks]
    float* st;     // columns: [groups of M, K]
};

template <typename T, bool VEC, bool BLOCKS>
__global__ void __launch_bounds__(32 * kTileWarps)
    fp8_quant_tile_kernel(const T* __restrict__ X, const TileArgs a) {
    __shared__ float colmax[kTileWarps][kG];
    __shared__ float blockmax[kTileWarps];
    __shared__ __align__(16) uint8_t turn[kG * kTPitch];
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t tm = blockIdx.x / a.tiles_k, tk = blockIdx.x % a.tiles_k;
    const int64_t m0 = tm * kG + 8 * warp, k0 = tk * kG + 4 * lane;
    float v[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (m0 + i < a.M) {
            load4<VEC>(X + (m0 + i) * a.K, k0, a.K, v[i]);
        } else {
            v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.0f;
        }
    }
    Scale sc[4];  // of this thread's columns (or of the block, four times)
    if constexpr (BLOCKS) {
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = max_nan(mx, absmax4(v[i]));
        mx = warp_absmax(mx);
        if (lane == 0) blockmax[warp] = mx;
        __syncthreads();
        const Scale b = scale_of(warp_absmax(blockmax[lane & (kTileWarps - 1)]), a.eps);
        if (threadIdx.x == 0) a.s[tm * a.tiles_k + tk] = b.d;
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[j] = b;
    } else if (a.qt != nullptr) {
        float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] = max_nan(c[j], fabsf(v[i][j]));
        *reinterpret_cast<float4*>(&colmax[warp][4 * lane]) = make_float4(c[0], c[1], c[2], c[3]);
        __syncthreads();
        if (threadIdx.x < kG) {
            float mx = colmax[0][threadIdx.x];
#pragma unroll
            for (int w = 1; w < kTileWarps; ++w) mx = max_nan(mx, colmax[w][threadIdx.x]);
            const int64_t k = tk * kG + threadIdx.x;
            const Scale t = scale_of(mx, a.eps);
            if (k < a.K) a.st[tm * a.K + k] = t.d;
            colmax[0][threadIdx.x] = t.ratio;  // column threadIdx.x is this thread's alone
        }
        __syncthreads();
        const float4 r = *reinterpret_cast<const float4*>(&colmax[0][4 * lane]);
        sc[0].ratio = r.x, sc[1].ratio = r.y, sc[2].ratio = r.z, sc[3].ratio = r.w;
    }
    if (a.q != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (m0 + i >= a.M) break;
            float ratio = sc[0].ratio;
            if constexpr (!BLOCKS) {
                const Scale r = scale_of(warp_absmax(absmax4(v[i])), a.eps);
                ratio = r.ratio;
                if (lane == 0) a.s[tk * a.M + m0 + i] = r.d;
            }
            // the last group's codes are padded with zeros to the pitch
            if (k0 < a.pitch)
                *reinterpret_cast<uint32_t*>(a.q + (m0 + i) * a.pitch + k0) = keep(codes4(v[i], ratio), a.K - k0);
        }
    }
    if (a.qt == nullptr) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float lo[4] = {v[0][j], v[1][j], v[2][j], v[3][j]}, hi[4] = {v[4][j], v[5][j], v[6][j], v[7][j]};
        *reinterpret_cast<uint2*>(turn + (4 * lane + j) * kTPitch + 8 * warp) =
            make_uint2(keep(codes4(lo, sc[j].ratio), a.M - m0), keep(codes4(hi, sc[j].ratio), a.M - m0 - 4));
    }
    __syncthreads();
#pragma unroll
    for (int p = threadIdx.x; p < kG * kG / 16; p += 32 * kTileWarps) {
        const int c = p / (kG / 16), piece = p % (kG / 16);
        const int64_t k = tk * kG + c, m = tm * kG + 16 * piece;
        if (k < a.K && m < a.pitch_t)
            *reinterpret_cast<uint4*>(a.qt + k * a.pitch_t + m) =
                *reinterpret_cast<const uint4*>(turn + c * kTPitch + 16 * piece);
    }
}

template <typename T, bool BLOCKS>
cudaError_t launch_tiles(const T* X, const TileArgs& a, cudaStream_t stream) {
    const int64_t tiles = (a.M + kG - 1) / kG * a.tiles_k;
    if (tiles >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(tiles)), block(32 * kTileWarps);
    return a.K % 4 == 0
               ? launch_pdl(fp8_quant_tile_kernel<T, true, BLOCKS>, grid, block, 0, stream, dim3(kNoCluster), X, a)
               : launch_pdl(fp8_quant_tile_kernel<T, false, BLOCKS>, grid, block, 0, stream, dim3(kNoCluster), X, a);
}

template <typename T>
cudaError_t launch_rows(const T* X, int64_t M, int64_t K, float eps, uint8_t* q, float* s, cudaStream_t stream) {
    const int64_t G = (K + kG - 1) / kG;
    int wpr = 1;
    while (wpr < kRowWarps && static_cast<int64_t>(wpr) * kU < G) wpr *= 2;
    const int rows = kRowWarps / wpr;
    const int64_t y = (G + wpr * kU - 1) / (wpr * kU);
    const dim3 grid(static_cast<unsigned>((M + rows - 1) / rows), static_cast<unsigned>(y < 65535 ? y : 65535));
    const dim3 block(32, kRowWarps);
    const int64_t pitch = fp8_row_bytes(K);
    return K % 4 == 0 ? launch_pdl(fp8_quant_rows_kernel<T, true>, grid, block, 0, stream, dim3(kNoCluster), X, M, K,
                                   pitch, eps, q, s, wpr)
                      : launch_pdl(fp8_quant_rows_kernel<T, false>, grid, block, 0, stream, dim3(kNoCluster), X, M, K,
                                   pitch, eps, q, s, wpr);
}

}  // namespace

int64_t fp8_row_bytes(int64_t K) { return (K + 15) / 16 * 16; }

cudaError_t launch_fp8_quantize_act(const void* X, bool x_bf16, int64_t M, int64_t K, float eps, uint8_t* q, float* s,
                                    uint8_t* qt, float* st, cudaStream_t stream) {
    if (qt == nullptr)
        return x_bf16 ? launch_rows(static_cast<const __nv_bfloat16*>(X), M, K, eps, q, s, stream)
                      : launch_rows(static_cast<const float*>(X), M, K, eps, q, s, stream);
    const TileArgs a{M, K, (K + kG - 1) / kG, fp8_row_bytes(K), fp8_row_bytes(M), eps, q, qt, s, st};
    return x_bf16 ? launch_tiles<__nv_bfloat16, false>(static_cast<const __nv_bfloat16*>(X), a, stream)
                  : launch_tiles<float, false>(static_cast<const float*>(X), a, stream);
}

cudaError_t launch_fp8_quantize_weights(const void* W, bool w_bf16, int64_t N, int64_t K, float eps, uint8_t* q,
                                        float* s, uint8_t* qt, cudaStream_t stream) {
    const TileArgs a{N, K, (K + kG - 1) / kG, fp8_row_bytes(K), fp8_row_bytes(N), eps, q, qt, s, nullptr};
    return w_bf16 ? launch_tiles<__nv_bfloat16, true>(static_cast<const __nv_bfloat16*>(W), a, stream)
                  : launch_tiles<float, true>(static_cast<const float*>(W), a, stream);
}

}  // namespace bl
