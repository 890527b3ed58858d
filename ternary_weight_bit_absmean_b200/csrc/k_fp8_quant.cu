// k_fp8_quant.cu -- e4m3 codes with one fp32 scale for each block of 128, the operands of
// the 8-bit floating-point product (k_fp8_gemm.cu) for layers that are left unternarised.
// Scaling by the largest magnitude to the largest code, without a zero point, as the int8
// quantiser does ("1-bit & Ternary LLMs", block "BitNet (Oct 2023)").
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
__device__ __forceinline__ uint32_t keep(uint32_t codes, int n) {
    return n >= 4 ? codes : n <= 0 ? 0u : codes & ((1u << (8 * n)) - 1u);
}

// Elements k .. k+3 of a row of K as they lie in memory, zeros past its end (all bits zero is a
// zero in either type).  Loading and converting are apart so that a thread's loads are all on
// their way before the first is needed: load() of every group, then settle() of every group,
// then the values.  VEC: K % 4 == 0 (k is), so the four are there or not together and lie on
// their own alignment.  In other rows four fp32 loads of neighbouring lanes still fill whole
// lines (8191 x 4099: 28 us, 92 % of the copy rate).  In bf16 there are twice as many loads to a
// byte: there the two aligned groups of four around the four are loaded and the four cut out of
// them (tiles of 4095 x 4099 both ways 33 -> 25 us, weights 28.5 -> 21, rows of 8191 x 4099
// 33 -> 31).
template <typename T, bool VEC>
struct Raw4;
template <bool VEC>
struct Raw4<float, VEC> {
    float4 a;
    __device__ __forceinline__ void load(const float* row, int k, int K, const float*) {
        a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if constexpr (VEC) {
            if (k < K) a = __ldg(reinterpret_cast<const float4*>(row + k));
        } else {
            if (k < K) a.x = __ldg(row + k);
            if (k + 1 < K) a.y = __ldg(row + k + 1);
            if (k + 2 < K) a.z = __ldg(row + k + 2);
            if (k + 3 < K) a.w = __ldg(row + k + 3);
        }
    }
    __device__ __forceinline__ void settle(const float*, int, int) {}
    __device__ __forceinline__ float value(int j) const { return j == 0 ? a.x : j == 1 ? a.y : j == 2 ? a.z : a.w; }
    __device__ __forceinline__ void values(float (&v)[4]) const { v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w; }
};
template <>
struct Raw4<__nv_bfloat16, true> {
    uint16_t h[4];
    __device__ __forceinline__ void load(const __nv_bfloat16* row, int k, int K, const __nv_bfloat16*) {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(row + k);
        uint2 a = make_uint2(0u, 0u);
        if (k < K) a = __ldg(reinterpret_cast<const uint2*>(p));
        *reinterpret_cast<uint2*>(h) = a;
    }
    __device__ __forceinline__ void settle(const __nv_bfloat16*, int, int) {}
    __device__ __forceinline__ float value(int j) const {
        return __uint_as_float(static_cast<uint32_t>(h[j]) << 16);
    }
    __device__ __forceinline__ void values(float (&v)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = value(i);
    }
};
template <>
struct Raw4<__nv_bfloat16, false> {
    uint2 a, b;  // b: the group behind a's, until settle()
    __device__ __forceinline__ static int offset(const __nv_bfloat16* p) {
        return static_cast<int>(reinterpret_cast<uintptr_t>(p) >> 1) & 3;
    }
    // `end` is the end of the matrix, which may lie inside an aligned group
    __device__ __forceinline__ void load(const __nv_bfloat16* row, int k, int K, const __nv_bfloat16* end) {
        a = b = make_uint2(0u, 0u);
        if (k >= K) return;
        const uint16_t* at = reinterpret_cast<const uint16_t*>(row + k) - offset(row + k);
        if (at + 8 <= reinterpret_cast<const uint16_t*>(end)) {
            a = __ldg(reinterpret_cast<const uint2*>(at));
            b = __ldg(reinterpret_cast<const uint2*>(at) + 1);
        } else {
            const int there = static_cast<int>(reinterpret_cast<const uint16_t*>(end) - at);
            auto get = [&](int i) { return i < there ? static_cast<uint32_t>(__ldg(at + i)) << (16 * (i & 1)) : 0u; };
            a = make_uint2(get(0) | get(1), get(2) | get(3));
            b = make_uint2(get(4) | get(5), get(6) | get(7));
        }
    }
    __device__ __forceinline__ void settle(const __nv_bfloat16* row, int k, int K) {
        const int off = offset(row + k), n = K - k;
        uint32_t third = b.x;
        if (off & 2) a = make_uint2(a.y, b.x), third = b.y;
        if (off & 1) a = make_uint2(__funnelshift_r(a.x, a.y, 16), __funnelshift_r(a.y, third, 16));
        if (n < 4) a.y &= n < 3 ? 0u : 0xFFFFu;
        if (n < 2) a.x &= n < 1 ? 0u : 0xFFFFu;
    }
    __device__ __forceinline__ float value(int j) const {
        const uint32_t w = j < 2 ? a.x : a.y;
        return __uint_as_float((j & 1) ? (w & 0xFFFF0000u) : (w << 16));
    }
    __device__ __forceinline__ void values(float (&v)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = value(i);
    }
};

__device__ __forceinline__ float absmax4(const float (&v)[4]) {
    return max_nan(max_nan(fabsf(v[0]), fabsf(v[1])), max_nan(fabsf(v[2]), fabsf(v[3])));
}

// ------------------------------------------------------------------ rows alone --
// A warp takes kU groups, four elements a lane (a load is a whole group: 256 or 512
// neighbouring bytes, a store 128): 2^LG neighbouring groups of each of kU / 2^LG rows.  The
// two quotients of a scale cost more instructions than the rest of its group, so lane u
// computes those of group u for the whole warp.
constexpr int kU = 8;
constexpr int kRowWarps = 8;

template <typename T, bool VEC, int LG>
__global__ void __launch_bounds__(32 * kRowWarps, sizeof(T) == 4 || VEC ? 5 : 4)
    fp8_quant_rows_kernel(const T* __restrict__ X, int64_t M, int64_t K, int64_t pitch, float eps,
                          uint8_t* __restrict__ q, float* __restrict__ s, uint32_t spans) {
    pdl_wait_then_release();
    constexpr int kAcross = 1 << LG, kRows = kU >> LG;
    const int lane = threadIdx.x;
    // warps: `spans` of them side by side cover a row
    const uint32_t warp = blockIdx.x * kRowWarps + threadIdx.y;
    const int64_t m0 = static_cast<int64_t>(warp / spans) * kRows;
    const int64_t g0 = static_cast<int64_t>(warp % spans) * kAcross;
    if (m0 >= M) return;
    const int rows = M - m0 < kRows ? static_cast<int>(M - m0) : kRows;
    // what is left of a row from the warp's first group on, at most a span and a bit
    const int64_t rest = K - g0 * kG;
    const int n = rest < 2 * kAcross * kG ? static_cast<int>(rest) : 2 * kAcross * kG;
    const T* x0 = X + m0 * K + g0 * kG;
    Raw4<T, VEC> x[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
        x[u].load(x0 + (u / kAcross) * K, u % kAcross * kG + 4 * lane, u / kAcross < rows ? n : 0, X + M * K);
#pragma unroll
    for (int u = 0; u < kU; ++u)
        x[u].settle(x0 + (u / kAcross) * K, u % kAcross * kG + 4 * lane, u / kAcross < rows ? n : 0);
    float absmax = 0.0f;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        float v[4];
        x[u].values(v);
        const float m = warp_absmax(absmax4(v));
        if (lane == u) absmax = m;
    }
    const Scale mine = scale_of(absmax, eps);
    if (lane < kU && lane / kAcross < rows && lane % kAcross * kG < n)
        s[(g0 + lane % kAcross) * M + m0 + lane / kAcross] = mine.d;
    uint8_t* q0 = q + m0 * pitch + g0 * kG + 4 * lane;
    const int room = n + static_cast<int>(pitch - K);  // with the row's padding
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const float ratio = __shfl_sync(0xFFFFFFFFu, mine.ratio, u);
        const int k = u % kAcross * kG + 4 * lane;
        float v[4];
        x[u].values(v);
        if (u / kAcross < rows && k < room)
            *reinterpret_cast<uint32_t*>(q0 + (u / kAcross) * pitch + u % kAcross * kG) =
                keep(codes4(v, ratio), n - k);
    }
}

// ----------------------------------------------------------- 128 x 128 tiles --
// 16 warps hold a tile in registers: warp w rows 8 w .. 8 w + 7, lane l columns 4 l .. 4 l + 3
// (a load is a whole row of the tile).  Row groups are reduced inside a warp, column groups
// and blocks over the warps through shared memory.  Transposed codes are turned in shared
// memory (a thread's eight rows of a column are eight neighbouring bytes there; the sixteen
// eight-byte units of a column are swizzled by the lane that writes them, so that neither
// side has bank conflicts) and leave as 16-byte pieces of 128-byte runs.
constexpr int kTileWarps = 16;

struct TileArgs {
    int64_t M, K, tiles_k;
    int64_t pitch, pitch_t;
    float eps;
    uint8_t* q;    // [M, pitch] or NULL
    uint8_t* qt;   // [K, pitch_t] or NULL
    float* s;      // rows: [groups of K, M]; blocks: [row blocks, column blocks]
    float* st;     // columns: [groups of M, K]
};

// Three resident blocks for bf16 (8192 x 8192 weights in both orientations: 59.5 -> 55.0 us with
// them); the fp32 values take too many registers for that.
template <typename T, bool VEC, bool BLOCKS>
__global__ void __launch_bounds__(32 * kTileWarps, sizeof(T) == 2 && VEC ? 3 : 2)
    fp8_quant_tile_kernel(const T* __restrict__ X, const TileArgs a) {
    __shared__ float colmax[kTileWarps][kG];
    __shared__ float blockmax[kTileWarps];
    __shared__ __align__(16) uint8_t turn[kG * kG];
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t tm = blockIdx.x / a.tiles_k, tk = blockIdx.x % a.tiles_k;
    const int64_t m0 = tm * kG + 8 * warp, k0 = tk * kG + 4 * lane;
    // rows and columns of the matrix from this thread's first on, at most the tile's
    const int rows = a.M - m0 < 8 ? static_cast<int>(a.M - m0) : 8;
    const int cols = a.K - tk * kG < kG ? static_cast<int>(a.K - tk * kG) : kG;
    const T* x0 = X + m0 * a.K + tk * kG;
    Raw4<T, VEC> x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i].load(x0 + i * a.K, 4 * lane, i < rows ? cols : 0, X + a.M * a.K);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i].settle(x0 + i * a.K, 4 * lane, i < rows ? cols : 0);
    Scale sc[4];  // of this thread's columns (or of the block, four times)
    if constexpr (BLOCKS) {
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v[4];
            x[i].values(v);
            mx = max_nan(mx, absmax4(v));
        }
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
        for (int i = 0; i < 8; ++i) {
            float v[4];
            x[i].values(v);
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] = max_nan(c[j], fabsf(v[j]));
        }
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
        Scale mine = sc[0];
        if constexpr (!BLOCKS) {  // lane i computes the scale of row i for the warp
            float absmax = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float v[4];
                x[i].values(v);
                const float m = warp_absmax(absmax4(v));
                if (lane == i) absmax = m;
            }
            mine = scale_of(absmax, a.eps);
            if (lane < 8 && lane < rows) a.s[tk * a.M + m0 + lane] = mine.d;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float ratio = BLOCKS ? mine.ratio : __shfl_sync(0xFFFFFFFFu, mine.ratio, i);
            // the last group's codes are padded with zeros to the pitch
            float v[4];
            x[i].values(v);
            if (i < rows && k0 < a.pitch)
                *reinterpret_cast<uint32_t*>(a.q + (m0 + i) * a.pitch + k0) = keep(codes4(v, ratio), cols - 4 * lane);
        }
    }
    if (a.qt == nullptr) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float lo[4] = {x[0].value(j), x[1].value(j), x[2].value(j), x[3].value(j)};
        const float hi[4] = {x[4].value(j), x[5].value(j), x[6].value(j), x[7].value(j)};
        *reinterpret_cast<uint2*>(turn + (4 * lane + j) * kG + 8 * (warp ^ (lane & 15))) =
            make_uint2(keep(codes4(lo, sc[j].ratio), rows), keep(codes4(hi, sc[j].ratio), rows - 4));
    }
    __syncthreads();
#pragma unroll
    for (int p = threadIdx.x; p < kG * kG / 16; p += 32 * kTileWarps) {
        const int c = p / (kG / 16), piece = p % (kG / 16);
        const int64_t k = tk * kG + c, m = tm * kG + 16 * piece;
        const int swizzle = (c >> 2) & 15;  // of the lane that wrote the column
        const uint4 u = *reinterpret_cast<const uint4*>(turn + c * kG + 16 * (piece ^ (swizzle >> 1)));
        if (k < a.K && m < a.pitch_t)
            *reinterpret_cast<uint4*>(a.qt + k * a.pitch_t + m) =
                (swizzle & 1) ? make_uint4(u.z, u.w, u.x, u.y) : u;
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
    int lg = 0;  // groups of a row that a warp takes: 1, 2, 4 or 8
    while (lg < 3 && (int64_t(1) << lg) < G) ++lg;
    const int64_t spans = (G + (1 << lg) - 1) >> lg;
    const int64_t rows = int64_t(kU) >> lg;
    const int64_t blocks = ((M + rows - 1) / rows * spans + kRowWarps - 1) / kRowWarps;
    if (blocks >= (int64_t(1) << 28)) return cudaErrorInvalidValue;  // 32-bit warp numbers
    const dim3 grid(static_cast<unsigned>(blocks)), block(32, kRowWarps);
    const int64_t pitch = fp8_row_bytes(K);
    auto run = [&](auto kernel) {
        return launch_pdl(kernel, grid, block, 0, stream, dim3(kNoCluster), X, M, K, pitch, eps, q, s,
                          static_cast<uint32_t>(spans));
    };
    const bool vec = K % 4 == 0;
    switch (lg) {
        case 0: return vec ? run(fp8_quant_rows_kernel<T, true, 0>) : run(fp8_quant_rows_kernel<T, false, 0>);
        case 1: return vec ? run(fp8_quant_rows_kernel<T, true, 1>) : run(fp8_quant_rows_kernel<T, false, 1>);
        case 2: return vec ? run(fp8_quant_rows_kernel<T, true, 2>) : run(fp8_quant_rows_kernel<T, false, 2>);
        default: return vec ? run(fp8_quant_rows_kernel<T, true, 3>) : run(fp8_quant_rows_kernel<T, false, 3>);
    }
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
