// k_norm.cu -- RMSNorm / LayerNorm of a token on their own, forward and backward.
//
// "1-bit & Ternary LLMs", block "BitNet (Oct 2023)": y = W~ . Quant(LN(x)); the training
// pseudocode of the same page quantises LN(x) as well.  The fused norm + quantiser of
// k_quant.cu serves the ternary layers' forward; the kernels here give the normalised
// activations themselves and carry the gradient that the straight-through backward
// leaves at them on to x and to the norm's weight and bias.
//
//   mu = 0 (RMS) or mean_k x;  r = 1 / sqrt(mean_k (x - mu)^2 + eps);  n = (x - mu) r
//   forward    y = n w + b
//   backward   g = dy w;  c1 = mean_k(g n);  c2 = 0 (RMS) or mean_k g
//              dx = r (g - c2 - n c1),  dw = sum_m dy n,  db = sum_m dy
//
// The backward takes mu and r from x again instead of reading saved ones: the row is on
// chip anyway for n.  All sums are fp32: a thread adds its elements in order, the threads
// of a row add in a tree, and the squares are of the already centred values, so a large
// mean costs no digits.
//
// Both are bound by memory (a row is read once, kept in registers, and written once).
// `TPR` threads hold a row, up to CH chunks of eight elements each; short rows share a
// block.  The column sums of the backward stay in the registers of the threads that own
// the columns while a block walks over its rows; they are added over the row groups of a
// block in shared memory and over the blocks by a second kernel, always in the same
// order, so the results do not change from run to run.
#include <cuda_bf16.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "bl_device.cuh"
#include "bl_internal.h"

namespace bl {
namespace {

constexpr int kE = 8;  // elements of a chunk

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// Element e of chunk c of a thread sits at row offset elem<VEC>(c, e): eight neighbours per
// chunk when the rows are 16-byte aligned (K % 8 == 0), else neighbouring threads hold
// neighbouring elements so that single-element accesses still coalesce.
template <bool VEC>
__device__ __forceinline__ int64_t elem(int c, int e, int t, int tpr) {
    const int64_t chunk = static_cast<int64_t>(c) * tpr;
    return VEC ? (chunk + t) * kE + e : (chunk * kE + static_cast<int64_t>(e) * tpr + t);
}

template <bool VEC>
__device__ __forceinline__ void load_chunk(const float* row, int c, int t, int tpr, int64_t K, float (&v)[kE]) {
    if constexpr (VEC) {
        const int64_t k = elem<true>(c, 0, t, tpr);
        if (k < K) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(row + k));
            const float4 b = __ldg(reinterpret_cast<const float4*>(row + k + 4));
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int e = 0; e < kE; ++e) v[e] = 0.0f;
        }
    } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const int64_t k = elem<false>(c, e, t, tpr);
            v[e] = k < K ? __ldg(row + k) : 0.0f;
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void load_chunk(const __nv_bfloat16* row, int c, int t, int tpr, int64_t K,
                                           float (&v)[kE]) {
    if constexpr (VEC) {
        const int64_t k = elem<true>(c, 0, t, tpr);
        uint4 a = make_uint4(0, 0, 0, 0);
        if (k < K) a = __ldg(reinterpret_cast<const uint4*>(row + k));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const int64_t k = elem<false>(c, e, t, tpr);
            v[e] = k < K ? __bfloat162float(row[k]) : 0.0f;
        }
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}

// One chunk of a row of `out` (fp32 or bf16 by `bf16`).
template <bool VEC>
__device__ __forceinline__ void store_chunk(void* out, bool bf16, int64_t row_off, int c, int t, int tpr, int64_t K,
                                            const float (&v)[kE]) {
    if constexpr (VEC) {
        const int64_t k = elem<true>(c, 0, t, tpr);
        if (k >= K) return;
        if (bf16) {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + row_off + k) =
                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        } else {
            float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + row_off + k);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const int64_t k = elem<false>(c, e, t, tpr);
            if (k >= K) continue;
            if (bf16)
                static_cast<__nv_bfloat16*>(out)[row_off + k] = __float2bfloat16_rn(v[e]);
            else
                static_cast<float*>(out)[row_off + k] = v[e];
        }
    }
}

// Sums of two values over the TPR threads of a row (TPR a multiple of 32; the group's
// threads call it together).  `slot` alternates between calls: a slot is written again
// only after the barrier of the call in between, which every reader has then passed.
struct RowSum {
    float2* buf;  // [2][32] of this row group
    int t, tpr, group;
    int slot = 0;
    __device__ __forceinline__ float2 operator()(float a, float b) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        if (tpr == 32) return make_float2(a, b);
        float2* s = buf + 32 * slot;
        slot ^= 1;
        if ((t & 31) == 0) s[t >> 5] = make_float2(a, b);
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
        const float2 v = (t & 31) < (tpr >> 5) ? s[t & 31] : make_float2(0.0f, 0.0f);
        a = v.x, b = v.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        return make_float2(a, b);
    }
};

constexpr int kMaxGroups = 8;   // row groups of a block
constexpr int kMaxThreads = 1024;

struct FwdArgs {
    const float* w;
    const float* b;
    int64_t M, K;
    bool layer;
    float eps, inv_k;
    void* out;
    bool out_bf16;
};

template <typename TX, bool VEC, int CH>
__global__ void __launch_bounds__(kMaxThreads) norm_forward_kernel(const TX* __restrict__ X, const FwdArgs a) {
    __shared__ float2 sums[kMaxGroups][64];
    const int t = threadIdx.x, tpr = blockDim.x, group = threadIdx.y;
    pdl_wait_then_release();
    RowSum row_sum{sums[group], t, tpr, group};
    const int64_t m = static_cast<int64_t>(blockIdx.x) * blockDim.y + group;
    if (m >= a.M) return;  // a whole group leaves together
    const TX* row = X + m * a.K;
    float x[CH][kE];
#pragma unroll
    for (int c = 0; c < CH; ++c) load_chunk<VEC>(row, c, t, tpr, a.K, x[c]);
    float mu = 0.0f;
    if (a.layer) {
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int e = 0; e < kE; ++e) s += x[c][e];
        mu = row_sum(s, 0.0f).x * a.inv_k;
    }
    float v = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            if (elem<VEC>(c, e, t, tpr) < a.K) {
                x[c][e] -= mu;
                v = fmaf(x[c][e], x[c][e], v);
            }
        }
    const float r = 1.0f / sqrtf(row_sum(v, 0.0f).x * a.inv_k + a.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        float w[kE], b[kE];
        if (a.w != nullptr) load_chunk<VEC>(a.w, c, t, tpr, a.K, w);
        if (a.b != nullptr) load_chunk<VEC>(a.b, c, t, tpr, a.K, b);
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            float y = x[c][e] * r;
            if (a.w != nullptr) y *= w[e];
            if (a.b != nullptr) y += b[e];
            x[c][e] = y;
        }
        store_chunk<VEC>(a.out, a.out_bf16, m * a.K, c, t, tpr, a.K, x[c]);
    }
}

// Rows too long for the registers of a block: three passes over the row (it stays in the
// caches between them).
template <typename TX>
__global__ void __launch_bounds__(kMaxThreads) norm_forward_long_kernel(const TX* __restrict__ X, const FwdArgs a) {
    __shared__ float2 sums[64];
    const int t = threadIdx.x, tpr = blockDim.x;
    pdl_wait_then_release();
    RowSum row_sum{sums, t, tpr, 0};
    const int64_t m = blockIdx.x;
    const TX* row = X + m * a.K;
    float mu = 0.0f;
    if (a.layer) {
        float s = 0.0f;
        for (int64_t k = t; k < a.K; k += tpr) s += to_f32(row[k]);
        mu = row_sum(s, 0.0f).x * a.inv_k;
    }
    float v = 0.0f;
    for (int64_t k = t; k < a.K; k += tpr) {
        const float d = to_f32(row[k]) - mu;
        v = fmaf(d, d, v);
    }
    const float r = 1.0f / sqrtf(row_sum(v, 0.0f).x * a.inv_k + a.eps);
    for (int64_t k = t; k < a.K; k += tpr) {
        float y = (to_f32(row[k]) - mu) * r;
        if (a.w != nullptr) y *= __ldg(a.w + k);
        if (a.b != nullptr) y += __ldg(a.b + k);
        if (a.out_bf16)
            static_cast<__nv_bfloat16*>(a.out)[m * a.K + k] = __float2bfloat16_rn(y);
        else
            static_cast<float*>(a.out)[m * a.K + k] = y;
    }
}

struct BwdArgs {
    const float* w;
    int64_t M, K;
    bool layer;
    float eps, inv_k;
    void* dx;
    bool dx_bf16;
    float* dw;  // [gridDim.x, K] partial sums (the result itself with one block), or NULL
    float* db;
};

// One row at a time per group; the group's threads keep the column sums of their columns.
template <typename TX, typename TD, bool VEC, int CH>
__global__ void __launch_bounds__(CH <= 2 ? 512 : 256)
    norm_backward_kernel(const TX* __restrict__ X, const TD* __restrict__ dY, const BwdArgs a) {
    __shared__ float2 sums[kMaxGroups][64];
    extern __shared__ float cols[];  // [2][tpr * CH * kE] column sums of the block's groups
    const int t = threadIdx.x, tpr = blockDim.x, group = threadIdx.y, groups = blockDim.y;
    pdl_wait_then_release();
    RowSum row_sum{sums[group], t, tpr, group};
    float dw[CH][kE], db[CH][kE];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < kE; ++e) dw[c][e] = db[c][e] = 0.0f;

    for (int64_t m = static_cast<int64_t>(blockIdx.x) * groups + group; m < a.M;
         m += static_cast<int64_t>(gridDim.x) * groups) {
        const TX* row = X + m * a.K;
        const TD* drow = dY + m * a.K;
        float x[CH][kE], d[CH][kE];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            load_chunk<VEC>(row, c, t, tpr, a.K, x[c]);
            load_chunk<VEC>(drow, c, t, tpr, a.K, d[c]);
        }
        float mu = 0.0f, c2 = 0.0f;
        if (a.layer) {
            float s = 0.0f, sg = 0.0f;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                float w[kE];
                if (a.w != nullptr) load_chunk<VEC>(a.w, c, t, tpr, a.K, w);
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    s += x[c][e];
                    sg = a.w != nullptr ? fmaf(d[c][e], w[e], sg) : sg + d[c][e];
                }
            }
            const float2 both = row_sum(s, sg);
            mu = both.x * a.inv_k;
            c2 = both.y * a.inv_k;
        }
        float v = 0.0f, gx = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float w[kE];
            if (a.w != nullptr) load_chunk<VEC>(a.w, c, t, tpr, a.K, w);
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                if (elem<VEC>(c, e, t, tpr) < a.K) {
                    x[c][e] -= mu;
                    v = fmaf(x[c][e], x[c][e], v);
                    const float g = a.w != nullptr ? d[c][e] * w[e] : d[c][e];
                    gx = fmaf(g, x[c][e], gx);
                }
            }
        }
        const float2 both = row_sum(v, gx);
        const float r = 1.0f / sqrtf(both.x * a.inv_k + a.eps);
        const float c1 = both.y * a.inv_k * r;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float w[kE], o[kE];
            if (a.w != nullptr) load_chunk<VEC>(a.w, c, t, tpr, a.K, w);
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                const float n = x[c][e] * r;
                const float g = a.w != nullptr ? d[c][e] * w[e] : d[c][e];
                o[e] = r * ((g - c2) - n * c1);
                dw[c][e] = fmaf(d[c][e], n, dw[c][e]);
                db[c][e] += d[c][e];
            }
            store_chunk<VEC>(a.dx, a.dx_bf16, m * a.K, c, t, tpr, a.K, o);
        }
    }
    if (a.dw == nullptr && a.db == nullptr) return;
    // the groups add their column sums in shared memory, one after the other
    const int width = tpr * CH * kE;
    for (int g = 0; g < groups; ++g) {
        if (g == group) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    const int k = (c * kE + e) * tpr + t;
                    if (g == 0) {
                        cols[k] = dw[c][e];
                        cols[width + k] = db[c][e];
                    } else {
                        cols[k] = dw[c][e] += cols[k];
                        cols[width + k] = db[c][e] += cols[width + k];
                    }
                }
        }
        if (g + 1 < groups) __syncthreads();
    }
    if (group + 1 != groups) return;
    const int64_t off = static_cast<int64_t>(blockIdx.x) * a.K;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        // rows of a partial-sum matrix start anywhere: element stores unless K % 8 == 0
        if (a.dw != nullptr) store_chunk<VEC>(a.dw, false, off, c, t, tpr, a.K, dw[c]);
        if (a.db != nullptr) store_chunk<VEC>(a.db, false, off, c, t, tpr, a.K, db[c]);
    }
}

// Rows too long for the registers: dx row by row as in norm_forward_long_kernel, keeping
// (mu, r) of every row for the column kernel below.
template <typename TX, typename TD>
__global__ void __launch_bounds__(kMaxThreads)
    norm_backward_long_kernel(const TX* __restrict__ X, const TD* __restrict__ dY, const BwdArgs a,
                              float2* __restrict__ stats) {
    __shared__ float2 sums[64];
    const int t = threadIdx.x, tpr = blockDim.x;
    pdl_wait_then_release();
    RowSum row_sum{sums, t, tpr, 0};
    const int64_t m = blockIdx.x;
    const TX* row = X + m * a.K;
    const TD* drow = dY + m * a.K;
    auto grad = [&](int64_t k) {
        const float d = to_f32(drow[k]);
        return a.w != nullptr ? d * __ldg(a.w + k) : d;
    };
    float mu = 0.0f, c2 = 0.0f;
    if (a.layer) {
        float s = 0.0f, sg = 0.0f;
        for (int64_t k = t; k < a.K; k += tpr) {
            s += to_f32(row[k]);
            sg += grad(k);
        }
        const float2 both = row_sum(s, sg);
        mu = both.x * a.inv_k;
        c2 = both.y * a.inv_k;
    }
    float v = 0.0f, gx = 0.0f;
    for (int64_t k = t; k < a.K; k += tpr) {
        const float x = to_f32(row[k]) - mu;
        v = fmaf(x, x, v);
        gx = fmaf(grad(k), x, gx);
    }
    const float2 both = row_sum(v, gx);
    const float r = 1.0f / sqrtf(both.x * a.inv_k + a.eps);
    const float c1 = both.y * a.inv_k * r;
    for (int64_t k = t; k < a.K; k += tpr) {
        const float n = (to_f32(row[k]) - mu) * r;
        const float o = r * ((grad(k) - c2) - n * c1);
        if (a.dx_bf16)
            static_cast<__nv_bfloat16*>(a.dx)[m * a.K + k] = __float2bfloat16_rn(o);
        else
            static_cast<float*>(a.dx)[m * a.K + k] = o;
    }
    if (t == 0 && stats != nullptr) stats[m] = make_float2(mu, r);
}

// Column sums of a strip of rows from x, dy and the rows' (mu, r): a thread owns a column.
template <typename TX, typename TD>
__global__ void __launch_bounds__(256)
    norm_columns_long_kernel(const TX* __restrict__ X, const TD* __restrict__ dY, const BwdArgs a,
                             const float2* __restrict__ stats, int64_t rows_per_block) {
    pdl_wait_then_release();
    const int64_t m0 = blockIdx.x * rows_per_block;
    const int64_t m1 = m0 + rows_per_block < a.M ? m0 + rows_per_block : a.M;
    for (int64_t k = blockIdx.y * 256 + threadIdx.x; k < a.K; k += static_cast<int64_t>(gridDim.y) * 256) {
        float dw = 0.0f, db = 0.0f;
#pragma unroll 4
        for (int64_t m = m0; m < m1; ++m) {
            const float2 st = __ldg(stats + m);
            const float d = to_f32(dY[m * a.K + k]);
            dw = fmaf(d, (to_f32(X[m * a.K + k]) - st.x) * st.y, dw);
            db += d;
        }
        if (a.dw != nullptr) a.dw[blockIdx.x * a.K + k] = dw;
        if (a.db != nullptr) a.db[blockIdx.x * a.K + k] = db;
    }
}

// dw and db from the blocks' partial sums: 32 columns a block, 32 strips of partial rows.
__global__ void __launch_bounds__(1024)
    norm_reduce_kernel(const float* __restrict__ pw, const float* __restrict__ pb, int parts, int64_t K, float* dw,
                       float* db) {
    __shared__ float s[32][33];
    pdl_wait_then_release();
    const float* p = blockIdx.y == 0 ? (pw != nullptr ? pw : pb) : pb;
    float* out = blockIdx.y == 0 ? (pw != nullptr ? dw : db) : db;
    const int64_t k = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    float v = 0.0f;
    if (k < K)
        for (int i = threadIdx.y; i < parts; i += 32) v += __ldg(p + i * K + k);
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    v = s[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int64_t ko = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.y;
    if (threadIdx.x == 0 && ko < K) out[ko] = v;
}

// Threads of a row and row groups of a block for rows of K elements in CH chunks a thread.
struct Shape {
    int tpr, groups;
};
Shape shape_of(int64_t K, int ch) {
    const int64_t chunks = (K + kE - 1) / kE;
    const int tpr = static_cast<int>((chunks + ch - 1) / ch + 31) / 32 * 32;
    int groups = 256 / tpr;
    return Shape{tpr, groups < 1 ? 1 : groups > kMaxGroups ? kMaxGroups : groups};
}

constexpr int64_t kFwdMaxK = int64_t(kMaxThreads) * 4 * kE;
constexpr int64_t kBwdMaxK = int64_t(256) * 4 * kE;

// Chunks a thread: one for rows that then still fill a warp group, up to four.
int chunks_of(int64_t K) {
    const int64_t chunks = (K + kE - 1) / kE;
    return chunks <= 128 ? 1 : chunks <= 256 ? 2 : 4;
}

template <typename TX, bool VEC>
cudaError_t forward_t(const TX* X, const FwdArgs& a, cudaStream_t stream) {
    const int ch = chunks_of(a.K);
    const Shape s = shape_of(a.K, ch);
    const dim3 grid(static_cast<unsigned>((a.M + s.groups - 1) / s.groups)), block(s.tpr, s.groups);
    switch (ch) {
        case 1: return launch_pdl(norm_forward_kernel<TX, VEC, 1>, grid, block, 0, stream, dim3(kNoCluster), X, a);
        case 2: return launch_pdl(norm_forward_kernel<TX, VEC, 2>, grid, block, 0, stream, dim3(kNoCluster), X, a);
        default: return launch_pdl(norm_forward_kernel<TX, VEC, 4>, grid, block, 0, stream, dim3(kNoCluster), X, a);
    }
}

template <typename TX>
cudaError_t forward_x(const TX* X, const FwdArgs& a, cudaStream_t stream) {
    if (a.K > kFwdMaxK)
        return launch_pdl(norm_forward_long_kernel<TX>, dim3(static_cast<unsigned>(a.M)), dim3(kMaxThreads), 0, stream,
                          dim3(kNoCluster), X, a);
    return a.K % kE == 0 ? forward_t<TX, true>(X, a, stream) : forward_t<TX, false>(X, a, stream);
}

// Blocks of the backward: each leaves one row of partial column sums.
int backward_blocks(int64_t M, int64_t K) {
    const int64_t per = K <= kBwdMaxK ? shape_of(K, chunks_of(K)).groups : 16;
    const int64_t want = (M + per - 1) / per;
    const int64_t most = 2 * 148;
    return static_cast<int>(want < most ? want : most);
}

template <typename TX, typename TD, bool VEC, int CH>
cudaError_t backward_c(const TX* X, const TD* dY, const BwdArgs& a, cudaStream_t stream) {
    const Shape s = shape_of(a.K, CH);
    const size_t smem = static_cast<size_t>(2) * s.tpr * CH * kE * sizeof(float);
    static PerContextOnce attr;
    cudaError_t e = attr.run([] {
        return cudaFuncSetAttribute(norm_backward_kernel<TX, TD, VEC, CH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(2 * 256 * 4 * kE * sizeof(float)));
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_backward_kernel<TX, TD, VEC, CH>, dim3(backward_blocks(a.M, a.K)), dim3(s.tpr, s.groups),
                      smem, stream, dim3(kNoCluster), X, dY, a);
}

template <typename TX, typename TD>
cudaError_t backward_t(const TX* X, const TD* dY, const BwdArgs& a, float2* stats, cudaStream_t stream) {
    if (a.K > kBwdMaxK) {
        cudaError_t e = launch_pdl(norm_backward_long_kernel<TX, TD>, dim3(static_cast<unsigned>(a.M)),
                                   dim3(kMaxThreads), 0, stream, dim3(kNoCluster), X, dY, a, stats);
        if (e != cudaSuccess || (a.dw == nullptr && a.db == nullptr)) return e;
        const int parts = backward_blocks(a.M, a.K);
        const int64_t rows = (a.M + parts - 1) / parts;
        const int64_t strips = (a.K + 255) / 256;
        return launch_pdl(norm_columns_long_kernel<TX, TD>,
                          dim3(parts, static_cast<unsigned>(strips < 65535 ? strips : 65535)), dim3(256), 0, stream,
                          dim3(kNoCluster), X, dY, a, static_cast<const float2*>(stats), rows);
    }
    const int ch = chunks_of(a.K);
    if (a.K % kE == 0) {
        switch (ch) {
            case 1: return backward_c<TX, TD, true, 1>(X, dY, a, stream);
            case 2: return backward_c<TX, TD, true, 2>(X, dY, a, stream);
            default: return backward_c<TX, TD, true, 4>(X, dY, a, stream);
        }
    }
    switch (ch) {
        case 1: return backward_c<TX, TD, false, 1>(X, dY, a, stream);
        case 2: return backward_c<TX, TD, false, 2>(X, dY, a, stream);
        default: return backward_c<TX, TD, false, 4>(X, dY, a, stream);
    }
}

int64_t align16(int64_t n) { return (n + 15) / 16 * 16; }

}  // namespace

cudaError_t launch_norm_forward(const void* X, bool x_bf16, const float* w, const float* b, int64_t M, int64_t K,
                                int kind, float eps, void* Y, bool y_bf16, cudaStream_t stream) {
    const FwdArgs a{w, b, M, K, kind == 1, eps, 1.0f / static_cast<float>(K), Y, y_bf16};
    return x_bf16 ? forward_x(static_cast<const __nv_bfloat16*>(X), a, stream)
                  : forward_x(static_cast<const float*>(X), a, stream);
}

// Partial column sums of dw and db, and the rows' statistics for rows that do not fit the
// registers.
size_t norm_backward_workspace(int64_t M, int64_t K) {
    const int64_t parts = backward_blocks(M, K);
    int64_t bytes = parts > 1 ? 2 * align16(parts * K * 4) : 0;
    if (K > kBwdMaxK) bytes += align16(M * 8);
    return static_cast<size_t>(bytes);
}

cudaError_t launch_norm_backward(const void* dY, bool dy_bf16, const void* X, bool x_bf16, const float* w, int64_t M,
                                 int64_t K, int kind, float eps, void* dX, bool dx_bf16, float* dw, float* db,
                                 void* ws, cudaStream_t stream) {
    const int parts = backward_blocks(M, K);
    const int64_t part_bytes = align16(static_cast<int64_t>(parts) * K * 4);
    uint8_t* p = static_cast<uint8_t*>(ws);
    BwdArgs a{w, M, K, kind == 1, eps, 1.0f / static_cast<float>(K), dX, dx_bf16, dw, db};
    if (parts > 1) {
        if (dw != nullptr) a.dw = reinterpret_cast<float*>(p);
        if (db != nullptr) a.db = reinterpret_cast<float*>(p + part_bytes);
        p += 2 * part_bytes;
    }
    float2* stats = K > kBwdMaxK ? reinterpret_cast<float2*>(p) : nullptr;
    cudaError_t e;
    if (x_bf16) {
        const auto* x = static_cast<const __nv_bfloat16*>(X);
        e = dy_bf16 ? backward_t(x, static_cast<const __nv_bfloat16*>(dY), a, stats, stream)
                    : backward_t(x, static_cast<const float*>(dY), a, stats, stream);
    } else {
        const auto* x = static_cast<const float*>(X);
        e = dy_bf16 ? backward_t(x, static_cast<const __nv_bfloat16*>(dY), a, stats, stream)
                    : backward_t(x, static_cast<const float*>(dY), a, stats, stream);
    }
    if (e != cudaSuccess || parts == 1 || (dw == nullptr && db == nullptr)) return e;
    const dim3 grid(static_cast<unsigned>((K + 31) / 32), dw != nullptr && db != nullptr ? 2 : 1);
    return launch_pdl(norm_reduce_kernel, grid, dim3(32, 32), 0, stream, dim3(kNoCluster),
                      static_cast<const float*>(a.dw), static_cast<const float*>(a.db), parts, K, dw, db);
}

}  // namespace bl
