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
// of a row add in a tree.
//
// Layer kind: a mean from a plain fp32 sum is some units in its last place off, which for
// |mean| >> sigma shifts every n of the row by error / sigma (1e4 + 0.1 N(0,1), K = 3200: 8e-3).
// So the sum runs over x - ref, with ref the mean of four neighbouring elements of the row, and
//   mu + lo = ref + mean_k (x - ref),  c = x - mu,  n = (c - lo) r,
//   mean_k (x - mean)^2 = mean_k c^2 - lo^2,   mean_k(g n) = (mean_k(g c) - lo mean_k g) r
// where lo is what rounding the mean to fp32 leaves over.  The differences are right to half a unit
// of their own, so what is left is the rounding of a sum of them, whatever the mean; a constant
// row's are all zero.  Cost: one subtraction an element (8192 x 8192 bf16 with a bias: forward 52
// -> 55 us, backward 113.5 -> 116.5).
//
// Both are bound by memory: a row is read once, held in registers as it came, and written once.
// A matrix is cut into chunks of eight elements of its flat order, whatever K is, so that every
// access is 16 bytes wide on 16-byte boundaries in each of the matrices; a row's first and last
// chunk may belong to its neighbours in part, and those elements are masked.
//
// Forward: many small blocks, each thread one to four chunks of a row; the blocks on an SM
// overlap one another's loads, sums and stores.
// Backward: the threads of a row also keep the sums of their columns, which fills the register
// file with one resident block.  There a ring of rows in shared memory, filled by one warp with
// bulk copies, keeps the memory busy meanwhile.  Short rows share the block between groups of
// threads.  Rows of more than kSlice columns are split over a cluster of blocks that exchange
// their row sums through distributed shared memory.
//
// The column sums of the backward stay in the registers of the threads that own the columns
// while a block walks over its rows; they are added over the groups of a block in shared memory
// and over the blocks by a second kernel, always in the same order, so the results do not
// change from run to run.
#include <cuda_bf16.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "bl_device.cuh"
#include "bl_internal.h"
#include "bl_wait.cuh"

namespace bl {
namespace {

constexpr int kE = 8;            // elements of a chunk
constexpr int kSlice = 9712;     // most columns of a block of the backward
constexpr int kMaxCluster = 8;
constexpr int kMaxGroups = 24;   // groups of threads of a block
constexpr int kMaxThreads = 1024;
constexpr int kMaxStages = 8;
constexpr int kRingBytes = 208 * 1024;
constexpr int kParts = 148;      // most blocks or clusters: one per SM
constexpr unsigned long long kLandNs = 1000000ull;  // 1 ms: see Place::finish

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}

// The elements [lo, hi) of a chunk that belong to the row (all eight where rows are whole
// chunks).
struct Mask {
    int lo, hi;
    __device__ __forceinline__ bool any() const { return lo < hi; }
    __device__ __forceinline__ bool all() const { return lo <= 0 && hi >= kE; }
    __device__ __forceinline__ bool has(int e) const { return e >= lo && e < hi; }
};

// A chunk as it lies in memory, and its values.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
    float4 a, b;
    // what the compiler cannot see through: the values are converted and used from here, not held
    __device__ __forceinline__ void pin() {
        asm volatile("" : "+f"(a.x), "+f"(a.y), "+f"(a.z), "+f"(a.w), "+f"(b.x), "+f"(b.y), "+f"(b.z), "+f"(b.w));
    }
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void load_global(const float* p) {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p + 4));
    }
    __device__ __forceinline__ void clear() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    // the first n (1 to 7) elements
    __device__ __forceinline__ void load_some(const float* p, int n) {
        auto get = [&](int e) { return e < n ? __ldg(p + e) : 0.0f; };
        a = make_float4(get(0), get(1), get(2), get(3));
        b = make_float4(get(4), get(5), get(6), get(7));
    }
    __device__ __forceinline__ void keep(const Mask& m) {
        auto pick = [&](int e, float v) { return m.has(e) ? v : 0.0f; };
        a = make_float4(pick(0, a.x), pick(1, a.y), pick(2, a.z), pick(3, a.w));
        b = make_float4(pick(4, b.x), pick(5, b.y), pick(6, b.z), pick(7, b.w));
    }
    __device__ __forceinline__ float operator[](int e) const {
        switch (e) {
            case 0: return a.x;
            case 1: return a.y;
            case 2: return a.z;
            case 3: return a.w;
            case 4: return b.x;
            case 5: return b.y;
            case 6: return b.z;
            default: return b.w;
        }
    }
};
template <>
struct Raw<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void pin() { asm volatile("" : "+r"(a.x), "+r"(a.y), "+r"(a.z), "+r"(a.w)); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void load_global(const __nv_bfloat16* p) {
        a = __ldg(reinterpret_cast<const uint4*>(p));
    }
    __device__ __forceinline__ void clear() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void load_some(const __nv_bfloat16* p, int n) {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
        auto get = [&](int e) { return e < n ? static_cast<uint32_t>(__ldg(h + e)) << (16 * (e & 1)) : 0u; };
        a = make_uint4(get(0) | get(1), get(2) | get(3), get(4) | get(5), get(6) | get(7));
    }
    __device__ __forceinline__ void keep(const Mask& m) {
        auto half = [&](int e) { return (m.has(e) ? 0xFFFFu : 0u) | (m.has(e + 1) ? 0xFFFF0000u : 0u); };
        a = make_uint4(a.x & half(0), a.y & half(2), a.z & half(4), a.w & half(6));
    }
    __device__ __forceinline__ float operator[](int e) const {
        const uint32_t w = e < 2 ? a.x : e < 4 ? a.y : e < 6 ? a.z : a.w;
        return __uint_as_float((e & 1) ? (w & 0xFFFF0000u) : (w << 16));
    }
};

// The mean of four elements, exact if they are one value.
__device__ __forceinline__ float mean_of(float a, float b, float c, float d) {
    return fmaf(a, 0.25f, 0.25f * b) + fmaf(c, 0.25f, 0.25f * d);
}
__device__ __forceinline__ float mean_of(const float4& v) { return mean_of(v.x, v.y, v.z, v.w); }
__device__ __forceinline__ float mean_of(const uint2& v) {  // bf16
    return mean_of(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                   __uint_as_float(v.y & 0xFFFF0000u));
}
template <typename T>
struct Four;
template <>
struct Four<float> {
    using Type = float4;
};
template <>
struct Four<__nv_bfloat16> {
    using Type = uint2;
};

// What the layer kind's sums are taken from (see the top): the mean of the first four elements of a
// row of n that lie on their own alignment, or its first element where no four do.  The row starts
// `skip` elements behind a chunk's start.
template <typename T>
__device__ __forceinline__ float reference(const T* row, int skip, int64_t n) {
    const int ahead = -skip & 3;
    if (ahead + 4 > n) return to_f32(row[0]);
    return mean_of(*reinterpret_cast<const typename Four<T>::Type*>(row + ahead));
}

// ref + delta in two parts: the rounded sum and what that leaves over.
struct Mean {
    float mu, lo;
};
__device__ __forceinline__ Mean mean_from(float ref, float delta) {
    const float mu = ref + delta, b = mu - ref;
    return Mean{mu, (ref - (mu - b)) + (delta - b)};
}

// 1 / sqrt(variance + eps) from the sum of c^2, and shift with n = c r + shift.  (Without a mean
// lo is 0, and adding -0 changes no value.)
struct Spread {
    float r, shift;
};
__device__ __forceinline__ Spread spread_of(bool layer, float sum_cc, float lo, float inv_k, float eps) {
    if (!layer) return Spread{__frsqrt_rn(fmaf(sum_cc, inv_k, eps)), -0.0f};
    const float r = __frsqrt_rn(fmaf(-lo, lo, sum_cc * inv_k) + eps);
    return Spread{r, -lo * r};
}

// A chunk of the output at flat element `flat`, as fp32 or bf16.
__device__ __forceinline__ void store_flat(void* out, bool bf16, int64_t flat, const Mask& m, const float (&v)[kE]) {
    if (m.all()) {
        if (bf16) {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + flat) =
                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        } else {
            float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + flat);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        if (!m.has(e)) continue;
        if (bf16)
            static_cast<__nv_bfloat16*>(out)[flat + e] = __float2bfloat16_rn(v[e]);
        else
            static_cast<float*>(out)[flat + e] = v[e];
    }
}

// Eight values of a vector over `total` columns from column k (which may be masked or unaligned: then
// the three aligned groups of four around them are loaded and the eight cut out; element by element
// the forward of 5470 x 4859 with weight and bias takes 69 us, so 53).
template <bool EDGE>
__device__ __forceinline__ void load_vector(const float* p, float fill, int64_t k, int64_t total, const Mask& m,
                                            float (&v)[kE]) {
    if (!EDGE && p != nullptr && m.any()) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p + k)), b = __ldg(reinterpret_cast<const float4*>(p + k + 4));
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        return;
    }
    const int64_t at = k & ~int64_t(3);
    if (EDGE && p != nullptr && m.all() && at + 12 <= total) {
        const float4* g = reinterpret_cast<const float4*>(p + at);
        const float4 a = __ldg(g), b = __ldg(g + 1), c = __ldg(g + 2);
        const float w[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
        const int off = static_cast<int>(k) & 3;
        float u[10];
#pragma unroll
        for (int e = 0; e < 10; ++e) u[e] = (off & 2) ? w[e + 2] : w[e];
#pragma unroll
        for (int e = 0; e < kE; ++e) v[e] = (off & 1) ? u[e + 1] : u[e];
        return;
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) v[e] = p != nullptr && m.has(e) ? __ldg(p + k + e) : fill;
}

// Sums of two values over the threads of a group.  Slots alternate between calls: one is written
// again only after a barrier that every reader of it has passed.  HALVES: each half of a warp adds
// one of the two, which takes half the exchanges and some registers (backward of 8192 x 8192 layer
// fp32 193 -> 142 us, 4096 x 16384 241 -> 177; the 640 threads with two chunks, whose registers are
// short, add both in every lane: 8192 x 4096 layer bf16 72 us, with halves 75, 8192 x 8640 RMS 120
// and 123).
template <bool HALVES>
struct GroupSum {
    float2* buf;  // [2][32] of this group
    int t, tpr, group;
    uint32_t calls = 0;
    __device__ __forceinline__ float2 operator()(float a, float b) {
        if constexpr (HALVES) {
            const bool upper = (t & 16) != 0;
            float v = upper ? b : a;
            v += __shfl_xor_sync(0xFFFFFFFFu, upper ? a : b, 16);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            if (tpr > 32) {
                // the warps' sums of a, then those of b
                float* s = reinterpret_cast<float*>(buf + 32 * (calls & 1)) + 2 * (t & 16);
                const int i = t & 15, n = tpr >> 5;
                if (i == 0) s[t >> 5] = v;
                asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
                v = i < n ? s[i] : 0.0f;
                if (i + 16 < n) v += s[i + 16];
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            }
            a = __shfl_sync(0xFFFFFFFFu, v, 0);
            b = __shfl_sync(0xFFFFFFFFu, v, 16);
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
                b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
            }
            if (tpr > 32) {
                float2* s = buf + 32 * (calls & 1);
                if ((t & 31) == 0) s[t >> 5] = make_float2(a, b);
                asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
                const float2 v = (t & 31) < (tpr >> 5) ? s[t & 31] : make_float2(0.0f, 0.0f);
                a = v.x, b = v.y;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
                    b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
                }
            }
        }
        ++calls;
        return make_float2(a, b);
    }
};

// -------------------------------------------------------------------------- forward --

struct FwdArgs {
    const float* w;
    const float* b;
    int64_t M, K;
    bool layer;
    float eps, inv_k;
    void* out;
    bool out_bf16;
};

// block: x = threads of a row, y = groups of them.  A group takes R neighbouring rows together:
// their sums share a latency and they share the loads of weight and bias.  EDGE: rows are not
// whole chunks.
template <typename TX, bool EDGE, int CH, int R, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) norm_forward_kernel(const TX* __restrict__ X, const FwdArgs a) {
    __shared__ float2 sums[8][64];
    const int t = threadIdx.x, tpr = blockDim.x, group = threadIdx.y;
    pdl_wait_then_release();
    GroupSum<true> row_sum{sums[group], t, tpr, group};
    const int64_t m0 = (static_cast<int64_t>(blockIdx.x) * blockDim.y + group) * R;
    if (m0 >= a.M) return;  // a whole group leaves together
    const int64_t total = a.M * a.K;
    // row r: element 0 of its chunk c is flat element flat(r, c), column col(r, c) of the row
    auto skip = [&](int r) { return EDGE ? static_cast<int>((m0 + r) * a.K & (kE - 1)) : 0; };
    auto col = [&](int r, int c) { return static_cast<int64_t>(c * tpr + t) * kE - skip(r); };
    auto flat = [&](int r, int c) { return (m0 + r) * a.K + col(r, c); };
    auto mask = [&](int r, int c) {
        const int64_t k = col(r, c);
        if (R > 1 && m0 + r >= a.M) return Mask{0, 0};
        if constexpr (EDGE)
            return Mask{k < 0 ? static_cast<int>(-k) : 0, a.K - k < kE ? static_cast<int>(a.K - k) : kE};
        else
            return Mask{0, k < a.K ? kE : 0};
    };
    Raw<TX> x[R][CH];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            x[r][c].clear();
            if (!mask(r, c).any()) continue;
            if (!EDGE || flat(r, c) + kE <= total)
                x[r][c].load_global(X + flat(r, c));
            else  // the matrix's last chunk
                x[r][c].load_some(X + flat(r, c), static_cast<int>(total - flat(r, c)));
        }
    if constexpr (EDGE) {  // zeros in place of the neighbouring rows' elements
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const Mask k = mask(r, c);
                if (k.any() && !k.all()) x[r][c].keep(k);
            }
    }
    auto values = [&](int r, int c, float(&v)[kE]) {
#pragma unroll
        for (int e = 0; e < kE; ++e) v[e] = x[r][c][e];
    };
    // both of the sums that GroupSum takes are of rows: row 0 and row R - 1
    float mu[R], lo[R];
#pragma unroll
    for (int r = 0; r < R; ++r) mu[r] = lo[r] = 0.0f;
    if (a.layer) {
        float s[R], ref[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            ref[r] = R == 1 || m0 + r < a.M ? reference(X + (m0 + r) * a.K, EDGE ? skip(r) : 0, a.K) : 0.0f;
            s[r] = 0.0f;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const Mask k = mask(r, c);
                float v[kE];
                values(r, c, v);
                const float from = k.any() ? ref[r] : 0.0f;  // a chunk that is not the row's is zeros
#pragma unroll
                for (int e = 0; e < kE; ++e) v[e] -= from;
                if (EDGE && !k.all())
#pragma unroll
                    for (int e = 0; e < kE; ++e)
                        if (!k.has(e)) v[e] = 0.0f;
#pragma unroll
                for (int e = 0; e < kE; ++e) s[r] += v[e];
            }
        }
        const float2 both = row_sum(s[0], R > 1 ? s[R - 1] : 0.0f);
        const Mean first = mean_from(ref[0], both.x * a.inv_k), second = mean_from(ref[R - 1], both.y * a.inv_k);
        mu[0] = first.mu, lo[0] = first.lo;
        if constexpr (R > 1) mu[1] = second.mu, lo[1] = second.lo;
    }
    float q[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        q[r] = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const Mask k = mask(r, c);
            if (!k.any()) continue;
            float v[kE];
            values(r, c, v);
#pragma unroll
            for (int e = 0; e < kE; ++e) v[e] -= mu[r];
            if (EDGE && a.layer && !k.all())
#pragma unroll
                for (int e = 0; e < kE; ++e)
                    if (!k.has(e)) v[e] = 0.0f;
#pragma unroll
            for (int e = 0; e < kE; ++e) q[r] = fmaf(v[e], v[e], q[r]);
        }
    }
    const float2 both = row_sum(q[0], R > 1 ? q[R - 1] : 0.0f);
    Spread of[R];
    of[0] = spread_of(a.layer, both.x, lo[0], a.inv_k, a.eps);
    if constexpr (R > 1) of[1] = spread_of(a.layer, both.y, lo[1], a.inv_k, a.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        float w[kE], b[kE];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const Mask k = mask(r, c);
            if (EDGE || r == 0) {  // whole chunks have the same columns in every row
                load_vector<EDGE>(a.w, 1.0f, col(r, c), a.K, k, w);
                load_vector<EDGE>(a.b, 0.0f, col(r, c), a.K, k, b);
            }
            if (!k.any()) continue;
            float v[kE];
            values(r, c, v);
#pragma unroll
            for (int e = 0; e < kE; ++e) v[e] = fmaf(v[e] - mu[r], of[r].r, of[r].shift) * w[e] + b[e];
            store_flat(a.out, a.out_bf16, flat(r, c), k, v);
        }
    }
}

// The two sums over a whole block, for rows too long for its registers.
struct BlockSum {
    float2* buf;  // [2][32]
    int t, tpr;
    int slot = 0;
    __device__ __forceinline__ float2 operator()(float a, float b) {
        float2* s = buf + 32 * slot;
        slot ^= 1;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        if ((t & 31) == 0) s[t >> 5] = make_float2(a, b);
        __syncthreads();
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

// Rows too long for the registers of a block: three passes over the row (it stays in the caches
// between them).
template <typename TX>
__global__ void __launch_bounds__(kMaxThreads) norm_forward_long_kernel(const TX* __restrict__ X, const FwdArgs a) {
    __shared__ float2 sums[64];
    const int t = threadIdx.x, tpr = blockDim.x;
    pdl_wait_then_release();
    BlockSum row_sum{sums, t, tpr};
    const int64_t m = blockIdx.x;
    const TX* row = X + m * a.K;
    float mu = 0.0f, lo = 0.0f;
    if (a.layer) {
        const float ref = reference(row, static_cast<int>(m * a.K & (kE - 1)), a.K);
        float s = 0.0f;
        for (int64_t k = t; k < a.K; k += tpr) s += to_f32(row[k]) - ref;
        const Mean mean = mean_from(ref, row_sum(s, 0.0f).x * a.inv_k);
        mu = mean.mu, lo = mean.lo;
    }
    float v = 0.0f;
    for (int64_t k = t; k < a.K; k += tpr) {
        const float d = to_f32(row[k]) - mu;
        v = fmaf(d, d, v);
    }
    const Spread of = spread_of(a.layer, row_sum(v, 0.0f).x, lo, a.inv_k, a.eps);
    for (int64_t k = t; k < a.K; k += tpr) {
        float y = fmaf(to_f32(row[k]) - mu, of.r, of.shift);
        if (a.w != nullptr) y *= __ldg(a.w + k);
        if (a.b != nullptr) y += __ldg(a.b + k);
        if (a.out_bf16)
            static_cast<__nv_bfloat16*>(a.out)[m * a.K + k] = __float2bfloat16_rn(y);
        else
            static_cast<float*>(a.out)[m * a.K + k] = y;
    }
}

// ------------------------------------------------- backward: the ring of rows --

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// What a block works on.  Group g of batch i takes row first + i * step + g; with rows that are
// not whole chunks the number of rows in step is a multiple of eight, so that a group's rows
// all start at the same place of a chunk and a thread's columns stay the same.
struct Shape {
    int64_t M, K;
    int tpr, groups;     // threads of a row, rows at a time
    int stages;
    int slot_x, slot_d;  // bytes of a slot for x and for dy
    int slice;           // columns of a block
};

struct Control {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t cross[2];                    // row sums of the blocks of the cluster
    float4 cross_sums[2][kMaxCluster];
    float2 sums[kMaxGroups][64];
    int abort;
    int issued;                           // loads of the ring
    unsigned long long wait_ns;
    // wait_on with the limit in shared memory, where it takes no registers (as an argument: 8192 x 4096
    // layer bf16 82 us, so 72)
    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) {
        return wait_on(bar, parity, &abort, [this] { return *static_cast<volatile unsigned long long*>(&wait_ns); });
    }
};

// GroupSum, then over the blocks of the cluster (each sends its sums to all).  A slot is
// written again only after the other blocks' next sums, sent by threads that have read it.
template <bool HALVES>
struct RowSum {
    GroupSum<HALVES> local;
    Control* ctl;
    int cluster;
    uint32_t rank;
    __device__ __forceinline__ float2 operator()(float a, float b) {
        const uint32_t call = local.calls;
        const float2 own = local(a, b);
        if (cluster == 1) return own;
        exchange(call, make_float4(own.x, own.y, 0.0f, 0.0f));
        float2 all = make_float2(0.0f, 0.0f);
        for (int i = 0; i < cluster; ++i) {
            const float4 v = ctl->cross_sums[call & 1][i];
            all.x += v.x, all.y += v.y;
        }
        return all;
    }
    // The same where a is a sum over this block's `slice` columns (the last block's: the rest of K)
    // of differences from its own ref: returns their sum from the first block's ref, and that.
    __device__ __forceinline__ float3 from_ref(float a, float b, float ref, int slice, int64_t K) {
        const uint32_t call = local.calls;
        const float2 own = local(a, b);
        if (cluster == 1) return make_float3(own.x, own.y, ref);
        exchange(call, make_float4(own.x, own.y, ref, 0.0f));
        const float4* s = ctl->cross_sums[call & 1];
        const float first = s[0].z;
        float2 all = make_float2(0.0f, 0.0f);
        for (int i = 0; i < cluster; ++i) {
            const float4 v = s[i];
            const float n = static_cast<float>(i + 1 < cluster ? slice : static_cast<int>(K - int64_t(i) * slice));
            all.x += fmaf(n, v.z - first, v.x);
            all.y += v.y;
        }
        return make_float3(all.x, all.y, first);
    }
    // After a wait was given up nothing is sent or expected any more (the slot's phase before may not have
    // ended), and the other blocks give up in turn.
    __device__ __forceinline__ void exchange(uint32_t call, const float4& own) {
        const int slot = static_cast<int>(call & 1), t = local.t;
        const uint32_t bar = smem_u32(&ctl->cross[slot]);
        if (t < cluster && !*static_cast<volatile int*>(&ctl->abort)) {
            if (t == 0) mbar_arrive_expect_tx(bar, 16u * static_cast<uint32_t>(cluster));
            const uint32_t dst = mapa_shared(smem_u32(&ctl->cross_sums[slot][rank]), static_cast<uint32_t>(t));
            const uint32_t rbar = mapa_shared(bar, static_cast<uint32_t>(t));
            asm volatile(
                "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
                "r"(__float_as_uint(own.x)), "r"(__float_as_uint(own.y)), "r"(__float_as_uint(own.z)),
                "r"(__float_as_uint(own.w)), "r"(rbar)
                : "memory");
        }
        ctl->wait(bar, (call >> 1) & 1u);
    }
};

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// Where a block stands.
struct Place {
    Control* ctl;
    uint8_t* ring;
    int t, group, tpr;
    bool producer;
    int cluster;
    uint32_t rank;
    int64_t first, step;  // its batches start at rows first, first + step, ...
    int k0, ks;           // its columns
    __device__ __forceinline__ Place(uint8_t* smem, const Shape& s, unsigned long long wait_ns) {
        ctl = reinterpret_cast<Control*>(smem);
        ring = smem + ((sizeof(Control) + 127) & ~size_t(127));
        tpr = s.tpr;
        producer = static_cast<int>(threadIdx.x) >= tpr * s.groups;
        group = threadIdx.x / tpr;
        t = threadIdx.x - group * tpr;
        cluster = static_cast<int>(cluster_size());
        rank = cluster_ctarank();
        first = static_cast<int64_t>(blockIdx.x / cluster) * s.groups;
        step = static_cast<int64_t>(gridDim.x / cluster) * s.groups;
        k0 = static_cast<int>(rank) * s.slice;
        ks = s.K - k0 < s.slice ? static_cast<int>(s.K - k0) : s.slice;
        if (threadIdx.x == 0) {
            for (int i = 0; i < s.stages; ++i) {
                mbar_init(smem_u32(&ctl->full[i]), 1);
                mbar_init(smem_u32(&ctl->empty[i]), tpr * s.groups / 32);
            }
            mbar_init(smem_u32(&ctl->cross[0]), 1);
            mbar_init(smem_u32(&ctl->cross[1]), 1);
            ctl->abort = ctl->issued = 0;
            ctl->wait_ns = wait_ns;
            mbar_fence_init();
        }
        pdl_wait_then_release();
        __syncthreads();
        if (cluster > 1) cluster_sync_all();  // every block's barriers exist
    }
    // The flat elements of the batch of rows that starts at row m, as whole chunks: [begin, end),
    // end cut at the matrix's last whole chunk.  (With a cluster there is one row, cut to its
    // slice.)
    __device__ __forceinline__ void span(const Shape& s, int64_t m, int64_t& begin, int64_t& end) const {
        const int64_t rows = s.M - m < s.groups ? s.M - m : s.groups;
        begin = (m * s.K + k0) & ~int64_t(kE - 1);
        end = ((cluster > 1 ? m * s.K + k0 + ks : (m + rows) * s.K) + kE - 1) & ~int64_t(kE - 1);
        const int64_t most = (s.M * s.K) & ~int64_t(kE - 1);
        if (end > most) end = most;
        if (end < begin) end = begin;
    }
    __device__ __forceinline__ void finish(const Shape& s, int32_t* err) const {
        __syncthreads();
        if (cluster > 1) cluster_sync_all();
        if (threadIdx.x == 0 && *static_cast<volatile int*>(&ctl->abort)) {
            // a wait was given up: loads of the ring may be in flight
            for (int i = 0; i < s.stages; ++i) {
                const int fills = fills_of(ctl->issued, s.stages, i);
                if (fills > 0) drain_wait(smem_u32(&ctl->full[i]), static_cast<uint32_t>((fills - 1) & 1));
            }
            // And sums of the cluster's other blocks, which have all ended.  How many they sent before
            // they gave up is not known here, so the block stays until they must have landed.  (A block
            // that has not given up has waited for every sum that was sent to it.)
            const unsigned long long t0 = globaltimer_ns();
            while (cluster > 1 && globaltimer_ns() - t0 < kLandNs) {
            }
            if (err != nullptr) atomicOr(err, kErrBitTimeout);
        }
    }
};

// One lane fills the ring, in the order in which the batches are worked on.
template <typename TX, typename TD>
__device__ __forceinline__ void fill_ring(const Place& pl, const Shape& s, const TX* X, const TD* dY,
                                          unsigned long long wait_ns, int stall_after) {
    if (threadIdx.x % 32 != 0) return;
    int issued = 0;
    for (int64_t m = pl.first; m < s.M; m += pl.step, ++issued) {
        const int stage = issued % s.stages;
        if (!wait_on(smem_u32(&pl.ctl->empty[stage]), static_cast<uint32_t>(((issued / s.stages) & 1) ^ 1),
                     &pl.ctl->abort, wait_ns))
            break;
        if (issued == stall_after) {  // the bounded-wait test: stop issuing
            stall_until_abort(&pl.ctl->abort, 4 * wait_ns);
            break;
        }
        const uint32_t bar = smem_u32(&pl.ctl->full[stage]);
        const uint32_t slot = smem_u32(pl.ring) + static_cast<uint32_t>(stage * (s.slot_x + s.slot_d));
        int64_t begin, end;
        pl.span(s, m, begin, end);
        const uint32_t n = static_cast<uint32_t>(end - begin);
        if (s.M * s.K - end < kE) {
            // the matrix ends inside a chunk, which no bulk copy may read as a whole: its
            // elements come one by one (and are visible to who waits for the barrier)
            uint8_t* raw = pl.ring + stage * (s.slot_x + s.slot_d);
            for (int64_t i = end; i < s.M * s.K; ++i) {
                reinterpret_cast<TX*>(raw)[i - begin] = X[i];
                reinterpret_cast<TD*>(raw + s.slot_x)[i - begin] = dY[i];
            }
        }
        mbar_arrive_expect_tx(bar, n * static_cast<uint32_t>(sizeof(TX) + sizeof(TD)));
        if (n > 0) {
            bulk_load(slot, X + begin, n * static_cast<uint32_t>(sizeof(TX)), bar);
            bulk_load(slot + s.slot_x, dY + begin, n * static_cast<uint32_t>(sizeof(TD)), bar);
        }
    }
    pl.ctl->issued = issued;
}

struct BwdArgs {
    Shape s;
    const float* w;
    float eps, inv_k;
    void* dx;
    bool dx_bf16;
    float* dw;  // [blocks or clusters, K] partial sums (the result itself with one), or NULL
    float* db;
    int32_t* err;
    unsigned long long wait_ns;  // limit of every wait (2 s outside the bounded-wait test)
    int stall_after;             // the ring's producers stop after this many loads (< 0: never)
};

// LAYER: the kind, known when compiling, so that RMS rows pay nothing for the mean (8192 x 8640: 121
// us, with a test at run time 145).  DB: with the bias's gradient (its sums take registers).
template <typename TX, typename TD, bool EDGE, bool LAYER, bool DB, int CH, int THREADS>
__global__ void __launch_bounds__(THREADS)
    norm_backward_kernel(const TX* __restrict__ X, const TD* __restrict__ dY, const __grid_constant__ BwdArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr bool kHalves = THREADS < 640 || CH == 1;
    const Shape& s = a.s;
    Place pl(smem, s, a.wait_ns);
    const int t = pl.t, tpr = pl.tpr;
    // this thread's columns: element 0 of chunk c is column k0 + (c tpr + t) 8 - skip
    const int skip = EDGE ? static_cast<int>(((pl.first + pl.group) * s.K + pl.k0) & (kE - 1)) : 0;
    Mask mask[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int k = (c * tpr + t) * kE - skip;
        mask[c] = EDGE ? Mask{k < 0 ? -k : 0, pl.ks - k < kE ? pl.ks - k : kE} : Mask{0, k < pl.ks ? kE : 0};
    }
    float dw[CH][kE], db[DB ? CH : 1][kE];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            dw[c][e] = 0.0f;
            if constexpr (DB) db[c][e] = 0.0f;
        }
    if (pl.producer) {
        fill_ring<TX, TD>(pl, s, X, dY, a.wait_ns, a.stall_after);
    } else {
        RowSum<kHalves> row_sum{GroupSum<kHalves>{pl.ctl->sums[pl.group], t, tpr, pl.group}, pl.ctl, pl.cluster,
                                pl.rank};
        float w[CH][kE];
#pragma unroll
        for (int c = 0; c < CH; ++c) load_vector<EDGE>(a.w, 1.0f, pl.k0 + (c * tpr + t) * kE - skip, s.K, mask[c], w[c]);
        // where the thread's chunks are in a slot: the same in every batch (see Shape)
        const int64_t row0 = pl.first * s.K + pl.k0;
        const int at = static_cast<int>((pl.first + pl.group) * s.K + pl.k0 - skip - (row0 & ~int64_t(kE - 1))) + t * kE;
        int64_t flat = (pl.first + pl.group) * s.K + pl.k0 - skip + t * kE;  // of chunk 0, in the matrix
        const int64_t flat_step = pl.step * s.K;
        // values converted once with one chunk; with two that costs more (120 -> 131 us for 8192 x
        // 8640 RMS), and the raw chunk is converted in each pass
        constexpr bool kOnce = CH == 1;
        // Two chunks, both gradients and both sums in 96 registers: held from one pass to the next, the
        // converted values spill (8192 x 4096 bf16 114 us against 72, 8192 x 8640 bf16 x, fp32 dy 287
        // against 218), so each pass starts from the raw chunks, and addresses from the row.
        constexpr bool kTight = LAYER && DB && THREADS == 640;
        auto drop = [&](Raw<TX>(&x)[CH], Raw<TD>(&d)[CH]) {
            if constexpr (kTight)
#pragma unroll
                for (int c = 0; c < CH; ++c) x[c].pin(), d[c].pin();
        };
        int stage = 0;
        uint32_t phase = 0;
        for (int64_t m = pl.first + pl.group; m - pl.group < s.M; m += pl.step, flat += flat_step) {
            // a wait that gives up does not end the loop (the group's barriers would no longer match):
            // the rest runs on what is there, and the block reports it at the end
            pl.ctl->wait(smem_u32(&pl.ctl->full[stage]), phase);
            const bool live = m < s.M;
            const uint8_t* slot = pl.ring + stage * (s.slot_x + s.slot_d);
            Raw<TX> x[CH];
            Raw<TD> d[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int i = at + c * tpr * kE;
                if (live && mask[c].any()) {
                    x[c].load(reinterpret_cast<const TX*>(slot) + i);
                    d[c].load(reinterpret_cast<const TD*>(slot + s.slot_x) + i);
                } else {
                    x[c].clear();
                    d[c].clear();
                }
            }
            float ref = 0.0f;
            if (LAYER && live) {  // here as well: the slot is given back below
                ref = reference(reinterpret_cast<const TX*>(slot) + at - t * kE + skip, EDGE ? skip : 0, pl.ks);
            }
            __syncwarp();
            if ((t & 31) == 0) mbar_arrive(smem_u32(&pl.ctl->empty[stage]));
            if (++stage == s.stages) {
                stage = 0;
                phase ^= 1u;
            }
            if (!live) continue;  // rows of a batch past the last one: the whole group skips
            // the values of chunk c; where they are not the row's, x is ref and dy zero
            auto convert = [&](int c, float(&xv)[kE], float(&dv)[kE]) {
#pragma unroll
                for (int e = 0; e < kE; ++e) xv[e] = x[c][e], dv[e] = d[c][e];
                if (EDGE && !mask[c].all())
#pragma unroll
                    for (int e = 0; e < kE; ++e)
                        if (!mask[c].has(e)) xv[e] = ref, dv[e] = 0.0f;
            };
            float xs[kOnce ? CH : 1][kE], ds[kOnce ? CH : 1][kE];
            if constexpr (kOnce)
#pragma unroll
                for (int c = 0; c < CH; ++c) convert(c, xs[c], ds[c]);
            auto values = [&](int c, float(&xv)[kE], float(&dv)[kE]) {
                if constexpr (kOnce) {
#pragma unroll
                    for (int e = 0; e < kE; ++e) xv[e] = xs[c][e], dv[e] = ds[c][e];
                } else {
                    convert(c, xv, dv);
                }
            };
            float mu = 0.0f, lo = 0.0f, c2 = 0.0f;
            if constexpr (LAYER) {
                float sum = 0.0f, sg = 0.0f;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    float xv[kE], dv[kE];
                    values(c, xv, dv);
                    const float from = EDGE || mask[c].any() ? ref : 0.0f;  // a chunk that is not the row's is zeros
#pragma unroll
                    for (int e = 0; e < kE; ++e) {
                        sum += xv[e] - from;
                        sg = fmaf(dv[e], w[c][e], sg);
                    }
                }
                const float3 all = row_sum.from_ref(sum, sg, ref, s.slice, s.K);
                const Mean mean = mean_from(all.z, all.x * a.inv_k);
                mu = mean.mu, lo = mean.lo;
                c2 = all.y * a.inv_k;
                drop(x, d);
            }
            float v = 0.0f, gx = 0.0f;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                if (!mask[c].any()) continue;
                float xv[kE], dv[kE];
                values(c, xv, dv);
#pragma unroll
                for (int e = 0; e < kE; ++e) xv[e] -= mu;
                if (EDGE && !mask[c].all())
#pragma unroll
                    for (int e = 0; e < kE; ++e)
                        if (!mask[c].has(e)) xv[e] = 0.0f;
                if constexpr (kOnce)
#pragma unroll
                    for (int e = 0; e < kE; ++e) xs[c][e] = xv[e];
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    v = fmaf(xv[e], xv[e], v);
                    gx = fmaf(dv[e] * w[c][e], xv[e], gx);
                }
            }
            const float2 both = row_sum(v, gx);
            drop(x, d);
            const Spread of = spread_of(LAYER, both.x, lo, a.inv_k, a.eps);
            const float r = of.r;
            const float c1 = fmaf(-lo, c2, both.y * a.inv_k) * r;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                if (!mask[c].any()) continue;
                float xv[kE], dv[kE];
                values(c, xv, dv);
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    const float n = fmaf(kOnce ? xv[e] : xv[e] - mu, r, of.shift);
                    dw[c][e] = fmaf(dv[e], n, dw[c][e]);
                    if constexpr (DB) db[c][e] += dv[e];
                    xv[e] = r * fmaf(-n, c1, fmaf(dv[e], w[c][e], -c2));
                }
                const int64_t first = kTight ? m * s.K + (pl.k0 - skip + t * kE) : flat;
                store_flat(a.dx, a.dx_bf16, first + c * tpr * kE, mask[c], xv);
            }
        }
    }
    if (a.dw != nullptr || DB) {
        // every group leaves its column sums in shared memory (the ring is free: every copy has
        // landed and been read), and they are added in the groups' order
        float* cols = reinterpret_cast<float*>(pl.ring);
        const int ks = pl.ks, all = s.groups * ks;
        __syncthreads();
        if (!pl.producer) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int k = (c * tpr + t) * kE - skip;
                float* p = cols + pl.group * ks + k;
                if (!EDGE && mask[c].any()) {
                    *reinterpret_cast<float4*>(p) = make_float4(dw[c][0], dw[c][1], dw[c][2], dw[c][3]);
                    *reinterpret_cast<float4*>(p + 4) = make_float4(dw[c][4], dw[c][5], dw[c][6], dw[c][7]);
                    if constexpr (DB) {
                        *reinterpret_cast<float4*>(p + all) = make_float4(db[c][0], db[c][1], db[c][2], db[c][3]);
                        *reinterpret_cast<float4*>(p + all + 4) = make_float4(db[c][4], db[c][5], db[c][6], db[c][7]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < kE; ++e) {
                        if (!mask[c].has(e)) continue;
                        p[e] = dw[c][e];
                        if constexpr (DB) p[all + e] = db[c][e];
                    }
                }
            }
        }
        __syncthreads();
        const int64_t off = static_cast<int64_t>(blockIdx.x / pl.cluster) * s.K + pl.k0;
        for (int k = threadIdx.x; k < ks; k += blockDim.x) {
            float sw = 0.0f, sb = 0.0f;
            for (int g = 0; g < s.groups; ++g) {
                sw += cols[g * ks + k];
                if constexpr (DB) sb += cols[all + g * ks + k];
            }
            if (a.dw != nullptr) a.dw[off + k] = sw;
            if constexpr (DB) a.db[off + k] = sb;
        }
    }
    pl.finish(s, a.err);
}

struct LongBwdArgs {
    const float* w;
    int64_t M, K;
    bool layer;
    float eps, inv_k;
    void* dx;
    bool dx_bf16;
    float* dw;  // [strips of rows, K] partial sums (the result itself with one), or NULL
    float* db;
};

// Rows longer than a cluster's slices: dx row by row as in norm_forward_long_kernel, keeping
// (mu, r, shift) of every row for the column kernel below.
template <typename TX, typename TD>
__global__ void __launch_bounds__(kMaxThreads)
    norm_backward_long_kernel(const TX* __restrict__ X, const TD* __restrict__ dY, const LongBwdArgs a,
                              float4* __restrict__ stats) {
    __shared__ float2 sums[64];
    const int t = threadIdx.x, tpr = blockDim.x;
    pdl_wait_then_release();
    BlockSum row_sum{sums, t, tpr};
    const int64_t m = blockIdx.x;
    const TX* row = X + m * a.K;
    const TD* drow = dY + m * a.K;
    auto grad = [&](int64_t k) {
        const float d = to_f32(drow[k]);
        return a.w != nullptr ? d * __ldg(a.w + k) : d;
    };
    float mu = 0.0f, lo = 0.0f, c2 = 0.0f;
    if (a.layer) {
        const float ref = reference(row, static_cast<int>(m * a.K & (kE - 1)), a.K);
        float s = 0.0f, sg = 0.0f;
        for (int64_t k = t; k < a.K; k += tpr) {
            s += to_f32(row[k]) - ref;
            sg += grad(k);
        }
        const float2 both = row_sum(s, sg);
        const Mean mean = mean_from(ref, both.x * a.inv_k);
        mu = mean.mu, lo = mean.lo;
        c2 = both.y * a.inv_k;
    }
    float v = 0.0f, gx = 0.0f;
    for (int64_t k = t; k < a.K; k += tpr) {
        const float x = to_f32(row[k]) - mu;
        v = fmaf(x, x, v);
        gx = fmaf(grad(k), x, gx);
    }
    const float2 both = row_sum(v, gx);
    const Spread of = spread_of(a.layer, both.x, lo, a.inv_k, a.eps);
    const float c1 = fmaf(-lo, c2, both.y * a.inv_k) * of.r;
    for (int64_t k = t; k < a.K; k += tpr) {
        const float n = fmaf(to_f32(row[k]) - mu, of.r, of.shift);
        const float o = of.r * ((grad(k) - c2) - n * c1);
        if (a.dx_bf16)
            static_cast<__nv_bfloat16*>(a.dx)[m * a.K + k] = __float2bfloat16_rn(o);
        else
            static_cast<float*>(a.dx)[m * a.K + k] = o;
    }
    if (t == 0 && stats != nullptr) stats[m] = make_float4(mu, of.r, of.shift, 0.0f);
}

// Column sums of a strip of rows from x, dy and the rows' (mu, r, shift): a thread owns a column.
template <typename TX, typename TD>
__global__ void __launch_bounds__(256)
    norm_columns_long_kernel(const TX* __restrict__ X, const TD* __restrict__ dY, const LongBwdArgs a,
                             const float4* __restrict__ stats, int64_t rows_per_block) {
    pdl_wait_then_release();
    const int64_t m0 = blockIdx.x * rows_per_block;
    const int64_t m1 = m0 + rows_per_block < a.M ? m0 + rows_per_block : a.M;
    for (int64_t k = blockIdx.y * 256 + threadIdx.x; k < a.K; k += static_cast<int64_t>(gridDim.y) * 256) {
        float dw = 0.0f, db = 0.0f;
#pragma unroll 4
        for (int64_t m = m0; m < m1; ++m) {
            const float4 st = __ldg(stats + m);
            const float d = to_f32(dY[m * a.K + k]);
            dw = fmaf(d, fmaf(to_f32(X[m * a.K + k]) - st.x, st.y, st.z), dw);
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

// --------------------------------------------------------------------- launches --

// Chunks that a row of K elements can touch.
int64_t chunks_of(int64_t K) { return K % kE == 0 ? K / kE : (K + kE - 2) / kE + 1; }

// Forward: up to 8192 columns in blocks of up to 256 threads, many of which share an SM; longer
// rows in one block of up to 1024 threads with four chunks each.
constexpr int64_t kFwdMaxChunks = int64_t(kMaxThreads) * 4;

template <typename TX, bool EDGE>
cudaError_t forward_t(const TX* X, const FwdArgs& a, cudaStream_t stream) {
    const int64_t chunks = chunks_of(a.K);
    const int ch = chunks <= 128 ? 1 : chunks <= 256 ? 2 : 4;
    const int tpr = static_cast<int>(((chunks + ch - 1) / ch + 31) / 32 * 32);
    // several rows share a block of 256 threads, and a group takes two rows, as long as the
    // blocks still cover the SMs
    const int64_t spread = (a.M + kParts - 1) / kParts;
    int groups = 256 / tpr;
    if (groups > spread) groups = static_cast<int>(spread);
    if (groups < 1) groups = 1;
    const bool two = sizeof(TX) == 2 && !EDGE && tpr <= 256 && 2 * groups <= spread;
    const int64_t rows = two ? 2 * groups : groups;
    const dim3 grid(static_cast<unsigned>((a.M + rows - 1) / rows)), block(tpr, groups);
    auto run = [&](auto kernel) { return launch_pdl(kernel, grid, block, 0, stream, dim3(kNoCluster), X, a); };
    if constexpr (sizeof(TX) == 2 && !EDGE) {
        if (two) {
            if (ch == 1) return run(norm_forward_kernel<TX, EDGE, 1, 2, 256, 5>);
            if (ch == 2) return run(norm_forward_kernel<TX, EDGE, 2, 2, 256, 5>);
            return run(norm_forward_kernel<TX, EDGE, 4, 2, 256, 4>);
        }
    }
    if (ch == 1) return run(norm_forward_kernel<TX, EDGE, 1, 1, 256, 6>);
    if (ch == 2) return run(norm_forward_kernel<TX, EDGE, 2, 1, 256, 5>);
    if (tpr <= 256) return run(norm_forward_kernel<TX, EDGE, 4, 1, 256, 4>);
    return run(norm_forward_kernel<TX, EDGE, 4, 1, kMaxThreads, 1>);
}

template <typename TX>
cudaError_t forward_x(const TX* X, const FwdArgs& a, cudaStream_t stream) {
    if (chunks_of(a.K) > kFwdMaxChunks)
        return launch_pdl(norm_forward_long_kernel<TX>, dim3(static_cast<unsigned>(a.M)), dim3(kMaxThreads), 0, stream,
                          dim3(kNoCluster), X, a);
    return a.K % kE == 0 ? forward_t<TX, false>(X, a, stream) : forward_t<TX, true>(X, a, stream);
}

// Backward: how rows of K columns are laid over blocks.  Up to kSlice columns a row is one block's;
// longer ones go to the smallest cluster whose slices fit (a power of two up to eight).  Several
// rows share a block as long as the rows still spread over all SMs.
//
// A thread owns one chunk in rows of up to 384 and two or three above.  What decides is how many warps
// the registers of its columns (x, dy, w, dw and with a bias db) leave room for: a warp too many on
// one of the SM's four schedulers takes registers from all of them, and the sums spill.
//   - two chunks from there to 4096 columns, so that two rows fit a block: 8192 x 3200 RMS 54 -> 48 us,
//     layer fp32 93 -> 65, 8192 x 4096 layer bf16 86 -> 72 (in fp32 with a bias it loses, 105 -> 118,
//     without one it gains, 118 -> 108).  With fewer rows than SMs one chunk is quicker (32 x 4096: 6.6
//     against 6.0 us).
//   - three chunks where two would need sixteen warps beside the one that fills the ring: 8192 x 8192
//     layer 236 -> 142 us in fp32, 143 -> 117 in bf16 (RMS 116 either way).
// The layout does not depend on which outputs are asked for, so leaving out db changes no bit of dw.
struct Plan {
    int cluster, chunks;  // blocks of a row, chunks of a thread
    Shape s;
    int parts;            // blocks or clusters
};

bool is_long(int64_t K) { return K > int64_t(kSlice) * kMaxCluster; }

Plan plan_of(int64_t M, int64_t K, int ex, int ed) {
    Plan p{};
    p.cluster = 1;
    while ((K + p.cluster - 1) / p.cluster > kSlice) p.cluster *= 2;
    const int64_t slice = ((K + p.cluster - 1) / p.cluster + kE - 1) / kE * kE;
    const int64_t chunks = chunks_of(p.cluster > 1 ? slice - (K % kE != 0) : K);  // unaligned: one more
    const int64_t spread = (M + kParts - 1) / kParts;  // rows of a block when all SMs have some
    p.chunks = chunks <= (spread > 1 ? 384 : 513) ? 1 : chunks > 960 && chunks <= 1056 ? 3 : 2;
    Shape& s = p.s;
    s.M = M;
    s.K = K;
    s.slice = static_cast<int>(p.cluster > 1 ? slice : K);
    s.tpr = static_cast<int>(((chunks + p.chunks - 1) / p.chunks + 31) / 32 * 32);
    const int fit = p.cluster > 1 ? 1 : (p.chunks == 1 ? 768 : 608) / s.tpr;
    s.groups = fit < kMaxGroups ? fit : kMaxGroups;
    if (s.groups >= 8 && s.groups * s.tpr == 768) --s.groups;  // room for 80 registers, see below
    if (s.groups > spread) s.groups = static_cast<int>(spread);
    const int64_t batches = (M + s.groups - 1) / s.groups;
    const int most = kParts / p.cluster;
    p.parts = static_cast<int>(batches < most ? batches : most);
    if (K % kE != 0) {
        // rows in step a multiple of eight (see Shape)
        int unit = kE;
        while (unit > 1 && (unit / 2) * s.groups % kE == 0) unit /= 2;
        p.parts = p.parts < unit ? unit : p.parts / unit * unit;
    }
    // a slot: the rows' elements and up to seven on either side
    const int64_t cols = ((p.cluster > 1 ? slice : K * s.groups) + 2 * kE) / kE * kE + kE;
    s.slot_x = static_cast<int>(cols * ex);
    s.slot_d = static_cast<int>(cols * ed);
    const int n = kRingBytes / (s.slot_x + s.slot_d);
    s.stages = n < kMaxStages ? n : kMaxStages;
    return p;
}

size_t smem_of(const Plan& p) {
    size_t ring = static_cast<size_t>(p.s.stages) * (p.s.slot_x + p.s.slot_d);
    const size_t cols = static_cast<size_t>(2) * p.s.groups * p.s.slice * sizeof(float);  // column sums
    if (ring < cols) ring = cols;
    return ((sizeof(Control) + 127) & ~size_t(127)) + ring;
}

constexpr int kSmemMost = 227 * 1024;
static_assert(((sizeof(Control) + 127) & ~size_t(127)) + kRingBytes <= kSmemMost, "shared memory");

int backward_parts(int64_t M, int64_t K) {
    if (!is_long(K)) return plan_of(M, K, 4, 4).parts;  // does not depend on the types
    const int64_t strips = (M + 15) / 16;
    return static_cast<int>(strips < kParts ? strips : kParts);
}

template <typename TX, typename TD, bool EDGE, bool LAYER, bool DB, int CH, int THREADS>
cudaError_t backward_c(const TX* X, const TD* dY, const Plan& p, const BwdArgs& a, cudaStream_t stream) {
    static PerContextOnce attr;
    cudaError_t e = attr.run([] {
        return cudaFuncSetAttribute(norm_backward_kernel<TX, TD, EDGE, LAYER, DB, CH, THREADS>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_backward_kernel<TX, TD, EDGE, LAYER, DB, CH, THREADS>,
                      dim3(static_cast<unsigned>(p.parts * p.cluster)), dim3(p.s.tpr * p.s.groups + 32), smem_of(p), stream,
                      p.cluster > 1 ? dim3(p.cluster, 1, 1) : dim3(kNoCluster), X, dY, a);
}

// The kernel whose limit of threads leaves the most registers: 80 with up to 768, 128 with up to 512,
// 168 with up to 384 (8192 x 7680 layer fp32 at 128 registers 142 us, at the 96 of 640 threads 219).
// Without a bias 96 are enough for rows of whole chunks (up to 80 bytes spill in fp32, up to 160 in
// other rows), and what more there is only lets the compiler move loads (8192 x 7680 RMS: 101 against
// 110 us).
template <typename TX, typename TD, bool EDGE, bool LAYER>
cudaError_t backward_e(const TX* X, const TD* dY, const Plan& p, const BwdArgs& a, cudaStream_t stream) {
    if (a.db != nullptr) {
        if (p.chunks == 1)
            return p.s.tpr * p.s.groups < 768 ? backward_c<TX, TD, EDGE, LAYER, true, 1, 768>(X, dY, p, a, stream)
                                              : backward_c<TX, TD, EDGE, LAYER, true, 1, 800>(X, dY, p, a, stream);
        if (p.chunks == 3) return backward_c<TX, TD, EDGE, LAYER, true, 3, 384>(X, dY, p, a, stream);
        if (p.s.tpr * p.s.groups < 512) return backward_c<TX, TD, EDGE, LAYER, true, 2, 512>(X, dY, p, a, stream);
        return backward_c<TX, TD, EDGE, LAYER, true, 2, 640>(X, dY, p, a, stream);
    }
    if (p.chunks == 1)
        return p.s.tpr * p.s.groups < 768 ? backward_c<TX, TD, EDGE, LAYER, false, 1, 768>(X, dY, p, a, stream)
                                          : backward_c<TX, TD, EDGE, LAYER, false, 1, 800>(X, dY, p, a, stream);
    if (p.chunks == 3) return backward_c<TX, TD, EDGE, LAYER, false, 3, 384>(X, dY, p, a, stream);
    return backward_c<TX, TD, EDGE, LAYER, false, 2, 640>(X, dY, p, a, stream);
}

struct BwdCall {
    const float* w;
    int64_t M, K;
    bool layer;
    float eps;
    void* dx;
    bool dx_bf16;
    float* dw;  // where the kernels leave their sums: partial ones with several parts
    float* db;
    float4* stats;
    int parts;
    int32_t* err;
};

template <typename TX, typename TD>
cudaError_t backward_t(const TX* X, const TD* dY, const BwdCall& c, cudaStream_t stream) {
    const float inv_k = 1.0f / static_cast<float>(c.K);
    if (is_long(c.K)) {
        const LongBwdArgs a{c.w, c.M, c.K, c.layer, c.eps, inv_k, c.dx, c.dx_bf16, c.dw, c.db};
        cudaError_t e = launch_pdl(norm_backward_long_kernel<TX, TD>, dim3(static_cast<unsigned>(c.M)),
                                   dim3(kMaxThreads), 0, stream, dim3(kNoCluster), X, dY, a, c.stats);
        if (e != cudaSuccess || (c.dw == nullptr && c.db == nullptr)) return e;
        const int64_t rows = (c.M + c.parts - 1) / c.parts;
        const int64_t strips = (c.K + 255) / 256;
        return launch_pdl(norm_columns_long_kernel<TX, TD>,
                          dim3(c.parts, static_cast<unsigned>(strips < 65535 ? strips : 65535)), dim3(256), 0, stream,
                          dim3(kNoCluster), X, dY, a, static_cast<const float4*>(c.stats), rows);
    }
    const Plan p = plan_of(c.M, c.K, sizeof(TX), sizeof(TD));
    const WaitTest wt = wait_test();
    const BwdArgs a{p.s, c.w, c.eps, inv_k, c.dx, c.dx_bf16, c.dw, c.db, c.err, wt.wait_ns, wt.stall_after};
    if (c.K % kE == 0)
        return c.layer ? backward_e<TX, TD, false, true>(X, dY, p, a, stream)
                       : backward_e<TX, TD, false, false>(X, dY, p, a, stream);
    return c.layer ? backward_e<TX, TD, true, true>(X, dY, p, a, stream)
                   : backward_e<TX, TD, true, false>(X, dY, p, a, stream);
}

int64_t align16(int64_t n) { return (n + 15) / 16 * 16; }

}  // namespace

cudaError_t launch_norm_forward(const void* X, bool x_bf16, const float* w, const float* b, int64_t M, int64_t K,
                                int kind, float eps, void* Y, bool y_bf16, cudaStream_t stream) {
    const FwdArgs a{w, b, M, K, kind == 1, eps, 1.0f / static_cast<float>(K), Y, y_bf16};
    return x_bf16 ? forward_x(static_cast<const __nv_bfloat16*>(X), a, stream)
                  : forward_x(static_cast<const float*>(X), a, stream);
}

// Partial column sums of dw and db, and the statistics of rows longer than a cluster's slices.
size_t norm_backward_workspace(int64_t M, int64_t K) {
    const int64_t parts = backward_parts(M, K);
    int64_t bytes = parts > 1 ? 2 * align16(parts * K * 4) : 0;
    if (is_long(K)) bytes += 16 * M;
    return static_cast<size_t>(bytes);
}

cudaError_t launch_norm_backward(const void* dY, bool dy_bf16, const void* X, bool x_bf16, const float* w, int64_t M,
                                 int64_t K, int kind, float eps, void* dX, bool dx_bf16, float* dw, float* db,
                                 void* ws, int32_t* err, cudaStream_t stream) {
    const int parts = backward_parts(M, K);
    const int64_t part_bytes = align16(static_cast<int64_t>(parts) * K * 4);
    uint8_t* p = static_cast<uint8_t*>(ws);
    BwdCall c{w, M, K, kind == 1, eps, dX, dx_bf16, dw, db, nullptr, parts, err};
    if (parts > 1) {
        if (dw != nullptr) c.dw = reinterpret_cast<float*>(p);
        if (db != nullptr) c.db = reinterpret_cast<float*>(p + part_bytes);
        p += 2 * part_bytes;
    }
    if (is_long(K)) c.stats = reinterpret_cast<float4*>(p);
    cudaError_t e;
    if (x_bf16) {
        const auto* x = static_cast<const __nv_bfloat16*>(X);
        e = dy_bf16 ? backward_t(x, static_cast<const __nv_bfloat16*>(dY), c, stream)
                    : backward_t(x, static_cast<const float*>(dY), c, stream);
    } else {
        const auto* x = static_cast<const float*>(X);
        e = dy_bf16 ? backward_t(x, static_cast<const __nv_bfloat16*>(dY), c, stream)
                    : backward_t(x, static_cast<const float*>(dY), c, stream);
    }
    if (e != cudaSuccess || parts == 1 || (dw == nullptr && db == nullptr)) return e;
    const dim3 grid(static_cast<unsigned>((K + 31) / 32), dw != nullptr && db != nullptr ? 2 : 1);
    return launch_pdl(norm_reduce_kernel, grid, dim3(32, 32), 0, stream, dim3(kNoCluster),
                      static_cast<const float*>(c.dw), static_cast<const float*>(c.db), parts, K, dw, db);
}

}  // namespace bl
