// rmsnorm.cu -- moe_rmsnorm, moe_rmsnorm_quantize_fp8, moe_rmsnorm_backward.
//
// The root-mean-square norm in front of an MoE layer, with the addition of the
// residual stream fused in front and the e4m3 quantization of the FP8 dispatch
// behind it:
//   h = round(x + residual)                       (stored; h = x without one)
//   r = 1 / sqrt(mean(h^2) + eps),  y = h * r * weight
//   e4m3: scale = max|y| / 448 per block (1 for a zero block), q = e4m3(y / scale)
// The norm is taken of h as it is stored, so that the backward, which only has
// the stored h, is the gradient of exactly this function.  Everything between
// the loads and the one rounding of each output is float32; y itself is never
// rounded to bf16 on the way to e4m3.
//
// Backward, with g = dL/dy and gh the gradient that reaches h past the norm:
//   grad_x = r (g w) - h r^3 mean(g w h) + gh
//   grad_weight = sum over the rows of g h r      (float32, fixed order)
// r is recomputed: h has to be read anyway, and both sums share one reduction.
#include "common.cuh"

namespace moe {
namespace {

constexpr int kChunk = 8;                 // elements a thread moves at a time
constexpr int kMaxThreads = 1024;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kBwdThreads = 256;          // columns of one pass of the element-wise backward
constexpr int kBwdMaxBlocks = 608;        // rows of partial sums of grad_weight

// ------------------------------------------------------------ loads, stores

// Plain (coherent) loads: residual_out may be residual or x themselves.
__device__ __forceinline__ void load8(const uint16_t* p, float* f) {
    const uint4 v = ld_v4(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16lo_to_f32(w[i]);
        f[2 * i + 1] = bf16hi_to_f32(w[i]);
    }
}
__device__ __forceinline__ void load8(const float* p, float* f) {
    const uint4 a = ld_v4(p), b = ld_v4(p + 4);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void store8(uint16_t* p, const float* f) {
    st_v4(p, make_uint4(pack_bf16x2_rn(f[0], f[1]), pack_bf16x2_rn(f[2], f[3]),
                        pack_bf16x2_rn(f[4], f[5]), pack_bf16x2_rn(f[6], f[7])));
}
__device__ __forceinline__ void store8(float* p, const float* f) {
    st_v4(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                        __float_as_uint(f[3])));
    st_v4(p + 4, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                            __float_as_uint(f[7])));
}
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float f) { *p = f32_to_bf16_rn(f); }
__device__ __forceinline__ void store1(float* p, float f) { *p = f; }

// The value as it is stored in the activation type.
__device__ __forceinline__ float as_stored(const uint16_t*, float f) {
    return bf16_to_f32(f32_to_bf16_rn(f));
}
__device__ __forceinline__ float as_stored(const float*, float f) { return f; }

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t q4(const float* f, float s) {
    return e4m3x2(__fdiv_rn(f[0], s), __fdiv_rn(f[1], s)) |
           (e4m3x2(__fdiv_rn(f[2], s), __fdiv_rn(f[3], s)) << 16);
}

// Sum over the block's threads, the same value in each; `s` holds kMaxWarps
// floats, and the caller alternates two of them so that one barrier a row is
// enough.  The order is fixed by the block size.
__device__ __forceinline__ float block_sum(float v, float* s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return v;
    if (lane_id() == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = int(lane_id()) < nw ? s[lane_id()] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    return t;
}

// ------------------------------------------------------------------ forward

struct NormArgs {
    const void* x;
    const void* residual;     // NULL: none
    const void* weight;
    void* h_out;              // NULL without a residual
    void* out;                // y, or e4m3 codes
    float* scales;            // e4m3: [T, H/block]
    int64_t T;
    int64_t H;
    float eps;
    int lanes;                // e4m3: lanes that share a block (block / 8)
};

// One block a row, V chunks a thread held in registers between the two passes
// over the row.
template <typename X, typename W, int V, bool kQuant>
__global__ void __launch_bounds__(kMaxThreads)
rmsnorm_kernel(const NormArgs a) {
    __shared__ float s_part[2][kMaxWarps];
    const int chunks = int(a.H / kChunk);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
        const X* x = static_cast<const X*>(a.x) + row * a.H;
        float h[V][kChunk];
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            if (c < chunks) load8(x + c * kChunk, h[v]);
        }
        if (a.residual) {
            const X* res = static_cast<const X*>(a.residual) + row * a.H;
            X* ho = static_cast<X*>(a.h_out) + row * a.H;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = threadIdx.x + v * blockDim.x;
                if (c < chunks) {
                    float r[kChunk];
                    load8(res + c * kChunk, r);
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) h[v][i] = as_stored(x, h[v][i] + r[i]);
                    store8(ho + c * kChunk, h[v]);
                }
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            if (c < chunks) {
#pragma unroll
                for (int i = 0; i < kChunk; ++i) ss = fmaf(h[v][i], h[v][i], ss);
            }
        }
        const float r = rsqrtf(block_sum(ss, s_part[turn]) / float(a.H) + a.eps);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            float y[kChunk];
            if (c < chunks) {
                float w[kChunk];
                load8(static_cast<const W*>(a.weight) + c * kChunk, w);
#pragma unroll
                for (int i = 0; i < kChunk; ++i) y[i] = h[v][i] * r * w[i];
            }
            if (!kQuant) {
                if (c < chunks) store8(static_cast<X*>(a.out) + row * a.H + c * kChunk, y);
            } else {
                // the magnitude bits order like the magnitudes; a block's lanes
                // are consecutive and whole blocks fit a warp (block <= 256)
                uint32_t m = 0;
                if (c < chunks) {
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
                }
                for (int o = a.lanes >> 1; o > 0; o >>= 1)
                    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                const float amax = __uint_as_float(m);
                const float s = amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
                if (c < chunks) {
                    uint2* q = reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + row * a.H);
                    q[c] = make_uint2(q4(y, s), q4(y + 4, s));
                    if (c % a.lanes == 0) a.scales[row * (chunks / a.lanes) + c / a.lanes] = s;
                }
            }
        }
    }
}

// Rows that no 16-byte vector fits, or too long for the registers: two passes
// over the row, element by element; the second reads back what this thread
// wrote or read in the first.
template <typename X, typename W>
__global__ void __launch_bounds__(kMaxThreads)
rmsnorm_elements_kernel(const NormArgs a) {
    __shared__ float s_part[2][kMaxWarps];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
        const X* x = static_cast<const X*>(a.x) + row * a.H;
        const X* res = a.residual ? static_cast<const X*>(a.residual) + row * a.H : nullptr;
        X* ho = a.residual ? static_cast<X*>(a.h_out) + row * a.H : nullptr;
        float ss = 0.0f;
        for (int64_t i = threadIdx.x; i < a.H; i += blockDim.x) {
            float h = load1(x + i);
            if (res) {
                h = as_stored(x, h + load1(res + i));
                store1(ho + i, h);
            }
            ss = fmaf(h, h, ss);
        }
        const float r = rsqrtf(block_sum(ss, s_part[turn]) / float(a.H) + a.eps);
        const X* hs = res ? ho : x;
        X* y = static_cast<X*>(a.out) + row * a.H;
        for (int64_t i = threadIdx.x; i < a.H; i += blockDim.x)
            store1(y + i, load1(hs + i) * r * load1(static_cast<const W*>(a.weight) + i));
    }
}

// ----------------------------------------------------------------- backward

struct BwdArgs {
    const void* g;
    const void* gh;           // NULL: none
    const void* h;
    const void* weight;
    void* gx;
    float* partial;           // [gridDim.x, H]
    int64_t T;
    int64_t H;
    float eps;
};

// Sums of two values over the block at once.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2* s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    const int nw = blockDim.x >> 5;
    if (nw == 1) return make_float2(a, b);
    if (lane_id() == 0) s[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    float2 t = int(lane_id()) < nw ? s[lane_id()] : make_float2(0.0f, 0.0f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        t.x += __shfl_xor_sync(0xFFFFFFFFu, t.x, o);
        t.y += __shfl_xor_sync(0xFFFFFFFFu, t.y, o);
    }
    return t;
}

// Each block walks rows blockIdx.x, + gridDim.x, ... and keeps its columns'
// share of grad_weight in registers; the shares are summed over the blocks, in
// order, by rmsnorm_grad_weight_kernel.
template <typename X, typename W, int V>
__global__ void __launch_bounds__(kMaxThreads)
rmsnorm_backward_kernel(const BwdArgs a) {
    __shared__ float2 s_part[2][kMaxWarps];
    const int chunks = int(a.H / kChunk);
    float dw[V][kChunk] = {};
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
        const X* hp = static_cast<const X*>(a.h) + row * a.H;
        const X* gp = static_cast<const X*>(a.g) + row * a.H;
        float h[V][kChunk], g[V][kChunk];
        float ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            if (c < chunks) {
                load8(hp + c * kChunk, h[v]);
                load8(gp + c * kChunk, g[v]);
                float w[kChunk];
                load8(static_cast<const W*>(a.weight) + c * kChunk, w);
#pragma unroll
                for (int i = 0; i < kChunk; ++i) {
                    ss = fmaf(h[v][i], h[v][i], ss);
                    dot = fmaf(g[v][i] * w[i], h[v][i], dot);
                }
            }
        }
        const float2 t = block_sum2(ss, dot, s_part[turn]);
        const float r = rsqrtf(t.x / float(a.H) + a.eps);
        const float b = r * r * r * (t.y / float(a.H));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            if (c < chunks) {
                float w[kChunk], o[kChunk];
                load8(static_cast<const W*>(a.weight) + c * kChunk, w);
#pragma unroll
                for (int i = 0; i < kChunk; ++i) {
                    dw[v][i] = fmaf(g[v][i], h[v][i] * r, dw[v][i]);
                    o[i] = r * (g[v][i] * w[i]) - h[v][i] * b;
                }
                if (a.gh) {
                    float e[kChunk];
                    load8(static_cast<const X*>(a.gh) + row * a.H + c * kChunk, e);
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) o[i] += e[i];
                }
                store8(static_cast<X*>(a.gx) + row * a.H + c * kChunk, o);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = threadIdx.x + v * blockDim.x;
        if (c < chunks) store8(a.partial + int64_t(blockIdx.x) * a.H + c * kChunk, dw[v]);
    }
}

// Any H and alignment.  The block's share of grad_weight lives in its row of
// `partial`: every column is read and written by one thread only.
template <typename X, typename W>
__global__ void __launch_bounds__(kBwdThreads)
rmsnorm_backward_elements_kernel(const BwdArgs a) {
    __shared__ float2 s_part[2][kMaxWarps];
    float* part = a.partial + int64_t(blockIdx.x) * a.H;
    for (int64_t i = threadIdx.x; i < a.H; i += blockDim.x) part[i] = 0.0f;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
        const X* h = static_cast<const X*>(a.h) + row * a.H;
        const X* g = static_cast<const X*>(a.g) + row * a.H;
        float ss = 0.0f, dot = 0.0f;
        for (int64_t i = threadIdx.x; i < a.H; i += blockDim.x) {
            const float hv = load1(h + i);
            ss = fmaf(hv, hv, ss);
            dot = fmaf(load1(g + i) * load1(static_cast<const W*>(a.weight) + i), hv, dot);
        }
        const float2 t = block_sum2(ss, dot, s_part[turn]);
        const float r = rsqrtf(t.x / float(a.H) + a.eps);
        const float b = r * r * r * (t.y / float(a.H));
        for (int64_t i = threadIdx.x; i < a.H; i += blockDim.x) {
            const float hv = load1(h + i), gv = load1(g + i);
            part[i] = fmaf(gv, hv * r, part[i]);
            float o = r * (gv * load1(static_cast<const W*>(a.weight) + i)) - hv * b;
            if (a.gh) o += load1(static_cast<const X*>(a.gh) + row * a.H + i);
            store1(static_cast<X*>(a.gx) + row * a.H + i, o);
        }
    }
}

// grad_weight[c] = sum over the blocks' shares, in the blocks' order.
__global__ void rmsnorm_grad_weight_kernel(const float* __restrict__ partial, int blocks,
                                           int64_t H, float* __restrict__ gw) {
    const int64_t c = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (c >= H) return;
    float s = 0.0f;
    for (int b = 0; b < blocks; ++b) s += partial[int64_t(b) * H + c];
    gw[c] = s;
}

// --------------------------------------------------------------------- host

// Threads a row for V chunks each.
int row_threads(int64_t H, int V) {
    const int64_t need = (H / kChunk + V - 1) / V;
    return int((need + 31) / 32 * 32);
}

// The smallest number of chunks a thread whose block fits kMaxThreads; 0: the
// row does not fit.
int row_chunks(int64_t H) {
    for (int V = 1; V <= 4; V *= 2)
        if ((H / kChunk + V - 1) / V <= kMaxThreads) return V;
    return 0;
}

bool vectors_fit(int64_t H, std::initializer_list<const void*> ptrs) {
    if (H % kChunk != 0 || row_chunks(H) == 0) return false;
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return false;
    return true;
}

unsigned row_blocks(int64_t T) { return unsigned(min64(T, int64_t(1) << 20)); }

template <typename X, typename W, bool kQuant>
moe_status_t launch_norm(const NormArgs& a, bool vectors, cudaStream_t s) {
    const unsigned grid = row_blocks(a.T);
    if (!vectors) {
        rmsnorm_elements_kernel<X, W><<<grid, 256, 0, s>>>(a);
        return launch_status();
    }
    switch (row_chunks(a.H)) {
        case 1: rmsnorm_kernel<X, W, 1, kQuant><<<grid, row_threads(a.H, 1), 0, s>>>(a); break;
        case 2: rmsnorm_kernel<X, W, 2, kQuant><<<grid, row_threads(a.H, 2), 0, s>>>(a); break;
        default: rmsnorm_kernel<X, W, 4, kQuant><<<grid, row_threads(a.H, 4), 0, s>>>(a); break;
    }
    return launch_status();
}

template <bool kQuant>
moe_status_t dispatch_norm(const NormArgs& a, int dtype, int wdtype, bool vectors,
                           cudaStream_t s) {
    if (dtype == MOE_BF16)
        return wdtype == MOE_BF16 ? launch_norm<uint16_t, uint16_t, kQuant>(a, vectors, s)
                                  : launch_norm<uint16_t, float, kQuant>(a, vectors, s);
    return wdtype == MOE_BF16 ? launch_norm<float, uint16_t, kQuant>(a, vectors, s)
                              : launch_norm<float, float, kQuant>(a, vectors, s);
}

template <typename X, typename W>
moe_status_t launch_backward(const BwdArgs& a, unsigned grid, bool vectors, cudaStream_t s) {
    if (!vectors) {
        rmsnorm_backward_elements_kernel<X, W><<<grid, kBwdThreads, 0, s>>>(a);
        return launch_status();
    }
    switch (row_chunks(a.H)) {
        case 1: rmsnorm_backward_kernel<X, W, 1><<<grid, row_threads(a.H, 1), 0, s>>>(a); break;
        case 2: rmsnorm_backward_kernel<X, W, 2><<<grid, row_threads(a.H, 2), 0, s>>>(a); break;
        default: rmsnorm_backward_kernel<X, W, 4><<<grid, row_threads(a.H, 4), 0, s>>>(a); break;
    }
    return launch_status();
}

// Shapes and types that all three calls share.
moe_status_t check_norm(int dtype, int wdtype, int64_t T, int64_t H, float eps) {
    if (!dtype_ok(dtype) || !dtype_ok(wdtype) || T < 0 || H < 0 || !(eps >= 0.0f))
        return MOE_ERR_INVALID_ARG;
    if (T >= (int64_t(1) << 31) || H * int64_t(elem_size(moe_dtype_t(dtype))) >= (int64_t(1) << 31))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int backward_blocks(int64_t T) { return int(min64(T, kBwdMaxBlocks)); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_rmsnorm(const void* x, const void* residual, moe_dtype_t dtype,
                                    const void* weight, moe_dtype_t weight_dtype, int64_t T,
                                    int64_t H, float eps, void* residual_out, void* out,
                                    void* stream) {
    MOE_TRACE(__func__);
    const moe_status_t st = check_norm(dtype, weight_dtype, T, H, eps);
    if (st != MOE_OK) return st;
    if (T == 0 || H == 0) return MOE_OK;
    if (!x || !weight || !out || (residual && !residual_out)) return MOE_ERR_INVALID_ARG;
    if (!residual) residual_out = nullptr;
    const NormArgs a{x, residual, weight, residual_out, out, nullptr, T, H, eps, 0};
    const bool vectors = vectors_fit(H, {x, residual, weight, residual_out, out});
    return dispatch_norm<false>(a, dtype, weight_dtype, vectors, static_cast<cudaStream_t>(stream));
}

extern "C" moe_status_t moe_rmsnorm_quantize_fp8(const void* x, const void* residual,
                                                 moe_dtype_t dtype, const void* weight,
                                                 moe_dtype_t weight_dtype, int64_t T, int64_t H,
                                                 float eps, int block, void* residual_out,
                                                 void* x_q, float* scales, void* stream) {
    MOE_TRACE(__func__);
    const moe_status_t st = check_norm(dtype, weight_dtype, T, H, eps);
    if (st != MOE_OK) return st;
    if (block != 32 && block != 64 && block != 128 && block != 256) return MOE_ERR_UNSUPPORTED;
    if (H % block != 0) return MOE_ERR_INVALID_ARG;
    if (T == 0 || H == 0) return MOE_OK;
    if (row_chunks(H) == 0) return MOE_ERR_UNSUPPORTED;
    if (!x || !weight || !x_q || !scales || (residual && !residual_out)) return MOE_ERR_INVALID_ARG;
    if (!residual) residual_out = nullptr;
    if (!vectors_fit(H, {x, residual, weight, residual_out}) ||
        (reinterpret_cast<uintptr_t>(x_q) & 7u) || (reinterpret_cast<uintptr_t>(scales) & 3u))
        return MOE_ERR_INVALID_ARG;
    const NormArgs a{x, residual, weight, residual_out, x_q, scales, T, H, eps, block / kChunk};
    return dispatch_norm<true>(a, dtype, weight_dtype, true, static_cast<cudaStream_t>(stream));
}

extern "C" moe_status_t moe_rmsnorm_backward_workspace_size(int64_t T, int64_t H, size_t* bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_norm(MOE_F32, MOE_F32, T, H, 0.0f);
    if (st != MOE_OK) return st;
    *bytes = align_up(size_t(backward_blocks(T)) * size_t(H) * 4, kWsAlign) + kWsAlign;
    return MOE_OK;
}

extern "C" moe_status_t moe_rmsnorm_backward(const void* grad_y, const void* grad_h, const void* h,
                                             moe_dtype_t dtype, const void* weight,
                                             moe_dtype_t weight_dtype, int64_t T, int64_t H,
                                             float eps, void* grad_x, float* grad_weight,
                                             void* workspace, size_t workspace_bytes,
                                             void* stream) {
    MOE_TRACE(__func__);
    const moe_status_t st = check_norm(dtype, weight_dtype, T, H, eps);
    if (st != MOE_OK) return st;
    if (H == 0) return MOE_OK;
    if (!grad_weight) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0)
        return cudaMemsetAsync(grad_weight, 0, size_t(H) * 4, s) == cudaSuccess ? MOE_OK
                                                                               : MOE_ERR_CUDA;
    if (!grad_y || !h || !weight || !grad_x) return MOE_ERR_INVALID_ARG;
    size_t need = 0;
    const moe_status_t sz = moe_rmsnorm_backward_workspace_size(T, H, &need);
    if (sz != MOE_OK) return sz;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) ||
        workspace_bytes < need)
        return MOE_ERR_WORKSPACE;
    const unsigned grid = unsigned(backward_blocks(T));
    const BwdArgs a{grad_y, grad_h, h, weight, grad_x, static_cast<float*>(workspace), T, H, eps};
    const bool vectors = vectors_fit(H, {grad_y, grad_h, h, weight, grad_x});
    moe_status_t r;
    if (dtype == MOE_BF16)
        r = weight_dtype == MOE_BF16 ? launch_backward<uint16_t, uint16_t>(a, grid, vectors, s)
                                     : launch_backward<uint16_t, float>(a, grid, vectors, s);
    else
        r = weight_dtype == MOE_BF16 ? launch_backward<float, uint16_t>(a, grid, vectors, s)
                                     : launch_backward<float, float>(a, grid, vectors, s);
    if (r != MOE_OK) return r;
    rmsnorm_grad_weight_kernel<<<unsigned((H + 127) / 128), 128, 0, s>>>(a.partial, int(grid), H,
                                                                         grad_weight);
    return launch_status();
}
