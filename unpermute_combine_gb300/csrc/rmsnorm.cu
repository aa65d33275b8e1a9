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
#include "pipeline.cuh"

namespace moe {
namespace {

constexpr int kChunk = 8;                 // elements a thread moves at a time
constexpr int kMaxThreads = 1024;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kWarpRows = 8;              // rows of a block whose rows are a warp each
constexpr int kBwdMaxBlocks = 608;        // rows of partial sums of grad_weight
constexpr int kMaxTeams = 15;             // rows that a block of the backward works on at once
                                          // (a named barrier each, and 16 of them)
constexpr int kMaxRing = 8;               // rows that a team has in shared memory
constexpr int kRingBytes = 200 * 1024;

// ------------------------------------------------------------ loads, stores

// A chunk as it is stored: one 16-byte word of bf16, two of float32.  Rows wait in
// this form, which takes half the registers of their values.
template <typename X>
struct Raw {
    uint4 v[sizeof(X) / 2];
};

// Plain (coherent) loads: residual_out may be residual or x themselves.
template <typename X>
__device__ __forceinline__ Raw<X> load_raw(const X* p) {
    Raw<X> r;
#pragma unroll
    for (int i = 0; i < int(sizeof(X) / 2); ++i) r.v[i] = ld_v4(p + i * (16 / sizeof(X)));
    return r;
}
template <typename X>
__device__ __forceinline__ Raw<X> shared_raw(const X* p) {
    Raw<X> r;
#pragma unroll
    for (int i = 0; i < int(sizeof(X) / 2); ++i)
        r.v[i] = *reinterpret_cast<const uint4*>(p + i * (16 / sizeof(X)));
    return r;
}
template <typename X>
__device__ __forceinline__ void store_raw(X* p, const Raw<X>& r) {
#pragma unroll
    for (int i = 0; i < int(sizeof(X) / 2); ++i) st_v4(p + i * (16 / sizeof(X)), r.v[i]);
}
__device__ __forceinline__ void values(const Raw<uint16_t>& r, float* f) {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16lo_to_f32(w[i]);
        f[2 * i + 1] = bf16hi_to_f32(w[i]);
    }
}
__device__ __forceinline__ void values(const Raw<float>& r, float* f) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(r.v[i].x);
        f[4 * i + 1] = __uint_as_float(r.v[i].y);
        f[4 * i + 2] = __uint_as_float(r.v[i].z);
        f[4 * i + 3] = __uint_as_float(r.v[i].w);
    }
}
// Rounded to the stored type (float: as it is).
__device__ __forceinline__ Raw<uint16_t> rounded(const uint16_t*, const float* f) {
    Raw<uint16_t> r;
    r.v[0] = make_uint4(pack_bf16x2_rn(f[0], f[1]), pack_bf16x2_rn(f[2], f[3]),
                        pack_bf16x2_rn(f[4], f[5]), pack_bf16x2_rn(f[6], f[7]));
    return r;
}
__device__ __forceinline__ Raw<float> rounded(const float*, const float* f) {
    Raw<float> r;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        r.v[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                            __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
    return r;
}
template <typename X>
__device__ __forceinline__ void load8(const X* p, float* f) { values(load_raw(p), f); }
template <typename X>
__device__ __forceinline__ void shared8(const X* p, float* f) { values(shared_raw(p), f); }
template <typename X>
__device__ __forceinline__ void store8(X* p, const float* f) { store_raw(p, rounded(p, f)); }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float f) { *p = f32_to_bf16_rn(f); }
__device__ __forceinline__ void store1(float* p, float f) { *p = f; }

// The value as it is stored.
__device__ __forceinline__ float as_stored(const uint16_t*, float f) {
    return bf16_to_f32(f32_to_bf16_rn(f));
}
__device__ __forceinline__ float as_stored(const float*, float f) { return f; }

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
// four floats -> four e4m3 bytes of f / s.  inv = 1 / s: a product costs a tenth of
// a division, and is off by a float ulp, where y is by several.
__device__ __forceinline__ uint32_t q4(const float* f, float inv) {
    return e4m3x2(f[0] * inv, f[1] * inv) | (e4m3x2(f[2] * inv, f[3] * inv) << 16);
}
// The same by division, for a scale whose reciprocal overflows.
__device__ __forceinline__ uint32_t q4_divided(const float* f, float s) {
    return e4m3x2(__fdiv_rn(f[0], s), __fdiv_rn(f[1], s)) |
           (e4m3x2(__fdiv_rn(f[2], s), __fdiv_rn(f[3], s)) << 16);
}

// Sum over a row's threads (blockDim.x of them: a warp, or the block), the same
// value in each; `s` holds kMaxWarps floats, and the caller alternates two of them
// so that one barrier a row is enough.  The order is fixed by the block size.
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

// A row to blockDim.x threads (a warp, blockDim.y rows a block; or the block), V
// chunks a thread held in registers between the two passes over the row.
template <typename X, typename W, int V, bool kQuant>
__global__ void __launch_bounds__(V >= 4 ? kMaxThreads / 2 : kMaxThreads)
rmsnorm_kernel(const NormArgs a) {
    __shared__ float s_part[2][kMaxWarps];
    const int chunks = int(a.H / kChunk);
    int turn = 0;
    for (int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y; row < a.T;
         row += int64_t(gridDim.x) * blockDim.y, turn ^= 1) {
        const X* x = static_cast<const X*>(a.x) + row * a.H;
        Raw<X> h[V];
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            if (c < chunks) h[v] = load_raw(x + c * kChunk);
        }
        if (a.residual) {
            const X* res = static_cast<const X*>(a.residual) + row * a.H;
            X* ho = static_cast<X*>(a.h_out) + row * a.H;
            Raw<X> add[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = threadIdx.x + v * blockDim.x;
                if (c < chunks) add[v] = load_raw(res + c * kChunk);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = threadIdx.x + v * blockDim.x;
                if (c < chunks) {
                    float f[kChunk], g[kChunk];
                    values(h[v], f);
                    values(add[v], g);
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) f[i] += g[i];
                    h[v] = rounded(x, f);
                    store_raw(ho + c * kChunk, h[v]);
                }
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            if (c < chunks) {
                float f[kChunk];
                values(h[v], f);
#pragma unroll
                for (int i = 0; i < kChunk; ++i) ss = fmaf(f[i], f[i], ss);
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
                values(h[v], y);
#pragma unroll
                for (int i = 0; i < kChunk; ++i) y[i] = y[i] * r * w[i];
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
                    const float inv = __frcp_rn(s);
                    q[c] = s >= 0x1p-126f ? make_uint2(q4(y, inv), q4(y + 4, inv))
                                          : make_uint2(q4_divided(y, s), q4_divided(y + 4, s));
                    if (c % a.lanes == 0) a.scales[row * (chunks / a.lanes) + c / a.lanes] = s;
                }
            }
        }
    }
}

// The same for rows that no 16-byte vector fits: elements threadIdx.x, +
// blockDim.x, ..., eight of them a thread, in registers.
template <typename X, typename W>
__global__ void __launch_bounds__(kMaxThreads)
rmsnorm_odd_kernel(const NormArgs a) {
    __shared__ float s_part[2][kMaxWarps];
    const int H = int(a.H);
    int turn = 0;
    for (int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y; row < a.T;
         row += int64_t(gridDim.x) * blockDim.y, turn ^= 1) {
        const X* x = static_cast<const X*>(a.x) + row * a.H;
        float h[kChunk], ss = 0.0f;
#pragma unroll
        for (int v = 0; v < kChunk; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            h[v] = c < H ? load1(x + c) : 0.0f;
        }
        if (a.residual) {
            const X* res = static_cast<const X*>(a.residual) + row * a.H;
            float r[kChunk];
#pragma unroll
            for (int v = 0; v < kChunk; ++v) {
                const int c = threadIdx.x + v * blockDim.x;
                r[v] = c < H ? load1(res + c) : 0.0f;
            }
#pragma unroll
            for (int v = 0; v < kChunk; ++v) {
                const int c = threadIdx.x + v * blockDim.x;
                h[v] = as_stored(x, h[v] + r[v]);
                if (c < H) store1(static_cast<X*>(a.h_out) + row * a.H + c, h[v]);
            }
        }
#pragma unroll
        for (int v = 0; v < kChunk; ++v) ss = fmaf(h[v], h[v], ss);
        const float r = rsqrtf(block_sum(ss, s_part[turn]) / float(a.H) + a.eps);
#pragma unroll
        for (int v = 0; v < kChunk; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            if (c < H)
                store1(static_cast<X*>(a.out) + row * a.H + c,
                       h[v] * r * load1(static_cast<const W*>(a.weight) + c));
        }
    }
}

// Rows too long for the registers: two passes over the row, element by element;
// the second reads back what this thread wrote or read in the first.
template <typename X, typename W>
__global__ void __launch_bounds__(kMaxThreads)
rmsnorm_long_kernel(const NormArgs a) {
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
    int ring;                 // rows that a team has in shared memory
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

// Rows in teams of blockDim.x threads, blockDim.y teams a block.  A team has a ring
// of rows in shared memory (h, grad_y and grad_h of each), which bulk copies fill
// rows ahead, so that reading goes on while a row waits for its sums; V chunks a
// thread.  The columns' shares of grad_weight stay in registers over all rows of
// the block; its teams' shares are added up at the end, in order, and the blocks'
// by rmsnorm_grad_weight_kernel.
template <typename X, typename W, int V>
__global__ void __launch_bounds__(kMaxThreads)
rmsnorm_backward_kernel(const BwdArgs a, uint32_t* status) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[kMaxTeams][kMaxRing];
    __shared__ float2 s_part[2][kMaxWarps];
    __shared__ volatile int s_failed[kMaxTeams];
    const int team = threadIdx.y, teams = blockDim.y, nw = blockDim.x >> 5;
    const int warp = threadIdx.x >> 5;
    const int chunks = int(a.H / kChunk);
    const uint32_t row_bytes = uint32_t(a.H) * sizeof(X);
    const uint32_t slot_bytes = row_bytes * (a.gh ? 3 : 2);
    uint8_t* ring = smem + size_t(team) * a.ring * slot_bytes;
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.ring; ++i) mbar_init(smem_addr(&full[team][i]), 1);
        mbar_fence_init();
    }
    if (threadIdx.x == 0) s_failed[team] = 0;
    __syncthreads();
    const int64_t first = int64_t(blockIdx.x) * teams + team, step = int64_t(gridDim.x) * teams;
    const int64_t rows = first < a.T ? (a.T - first + step - 1) / step : 0;
    auto fill = [&](int64_t n) {                           // one thread: the team's n-th row
        const int slot = int(n % a.ring);
        const uint32_t bar = smem_addr(&full[team][slot]), dst = smem_addr(ring + slot * slot_bytes);
        const int64_t at = (first + n * step) * a.H;
        mbar_expect_tx(bar, slot_bytes);
        bulk_load(dst, static_cast<const X*>(a.h) + at, row_bytes, bar);
        bulk_load(dst + row_bytes, static_cast<const X*>(a.g) + at, row_bytes, bar);
        if (a.gh) bulk_load(dst + 2 * row_bytes, static_cast<const X*>(a.gh) + at, row_bytes, bar);
    };
    if (threadIdx.x == 0)
        for (int64_t n = 0; n < rows && n < a.ring; ++n) fill(n);
    float dw[V][kChunk] = {};
    for (int64_t n = 0; n < rows; ++n) {
        const int slot = int(n % a.ring);
        if (!mbar_wait(smem_addr(&full[team][slot]), uint32_t(n / a.ring) & 1u)) s_failed[team] = 1;
        const X* h = reinterpret_cast<const X*>(ring + slot * slot_bytes);
        const X* g = reinterpret_cast<const X*>(ring + slot * slot_bytes + row_bytes);
        float ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            if (c < chunks) {
                float hv[kChunk], gv[kChunk], w[kChunk];
                shared8(h + c * kChunk, hv);
                shared8(g + c * kChunk, gv);
                load8(static_cast<const W*>(a.weight) + c * kChunk, w);
#pragma unroll
                for (int i = 0; i < kChunk; ++i) {
                    ss = fmaf(hv[i], hv[i], ss);
                    dot = fmaf(gv[i] * w[i], hv[i], dot);
                }
            }
        }
        // over the team: shuffles, then its warps' sums by way of shared memory
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
            dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
        }
        if (nw > 1) {
            float2* part = s_part[n & 1] + team * nw;
            if (lane_id() == 0) part[warp] = make_float2(ss, dot);
            asm volatile("bar.sync %0, %1;" :: "r"(team + 1), "r"(blockDim.x) : "memory");
            const float2 t = int(lane_id()) < nw ? part[lane_id()] : make_float2(0.0f, 0.0f);
            ss = t.x;
            dot = t.y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
            }
        }
        __syncwarp();
        if (s_failed[team]) {                              // the same for the whole team here
            if (threadIdx.x == 0)                          // none of its copies stays in flight
                for (int64_t m = n + 1; m < n + a.ring && m < rows; ++m)
                    mbar_wait(smem_addr(&full[team][m % a.ring]), uint32_t(m / a.ring) & 1u);
            break;
        }
        const float r = rsqrtf(ss / float(a.H) + a.eps);
        const float b = r * r * r * (dot / float(a.H));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            if (c < chunks) {
                float hv[kChunk], gv[kChunk], w[kChunk], o[kChunk];
                shared8(h + c * kChunk, hv);
                shared8(g + c * kChunk, gv);
                load8(static_cast<const W*>(a.weight) + c * kChunk, w);
#pragma unroll
                for (int i = 0; i < kChunk; ++i) {
                    dw[v][i] = fmaf(gv[i], hv[i] * r, dw[v][i]);
                    o[i] = r * (gv[i] * w[i]) - hv[i] * b;
                }
                if (a.gh) {
                    float e[kChunk];
                    shared8(h + 2 * a.H + c * kChunk, e);
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) o[i] += e[i];
                }
                store8(static_cast<X*>(a.gx) + (first + n * step) * a.H + c * kChunk, o);
            }
        }
        // the row has been read by the whole team: its slot takes another
        if (nw > 1)
            asm volatile("bar.sync %0, %1;" :: "r"(team + 1), "r"(blockDim.x) : "memory");
        else
            __syncwarp();
        if (threadIdx.x == 0 && n + a.ring < rows) fill(n + a.ring);
    }
    __syncthreads();
    if (threadIdx.x == 0 && s_failed[team]) atomicExch(status, uint32_t(MOE_ERR_TIMEOUT));
    // the teams' shares one after the other, in the ring's place
    float* sum = reinterpret_cast<float*>(smem);
    for (int t = 0; t < teams; ++t) {
        if (t == team) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = threadIdx.x + v * blockDim.x;
                if (c < chunks) {
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) {
                        if (t > 0) dw[v][i] += sum[i * chunks + c];
                        if (t + 1 < teams) sum[i * chunks + c] = dw[v][i];
                    }
                    if (t + 1 == teams) store8(a.partial + int64_t(blockIdx.x) * a.H + c * kChunk, dw[v]);
                }
            }
        }
        __syncthreads();
    }
}

// Rows that no 16-byte vector fits: elements threadIdx.x, + blockDim.x, ..., eight
// of them a thread; the next row's are loaded while this one's are worked on.
template <typename X, typename W>
__global__ void __launch_bounds__(kMaxThreads)
rmsnorm_backward_odd_kernel(const BwdArgs a) {
    __shared__ float2 s_part[2][kMaxWarps];
    const int H = int(a.H);
    float dw[kChunk] = {}, h[kChunk], g[kChunk];
    auto load = [&](int64_t row, float* hv, float* gv) {
#pragma unroll
        for (int v = 0; v < kChunk; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            hv[v] = gv[v] = 0.0f;
            if (c < H) {
                hv[v] = load1(static_cast<const X*>(a.h) + row * a.H + c);
                gv[v] = load1(static_cast<const X*>(a.g) + row * a.H + c);
            }
        }
    };
    int turn = 0;
    int64_t row = blockIdx.x;
    if (row < a.T) load(row, h, g);
    for (; row < a.T; row += gridDim.x, turn ^= 1) {
        float e[kChunk] = {}, hn[kChunk], gn[kChunk], ss = 0.0f, dot = 0.0f;
        if (a.gh) {
#pragma unroll
            for (int v = 0; v < kChunk; ++v) {
                const int c = threadIdx.x + v * blockDim.x;
                if (c < H) e[v] = load1(static_cast<const X*>(a.gh) + row * a.H + c);
            }
        }
        if (row + gridDim.x < a.T) load(row + gridDim.x, hn, gn);
#pragma unroll
        for (int v = 0; v < kChunk; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            ss = fmaf(h[v], h[v], ss);
            if (c < H) dot = fmaf(g[v] * load1(static_cast<const W*>(a.weight) + c), h[v], dot);
        }
        const float2 t = block_sum2(ss, dot, s_part[turn]);
        const float r = rsqrtf(t.x / float(a.H) + a.eps);
        const float b = r * r * r * (t.y / float(a.H));
#pragma unroll
        for (int v = 0; v < kChunk; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            dw[v] = fmaf(g[v], h[v] * r, dw[v]);
            if (c < H)
                store1(static_cast<X*>(a.gx) + row * a.H + c,
                       r * (g[v] * load1(static_cast<const W*>(a.weight) + c)) - h[v] * b + e[v]);
            h[v] = hn[v];
            g[v] = gn[v];
        }
    }
#pragma unroll
    for (int v = 0; v < kChunk; ++v) {
        const int c = threadIdx.x + v * blockDim.x;
        if (c < H) a.partial[int64_t(blockIdx.x) * a.H + c] = dw[v];
    }
}

// Rows too long for the registers or the ring.  The block's share of grad_weight
// lives in its row of `partial`: every column is read and written by one thread
// only.
template <typename X, typename W>
__global__ void __launch_bounds__(kMaxThreads)
rmsnorm_backward_long_kernel(const BwdArgs a) {
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

// grad_weight[c] = sum over the blocks' shares: kSumGroups threads a column, each
// every kSumGroups-th share, and their sums in order.
constexpr int kSumCols = 32, kSumGroups = 16;

__global__ void __launch_bounds__(kSumCols * kSumGroups)
rmsnorm_grad_weight_kernel(const float* partial, int blocks, int64_t H, float* __restrict__ gw) {
    __shared__ float s_sum[kSumGroups][kSumCols];
    const int64_t c = int64_t(blockIdx.x) * kSumCols + threadIdx.x;
    wait_for_predecessor();
    float s = 0.0f;
    if (c < H) {
#pragma unroll 8
        for (int b = threadIdx.y; b < blocks; b += kSumGroups) s += __ldcg(partial + int64_t(b) * H + c);
    }
    s_sum[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < H) {
        for (int g = 1; g < kSumGroups; ++g) s += s_sum[g][threadIdx.x];
        gw[c] = s;
    }
}

// --------------------------------------------------------------------- host

int warps_up(int64_t n) { return int((n + 31) / 32 * 32); }

// The smallest number of chunks a thread whose block fits kMaxThreads; 0: the row
// does not fit.
int row_chunks(int64_t H) {
    if (H / kChunk <= kMaxThreads) return 1;
    if (H / kChunk <= 2 * kMaxThreads) return 2;
    return H / kChunk <= 8 * (kMaxThreads / 2) ? 8 : 0;
}

// Rows of at most kMaxThreads * kChunk elements are held by threads of eight.
bool odd_fits(int64_t H) { return H <= int64_t(kMaxThreads) * kChunk; }

bool vectors_fit(int64_t H, std::initializer_list<const void*> ptrs) {
    if (H % kChunk != 0) return false;
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return false;
    return true;
}

template <typename X, typename W, bool kQuant>
moe_status_t launch_norm(const NormArgs& a, bool vectors, cudaStream_t s) {
    const auto grid = [&](int rows) { return unsigned(min64((a.T + rows - 1) / rows, int64_t(1) << 20)); };
    if (!vectors && odd_fits(a.H)) {
        const int threads = warps_up((a.H + kChunk - 1) / kChunk), rows = threads == 32 ? kWarpRows : 1;
        rmsnorm_odd_kernel<X, W><<<grid(rows), dim3(threads, rows), 0, s>>>(a);
        return launch_status();
    }
    if (!vectors || row_chunks(a.H) == 0) {
        rmsnorm_long_kernel<X, W><<<grid(1), kMaxThreads, 0, s>>>(a);
        return launch_status();
    }
    // Few rows: as many threads a row as it has chunks, which is the shortest way
    // through it.  Many: four chunks a thread, more loads in flight and more rows
    // an SM (16384 rows of 7168 in bf16: XX us, with one chunk 176).
    int V = row_chunks(a.H);
    const int64_t chunks = a.H / kChunk;
    if (a.T > 2 * sm_count() && chunks > 32) V = chunks > 64 && chunks <= 4 * (kMaxThreads / 2) ? 4 : max64(V, 2);
    const int threads = warps_up((chunks + V - 1) / V), rows = threads == 32 ? kWarpRows : 1;
    const dim3 block(threads, rows);
    switch (V) {
        case 1: rmsnorm_kernel<X, W, 1, kQuant><<<grid(rows), block, 0, s>>>(a); break;
        case 2: rmsnorm_kernel<X, W, 2, kQuant><<<grid(rows), block, 0, s>>>(a); break;
        case 4: rmsnorm_kernel<X, W, 4, kQuant><<<grid(rows), block, 0, s>>>(a); break;
        default: rmsnorm_kernel<X, W, 8, kQuant><<<grid(rows), block, 0, s>>>(a); break;
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

// The backward's blocks (rows of partial sums): the ring has one on every SM, the
// others as many as help.
template <typename X, typename W>
moe_status_t launch_backward(BwdArgs a, bool vectors, unsigned* blocks, cudaStream_t s) {
    const int64_t slot = a.H * int64_t(sizeof(X)) * (a.gh ? 3 : 2), chunks = a.H / kChunk;
    if (vectors && 2 * slot <= kRingBytes && chunks <= 2 * kMaxThreads) {
        const int V = chunks > 32 ? 2 : 1, threads = warps_up((chunks + V - 1) / V);
        // as many teams as fit, but no fewer blocks than SMs for them
        int teams = kMaxThreads / threads;
        teams = int(min64(min64(teams, kMaxTeams), kRingBytes / (2 * slot)));
        teams = int(max64(1, min64(teams, (a.T + sm_count() - 1) / sm_count())));
        a.ring = int(min64(kMaxRing, kRingBytes / (teams * slot)));
        *blocks = unsigned(min64((a.T + teams - 1) / teams, min64(sm_count(), kBwdMaxBlocks)));
        const size_t smem = size_t(max64(int64_t(teams) * a.ring * slot, a.H * 4));
        const auto kernel = V == 1 ? rmsnorm_backward_kernel<X, W, 1> : rmsnorm_backward_kernel<X, W, 2>;
        if (!opt_in_smem((const void*)kernel, kRingBytes)) return MOE_ERR_CUDA;
        uint32_t* status = device_status_word();
        if (!status) return MOE_ERR_CUDA;
        kernel<<<*blocks, dim3(threads, teams), smem, s>>>(a, status);
        return launch_status();
    }
    *blocks = unsigned(min64(a.T, kBwdMaxBlocks));
    if (odd_fits(a.H))
        rmsnorm_backward_odd_kernel<X, W><<<*blocks, warps_up((a.H + kChunk - 1) / kChunk), 0, s>>>(a);
    else
        rmsnorm_backward_long_kernel<X, W><<<*blocks, kMaxThreads, 0, s>>>(a);
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
    *bytes = align_up(size_t(min64(T, kBwdMaxBlocks)) * size_t(H) * 4, kWsAlign) + kWsAlign;
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
    unsigned blocks = 0;
    const BwdArgs a{grad_y, grad_h, h, weight, grad_x, static_cast<float*>(workspace), T, H, eps, 0};
    const bool vectors = vectors_fit(H, {grad_y, grad_h, h, weight, grad_x});
    moe_status_t r;
    if (dtype == MOE_BF16)
        r = weight_dtype == MOE_BF16 ? launch_backward<uint16_t, uint16_t>(a, vectors, &blocks, s)
                                     : launch_backward<uint16_t, float>(a, vectors, &blocks, s);
    else
        r = weight_dtype == MOE_BF16 ? launch_backward<float, uint16_t>(a, vectors, &blocks, s)
                                     : launch_backward<float, float>(a, vectors, &blocks, s);
    if (r != MOE_OK) return r;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((H + kSumCols - 1) / kSumCols));
    cfg.blockDim = dim3(kSumCols, kSumGroups);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rmsnorm_grad_weight_kernel, a.partial, int(blocks), H,
                              grad_weight) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
