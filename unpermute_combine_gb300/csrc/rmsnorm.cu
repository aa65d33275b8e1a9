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
// With the normed row n = h r the first is r (g w - n (r mean(g w h))) + gh, and so
// it is computed: r^3 leaves float32's range where rows are as large as 1e13 or as
// small as 1e-13.
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

__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float f) { *p = f32_to_bf16_rn(f); }
__device__ __forceinline__ void store1(float* p, float f) { *p = f; }

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
// Rows that are no multiple of 16 bytes start off a 16-byte boundary, each by its
// own shift, but all of a call's tensors by the same one.  Their chunks are those
// of the aligned memory: chunk c has the elements from 8 c - shift on, and the
// first and the last have some that are another row's.
template <typename X>
__device__ __forceinline__ int row_shift(int64_t row, int64_t H) {
    return int(row * H) & int(16 / sizeof(X) - 1);
}

// The chunk from element p on.  Elements of the rows next to this one come along
// (clear_others takes them out), but nothing past the tensor's end, `left` elements
// from the row's start, is read.
template <bool kShift, typename X>
__device__ __forceinline__ Raw<X> load_at(const X* row, int p, int H, int64_t left) {
    if constexpr (kShift) {
        if (p + kChunk > left) {
            float f[kChunk];
#pragma unroll
            for (int i = 0; i < kChunk; ++i) f[i] = p + i >= 0 && p + i < H ? load1(row + p + i) : 0.0f;
            return rounded(row, f);
        }
    }
    return load_raw(row + p);
}
template <bool kShift>
__device__ __forceinline__ void clear_others(float* f, int p, int H) {
    if constexpr (kShift) {
        if (p < 0 || p + kChunk > H) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i)
                if (p + i < 0 || p + i >= H) f[i] = 0.0f;
        }
    }
}
template <bool kShift, typename X>
__device__ __forceinline__ void store_at(X* row, int p, int H, const Raw<X>& r) {
    if constexpr (kShift) {
        if (p < 0 || p + kChunk > H) {
            float f[kChunk];
            values(r, f);
#pragma unroll
            for (int i = 0; i < kChunk; ++i)
                if (p + i >= 0 && p + i < H) store1(row + p + i, f[i]);
            return;
        }
    }
    store_raw(row + p, r);
}
// A chunk of the weight, which the shift moves off its own boundaries.  (Out of two
// aligned chunks by selects: no faster.)
template <bool kShift, typename W>
__device__ __forceinline__ void weight_at(const W* w, int p, int H, float* f) {
    if constexpr (kShift) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) f[i] = load1(w + min(max(p + i, 0), H - 1));
    } else {
        load8(w + p, f);
    }
}

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
// Products of two floats at once.
__device__ __forceinline__ uint64_t both(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// Two e4m3 bytes of y / s, each the code of the correctly rounded quotient: the product
// with inv = 1 / s and its remainder put back (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990).  Of -y and -inv, so that the
// zeros keep their signs.
__device__ __forceinline__ uint32_t quotients(float ny0, float ny1, uint64_t s, uint64_t ninv) {
    const uint64_t ny = both(ny0, ny1), q = mul2(ny, ninv), r = fma2(fma2(q, s, ny), ninv, q);
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
    return e4m3x2(a, b);
}
// 8 negated floats -> 8 e4m3 bytes of y / s.  The reciprocal is an approximation (an ulp
// off) and a Newton step: the rounded 1 / s, or for a few s an ulp off.  Every s with
// every y next to a boundary of two codes was compared with the division, from
// approximations up to 3 ulp off: the codes are the same, but for one y of the s whose
// significand is all ones.  That s is divided by, as are an infinite one and those so
// small that a remainder underflows (a code other than 0 has a quotient of 2^-10 or more,
// whose remainder is a multiple of 2^-56 s).  8192 rows of 4096: 46.5 us, 46.1 with the
// product alone (which had other codes now and then), 55.0 with divisions throughout.
__device__ __forceinline__ uint2 q8(const float* ny, float s) {
    if (s >= 0x1p-90f && s <= 0x1.fffffep+127f && (~__float_as_uint(s) & 0x7FFFFFu)) {
        float ninv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ninv) : "f"(-s));
        ninv = fmaf(fmaf(s, ninv, 1.0f), ninv, ninv);
        const uint64_t ss = both(s, s), ii = both(ninv, ninv);
        return make_uint2(quotients(ny[0], ny[1], ss, ii) | quotients(ny[2], ny[3], ss, ii) << 16,
                          quotients(ny[4], ny[5], ss, ii) | quotients(ny[6], ny[7], ss, ii) << 16);
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = e4m3x2(__fdiv_rn(ny[2 * i], -s), __fdiv_rn(ny[2 * i + 1], -s));
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
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
// chunks a thread held in registers between the two passes over the row.  Bound
// by memory: 16384 rows of 7168 in bf16 with a residual take 136 us, 6.9 TB/s (a
// copy: 6.7); with e4m3 output 156 us, 5.3 TB/s, where 71% of the issue slots are
// taken (290 warp instructions for 8 elements of each lane, against 145 without the
// quantization; the divisions by a.lanes are some of them); rows of 7001 elements 150 us.  64
// registers where a thread has 64 bytes: with 76, the e4m3 form took 176 us.
template <typename X, typename W, int V, bool kQuant, bool kShift>
__global__ void __launch_bounds__(V >= 4 ? kMaxThreads / 2 : kMaxThreads, V == 4 ? 2 : 1)
rmsnorm_kernel(const NormArgs a) {
    __shared__ float s_part[2][kMaxWarps];
    const int H = int(a.H);
    int turn = 0;
    for (int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y; row < a.T;
         row += int64_t(gridDim.x) * blockDim.y, turn ^= 1) {
        const X* x = static_cast<const X*>(a.x) + row * a.H;
        const int shift = kShift ? row_shift<X>(row, a.H) : 0;
        const int chunks = (H + shift + kChunk - 1) / kChunk;
        const int64_t left = (a.T - row) * a.H;
        Raw<X> h[V];
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            if (c < chunks) h[v] = load_at<kShift>(x, c * kChunk - shift, H, left);
        }
        if (a.residual) {
            const X* res = static_cast<const X*>(a.residual) + row * a.H;
            X* ho = static_cast<X*>(a.h_out) + row * a.H;
            Raw<X> add[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = threadIdx.x + v * blockDim.x;
                if (c < chunks) add[v] = load_at<kShift>(res, c * kChunk - shift, H, left);
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
                    store_at<kShift>(ho, c * kChunk - shift, H, h[v]);
                }
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            if (c < chunks) {
                float f[kChunk];
                values(h[v], f);
                clear_others<kShift>(f, c * kChunk - shift, H);
#pragma unroll
                for (int i = 0; i < kChunk; ++i) ss = fmaf(f[i], f[i], ss);
            }
        }
        const float root = rsqrtf(block_sum(ss, s_part[turn]) / float(a.H) + a.eps);
        const float r = kQuant ? -root : root;             // (q8 takes -y)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            float y[kChunk];
            if (c < chunks) {
                float w[kChunk];
                weight_at<kShift>(static_cast<const W*>(a.weight), c * kChunk - shift, H, w);
                values(h[v], y);
#pragma unroll
                for (int i = 0; i < kChunk; ++i) y[i] = y[i] * r * w[i];
            }
            if (!kQuant) {
                if (c < chunks)
                    store_at<kShift>(static_cast<X*>(a.out) + row * a.H, c * kChunk - shift, H,
                                     rounded(x, y));
            } else {
                // a block's lanes are consecutive and whole blocks fit a warp
                float amax = 0.0f;
                if (c < chunks) {
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) amax = fmaxf(amax, fabsf(y[i]));
                }
                for (int o = a.lanes >> 1; o > 0; o >>= 1)
                    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
                // amax / 448: the product with 1/448, and its remainder put back; no scale
                // is 0, by which a 0 beside the smallest floats would become NaN
                float s = amax * (1.0f / 448.0f);
                s = fmaf(fmaf(s, -448.0f, amax), 1.0f / 448.0f, s);
                if (!(s >= 0x1p-126f)) s = amax > 0.0f ? fmaxf(__fdiv_rn(amax, 448.0f), 0x1p-149f) : 1.0f;
                if (c < chunks) {
                    uint2* q = reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + row * a.H);
                    q[c] = q8(y, s);
                    if (c % a.lanes == 0) a.scales[row * (chunks / a.lanes) + c / a.lanes] = s;
                }
            }
        }
    }
}

// The same for tensors that do not start on a 16-byte boundary: elements
// threadIdx.x, + blockDim.x, ..., eight of them a thread, in registers.  Bound by loads
// of single elements: 16384 rows of 7168 in bf16 405 us.
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
    bool ring_gh;             // rows of gh among them
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

// Bytes of a row's place in the ring.
template <typename X, bool kShift>
__host__ __device__ constexpr uint32_t slot_size(int64_t H, bool three) {
    const int64_t most = kShift ? (H + int64_t(16 / sizeof(X)) - 1 + kChunk - 1) / kChunk * kChunk : H;
    return uint32_t(most * int64_t(sizeof(X))) * (three ? 3 : 2);
}

// Rows in teams of blockDim.x threads, blockDim.y teams a block.  A team has a ring
// of rows in shared memory (h, grad_y and grad_h of each, or the first two where only
// they have room twice), which bulk copies fill rows ahead, so that reading goes on
// while a row waits for its sums; V chunks a thread.  The columns' shares of
// grad_weight stay in registers over all rows of the block; its teams' shares are
// added up at the end, in order, and the blocks' by rmsnorm_grad_weight_kernel.
// Bound by memory on long batches (16384 rows of 7168 in bf16 with grad_h: 144 us,
// 6.5 TB/s), by the way in and out of the ring on short ones (4096 rows of 2048, 3.4
// rows a team: 22 us with the second launch, of which 10 move the bytes).  Shifted rows
// (7172 wide: 184 us) pay a barrier more and the repair of their edges before a row's
// sums.  float32 rows of 12000, whose grad_h is loaded when it is added: 150 us for 4096,
// memory 118 (8528, with grad_h in the ring: 88, memory 84).  One row a
// block at a time, without a ring: 295 and 44 us.  Packed float instructions and
// fewer shuffles: no faster, though 70% of the issue slots are taken.
template <typename X, typename W, int V, bool kShift>
__global__ void __launch_bounds__(kMaxThreads)
rmsnorm_backward_kernel(const BwdArgs a, uint32_t* status) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[kMaxTeams][kMaxRing];
    __shared__ float2 s_part[2][kMaxWarps];
    __shared__ volatile int s_failed[kMaxTeams];
    const int team = threadIdx.y, teams = blockDim.y, nw = blockDim.x >> 5;
    const int warp = threadIdx.x >> 5;
    const int H = int(a.H);
    const int64_t first = int64_t(blockIdx.x) * teams + team, step = int64_t(gridDim.x) * teams;
    // (step is a multiple of 8 where there is a shift: it is the same for all of a
    // team's rows, and a thread's chunks are the same columns in all of them)
    const int shift = kShift ? row_shift<X>(first, a.H) : 0;
    const int chunks = (H + shift + kChunk - 1) / kChunk;
    const uint32_t slot_bytes = slot_size<X, kShift>(a.H, a.ring_gh);
    const uint32_t row_bytes = slot_bytes / (a.ring_gh ? 3 : 2);
    uint8_t* ring = smem + size_t(team) * a.ring * slot_bytes;
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.ring; ++i) mbar_init(smem_addr(&full[team][i]), 1);
        mbar_fence_init();
    }
    if (threadIdx.x == 0) s_failed[team] = 0;
    __syncthreads();
    const int64_t rows = first < a.T ? (a.T - first + step - 1) / step : 0;
    // elements of the team's n-th row, from its shift on, that bulk copies bring: whole
    // 16-byte words, of which the tensor's last may be cut off
    constexpr int kWord = int(16 / sizeof(X));
    auto brought = [&](int64_t n) -> int {
        if (!kShift) return H;
        const int64_t at = (first + n * step) * a.H - shift, left = a.T * a.H - at;
        const int whole = (H + shift + kWord - 1) / kWord * kWord;
        return left >= whole ? whole : int(left / kWord * kWord);
    };
    auto fill = [&](int64_t n) {                           // one thread: the team's n-th row
        const int slot = int(n % a.ring);
        const uint32_t bar = smem_addr(&full[team][slot]), dst = smem_addr(ring + slot * slot_bytes);
        const uint32_t bytes = uint32_t(brought(n)) * uint32_t(sizeof(X));
        const int64_t at = (first + n * step) * a.H - shift;
        mbar_expect_tx(bar, bytes * (a.ring_gh ? 3 : 2));
        if (kShift && bytes == 0) return;
        bulk_load(dst, static_cast<const X*>(a.h) + at, bytes, bar);
        bulk_load(dst + row_bytes, static_cast<const X*>(a.g) + at, bytes, bar);
        if (a.ring_gh) bulk_load(dst + 2 * row_bytes, static_cast<const X*>(a.gh) + at, bytes, bar);
    };
    if (threadIdx.x == 0)
        for (int64_t n = 0; n < rows && n < a.ring; ++n) fill(n);
    Raw<W> weight[V];
    float dw[V][kChunk] = {};
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = threadIdx.x + v * blockDim.x;
        if (c < chunks) {
            float f[kChunk];
            weight_at<kShift>(static_cast<const W*>(a.weight), c * kChunk - shift, H, f);
            weight[v] = rounded(static_cast<const W*>(a.weight), f);
        }
    }
    for (int64_t n = 0; n < rows; ++n) {
        const int slot = int(n % a.ring);
        if (!mbar_wait(smem_addr(&full[team][slot]), uint32_t(n / a.ring) & 1u)) s_failed[team] = 1;
        uint8_t* row = ring + slot * slot_bytes;
        if constexpr (kShift) {
            // The first and the last chunk are put right in place, once: other rows'
            // elements become 0, and what no copy brings is loaded.  (In registers,
            // at each reading: 350 us instead of 189 for 16384 rows of 7172.)
            if (threadIdx.x < 2 * kChunk) {
                const int i = (threadIdx.x < kChunk ? 0 : chunks - 1) * kChunk +
                              int(threadIdx.x & (kChunk - 1));
                const bool inside = i >= shift && i < H + shift;
                if (!inside || i >= brought(n)) {
                    const int64_t at = (first + n * step) * a.H + i - shift;
                    X* edge = reinterpret_cast<X*>(row) + i;
                    const int pitch = int(row_bytes / sizeof(X));
                    edge[0] = inside ? static_cast<const X*>(a.h)[at] : X(0);
                    edge[pitch] = inside ? static_cast<const X*>(a.g)[at] : X(0);
                    if (a.ring_gh) edge[2 * pitch] = inside ? static_cast<const X*>(a.gh)[at] : X(0);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the next copy
                }
            }
            if (nw > 1)
                asm volatile("bar.sync %0, %1;" :: "r"(team + 1), "r"(blockDim.x) : "memory");
            else
                __syncwarp();
        }
        // chunk c of the row's `which`th tensor
        auto chunk = [&](int which, int c, float* f) {
            shared8(reinterpret_cast<const X*>(row + which * row_bytes) + c * kChunk, f);
        };
        float ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            if (c < chunks) {
                float hv[kChunk], gv[kChunk], w[kChunk];
                chunk(0, c, hv);
                chunk(1, c, gv);
                values(weight[v], w);
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
        const float b = r * (dot / float(a.H));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            if (c < chunks) {
                float hv[kChunk], gv[kChunk], w[kChunk], o[kChunk];
                chunk(0, c, hv);
                chunk(1, c, gv);
                values(weight[v], w);
#pragma unroll
                for (int i = 0; i < kChunk; ++i) {
                    const float n = hv[i] * r;
                    dw[v][i] = fmaf(gv[i], n, dw[v][i]);
                    o[i] = r * fmaf(-n, b, gv[i] * w[i]);
                }
                const int64_t at = first + n * step;
                if (a.gh) {
                    float e[kChunk];
                    if (sizeof(X) == 2 || a.ring_gh)       // (bf16 rows always have room)
                        chunk(2, c, e);
                    else
                        values(load_at<kShift>(static_cast<const X*>(a.gh) + at * a.H, c * kChunk - shift,
                                               H, (a.T - at) * a.H), e);
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) o[i] += e[i];
                }
                X* gx = static_cast<X*>(a.gx) + at * a.H;
                store_at<kShift>(gx, c * kChunk - shift, H, rounded(gx, o));
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
    // the teams' shares side by side in the ring's place (4 H bytes each, and a ring
    // has at least 8 H for a team), then a column's sum over the teams, in order
    float* share = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = threadIdx.x + v * blockDim.x, p = c * kChunk - shift;
        if (c >= chunks) continue;
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
            if (!kShift || (p + i >= 0 && p + i < H)) share[team * H + p + i] = dw[v][i];
    }
    __syncthreads();
    const int threads = blockDim.x * blockDim.y;
    for (int c = team * blockDim.x + threadIdx.x; c < H; c += threads) {
        float sum = share[c];
        for (int t = 1; t < teams; ++t) sum += share[t * H + c];
        a.partial[int64_t(blockIdx.x) * a.H + c] = sum;
    }
}

// Tensors that do not start on a 16-byte boundary: elements threadIdx.x, +
// blockDim.x, ..., eight of them a thread; the next row's are loaded while this one's are
// worked on.  Bound by loads of single elements: 16384 rows of 7168 in bf16 610 us.
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
        const float b = r * (t.y / float(a.H));
#pragma unroll
        for (int v = 0; v < kChunk; ++v) {
            const int c = threadIdx.x + v * blockDim.x;
            const float n = h[v] * r;
            dw[v] = fmaf(g[v], n, dw[v]);
            if (c < H)
                store1(static_cast<X*>(a.gx) + row * a.H + c,
                       fmaf(r, fmaf(-n, b, g[v] * load1(static_cast<const W*>(a.weight) + c)), e[v]));
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
// only.  Bound by reading every row twice, element by element, and the share with it:
// 4096 rows of 16384 in bf16 443 us, of 20000 in float32 605, three and five times what
// the bytes take.
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
        const float b = r * (t.y / float(a.H));
        for (int64_t i = threadIdx.x; i < a.H; i += blockDim.x) {
            const float n = load1(h + i) * r, gv = load1(g + i);
            part[i] = fmaf(gv, n, part[i]);
            float o = r * fmaf(-n, b, gv * load1(static_cast<const W*>(a.weight) + i));
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
    const int64_t chunks = (H + kChunk - 1) / kChunk;
    if (chunks <= kMaxThreads) return 1;
    if (chunks <= 2 * kMaxThreads) return 2;
    return chunks <= 8 * (kMaxThreads / 2) ? 8 : 0;
}

// Rows of at most kMaxThreads * kChunk elements are held by threads of eight.
bool odd_fits(int64_t H) { return H <= int64_t(kMaxThreads) * kChunk; }

// Whether every pointer is on a boundary of its element.
bool on_elements(int dtype, std::initializer_list<const void*> ptrs) {
    const uintptr_t low = elem_size(moe_dtype_t(dtype)) - 1;
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & low) return false;
    return true;
}

// How a call's rows lie: on 16-byte boundaries, in memory that starts on one, or not.
enum Rows : int { kVectors, kShifted, kElements };

Rows rows_of(int64_t H, const void* weight, std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return kElements;
    return H % kChunk == 0 && aligned16(weight) ? kVectors : kShifted;
}

template <typename X, typename W, bool kQuant>
moe_status_t launch_norm(const NormArgs& a, Rows how, cudaStream_t s) {
    const auto grid = [&](int rows) { return unsigned(min64((a.T + rows - 1) / rows, int64_t(1) << 20)); };
    if (how == kElements && odd_fits(a.H)) {
        const int threads = warps_up((a.H + kChunk - 1) / kChunk), rows = threads == 32 ? kWarpRows : 1;
        rmsnorm_odd_kernel<X, W><<<grid(rows), dim3(threads, rows), 0, s>>>(a);
        return launch_status();
    }
    const int64_t most = a.H + (how == kShifted ? kChunk : 0);    // with the shift
    int V = row_chunks(most);
    if (how == kElements || V == 0) {
        rmsnorm_long_kernel<X, W><<<grid(1), kMaxThreads, 0, s>>>(a);
        return launch_status();
    }
    // Few rows: as many threads a row as it has chunks, which is the shortest way
    // through it.  Many: 64 bytes a thread, more loads in flight and more rows an SM
    // (16384 rows of 7168 in bf16: 136 us, with 32 bytes 149, with 16 176).
    const int64_t chunks = (most + kChunk - 1) / kChunk;
    constexpr int kWide = sizeof(X) == 2 ? 4 : 2;
    if (a.T > 2 * sm_count() && chunks > 32) V = int(max64(V, chunks > 64 ? kWide : 2));
    const int threads = warps_up((chunks + V - 1) / V), rows = threads == 32 ? kWarpRows : 1;
    const dim3 block(threads, rows);
    constexpr bool kMay = !kQuant;                         // e4m3 rows are never shifted
#define MOE_NORM(v)                                                                              \
    do {                                                                                         \
        if (kMay && how == kShifted)                                                             \
            rmsnorm_kernel<X, W, v, kQuant, kMay><<<grid(rows), block, 0, s>>>(a);               \
        else                                                                                     \
            rmsnorm_kernel<X, W, v, kQuant, false><<<grid(rows), block, 0, s>>>(a);              \
    } while (0)
    if (V == 1) MOE_NORM(1);
    else if (V == 2) MOE_NORM(2);
    else if (V == kWide) MOE_NORM(kWide);
    else MOE_NORM(8);
#undef MOE_NORM
    return launch_status();
}

template <bool kQuant>
moe_status_t dispatch_norm(const NormArgs& a, int dtype, int wdtype, Rows how,
                           cudaStream_t s) {
    if (dtype == MOE_BF16)
        return wdtype == MOE_BF16 ? launch_norm<uint16_t, uint16_t, kQuant>(a, how, s)
                                  : launch_norm<uint16_t, float, kQuant>(a, how, s);
    return wdtype == MOE_BF16 ? launch_norm<float, uint16_t, kQuant>(a, how, s)
                              : launch_norm<float, float, kQuant>(a, how, s);
}

template <typename X, typename W, bool kShift>
moe_status_t launch_ring(BwdArgs a, unsigned* blocks, cudaStream_t s) {
    // The teams follow from the size of three tensors' rows, with grad_h or without: the
    // order of grad_weight's sums is the same.
    const int64_t most_slot = slot_size<X, kShift>(a.H, true);
    a.ring_gh = a.gh && 2 * most_slot <= kRingBytes;
    const int64_t slot = slot_size<X, kShift>(a.H, a.ring_gh);
    const int64_t chunks = most_slot / 3 / int64_t(kChunk * sizeof(X));
    const int V = chunks > 32 ? 2 : 1;
    const int threads = warps_up((chunks + V - 1) / V);
    // as many teams as fit (16384 rows of 2048 in bf16: 57 us with 8, 98 with 2, 173
    // with 1), but no fewer blocks than SMs for them
    int teams = int(min64(min64(kMaxThreads / threads, kMaxTeams), kRingBytes / (2 * most_slot)));
    teams = int(max64(1, min64(teams, (a.T + sm_count() - 1) / sm_count())));
    a.ring = int(min64(kMaxRing, kRingBytes / (teams * slot)));
    int64_t most = min64(sm_count(), kBwdMaxBlocks);
    if (kShift && most >= 8) most -= most % 8;             // the step between a team's rows
    *blocks = unsigned(min64((a.T + teams - 1) / teams, most));
    const size_t smem = size_t(teams) * a.ring * slot;
    const auto kernel = V == 1 ? rmsnorm_backward_kernel<X, W, 1, kShift>
                               : rmsnorm_backward_kernel<X, W, 2, kShift>;
    if (!opt_in_smem((const void*)kernel, kRingBytes)) return MOE_ERR_CUDA;
    uint32_t* status = device_status_word();
    if (!status) return MOE_ERR_CUDA;
    kernel<<<*blocks, dim3(threads, teams), smem, s>>>(a, status);
    return launch_status();
}

// The backward's blocks (rows of partial sums): the ring has one on every SM, the
// others as many as help.
template <typename X, typename W>
moe_status_t launch_backward(const BwdArgs& a, Rows how, unsigned* blocks, cudaStream_t s) {
    if (how != kElements && 2 * int64_t(slot_size<X, true>(a.H, false)) <= kRingBytes &&
        a.H + kChunk <= 2 * kMaxThreads * kChunk) {
        if (how == kVectors) return launch_ring<X, W, false>(a, blocks, s);
        // a shift wants blocks by eights, or no second row for a team
        if (sm_count() >= 8 || a.T <= sm_count()) return launch_ring<X, W, true>(a, blocks, s);
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
    if (!x || !weight || !out || (residual && (!residual_out || residual_out == out)))
        return MOE_ERR_INVALID_ARG;
    if (!residual) residual_out = nullptr;
    if (!on_elements(dtype, {x, residual, residual_out, out}) || !on_elements(weight_dtype, {weight}))
        return MOE_ERR_INVALID_ARG;
    const NormArgs a{x, residual, weight, residual_out, out, nullptr, T, H, eps, 0};
    const Rows how = rows_of(H, weight, {x, residual, residual_out, out});
    return dispatch_norm<false>(a, dtype, weight_dtype, how, static_cast<cudaStream_t>(stream));
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
    if (rows_of(H, weight, {x, residual, residual_out}) != kVectors ||
        (reinterpret_cast<uintptr_t>(x_q) & 7u) || (reinterpret_cast<uintptr_t>(scales) & 3u))
        return MOE_ERR_INVALID_ARG;
    const NormArgs a{x, residual, weight, residual_out, x_q, scales, T, H, eps, block / kChunk};
    return dispatch_norm<true>(a, dtype, weight_dtype, kVectors, static_cast<cudaStream_t>(stream));
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
    if (!grad_weight || !on_elements(MOE_F32, {grad_weight})) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0)
        return cudaMemsetAsync(grad_weight, 0, size_t(H) * 4, s) == cudaSuccess ? MOE_OK
                                                                               : MOE_ERR_CUDA;
    if (!grad_y || !h || !weight || !grad_x) return MOE_ERR_INVALID_ARG;
    if (!on_elements(dtype, {grad_y, grad_h, h, grad_x}) || !on_elements(weight_dtype, {weight}))
        return MOE_ERR_INVALID_ARG;
    size_t need = 0;
    const moe_status_t sz = moe_rmsnorm_backward_workspace_size(T, H, &need);
    if (sz != MOE_OK) return sz;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) ||
        workspace_bytes < need)
        return MOE_ERR_WORKSPACE;
    unsigned blocks = 0;
    const BwdArgs a{grad_y, grad_h, h, weight, grad_x, static_cast<float*>(workspace), T, H, eps, 0, false};
    const Rows how = rows_of(H, weight, {grad_y, grad_h, h, grad_x});
    moe_status_t r;
    if (dtype == MOE_BF16)
        r = weight_dtype == MOE_BF16 ? launch_backward<uint16_t, uint16_t>(a, how, &blocks, s)
                                     : launch_backward<uint16_t, float>(a, how, &blocks, s);
    else
        r = weight_dtype == MOE_BF16 ? launch_backward<float, uint16_t>(a, how, &blocks, s)
                                     : launch_backward<float, float>(a, how, &blocks, s);
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
