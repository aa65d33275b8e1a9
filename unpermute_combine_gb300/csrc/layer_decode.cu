// layer_decode.cu -- moe_layer_decode, moe_layer_decode_indices: a whole MoE
// layer for a few tokens.
//
//   out[t] = sum_j p[t,j] * (silu(x_t Wg[e]^T) * (x_t Wu[e]^T)) Wd[e]^T,  e = idx[t,j]
//
// With up to 64 tokens a layer is bound by reading the weights of the experts
// that some token chose, once: 6 H I bytes each.  Two kernels read them: the
// first the up projections (into the hidden rows, in the workspace), the
// second the down projections and, in the last block that finishes a strip of
// output columns, the weighted sum over a token's slots in slot order, so that
// the result does not depend on which block that is.  Every block works the
// routing out for itself (top-k, softmax, each expert's tokens) in shared
// memory: 64 tokens are too few for a launch of their own.
#include "pipeline.cuh"

namespace moe {
namespace {

constexpr int kMaxTokens = 64;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 32;                 // weight rows of one work item
constexpr int kTok = 4;                   // tokens a warp multiplies a weight row with at a time

struct LayerArgs {
    const void* x;              // bf16 [T,H], or e4m3 codes
    const float* x_scales;      // NULL (bf16 x), or [T, H/128]
    const float* logits;        // NULL: the choices are given
    const int32_t* given_idx;   // [T,k], -1 = empty slot
    const float* given_w;       // [T,k]
    int32_t* topk_idx;          // written from the logits
    float* topk_w;
    const uint16_t* w_up;       // [E,2I,H] packed
    const uint16_t* w_down;     // [E,H,I] packed
    uint16_t* out;              // [T,H] bf16
    WsHeader* header;
    uint32_t* arrivals;         // [H / kRows] blocks that finished a strip's products
    float* hidden;              // [T*k, I]
    float* y;                   // [T*k, H]
    int T, E, k;
    int64_t H, I;
};

// ----------------------------------------------------------------- routing

// What every block knows of the routing, in shared memory.  A slot is a row of
// the workspace: experts in order, an expert's tokens in order.
struct Routing {
    float* w;                   // [T*k]
    unsigned long long* mask;   // [E] tokens of each expert
    int16_t* idx;               // [T*k] expert, -1 = empty
    uint16_t* first;            // [E] first slot of each expert
    uint16_t* active;           // [min(E, T*k)] experts with tokens
    uint8_t* token;             // [T*k] token of each slot
    int* count;                 // [2]: active experts, bad choices
};

__host__ __device__ inline size_t routing_bytes(int T, int E, int k) {
    const size_t n = size_t(T) * k;
    const size_t b = 16 + n * 4 + size_t(E) * 8 + n * 2 + size_t(E) * 2 + (size_t(E) + 1) * 2 + n;
    return (b + 127) / 128 * 128;
}

__device__ __forceinline__ Routing carve_routing(uint8_t* p, int T, int E, int k) {
    const int n = T * k;
    Routing r;
    r.count = reinterpret_cast<int*>(p);
    r.mask = reinterpret_cast<unsigned long long*>(p + 16);
    r.w = reinterpret_cast<float*>(r.mask + E);
    r.idx = reinterpret_cast<int16_t*>(r.w + n);
    r.first = reinterpret_cast<uint16_t*>(r.idx + n);
    r.active = r.first + E;
    r.token = reinterpret_cast<uint8_t*>(r.active + E + 1);
    return r;
}

// Order-preserving key of a float; -0 is +0, as for a comparison of floats.
__device__ __forceinline__ uint32_t logit_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_logit(uint32_t u) {
    return __uint_as_float(u ^ (uint32_t(int32_t(~u) >> 31) | 0x80000000u));
}

// The warp's token: its k largest logits, largest first, equal ones by id, and
// their softmax.  Lane j gets choice j.
template <int NV>
__device__ __forceinline__ void top_k(const float* logits, int E, int k, int& id, float& weight) {
    const int lane = int(lane_id());
    uint32_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        key[i] = e < E ? logit_key(logits[e]) : 0u;
    }
    uint32_t my_key = 0;
    id = -1;
    for (int j = 0; j < k; ++j) {
        uint32_t best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < NV; ++i)
            if (key[i] > best) { best = key[i]; at = i; }
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
        const uint32_t e = __reduce_min_sync(0xFFFFFFFFu,
                                             best == top ? uint32_t(lane + 32 * at) : 0xFFFFFFFFu);
        if ((e & 31u) == uint32_t(lane)) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (uint32_t(i) == (e >> 5)) key[i] = 0u;
        }
        if (lane == j) { my_key = top; id = e < uint32_t(E) ? int(e) : -1; }
    }
    const float v = key_logit(my_key), v0 = __shfl_sync(0xFFFFFFFFu, v, 0);
    const float p = lane < k ? expf(v - v0) : 0.0f;
    float sum = p;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    weight = __fdiv_rn(p, sum);
}

// All threads of the block; ends with a barrier.  Block 0 of the first kernel
// writes the choices out (`publish`).
__device__ void route(const LayerArgs& a, const Routing& r, bool publish) {
    const int lane = int(lane_id()), warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int T = a.T, E = a.E, k = a.k, n = T * k;
    for (int e = threadIdx.x; e < E; e += blockDim.x) r.mask[e] = 0ull;
    if (threadIdx.x == 0) r.count[1] = 0;
    __syncthreads();
    for (int t = warp; t < T; t += warps) {
        int id = -1;
        float w = 0.0f;
        if (a.logits) {
            const float* lg = a.logits + int64_t(t) * E;
            if (E <= 64) top_k<2>(lg, E, k, id, w);
            else if (E <= 256) top_k<8>(lg, E, k, id, w);
            else top_k<32>(lg, E, k, id, w);
            if (publish && lane < k) {
                a.topk_idx[t * k + lane] = id;
                a.topk_w[t * k + lane] = w;
            }
        } else {
            int bad = 0;
            if (lane < k) {
                id = a.given_idx[t * k + lane];
                w = a.given_w[t * k + lane];
                bad = id < -1 || id >= E;
                if (id < 0 || id >= E) id = -1;
            }
            // an expert named twice: the first slot keeps it
            const unsigned same = __match_any_sync(0xFFFFFFFFu, id < 0 ? -1 - lane : id);
            if (id >= 0 && (same & ((1u << lane) - 1u))) { id = -1; bad = 1; }
            if (bad) r.count[1] = 1;
        }
        if (lane < k) {
            r.idx[t * k + lane] = int16_t(id);
            r.w[t * k + lane] = w;
            if (id >= 0) atomicOr(&r.mask[id], 1ull << t);
        }
    }
    __syncthreads();
    if (warp == 0) {
        int slots = 0, act = 0;
        for (int base = 0; base < E; base += 32) {
            const int e = base + lane;
            const int c = e < E ? __popcll(r.mask[e]) : 0;
            int incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (lane >= o) incl += v;
            }
            const unsigned some = __ballot_sync(0xFFFFFFFFu, c > 0);
            if (e < E) r.first[e] = uint16_t(slots + incl - c);
            if (c > 0) r.active[act + __popc(some & ((1u << lane) - 1u))] = uint16_t(e);
            slots += __shfl_sync(0xFFFFFFFFu, incl, 31);
            act += __popc(some);
        }
        if (lane == 0) r.count[0] = act;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int e = r.idx[i], t = i / k;
        if (e >= 0) r.token[r.first[e] + __popcll(r.mask[e] & ((1ull << t) - 1ull))] = uint8_t(t);
    }
    __syncthreads();
}

// The slot of (t, j), or -1.
__device__ __forceinline__ int slot_of(const Routing& r, int t, int i) {
    const int e = r.idx[i];
    return e < 0 ? -1 : r.first[e] + __popcll(r.mask[e] & ((1ull << t) - 1ull));
}

// ---------------------------------------------------------------- products

__device__ __forceinline__ void unpack8(uint4 v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16lo_to_f32(w[i]);
        f[2 * i + 1] = bf16hi_to_f32(w[i]);
    }
}

// Elements [c, c + 8) of token t's row.
__device__ __forceinline__ void load_x8(const LayerArgs& a, int t, int64_t c, float* f) {
    if (!a.x_scales) {
        unpack8(ld_v4(static_cast<const uint16_t*>(a.x) + t * a.H + c), f);
        return;
    }
    const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.x) + t * a.H + c);
    const float s = a.x_scales[t * (a.H / 128) + c / 128];
    e4m3x2_to_f32(q.x & 0xFFFFu, f[0], f[1]);
    e4m3x2_to_f32(q.x >> 16, f[2], f[3]);
    e4m3x2_to_f32(q.y & 0xFFFFu, f[4], f[5]);
    e4m3x2_to_f32(q.y >> 16, f[6], f[7]);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= s;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// hidden[slot, j] = silu(gate) * up
__global__ void __launch_bounds__(kThreads) layer_up_kernel(const LayerArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    const Routing r = carve_routing(smem, a.T, a.E, a.k);
    const int lane = int(lane_id()), warp = threadIdx.x >> 5;
    route(a, r, a.logits && blockIdx.x == 0);
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) {
            a.header->status = r.count[1] ? MOE_ERR_DEVICE_CHECK : MOE_OK;
            a.header->detail = 0;
        }
        for (int64_t i = threadIdx.x; i < a.H / kRows; i += blockDim.x) a.arrivals[i] = 0u;
    }
    const int strips = int(a.I / kRows), items = r.count[0] * strips;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int e = r.active[item / strips];
        const int first = r.first[e], n = __popcll(r.mask[e]);
        for (int j = (item % strips) * kRows + warp; j < (item % strips + 1) * kRows; j += kWarps) {
            const uint16_t* wg = a.w_up + (int64_t(e) * 2 * a.I + (j / 128) * 256 + j % 128) * a.H;
            const uint16_t* wu = wg + 128 * a.H;
            for (int t0 = 0; t0 < n; t0 += kTok) {
                float g[kTok] = {}, u[kTok] = {};
                for (int64_t c = lane * 8; c < a.H; c += 256) {
                    float fg[8], fu[8];
                    unpack8(ld_nc_v4(wg + c), fg);
                    unpack8(ld_nc_v4(wu + c), fu);
#pragma unroll
                    for (int q = 0; q < kTok; ++q) {
                        if (t0 + q < n) {
                            float fx[8];
                            load_x8(a, r.token[first + t0 + q], c, fx);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                g[q] = fmaf(fg[i], fx[i], g[q]);
                                u[q] = fmaf(fu[i], fx[i], u[q]);
                            }
                        }
                    }
                }
#pragma unroll
                for (int q = 0; q < kTok; ++q) {
                    const float gs = warp_sum(g[q]), us = warp_sum(u[q]);
                    if (lane == 0 && t0 + q < n)
                        a.hidden[int64_t(first + t0 + q) * a.I + j] = gs / (1.0f + expf(-gs)) * us;
                }
            }
        }
    }
}

// y[slot, h], and the last block of a strip of output columns adds it up.
__global__ void __launch_bounds__(kThreads) layer_down_kernel(const LayerArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int s_last;
    const Routing r = carve_routing(smem, a.T, a.E, a.k);
    const int lane = int(lane_id()), warp = threadIdx.x >> 5;
    route(a, r, false);
    const int act = r.count[0], strips = int(a.H / kRows), items = act * strips;
    if (act == 0) {                                       // every slot is empty
        for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < a.T * a.H;
             i += int64_t(gridDim.x) * kThreads)
            a.out[i] = 0;
        return;
    }
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int e = r.active[item % act], strip = item / act;
        const int first = r.first[e], n = __popcll(r.mask[e]);
        for (int h = strip * kRows + warp; h < (strip + 1) * kRows; h += kWarps) {
            const uint16_t* wd = a.w_down + (int64_t(e) * a.H + h) * a.I;
            for (int t0 = 0; t0 < n; t0 += kTok) {
                float s[kTok] = {};
                for (int64_t c = lane * 8; c < a.I; c += 256) {
                    float f[8];
                    unpack8(ld_nc_v4(wd + c), f);
#pragma unroll
                    for (int q = 0; q < kTok; ++q) {
                        if (t0 + q < n) {
                            const float* hp = a.hidden + int64_t(first + t0 + q) * a.I + c;
#pragma unroll
                            for (int i = 0; i < 8; ++i) s[q] = fmaf(f[i], hp[i], s[q]);
                        }
                    }
                }
#pragma unroll
                for (int q = 0; q < kTok; ++q) {
                    const float v = warp_sum(s[q]);
                    if (lane == 0 && t0 + q < n) a.y[int64_t(first + t0 + q) * a.H + h] = v;
                }
            }
        }
        // the block that arrives last sees every other block's products
        __syncthreads();
        if (threadIdx.x == 0) {
            __threadfence();
            s_last = atomicAdd(&a.arrivals[strip], 1u) == uint32_t(act - 1);
            __threadfence();
        }
        __syncthreads();
        if (s_last) {
            for (int i = threadIdx.x; i < a.T * kRows; i += kThreads) {
                const int t = i / kRows;
                const int64_t h = int64_t(strip) * kRows + i % kRows;
                float s = 0.0f;
                for (int j = 0; j < a.k; ++j) {
                    const int slot = slot_of(r, t, t * a.k + j);
                    if (slot >= 0) s = fmaf(r.w[t * a.k + j], __ldcg(a.y + slot * a.H + h), s);
                }
                a.out[t * a.H + h] = f32_to_bf16_rn(s);
            }
        }
        __syncthreads();
    }
}

// -------------------------------------------------------------------- host

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

moe_status_t check_layer(int64_t T, int E, int k, int64_t H, int64_t I) {
    if (T < 0 || E < 1 || k < 1 || H < 1 || I < 1) return MOE_ERR_INVALID_ARG;
    if (T > kMaxTokens || E > kMaxExperts || k > kMaxTopK || k > E || H % 256 != 0 || I % 128 != 0)
        return MOE_ERR_UNSUPPORTED;
    if (int64_t(E) * 2 * I >= (int64_t(1) << 31) || int64_t(E) * H >= (int64_t(1) << 31))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

struct Layout { size_t arrivals, hidden, y, total; };

Layout workspace_layout(int64_t T, int k, int64_t H, int64_t I) {
    const size_t n = size_t(T) * k;
    Layout l;
    l.arrivals = kWsAlign;
    l.hidden = l.arrivals + align_up(size_t(H / kRows) * 4, kWsAlign);
    l.y = l.hidden + align_up(n * size_t(I) * 4, kWsAlign);
    l.total = l.y + align_up(n * size_t(H) * 4, kWsAlign);
    return l;
}

moe_status_t layer(LayerArgs a, int64_t T, void* workspace, size_t workspace_bytes,
                   cudaStream_t s) {
    const moe_status_t st = check_layer(T, a.E, a.k, a.H, a.I);
    if (st != MOE_OK) return st;
    const Layout l = workspace_layout(T, a.k, a.H, a.I);
    const bool choices = a.logits ? a.topk_idx && a.topk_w : a.given_idx && a.given_w;
    if (T > 0 && (!a.x || !choices || !a.w_up || !a.w_down || !a.out)) return MOE_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) ||
        workspace_bytes < l.total)
        return MOE_ERR_WORKSPACE;
    if (!aligned16(a.x) || !aligned16(a.w_up) || !aligned16(a.w_down) || !aligned16(a.out) ||
        !aligned4(a.x_scales) || !aligned4(a.logits) || !aligned4(a.given_idx) ||
        !aligned4(a.given_w) || !aligned4(a.topk_idx) || !aligned4(a.topk_w))
        return MOE_ERR_INVALID_ARG;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.header = reinterpret_cast<WsHeader*>(ws);
    if (T == 0)
        return cudaMemsetAsync(ws, 0, 8, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    a.T = int(T);
    a.arrivals = reinterpret_cast<uint32_t*>(ws + l.arrivals);
    a.hidden = reinterpret_cast<float*>(ws + l.hidden);
    a.y = reinterpret_cast<float*>(ws + l.y);
    const size_t smem = routing_bytes(a.T, a.E, a.k);
    const unsigned grid = unsigned(sm_count() * 4);
    layer_up_kernel<<<grid, kThreads, smem, s>>>(a);
    if (launch_status() != MOE_OK) return MOE_ERR_CUDA;
    layer_down_kernel<<<grid, kThreads, smem, s>>>(a);
    return launch_status();
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_layer_decode_workspace_size(int64_t T, int E, int k, int64_t H,
                                                        int64_t I, size_t* bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_layer(T, E, k, H, I);
    if (st != MOE_OK) return st;
    *bytes = workspace_layout(T, k, H, I).total;
    return MOE_OK;
}

extern "C" moe_status_t moe_layer_decode(const void* x, const float* x_scales, const float* logits,
                                         int64_t T, int E, int k, int64_t H, int64_t I,
                                         const void* w_up_packed, const void* w_down_packed,
                                         int32_t* topk_idx, float* topk_w, void* out,
                                         void* workspace, size_t workspace_bytes, void* stream) {
    MOE_TRACE(__func__);
    if (T > 0 && !logits) return MOE_ERR_INVALID_ARG;
    LayerArgs a{};
    a.x = x;
    a.x_scales = x_scales;
    a.logits = logits;
    a.topk_idx = topk_idx;
    a.topk_w = topk_w;
    a.w_up = static_cast<const uint16_t*>(w_up_packed);
    a.w_down = static_cast<const uint16_t*>(w_down_packed);
    a.out = static_cast<uint16_t*>(out);
    a.E = E;
    a.k = k;
    a.H = H;
    a.I = I;
    return layer(a, T, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" moe_status_t moe_layer_decode_indices(const void* x, const float* x_scales,
                                                 const int32_t* topk_idx, const float* topk_w,
                                                 int64_t T, int E, int k, int64_t H, int64_t I,
                                                 const void* w_up_packed,
                                                 const void* w_down_packed, void* out,
                                                 void* workspace, size_t workspace_bytes,
                                                 void* stream) {
    MOE_TRACE(__func__);
    LayerArgs a{};
    a.x = x;
    a.x_scales = x_scales;
    a.given_idx = topk_idx;
    a.given_w = topk_w;
    a.w_up = static_cast<const uint16_t*>(w_up_packed);
    a.w_down = static_cast<const uint16_t*>(w_down_packed);
    a.out = static_cast<uint16_t*>(out);
    a.E = E;
    a.k = k;
    a.H = H;
    a.I = I;
    return layer(a, T, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}
