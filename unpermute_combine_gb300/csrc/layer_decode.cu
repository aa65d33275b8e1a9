// layer_decode.cu -- moe_layer_decode, moe_layer_decode_indices: a whole MoE
// layer for a few tokens.
//
//   out[t] = sum_j p[t,j] * (silu(x_t Wg[e]^T) * (x_t Wu[e]^T)) Wd[e]^T,  e = idx[t,j]
//
// With up to 64 tokens a layer is bound by reading the weights of the experts
// that some token chose, once: 6 H I bytes each.  Two kernels stream them, the
// up projections and then the down projections, through the tensor cores with
// the operands swapped: 128 weight rows are the A tile (M = 128) and the few
// tokens of an expert the B tile (N = 16, 32, 48 or 64), so no part of the tile
// is padding that has to be read, and the weights go from TMA to shared memory
// to tcgen05.mma without passing a register.
//   warp 0       TMA producer: stages of 128 weight rows x 64 (16 KB) in a ring
//                that fills half of the SM's shared memory, so that two blocks
//                of either kernel fit an SM
//   warp 1       one thread issues the MMAs
//   warps 2..5   fill the B tiles: gathered token rows (e4m3 codes times their
//                scale) or hidden rows, one warp a stage, so that the latency of
//                four gathers overlaps (warp 2 also allocates the tensor memory)
//   warps 6..9   epilogue: silu(gate) * up, or the down products
// Precision: the MMA's operands are bf16, but a hidden value, and an e4m3 code
// times its scale, are not bf16 values.  Both are split into a bf16 value and
// the bf16 value of the rest (16 bits together) and take two MMAs into the same
// accumulator; the tensor cores idle here, so the second one costs nothing.
// The second kernel is launched to overlap the first (programmatic dependent
// launch): its blocks take the place of blocks that finish, and stream the down
// projections, which do not depend on the first kernel, until their rings are
// full; only then do they wait for it.
// The last block to finish a strip of 128 output columns adds a token's slots
// up, in slot order, so the result does not depend on which block that is.
// Every block works the routing out for itself (top-k, softmax, each expert's
// tokens) in shared memory: 64 tokens are too few for a launch of their own.
// Every wait on an mbarrier is bounded; one that gives up records
// MOE_ERR_TIMEOUT in the workspace status word.
#include "tensor_core.cuh"

namespace moe {
namespace {

constexpr int kMaxTokens = 64;
constexpr int kM = 128;                   // weight rows of one tile
constexpr int kK = 64;                    // K of a stage: one 128-byte swizzle row
constexpr int kBox = 64;                  // weight rows of one TMA box
constexpr int kTileBytes = kM * kK * 2;
constexpr int kUpCols = 64;               // hidden columns of an up tile: 64 gate + 64 up rows
constexpr int kMaxStages = 8;
constexpr int kLoaders = 4;               // warps that fill B tiles
constexpr int kThreads = 320;
constexpr int kExchBytes = 16 * kUpCols * 4;   // up values on their way to the gate's threads
constexpr int kBlocksPerSm = 2;
constexpr int kSmemBudget = 111 * 1024;   // dynamic shared memory of a block, two on an SM
constexpr int kMaxParts = 8;              // splits of the down projections' K

struct LayerArgs {
    const void* x;              // bf16 [T,H], or e4m3 codes
    const float* x_scales;      // NULL (bf16 x), or [T, H/128]
    const float* logits;        // NULL: the choices are given
    const int32_t* given_idx;   // [T,k], -1 = empty slot
    const float* given_w;       // [T,k]
    int32_t* topk_idx;          // written from the logits
    float* topk_w;
    uint16_t* out;              // [T,H] bf16
    WsHeader* header;
    uint32_t* arrivals;         // [H / kM] products of a strip that are done
    uint16_t* hidden;           // [2][T*k, I] bf16: the values, and what they leave
    float* y;                   // [parts][slots, H]
    int T, E, k;
    int64_t H, I;
    int nmax;                   // rows of a B tile: T rounded up to 16
    int stages;
    int spread;                 // blocks that fit the GPU at once
};

// ----------------------------------------------------------------- routing

// What every block knows of the routing, in shared memory.  A slot is a row of
// the workspace: experts in order, an expert's tokens in order.
struct Routing {
    float* w;                   // [T*k]
    unsigned long long* mask;   // [E] tokens of each expert
    int16_t* slot;              // [T*k] slot of a choice, -1 = empty
    uint16_t* first;            // [E] first slot of each expert
    uint16_t* active;           // [min(E, T*k)] experts with tokens
    uint8_t* token;             // [T*k] token of each slot
    int* count;                 // [3]: active experts, bad choices, slots
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
    r.slot = reinterpret_cast<int16_t*>(r.w + n);
    r.first = reinterpret_cast<uint16_t*>(r.slot + n);
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

// All threads of the block; ends with a barrier.  `publish`: writes the choices
// out.
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
            r.slot[t * k + lane] = int16_t(id);      // the expert, until slots are known
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
        if (lane == 0) { r.count[0] = act; r.count[2] = slots; }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int e = r.slot[i], t = i / k;
        if (e >= 0) {
            const int slot = r.first[e] + __popcll(r.mask[e] & ((1ull << t) - 1ull));
            r.token[slot] = uint8_t(t);
            r.slot[i] = int16_t(slot);
        }
    }
    __syncthreads();
}

// ------------------------------------------------------------------- tiles

// One work item: the tile of 128 weight rows at `strip` of an expert, over the
// stages [k0, k1) of its K.
struct Item {
    int e, first, n;            // expert, its first slot, its tokens
    int strip, part, k0, k1;
};

struct Work { int act, strips, parts, steps, items; };

template <bool kUp>
__device__ __forceinline__ Work work_of(const LayerArgs& a, const Routing& r) {
    Work w;
    w.act = r.count[0];
    w.strips = int(kUp ? a.I / kUpCols : a.H / kM);
    w.steps = int((kUp ? a.H : a.I) / kK);
    w.parts = 1;
    // the down products are sums over K, which may be cut to give more blocks work
    if (!kUp && w.act > 0)
        w.parts = max(1, min(min(kMaxParts, w.steps / 2), a.spread / (w.act * w.strips)));
    w.items = w.act * w.strips * w.parts;
    return w;
}

// Up: an expert's strips one after the other.  Down: a strip's experts and
// parts one after the other, so that strips finish, and are added up, early.
template <bool kUp>
__device__ __forceinline__ Item item_of(const Work& w, const Routing& r, int i) {
    Item it;
    const int q = kUp ? i : i / w.parts;
    it.part = kUp ? 0 : i % w.parts;
    const int act = kUp ? q / w.strips : q % w.act;
    it.strip = kUp ? q % w.strips : q / w.act;
    it.e = r.active[act];
    it.first = r.first[it.e];
    it.n = __popcll(r.mask[it.e]);
    it.k0 = it.part * w.steps / w.parts;
    it.k1 = (it.part + 1) * w.steps / w.parts;
    return it;
}

__device__ __forceinline__ int columns(int n) { return (n + 15) & ~15; }

// A float's bf16 value, and the bf16 value of what that leaves (0 for an
// infinity, so that it stays one).
__device__ __forceinline__ float bf16_rest(float v, float hi) {
    return (__float_as_uint(hi) & 0x7F800000u) == 0x7F800000u ? 0.0f : v - hi;
}

__device__ __forceinline__ void split8(const float* v, uint4& hi, uint4& lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = v[2 * i], b = v[2 * i + 1];
        h[i] = pack_bf16x2_rn(a, b);
        l[i] = pack_bf16x2_rn(bf16_rest(a, bf16lo_to_f32(h[i])), bf16_rest(b, bf16hi_to_f32(h[i])));
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

__device__ __forceinline__ uint4 ld_cg_v4(const void* p) {
    return __ldcg(static_cast<const uint4*>(p));
}

// Chunk c (8 values of K) of B row `row` in a tile with 128-byte swizzle.
__device__ __forceinline__ void put_chunk(uint8_t* tile, int row, int c, uint4 v) {
    *reinterpret_cast<uint4*>(tile + row * 128 + ((c ^ (row & 7)) << 4)) = v;
}

__device__ __forceinline__ void bar_epilogue() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Whether any of the epilogue's 128 threads says so; all of them get to know.
__device__ __forceinline__ bool any_epilogue(bool v) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n"
        " bar.red.or.pred p, 1, 128, q;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(r) : "r"(uint32_t(v)) : "memory");
    return r != 0;
}

// out[t, strip] = sum over the slots, in order, of the weighted down products.
// 128 threads: lane = 4 columns, warp = every fourth token.
__device__ void add_up(const LayerArgs& a, const Routing& r, const Work& w, int strip) {
    const int lane = int(lane_id());
    const int64_t h = int64_t(strip) * kM + lane * 4, part = int64_t(r.count[2]) * a.H;
    for (int t = (threadIdx.x >> 5) & 3; t < a.T; t += 4) {
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int j = 0; j < a.k; ++j) {
            const int slot = r.slot[t * a.k + j];
            if (slot < 0) continue;
            const float* p = a.y + int64_t(slot) * a.H + h;
            float4 v = __ldcg(reinterpret_cast<const float4*>(p));
            for (int q = 1; q < w.parts; ++q) {
                const float4 o = __ldcg(reinterpret_cast<const float4*>(p + q * part));
                v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
            }
            const float pw = r.w[t * a.k + j];
            s.x = fmaf(pw, v.x, s.x);
            s.y = fmaf(pw, v.y, s.y);
            s.z = fmaf(pw, v.z, s.z);
            s.w = fmaf(pw, v.w, s.w);
        }
        *reinterpret_cast<uint2*>(a.out + t * a.H + h) =
            make_uint2(pack_bf16x2_rn(s.x, s.y), pack_bf16x2_rn(s.z, s.w));
    }
}

// kUp: hidden = silu(x Wg^T) * (x Wu^T) of every active expert's tokens;
// otherwise y = hidden Wd^T, and out.  kB2: the B rows come in two bf16 parts
// (e4m3 x, or hidden rows).
template <bool kUp, bool kB2>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
layer_kernel(const __grid_constant__ CUtensorMap map_w, const LayerArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_a[kMaxStages], full_b[kMaxStages], empty[kMaxStages];
    __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_failed;
    __shared__ int s_last;

    const int warp = threadIdx.x >> 5, lane = int(lane_id());
    const int b_bytes = a.nmax * 128 * (kB2 ? 2 : 1), stage_bytes = kTileBytes + b_bytes;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    float* exch = reinterpret_cast<float*>(ring + a.stages * stage_bytes);     // [16][kUpCols]
    const Routing r = carve_routing(ring + a.stages * stage_bytes + kExchBytes, a.T, a.E, a.k);

    if (threadIdx.x == 0) {
        s_failed = 0;
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(smem_addr(&full_a[s]), 1);
            mbar_init(smem_addr(&full_b[s]), 1);
            mbar_init(smem_addr(&empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&acc_full[b]), 1);
            mbar_init(smem_addr(&acc_empty[b]), 128);
        }
        mbar_fence_init();
    }
    // two accumulators of nmax fp32 columns, a power of two of at least 32
    const uint32_t tmem_cols = a.nmax <= 16 ? 32u : a.nmax <= 32 ? 64u : 128u;
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_addr(&s_tmem)), "r"(tmem_cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    route(a, r, kUp && a.logits && blockIdx.x == 0);       // ends with a barrier
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const Work w = work_of<kUp>(a, r);
    if (kUp) {
        // every block of this kernel is resident and has its tensor memory
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        if (blockIdx.x == 0) {
            if (threadIdx.x == 0) {
                a.header->status = r.count[1] ? MOE_ERR_DEVICE_CHECK : MOE_OK;
                a.header->detail = 0;
            }
            for (int64_t i = threadIdx.x; i < a.H / kM; i += blockDim.x) a.arrivals[i] = 0u;
        }
    } else if (w.items == 0) {                             // every slot is empty
        for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < a.T * a.H;
             i += int64_t(gridDim.x) * kThreads)
            a.out[i] = 0;
    }

    if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------- TMA producer
            uint32_t it = 0;
            for (int i = blockIdx.x; i < w.items && !s_failed; i += gridDim.x) {
                const Item m = item_of<kUp>(w, r, i);
                // the two boxes: 64 gate rows and the matching up rows, or 128 rows of Wd
                const int row = kUp ? int(m.e * 2 * a.I) + m.strip / 2 * 256 + m.strip % 2 * 64
                                    : int(m.e * a.H) + m.strip * kM;
                const int row2 = row + (kUp ? 128 : kBox);
                for (int ks = m.k0; ks < m.k1; ++ks, ++it) {
                    const int s = it % a.stages;
                    const uint32_t turn = it / a.stages;
                    if (!kUp && turn == 1 && s == 0) wait_for_predecessor();   // the ring is full
                    if (!mbar_wait(smem_addr(&empty[s]), (turn & 1u) ^ 1u)) { s_failed = 1; break; }
                    const uint32_t dst = smem_addr(ring + s * stage_bytes);
                    const uint32_t bar = smem_addr(&full_a[s]);
                    mbar_expect_tx(bar, kTileBytes);
                    tma_load_2d(dst, &map_w, ks * kK, row, bar);
                    tma_load_2d(dst + kTileBytes / 2, &map_w, ks * kK, row2, bar);
                }
            }
            // a block that gave up leaves no copy of its own in flight
            if (s_failed)
                for (uint32_t b = it > uint32_t(a.stages) ? it - a.stages : 0; b < it; ++b)
                    mbar_wait(smem_addr(&full_a[b % a.stages]), (b / a.stages) & 1u);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ------------------------------------------------------ MMA issuer
            if (!kUp) wait_for_predecessor();
            uint32_t it = 0, tile = 0;
            for (int i = blockIdx.x; i < w.items && !s_failed; i += gridDim.x, ++tile) {
                const Item m = item_of<kUp>(w, r, i);
                const uint32_t idesc = idesc_bf16(kM, columns(m.n));
                const uint32_t buf = tile & 1u, acc = tmem + buf * a.nmax;
                if (!mbar_wait(smem_addr(&acc_empty[buf]), ((tile >> 1) & 1u) ^ 1u)) { s_failed = 1; break; }
                tc_fence_after();
                for (int ks = m.k0; ks < m.k1; ++ks, ++it) {
                    const int s = it % a.stages;
                    const uint32_t ph = (it / a.stages) & 1u;
                    if (!mbar_wait(smem_addr(&full_b[s]), ph) ||
                        !mbar_wait(smem_addr(&full_a[s]), ph)) { s_failed = 1; break; }
                    tc_fence_after();
                    const uint32_t wa = smem_addr(ring + s * stage_bytes), xb = wa + kTileBytes;
#pragma unroll
                    for (int kk = 0; kk < kK / 16; ++kk) {
                        const uint64_t ad = smem_desc_k128(wa + kk * 32);
                        mma_bf16(acc, ad, smem_desc_k128(xb + kk * 32), idesc, ks != m.k0 || kk);
                        if (kB2)
                            mma_bf16(acc, ad, smem_desc_k128(xb + a.nmax * 128 + kk * 32), idesc, 1);
                    }
                    mma_commit(smem_addr(&empty[s]));
                }
                if (s_failed) break;
                mma_commit(smem_addr(&acc_full[buf]));
            }
        }
    } else if (warp < 2 + kLoaders) {
        // ----------------------------------------------------------- B loaders
        if (!kUp) wait_for_predecessor();                  // the hidden rows
        // No more warps than stages: a warp that waits for a stage has seen the
        // use before its own last one end, so the stage's barrier can be at most
        // one phase behind and the parity is not mistaken for an older one.
        const uint32_t loaders = min(kLoaders, a.stages), mine = warp - 2;
        uint32_t it = 0;
        bool stop = false;                                 // the same in all lanes
        for (int i = blockIdx.x; i < w.items && !stop; i += gridDim.x) {
            const Item m = item_of<kUp>(w, r, i);
            const int chunks = m.n * 8;
            for (int ks = m.k0; ks < m.k1; ++ks, ++it) {
                if (it % loaders != mine) continue;
                const int s = it % a.stages;
                uint8_t* tile = ring + s * stage_bytes + kTileBytes;
                bool ready = false;
                for (int c0 = 0; c0 < chunks; c0 += 128) {
                    // up to four chunks a lane in flight; the first ones before the wait
                    uint4 v[4], v2[4];
                    float sc[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int c = c0 + q * 32 + lane, row = c >> 3, col = ks * kK + (c & 7) * 8;
                        if (c >= chunks) continue;
                        if (kUp && !kB2) {
                            v[q] = ld_nc_v4(static_cast<const uint16_t*>(a.x) +
                                            r.token[m.first + row] * a.H + col);
                        } else if (kUp) {
                            const int t = r.token[m.first + row];
                            const uint2 code = __ldg(reinterpret_cast<const uint2*>(
                                static_cast<const uint8_t*>(a.x) + t * a.H + col));
                            v[q].x = code.x;
                            v[q].y = code.y;
                            sc[q] = __ldg(a.x_scales + t * (a.H / 128) + col / 128);
                        } else {
                            const uint16_t* p = a.hidden + int64_t(m.first + row) * a.I + col;
                            v[q] = ld_cg_v4(p);
                            v2[q] = ld_cg_v4(p + int64_t(a.T) * a.k * a.I);
                        }
                    }
                    if (!ready) {
                        ready = mbar_wait(smem_addr(&empty[s]), ((it / a.stages) & 1u) ^ 1u);
                        if (!ready) { s_failed = 1; break; }
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int c = c0 + q * 32 + lane, row = c >> 3;
                        if (c >= chunks) continue;
                        if (kUp && kB2) {
                            float f[8];
                            e4m3x2_to_f32(v[q].x & 0xFFFFu, f[0], f[1]);
                            e4m3x2_to_f32(v[q].x >> 16, f[2], f[3]);
                            e4m3x2_to_f32(v[q].y & 0xFFFFu, f[4], f[5]);
                            e4m3x2_to_f32(v[q].y >> 16, f[6], f[7]);
#pragma unroll
                            for (int e = 0; e < 8; ++e) f[e] *= sc[q];
                            split8(f, v[q], v2[q]);
                        }
                        put_chunk(tile, row, c & 7, v[q]);
                        if (kB2) put_chunk(tile + a.nmax * 128, row, c & 7, v2[q]);
                    }
                }
                // each thread orders its writes before the tensor core's reads
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                stop = __any_sync(0xFFFFFFFFu, s_failed != 0);
                if (stop) break;
                if (lane == 0) mbar_arrive(smem_addr(&full_b[s]));
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        if (!kUp) wait_for_predecessor();                  // the arrival counts
        const int q = warp & 3, row = q * 32 + lane;       // TMEM lane quadrant, weight row
        uint32_t tile = 0;
        for (int i = blockIdx.x; i < w.items; i += gridDim.x, ++tile) {
            const Item m = item_of<kUp>(w, r, i);
            const uint32_t buf = tile & 1u, acc = tmem + buf * a.nmax + (uint32_t(q * 32) << 16);
            const bool ok = !s_failed && mbar_wait(smem_addr(&acc_full[buf]), (tile >> 1) & 1u);
            // all 128 threads go on, or none
            if (any_epilogue(!ok)) { s_failed = 1; break; }
            tc_fence_after();
            for (int c0 = 0; c0 < m.n; c0 += 16) {
                float v[16];
                tmem_ld16(acc + c0, v);
                if (kUp) {
                    // rows 0-63 hold the gate, rows 64-127 the up values
                    if (q >= 2) {
#pragma unroll
                        for (int c = 0; c < 16; ++c) exch[c * kUpCols + row - 64] = v[c];
                    }
                    bar_epilogue();
                    if (q < 2) {
                        uint16_t* hp = a.hidden + int64_t(m.first + c0) * a.I + m.strip * kUpCols + row;
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            if (c0 + c >= m.n) break;
                            const float h = v[c] / (1.0f + expf(-v[c])) * exch[c * kUpCols + row];
                            const uint16_t hi = f32_to_bf16_rn(h);
                            hp[c * a.I] = hi;
                            hp[(int64_t(a.T) * a.k + c) * a.I] =
                                f32_to_bf16_rn(bf16_rest(h, bf16_to_f32(hi)));
                        }
                    }
                    bar_epilogue();
                } else {
                    float* yp = a.y + (int64_t(m.part) * r.count[2] + m.first + c0) * a.H +
                                m.strip * kM + row;
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        if (c0 + c < m.n) yp[c * a.H] = v[c];
                }
            }
            tc_fence_before();
            mbar_arrive(smem_addr(&acc_empty[buf]));
            if (!kUp) {
                bar_epilogue();
                if (row == 0) {
                    __threadfence();
                    s_last = atomicAdd(&a.arrivals[m.strip], 1u) == uint32_t(w.act * w.parts - 1);
                    __threadfence();
                }
                bar_epilogue();
                if (s_last) add_up(a, r, w, m.strip);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (s_failed && threadIdx.x == 0) {
        a.header->status = MOE_ERR_TIMEOUT;
        a.header->detail = blockIdx.x;
    }
    __syncwarp();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                     :: "r"(tmem), "r"(tmem_cols) : "memory");
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

// Items that the down projections may be split into: a bound of the blocks that
// any GPU of this kind holds at once.
constexpr int64_t kSpread = 320;

struct Layout { size_t arrivals, hidden, y, total; };

Layout workspace_layout(int64_t T, int k, int64_t H, int64_t I) {
    const size_t n = size_t(T) * k;
    Layout l;
    l.arrivals = kWsAlign;
    l.hidden = l.arrivals + align_up(size_t(H / kM) * 4, kWsAlign);
    l.y = l.hidden + align_up(n * size_t(I) * 4, kWsAlign);
    // unsplit: n rows of H; split: no more than kSpread strips of kM columns
    // over at most T tokens of an expert (work_of)
    l.total = l.y + align_up(max64(int64_t(n) * H, T * kSpread * kM) * 4, kWsAlign);
    return l;
}

int stage_bytes(const LayerArgs& a, bool two_parts) {
    return kTileBytes + a.nmax * 128 * (two_parts ? 2 : 1);
}

// As many stages as half of an SM's shared memory holds: 2 (64 tokens, 1024
// experts, k = 32, two parts) to 8; 5 for up to 16 tokens.
int ring_stages(const LayerArgs& a, bool two_parts) {
    const int left = kSmemBudget - 1024 - kExchBytes - int(routing_bytes(a.T, a.E, a.k));
    const int n = left / stage_bytes(a, two_parts);
    return n < kMaxStages ? n : kMaxStages;
}

size_t smem_bytes(const LayerArgs& a, bool two_parts) {
    return 1024 + size_t(a.stages) * stage_bytes(a, two_parts) + kExchBytes +
           routing_bytes(a.T, a.E, a.k);
}

moe_status_t layer(LayerArgs a, const void* w_up, const void* w_down, int64_t T, void* workspace, size_t workspace_bytes,
                   cudaStream_t s) {
    const moe_status_t st = check_layer(T, a.E, a.k, a.H, a.I);
    if (st != MOE_OK) return st;
    const Layout l = workspace_layout(T, a.k, a.H, a.I);
    const bool choices = a.logits ? a.topk_idx && a.topk_w : a.given_idx && a.given_w;
    if (T > 0 && (!a.x || !choices || !w_up || !w_down || !a.out)) return MOE_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) ||
        workspace_bytes < l.total)
        return MOE_ERR_WORKSPACE;
    if (!aligned16(a.x) || !aligned16(w_up) || !aligned16(w_down) || !aligned16(a.out) ||
        !aligned4(a.x_scales) || !aligned4(a.logits) || !aligned4(a.given_idx) ||
        !aligned4(a.given_w) || !aligned4(a.topk_idx) || !aligned4(a.topk_w))
        return MOE_ERR_INVALID_ARG;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.header = reinterpret_cast<WsHeader*>(ws);
    if (T == 0)
        return cudaMemsetAsync(ws, 0, 8, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    a.T = int(T);
    a.arrivals = reinterpret_cast<uint32_t*>(ws + l.arrivals);
    a.hidden = reinterpret_cast<uint16_t*>(ws + l.hidden);
    a.y = reinterpret_cast<float*>(ws + l.y);
    a.nmax = (a.T + 15) / 16 * 16;
    a.spread = int(min64(int64_t(sm_count()) * kBlocksPerSm, kSpread));

    CUtensorMap m_up, m_down;
    if (!make_map(&m_up, w_up, int64_t(a.E) * 2 * a.I, a.H, kBox) ||
        !make_map(&m_down, w_down, int64_t(a.E) * a.H, a.I, kBox))
        return MOE_ERR_CUDA;
    const int64_t experts = min64(a.E, T * a.k);
    const auto blocks = [&](int64_t items) { return unsigned(min64(items, a.spread)); };
    const bool fp8 = a.x_scales != nullptr;
    const auto up = fp8 ? layer_kernel<true, true> : layer_kernel<true, false>;
    const auto down = layer_kernel<false, true>;
    a.stages = ring_stages(a, fp8);
    size_t smem = smem_bytes(a, fp8);
    if (!opt_in_smem((const void*)up, int(smem))) return MOE_ERR_CUDA;
    up<<<blocks(experts * (a.I / kUpCols)), kThreads, smem, s>>>(m_up, a);
    if (launch_status() != MOE_OK) return MOE_ERR_CUDA;
    a.stages = ring_stages(a, true);
    smem = smem_bytes(a, true);
    if (!opt_in_smem((const void*)down, int(smem))) return MOE_ERR_CUDA;
    return launch_dependent(down, unsigned(a.spread), kThreads, smem, s, m_down, a) == cudaSuccess
               ? MOE_OK : MOE_ERR_CUDA;
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
    a.out = static_cast<uint16_t*>(out);
    a.E = E;
    a.k = k;
    a.H = H;
    a.I = I;
    return layer(a, w_up_packed, w_down_packed, T, workspace, workspace_bytes,
                 static_cast<cudaStream_t>(stream));
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
    a.out = static_cast<uint16_t*>(out);
    a.E = E;
    a.k = k;
    a.H = H;
    a.I = I;
    return layer(a, w_up_packed, w_down_packed, T, workspace, workspace_bytes,
                 static_cast<cudaStream_t>(stream));
}
