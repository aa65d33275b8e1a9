// layer_decode.cu -- moe_layer_decode, moe_layer_decode_indices: a whole MoE
// layer for a few tokens.
//
//   out[t] = sum_j p[t,j] * (silu(x_t Wg[e]^T) * (x_t Wu[e]^T)) Wd[e]^T,  e = idx[t,j]
//
// With up to 64 tokens a layer is bound by reading the weights of the experts
// that some token chose, once: 6 H I bytes each.  Two kernels stream them, the
// up projections and then the down projections, through the tensor cores with
// the operands swapped: up to 128 weight rows are the A tile (M = 128) and a
// group of up to 64 tokens of one expert the B tile (N), so nothing that is read
// is padding, and the weights go from TMA to shared memory to tcgen05.mma
// without passing a register.  A third, small kernel adds a token's slots up.
//   warp 0       TMA producer: stages of weight rows x 64 or 128 of K, in a ring
//                that fills half of the SM's shared memory, so that two blocks
//                of either kernel fit an SM
//   warp 1       one thread issues the MMAs
//   warps 2..5   fill the B tiles: gathered token rows (e4m3 codes times their
//                scale) or hidden rows, one warp a stage, so that the latency of
//                four gathers overlaps (warp 2 also allocates the tensor memory)
//   warps 6..9   epilogue: silu(gate) * up, or the down products
// Precision: the MMA's operands are bf16, but a hidden value, and an e4m3 code
// times its scale, are not bf16 values.  Both are split into a bf16 value and
// the bf16 value of the rest (16 bits together), which stand side by side as
// columns of one B tile; the epilogue adds the two columns.  An MMA this narrow
// takes as long as its A tile, so the second part costs next to nothing.
// The second kernel is launched to overlap the first (programmatic dependent
// launch): its blocks take the place of blocks that finish, and stream the down
// projections, which do not depend on the first kernel, until their rings are
// full; only then do they wait for it.
// Every block works the routing out for itself (top-k, softmax, each expert's
// tokens) in shared memory: 64 tokens are too few for a launch of their own.
// Every wait on an mbarrier is bounded; one that gives up records
// MOE_ERR_TIMEOUT in the workspace status word.
#include "tensor_core.cuh"

namespace moe {
namespace {

constexpr int kMaxTokens = 64;
constexpr int kM = 128;                   // rows of an MMA, weight rows of a down tile
constexpr int kBigBox = 64, kSmallBox = 16;    // weight rows of a TMA box
constexpr int kMaxStages = 16;
constexpr int kLoaders = 4;               // warps that fill B tiles
constexpr int kThreads = 320;
constexpr int kExchBytes = 8 * 64 * 4;    // up values on their way to the gate's threads
constexpr int kBlocksPerSm = 2;
constexpr int kSmemBytes = 111 * 1024;    // dynamic shared memory of a block, two on an SM
constexpr int kMaxParts = 8;              // splits of the down projections' K
constexpr int kSumThreads = 128;

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
    int* slots;                 // [2 + T*k]: units, slots in use, slot of each choice
    float* weights;             // [T*k]
    uint16_t* hidden;           // [2][T*k, I] bf16: the values, and what they leave
    float* y;                   // [parts][slots, H]
    int T, E, k;
    int64_t H, I;
    int spread;                 // blocks that fit the GPU at once
    uint32_t tmem_cols;
};

// ----------------------------------------------------------------- routing

// What every block knows of the routing, in shared memory.  A slot is a row of
// the workspace: experts in order, an expert's tokens in order.  A unit is a
// group of an expert's tokens that share a B tile.
struct Routing {
    float* w;                   // [T*k]
    unsigned long long* mask;   // [E] tokens of each expert
    int16_t* slot;              // [T*k] slot of a choice, -1 = empty
    uint16_t* first;            // [E] first slot of each expert
    uint16_t* unit;             // [T*k] expert of each unit
    uint8_t* group;             // [T*k] which group of the expert's tokens it is
    uint8_t* token;             // [T*k] token of each slot
    int* count;                 // [4]: units, bad choices, slots, tokens of a group
};

__host__ __device__ inline size_t routing_bytes(int T, int E, int k) {
    const size_t n = size_t(T) * k;
    const size_t b = 16 + size_t(E) * 8 + n * 4 + n * 2 + size_t(E) * 2 + n * 2 + n + n;
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
    r.unit = r.first + E;
    r.group = reinterpret_cast<uint8_t*>(r.unit + n);
    r.token = r.group + n;
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
        // Tokens of a group: a large group keeps its rows' place in every stage
        // and leaves less of the ring to weights, a small one reads the weights
        // of an expert with more tokens again, from L2.  16, unless that is a
        // tenth more reads; then 32, by the same rule; then 64.
        int act = 0, by16 = 0, by32 = 0;
        for (int e = lane; e < E; e += 32) {
            const int c = __popcll(r.mask[e]);
            act += c > 0;
            by16 += (c + 15) / 16;
            by32 += (c + 31) / 32;
        }
        act = __reduce_add_sync(0xFFFFFFFFu, act);
        by16 = __reduce_add_sync(0xFFFFFFFFu, by16);
        by32 = __reduce_add_sync(0xFFFFFFFFu, by32);
        const int g = by16 * 10 <= act * 11 ? 16 : by32 * 10 <= act * 11 ? 32 : 64;
        int slots = 0, units = 0;
        for (int base = 0; base < E; base += 32) {
            const int e = base + lane;
            const int c = e < E ? __popcll(r.mask[e]) : 0, u = (c + g - 1) / g;
            int both = c << 16 | u, incl = both;           // at most 2048 of each
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (lane >= o) incl += v;
            }
            if (e < E) r.first[e] = uint16_t(slots + (incl >> 16) - c);
            for (int i = 0; i < u; ++i) {
                r.unit[units + (incl & 0xFFFF) - u + i] = uint16_t(e);
                r.group[units + (incl & 0xFFFF) - u + i] = uint8_t(i);
            }
            const int all = __shfl_sync(0xFFFFFFFFu, incl, 31);
            slots += all >> 16;
            units += all & 0xFFFF;
        }
        if (lane == 0) { r.count[0] = units; r.count[2] = slots; r.count[3] = g; }
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

// How the routing is cut into work items, the same in every block.
struct Work {
    int units, strips, parts, items;
    int cols;                   // up: hidden columns of a tile (as many gate and up rows)
    int rows;                   // weight rows of a tile
    int group, subs, steps;     // tokens of a B tile; sub-tiles of a stage; stages of K
    int stage_bytes, stages;
};

// parts of the down projections' K, so that there is work for every block
__device__ __forceinline__ int down_parts(const LayerArgs& a, int units) {
    const int strips = int(a.H / kM), most = int(min64(kMaxParts, a.I / 128));
    return units > 0 ? max(1, min(most, a.spread / (units * strips))) : 1;
}

template <bool kUp, bool kB2>
__device__ __forceinline__ Work work_of(const LayerArgs& a, const Routing& r, int ring_bytes) {
    Work w;
    w.units = r.count[0];
    w.group = r.count[3];
    w.parts = kUp ? 1 : down_parts(a, w.units);
    // narrower up tiles where there are not enough wide ones for every block
    w.cols = 64;
    if (kUp)
        while (w.cols > 16 && w.units * int(a.I / w.cols) * 4 < a.spread * 3) w.cols /= 2;
    w.rows = kUp ? 2 * w.cols : kM;
    w.strips = int(kUp ? a.I / w.cols : a.H / kM);
    w.items = w.units * w.strips * w.parts;
    // two sub-tiles a stage (256 bytes of a row) where three such stages fit
    const int sub = (w.rows + w.group * (kB2 ? 2 : 1)) * 128;
    const int left = ring_bytes - (kM - w.rows) * 128;     // an MMA reads kM rows all the same
    w.subs = 6 * sub <= left ? 2 : 1;
    w.stage_bytes = w.subs * sub;
    w.stages = min(kMaxStages, left / w.stage_bytes);
    w.steps = int((kUp ? a.H : a.I) / (64 * w.subs));
    return w;
}

// One work item: a tile of weight rows over the stages [k0, k1) of its K.
struct Item {
    int e, first, n;            // expert, the unit's first slot, its tokens
    int strip, part, k0, k1;
};

// Up: a unit's strips one after the other.  Down: a strip's units and parts.
template <bool kUp>
__device__ __forceinline__ Item item_of(const Work& w, const Routing& r, int i) {
    Item it;
    const int q = kUp ? i : i / w.parts;
    it.part = kUp ? 0 : i % w.parts;
    const int unit = kUp ? q / w.strips : q % w.units;
    it.strip = kUp ? q % w.strips : q / w.units;
    it.e = r.unit[unit];
    const int at = r.group[unit] * w.group;
    it.first = r.first[it.e] + at;
    it.n = min(w.group, __popcll(r.mask[it.e]) - at);
    it.k0 = it.part * w.steps / w.parts;
    it.k1 = (it.part + 1) * w.steps / w.parts;
    return it;
}

// B rows of n tokens: each part of two takes a multiple of 8, one alone of 16,
// so that N is a multiple of 16.
template <bool kB2>
__device__ __forceinline__ int b_rows(int n) { return kB2 ? (n + 7) & ~7 : (n + 15) & ~15; }

// What a float's bf16 value leaves of it (0 for an infinity, so that it stays one).
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

// Chunk c (8 values of K) of a B row in a sub-tile with 128-byte swizzle.
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

// kUp: hidden = silu(x Wg^T) * (x Wu^T) of every active expert's tokens;
// otherwise y = hidden Wd^T.  kB2: the B rows come in two bf16 parts (e4m3 x,
// or hidden rows).
template <bool kUp, bool kB2>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
layer_kernel(const __grid_constant__ CUtensorMap map_big,
             const __grid_constant__ CUtensorMap map_small, const LayerArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_a[kMaxStages], full_b[kMaxStages], empty[kMaxStages];
    __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_failed;

    const int warp = threadIdx.x >> 5, lane = int(lane_id());
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    const int ring_bytes = kSmemBytes - 1024 - kExchBytes - int(routing_bytes(a.T, a.E, a.k));
    float* exch = reinterpret_cast<float*>(ring + ring_bytes);                 // [8][cols]
    const Routing r = carve_routing(ring + ring_bytes + kExchBytes, a.T, a.E, a.k);

    if (threadIdx.x == 0) {
        s_failed = 0;
        for (int s = 0; s < kMaxStages; ++s) {
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
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_addr(&s_tmem)), "r"(a.tmem_cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    route(a, r, kUp && a.logits && blockIdx.x == 0);       // ends with a barrier
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const Work w = work_of<kUp, kB2>(a, r, ring_bytes);
    const int b_sub = w.group * (kB2 ? 2 : 1) * 128, a_sub = w.rows * 128;
    // every block of this kernel is resident and has its tensor memory
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (kUp && blockIdx.x == 0) {                          // for the sum over slots
        if (threadIdx.x == 0) {
            a.header->status = r.count[1] ? MOE_ERR_DEVICE_CHECK : MOE_OK;
            a.header->detail = 0;
            a.slots[0] = w.units;
            a.slots[1] = r.count[2];
        }
        for (int i = threadIdx.x; i < a.T * a.k; i += kThreads) {
            a.slots[2 + i] = r.slot[i];
            a.weights[i] = r.w[i];
        }
    }

    if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------- TMA producer
            uint32_t it = 0;
            for (int i = blockIdx.x; i < w.items && !s_failed; i += gridDim.x) {
                const Item m = item_of<kUp>(w, r, i);
                // gate rows and the matching up rows (blocks of 128 each), or rows of Wd
                const int col = m.strip * w.cols;
                const int row = kUp ? int(m.e * 2 * a.I) + col / 128 * 256 + col % 128
                                    : int(m.e * a.H) + m.strip * kM;
                const int row2 = row + (kUp ? 128 : kM / 2), half = w.rows / 2;
                for (int ks = m.k0; ks < m.k1; ++ks, ++it) {
                    const int s = it % w.stages;
                    const uint32_t turn = it / w.stages;
                    if (!kUp && turn == 1 && s == 0) wait_for_predecessor();   // the ring is full
                    if (!mbar_wait(smem_addr(&empty[s]), (turn & 1u) ^ 1u)) { s_failed = 1; break; }
                    const uint32_t bar = smem_addr(&full_a[s]);
                    mbar_expect_tx(bar, w.subs * a_sub);
                    for (int u = 0; u < w.subs; ++u) {
                        const uint32_t dst = smem_addr(ring + s * w.stage_bytes + u * a_sub);
                        const int c = (ks * w.subs + u) * 64;
                        if (half == kBigBox) {
                            tma_load_2d(dst, &map_big, c, row, bar);
                            tma_load_2d(dst + kBigBox * 128, &map_big, c, row2, bar);
                        } else {
                            for (int b = 0; b < half; b += kSmallBox) {
                                tma_load_2d(dst + b * 128, &map_small, c, row + b, bar);
                                tma_load_2d(dst + (half + b) * 128, &map_small, c, row2 + b, bar);
                            }
                        }
                    }
                }
            }
            // a block that gave up leaves no copy of its own in flight
            if (s_failed)
                for (uint32_t b = it > uint32_t(w.stages) ? it - w.stages : 0; b < it; ++b)
                    mbar_wait(smem_addr(&full_a[b % w.stages]), (b / w.stages) & 1u);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ------------------------------------------------------ MMA issuer
            if (!kUp) wait_for_predecessor();
            uint32_t it = 0, tile = 0;
            for (int i = blockIdx.x; i < w.items && !s_failed; i += gridDim.x, ++tile) {
                const Item m = item_of<kUp>(w, r, i);
                const uint32_t idesc = idesc_bf16(kM, b_rows<kB2>(m.n) * (kB2 ? 2 : 1));
                const uint32_t buf = tile & 1u, acc = tmem + buf * (a.tmem_cols / 2);
                if (!mbar_wait(smem_addr(&acc_empty[buf]), ((tile >> 1) & 1u) ^ 1u)) { s_failed = 1; break; }
                tc_fence_after();
                for (int ks = m.k0; ks < m.k1; ++ks, ++it) {
                    const int s = it % w.stages;
                    const uint32_t ph = (it / w.stages) & 1u;
                    if (!mbar_wait(smem_addr(&full_b[s]), ph) ||
                        !mbar_wait(smem_addr(&full_a[s]), ph)) { s_failed = 1; break; }
                    tc_fence_after();
                    const uint32_t wa = smem_addr(ring + s * w.stage_bytes), xb = wa + w.subs * a_sub;
                    for (int u = 0; u < w.subs; ++u) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_bf16(acc, smem_desc_k128(wa + u * a_sub + kk * 32),
                                     smem_desc_k128(xb + u * b_sub + kk * 32), idesc,
                                     ks != m.k0 || u || kk);
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
        const uint32_t loaders = min(kLoaders, w.stages), mine = warp - 2;
        const int row_chunks = 8 * w.subs, row_shift = w.subs == 2 ? 4 : 3;
        uint32_t it = 0;
        bool stop = false;                                 // the same in all lanes
        for (int i = blockIdx.x; i < w.items && !stop; i += gridDim.x) {
            const Item m = item_of<kUp>(w, r, i);
            const int chunks = m.n * row_chunks, part2 = b_rows<kB2>(m.n) * 128;
            for (int ks = m.k0; ks < m.k1; ++ks, ++it) {
                if (it % loaders != mine) continue;
                const int s = it % w.stages;
                uint8_t* tile = ring + s * w.stage_bytes + w.subs * a_sub;
                bool ready = false;
                for (int c0 = 0; c0 < chunks; c0 += 128) {
                    // up to four chunks a lane in flight; the first ones before the wait
                    uint4 v[4], v2[4];
                    float sc[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int c = c0 + q * 32 + lane, row = c >> row_shift;
                        const int col = (ks * row_chunks + (c & (row_chunks - 1))) * 8;
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
                            v[q] = __ldcg(reinterpret_cast<const uint4*>(p));
                            v2[q] = __ldcg(reinterpret_cast<const uint4*>(p + int64_t(a.T) * a.k * a.I));
                        }
                    }
                    if (!ready) {
                        ready = mbar_wait(smem_addr(&empty[s]), ((it / w.stages) & 1u) ^ 1u);
                        if (!ready) { s_failed = 1; break; }
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int c = c0 + q * 32 + lane, row = c >> row_shift;
                        const int j = c & (row_chunks - 1);
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
                        uint8_t* sub = tile + (j >> 3) * b_sub;
                        put_chunk(sub, row, j & 7, v[q]);
                        if (kB2) put_chunk(sub + part2, row, j & 7, v2[q]);
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
        if (!kUp) wait_for_predecessor();                  // y may still be read
        const int q = warp & 3, row = q * 32 + lane;       // TMEM lane quadrant, tile row
        uint32_t tile = 0;
        for (int i = blockIdx.x; i < w.items; i += gridDim.x, ++tile) {
            const Item m = item_of<kUp>(w, r, i);
            const uint32_t buf = tile & 1u;
            const uint32_t acc = tmem + buf * (a.tmem_cols / 2) + (uint32_t(q * 32) << 16);
            const bool ok = !s_failed && mbar_wait(smem_addr(&acc_full[buf]), (tile >> 1) & 1u);
            // all 128 threads go on, or none
            if (any_epilogue(!ok)) { s_failed = 1; break; }
            tc_fence_after();
            for (int c0 = 0; c0 < m.n; c0 += 8) {
                float v[8];
                tmem_ld8(acc + c0, v);
                if (kB2) {
                    float lo[8];
                    tmem_ld8(acc + b_rows<kB2>(m.n) + c0, lo);
#pragma unroll
                    for (int c = 0; c < 8; ++c) v[c] += lo[c];
                }
                if (kUp) {
                    // the tile's first rows hold the gate, the next ones the up values
                    if (row >= w.cols && row < 2 * w.cols) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) exch[c * 64 + row - w.cols] = v[c];
                    }
                    bar_epilogue();
                    if (row < w.cols) {
                        uint16_t* hp = a.hidden + int64_t(m.first + c0) * a.I + m.strip * w.cols + row;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            if (c0 + c >= m.n) break;
                            const float h = v[c] / (1.0f + expf(-v[c])) * exch[c * 64 + row];
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
                    for (int c = 0; c < 8; ++c)
                        if (c0 + c < m.n) yp[c * a.H] = v[c];
                }
            }
            tc_fence_before();
            mbar_arrive(smem_addr(&acc_empty[buf]));
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
                     :: "r"(tmem), "r"(a.tmem_cols) : "memory");
}

// out[t] = sum over the slots, in order, of the weighted down products.  A thread
// has 4 columns of a token.
__global__ void __launch_bounds__(kSumThreads) layer_sum_kernel(const LayerArgs a) {
    __shared__ int s_slot[kMaxTopK];
    __shared__ float s_w[kMaxTopK];
    const int t = blockIdx.y;
    const int64_t h = (int64_t(blockIdx.x) * kSumThreads + threadIdx.x) * 4;
    wait_for_predecessor();
    if (int(threadIdx.x) < a.k) {
        s_slot[threadIdx.x] = __ldcg(a.slots + 2 + t * a.k + threadIdx.x);
        s_w[threadIdx.x] = __ldcg(a.weights + t * a.k + threadIdx.x);
    }
    const int parts = down_parts(a, __ldcg(a.slots));
    const int64_t part = int64_t(__ldcg(a.slots + 1)) * a.H;
    __syncthreads();
    if (h >= a.H) return;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int q = 0; q < parts; ++q) {
#pragma unroll 8
        for (int j = 0; j < a.k; ++j) {
            const int slot = s_slot[j];
            const float w = s_w[j];
            // no branch around the load, so that eight of them are in flight
            const float4 v = __ldcg(reinterpret_cast<const float4*>(a.y + q * part +
                                                                    int64_t(max(slot, 0)) * a.H + h));
            if (slot >= 0) {
                s.x = fmaf(w, v.x, s.x);
                s.y = fmaf(w, v.y, s.y);
                s.z = fmaf(w, v.z, s.z);
                s.w = fmaf(w, v.w, s.w);
            }
        }
    }
    *reinterpret_cast<uint2*>(a.out + t * a.H + h) =
        make_uint2(pack_bf16x2_rn(s.x, s.y), pack_bf16x2_rn(s.z, s.w));
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

// Most blocks that the kernels are launched with, whatever the GPU: a bound of
// the items that the down projections are split into.
constexpr int64_t kSpread = 320;

struct Layout { size_t slots, weights, hidden, y, total; };

Layout workspace_layout(int64_t T, int k, int64_t H, int64_t I) {
    const size_t n = size_t(T) * k;
    Layout l;
    l.slots = kWsAlign;
    l.weights = l.slots + align_up((2 + n) * 4, kWsAlign);
    l.hidden = l.weights + align_up(n * 4, kWsAlign);
    l.y = l.hidden + align_up(n * size_t(I) * 4, kWsAlign);
    // not split: n rows of H; split: kSpread items of at most T tokens and kM columns
    l.total = l.y + align_up(max64(int64_t(n) * H, T * kSpread * kM) * 4, kWsAlign);
    return l;
}

moe_status_t layer(LayerArgs a, const void* w_up, const void* w_down, int64_t T, void* workspace,
                   size_t workspace_bytes, cudaStream_t s) {
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
    a.slots = reinterpret_cast<int*>(ws + l.slots);
    a.weights = reinterpret_cast<float*>(ws + l.weights);
    a.hidden = reinterpret_cast<uint16_t*>(ws + l.hidden);
    a.y = reinterpret_cast<float*>(ws + l.y);
    a.spread = int(min64(int64_t(sm_count()) * kBlocksPerSm, kSpread));

    CUtensorMap up_big, up_small, down_big;
    if (!make_map(&up_big, w_up, int64_t(a.E) * 2 * a.I, a.H, kBigBox) ||
        !make_map(&up_small, w_up, int64_t(a.E) * 2 * a.I, a.H, kSmallBox) ||
        !make_map(&down_big, w_down, int64_t(a.E) * a.H, a.I, kBigBox))
        return MOE_ERR_CUDA;
    const bool fp8 = a.x_scales != nullptr;
    const auto up = fp8 ? layer_kernel<true, true> : layer_kernel<true, false>;
    const auto down = layer_kernel<false, true>;
    if (!opt_in_smem((const void*)up, kSmemBytes) || !opt_in_smem((const void*)down, kSmemBytes))
        return MOE_ERR_CUDA;
    // two accumulators of as many columns as a B tile has rows, a power of two
    const auto cols = [&](bool two) { return (T <= 16 ? 32u : T <= 32 ? 64u : 128u) << (two ? 1 : 0); };
    a.tmem_cols = cols(fp8);
    up<<<unsigned(a.spread), kThreads, kSmemBytes, s>>>(up_big, up_small, a);
    if (launch_status() != MOE_OK) return MOE_ERR_CUDA;
    a.tmem_cols = cols(true);
    if (launch_dependent(down, unsigned(a.spread), kThreads, kSmemBytes, s, down_big, down_big,
                         a) != cudaSuccess)
        return MOE_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((a.H + 4 * kSumThreads - 1) / (4 * kSumThreads)), unsigned(T));
    cfg.blockDim = dim3(kSumThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, layer_sum_kernel, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
