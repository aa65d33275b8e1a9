// layer_decode.cu -- moe_layer_decode, moe_layer_decode_indices: a whole MoE
// layer for a few tokens, in one launch.
//
//   out[t] = sum_j p[t,j] * (silu(x_t Wg[e]^T) * (x_t Wu[e]^T)) Wd[e]^T,  e = idx[t,j]
//
// With up to 64 tokens a layer is bound by reading the weights of the experts
// that some token chose, once: 6 H I bytes each.  One block on every SM streams
// them, first the up projections and then the down projections, through the
// tensor cores with the operands swapped: up to 128 weight rows are the A tile
// (M = 128) and a group of up to 64 tokens of one expert the B tile (N), so
// nothing that is read is padding, and the weights go from TMA to shared memory
// to tcgen05.mma without passing a register.
//   warp 0        TMA producer: stages of weight rows x up to 256 of K, in a
//                 ring that fills the SM's shared memory
//   warp 1        one thread issues the MMAs
//   warps 2..10   fill the up phase's B tiles with gathered token rows (asynchronous
//                 copies; e4m3 codes times their scale through registers), one or
//                 several warps a stage, so that the latency of several gathers
//                 overlaps (warp 2 also has the tensor memory)
//   warp 11       waits for the other blocks, and copies hidden rows into the down
//                 phase's B tiles
//   warps 12..15  epilogue: silu(gate) * up, or the down products
// The issuing threads are elected (elect_one): one token, 2 of 64 experts,
// H = 4096, I = 2048: 34.4 us against 39.5 behind a test of the lane.  Where
// memory is the bound throughout it costs 1 to 2% (the last case below).
// What bounds many tokens of an expert (64 tokens, 8 of 8 experts, H = 4096, I = 2048:
// 95 us, weights 60): every tile of weight rows brings its own copy of the unit's
// token rows, half as many bytes again as the weights, or as many in the down phase
// and for e4m3 rows, which come in two parts; and the rows leave the ring 3 or 4 stages.
// Precision: the MMA's operands are bf16, but a hidden value, and an e4m3 code
// times its scale, are not bf16 values.  Both are split into a bf16 value and
// the bf16 value of the rest (16 bits together, off by 2^-17 at most, where the output
// is rounded to 2^-8), which stand side by side as
// columns of one B tile; the epilogue adds the two columns.  An MMA this narrow
// takes as long as the read of its A tile (37 cycles measured, a fifth of the
// time that the tile takes to arrive), so the second part costs next to nothing.
// The blocks meet twice (a cooperative launch, so that all of them are
// resident): before the hidden rows are read, and before the down products of a
// token's choices are added up.  The weights do not depend on the hidden rows,
// so a block's ring fills with down projections while it waits.
// Every block works the routing out for itself (top-k, softmax, each expert's
// tokens) in shared memory: a launch of its own would take longer.
// Measured (one call after another in a CUDA graph, other weights each time; the GPUs
// differ by up to 4%, and calls from Python take 1 to 4% more): one token, 6 of 64
// experts, H = 2048, I = 1408: 32.5-33.0 us, of which 10 + 4 stream the weights; the
// rest is latency (routing 4 us, the two meetings, the last sum).  16 tokens of
// these: 129-131 us, 6.2 TB/s; 64 tokens over 256 experts, H = 7168, I = 2048:
// 2.82-2.88 ms, 6.8 TB/s (a copy on the same GPU: 6.7).  Three launches, with
// the down projections' overlapping the up projections', were as fast for one token
// and slower in between (139 us for the 16 tokens, where one launch had 132): each
// launch worked the routing out anew.  Dot products by warps, without tensor cores: 82 us, 439 us, 12.2 ms.
// Every wait is bounded; one that gives up records MOE_ERR_TIMEOUT in the
// workspace status word.
#include <atomic>

#include "tensor_core.cuh"

namespace moe {
namespace {

constexpr int kMaxTokens = 64;
constexpr int kMaxSize = 1 << 20;         // of H and I
constexpr int kM = 128;                   // rows of an MMA, weight rows of a down tile
constexpr int kRowBox = 8, kRowBigBox = 32;    // hidden rows of one
constexpr int kMaxStages = 16;
constexpr int kLoaders = 9;               // warps that fill B tiles
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kEpilogue = 3 + kLoaders;   // its first warp
static_assert(kEpilogue + 4 == kWarps && kEpilogue % 4 == 0, "warp roles");
constexpr int kFly = 8;                   // chunks that a loader's lane has in flight
constexpr int kExchBytes = 2 * 8 * 64 * 4;    // gate and up values on their way to each other
constexpr int kSmemBytes = 226 * 1024;    // dynamic shared memory of a block, one on an SM
constexpr int kMaxParts = 8;              // parts of a down tile's K
constexpr uint32_t kTmemCols = 256;       // two accumulators of up to 128 columns
// Most blocks of a launch, whatever the GPU.
constexpr int kMaxBlocks = 160;

// What the blocks meet by, at the same place of every workspace.
struct Meeting {
    uint64_t epoch;                       // the token of the last call, if nobody wrote over it
    uint64_t pad[31];
    uint64_t flag[2][kMaxBlocks];         // a block sets its own to the call's token
};

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
    Meeting* meeting;
    uint64_t nonce;             // another one for each call from the host
    uint16_t* hidden;           // [2][T*k, I] bf16: the values, and what they leave
    float* y;                   // [T*k, H], a row for each choice
    float* parts;               // [2 * kMaxBlocks][min(group, T)][kM]: tiles that are cut
    int T, E, k;
    int H, I;
};

// ----------------------------------------------------------------- routing

// What every block knows of the routing, in shared memory.  A slot is a row of
// the workspace: experts in order, an expert's tokens in order.  A unit is a
// group of an expert's tokens that share a B tile.
struct Routing {
    float* w;                   // [T*k]
    uint32_t* mask;             // [E][2] tokens of each expert, a bit each
    int16_t* expert;            // [T*k] expert of a choice, -1 = empty
    uint16_t* first;            // [E] first slot of each expert
    uint16_t* units;            // [E] its first unit
    uint16_t* unit;             // [T*k] expert of each unit
    uint8_t* group;             // [T*k] which group of the expert's tokens it is
    uint8_t* token;             // [T*k] token of each slot
    uint16_t* choice;           // [T*k] t*k + j of each slot
    int* count;                 // [4]: units, bad choices, tokens of a group
    int* sums;                  // [3 * kWarps] a warp's sums over its experts
};

__host__ __device__ inline size_t routing_bytes(int T, int E, int k) {
    const size_t n = size_t(T) * k;
    const size_t b = 16 + 12 * kWarps + size_t(E) * 12 + n * 12;
    return (b + 127) / 128 * 128;
}

__device__ __forceinline__ Routing carve_routing(uint8_t* p, int T, int E, int k) {
    const int n = T * k;
    Routing r;
    r.count = reinterpret_cast<int*>(p);
    r.sums = r.count + 4;
    r.mask = reinterpret_cast<uint32_t*>(r.sums + 3 * kWarps);
    r.w = reinterpret_cast<float*>(r.mask + 2 * E);
    r.expert = reinterpret_cast<int16_t*>(r.w + n);
    r.first = reinterpret_cast<uint16_t*>(r.expert + n);
    r.units = r.first + E;
    r.unit = r.units + E;
    r.choice = r.unit + n;
    r.group = reinterpret_cast<uint8_t*>(r.choice + n);
    r.token = r.group + n;
    return r;
}

// How many tokens expert e has, and how many of them come before token t.
__device__ __forceinline__ int tokens_of(const Routing& r, int e) {
    return __popc(r.mask[2 * e]) + __popc(r.mask[2 * e + 1]);
}
__device__ __forceinline__ int tokens_before(const Routing& r, int e, int t) {
    const uint32_t below = (1u << (t & 31)) - 1u;
    return t < 32 ? __popc(r.mask[2 * e] & below)
                  : __popc(r.mask[2 * e]) + __popc(r.mask[2 * e + 1] & below);
}

// Order-preserving key of a float; -0 is +0, as for a comparison of floats.
__device__ __forceinline__ uint32_t logit_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_logit(uint32_t u) {
    return __uint_as_float(u ^ (uint32_t(int32_t(~u) >> 31) | 0x80000000u));
}

__device__ __forceinline__ void note_choice(const Routing& r, int t, int i, int id, float w) {
    r.expert[i] = int16_t(id);
    r.w[i] = w;
    if (id >= 0) atomicOr(&r.mask[2 * id + (t >> 5)], 1u << (t & 31));
}

// The choices from the logits.  `lanes` lanes a token, 32 / lanes tokens a warp;
// a lane has the keys of NV consecutive experts (E <= lanes * NV, k <= lanes).
template <int NV>
__device__ __forceinline__ void choose(const LayerArgs& a, const Routing& r, int lanes, bool publish) {
    const int lane = int(lane_id()) & (lanes - 1), base = int(lane_id()) & ~(lanes - 1);
    const uint32_t group = lanes == 32 ? 0xFFFFFFFFu : (1u << lanes) - 1u;
    bool clear = false;
    // whole warps go round, with tokens that do not exist among theirs
    for (int t0 = 0; t0 < a.T; t0 += kThreads / lanes) {
        const int t = t0 + threadIdx.x / lanes;
        uint32_t key[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = lane * NV + i;
            key[i] = t < a.T && e < a.E ? logit_key(__ldg(a.logits + int64_t(t) * a.E + e)) : 0u;
        }
        if (!clear) { __syncthreads(); clear = true; }     // the masks are
        if (t0 + int(threadIdx.x & ~31) / lanes >= a.T) continue;
        uint32_t my_key = 0;
        int my_id = -1;
#pragma unroll 1
        for (int j = 0; j < a.k; ++j) {
            // the largest key left; 0: taken, or none
            uint32_t best = key[0];
            int at = 0;
#pragma unroll
            for (int i = 1; i < NV; ++i)
                if (key[i] > best) { best = key[i]; at = i; }
            uint32_t top = best;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const uint32_t v = __shfl_xor_sync(0xFFFFFFFFu, top, o);
                if (o < lanes) top = max(top, v);
            }
            // equal ones: the lowest lane has the lowest id
            const uint32_t have = (__ballot_sync(0xFFFFFFFFu, best == top) >> base) & group;
            const int from = __ffs(int(have)) - 1;
            const int e = __shfl_sync(0xFFFFFFFFu, lane * NV + at, base + from);
            if (lane == from) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (i == at) key[i] = 0u;
            }
            if (lane == j) { my_key = top; my_id = top != 0u ? e : -1; }   // (0: no key is left)
        }
        // lane j has choice j; their softmax
        const float v = key_logit(my_key), v0 = __shfl_sync(0xFFFFFFFFu, v, base);
        const float p = lane < a.k ? expf(v - v0) : 0.0f;
        float sum = p;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float u = __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            if (o < lanes) sum += u;
        }
        const float w = __fdiv_rn(p, sum);
        if (t < a.T && lane < a.k) {
            const int i = t * a.k + lane;
            if (publish) {
                a.topk_idx[i] = my_id;
                a.topk_w[i] = w;
            }
            note_choice(r, t, i, my_id, w);
        }
    }
    __syncthreads();
}

// All threads of the block; the caller ends it with a barrier.  `publish`: writes the choices
// out.
__device__ __forceinline__ void route(const LayerArgs& a, const Routing& r, bool publish) {
    const int lane = int(lane_id()), warp = threadIdx.x >> 5;
    const int T = a.T, E = a.E, k = a.k, n = T * k;
    for (int e = threadIdx.x; e < 2 * E; e += kThreads) r.mask[e] = 0u;
    if (threadIdx.x == 0) r.count[1] = 0;
    if (a.logits) {
        // a warp a token; 8 lanes where there are more tokens than warps and few experts
        if (E <= 256) choose<8>(a, r, T > kWarps && E <= 64 && k <= 8 ? 8 : 32, publish);
        else choose<32>(a, r, 32, publish);
    } else {
        __syncthreads();
        for (int t = warp; t < T; t += kWarps) {
            int id = -1, bad = 0;
            float w = 0.0f;
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
            if (lane < k) note_choice(r, t, t * k + lane, id, w);
        }
        __syncthreads();
    }
    if (n <= 32 && T <= 8) {
        // Few choices: a warp has one in each lane, and the experts in the order of
        // their first choices.  A unit takes all of an expert's tokens.
        if (warp == 0) {
            const int e = lane < n ? r.expert[lane] : -1;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, e < 0 ? -1 - lane : e);
            const unsigned below = (1u << lane) - 1u;
            const bool leads = e >= 0 && !(same & below);
            const int c = leads ? __popc(same) : 0, unit = __popc(__ballot_sync(0xFFFFFFFFu, leads) & below);
            int slot = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, slot, o);
                if (lane >= o) slot += v;
            }
            slot = __shfl_sync(0xFFFFFFFFu, slot - c, __ffs(int(same)) - 1) + __popc(same & below);
            if (leads) {
                r.first[e] = uint16_t(slot);
                r.units[e] = uint16_t(unit);
                r.unit[unit] = uint16_t(e);
                r.group[unit] = 0;
            }
            if (e >= 0) {
                r.token[slot] = uint8_t(lane / k);
                r.choice[slot] = uint16_t(lane);
            }
            const int units = __popc(__ballot_sync(0xFFFFFFFFu, leads));
            if (lane == 0) { r.count[0] = units; r.count[2] = 8; }
        }
        __syncthreads();
        return;
    }
    // Prefix sums over the experts, `mine` of them a thread: tokens, and units of
    // 8, 16, 32 or 64 tokens.  Two sums to a word; each is at most 2048.
    const int mine = (E + kThreads - 1) / kThreads, e0 = min(threadIdx.x * mine, E);
    const int e1 = min(e0 + mine, E);
    int lo = 0, hi = 0, ex = 0;                            // tokens, by 8; by 16, by 32; by 64
#pragma unroll 1
    for (int e = e0; e < e1; ++e) {
        const int c = tokens_of(r, e);
        lo += c << 16 | (c + 7) / 8;
        hi += (c + 15) / 16 << 16 | (c + 31) / 32;
        ex += (c + 63) / 64;
    }
    int ilo = lo, ihi = hi, iex = ex;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, ilo, o), u = __shfl_up_sync(0xFFFFFFFFu, ihi, o);
        const int x = __shfl_up_sync(0xFFFFFFFFu, iex, o);
        if (lane >= o) { ilo += v; ihi += u; iex += x; }
    }
    if (lane == 31) { r.sums[warp] = ilo; r.sums[kWarps + warp] = ihi; r.sums[2 * kWarps + warp] = iex; }
    __syncthreads();
    int all_lo = 0, all_hi = 0, act = 0;
    ilo -= lo;
    ihi -= hi;
    iex -= ex;
#pragma unroll 4
    for (int i = 0; i < kWarps; ++i) {
        if (i == warp) { ilo += all_lo; ihi += all_hi; iex += act; }
        all_lo += r.sums[i];
        all_hi += r.sums[kWarps + i];
        act += r.sums[2 * kWarps + i];
    }
    // Tokens of a group: a large group keeps its rows' place in every stage and
    // leaves less of the ring to weights, a small one reads the weights of an
    // expert with more tokens again, from L2.  8, unless that is a tenth more
    // reads; then 16 and 32, by the same rule; then 64.
    const int by8 = all_lo & 0xFFFF, by16 = all_hi >> 16, by32 = all_hi & 0xFFFF;
    const int g = by8 * 10 <= act * 11 ? 8 : by16 * 10 <= act * 11 ? 16 : by32 * 10 <= act * 11 ? 32 : 64;
    int slot = ilo >> 16;
    int unit = g == 8 ? ilo & 0xFFFF : g == 16 ? ihi >> 16 : g == 32 ? ihi & 0xFFFF : iex;
#pragma unroll 1
    for (int e = e0; e < e1; ++e) {
        const int c = tokens_of(r, e);
        r.first[e] = uint16_t(slot);
        r.units[e] = uint16_t(unit);
        slot += c;
        for (int q = 0; q * g < c; ++q, ++unit) {
            r.unit[unit] = uint16_t(e);
            r.group[unit] = uint8_t(q);
        }
    }
    if (threadIdx.x == kThreads - 1) {
        r.count[0] = g == 8 ? by8 : g == 16 ? by16 : g == 32 ? by32 : act;
        r.count[2] = g;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int e = r.expert[i], t = i / k;
        if (e >= 0) {
            const int slot = r.first[e] + tokens_before(r, e, t);
            r.token[slot] = uint8_t(t);
            r.choice[slot] = uint16_t(i);
        }
    }
}

// ----------------------------------------------------------------- meeting

// The token that the blocks of this call meet by: the epoch word of the workspace
// and the call's own nonce, mixed (the finalizer of Steele, Lea & Flood, "Fast
// splittable pseudorandom number generators", 2014).  Whatever the workspace
// holds, a flag must not equal the token before its block has set it.  Data of
// other calls does so by chance only, with 64 bits.  Flags of an earlier call are
// the danger: a replayed graph repeats its nonce, and where another of its nodes
// writes the epoch word, the token too.  So no call leaves a flag that a later one
// could take:
//   - a block clears its flag of the second meeting before it arrives at the first,
//     and nobody reads those flags before the first meeting is over;
//   - block 0 clears the flags of the first meeting after the second, at which a
//     block arrives only once it has read them for the last time, or without reading
//     them if it has nothing to wait for.
__device__ __forceinline__ uint64_t meeting_token(uint64_t epoch, uint64_t nonce) {
    uint64_t z = epoch + nonce * 0x9E3779B97F4A7C15ull;
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}

// One thread, after everything that the block wrote (and a barrier of it).
__device__ __forceinline__ void arrive(const LayerArgs& a, int which, uint64_t token) {
    asm volatile("fence.acq_rel.gpu;\n st.relaxed.gpu.global.u64 [%0], %1;"
                 :: "l"(&a.meeting->flag[which][blockIdx.x]), "l"(token) : "memory");
}

// One warp: waits until every block has arrived; false after kMeetPolls polls
// (each takes over half a microsecond).
constexpr int kMeetPolls = 1 << 22;

__device__ __forceinline__ bool wait_for_blocks(const LayerArgs& a, int which, uint64_t token) {
    const uint64_t* flag = a.meeting->flag[which] + lane_id();
    bool here = false;
#pragma unroll 1
    for (int i = 0; i < kMeetPolls && !here; ++i) {
        uint64_t v[kMaxBlocks / 32];                       // all on their way at once
#pragma unroll
        for (int b = 0; b < kMaxBlocks / 32; ++b)
            asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v[b]) : "l"(flag + 32 * b) : "memory");
        here = true;
#pragma unroll
        for (int b = 0; b < kMaxBlocks / 32; ++b)
            here &= v[b] == token || int(lane_id()) + 32 * b >= int(gridDim.x);
        here = __all_sync(0xFFFFFFFFu, here);
    }
    asm volatile("fence.acq_rel.gpu;" ::: "memory");
    __syncwarp();                                          // what one lane has seen, all have
    return here;
}

// One copy of the wait's code for all of the roles.
__device__ __noinline__ bool bar_wait(uint32_t bar, uint32_t parity) { return mbar_wait(bar, parity); }

// ------------------------------------------------------------------- tiles

// How the routing is cut into a phase's work items, the same in every block.  A
// tile is 64 gate rows and the matching up rows, or 128 rows of Wd, for one
// unit; the blocks take the items in turn.  The tiles of the last round, which
// would leave most blocks without work, are cut further, into fewer columns or
// into parts of K, so that it is a short one.
struct Work {
    int units, strips;          // tiles: units * strips
    int whole, items;           // tiles that are one item each; items
    int cuts;                   // items of each of the other tiles
    int group;                  // tokens of a B tile
    int subs, shift, ksubs;     // sub-tiles (64 of K) of a stage, its logarithm; of all K
    int stage_bytes, stages;
    int teams, team;            // of loader warps, a stage each; warps of one
    int a_sub, b_sub;           // bytes of a sub-tile
    bool two;                   // the B rows come in two bf16 parts
};

// Rounds that `items` take.
__device__ __forceinline__ int rounds(int items) { return (items + int(gridDim.x) - 1) / int(gridDim.x); }

// (A whole warp.)
__device__ __forceinline__ Work work_of(const LayerArgs& a, const Routing& r, int ring_bytes, bool up) {
    Work w;
    w.units = r.count[0];
    w.group = r.count[2];
    w.two = !up || a.x_scales;
    w.strips = up ? a.I / 64 : a.H / kM;
    const int tiles = w.units * w.strips, rest = tiles % int(gridDim.x);
    w.whole = tiles - rest;
    // An item's own cost is taken as 16 of the 64 columns, and as half a step of
    // 128 of K.  No more than two rounds of parts: that bounds the workspace.  A
    // lane tries each number of cuts.
    const int c = up ? 1 << (lane_id() & 3) : 1 + int(lane_id() & 7), steps = a.I / 128;
    const bool may = up ? c <= 4 : c == 1 || (c <= min(kMaxParts, steps) && c * rest <= 2 * int(gridDim.x));
    const int cost = rounds(rest * c) * (up ? 64 / c + 16 : 2 * ((steps + c - 1) / c) + 1);
    // the cheapest, of equal ones the fewest cuts
    w.cuts = int(__reduce_min_sync(0xFFFFFFFFu, may ? uint32_t(cost) << 4 | uint32_t(c) : 0xFFFFFFFFu) & 15u);
    w.items = w.whole + rest * w.cuts;
    const int rows = up && w.whole == 0 ? kM / w.cuts : kM;    // of the largest item
    // As much of a row in one stage, up to 512 bytes, as leaves three stages: rows
    // are far apart, and memory is slower the shorter the pieces (16 tokens, 64
    // experts, H = 2048: 154 us with 128 bytes, 135 with 256, 132 with 512).
    w.a_sub = rows * 128;
    w.b_sub = w.two ? w.group * 256 : max(w.group, 16) * 128;
    const int sub = w.a_sub + w.b_sub;
    const int left = ring_bytes - (kM - rows) * 128;       // an MMA reads kM rows all the same
    w.shift = 12 * sub <= left ? 2 : 6 * sub <= left ? 1 : 0;
    w.subs = 1 << w.shift;
    w.stage_bytes = w.subs * sub;
    w.stages = min(kMaxStages, left / w.stage_bytes);
    w.teams = min(kLoaders, w.stages);
    w.team = kLoaders / w.teams;
    w.ksubs = (up ? a.H : a.I) / 64;
    return w;
}

// One work item: (part of) a tile over the sub-tiles [k0, k1) of its K.
struct Item {
    int e, first, n;            // expert, the unit's first slot, its tokens
    int strip;
    int cols, col;              // up: hidden columns, the first of them
    int cut;                    // down: which part among all parts, -1: the whole tile
    int k0, k1;
};

// Up: a unit's strips one after the other.  Down: a strip's units.
__device__ __forceinline__ Item item_of(const Work& w, const Routing& r, int i, bool up) {
    Item it;
    int tile = i, cut = 0, cuts = 1;
    it.cut = -1;
    if (i >= w.whole) {
        const int j = i - w.whole;
        cuts = w.cuts;
        tile = j / cuts;
        cut = j - tile * cuts;
        tile += w.whole;
        if (cuts > 1) it.cut = j;
    }
    int unit;
    it.k0 = 0;
    it.k1 = w.ksubs;
    it.cols = 64;
    if (up) {
        unit = tile / w.strips;
        it.strip = tile - unit * w.strips;
        it.cols /= cuts;
        it.col = it.strip * 64 + cut * it.cols;
    } else {
        it.strip = tile / w.units;
        unit = tile - it.strip * w.units;
        it.k0 = cut * w.ksubs / cuts;
        it.k1 = (cut + 1) * w.ksubs / cuts;
        it.col = 0;
    }
    it.e = r.unit[unit];
    const int at = r.group[unit] * w.group;
    it.first = r.first[it.e] + at;
    it.n = min(w.group, tokens_of(r, it.e) - at);
    return it;
}

// B rows of n tokens: each part of two takes a multiple of 8, one alone of 16,
// so that N is a multiple of 16.
__device__ __forceinline__ int b_rows(int n, bool two) { return two ? (n + 7) & ~7 : (n + 15) & ~15; }

// What a float's bf16 value leaves of it (0 for an infinity, so that it stays one).
__device__ __forceinline__ float bf16_rest(float v, float hi) {
    return (__float_as_uint(hi) & 0x7F800000u) == 0x7F800000u ? 0.0f : v - hi;
}

// Chunk c (8 values of K) of a B row in a sub-tile with 128-byte swizzle.
__device__ __forceinline__ void put_chunk(uint8_t* tile, int row, int c, uint4 v) {
    *reinterpret_cast<uint4*>(tile + row * 128 + ((c ^ (row & 7)) << 4)) = v;
}

// 8 e4m3 codes times their scale, as bf16 values and what they leave.
__device__ __forceinline__ void split_codes(uint2 code, float scale, uint4& hi, uint4& lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        e4m3x2_to_f32((i < 2 ? code.x : code.y) >> (16 * (i & 1)), a, b);
        a *= scale;
        b *= scale;
        h[i] = pack_bf16x2_rn(a, b);
        l[i] = pack_bf16x2_rn(bf16_rest(a, bf16lo_to_f32(h[i])), bf16_rest(b, bf16hi_to_f32(h[i])));
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
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

// Threads that share 4 columns of the last sum: 8 while that leaves each at most one such
// share; threads of all shares (a multiple of a warp's).
__device__ __forceinline__ int sum_lanes(const LayerArgs& a) {
    return a.T * (a.H / 4) * 8 <= int(gridDim.x) * kThreads ? 8 : 1;
}
__device__ __forceinline__ int sum_threads(const LayerArgs& a) { return a.T * (a.H / 4) * sum_lanes(a); }

// out[t] = sum over the choices of the weighted down products.  `lanes`
// neighbouring threads have 4 columns of a token, each a share of the choices
// (and of their parts); the order of the sum depends on `lanes` alone.
__device__ __forceinline__ void add_up(const LayerArgs& a, const Routing& r, const Work& w, int lanes,
                                       int i) {
    constexpr int kMany = 4;                               // loads in flight
    const int quad = i / lanes, mine = i & (lanes - 1);
    const int quads = a.H / 4, t = quad / quads, h = (quad - t * quads) * 4;
    const int cuts = w.items > w.whole ? w.cuts : 1, n = a.k * cuts;
    const int tile0 = h / kM * w.units, rows = min(w.group, a.T);
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int m0 = mine; m0 < n; m0 += kMany * lanes) {
        float4 v[kMany];
        float p[kMany];
#pragma unroll
        for (int q = 0; q < kMany; ++q) {
            const int m = m0 + q * lanes, j = m / cuts, cut = m - j * cuts;
            v[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            p[q] = 0.0f;
            const int e = m < n ? r.expert[t * a.k + j] : -1;
            if (e < 0) continue;
            const int at = tokens_before(r, e, t);         // the token's place in the expert
            const int tile = tile0 + r.units[e] + at / w.group;
            const float* y = a.y + int64_t(t * a.k + j) * a.H + h;
            if (cuts > 1 && tile >= w.whole)
                y = a.parts + (int64_t((tile - w.whole) * cuts + cut) * rows + at % w.group) * kM + h % kM;
            else if (cut > 0)
                continue;
            v[q] = __ldcg(reinterpret_cast<const float4*>(y));
            p[q] = r.w[t * a.k + j];
        }
#pragma unroll
        for (int q = 0; q < kMany; ++q) {
            s.x = fmaf(p[q], v[q].x, s.x);
            s.y = fmaf(p[q], v[q].y, s.y);
            s.z = fmaf(p[q], v[q].z, s.z);
            s.w = fmaf(p[q], v[q].w, s.w);
        }
    }
#pragma unroll 1
    for (int o = 1; o < lanes; o <<= 1) {
        s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, o);
        s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, o);
        s.z += __shfl_xor_sync(0xFFFFFFFFu, s.z, o);
        s.w += __shfl_xor_sync(0xFFFFFFFFu, s.w, o);
    }
    if (mine == 0)
        *reinterpret_cast<uint2*>(a.out + int64_t(t) * a.H + h) =
            make_uint2(pack_bf16x2_rn(s.x, s.y), pack_bf16x2_rn(s.z, s.w));
}

// Starts the copy of chunk c of a row of a B tile.
__device__ __forceinline__ void copy_chunk(uint8_t* tile, int row, int c, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 :: "r"(smem_addr(tile + row * 128 + ((c ^ (row & 7)) << 4))), "l"(from) : "memory");
}

// A stage's B tiles from rows of bf16, chunks of 16 bytes: asynchronous copies, all of
// them in flight at once (through registers, 8 at a time: 64 tokens of 8 experts of 4096
// by 2048, 108 us against 97).  Wants 16 bytes of alignment, which x has.
__device__ __forceinline__ void load_stage(const LayerArgs& a, const Routing& r, const Work& w,
                                           const Item& m, int k, int cols, int member, uint8_t* tile) {
    const int row_chunks = 8 * w.subs, row_shift = 3 + w.shift, chunks = m.n * row_chunks;
#pragma unroll 4
    for (int c = member * 32 + int(lane_id()); c < chunks; c += w.team * 32) {
        const int row = c >> row_shift, j = c & (row_chunks - 1);
        if (j >= cols) continue;
        const int64_t at = int64_t(r.token[m.first + row]) * a.H + k * 64 + j * 8;
        copy_chunk(tile + (j >> 3) * w.b_sub, row, j & 7, static_cast<const uint16_t*>(a.x) + at);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// The same from e4m3 codes and their scales, chunks of 8 codes, as values in two parts.
// Loads what comes first before it waits for the stage; false: the wait ran out.
__device__ __forceinline__ bool load_codes(const LayerArgs& a, const Routing& r, const Work& w,
                                           const Item& m, int k, int cols, int member, uint8_t* tile,
                                           uint32_t empty, uint32_t parity) {
    const int row_chunks = 8 * w.subs, row_shift = 3 + w.shift, chunks = m.n * row_chunks;
    const int part2 = b_rows(m.n, true) * 128;
    bool ready = false;
#pragma unroll 1
    for (int c0 = member * 32 * kFly; c0 < chunks || !ready; c0 += w.team * 32 * kFly) {
        // (a warp may have no chunk) no branch around a load, so that all of them are in
        // flight
        uint2 code[kFly];
        float scale[kFly];
#pragma unroll
        for (int q = 0; q < kFly; ++q) {
            const int c = min(c0 + q * 32 + int(lane_id()), chunks - 1);
            const int j = min(c & (row_chunks - 1), cols - 1);
            const int t = r.token[m.first + (c >> row_shift)], col = k * 64 + j * 8;
            code[q] = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.x) +
                                                           int64_t(t) * a.H + col));
            scale[q] = __ldg(a.x_scales + int64_t(t) * (a.H / 128) + col / 128);
        }
        if (!ready) ready = bar_wait(empty, parity);
        if (!ready) return false;
#pragma unroll
        for (int q = 0; q < kFly; ++q) {
            const int c = c0 + q * 32 + int(lane_id()), row = c >> row_shift, j = c & (row_chunks - 1);
            if (c >= chunks || j >= cols) continue;
            uint8_t* sub = tile + (j >> 3) * w.b_sub;
            uint4 hi, lo;
            split_codes(code[q], scale[q], hi, lo);
            put_chunk(sub, row, j & 7, hi);
            put_chunk(sub + part2, row, j & 7, lo);
        }
    }
    return true;
}

// The up phase's B tiles: the tokens' rows.  Loader warps, teams of w.team of them;
// a team fills a stage.  kTwo: x is e4m3 codes.
template <bool kTwo>
__device__ __forceinline__ void load_tokens(const LayerArgs& a, const Routing& r, const Work& work,
                                            uint8_t* ring, uint64_t* empty, uint64_t* full,
                                            volatile int* failed) {
    const Work w = work;
    const int lane = int(lane_id()), warp = int(threadIdx.x >> 5) - 2;
    // No more teams than stages: a warp that waits for a stage has seen the use
    // before its own last one end, so the stage's barrier can be at most one phase
    // behind and the parity is not mistaken for an older one.
    const int mine = warp / w.team, member = warp - mine * w.team;
    if (mine >= w.teams) return;
    uint32_t it = 0;
#pragma unroll 1
    for (int i = blockIdx.x; i < w.items; i += gridDim.x) {
        const Item m = item_of(w, r, i, true);
#pragma unroll 1
        for (int k = m.k0; k < m.k1; k += w.subs, ++it) {
            if (int(it % w.teams) != mine) continue;
            const int s = it % w.stages, cols = min(w.subs, m.k1 - k) * 8;
            const uint32_t bar = smem_addr(&empty[s]), parity = ((it / w.stages) & 1u) ^ 1u;
            uint8_t* tile = ring + s * w.stage_bytes + w.subs * w.a_sub;
            if constexpr (kTwo) {
                if (!load_codes(a, r, w, m, k, cols, member, tile, bar, parity)) *failed = 1;
            } else {
                if (bar_wait(bar, parity)) load_stage(a, r, w, m, k, cols, member, tile);
                else *failed = 1;
            }
            // each thread orders its writes before the tensor core's reads, and the warp
            // its threads' before the one arrival
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (__any_sync(0xFFFFFFFFu, *failed != 0)) return;
            if (lane == 0) mbar_arrive(smem_addr(&full[s]));
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1)
layer_kernel(const __grid_constant__ CUtensorMap map_up, const __grid_constant__ CUtensorMap map_up32,
             const __grid_constant__ CUtensorMap map_up16,
             const __grid_constant__ CUtensorMap map_down, const __grid_constant__ CUtensorMap map_hidden,
             const __grid_constant__ CUtensorMap map_hidden_big, const LayerArgs a) {
    extern __shared__ uint8_t smem_raw[];
    // a phase has its own barriers of the ring, and a ring of its own shape
    __shared__ __align__(8) uint64_t full_a[2][kMaxStages], full_b[2][kMaxStages], empty[2][kMaxStages];
    __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2];
    __shared__ __align__(8) uint64_t up_done, met;         // once each
    __shared__ uint32_t s_tmem;
    __shared__ uint64_t s_token;
    __shared__ volatile int s_failed;
    __shared__ int s_late;
    __shared__ Work s_work[2];

    const int warp = threadIdx.x >> 5, lane = int(lane_id());
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    const int ring_bytes = kSmemBytes - 1024 - kExchBytes - int(routing_bytes(a.T, a.E, a.k));
    float* exch = reinterpret_cast<float*>(ring + ring_bytes);                 // [2][8][64]
    const Routing r = carve_routing(ring + ring_bytes + kExchBytes, a.T, a.E, a.k);

    // the tokens' rows, on their way to L2 while the routing is worked out
    if (blockIdx.x * kThreads + threadIdx.x < a.T * (a.H / 128) * (a.x_scales ? 1 : 2))
        asm volatile("prefetch.global.L2 [%0];" :: "l"(static_cast<const uint8_t*>(a.x) +
            int64_t(blockIdx.x * kThreads + threadIdx.x) * 128) : "memory");
    if (threadIdx.x < 2 * kMaxStages) {
        const int p = threadIdx.x / kMaxStages, s = threadIdx.x % kMaxStages;
        mbar_init(smem_addr(&full_a[p][s]), 1);
        mbar_init(smem_addr(&empty[p][s]), 1);
        if (s < 2) {
            mbar_init(smem_addr(p ? &acc_full[s] : &acc_empty[s]), p ? 1 : 128);
        } else if (threadIdx.x == 2) {
            mbar_init(smem_addr(&up_done), 1);
            mbar_init(smem_addr(&met), 1);
            s_failed = 0;
        }
        mbar_fence_init();
    } else if (warp == 1) {
        if (lane == 0) {
            prefetch_map(&map_up);
            prefetch_map(&map_up32);
            prefetch_map(&map_up16);
            prefetch_map(&map_down);
            prefetch_map(&map_hidden);
            prefetch_map(&map_hidden_big);
        }
    } else if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_addr(&s_tmem)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else if (threadIdx.x == 3 * 32) {
        uint64_t epoch;
        asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(epoch) : "l"(&a.meeting->epoch) : "memory");
        s_token = meeting_token(epoch, a.nonce);
        asm volatile("st.relaxed.gpu.global.u64 [%0], %1;"
                     :: "l"(&a.meeting->flag[1][blockIdx.x]), "l"(uint64_t(0)) : "memory");
    }
    tc_fence_before();
    route(a, r, a.logits && blockIdx.x == 0);
    if (warp >= kWarps - 2) {                              // two warps that may have no choices
        const Work w = work_of(a, r, ring_bytes, (warp & 1) == 0);
        if (lane == 0) s_work[warp & 1] = w;
        if (lane < kMaxStages) mbar_init(smem_addr(&full_b[warp & 1][lane]), (warp & 1) ? 1 : w.team);
        mbar_fence_init();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    if (blockIdx.x == 0 && threadIdx.x == kThreads - 1) {
        a.header->status = r.count[1] ? MOE_ERR_DEVICE_CHECK : MOE_OK;
        a.header->detail = 0;
    }

    // Every role: the up phase, then the down phase.  Items of a phase go to the
    // blocks in turn.
    if (warp == 0) {
        if (elect_one()) {
            // ---------------------------------------------------- TMA producer
            // weights leave L2 before what every call needs again
            const uint64_t once = policy_evict_first();
#pragma unroll 1
            for (int phase = 0; phase < 2; ++phase) {
                const bool up = phase == 0;
                const Work w = s_work[phase];
                // A stage's weights, from sub-tile k on: gate rows and the matching up rows
                // (blocks of 128 each), or rows of Wd.
                auto copy = [&](const Work& w, const Item& m, int k, uint32_t dst, uint32_t bar) {
                    const int row = up ? m.e * 2 * a.I + m.col / 128 * 256 + m.col % 128
                                       : m.e * a.H + m.strip * kM;
                    const int row2 = row + (up ? 128 : kM / 2), half = m.cols;
                    const CUtensorMap* map = !up ? &map_down : half == 64 ? &map_up
                                             : half == 32 ? &map_up32 : &map_up16;
#pragma unroll 1
                    for (int u = 0; u < min(w.subs, m.k1 - k); ++u) {
                        const int c = (k + u) * 64;
                        const uint32_t to = dst + u * w.a_sub;
                        tma_load_2d_hint(to, map, c, row, bar, once);
                        tma_load_2d_hint(to + half * 128, map, c, row2, bar, once);
                    }
                };
                uint32_t it = 0;
#pragma unroll 1
                for (int i = blockIdx.x; i < w.items && !s_failed; i += gridDim.x) {
                    const Item m = item_of(w, r, i, up);
#pragma unroll 1
                    for (int k = m.k0; k < m.k1; k += w.subs, ++it) {
                        const int s = it % w.stages;
                        if (!bar_wait(smem_addr(&empty[phase][s]), ((it / w.stages) & 1u) ^ 1u)) {
                            s_failed = 1;
                            break;
                        }
                        const uint32_t bar = smem_addr(&full_a[phase][s]);
                        mbar_expect_tx(bar, min(w.subs, m.k1 - k) * m.cols * 256);
                        copy(w, m, k, smem_addr(ring + s * w.stage_bytes), bar);
                    }
                }
                // The ring takes another shape once its MMAs have read it.  A block
                // that gave up leaves no copy of its own in flight.
#pragma unroll 1
                for (uint32_t b = it > uint32_t(w.stages) ? it - w.stages : 0; b < it; ++b) {
                    const int s = b % w.stages;
                    const uint32_t ph = (b / w.stages) & 1u;
                    if (!s_failed && !bar_wait(smem_addr(&empty[phase][s]), ph)) s_failed = 1;
                    if (s_failed) bar_wait(smem_addr(&full_a[phase][s]), ph);
                }
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            // ------------------------------------------------------ MMA issuer
            uint32_t tile = 0;
#pragma unroll 1
            for (int phase = 0; phase < 2; ++phase) {
                const bool up = phase == 0;
                const Work w = s_work[phase];
                uint32_t it = 0;
#pragma unroll 1
                for (int i = blockIdx.x; i < w.items && !s_failed; i += gridDim.x, ++tile) {
                    const Item m = item_of(w, r, i, up);
                    const uint32_t idesc = idesc_bf16(kM, b_rows(m.n, w.two) * (w.two ? 2 : 1));
                    const uint32_t buf = tile & 1u, acc = tmem + buf * (kTmemCols / 2);
                    if (!bar_wait(smem_addr(&acc_empty[buf]), ((tile >> 1) & 1u) ^ 1u)) {
                        s_failed = 1;
                        break;
                    }
                    tc_fence_after();
#pragma unroll 1
                    for (int k = m.k0; k < m.k1; k += w.subs, ++it) {
                        const int s = it % w.stages;
                        const uint32_t ph = (it / w.stages) & 1u;
                        if (!bar_wait(smem_addr(&full_b[phase][s]), ph) ||
                            !bar_wait(smem_addr(&full_a[phase][s]), ph)) {
                            s_failed = 1;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t wa = smem_addr(ring + s * w.stage_bytes);
#pragma unroll 1
                        for (int u = 0; u < min(w.subs, m.k1 - k); ++u) {
                            // along K inside the swizzled row: 16 values, 32 bytes, 2 in the
                            // descriptor's address
                            const uint64_t ad = smem_desc_k128(wa + u * w.a_sub);
                            const uint64_t bd = smem_desc_k128(wa + w.subs * w.a_sub + u * w.b_sub);
                            mma_bf16(acc, ad, bd, idesc, k != m.k0 || u);
#pragma unroll
                            for (int kk = 1; kk < 4; ++kk)
                                mma_bf16(acc, ad + 2 * kk, bd + 2 * kk, idesc, 1);
                        }
                        mma_commit(smem_addr(&empty[phase][s]));
                    }
                    if (s_failed) break;
                    mma_commit(smem_addr(&acc_full[buf]));
                }
            }
        }
    } else if (warp == kEpilogue - 1) {
        // ------------------------------ waits for the other blocks; B tiles, down phase
        // (and for its own block's MMAs, which have to have read the ring that the copies go to)
        // A block with neither down products nor a share of the last sum waits for nobody.
        if (int(blockIdx.x) < s_work[1].items || int(blockIdx.x) * kThreads < sum_threads(a)) {
            if (!wait_for_blocks(a, 0, s_token)) s_failed = 1;
            if (!bar_wait(smem_addr(&up_done), 0)) s_failed = 1;
            __syncwarp();
        }
        if (elect_one()) {
            mbar_arrive(smem_addr(&met));
            // the hidden rows, which other blocks' threads wrote and copies now read
            asm volatile("fence.proxy.async;" ::: "memory");
            const Work w = s_work[1];
            uint32_t it = 0;
#pragma unroll 1
            for (int i = blockIdx.x; i < w.items && !s_failed; i += gridDim.x) {
                const Item m = item_of(w, r, i, false);
                const int rows = b_rows(m.n, true);        // (a row more than n is another unit's)
#pragma unroll 1
                for (int k = m.k0; k < m.k1; k += w.subs, ++it) {
                    const int s = it % w.stages, subs = min(w.subs, m.k1 - k);
                    if (!bar_wait(smem_addr(&empty[1][s]), ((it / w.stages) & 1u) ^ 1u)) {
                        s_failed = 1;
                        break;
                    }
                    const uint32_t bar = smem_addr(&full_b[1][s]);
                    mbar_expect_tx(bar, subs * rows * 256);
#pragma unroll 1
                    for (int u = 0; u < subs; ++u) {
                        const uint32_t dst = smem_addr(ring + s * w.stage_bytes + w.subs * w.a_sub + u * w.b_sub);
#pragma unroll 1
                        for (int b = 0; b < rows;) {
                            const bool big = rows - b >= kRowBigBox;
                            const CUtensorMap* map = big ? &map_hidden_big : &map_hidden;
                            tma_load_2d(dst + b * 128, map, (k + u) * 64, m.first + b, bar);
                            tma_load_2d(dst + (rows + b) * 128, map, (k + u) * 64,
                                        a.T * a.k + m.first + b, bar);
                            b += big ? kRowBigBox : kRowBox;
                        }
                    }
                }
            }
            if (s_failed)                                  // none of its copies stays in flight
                for (uint32_t b = it > uint32_t(w.stages) ? it - w.stages : 0; b < it; ++b)
                    bar_wait(smem_addr(&full_b[1][b % w.stages]), (b / w.stages) & 1u);
        }
    } else if (warp < 2 + kLoaders) {
        // -------------------------------------------------- B loaders, up phase
        if (s_work[0].two)
            load_tokens<true>(a, r, s_work[0], ring, empty[0], full_b[0], &s_failed);
        else
            load_tokens<false>(a, r, s_work[0], ring, empty[0], full_b[0], &s_failed);
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3, row = q * 32 + lane;       // TMEM lane quadrant, tile row
        uint32_t tile = 0;
#pragma unroll 1
        for (int phase = 0; phase < 2; ++phase) {
            const bool up = phase == 0;
            const Work w = s_work[phase];
#pragma unroll 1
            for (int i = blockIdx.x; i < w.items; i += gridDim.x, ++tile) {
                const Item m = item_of(w, r, i, up);
                const uint32_t buf = tile & 1u;
                const uint32_t acc = tmem + buf * (kTmemCols / 2) + (uint32_t(q * 32) << 16);
                const bool ok = !s_failed && bar_wait(smem_addr(&acc_full[buf]), (tile >> 1) & 1u);
                // all 128 threads go on, or none
                if (any_epilogue(!ok)) { s_failed = 1; break; }
                tc_fence_after();
#pragma unroll 1
                for (int c0 = 0; c0 < m.n; c0 += 8) {
                    float v[8];
                    tmem_ld8(acc + c0, v);
                    if (w.two) {
                        float lo[8];
                        tmem_ld8(acc + b_rows(m.n, true) + c0, lo);
                        // (an infinite weight times a part that is 0, or of the other sign, would
                        // make NaN of the infinity that the first part has)
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            if (fabsf(v[c]) <= 0x1.fffffep+127f) v[c] += lo[c];
                    }
                    if (up) {
                        // The tile's first rows hold the gate, the next ones the up values.  A
                        // gate's thread works on the first 4 tokens, an up value's on the others;
                        // the threads of every other 8 tokens have the same half of `exch`.
                        const bool gate = row < m.cols;
                        const int col = gate ? row : row - m.cols, c1 = gate ? 0 : 4;
                        float* ex = exch + (c0 & 8) * 64 + col;
                        if (col < m.cols) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) ex[(4 - c1 + c) * 64] = gate ? v[4 + c] : v[c];
                        }
                        bar_epilogue();
                        if (col < m.cols) {
                            uint16_t* hp = a.hidden + int64_t(m.first + c0 + c1) * a.I + m.col + col;
                            float h[4];
                            // silu by the fast exponential and quotient, as in the grouped
                            // layer: off by some 2^-22 and |g| 2^-24, below the 2^-17 that the
                            // row is kept to
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const float other = ex[(c1 + c) * 64], g = gate ? v[c] : other;
                                h[c] = __fdividef(g, 1.0f + __expf(-g)) * (gate ? other : v[4 + c]);
                            }
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                if (c0 + c1 + c >= m.n) continue;
                                const uint16_t hi = f32_to_bf16_rn(h[c]);
                                hp[int64_t(c) * a.I] = hi;
                                hp[(int64_t(a.T) * a.k + c) * a.I] =
                                    f32_to_bf16_rn(bf16_rest(h[c], bf16_to_f32(hi)));
                            }
                        }
                    } else {
                        float* yp = a.y + m.strip * kM + row;
                        float* pp = a.parts + (int64_t(m.cut) * min(w.group, a.T) + c0) * kM + row;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            if (c0 + c >= m.n) break;
                            if (m.cut >= 0) pp[c * kM] = v[c];
                            else yp[int64_t(r.choice[m.first + c0 + c]) * a.H] = v[c];
                        }
                    }
                }
                tc_fence_before();
                mbar_arrive(smem_addr(&acc_empty[buf]));
            }
            // (also where this block gave up: the others go on, and end)
            bar_epilogue();
            if (row == 0) {
                if (up) mbar_arrive(smem_addr(&up_done));
                else if (!bar_wait(smem_addr(&met), 0)) s_failed = 1;
                arrive(a, phase, s_token);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                     :: "r"(tmem), "r"(kTmemCols) : "memory");
    // the sum over a token's choices, of every block's products
    const int lanes = sum_lanes(a);
    if (int(blockIdx.x) * kThreads < sum_threads(a)) {
        if (warp == 0) {
            const bool there = wait_for_blocks(a, 1, s_token);
            if (lane == 0) s_late = !there;
        }
        __syncthreads();
        if (s_late) s_failed = 1;
        // block 0 (which has a share of the sum, whatever the shape): nobody reads this
        // call's epoch or the first meeting's flags any more
        if (blockIdx.x == 0) {
            if (threadIdx.x < kMaxBlocks) a.meeting->flag[0][threadIdx.x] = 0;
            if (threadIdx.x == kMaxBlocks) a.meeting->epoch = s_token;
        }
        const Work w = s_work[1];
#pragma unroll 1
        for (int i = blockIdx.x * kThreads + threadIdx.x; i < sum_threads(a); i += gridDim.x * kThreads)
            add_up(a, r, w, lanes, i);
    }
    if (threadIdx.x == 0 && s_failed) {
        a.header->status = MOE_ERR_TIMEOUT;
        a.header->detail = blockIdx.x;
    }
}

// -------------------------------------------------------------------- host

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

moe_status_t check_layer(int64_t T, int E, int k, int64_t H, int64_t I) {
    if (T < 0 || E < 1 || k < 1 || H < 1 || I < 1) return MOE_ERR_INVALID_ARG;
    if (T > kMaxTokens || E > kMaxExperts || k > kMaxTopK || k > E || H % 256 != 0 || I % 128 != 0)
        return MOE_ERR_UNSUPPORTED;
    if (H > kMaxSize || I > kMaxSize) return MOE_ERR_UNSUPPORTED;    // (int arithmetic below)
    if (int64_t(E) * 2 * I >= (int64_t(1) << 31) || int64_t(E) * H >= (int64_t(1) << 31))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

struct Layout { size_t meeting, hidden, y, parts, total; };

Layout workspace_layout(int64_t T, int k, int64_t H, int64_t I) {
    const size_t n = size_t(T) * k;
    Layout l;
    l.meeting = kWsAlign;
    l.hidden = l.meeting + align_up(sizeof(Meeting), kWsAlign);
    l.y = l.hidden + align_up(n * size_t(I) * 4, kWsAlign);
    l.parts = l.y + align_up(n * size_t(H) * 4, kWsAlign);
    l.total = l.parts + align_up(size_t(2 * kMaxBlocks) * T * kM * 4, kWsAlign);
    return l;
}

moe_status_t layer(LayerArgs a, const void* w_up, const void* w_down, int64_t T, int64_t H,
                   int64_t I, void* workspace, size_t workspace_bytes, cudaStream_t s) {
    const moe_status_t st = check_layer(T, a.E, a.k, H, I);
    if (st != MOE_OK) return st;
    const Layout l = workspace_layout(T, a.k, H, I);
    const bool choices = a.logits ? a.topk_idx && a.topk_w : a.given_idx && a.given_w;
    if (T > 0 && (!a.x || !choices || !w_up || !w_down || !a.out || a.out == a.x))
        return MOE_ERR_INVALID_ARG;
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
    a.H = int(H);
    a.I = int(I);
    a.meeting = reinterpret_cast<Meeting*>(ws + l.meeting);
    a.hidden = reinterpret_cast<uint16_t*>(ws + l.hidden);
    a.y = reinterpret_cast<float*>(ws + l.y);
    a.parts = reinterpret_cast<float*>(ws + l.parts);
    static std::atomic<uint64_t> calls{0};
    a.nonce = calls.fetch_add(1, std::memory_order_relaxed) + 1;

    // boxes of half a tile's rows
    CUtensorMap up, up32, up16, down, hidden, hidden_big;
    if (!make_map(&up, w_up, a.E * 2 * I, H, 64) || !make_map(&up32, w_up, a.E * 2 * I, H, 32) ||
        !make_map(&up16, w_up, a.E * 2 * I, H, 16) || !make_map(&down, w_down, a.E * H, I, kM / 2) ||
        !make_map(&hidden, a.hidden, 2 * T * a.k, I, kRowBox) ||
        !make_map(&hidden_big, a.hidden, 2 * T * a.k, I, kRowBigBox) ||
        !opt_in_smem((const void*)layer_kernel, kSmemBytes))
        return MOE_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(min64(sm_count(), kMaxBlocks)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, layer_kernel, up, up32, up16, down, hidden, hidden_big, a) != cudaSuccess) {
        cudaGetLastError();                                // not the next call's
        return MOE_ERR_CUDA;
    }
    return MOE_OK;
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
    return layer(a, w_up_packed, w_down_packed, T, H, I, workspace, workspace_bytes,
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
    return layer(a, w_up_packed, w_down_packed, T, H, I, workspace, workspace_bytes,
                 static_cast<cudaStream_t>(stream));
}
