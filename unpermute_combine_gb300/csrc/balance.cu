// balance.cu -- moe_balance_loss and moe_balance_loss_backward.
//
// The loss that keeps a router's load even ("从零理解 MoE 算子" §3 and §18 describe
// the router and what an uneven load costs), per sequence s of n tokens, with p the
// softmax of the logits over all experts, or their sigmoids divided by the sum:
//   loss = coef / S * sum_s sum_e f[s,e] P[s,e],  f = counts E / (k n), P = mean of p
// and the router's z loss, z_coef * mean(logsumexp(logits)^2).
//
// Forward: blocks of a fixed chunk of tokens (the chunks' number does not depend on
// the GPU) read the logits once; a row is a few lanes' of a warp, and its p are added
// to sums in registers.  What a block has of one sequence is a piece, with number
// chunk + sequence: along the tokens each new piece raises one of the two, so that no
// two pieces share a number and none has to be looked up.  A second kernel adds the
// pieces of each sequence; the block that ends last adds the sequences.  Sums have a
// fixed order throughout, and counts are whole numbers, so that the same inputs give
// the same bits.
//
// Backward, with a = coef E / (S k n^2) counts, the gradient of p summed over a row:
//   grad = p (a - sum_j a_j p_j) [(1 - sigmoid)] + z_coef 2 / tokens lse softmax
// a is taken less its mean, (counts E - sum counts), which is exact in whole numbers
// and leaves the difference as it is: p sums to 1.  In a balanced layer the a of all
// experts are nearly equal, and the difference of the plain a and their mean would
// lose most of its digits.
#include <type_traits>

#include "common.cuh"
#include "pipeline.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMostChunks = 608;       // of tokens, in the forward pass
constexpr int kLeastChunk = 32;         // tokens

struct Sequences {
    const int32_t* offsets;             // [S+1], or NULL: one sequence of all tokens
    int S;
    int64_t T;

    __device__ int64_t at(int s) const {          // clamped into [0, T]
        if (!offsets) return s == 0 ? 0 : T;
        return min64(max64(int64_t(__ldg(offsets + s)), 0), T);
    }
    // The last sequence that begins at or before token t (0 if none does).
    __device__ int find(int64_t t) const {
        int lo = 0, hi = S - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (at(mid) <= t) lo = mid; else hi = mid - 1;
        }
        return lo;
    }
    __device__ bool bad(int s) const {
        if (!offsets) return false;
        const int a = __ldg(offsets + s), b = __ldg(offsets + s + 1);
        return a < 0 || b < a || b > T;
    }
};

// A row's values over the G lanes of a group, V a lane (a multiple of 4), four of them side
// by side (VEC) or each G from the next.
template <int G, int V, bool VEC>
struct Row {
    float2 v[V / 2];

    static __device__ int expert(int i, int lane) {
        return VEC ? i / 4 * (G * 4) + lane * 4 + i % 4 : i * G + lane;
    }
    __device__ float& at(int i) { return i % 2 ? v[i / 2].y : v[i / 2].x; }

    __device__ void load(const float* row, int E, int lane, float none) {
        if (VEC) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const int e = expert(i, lane);
                const float4 q = e < E ? *reinterpret_cast<const float4*>(row + e)
                                       : make_float4(none, none, none, none);
                v[i / 2] = make_float2(q.x, q.y), v[i / 2 + 1] = make_float2(q.z, q.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = expert(i, lane);
                at(i) = e < E ? row[e] : none;
            }
        }
    }
    __device__ void store(float* row, int E, int lane) {
        if (VEC) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const int e = expert(i, lane);
                if (e < E)
                    *reinterpret_cast<float4*>(row + e) =
                        make_float4(v[i / 2].x, v[i / 2].y, v[i / 2 + 1].x, v[i / 2 + 1].y);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = expert(i, lane);
                if (e < E) row[e] = at(i);
            }
        }
    }
    __device__ float sum() const {
        float2 s = v[0];
#pragma unroll
        for (int i = 1; i < V / 2; ++i) s = add2(s, v[i]);
        return s.x + s.y;
    }
    __device__ float max() const {
        float m = fmaxf(v[0].x, v[0].y);
#pragma unroll
        for (int i = 1; i < V / 2; ++i) m = fmaxf(m, fmaxf(v[i].x, v[i].y));
        return m;
    }
};

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// 2^x and 1/x by one operation of the special function unit, results below 2^-126 as 0 (off
// by about 2^-22 relative; exp(x) = 2^(x log2 e) by 2^-23 |x| more): the functions for all
// floats take two to four instructions more, of some ten an element.
constexpr float kLog2E = 1.4426950408889634f;

__device__ __forceinline__ float exp2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_ftz(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Sums of exp(x) within these bounds: no x is past 63, none that counts is lost, and the
// row needs no shift by its largest.
constexpr float kLeastSum = 0x1p-60f, kMostSum = 0x1p90f;

// Scores of a row of logits x: the softmax is u * inv; with the sigmoid the scores are
// sig * part, keep is one less the sigmoid.
template <int G, int V, bool VEC>
struct Scores {
    Row<G, V, VEC> u, sig, keep;
    float inv, part, lse;
};

// Nearly every row is one exponential u = exp(x) an element and, with the sigmoid, one
// reciprocal r = 1 / (1 + u): the sigmoid u r, one less it r.  Instructions bound the
// kernels, not memory, unless they are few: rows of 32 lanes with a shift by the largest,
// three functions and single floats took 204 for 8 elements of a lane (45 us for 131072 x
// 256, whose logits take 20 us to read).
// Other rows are shifted by their largest m.  If that is far below 0 the sigmoids are their
// exponentials to float32's last bit, and their shares the softmax; if far above, they are
// taken one by one.  A row of nothing but -inf has scores of 0 and an lse of 0.
template <int G, int V, bool VEC, bool SIGMOID>
__device__ __forceinline__ Scores<G, V, VEC> row_scores(const Row<G, V, VEC>& row) {
    Scores<G, V, VEC> s;
    Row<G, V, VEC> x = row;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const float2 t = mul2(x.v[i], both(kLog2E));
        s.u.v[i] = make_float2(exp2_ftz(t.x), exp2_ftz(t.y));
    }
    float sum = group_sum<G>(s.u.sum());
    const bool odd = !(sum >= kLeastSum && sum <= kMostSum);
    bool none = false;
    float shift = 0.0f;
    if (SIGMOID) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 t = add2(s.u.v[i], both(1.0f));
            s.keep.v[i] = make_float2(rcp_ftz(t.x), rcp_ftz(t.y));
            s.sig.v[i] = mul2(s.u.v[i], s.keep.v[i]);
        }
    }
    if (__any_sync(0xFFFFFFFFu, odd)) {
        const float m = group_max<G>(x.max());
        none = odd && sum == 0.0f && m == -INFINITY;         // (a NaN's sum is NaN)
        shift = odd && !none ? m : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (odd) s.u.at(i) = exp2_ftz((x.at(i) - shift) * kLog2E);
            if (SIGMOID && odd) {
                const bool off = m < 0.0f;
                s.keep.at(i) = off ? 1.0f : rcp_ftz(1.0f + exp2_ftz(x.at(i) * kLog2E));
                s.sig.at(i) = off ? s.u.at(i) : rcp_ftz(1.0f + exp2_ftz(-x.at(i) * kLog2E));
            }
        }
        const float again = group_sum<G>(s.u.sum());
        if (odd) sum = again;
    }
    // (__logf is off by 2^-21.4 near 1, about as far as the sum is: 2^-22 and its additions)
    s.lse = none ? 0.0f : shift + __logf(sum);
    s.inv = none ? 0.0f : rcp_ftz(sum);
    if (SIGMOID) {
        const float total = group_sum<G>(s.sig.sum());
        s.part = none ? 0.0f : rcp_ftz(total);
    }
    return s;
}

// ---------------------------------------------------------------- forward

struct Pieces {                         // the workspace behind its header
    uint32_t* ticket;
    uint32_t* bad;                      // [chunks] a choice out of range
    float* z;                           // [pieces]
    float* seq_loss;                    // [S * slices]
    float* seq_z;                       // [S]
    float* sums;                        // [pieces][E]
    int32_t* counts;                    // [pieces][E]
};

// 131072 x 256: 27 us with the sigmoid and 26 with the softmax where nothing else is in L2 (5.1
// TB/s of logits and choices), 33 for both behind a gradient whose stores leave L2 meanwhile.
// With the sigmoid 143 instructions of a warp a row; the softmax's are fewer and take as long:
// neither the issue slots (62%) nor memory is full.  Rows of 8 values a lane have four blocks an SM, all chunks in one wave, which the
// bound keeps: with 77 or 78 registers, three blocks and two waves, it is 15 us more.
template <int G, int V, bool VEC, bool SIGMOID>
__global__ void __launch_bounds__(kThreads, V <= 8 ? 4 : V <= 16 ? 2 : 0)
balance_pieces_kernel(const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
                      Sequences seq, int E, int k, int64_t chunk, Pieces out) {
    constexpr int kSide = 32 / G, kStep = kWarps * kSide;      // rows of a warp, of the block at once
    constexpr bool kFar = V <= 8;                     // registers for two rows to come
    constexpr int kAhead = kFar ? 2 * kStep : kStep;
    extern __shared__ float s_sums[];                 // [warps][E], then the counts [E]
    __shared__ float s_z[kWarps];
    __shared__ int s_bad;
    int* s_counts = reinterpret_cast<int*>(s_sums + kWarps * E);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x % G, side = threadIdx.x % 32 / G;
    const int64_t first = int64_t(blockIdx.x) * chunk, last = min64(first + chunk, seq.T);
    if (blockIdx.x == 0 && threadIdx.x == 0) *out.ticket = 0;
    if (threadIdx.x == 0) s_bad = 0;
    for (int s = seq.find(first); s < seq.S; ++s) {
        const int64_t begin = seq.at(s);
        if (begin >= last) break;
        const int64_t a = max64(begin, first), b = min64(seq.at(s + 1), last);
        if (a >= b) {                   // past sequences without tokens, of which there may be many
            s = max(s, seq.find(a) - 1);
            continue;
        }
        // the next rows load while these are worked on
        const int n = int(b - a), r1 = warp * kSide;
        const float* rows = logits + a * E;
        Row<G, V, VEC> next, later;
        auto row_at = [&](int r) { return rows + int64_t(min(r + side, n - 1)) * E; };
        if (r1 < n) next.load(row_at(r1), E, lane, -INFINITY);
        if (kFar && r1 + kStep < n) later.load(row_at(r1 + kStep), E, lane, -INFINITY);
        for (int e = threadIdx.x; e < E; e += kThreads) s_counts[e] = 0;
        __syncthreads();
        bool bad = false;
        const int slots = n * k;
        for (int i = threadIdx.x; i < slots; i += 4 * kThreads) {
            int id[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                id[j] = i + j * kThreads < slots ? __ldg(topk_idx + a * k + i + j * kThreads) : -1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (id[j] >= 0 && id[j] < E) atomicAdd(s_counts + id[j], 1);
                else bad |= id[j] != -1;
            }
        }
        if (bad) s_bad = 1;
        Row<G, V, VEC> acc;
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) acc.v[i] = make_float2(0.0f, 0.0f);
        for (int r = r1; r < n; r += kStep) {
            const Row<G, V, VEC> row = next;
            const bool live = r + side < n;
            if (kFar) next = later;
            if (r + kAhead < n) (kFar ? later : next).load(row_at(r + kAhead), E, lane, -INFINITY);
            const Scores<G, V, VEC> sc = row_scores<G, V, VEC, SIGMOID>(row);
            // a row past the last adds nothing
            const float part = SIGMOID ? sc.part : sc.inv;
            const float2 f = both(live ? part : 0.0f);
            if (live) z += sc.lse * sc.lse;
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
                acc.v[i] = fma2(SIGMOID ? sc.sig.v[i] : sc.u.v[i], f, acc.v[i]);
        }
        // rows side by side in the warp, then the warps
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int o = G; o < 32; o <<= 1) acc.at(i) += __shfl_xor_sync(0xFFFFFFFFu, acc.at(i), o);
            const int e = Row<G, V, VEC>::expert(i, lane);
            if (side == 0 && e < E) s_sums[warp * E + e] = acc.at(i);
        }
#pragma unroll
        for (int o = G; o < 32; o <<= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
        if (threadIdx.x % 32 == 0) s_z[warp] = z;
        __syncthreads();
        const int64_t piece = int64_t(blockIdx.x) + s;
        for (int e = threadIdx.x; e < E; e += kThreads) {
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += s_sums[w * E + e];
            out.sums[piece * E + e] = sum;
            out.counts[piece * E + e] = s_counts[e];
        }
        if (threadIdx.x == 0) {
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += s_z[w];
            out.z[piece] = sum;
        }
        __syncthreads();
    }
    __syncthreads();
    if (threadIdx.x == 0) out.bad[blockIdx.x] = uint32_t(s_bad);
}

// Sum over the block of one float a thread, in a fixed order.
__device__ __forceinline__ float block_sum(float v, float* s_part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
    __syncthreads();
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += s_part[w];
    __syncthreads();
    return sum;
}

// Block (s, J experts): adds the pieces of sequence s, 256 / J of them side by side and four
// of each in flight; the block that ends last adds up the losses.  In float32: chains of
// float64 additions, slow on this GPU, were 12 us of a join of 256 pieces.  A sequence has
// kMostChunks pieces at most: chains of 19 additions over 32 threads, or 76 over the 8 of many
// sequences, off by 2^-19 or 2^-17.6 at the worst.
constexpr int kJoin = 8;                // few sequences; many: 32 experts a block

template <int J>
__global__ void __launch_bounds__(kThreads)
balance_join_kernel(Sequences seq, int E, int k, int64_t chunk, int chunks, float balance_coef,
                    float z_coef, Pieces in, float* __restrict__ loss,
                    int32_t* __restrict__ counts, float* __restrict__ mean_scores,
                    WsHeader* header) {
    constexpr int kSide = kThreads / J, kDeep = 4;
    __shared__ float s_sum[kWarps][J];
    __shared__ int s_count[kWarps][J];
    __shared__ float s_part[kWarps];
    __shared__ bool s_last;
    const int slices = (E + J - 1) / J;
    const int s = blockIdx.x / slices, slice = blockIdx.x % slices;
    const int col = threadIdx.x % J, side = threadIdx.x / J, e = slice * J + col;
    const int64_t a = seq.at(s), b = seq.at(s + 1), n = b - a;
    wait_for_predecessor();
    float sum = 0.0f, z = 0.0f;
    int count = 0;
    if (n > 0) {
        const int64_t p0 = a / chunk + s, p1 = (b - 1) / chunk + s;
        if (e < E)
            for (int64_t p = p0 + side; p <= p1; p += kSide * kDeep) {
                float v[kDeep];
                int c[kDeep];
#pragma unroll
                for (int i = 0; i < kDeep; ++i) {
                    const int64_t at = p + i * kSide;
                    v[i] = at <= p1 ? __ldcg(in.sums + at * E + e) : 0.0f;
                    c[i] = at <= p1 ? __ldcg(in.counts + at * E + e) : 0;
                }
#pragma unroll
                for (int i = 0; i < kDeep; ++i) sum += v[i], count += c[i];
            }
        if (slice == 0 && z_coef != 0.0f)
            for (int64_t p = p0 + threadIdx.x; p <= p1; p += kThreads) z += __ldcg(in.z + p);
    }
#pragma unroll
    for (int o = J; o < 32; o <<= 1) {
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        count += __shfl_xor_sync(0xFFFFFFFFu, count, o);
    }
    if (threadIdx.x % 32 < J) {
        s_sum[threadIdx.x / 32][col] = sum;
        s_count[threadIdx.x / 32][col] = count;
    }
    if (slice == 0) z = block_sum(z, s_part);
    else __syncthreads();
    if (threadIdx.x < 32) {
        sum = 0.0f, count = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += s_sum[w][col], count += s_count[w][col];
        float part = 0.0f;
        if (threadIdx.x < J && e < E) {
            const float mean = n > 0 ? sum / float(n) : 0.0f;
            counts[int64_t(s) * E + e] = count;
            mean_scores[int64_t(s) * E + e] = mean;
            if (n > 0) part = mean * float(count) * (float(E) / (float(k) * float(n)));
        }
#pragma unroll
        for (int o = J / 2; o > 0; o >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, o);
        if (threadIdx.x == 0) {
            in.seq_loss[blockIdx.x] = part;
            if (slice == 0) in.seq_z[s] = z;
            __threadfence();
            s_last = atomicAdd(in.ticket, 1u) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    float total = 0.0f, total_z = 0.0f;
    bool bad = false;
    for (int64_t i = threadIdx.x; i < int64_t(seq.S) * slices; i += kThreads)
        total += __ldcg(in.seq_loss + i);
    for (int i = threadIdx.x; i < seq.S; i += kThreads) {
        total_z += __ldcg(in.seq_z + i);
        bad |= seq.bad(i);
    }
    for (int i = threadIdx.x; i < chunks; i += kThreads) bad |= __ldcg(in.bad + i) != 0;
    total = block_sum(total, s_part);
    total_z = block_sum(total_z, s_part);
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        const int64_t tokens = max64(seq.at(seq.S) - seq.at(0), 1);
        loss[0] = balance_coef / float(seq.S) * total;
        loss[1] = z_coef != 0.0f ? z_coef / float(tokens) * total_z : 0.0f;
        header->status = bad ? MOE_ERR_DEVICE_CHECK : MOE_OK;
        header->detail = 0;
    }
}

// --------------------------------------------------------------- backward

// 131072 x 256: 47 us with the sigmoid (5.7 TB/s in and out, 236 instructions of a warp a row and
// 57% of the issue slots), 44 with the softmax (6.1 TB/s, 201 and 56%).
template <int G, int V, bool VEC, bool SIGMOID, bool ADD>
__global__ void __launch_bounds__(kThreads)
balance_backward_kernel(const float* __restrict__ logits, const int32_t* __restrict__ counts,
                        Sequences seq, int E, int k, int rounds, float balance_coef, float z_coef,
                        const float* __restrict__ grad_loss, const float* grad_in, float* grad,
                        uint32_t* __restrict__ status) {
    constexpr int kSide = 32 / G;                     // rows of a warp at once
    constexpr bool kAhead = V <= 16;                  // registers for the next rows
    // all the offsets, a thread one or few: rows' walks below step over sequences without tokens
    bool bad = false;
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < seq.S;
         i += int64_t(gridDim.x) * kThreads)
        bad |= seq.bad(int(i));
    if (bad && status) atomicExch(status, uint32_t(MOE_ERR_DEVICE_CHECK));
    const int lane = threadIdx.x % G, side = threadIdx.x % 32 / G;
    // a warp's rows are one run
    const int64_t first = (int64_t(blockIdx.x) * kWarps + threadIdx.x / 32) * kSide * rounds;
    const int64_t last = min64(first + int64_t(kSide) * rounds, seq.T);
    if (first >= last) return;
    auto offset = [&](int64_t t) { return min64(t + side, last - 1) * E; };
    Row<G, V, VEC> next, next_add;
    if (kAhead) {
        next.load(logits + offset(first), E, lane, -INFINITY);
        if (ADD) next_add.load(grad_in + offset(first), E, lane, 0.0f);
    }
    const float g0 = grad_loss ? __ldg(grad_loss) : 1.0f, g1 = grad_loss ? __ldg(grad_loss + 1) : 1.0f;
    const float zc = 2.0f * z_coef * g1 / float(max64(seq.at(seq.S) - seq.at(0), 1));
    int s = seq.find(min64(first + side, last - 1));
    int64_t begin = 0, end = -1;                      // of sequence s
    Row<G, V, VEC> a;
    for (int64_t t0 = first; t0 < last; t0 += kSide) {
        const int64_t t = t0 + side;
        Row<G, V, VEC> row, add;
        if (kAhead) {
            row = next, add = next_add;
            if (t0 + kSide < last) {
                next.load(logits + offset(t0 + kSide), E, lane, -INFINITY);
                if (ADD) next_add.load(grad_in + offset(t0 + kSide), E, lane, 0.0f);
            }
        } else {
            row.load(logits + offset(t0), E, lane, -INFINITY);
            if (ADD) add.load(grad_in + offset(t0), E, lane, 0.0f);
        }
        // the sequence's counts less their mean (whole numbers), over n^2
        const bool fresh = end < 0 || (t >= end && s + 1 < seq.S);
        if (__any_sync(0xFFFFFFFFu, fresh)) {
            // the next one; past sequences without tokens, of which there may be many, by a search
            auto begun = [&] { return s + 1 < seq.S && seq.at(s + 1) <= t; };
            if (begun() && (++s, begun())) s = seq.find(t);
            begin = seq.at(s), end = seq.at(s + 1);
            int c[V], total = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = Row<G, V, VEC>::expert(i, lane);
                c[i] = e < E ? __ldg(counts + int64_t(s) * E + e) : 0;
                total += c[i];
            }
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
            const float n = float(max64(end - begin, 1));
            const float f = balance_coef * g0 / (float(seq.S) * float(k)) / n / n;
#pragma unroll
            for (int i = 0; i < V; ++i) a.at(i) = float(int64_t(c[i]) * E - total) * f;
        }
        Scores<G, V, VEC> sc = row_scores<G, V, VEC, SIGMOID>(row);
        Row<G, V, VEC>& p = SIGMOID ? sc.sig : sc.u;
        const float scale = SIGMOID ? sc.part : sc.inv;
        float2 dot2 = mul2(p.v[0], a.v[0]);
#pragma unroll
        for (int i = 1; i < V / 2; ++i) dot2 = fma2(p.v[i], a.v[i], dot2);
        const float dot = group_sum<G>(dot2.x + dot2.y) * scale;
        const bool inside = t >= begin && t < end;
        const float2 f = both(scale), less = both(-dot), zf = both(sc.lse * zc * sc.inv);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            float2 d = mul2(mul2(p.v[i], f), add2(a.v[i], less));
            if (SIGMOID) d = mul2(d, sc.keep.v[i]);
            if (zc != 0.0f) d = fma2(sc.u.v[i], zf, d);    // (an infinite lse times 0 is NaN)
            if (!inside) d = both(0.0f);              // (padding may hold anything)
            row.v[i] = ADD ? add2(d, add.v[i]) : d;
        }
        if (t < last) row.store(grad + t * E, E, lane);
    }
}

// ----------------------------------------------------------------- host side

int64_t chunk_tokens(int64_t T) {
    const int64_t c = (T + kMostChunks - 1) / kMostChunks;
    return c < kLeastChunk ? kLeastChunk : c;
}

int chunk_count(int64_t T) {
    const int64_t c = chunk_tokens(T), n = (T + c - 1) / c;
    return int(n > 0 ? n : 1);
}

// The workspace's parts; returns its size.
size_t pieces_layout(int64_t T, int E, int S, uint8_t* base, Pieces* p) {
    size_t at = kWsAlign;
    auto part = [&](size_t bytes) {
        uint8_t* q = base ? base + at : nullptr;
        at += align_up(bytes, kWsAlign);
        return q;
    };
    const size_t chunks = size_t(chunk_count(T)), pieces = chunks + size_t(S);
    Pieces w;
    w.ticket = reinterpret_cast<uint32_t*>(part(4));
    w.bad = reinterpret_cast<uint32_t*>(part(4 * chunks));
    w.z = reinterpret_cast<float*>(part(4 * pieces));
    w.seq_loss = reinterpret_cast<float*>(part(4 * size_t(S) * size_t((E + kJoin - 1) / kJoin)));
    w.seq_z = reinterpret_cast<float*>(part(4 * size_t(S)));
    w.sums = reinterpret_cast<float*>(part(4 * pieces * size_t(E)));
    w.counts = reinterpret_cast<int32_t*>(part(4 * pieces * size_t(E)));
    if (p) *p = w;
    return at;
}

moe_status_t check_balance(int64_t T, int E, int k, int S, int score) {
    if (T < 0 || E < 1 || k < 1 || k > E || S < 1) return MOE_ERR_INVALID_ARG;
    if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts || k > kMaxTopK || S > (1 << 24) || T >= (int64_t(1) << 31) / k)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// Calls go(G, V, VEC) as integral constants: lanes of a row and values of a lane, as few
// lanes as leave the values in registers; whether rows come by vectors.
template <typename F>
void with_row_shape(int E, bool vec, F go) {
    auto shape = [&](auto G, auto V) {
        vec ? go(G, V, std::true_type{}) : go(G, V, std::false_type{});
    };
#define MOE_SHAPE(G_, V_) shape(std::integral_constant<int, G_>{}, std::integral_constant<int, V_>{})
    if (E <= 8) MOE_SHAPE(2, 4);
    else if (E <= 16) MOE_SHAPE(4, 4);
    else if (E <= 32) MOE_SHAPE(8, 4);
    else if (E <= 64) MOE_SHAPE(8, 8);
    else if (E <= 128) MOE_SHAPE(16, 8);
    else if (E <= 256) MOE_SHAPE(32, 8);
    else if (E <= 512) MOE_SHAPE(32, 16);
    else MOE_SHAPE(32, 32);
#undef MOE_SHAPE
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_balance_loss_workspace_size(int64_t T, int E, int S, size_t* bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_balance(T, E, 1, S, MOE_SCORE_SOFTMAX);
    if (st != MOE_OK) return st;
    *bytes = pieces_layout(T, E, S, nullptr, nullptr);
    return MOE_OK;
}

extern "C" moe_status_t moe_balance_loss(const float* logits, const int32_t* topk_idx,
                                         const int32_t* seq_offsets, int64_t T, int E, int k, int S,
                                         moe_score_t score, float balance_coef, float z_coef,
                                         float* loss, int32_t* counts, float* mean_scores,
                                         void* workspace, size_t workspace_bytes, void* stream) {
    MOE_TRACE(__func__);
    const moe_status_t st = check_balance(T, E, k, S, score);
    if (st != MOE_OK) return st;
    if ((T > 0 && (!logits || !topk_idx)) || !loss || !counts || !mean_scores ||
        (!seq_offsets && S != 1) || !aligned4(logits) || !aligned4(topk_idx) ||
        !aligned4(seq_offsets) || !aligned4(loss) || !aligned4(counts) || !aligned4(mean_scores))
        return MOE_ERR_INVALID_ARG;
    Pieces p;
    const size_t need = pieces_layout(T, E, S, static_cast<uint8_t*>(workspace), &p);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) ||
        workspace_bytes < need)
        return MOE_ERR_WORKSPACE;
    const Sequences seq{seq_offsets, S, T};
    const int64_t chunk = chunk_tokens(T);
    const int chunks = chunk_count(T), smem = (kWarps + 1) * E * 4;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    with_row_shape(E, E % 4 == 0 && aligned16(logits), [&](auto G, auto V, auto vec) {
        auto go = [&](auto kernel) {
            kernel<<<chunks, kThreads, smem, s>>>(logits, topk_idx, seq, E, k, chunk, p);
        };
        if (score == MOE_SCORE_SIGMOID) go(balance_pieces_kernel<G(), V(), vec(), true>);
        else go(balance_pieces_kernel<G(), V(), vec(), false>);
    });
    if (launch_status() != MOE_OK) return MOE_ERR_CUDA;
    // 131072 tokens in 37 sequences, 256 experts: 1184 blocks of 8 experts took 11 us; one
    // sequence alone takes 8 us with 8 experts a block, 13 with 32
    const int slices = (E + kJoin - 1) / kJoin;
    const bool many = int64_t(S) * slices > 2 * sm_count();
    auto go = [&](auto kernel, int n) {
        return launch_dependent(kernel, unsigned(S) * unsigned(n), kThreads, 0, s, seq, E, k, chunk,
                                chunks, balance_coef, z_coef, p, loss, counts, mean_scores,
                                static_cast<WsHeader*>(workspace)) == cudaSuccess
                   ? launch_status() : MOE_ERR_CUDA;
    };
    return many ? go(balance_join_kernel<32>, (E + 31) / 32) : go(balance_join_kernel<kJoin>, slices);
}

extern "C" moe_status_t moe_balance_loss_backward(const float* logits, const int32_t* counts,
                                                  const int32_t* seq_offsets, int64_t T, int E,
                                                  int k, int S, moe_score_t score,
                                                  float balance_coef, float z_coef,
                                                  const float* grad_loss, const float* grad_in,
                                                  float* grad_logits, void* stream) {
    MOE_TRACE(__func__);
    const moe_status_t st = check_balance(T, E, k, S, score);
    if (st != MOE_OK) return st;
    if ((!seq_offsets && S != 1) || !aligned4(seq_offsets) || !aligned4(grad_loss))
        return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!logits || !counts || !grad_logits || !aligned4(logits) || !aligned4(counts) ||
        !aligned4(grad_in) || !aligned4(grad_logits) || grad_logits == logits)
        return MOE_ERR_INVALID_ARG;
    const Sequences seq{seq_offsets, S, T};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool vec = E % 4 == 0 && aligned16(logits) && aligned16(grad_logits) && aligned16(grad_in);
    with_row_shape(E, vec, [&](auto G, auto V, auto by_vec) {
        // a warp's rows, one run of `rounds` times as many as it takes at once: as many as
        // leave eight blocks an SM, 16 at most
        const int64_t side = kThreads / G();
        const int64_t each = T / (side * 8 * sm_count());
        const int rounds = int(each < 1 ? 1 : each > 16 ? 16 : each);
        const unsigned grid = unsigned((T + side * rounds - 1) / (side * rounds));
        auto go = [&](auto kernel) {
            kernel<<<grid, kThreads, 0, s>>>(logits, counts, seq, E, k, rounds, balance_coef, z_coef,
                                             grad_loss, grad_in, grad_logits, device_status_word());
        };
        constexpr int kG = G(), kV = V();
        constexpr bool kVec = by_vec();
        if (score == MOE_SCORE_SIGMOID)
            grad_in ? go(balance_backward_kernel<kG, kV, kVec, true, true>)
                    : go(balance_backward_kernel<kG, kV, kVec, true, false>);
        else
            grad_in ? go(balance_backward_kernel<kG, kV, kVec, false, true>)
                    : go(balance_backward_kernel<kG, kV, kVec, false, false>);
    });
    return launch_status();
}
