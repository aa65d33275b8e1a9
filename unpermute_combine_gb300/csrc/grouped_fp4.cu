// grouped_fp4.cu -- moe_grouped_matmul_fp4 and moe_grouped_swiglu_fp4: each
// expert's rows times its weights, both in e2m1 with block scales.
//
// The products of "从零理解 MoE 算子" §7 and §8 over expert-contiguous rows, on
// the tensor cores' block-scaled instructions: tcgen05.mma kind::mxf4nvf4 (blocks
// of 16, e4m3 scales) and kind::mxf4 (blocks of 32, powers of two) multiply 64
// columns of both operands with their scales and add in float32, at four times
// the rate of bf16.  A stage of the ring is 256 columns of the reduction: 128
// bytes of codes a row, in 128-byte-swizzled tiles, and the scales in the order in
// which tcgen05.cp takes them to tensor memory (fp4.cuh).
// Three shapes of tile, one kernel:
//   ROWS = 256  256 rows x 256 columns by the two blocks of a cluster (cta_group::2):
//               each has 128 of the rows and brings half of the weights, the leader
//               issues the MMAs of both.  A block alone with 128 x 256 read a third
//               more through L2, copied twice the scales for the same MMAs and ran at
//               3/4 of the rate.
//   ROWS = 128  128 x 128 by one block: less work, which pairs would spread over fewer
//               SMs, and more experts than a pair's schedule has room for (65536 rows, H = 7168,
//               I = 2048, blocks of 32: 256 experts 1320 us, 257 by such blocks 1890).
//   ROWS = 32   32 x 128, still MMAs of 128 rows, whose other rows read whatever lies
//               behind the 32: a few rows an expert, where the weights' way in is what
//               counts and rows' slots would take the place of weights in flight.
// Warps of a block:
//   warp 0       brings codes of rows and weights, and the weights' scales, by TMA
//   warp 1       copies a stage's scales to tensor memory and issues its MMAs
//   warps 2, 3   bring the rows' scales, one stage each in turn, where they are as the
//                quantizers leave them ([rows, K/block]; an expert's rows begin
//                anywhere): lane i loads those of rows i, i + 32, i + 64 and i + 96,
//                which in tensor memory's order lie side by side.  For pairs, whose
//                stages these loads held up (289 us for 16384 x 7168 x 7168 then, 276
//                without), a kernel puts them into the order of packed weights before,
//                for the hidden rows the first product does, and warp 0 brings them.
//   warps 4..7   epilogue: bf16 rows of y, by TMA where a warp's 32 rows are all the
//                expert's, or SwiGLU and the hidden rows' codes
// Persistent blocks take tiles in the order of grouped_swiglu.cu: experts, in an
// expert the column tiles, in those the row tiles.
// Measured: 16384 rows of four experts, 7168 x 7168, 252 us or 6.6 PFLOP/s, the tensor pipe
// 80% busy, until the card's power holds it at 280-295 us; 65536 rows through 64 experts, H =
// 7168, I = 2048, 924 us; 512 rows through them 236 us, 6.7 TB/s of weights; one row, 7168 x
// 2048, 8 us, most of it latency (offsets 0.8, the first tile 1.7, eight stages 2.4).
// Tensor memory has 512 columns: a pair's two accumulators of 256 overlap, so that
// stages' scales fit beside them; the epilogue takes the shared columns first.
// Every wait on an mbarrier is bounded; one that gives up leaves MOE_ERR_TIMEOUT in
// the workspace status word, and the kernel waits for its copies and winds down.
#include <mutex>

#include "fp4.cuh"
#include "tensor_core.cuh"

namespace moe {
namespace {

constexpr int BM = 128;                       // rows of a block's tile (TMEM lanes)
constexpr int kStageCols = kScaleCols;        // columns of the reduction in a stage
constexpr int kRowBytes = kStageCols / 2;     // their codes: one swizzle row
constexpr int kThreads = 256;
constexpr int kTmemCols = 512;
constexpr int kSmallRows = 16;                // rows of the short A box
constexpr int kTileBytes = 128 * kRowBytes;   // codes of 128 rows in a stage
constexpr int kPutCols = 64;                  // columns of y in a staging tile of a warp's 32 rows
constexpr int kPutBytes = 32 * kPutCols * 2;

template <int ROWS, int BLOCK>
struct Shape {
    static_assert(ROWS == 32 || ROWS == 128 || ROWS == 256, "a tile's rows");
    static constexpr int CTAS = ROWS == 256 ? 2 : 1;
    static constexpr int BN = 128 * CTAS;                           // columns of a tile
    static constexpr int kRows = ROWS / CTAS;                       // rows of a block
    static constexpr int kParts = scale_chunk_bytes(BLOCK) / kScalePart;   // TMEM copies a 128 rows
    static constexpr int kScales = scale_chunk_bytes(BLOCK);        // of 128 rows
    // a stage of one block: rows, weights, the rows' scales, those of all BN columns.  (An
    // MMA reads 128 rows from the stage's start: the stage is longer.)
    static constexpr int kWeights = kRows * kRowBytes, kRowScales = kWeights + kTileBytes,
                         kWeightScales = kRowScales + kScales,
                         kStageBytes = kWeightScales + CTAS * kScales;
    static_assert(kStageBytes >= kTileBytes && kStageBytes % 1024 == 0, "a stage");
    static constexpr int kStages = ROWS == 32 ? 8 : 5;
    static constexpr bool kPut = ROWS != 32;                        // y by way of shared memory
    static constexpr int kSmem = kStages * kStageBytes + (kPut ? 4 * 2 * kPutBytes : 0) + 1024;
    static constexpr int kExperts = CTAS == 2 ? 256 : kMaxExperts;  // room of the schedule
    static constexpr int kEpiWarps = kRows / 32;
    // Tensor memory: accumulators, then sets of a stage's scales.  With a set for every stage
    // of the ring a full stage says that its set's last MMAs are done; a pair's scales of
    // blocks of 16 have room for two, and their MMAs are waited for.
    static constexpr int kScaleSet = kParts * (4 + BN / 32);        // columns
    static constexpr int kSets = CTAS == 2 && BLOCK == 16 ? 2 : kStages;
    static constexpr int kScaleBase = kTmemCols - kSets * kScaleSet;
    static constexpr int kAcc1 = kScaleBase - BN < BN ? kScaleBase - BN : BN;
    static_assert(kAcc1 >= 0 && BN - kAcc1 <= 128, "tensor memory");
    static_assert(kSmem + 8 * kExperts + 512 <= 227 * 1024, "shared memory");
};

// Rows' scales in the packed order stand by blocks of kRows rows (32 or 128) of an expert's
// segment.  Block m of expert e has number row0 / kRows + e + m, which no two share: along
// the rows each next block raises one of the first two or the last.
__host__ __device__ inline int64_t scale_blocks(int64_t rows, int E, int block_rows) {
    return rows / block_rows + E + 1;
}

struct Fp4Args {
    const int32_t* offsets;       // [E+1] row segments
    int64_t n_rows;
    int E;
    int K;
    int64_t N;                    // weight rows of an expert
    int n_tiles;                  // column tiles of an expert
    const uint8_t* x_scales;      // [n_rows, K/block], or packed by blocks of rows
    int x_vec;                    // bytes of them that may be read at once: 16, 8, 4 or 1
    const uint8_t* w_scales;      // packed
    const float* alpha;           // [E] or NULL
    void* out;                    // bf16 y [n_rows, N], or hidden codes [n_rows, N/4]
    uint8_t* out_scales;          // hidden scales, packed by blocks of rows
    const float* hidden_scale;    // or NULL
    WsHeader* header;
    bool after_own;               // not the call's first kernel: rows or their scales are another's
};

// ------------------------------------------------------------- PTX helpers

// Shared-memory descriptors without their addresses (bits 0-13, in 16 bytes; a sum with one
// of shared memory's carries nowhere).  Codes: K-major tiles with the 128-byte swizzle, as
// smem_desc_k128.  Scales, for tcgen05.cp: no swizzle, 8-row groups of 16-byte rows 128 bytes
// apart.
constexpr uint64_t kTileDesc = uint64_t(1) << 16 | uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 |
                               uint64_t(2) << 61;
constexpr uint64_t kScaleDesc = uint64_t(128 >> 4) << 16 | uint64_t(128 >> 4) << 32 |
                                uint64_t(1) << 46;

// 32 rows of 16 bytes to the same four columns of all four quarters of the lanes (of each
// of a pair's blocks, from its own shared memory).
template <int CTAS>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t from) {
    if (CTAS == 2)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;"
                     :: "r"(tmem), "l"(from) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;"
                     :: "r"(tmem), "l"(from) : "memory");
}

// Instruction descriptor of the block-scaled kinds: e2m1 A and B (bits 7-9, 10-11
// = 1), N >> 3 in bits 17-22, scale type in bit 23 (1: exponent bytes), M >> 7 in
// bits 27-28, K = 64 (bit 31 = 0); which byte of a 32-bit column an MMA's scales
// begin at in bits 4-5 (B) and 29-30 (A).
template <int CTAS, int BLOCK>
__device__ __forceinline__ uint32_t idesc_fp4(uint32_t byte) {
    return (1u << 7) | (1u << 10) | (uint32_t(16 * CTAS) << 17) |
           (BLOCK == 32 ? 1u << 23 : 0u) | (uint32_t(BM * CTAS >> 7) << 27) | byte << 4 | byte << 29;
}

#define MOE_MMA_FP4(GROUP, KIND)                                                              \
    asm volatile(                                                                             \
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"                                         \
        " tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, [%4], [%5], p;\n}" \
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(scale_a), "r"(scale_b), "r"(accumulate)    \
        : "memory")

template <int CTAS, int BLOCK>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t scale_a, uint32_t scale_b, uint32_t accumulate) {
    if (BLOCK == 16) {
        if (CTAS == 2) MOE_MMA_FP4("2", "mxf4nvf4.block_scale.scale_vec::4X");
        else MOE_MMA_FP4("1", "mxf4nvf4.block_scale.scale_vec::4X");
    } else {
        if (CTAS == 2) MOE_MMA_FP4("2", "mxf4.block_scale.scale_vec::2X");
        else MOE_MMA_FP4("1", "mxf4.block_scale.scale_vec::2X");
    }
}
#undef MOE_MMA_FP4

// The barrier, of a pair's both blocks, completes when the MMAs and copies issued so far have.
template <int CTAS>
__device__ __forceinline__ void commit_all(uint32_t bar) {
    if (CTAS == 2)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
                     ".multicast::cluster.b64 [%0], %1;" :: "r"(bar), "h"(uint16_t(3)) : "memory");
    else
        mma_commit(bar);
}

// A tile by TMA, counted on `bar`: for a pair the leader's, whose address is one of the cluster.
template <int CTAS>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                          uint32_t bar) {
    if (CTAS == 2)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
            ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
            :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
    else
        tma_load_2d(dst, map, c0, c1, bar);
}

__device__ __forceinline__ void store_tile(const CUtensorMap* map, int c0, int c1, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
                 :: "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(src) : "memory");
}

// TMA reads that follow see what other kernels stored before a wait for them.
__device__ __forceinline__ void async_after_stores() {
    asm volatile("fence.proxy.async.global;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// The leader's barrier at the place of this block's.
template <int CTAS>
__device__ __forceinline__ uint32_t leaders(uint32_t bar) {
    if (CTAS == 1) return bar;
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(bar));
    return r;
}

// Arrival at the leader's barrier.  What it announces is for the tensor core alone: a proxy
// fence, or tcgen05's, stands before it, and no thread of the other block reads memory for
// it.  So it releases at the block's scope: at the cluster's it waited for every load and
// store of the thread, and a stage took 0.73 us instead of 0.4.
template <int CTAS>
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    if (CTAS == 2)
        asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
    else
        mbar_arrive(bar);
}

// All threads of the block, or of the pair's blocks.
template <int CTAS>
__device__ __forceinline__ void sync_blocks() {
    tc_fence_before();
    if (CTAS == 2) {
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    } else {
        __syncthreads();
    }
    tc_fence_after();
}

// 128 consecutive float columns of this thread's TMEM lane, with one wait for all: the next
// tile's MMAs wait for these loads.
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x128.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,"
        "%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
        "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,"
        "%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
        "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%128];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]),
          "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]),
          "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]),
          "=f"(v[48]), "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]),
          "=f"(v[56]), "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63]),
          "=f"(v[64]), "=f"(v[65]), "=f"(v[66]), "=f"(v[67]), "=f"(v[68]), "=f"(v[69]), "=f"(v[70]), "=f"(v[71]),
          "=f"(v[72]), "=f"(v[73]), "=f"(v[74]), "=f"(v[75]), "=f"(v[76]), "=f"(v[77]), "=f"(v[78]), "=f"(v[79]),
          "=f"(v[80]), "=f"(v[81]), "=f"(v[82]), "=f"(v[83]), "=f"(v[84]), "=f"(v[85]), "=f"(v[86]), "=f"(v[87]),
          "=f"(v[88]), "=f"(v[89]), "=f"(v[90]), "=f"(v[91]), "=f"(v[92]), "=f"(v[93]), "=f"(v[94]), "=f"(v[95]),
          "=f"(v[96]), "=f"(v[97]), "=f"(v[98]), "=f"(v[99]), "=f"(v[100]), "=f"(v[101]), "=f"(v[102]), "=f"(v[103]),
          "=f"(v[104]), "=f"(v[105]), "=f"(v[106]), "=f"(v[107]), "=f"(v[108]), "=f"(v[109]), "=f"(v[110]), "=f"(v[111]),
          "=f"(v[112]), "=f"(v[113]), "=f"(v[114]), "=f"(v[115]), "=f"(v[116]), "=f"(v[117]), "=f"(v[118]), "=f"(v[119]),
          "=f"(v[120]), "=f"(v[121]), "=f"(v[122]), "=f"(v[123]), "=f"(v[124]), "=f"(v[125]), "=f"(v[126]), "=f"(v[127])
        : "r"(taddr) : "memory");
}

// ------------------------------------------------------------- tile schedule

struct Tile { int e, m, n, row, rows; };      // first row, and rows of the segment from there

// tile_start[e]: tiles, of `tile_rows` rows, of the experts before e; row0: their
// offsets.
__device__ __forceinline__ Tile tile_at(int t, const int* tile_start, const int* row0, int E,
                                        int tile_rows) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tile_start[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int r0 = row0[lo], r1 = row0[lo + 1], mt = (r1 - r0 + tile_rows - 1) / tile_rows;
    const int r = t - tile_start[lo], n = mt == 1 ? r : r / mt, m = r - n * mt;
    return {lo, m, n, r0 + m * tile_rows, min(tile_rows, r1 - r0 - m * tile_rows)};
}

enum Epi : int { kPlain, kSwiglu };

// A lane's scales of a stage: those of four rows, `VALUES` words each.
template <int BLOCK> struct RowScales { uint32_t w[4][scale_chunk_bytes(BLOCK) / kScalePart]; };

// Scales of rows lane, lane + 32, ... of the tile from column chunk ks; 0 for rows
// past the segment and columns past K (a code there is 0, and 0 times a NaN is not).
template <int BLOCK>
__device__ __forceinline__ RowScales<BLOCK> load_scales(const uint8_t* scales, int64_t n_rows, int K,
                                                        int vec, int row, int rows, int ks, int lane) {
    constexpr int W = scale_chunk_bytes(BLOCK) / kScalePart, CB = 4 * W;
    const int64_t stride = K / BLOCK;
    const int left = min(CB, int(stride) - ks * CB);          // scale bytes of the chunk
    RowScales<BLOCK> s;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = lane + 32 * j;
#pragma unroll
        for (int i = 0; i < W; ++i) s.w[j][i] = 0;
        if (r >= rows) continue;
        const uint8_t* p = scales + (row + r) * stride + ks * CB;
        if (vec == CB) {
            if (W == 4) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
                s.w[j][0] = v.x, s.w[j][1] = v.y, s.w[j][W - 2] = v.z, s.w[j][W - 1] = v.w;
            } else {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
                s.w[j][0] = v.x, s.w[j][1] = v.y;
            }
        } else if (vec == 4) {
#pragma unroll
            for (int i = 0; i < W; ++i)
                if (4 * i < left) s.w[j][i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
        } else {
            // rows on any byte: the words around them, shifted, where those lie in the tensor
            const uintptr_t at = reinterpret_cast<uintptr_t>(p);
            const int off = int(at & 3);
            const uint32_t* q = reinterpret_cast<const uint32_t*>(at - off);
            if (p - off >= scales && p - off + CB + 4 <= scales + n_rows * stride) {
                uint32_t w[W + 1];
#pragma unroll
                for (int i = 0; i <= W; ++i) w[i] = __ldg(q + i);
#pragma unroll
                for (int i = 0; i < W; ++i) s.w[j][i] = __funnelshift_r(w[i], w[i + 1], 8 * off);
            } else {
#pragma unroll
                for (int i = 0; i < CB; ++i)
                    if (i < left) s.w[j][i / 4] |= uint32_t(__ldg(p + i)) << (8 * (i % 4));
            }
        }
        if (left < CB)
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const int n = left - 4 * i;
                if (n < 4) s.w[j][i] &= n > 0 ? (1u << (8 * n)) - 1u : 0u;
            }
    }
    return s;
}

// ------------------------------------------------------------- the kernel

struct Fp4Maps {
    CUtensorMap a, a_small, b, w_scales, x_scales, y;
};

// PACKED: the rows' scales are in the packed order.
template <int ROWS, int BLOCK, int EPI, bool PACKED>
__global__ void __cluster_dims__(ROWS == 256 ? 2 : 1, 1, 1) __launch_bounds__(kThreads, 1)
grouped_fp4_kernel(const __grid_constant__ Fp4Maps maps, const Fp4Args args) {
    using S = Shape<ROWS, BLOCK>;
    constexpr int CTAS = S::CTAS, BN = S::BN, kStages = S::kStages, kRows = S::kRows;
    static_assert(PACKED || CTAS == 1, "pairs take packed scales");
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[kStages];      // (the leader's are used)
    __shared__ __align__(8) uint64_t empty_bar[kStages];
    __shared__ __align__(8) uint64_t acc_full_bar[2];
    __shared__ __align__(8) uint64_t acc_free_bar;           // the next tile's MMAs may begin (leader's)
    __shared__ __align__(8) uint64_t drain_bar;
    __shared__ uint32_t s_tmem_base;
    __shared__ int s_tile_start[S::kExperts + 1];
    __shared__ int s_row0[S::kExperts + 1];
    __shared__ int s_warp_tiles[kThreads / 32];
    __shared__ int s_failed;
    __shared__ int s_bad;

    const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = args.E;
    const int rank = CTAS == 2 ? int(cluster_rank()) : 0;

    if (threadIdx.x == 32) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_addr(&full_bar[s]), PACKED ? 1 : 2);    // the copies, the rows' scales
            mbar_init(smem_addr(&empty_bar[s]), 1);
        }
        mbar_init(smem_addr(&acc_full_bar[0]), 1);
        mbar_init(smem_addr(&acc_full_bar[1]), 1);
        mbar_init(smem_addr(&acc_free_bar), S::kEpiWarps * CTAS);
        mbar_init(smem_addr(&drain_bar), 1);
        mbar_fence_init();
    }
    if (warp == 2) {
        if (CTAS == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                         :: "r"(smem_addr(&s_tmem_base)), "r"(kTmemCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                         :: "r"(smem_addr(&s_tmem_base)), "r"(kTmemCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    if (threadIdx.x == 0) {
        if (kRows == BM) prefetch_map(&maps.a);
        prefetch_map(&maps.a_small);
        prefetch_map(&maps.b);
        prefetch_map(&maps.w_scales);
        if (PACKED) prefetch_map(&maps.x_scales);
        s_failed = 0;
        s_bad = 0;
    }
    // The offsets are from before the first of a call's kernels, which has waited for them:
    // the others wait later, for what the one before them writes.
    if (!args.after_own) wait_for_predecessor();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // schedule from the offsets on the device, kEach experts a thread; offsets outside
    // [0, n_rows], or that decrease, leave no tile
    {
        constexpr int kEach = S::kExperts / kThreads;
        const int nr = int(args.n_rows), e0 = int(threadIdx.x) * kEach;
        int raw[kEach + 1], tiles[kEach], sum = 0;
        bool bad = false;
#pragma unroll
        for (int i = 0; i <= kEach; ++i) raw[i] = e0 + i <= E ? __ldg(args.offsets + e0 + i) : 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int r0 = min(max(raw[i], 0), nr), r1 = min(max(raw[i + 1], 0), nr);
            const bool on = e0 + i < E;
            bad |= on && (raw[i] < 0 || raw[i + 1] < raw[i] || raw[i + 1] > nr);
            tiles[i] = on && r1 > r0 ? (r1 - r0 + ROWS - 1) / ROWS * args.n_tiles : 0;
            if (e0 + i <= E) s_row0[e0 + i] = r0;
            sum += tiles[i];
        }
        if (e0 + kEach == E) s_row0[E] = min(max(raw[kEach], 0), nr);
        int incl = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
            if (lane >= off) incl += o;
        }
        if (lane == 31) s_warp_tiles[warp] = incl;
        __syncthreads();
        int before = incl - sum;
        for (int w = 0; w < warp; ++w) before += s_warp_tiles[w];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (e0 + i <= E) s_tile_start[e0 + i] = before;
            before += tiles[i];
        }
        if (e0 + kEach == E) s_tile_start[E] = before;
        if (bad) s_bad = 1;
    }
    sync_blocks<CTAS>();
    // A call's first kernel begins its status.  Another block's timeout comes two seconds
    // after its start, and blocks start in turn.
    if (threadIdx.x == 0 && blockIdx.x == 0 && !args.after_own) {
        args.header->status = MOE_OK;
        args.header->detail = 0;
    }

    const int total = s_bad ? 0 : s_tile_start[E];
    const int first = int(blockIdx.x) / CTAS, step = int(gridDim.x) / CTAS;
    const int k_stages = (args.K + kStageCols - 1) / kStageCols;
    const uint32_t tmem = s_tmem_base;
    const uint32_t full0 = leaders<CTAS>(smem_addr(&full_bar[0]));
    auto stage = [&](uint32_t it) { return smem + it % kStages * S::kStageBytes; };
    auto parity = [&](uint32_t it) { return it / kStages & 1u; };
    auto full_at = [&](uint32_t it) { return full0 + it % kStages * 8; };
    auto tile_of = [&](int t) { return tile_at(t, s_tile_start, s_row0, E, ROWS); };
    // rows of block r in a tile
    auto rows_of = [&](const Tile& at, int r) { return min(max(at.rows - r * BM, 0), kRows); };
    // the packed block of its rows' scales
    auto scale_block = [&](const Tile& at, int r) { return s_row0[at.e] / kRows + at.e + at.m * CTAS + r; };

    if (warp == 0 && elect_one()) {
        // ------------------------------------------------------ copies
        async_after_stores();
        uint32_t it = 0;
        const int nb_all = int((args.N + kScaleRows - 1) / kScaleRows);
        Tile at{};
        // few rows come in short boxes, more in one of all 128
        auto whole = [](int rows) { return kRows == BM && rows > BM / 2; };
        auto boxes = [](int rows) { return (rows + kSmallRows - 1) / kSmallRows; };
        auto row_bytes = [&](int rows) {
            const int codes = whole(rows) ? kTileBytes : boxes(rows) * kSmallRows * kRowBytes;
            return codes + (PACKED && rows > 0 ? S::kScales : 0);
        };
        auto load_weights = [&](int ks, uint32_t i) {        // and what the stage expects in all
            const int nb = at.n * (BN / kScaleRows), parts = min(BN / kScaleRows, nb_all - nb);
            const uint32_t st = stage(i), fb = full_at(i);
            if (rank == 0)
                mbar_expect_tx(fb, row_bytes(rows_of(at, 0)) + (CTAS == 2 ? row_bytes(rows_of(at, 1)) : 0) +
                                       CTAS * (kTileBytes + parts * S::kScales));
            load_tile<CTAS>(st + S::kWeights, &maps.b, ks * kRowBytes,
                            int(at.e * args.N) + at.n * BN + rank * 128, fb);
            // (each block of a pair has the scales of all the tile's columns)
            for (int h = 0; h < parts; ++h)
                load_tile<CTAS>(st + S::kWeightScales + h * S::kScales, &maps.w_scales, 0,
                                ((at.e * nb_all + nb + h) * k_stages + ks) * S::kParts, fb);
        };
        auto load_rows = [&](int ks, uint32_t i) {
            const int rows = rows_of(at, rank), row = at.row + rank * BM;
            const uint32_t st = stage(i), fb = full_at(i);
            if (PACKED && rows > 0)
                load_tile<CTAS>(st + S::kRowScales, &maps.x_scales, 0,
                                (scale_block(at, rank) * k_stages + ks) * S::kParts, fb);
            if (whole(rows)) {
                load_tile<CTAS>(st, &maps.a, ks * kRowBytes, row, fb);
            } else {
                for (int j = 0; j < boxes(rows); ++j)
                    load_tile<CTAS>(st + j * kSmallRows * kRowBytes, &maps.a_small, ks * kRowBytes,
                                    row + j * kSmallRows, fb);
            }
        };
        for (int t = first; t < total && !s_failed; t += step) {
            at = tile_of(t);
            int ks = 0;
            if (args.after_own && it == 0) {
                // the first stages' weights come while the kernel before still runs
                const int n = min(kStages, k_stages);
                for (int i = 0; i < n; ++i) load_weights(i, i);
                wait_for_predecessor();
                async_after_stores();
                for (; ks < n; ++ks, ++it) load_rows(ks, it);
            }
            for (; ks < k_stages; ++ks, ++it) {
                if (!mbar_wait(smem_addr(&empty_bar[it % kStages]), parity(it) ^ 1u)) {
                    s_failed = 1;
                    break;
                }
                load_weights(ks, it);
                load_rows(ks, it);
            }
        }
        // The last stages' commits arrive here too, which no next stage waits for, and nothing may
        // arrive at a block that has ended.
        const uint32_t last = it > kStages ? it - kStages : 0;
        for (uint32_t i = last; i < it && !s_failed; ++i)
            if (!mbar_wait(smem_addr(&empty_bar[i % kStages]), parity(i))) s_failed = 1;
        if (s_failed && rank == 0) {  // copies in flight land before the blocks end
            for (uint32_t i = last; i < it; ++i)
                mbar_wait(smem_addr(&full_bar[i % kStages]), parity(i));
        } else if (s_failed) {
            // the leader's last commit, behind its MMAs, and copies, which have no barrier
            // here: a millisecond
            mbar_wait(smem_addr(&drain_bar), 0);
            for (const uint64_t t0 = global_ns(); global_ns() - t0 < 1000000;) __nanosleep(1000);
        }
    } else if (warp == 1 && rank == 0 && elect_one()) {
        // ------------------------------------------------------ MMAs
        // The one thread's own instructions are what bounds a pair's stage of few MMAs, so
        // descriptors are a base and an offset of their low words, and the ring's place is
        // counted, not divided (297 -> 280 us for 16384 x 7168 x 7168).
        constexpr uint32_t kTileHi = uint32_t(kTileDesc >> 32), kScaleHi = uint32_t(kScaleDesc >> 32);
        const uint32_t tiles0 = uint32_t(kTileDesc) | smem >> 4;
        const uint32_t scales0 = uint32_t(kScaleDesc) | (smem + S::kRowScales) >> 4;
        auto desc = [](uint32_t hi, uint32_t lo) { return uint64_t(hi) << 32 | lo; };
        const uint32_t full = smem_addr(&full_bar[0]), empty = smem_addr(&empty_bar[0]);
        uint32_t s = 0, ph = 0, set = 0, tile = 0;   // stage of the ring and its parity, set of scales
        bool first_round = true;
        for (int t = first; t < total && !s_failed; t += step, ++tile) {
            // the epilogue of the tile before has taken the columns that this one writes
            // (all of its own accumulator's: the epilogue before that one is done)
            if (tile > 0 && !mbar_wait(smem_addr(&acc_free_bar), (tile - 1) & 1u)) {
                s_failed = 1;
                break;
            }
            const uint32_t acc = tmem + (tile & 1u) * S::kAcc1;
            for (int ks = 0; ks < k_stages; ++ks) {
                bool ok = mbar_wait(full + 8 * s, ph);
                if (S::kSets < kStages && (!first_round || s >= S::kSets)) {
                    const bool around = s < S::kSets;
                    ok = ok && mbar_wait(empty + 8 * (around ? s + kStages - S::kSets : s - S::kSets),
                                         around ? ph ^ 1u : ph);
                }
                if (!ok) { s_failed = 1; break; }
                tc_fence_after();
                const uint32_t at = s * (S::kStageBytes >> 4), a = tiles0 + at, sc = scales0 + at;
                const uint32_t ta = tmem + S::kScaleBase + set * S::kScaleSet;
                const uint32_t tb = ta + 4 * S::kParts;
#pragma unroll
                for (int p = 0; p < S::kParts; ++p) {
                    copy_scales<CTAS>(ta + 4 * p, desc(kScaleHi, sc + p * (kScalePart >> 4)));
#pragma unroll
                    for (int h = 0; h < BN / kScaleRows; ++h)
                        copy_scales<CTAS>(tb + p * (BN / 32) + 4 * h,
                                          desc(kScaleHi, sc + ((1 + h) * S::kScales + p * kScalePart >> 4)));
                }
                const int steps = min(4, (args.K - ks * kStageCols + 63) / 64);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    if (kk >= steps) break;
                    const int p = BLOCK == 16 ? kk : kk / 2;
                    mma_fp4<CTAS, BLOCK>(acc, desc(kTileHi, a + kk * 2),
                                         desc(kTileHi, a + (S::kWeights >> 4) + kk * 2),
                                         idesc_fp4<CTAS, BLOCK>(BLOCK == 16 ? 0 : kk % 2 * 2),
                                         ta + 4 * p, tb + p * (BN / 32), (ks | kk) != 0);
                }
                commit_all<CTAS>(empty + 8 * s);
                if (++s == kStages) s = 0, ph ^= 1u, first_round = false;
                if (++set == S::kSets) set = 0;
            }
            if (s_failed) break;
            commit_all<CTAS>(smem_addr(&acc_full_bar[tile & 1u]));
        }
        if (s_failed) {             // MMAs in flight end before tensor memory is freed
            commit_all<CTAS>(smem_addr(&drain_bar));
            mbar_wait(smem_addr(&drain_bar), 0);
        }
    } else if (!PACKED && (warp == 2 || warp == 3)) {
        // -------------------------------- scales of the rows (in a call's first kernel)
        uint32_t it = warp - 2;
        int t = first, ks = warp - 2;
        Tile at{};
        auto settle = [&] {                       // (t, ks) of the stage `it`
            bool moved = false;
            while (ks >= k_stages) ks -= k_stages, t += step, moved = true;
            if (moved && t < total) at = tile_of(t);
        };
        if (t < total) at = tile_of(t);
        settle();
        auto row_scales = [&](const Tile& of, int k) {
            return load_scales<BLOCK>(args.x_scales, args.n_rows, args.K, args.x_vec, of.row, of.rows, k,
                                      lane);
        };
        RowScales<BLOCK> next{};
        if (t < total) next = row_scales(at, ks);
        while (t < total && !__any_sync(0xFFFFFFFFu, s_failed)) {
            const RowScales<BLOCK> now = next;
            ks += 2;
            settle();
            if (t < total) next = row_scales(at, ks);
            const bool free = mbar_wait(smem_addr(&empty_bar[it % kStages]), parity(it) ^ 1u);
            if (!__all_sync(0xFFFFFFFFu, free)) { s_failed = 1; break; }
            const uint32_t dst = stage(it) + S::kRowScales + lane * 16;
#pragma unroll
            for (int p = 0; p < S::kParts; ++p)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                             :: "r"(dst + p * kScalePart), "r"(now.w[0][p]), "r"(now.w[1][p]),
                                "r"(now.w[2][p]), "r"(now.w[3][p]) : "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(full_at(it));
            it += 2;
        }
    } else if (warp >= 4 && warp < 4 + S::kEpiWarps) {
        // ------------------------------------------------------ epilogue
        const int quad = warp - 4;
        const uint32_t lanes = uint32_t(quad * 32) << 16;
        const uint32_t free_bar = leaders<CTAS>(smem_addr(&acc_free_bar));
        const uint32_t put0 = smem + kStages * S::kStageBytes + quad * 2 * kPutBytes;
        Fp4Unit unit{};
        if (EPI == kSwiglu) unit = fp4_unit(BLOCK == 16 ? args.hidden_scale : nullptr);
        uint32_t tile = 0, puts = 0;
        for (int t = first; t < total; t += step, ++tile) {
            const Tile at = tile_of(t);
            const int r = rank * BM + quad * 32 + lane;
            const bool live = r < at.rows;
            const bool all = r - lane + 32 <= at.rows;      // every row of the warp's 32
            const int64_t row = int64_t(at.row) + r;
            const float alpha = args.alpha ? __ldg(args.alpha + at.e) : 1.0f;
            const uint32_t second = tile & 1u;
            const bool full = !s_failed &&
                              mbar_wait(smem_addr(&acc_full_bar[second]), tile >> 1 & 1u);
            if (!__all_sync(0xFFFFFFFFu, full)) { s_failed = 1; break; }
            tc_fence_after();
            const uint32_t acc = tmem + second * S::kAcc1 + lanes;
            // 128 columns at a time; what a pair's accumulators share is in the first one's
            // last 128 and in the second's first
#pragma unroll 1
            for (int i = 0; i < CTAS; ++i) {
                const int h = CTAS == 2 && !second ? 1 - i : i;
                float v[128];
                __syncwarp();
                tmem_ld128(acc + h * 128, v);
                if (i == 0) {        // the next tile's accumulator may be written from here on
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_at<CTAS>(free_bar);
                }
                if (EPI == kSwiglu) {
                    // 64 columns of the gate, then 64 of up
                    const int64_t j0 = int64_t(at.n) * (BN / 2) + h * 64;
                    if (live && j0 < args.N / 2) {
                        uint32_t codes[8], bytes = 0;
#pragma unroll
                        for (int c = 0; c < 64; ++c) {
                            const float a = v[c] * alpha;
                            v[c] = __fdividef(a, 1.0f + __expf(-a)) * (v[64 + c] * alpha);
                        }
#pragma unroll
                        for (int c = 0; c < 64; c += BLOCK) {
                            float sc;
                            const uint32_t byte = fp4_scale<BLOCK>(amax_bits<BLOCK>(v + c), unit, sc);
                            fp4_codes<BLOCK, BLOCK>(v + c, byte, sc, codes + c / 8);
                            bytes |= byte << (8 * (c / BLOCK));
                        }
                        uint8_t* q = static_cast<uint8_t*>(args.out) + row * (args.N / 4) + j0 / 2;
                        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                                     :: "l"(q), "r"(codes[0]), "r"(codes[1]), "r"(codes[2]),
                                        "r"(codes[3]), "r"(codes[4]), "r"(codes[5]), "r"(codes[6]),
                                        "r"(codes[7]) : "memory");
                        // to their packed place: a word of four, or half of one
                        const int k2 = int((args.N / 2 + kStageCols - 1) / kStageCols);
                        const int col = int(j0 % kStageCols), in_block = quad * 32 + lane;
                        uint8_t* sc = args.out_scales +
                                      (int64_t(scale_block(at, rank)) * k2 + j0 / kStageCols) * S::kScales +
                                      in_block % 32 * 16 + in_block / 32 * 4;
                        if (BLOCK == 16) *reinterpret_cast<uint32_t*>(sc + col / 64 * kScalePart) = bytes;
                        else *reinterpret_cast<uint16_t*>(sc + col / 128 * kScalePart + col % 128 / 32) =
                                 uint16_t(bytes);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 128; c += kPutCols) {
                        const int64_t j = int64_t(at.n) * BN + h * 128 + c;
                        if (j >= args.N) break;
                        uint4 o[kPutCols / 8];
#pragma unroll
                        for (int g = 0; g < kPutCols / 8; ++g) {
                            const float* f = v + c + 8 * g;
                            o[g] = make_uint4(pack_bf16x2_rn(f[0] * alpha, f[1] * alpha),
                                              pack_bf16x2_rn(f[2] * alpha, f[3] * alpha),
                                              pack_bf16x2_rn(f[4] * alpha, f[5] * alpha),
                                              pack_bf16x2_rn(f[6] * alpha, f[7] * alpha));
                        }
                        if (S::kPut && all) {
                            // by way of shared memory: 128-byte rows, 16-byte piece g of row r at
                            // g ^ (r % 8); columns past N are left out by the map
                            const uint32_t put = put0 + (puts++ & 1u) * kPutBytes;
                            if (lane == 0) bulk_wait_read<1>();
                            __syncwarp();
#pragma unroll
                            for (int g = 0; g < kPutCols / 8; ++g)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                             :: "r"(put + lane * 128 + ((g ^ (lane & 7)) << 4)),
                                                "r"(o[g].x), "r"(o[g].y), "r"(o[g].z), "r"(o[g].w)
                                             : "memory");
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            __syncwarp();
                            if (lane == 0) {
                                store_tile(&maps.y, int(j), int(row), put);
                                bulk_commit();
                            }
                        } else if (live) {
                            uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(args.out) +
                                                                row * args.N + j);
#pragma unroll
                            for (int g = 0; g < kPutCols / 8; ++g)
                                if (j + 8 * g < args.N) d[g] = o[g];
                        }
                    }
                }
            }
        }
        if (EPI == kPlain && S::kPut && lane == 0) bulk_wait_all();       // every store has landed
        __syncwarp();
    }
    // what follows this kernel follows the one before it too
    if (args.after_own) wait_for_predecessor();
    sync_blocks<CTAS>();
    if (s_failed && threadIdx.x == 0) {
        args.header->status = MOE_ERR_TIMEOUT;
        args.header->detail = blockIdx.x;
    } else if (s_bad && threadIdx.x == 0 && blockIdx.x == 0) {
        atomicCAS(&args.header->status, uint32_t(MOE_OK), uint32_t(MOE_ERR_DEVICE_CHECK));
    }
    __syncwarp();
    if (warp == 2) {
        if (CTAS == 2)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;"
                         :: "r"(tmem), "r"(kTmemCols) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                         :: "r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// Rows' scales [n_rows, K/block] into the packed order by blocks of 128 rows of a segment, for
// pairs: a warp has one block's chunk of 256 columns, as warps 2 and 3 above.  The first
// kernel of its call; 6 us for 16384 x 7168, latency, of which the product's launch hides some.
constexpr int kPackThreads = 256;

template <int BLOCK>
__global__ void __launch_bounds__(kPackThreads)
pack_rows_kernel(const uint8_t* __restrict__ scales, int64_t n_rows, int K, int vec,
                 const int32_t* __restrict__ offsets, int E, int blocks, uint8_t* __restrict__ out,
                 WsHeader* header) {
    wait_for_predecessor();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        header->status = MOE_OK;
        header->detail = 0;
    }
    constexpr int kParts = scale_chunk_bytes(BLOCK) / kScalePart;
    const int lane = threadIdx.x & 31, chunks = (K + kStageCols - 1) / kStageCols;
    const int task = blockIdx.x * (kPackThreads / 32) + threadIdx.x / 32;
    const int b = task / chunks, ks = task - b * chunks;
    if (b >= blocks) return;
    auto row0 = [&](int e) { return min(max(int64_t(__ldg(offsets + e)), int64_t(0)), n_rows); };
    int lo = 0, hi = E - 1;                          // the last expert whose numbers begin by b
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (row0(mid) / BM + mid <= b) lo = mid; else hi = mid - 1;
    }
    const int64_t r0 = row0(lo), r1 = row0(lo + 1), row = r0 + (b - int(r0 / BM) - lo) * int64_t(BM);
    if (row < r0 || row >= r1) return;               // a number that no block has
    const RowScales<BLOCK> s = load_scales<BLOCK>(scales, n_rows, K, vec, int(row),
                                                  int(min64(BM, r1 - row)), ks, lane);
    uint4* dst = reinterpret_cast<uint4*>(out + (int64_t(b) * chunks + ks) * scale_chunk_bytes(BLOCK)) +
                 lane;
#pragma unroll
    for (int p = 0; p < kParts; ++p)
        dst[p * (kScalePart / 16)] = make_uint4(s.w[0][p], s.w[1][p], s.w[2][p], s.w[3][p]);
}

// ----------------------------------------------------------------- host side

// Map over row-major codes [rows, K] (K/2 bytes a row), box [box_rows, 256
// columns], 128-byte swizzle; reads past the last row or column return zeros.
bool make_map_fp4(CUtensorMap* map, const void* base, int64_t rows, int64_t K, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cuuint64_t(K / 2), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(K / 2)};
    const cuuint32_t box[2] = {kRowBytes, cuuint32_t(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Bytes of a row's scales that loads may take at once.
int scale_vec(const uint8_t* base, int64_t stride, int block) {
    const int chunk = kScaleCols / block;
    for (const int v : {chunk, 4})
        if (stride % v == 0 && aligned(base, v)) return v;
    return 1;
}

// Map over packed scales as rows of 512 bytes, box: those of 128 weight rows in a stage.
bool make_map_packed(CUtensorMap* map, const void* base, int64_t bytes, int parts) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {kScalePart / 4, cuuint64_t(bytes / kScalePart)};
    const cuuint64_t strides[1] = {kScalePart};
    const cuuint32_t box[2] = {kScalePart / 4, cuuint32_t(parts)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// Clusters of two of this kernel that the current device runs at once, looked up once.
template <int ROWS, int BLOCK, int EPI, bool PACKED>
int pair_count() {
    static std::mutex m;
    static int cached[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lock(m);
    if (!cached[dev]) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned(sm_count()) / 2 * 2);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Shape<ROWS, BLOCK>::kSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        const auto kernel = (const void*)grouped_fp4_kernel<ROWS, BLOCK, EPI, PACKED>;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) return 0;
        cached[dev] = n < sm_count() / 2 ? n : sm_count() / 2;
    }
    return cached[dev];
}

template <int ROWS, int BLOCK, int EPI, bool PACKED>
moe_status_t launch(const void* x_q, const void* w_q, Fp4Args a, cudaStream_t s) {
    using S = Shape<ROWS, BLOCK>;
    const int64_t chunks = (a.K + kStageCols - 1) / kStageCols;
    Fp4Maps m;
    if ((S::kRows == BM && !make_map_fp4(&m.a, x_q, a.n_rows, a.K, BM)) ||
        !make_map_fp4(&m.a_small, x_q, a.n_rows, a.K, kSmallRows) ||
        !make_map_fp4(&m.b, w_q, a.E * a.N, a.K, 128) ||
        !make_map_packed(&m.w_scales, a.w_scales, a.E * packed_scale_bytes(a.N, a.K, BLOCK), S::kParts) ||
        (PACKED && !make_map_packed(&m.x_scales, a.x_scales,
                                    scale_blocks(a.n_rows, a.E, S::kRows) * chunks * S::kScales,
                                    S::kParts)) ||
        (EPI == kPlain && S::kPut && !make_map(&m.y, a.out, a.n_rows, a.N, 32)))
        return MOE_ERR_CUDA;
    const auto kernel = grouped_fp4_kernel<ROWS, BLOCK, EPI, PACKED>;
    if (!opt_in_smem((const void*)kernel, S::kSmem)) return MOE_ERR_CUDA;
    int blocks = sm_count();
    if constexpr (S::CTAS == 2) blocks = 2 * pair_count<ROWS, BLOCK, EPI, PACKED>();
    if (blocks < 1) return MOE_ERR_CUDA;
    a.n_tiles = int((a.N + S::BN - 1) / S::BN);
    return launch_dependent(kernel, unsigned(blocks), kThreads, S::kSmem, s, m, a) == cudaSuccess
               ? launch_status() : MOE_ERR_CUDA;
}

// May pairs be the choice for M rows, or fewer?  Where M rows make no more tiles of 128 rows
// than of 256, blocks alone have no more rounds than pairs and a shorter stage.
bool pairs_pay(int64_t M, int E) {
    if (E > Shape<256, 16>::kExperts) return false;
    return E == 1 ? M > 128 : M / 128 > (E + 1) / 2;
}

// Rows of a tile for products of E experts, M rows, and for each an N and a K (nothing for a
// second of 0): those of the least estimated time in us.  The segments are known on the
// device alone, so that every expert is taken to have rows, and half a tile to be lost on
// each.  A tile's stage takes about 0.38 us by a pair, 0.32 by a block with 128 rows, and
// 0.22, bound by the weights' way in, with 32; pairs need one more kernel.  Measured on the
// experts' network (E = 64, H = 4096, I = 2048), tiles of 32, 128, 256 rows: 16 rows an
// expert 149, 147, 164 us; 48: 201, 165, 172; 128: 407, 235, 199; 512: 1450, 727, 449.
int tile_rows(int64_t M, int E, int64_t N0, int64_t K0, int64_t N1, int64_t K1) {
    const int64_t active = min64(E, M);
    auto time = [&](int rows, int cols, int64_t at_once, double stage) {
        const int64_t row_tiles = E == 1 ? (M + rows - 1) / rows : max64(active, M / rows + active / 2);
        auto part = [&](int64_t N, int64_t K) {
            const int64_t tiles = row_tiles * ((N + cols - 1) / cols);
            return double((tiles + at_once - 1) / at_once) * double((K + kStageCols - 1) / kStageCols);
        };
        return stage * (part(N0, K0) + part(N1, K1));
    };
    const int sms = sm_count();
    const double few = time(32, 128, sms, 0.22), some = time(128, 128, sms, 0.32);
    const double many = pairs_pay(M, E)
                            ? 2.0 + time(256, 256, sms > 1 ? sms / 2 : 1, 0.38) : some + 1.0;
    if (few <= some && few <= many) return 32;
    return some <= many ? 128 : 256;
}

// Bytes of rows' packed scales.
int64_t packed_rows_bytes(int64_t M, int E, int64_t K, int block, int block_rows) {
    return scale_blocks(M, E, block_rows) * ((K + kStageCols - 1) / kStageCols) * scale_chunk_bytes(block);
}

// The first product of a call: its rows' scales as the quantizers leave them, for pairs
// brought into the packed order first.
template <int BLOCK, int EPI>
moe_status_t first_product(int rows, const void* x_q, const void* w_q, Fp4Args a, uint8_t* packed,
                           cudaStream_t s) {
    const int64_t stride = a.K / BLOCK;
    a.x_vec = scale_vec(a.x_scales, stride, BLOCK);
    if (rows == 32) return launch<32, BLOCK, EPI, false>(x_q, w_q, a, s);
    if (rows == 128) return launch<128, BLOCK, EPI, false>(x_q, w_q, a, s);
    const int blocks = int(scale_blocks(a.n_rows, a.E, BM));
    const int64_t tasks = int64_t(blocks) * ((a.K + kStageCols - 1) / kStageCols);
    constexpr int kEach = kPackThreads / 32;
    if (launch_dependent(pack_rows_kernel<BLOCK>, unsigned((tasks + kEach - 1) / kEach), kPackThreads, 0,
                         s, a.x_scales, a.n_rows, a.K, a.x_vec, a.offsets, a.E, blocks, packed,
                         a.header) != cudaSuccess)
        return MOE_ERR_CUDA;
    a.x_scales = packed;
    a.after_own = true;
    return launch<256, BLOCK, EPI, true>(x_q, w_q, a, s);
}

template <int BLOCK>
moe_status_t second_product(int rows, const void* x_q, const void* w_q, const Fp4Args& a,
                            cudaStream_t s) {
    if (rows == 32) return launch<32, BLOCK, kPlain, true>(x_q, w_q, a, s);
    if (rows == 128) return launch<128, BLOCK, kPlain, true>(x_q, w_q, a, s);
    return launch<256, BLOCK, kPlain, true>(x_q, w_q, a, s);
}

moe_status_t check_product(int64_t M, int E, int64_t N, int64_t K, int block) {
    if (M < 0 || E < 1 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
    if (block != 16 && block != 32) return MOE_ERR_UNSUPPORTED;
    if (E > kMaxExperts || N % 8 != 0 || K % 32 != 0 || K >= (int64_t(1) << 24) ||
        M >= (int64_t(1) << 31) - BM || int64_t(E) * N >= (int64_t(1) << 31) - 256)
        return MOE_ERR_UNSUPPORTED;
    // tiles, and the scales' rows of 512 bytes, are counted in 32 bits
    if ((min64(E, M) + M / 32) * ((N + 127) / 128) >= (int64_t(1) << 31) ||
        E * packed_scale_bytes(N, K, block) / kScalePart >= (int64_t(1) << 31))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

moe_status_t check_layer(int64_t M, int E, int64_t H, int64_t I, int block) {
    if (M < 0 || E < 1 || H < 1 || I < 1) return MOE_ERR_INVALID_ARG;
    if (H % 64 != 0 || I % 64 != 0) return MOE_ERR_UNSUPPORTED;
    const moe_status_t st = check_product(M, E, 2 * I, H, block);
    return st != MOE_OK ? st : check_product(M, E, H, I, block);
}

bool workspace_ok(const void* workspace, size_t bytes, size_t need) {
    return workspace && aligned(workspace, kWsAlign) && bytes >= need;
}

}  // namespace
}  // namespace moe

using namespace moe;

namespace {

// Workspaces have room for what any tile that M rows or fewer may be given needs, so that the
// largest call's serves the smaller ones.  A product's: the status, and where pairs may be
// chosen the rows' packed scales.
size_t matmul_bytes(int64_t M, int E, int64_t K, int block) {
    return kWsAlign +
           (pairs_pay(M, E) ? align_up(size_t(packed_rows_bytes(M, E, K, block, BM)), kWsAlign) : 0);
}

// The layer's: besides, the hidden rows' codes and their packed scales, of which tiles of 32
// rows have the most blocks.
struct LayerParts {
    size_t hidden_q, hidden_scales, bytes;
};

LayerParts layer_parts(int64_t M, int E, int64_t H, int64_t I, int block) {
    LayerParts p;
    p.hidden_q = matmul_bytes(M, E, H, block);
    p.hidden_scales = p.hidden_q + align_up(size_t(M) * size_t(I / 2), kWsAlign);
    p.bytes = p.hidden_scales + align_up(size_t(packed_rows_bytes(M, E, I, block, 32)), kWsAlign);
    return p;
}

}  // namespace

extern "C" moe_status_t moe_grouped_matmul_fp4_workspace_size(int64_t M, int E, int64_t N, int64_t K,
                                                              int block, size_t* bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_product(M, E, N, K, block);
    if (st != MOE_OK) return st;
    *bytes = matmul_bytes(M, E, K, block);
    return MOE_OK;
}

extern "C" moe_status_t moe_grouped_matmul_fp4(const void* x_q, const void* x_scales,
                                               const void* w_q, const void* w_scales,
                                               const float* alpha, const int32_t* offsets,
                                               int64_t M, int E, int64_t N, int64_t K, int block,
                                               void* y, void* workspace, size_t workspace_bytes,
                                               void* stream) {
    MOE_TRACE(__func__);
    const moe_status_t st = check_product(M, E, N, K, block);
    if (st != MOE_OK) return st;
    if (!offsets || (M > 0 && (!x_q || !x_scales || !w_q || !w_scales || !y)))
        return MOE_ERR_INVALID_ARG;
    if (!aligned16(x_q) || !aligned16(w_q) || !aligned16(w_scales) || !aligned16(y) ||
        !aligned(alpha, 4) || !aligned(offsets, 4))
        return MOE_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes, matmul_bytes(M, E, K, block)))
        return MOE_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    WsHeader* header = static_cast<WsHeader*>(workspace);
    if (M == 0)
        return cudaMemsetAsync(header, 0, sizeof *header, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    const Fp4Args a{offsets, M, E, int(K), N, 0, static_cast<const uint8_t*>(x_scales), 0,
                    static_cast<const uint8_t*>(w_scales), alpha, y, nullptr, nullptr, header, false};
    uint8_t* packed = static_cast<uint8_t*>(workspace) + kWsAlign;
    const int rows = tile_rows(M, E, N, K, 0, 0);
    return block == 16 ? first_product<16, kPlain>(rows, x_q, w_q, a, packed, s)
                       : first_product<32, kPlain>(rows, x_q, w_q, a, packed, s);
}

extern "C" moe_status_t moe_grouped_swiglu_fp4_workspace_size(int64_t M, int E, int64_t H,
                                                              int64_t I, int block, size_t* bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_layer(M, E, H, I, block);
    if (st != MOE_OK) return st;
    *bytes = M > 0 ? layer_parts(M, E, H, I, block).bytes : kWsAlign;
    return MOE_OK;
}

extern "C" moe_status_t moe_grouped_swiglu_fp4(
    const void* x_q, const void* x_scales, const void* w_up_q, const void* w_up_scales,
    const void* w_down_q, const void* w_down_scales, const float* alpha_up,
    const float* alpha_down, const float* hidden_scale, const int32_t* offsets, int64_t M, int E,
    int64_t H, int64_t I, int block, void* y, void* workspace, size_t workspace_bytes,
    void* stream) {
    MOE_TRACE(__func__);
    const moe_status_t st = check_layer(M, E, H, I, block);
    if (st != MOE_OK) return st;
    if (!offsets || (M > 0 && (!x_q || !x_scales || !w_up_q || !w_up_scales || !w_down_q ||
                               !w_down_scales || !y)))
        return MOE_ERR_INVALID_ARG;
    if (!aligned16(x_q) || !aligned16(w_up_q) || !aligned16(w_up_scales) || !aligned16(w_down_q) ||
        !aligned16(w_down_scales) || !aligned16(y) || !aligned(alpha_up, 4) ||
        !aligned(alpha_down, 4) || !aligned(hidden_scale, 4) || !aligned(offsets, 4) ||
        (block == 32 && hidden_scale))
        return MOE_ERR_INVALID_ARG;
    const LayerParts parts = layer_parts(M, E, H, I, block);
    if (!workspace_ok(workspace, workspace_bytes, M > 0 ? parts.bytes : kWsAlign))
        return MOE_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    WsHeader* header = static_cast<WsHeader*>(workspace);
    if (M == 0)
        return cudaMemsetAsync(header, 0, sizeof *header, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const int rows = tile_rows(M, E, 2 * I, H, H, I);
    const Fp4Args up{offsets, M, E, int(H), 2 * I, 0, static_cast<const uint8_t*>(x_scales), 0,
                     static_cast<const uint8_t*>(w_up_scales), alpha_up, ws + parts.hidden_q,
                     ws + parts.hidden_scales, hidden_scale, header, false};
    const moe_status_t up_st = block == 16
        ? first_product<16, kSwiglu>(rows, x_q, w_up_q, up, ws + kWsAlign, s)
        : first_product<32, kSwiglu>(rows, x_q, w_up_q, up, ws + kWsAlign, s);
    if (up_st != MOE_OK) return up_st;
    const Fp4Args down{offsets, M, E, int(I), H, 0, ws + parts.hidden_scales, 0,
                       static_cast<const uint8_t*>(w_down_scales), alpha_down, y, nullptr, nullptr,
                       header, true};
    return block == 16 ? second_product<16>(rows, ws + parts.hidden_q, w_down_q, down, s)
                       : second_product<32>(rows, ws + parts.hidden_q, w_down_q, down, s);
}
