// Attention of a chunk of new tokens over the packed cache (sm_103a, tcgen05).
//
// Query i of a sequence sits at position kv_len + i and sees the tokens t <= its position
// (within a window and sinks, when set): the cache's packed tokens dequantized as c*s + z, its
// residual tokens as stored, and the chunk's own tokens as given. Rows are (query, head of the
// kv head's group) pairs, so the whole group shares every key and value tile.
//
// One CTA per SM, warp-specialized, over 128-token tiles:
//   warps 0-3, 4-7   softmax of row tiles 0 and 1 (128 rows each, thread = row): scores from TMEM,
//                    online softmax, probabilities back to TMEM as f16, output epilogue
//   warps 8-11       keys: codes, scales and zeros (or stored rows) to an f16 tile in shared memory
//   warps 12-15      values, the same
//   warps 16, 19     issue tcgen05.mma (kind::f16, M = N = 128), one for each softmax warpgroup: S = Q K^T from
//                    shared memory, O += P V with P from TMEM
//   warp 17          brings packed tokens into shared memory; warp 18 walks the CTA's work
// TMEM: for each row tile two score buffers of 64 tokens (64 columns, P over the first 32) and the
// output (128 columns). While the softmax works on one half of a key tile, the tensor core
// makes the scores of the next half and the other row tile's products: with one 128-token
// buffer per row tile, scores, softmax and products of a tile ran one after the other and took
// 5200 clocks a tile, against 2140 that the tensor core needs for both row tiles.
//
// Rounding: operands are f16 whatever the storage type. With bf16 storage a dequantized token is
// rounded once, fma(c, s, z) to 11 bits, as an f16 cache would hold it; with fp16 storage a key is kept
// in two f16 parts (split_grid) and the scores are two products. One part puts the scores of keys with
// outlier channels off by up to 2^-12 of their products: measured against 64 bits over 1000 to 32768
// tokens, outputs were 6e-4 to 1.1e-3 off (2-norm), where one rounding to fp16 is 2.1e-4 and one to
// bf16 1.7e-3; two parts give 3e-4 at fp16, and at bf16 would take 1373 us instead of 995 (2048 tokens
// over 32768) to bring 2.1e-3 - 2.6e-3 down to 1.7e-3. Stored bf16 tokens with |x| <= 65504 are
// exact in f16 down to 2^-14 (finer ones are rounded at 2^-24). Queries are scaled per row
// by a power of two into (1/2, 1], and the scale is applied to the fp32 scores. Probabilities are
// f16 relative to a running maximum that lags by at most 2^8. Scores, maxima, sums and
// outputs are fp32.
//
// Channels are stored in the order in which the code unpack yields them (pairs (i, i + 8) of 16
// channels at 2 bits, (i, i + 4) of 8 at 4 bits), the same for Q and K, and undone in the epilogue
// for V.
//
// Work is split evenly: the row of units is, for every (sequence, 256-row tile, kv head), the key
// tiles it sees plus an overhead; CTA c takes units [c U / C, (c + 1) U / C). A row tile that
// several CTAs share leaves fp32 records (acc, max, sum) that chunk_merge_kernel joins.
//
// Measured (GB300, 2-bit, 32 query heads on 8 kv heads, bf16): 2048 tokens over 32768 995 us, 1.14
// PFLOP/s, 60 % of what cuBLAS reaches; the TMEM pipe is busy 57 % and the issue slots 60 % of the
// time. Bound by the handoffs of a half tile (scores, softmax, products) together with the issue slots that
// unpacking takes: 450 us with the barriers alone, 783 with the products too, 805 with all but the
// softmax, 886 with all but the unpack. 4 tokens over 64 x 32768: 1.43 ms, 1.14 TB/s; there each tile has 16
// rows, and unpacking it (913 us by itself, eight warps that wait on each other's latencies) is what counts.
#pragma once
#include <type_traits>

#include "kivi_decode_impl.cuh"

namespace kivi {
namespace {

constexpr int kChunkSoftmaxWarps = 8;
constexpr int kChunkThreads = 20 * 32;
constexpr int kRows = 128;                // rows of a row tile
constexpr int kKeys = 128;                // tokens of a key tile
constexpr int kHalf = 64;                 // tokens of a score buffer
constexpr int kOpBytes = kRows * kD * 2;  // one 128 x 128 f16 operand tile
constexpr int kKvStages = 2;
// Registers per thread of the softmax, operand and issue warpgroups: setmaxnreg moves them from
// the launch's 96 x 640, and the three shares add up to it.
constexpr int kSoftmaxRegs = 120, kOperandRegs = 88, kIssueRegs = 64;
constexpr int kLaunchRegs = 96;           // what the launch bounds leave a thread
static_assert(kKvStages == 2, "the barriers' phases count pairs of tiles");
static_assert(kSoftmaxRegs >= kLaunchRegs && kOperandRegs <= kLaunchRegs && kIssueRegs <= kLaunchRegs,
              "setmaxnreg.inc must not lower a count, nor setmaxnreg.dec raise one");
static_assert(256 * kSoftmaxRegs + 256 * kOperandRegs + 128 * kIssueRegs <= kChunkThreads * kLaunchRegs, "shares of the launch's registers");
constexpr int kUnitOverhead = 3;          // units charged per (row tile pair, kv head)
constexpr int kMinChunkUnits = 2;
constexpr float kLag = 8.0f;              // log2 by which the softmax reference may lag behind

// ---------------------------------------------------------------- mbarrier, tcgen05

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// One arrival for the whole warp, after every lane's work before it: 128 arrivals of a warpgroup on
// one barrier are served one after the other.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// Waits for a phase, all lanes of the warp together; gives up (and tells the other roles) after
// about two seconds, so that no mistake in the schedule can hang the device. Both results are the
// same in every lane. The first try stands alone: a phase that is over costs 60 clocks this way and
// 190 with the limits in its loop, and the issuing warps wait six times per key tile.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* stop) {
    if (__all_sync(kFull, mbar_try(bar, parity))) return true;
    const long long t0 = clock64();
#pragma unroll 1
    while (!__all_sync(kFull, mbar_try(bar, parity))) {
        if (__any_sync(kFull, *stop != 0 || clock64() - t0 > 4000000000LL)) {
            *stop = 1;
            return false;
        }
    }
    return true;
}
// The same for a single lane.
__device__ __forceinline__ bool lane_wait(uint32_t bar, uint32_t parity, volatile int* stop) {
    const long long t0 = clock64();
    while (!mbar_try(bar, parity)) {
        if (*stop != 0 || clock64() - t0 > 4000000000LL) {
            *stop = 1;
            return false;
        }
    }
    return true;
}

// One lane of the (converged) warp, always the same one
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{ .reg .pred q; elect.sync _|q, 0xffffffff; selp.u32 %0, 1, 0, q; }" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 32 columns of this warp's 32 lanes
__device__ __forceinline__ void tc_ld32(float (&r)[32], uint32_t addr) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
          "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
          "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(addr));
}
__device__ __forceinline__ void tc_ld16(float (&r)[16], uint32_t addr) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(addr));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const float (&r)[32]) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(r);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
        ::"r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
          "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]),
          "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]),
          "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&u)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
        ::"r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
          "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(addr)
        : "memory");
}

// Two fp32 at a time
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
        "l"(reinterpret_cast<uint64_t&>(c)));
    return reinterpret_cast<float2&>(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return reinterpret_cast<float2&>(d);
}

// Operand tiles in shared memory: two blocks of 64 channels, each 128 rows of 128 bytes with the
// 16-byte chunks of a row XORed by its low three bits (the 128-byte swizzle).
__device__ __forceinline__ uint32_t op_addr(int row, int chunk) {   // chunk of 8 channels, 0 .. 15
    return static_cast<uint32_t>((chunk >> 3) * (kRows * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}
// Key stages. bf16: one key tile of 128 rows. f16: half a tile, 64 rows of each channel block, twice: the
// keys' leading parts and, behind them, their rests (split_grid). Two stages either way.
template <bool LO>
struct KeyStage {
    static constexpr int kBlock = (LO ? kHalf : kKeys) * 128;   // bytes of a 64-channel block
    static constexpr int kRest = 2 * kBlock;                    // where the rests begin (LO)
};
template <bool LO>
__device__ __forceinline__ uint32_t key_addr(int row, int chunk) {
    return static_cast<uint32_t>((chunk >> 3) * KeyStage<LO>::kBlock + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}
// Shared-memory descriptors, 128-byte swizzle, as (low word, high word): K-major (Q, K) has rows of 8
// every 1024 bytes; MN-major (V: channels contiguous) has 64-channel blocks every kRows * 128 bytes
// and groups of 8 tokens every 1024. Only the low word's address changes from one product to the next.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return ((addr & 0x3ffffu) >> 4) | ((lbo >> 4) << 16); }
// f32 accumulator, f16 operands, M = 128, N = 64 (scores) or 128; bit 16: B is MN-major
constexpr uint32_t kIdescQK = (1u << 4) | ((kHalf / 8) << 17) | ((kRows / 16) << 24);
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | ((kD / 8) << 17) | ((kRows / 16) << 24);

// One K = 16 step, A from shared memory or from TMEM; acc 0 overwrites D, 1 adds to it.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{ .reg .pred p; .reg .b64 x, y; mov.b64 x, {%1, %3}; mov.b64 y, {%2, %3}; setp.ne.b32 p, %5, 0;"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p; }"
        ::"r"(d), "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{ .reg .pred p; .reg .b64 y; mov.b64 y, {%2, %3}; setp.ne.b32 p, %5, 0;"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p; }"
        ::"r"(d), "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "r"(acc) : "memory");
}

// ---------------------------------------------------------------- the row of units

// One (sequence, pair of row tiles): rows [0, rows) of it hold the (query, head) pairs from
// row0 on; nt listed key tiles (tile i < st is tile i, the others i + skip).
struct ChunkItem {
    int64_t L;            // cached tokens
    int b, n, row0, rows; // sequence, its new tokens, first row, rows in this pair of tiles
    int nt, st, skip;
};

__device__ __forceinline__ bool chunk_seq(const ChunkArgs& a, int b, int64_t* L, int* n) {
    *n = a.n_new[b];
    *L = a.kv_len[b];
    if (*n < 0 || *n > a.max_new) {
        *n = 0;
        return false;
    }
    return *L >= 0 && *L <= a.max_kv_len && n_packed(*L, a.R, a.G) <= a.seqs[b].cap_tokens;
}

__device__ __forceinline__ ChunkItem chunk_item(const ChunkArgs& a, int idx) {
    ChunkItem it;
    it.b = idx / a.pairs;
    const int64_t row0 = static_cast<int64_t>(idx - it.b * a.pairs) * (2 * kRows);
    const int g = a.Hq / a.H;
    it.nt = it.st = it.skip = it.rows = 0;
    it.row0 = 0;
    if (!chunk_seq(a, it.b, &it.L, &it.n)) return it;
    const int64_t left = static_cast<int64_t>(it.n) * g - row0;
    if (left <= 0) return it;
    it.row0 = static_cast<int>(row0);
    it.rows = static_cast<int>(left < 2 * kRows ? left : 2 * kRows);
    const int64_t q0 = row0 / g, q1 = (row0 + it.rows - 1) / g;
    const int64_t hi = it.L + q1 + 1;                                     // tokens the last query sees
    const int nt = static_cast<int>((hi + kKeys - 1) / kKeys);
    it.nt = nt;
    if (a.window > 0) {
        const int64_t lo = it.L + q0 + 1 - a.window;                     // first token of the first query's window
        if (lo > 0) {
            const int64_t s = a.sinks < hi ? a.sinks : hi;
            const int st = static_cast<int>((s + kKeys - 1) / kKeys), w0 = static_cast<int>(lo / kKeys);
            if (w0 > st) {
                it.st = st;
                it.skip = w0 - st;
                it.nt = nt - it.skip;
            }
        }
    }
    return it;
}
__device__ __forceinline__ int64_t item_units(const ChunkItem& it) { return it.nt > 0 ? it.nt + kUnitOverhead : 0; }

// A CTA's share of the row of units; chunk_next yields its segments (a row tile pair of one kv
// head, listed key tiles [x0, x1)).
struct ChunkWalk {
    int64_t lo, hi, pos;        // this CTA's units, first unit of item idx
    int64_t U;
    int idx, C, h;
};
struct ChunkSeg {
    ChunkItem it;
    int h, x0, x1;
    int nseg;   // CTAs that share it
};

__device__ __forceinline__ bool chunk_next(const ChunkArgs& a, ChunkWalk& w, ChunkSeg& s) {
    const int items = a.nseq * a.pairs;   // below 2^31, by the entry point
    while (w.idx < items && w.pos < w.hi) {
        s.it = chunk_item(a, w.idx);
        const int64_t u = item_units(s.it);
        for (; u > 0 && w.h < a.H; ++w.h) {
            const int64_t first = w.pos + w.h * u + kUnitOverhead, end = first + s.it.nt;
            if (first - kUnitOverhead >= w.hi) return false;
            const int64_t x0 = (w.lo > first ? w.lo : first) - first, x1 = (w.hi < end ? w.hi : end) - first;
            if (x1 > x0) {
                s.h = w.h++;
                s.x0 = static_cast<int>(x0);
                s.x1 = static_cast<int>(x1);
                s.nseg = static_cast<int>(owner(end - 1, w.U, w.C) - owner(first, w.U, w.C)) + 1;
                return true;
            }
        }
        w.pos += u * a.H;
        ++w.idx;
        w.h = 0;
    }
    return false;
}

// Raw packed tokens on their way from memory: a stage holds two subtiles (32 tokens
// of one kv head each: codes, scales and zeros of keys and values). As many stages as fit
// beside the operand tiles.
template <int KB, int VB>
struct RawLayout {
    static constexpr int kKc = 0, kKs = kTile * kD * KB / 8, kKz = kKs + kD * 2, kVc = kKz + kD * 2;
    static constexpr int kVs = kVc + kTile * kD * VB / 8, kVz = kVs + 256, kSub = kVz + 256;   // 128 of the last two used when G = 64
    static constexpr int kBytes = 2 * kSub;
    static constexpr int kStages = KB + VB == 4 ? 5 : KB + VB == 6 ? 4 : 3;
};
constexpr int kRawMax = 5;
constexpr int kSegs = 4;                  // segments announced ahead (warp 18 walks, every role follows)
constexpr int kSegReaders = 19;           // every warp but the walking one

struct ChunkShared {
    uint64_t k_full[2 * kKvStages], k_empty[kKvStages], v_full[kKvStages], v_empty[kKvStages];
    uint64_t s_full[4], p_full[4], o_step[4];   // [softmax warpgroup][half]
    uint64_t q_full[2 * kSegs];                 // [segment slot][softmax warpgroup]
    uint64_t raw_full[kRawMax], raw_empty[kRawMax], hand_full, hand_empty, seg_full[kSegs], seg_empty[kSegs];
    ChunkSeg seg[kSegs];
    float hand_m[kRows], hand_l[kRows];   // state of the second softmax warpgroup at the end of a narrow segment
    int64_t warp_sum[kChunkThreads / 32];
    int64_t lo, hi, pos, U;
    int idx, C, h;
    uint32_t tmem;
    int stop;
};
template <int KB, int VB>
constexpr int chunk_smem() {
    constexpr int bytes = 2 * kOpBytes + 2 * kKvStages * kOpBytes + RawLayout<KB, VB>::kStages * RawLayout<KB, VB>::kBytes +
                          1024 + static_cast<int>(sizeof(ChunkShared));
    static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
    return bytes;
}

// ---------------------------------------------------------------- operand tiles

// Position p (0 .. 15) of a 16-channel span holds channel perm(p): the order code_pair yields.
template <int BITS>
__host__ __device__ constexpr int span_channel(int p) {
    return BITS == 2 ? (p >> 1) + 8 * (p & 1) : (p & 8) + ((p & 7) >> 1) + 4 * (p & 1);
}

// The f16 pairs of span positions (2 i, 2 i + 1), i = 0 .. 7, from 16 values of 16 bits in channel order
// (eight words).
template <int BITS>
__device__ __forceinline__ void pair_words(const uint32_t (&w)[8], uint32_t (&out)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c0 = span_channel<BITS>(2 * i), c1 = span_channel<BITS>(2 * i + 1);
        out[i] = prmt(w[c0 >> 1], w[c1 >> 1], (c0 & 1) ? 0x7632u : 0x5410u);   // c0 and c1 have equal parity
    }
}
// The same from stored values of type DT, converted to f16.
template <int BITS, int DT>
__device__ __forceinline__ void pair_stored(const uint32_t (&w)[8], uint32_t (&out)[8]) {
    if constexpr (DT == KIVI_F16) {
        pair_words<BITS>(w, out);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c0 = span_channel<BITS>(2 * i), c1 = span_channel<BITS>(2 * i + 1);
            const float x0 = __uint_as_float((c0 & 1) ? w[c0 >> 1] & 0xffff0000u : w[c0 >> 1] << 16);
            const float x1 = __uint_as_float((c1 & 1) ? w[c1 >> 1] & 0xffff0000u : w[c1 >> 1] << 16);
            out[i] = pack_h2(x0, x1);
        }
    }
}
// The exact f16 codes of a span (BITS words) as pairs in the same order.
template <int BITS>
__device__ __forceinline__ void pair_codes(const uint32_t (&w)[BITS / 2], uint32_t (&out)[8]) {
    if constexpr (BITS == 2) {
        const uint32_t ws = w[0] >> CodeShift<2>::kValue;
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = code_slot<2>(w[0], ws, i);
    } else {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const uint32_t ws = w[m] >> CodeShift<4>::kValue;
#pragma unroll
            for (int i = 0; i < 4; ++i) out[4 * m + i] = code_slot<4>(w[m], ws, i);
        }
    }
}

__device__ __forceinline__ void load8(uint32_t (&w)[8], const void* p) {
    const uint4* q = static_cast<const uint4*>(p);
    const uint4 a = __ldg(q), b = __ldg(q + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// Splits scale and zero of two channels, s = sh + sl and z = zh + zl exactly, with sh and zh on a grid so
// coarse that c sh + zh is an f16 number for every code c. Let 2^e <= max(|z|, |qmax s + z|) < 2^(e + 1). Adding and
// taking away 1.5 * 2^(e + 2), whose last bit is worth 2^(e - 8), rounds s and z to multiples of 2^(e - 8); the
// levels c sh + zh are then below 2^10 of those. A dequantized key is fma(c, sh, zh), exact, plus
// fma(c, sl, zl), at most 2^(e - 5) and rounded at 2^-11 of that: together 2^-16 of the largest level
// where one f16 number gives 2^-11. From 2^13 on, where the sums could overflow, sh = s and zh = z, one
// rounding as with bf16.
template <int BITS>
__device__ __forceinline__ void split_grid(uint32_t s, uint32_t z, uint32_t& sh, uint32_t& zh, uint32_t& sl, uint32_t& zl) {
    constexpr uint32_t kQmax = BITS == 2 ? 0x42004200u : 0x4B804B80u;   // 3 or 15
    const uint32_t m = hmax2(z & 0x7fff7fffu, hfma2(kQmax, s, z) & 0x7fff7fffu);
    const uint32_t big = (((m + 0x10001000u) & 0x80008000u) >> 15) * 0xffffu;   // halves from 2^13 on
    const uint32_t c = (((m & 0x7C007C00u) + 0x08000800u) | 0x02000200u) & ~big;
    sh = hsub2(hadd2(s, c), c);
    zh = hsub2(hadd2(z, c), c);
    sl = hsub2(s, sh);
    zl = hsub2(z, zh);
}

// A warp's part of a packed subtile (32 tokens): lane (row_lo = lane % 8, span) has rows row_lo + 8 k of
// one 16-channel span, k = 0 .. 3, so that the span's key scales are read and paired once for four rows and
// the eight lanes of a store phase hit eight rows, whose chunks lie in distinct banks under the swizzle.
// st: the raw stage, already at the lane's place (row_lo, span) of each part; dst: the operand tile at row
// row_lo of the subtile, a0 and a1 the lane's chunk offsets; gsh = log2 G.
template <int KB, int VB, bool VALUES, bool LO>
__device__ __forceinline__ void fill_packed(const unsigned char* st, int gsh, int row_lo, int span, unsigned char* dst, uint32_t a0,
                                            uint32_t a1) {
    using Raw = RawLayout<KB, VB>;
    constexpr int BITS = VALUES ? VB : KB;
    constexpr int kRowBytes = kD * BITS / 8, kSpanBytes = 2 * BITS;
    const unsigned char* codes = st + (VALUES ? Raw::kVc : Raw::kKc) + row_lo * kRowBytes + span * kSpanBytes;
    // every load of the subtile before its first store (a store could alias a later load, so the
    // compiler would keep them in order)
    uint32_t w[4][BITS / 2], sc[8], zr[8], s1[4], z1[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (BITS == 2) {
            w[k][0] = *reinterpret_cast<const uint32_t*>(codes + 8 * k * kRowBytes);
        } else {
            const uint2 x = *reinterpret_cast<const uint2*>(codes + 8 * k * kRowBytes);
            w[k][0] = x.x;
            w[k][1] = x.y;
        }
    }
    if constexpr (!VALUES) {
        auto row = [&](int at, uint32_t (&out)[8]) {
            const uint4 a = *reinterpret_cast<const uint4*>(st + at + span * 32), b = *reinterpret_cast<const uint4*>(st + at + span * 32 + 16);
            const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            pair_words<BITS>(x, out);
        };
        row(Raw::kKs, sc);
        row(Raw::kKz, zr);
    } else {
        const int vsh = 8 - gsh;   // log2 of the bytes of a token's value scales, 2 D / G
        const unsigned char* meta = st + Raw::kVs + (row_lo << vsh) + (((span * 16) >> gsh) << 1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            s1[k] = *reinterpret_cast<const uint16_t*>(meta + ((8 * k) << vsh));
            z1[k] = *reinterpret_cast<const uint16_t*>(meta + ((8 * k) << vsh) + (Raw::kVz - Raw::kVs));
        }
    }
    if constexpr (!VALUES && LO) {
        // by eight channels (one chunk of the row), so that the split scales of both do not have to be held
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            uint32_t sh[4], zh[4], sl[4], zl[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) split_grid<BITS>(sc[4 * p + i], zr[4 * p + i], sh[i], zh[i], sl[i], zl[i]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t c;
                    if constexpr (BITS == 2) c = code_slot<2>(w[k][0], w[k][0] >> CodeShift<2>::kValue, 4 * p + i);
                    else c = code_slot<4>(w[k][p], w[k][p] >> CodeShift<4>::kValue, i);
                    hi[i] = hfma2(c, sh[i], zh[i]);
                    lo[i] = hfma2(c, sl[i], zl[i]);
                }
                unsigned char* to = dst + (p == 0 ? a0 : a1) + 1024 * k;
                *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(to + KeyStage<LO>::kRest) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t c[8];
            pair_codes<BITS>(w[k], c);
            if constexpr (VALUES) {
                const uint32_t s2 = prmt(s1[k], s1[k], 0x1010u), z2 = prmt(z1[k], z1[k], 0x1010u);
#pragma unroll
                for (int i = 0; i < 8; ++i) c[i] = hfma2(c[i], s2, z2);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) c[i] = hfma2(c[i], sc[i], zr[i]);
            }
            *reinterpret_cast<uint4*>(dst + a0 + 1024 * k) = make_uint4(c[0], c[1], c[2], c[3]);
            *reinterpret_cast<uint4*>(dst + a1 + 1024 * k) = make_uint4(c[4], c[5], c[6], c[7]);
        }
    }
}

// Stored tokens (the ring's and the chunk's own) of a kv head.
struct ChunkStored {
    const uint16_t *res, *fresh;
    int L, end;   // cached tokens; cached and new ones
    int ring;
};
// One row of a lane's span at token t; a row behind the last token is zeros.
__device__ __forceinline__ void load_row(const ChunkStored& s, int t, int span, uint32_t (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0;
    if (t < s.L) load8(w, s.res + static_cast<int64_t>(t % s.ring) * kD + span * 16);
    else if (t < s.end) load8(w, s.fresh + static_cast<int64_t>(t - s.L) * kD + span * 16);
}
// The four rows of a lane of the stored subtile at token tb.
__device__ __forceinline__ void load_stored(const ChunkStored& s, int tb, int row_lo, int span, uint32_t (&w)[4][8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) load_row(s, tb + row_lo + 8 * k, span, w[k]);
}

// ---------------------------------------------------------------- the kernel

// Records of row tile pairs that several CTAs share: slot 2 c of CTA c for a pair begun by an
// earlier CTA, 2 c + 1 for one begun here. A slot holds, per row tile, acc as [32 channel quads][128 rows]
// float4, then max[128] and sum[128].
constexpr int64_t kRecFloats = kRows * (kD + 2);
__device__ __forceinline__ float* chunk_record(const ChunkArgs& a, int64_t slot, int tile) {
    return a.records + (slot * a.rec_tiles + tile) * kRecFloats;
}

// One thread's row of the output: 32 channels from c0 on.
template <int DT>
__device__ __forceinline__ void store32(void* out, int64_t row, int c0, const float (&x)[32]) {
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row * kD + c0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float lo = x[8 * i + 2 * k], hi = x[8 * i + 2 * k + 1];
            if constexpr (DT == KIVI_F16) w[k] = pack_h2(lo, hi);
            else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(hi), "f"(lo));
        }
        o[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int KB, int VB, int DT>
__global__ void __launch_bounds__(kChunkThreads, 1) chunk_kernel(ChunkArgs a) {
    extern __shared__ unsigned char raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    unsigned char* sq_tile = smem;                                   // [2] query tiles
    unsigned char* sk_tile = smem + 2 * kOpBytes;                    // [kKvStages]
    unsigned char* sv_tile = sk_tile + kKvStages * kOpBytes;         // [kKvStages]
    using Raw = RawLayout<KB, VB>;
    constexpr bool LO = DT == KIVI_F16;    // keys in two parts: an f16 output would show one's rounding, a bf16 one hardly does
    unsigned char* raw_ring = sv_tile + kKvStages * kOpBytes;        // [Raw::kStages] raw packed subtiles
    ChunkShared& sh = *reinterpret_cast<ChunkShared*>(raw_ring + Raw::kStages * Raw::kBytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
    const int g = a.Hq / a.H;
    volatile int* stop = &sh.stop;
    asm volatile("griddepcontrol.launch_dependents;");

    // sequences without valid lengths: NaN rows and a status
    for (int b = c; b < a.nseq; b += gridDim.x) {
        int64_t L;
        int n;
        if (chunk_seq(a, b, &L, &n)) continue;
        uint16_t* o = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(a.q_start[b]) * a.Hq * kD;
        for (int64_t i = tid; i < static_cast<int64_t>(n) * a.Hq * kD; i += kChunkThreads) o[i] = 0x7fff;   // NaN in both types
        if (tid == 0) set_status(a.status, KIVI_ERR_LENGTH);
    }

    if (tid == 0) {
        for (int i = 0; i < kKvStages; ++i) {
            // (f16: a stage has a barrier for even tiles and one for odd ones, so that an issuing warp that takes every
            // other tile sees every phase of the one it waits for; a parity tells two neighbouring phases apart only)
            mbar_init(smem_u32(&sh.k_full[2 * i]), LO ? 2 : 4);
            mbar_init(smem_u32(&sh.k_full[2 * i + 1]), LO ? 2 : 4);
            mbar_init(smem_u32(&sh.k_empty[i]), 2);   // one per issuing warp
            mbar_init(smem_u32(&sh.v_full[i]), 4);
            mbar_init(smem_u32(&sh.v_empty[i]), 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.s_full[2 * i]), 1);
            mbar_init(smem_u32(&sh.s_full[2 * i + 1]), 1);
            mbar_init(smem_u32(&sh.p_full[2 * i]), 4);
            mbar_init(smem_u32(&sh.p_full[2 * i + 1]), 4);
            mbar_init(smem_u32(&sh.o_step[2 * i]), 1);
            mbar_init(smem_u32(&sh.o_step[2 * i + 1]), 1);
        }
        for (int i = 0; i < Raw::kStages; ++i) {
            mbar_init(smem_u32(&sh.raw_full[i]), 32);   // the loader's lanes
            mbar_init(smem_u32(&sh.raw_empty[i]), 4);   // the warps that read a subtile
        }
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(smem_u32(&sh.q_full[2 * i]), 4);
            mbar_init(smem_u32(&sh.q_full[2 * i + 1]), 4);
            mbar_init(smem_u32(&sh.seg_full[i]), 1);
            mbar_init(smem_u32(&sh.seg_empty[i]), kSegReaders);
        }
        mbar_init(smem_u32(&sh.hand_full), 4);
        mbar_init(smem_u32(&sh.hand_empty), 4);
        sh.stop = 0;
        sh.idx = INT32_MAX;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 16) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }

    // units of each thread's run of items, their exclusive prefix and the total
    const int items = a.nseq * a.pairs, per = (items + kChunkThreads - 1) / kChunkThreads;
    const int i0 = static_cast<int>(static_cast<int64_t>(tid) * per < items ? static_cast<int64_t>(tid) * per : items);
    const int i1 = items - i0 < per ? items : i0 + per;
    int64_t mine = 0;
    for (int i = i0; i < i1; ++i) mine += item_units(chunk_item(a, i)) * a.H;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sh.warp_sum[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int64_t before = 0, U = 0;
    for (int w = 0; w < kChunkThreads / 32; ++w) {
        before += w < warp ? sh.warp_sum[w] : 0;
        U += sh.warp_sum[w];
    }
    const int64_t by_size = U / kMinChunkUnits > 1 ? U / kMinChunkUnits : 1;
    const int64_t C = by_size < gridDim.x ? by_size : gridDim.x;
    if (U > 0 && c < C) {
        const int64_t lo = c * U / C, start = before + incl - mine;
        if (lo >= start && lo < start + mine) {
            int64_t p = start;
            for (int i = i0; i < i1; ++i) {
                const int64_t u = item_units(chunk_item(a, i));
                if (lo < p + u * a.H) {
                    sh.lo = lo;
                    sh.hi = (c + 1) * U / C;
                    sh.pos = p;
                    sh.idx = i;
                    sh.U = U;
                    sh.C = static_cast<int>(C);
                    sh.h = static_cast<int>((lo - p) / u);
                    break;
                }
                p += u * a.H;
            }
        }
    }
    if (tid == 0) a.info[c].nseg = 0;
    __syncthreads();
    const uint32_t tmem = sh.tmem;
    bool ok = true;
    // segment i of this CTA in sh.seg: whether there is one, and the word that this warp is done with it
    auto seg_next = [&](uint32_t i) {
        ok = warp_wait(smem_u32(&sh.seg_full[i % kSegs]), (i / kSegs) & 1, stop);
        return ok && sh.seg[i % kSegs].x1 > 0;
    };
    auto seg_done = [&](uint32_t i) {
        warp_arrive(smem_u32(&sh.seg_empty[i % kSegs]));
    };

    if (warp < kChunkSoftmaxWarps) {
        // ------------------------------------------------ softmax
        // Wide segments: warpgroup t has row tile t. Narrow ones (at most 128 rows): both have the one row
        // tile, and take its key tiles in turn, each with its own state and output columns, joined at the end.
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int wg = warp >> 2, r = tid & 127;
        const uint32_t lane_off = static_cast<uint32_t>(warp & 3) << 21;     // this warp's 32 TMEM lanes
        const uint32_t t_s = tmem + lane_off + wg * kKeys, t_o = tmem + lane_off + 2 * kKeys + wg * kD;
        uint32_t ns = 0, nh = 0;    // key tiles and handed states so far
        for (uint32_t si = 0; ok && seg_next(si); seg_done(si), ++si) {
            const ChunkSeg& s = sh.seg[si % kSegs];
            const bool narrow = s.it.rows <= kRows;
            const int tile = narrow ? 0 : wg, step = narrow ? 2 : 1;
            const int row = s.it.row0 + tile * kRows + r;
            const bool live = tile * kRows + r < s.it.rows;
            const bool warp_live = tile * kRows + (r & ~31) < s.it.rows;     // some row of this warp is real
            const int qi = row / g;
            const int64_t qrow = (static_cast<int64_t>(a.q_start[s.it.b]) + qi) * a.Hq + s.h * g + (row - qi * g);
            float sl = 1.0f;        // log2 units per score of this thread's row
            // This warp's 32 rows of Q, 16 lanes a row, scaled by a power of two to |q| in (1/2, 1], in K's channel
            // order. (A lane per row took 12000 .. 14000 clocks a segment, this 9000 .. 12000.)
            {
                const int chunk = lane & 15, base = s.it.row0 + tile * kRows + (r & ~31), end = s.it.row0 + s.it.rows;
                const int64_t q0 = static_cast<int64_t>(a.q_start[s.it.b]) * a.Hq + s.h * g;   // the first query's first head
                unsigned char* qt = sq_tile + tile * kOpBytes;
                int e_mine = 0;
                int row_k = base + (lane >> 4), qk = row_k / g, hk = row_k - qk * g;    // this lane's next row: query and head
#pragma unroll 1
                for (int k0 = 0; k0 < 16; k0 += 8) {
                    uint4 x[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        x[k] = row_k < end ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                                                  (q0 + static_cast<int64_t>(qk) * a.Hq + hk) * kD) + chunk)
                                           : make_uint4(0, 0, 0, 0);
                        row_k += 2;
                        hk += 2;
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (hk >= g) {
                                hk -= g;
                                ++qk;
                            }
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                        float mx = 0.0f;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mx = fmaxf(mx, fmaxf(fabsf(widen<DT>(static_cast<uint16_t>(w[i]))), fabsf(widen<DT>(static_cast<uint16_t>(w[i] >> 16)))));
#pragma unroll
                        for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
                        // 2^e above mx (from its exponent field; a zero row takes any), kept where 2^e and 2^-e are normal
                        int e = static_cast<int>(__float_as_uint(mx) >> 23) - 126;
                        e = e < -126 ? -126 : e > 126 ? 126 : e;
                        const float pre = a.scale_log2 == 0.0f ? 0.0f : copysignf(__uint_as_float(static_cast<uint32_t>(127 - e) << 23), a.scale_log2);
                        const int rk = (r & ~31) + 2 * (k0 + k) + (lane >> 4);
                        const int e_row = __shfl_sync(kFull, e, 16 * (lane & 1));   // of row 2 (k0 + k) + (lane & 1)
                        if (lane >> 1 == k0 + k) e_mine = e_row;
                        if (wg != tile) continue;      // a narrow segment's second warpgroup: the tile is the first's to fill
                        uint32_t f[4], o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            f[i] = pack_h2(widen<DT>(static_cast<uint16_t>(w[i])) * pre, widen<DT>(static_cast<uint16_t>(w[i] >> 16)) * pre);
                        if constexpr (KB == 2) {
                            // pairs (i, i + 8) of 16 channels: this lane has eight of them, its neighbour the others
                            const bool upper = chunk & 1;
                            const uint32_t g0 = __shfl_xor_sync(kFull, upper ? f[0] : f[2], 1), g1 = __shfl_xor_sync(kFull, upper ? f[1] : f[3], 1);
                            const uint32_t a0 = upper ? g0 : f[0], a1 = upper ? g1 : f[1], b0 = upper ? f[2] : g0, b1 = upper ? f[3] : g1;
                            o[0] = prmt(a0, b0, 0x5410u);
                            o[1] = prmt(a0, b0, 0x7632u);
                            o[2] = prmt(a1, b1, 0x5410u);
                            o[3] = prmt(a1, b1, 0x7632u);
                        } else {
                            o[0] = prmt(f[0], f[2], 0x5410u);   // pairs (i, i + 4) of eight channels
                            o[1] = prmt(f[0], f[2], 0x7632u);
                            o[2] = prmt(f[1], f[3], 0x5410u);
                            o[3] = prmt(f[1], f[3], 0x7632u);
                        }
                        *reinterpret_cast<uint4*>(qt + op_addr(rk, chunk)) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
                // (both warpgroups arrive, in narrow segments too: each is done with the segment before)
                if (wg == tile) proxy_fence();
                warp_arrive(smem_u32(&sh.q_full[2 * (si % kSegs) + wg]));
                __syncwarp();
                if (a.scale_log2 != 0.0f) sl = fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 + e_mine) << 23);
            }
            // tokens this row sees: [lo, pos] and [0, sinks)
            const int len = static_cast<int>(s.it.L), pos = len + qi;
            const int lo = a.window > 0 ? pos + 1 - a.window : 0;
            const int snk = a.window > 0 ? a.sinks : 0;
            const int tile_first = len + (s.it.row0 + tile * kRows) / g;   // position of the row tile's first query
            const int tile_last = len + (s.it.row0 + tile * kRows + kRows - 1) / g;

            float m = -CUDART_INF_F;         // reference maximum, log2 units
            float2 l[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};   // parts of the row's sum
            const int j0 = s.x0 + (narrow ? wg : 0);
            for (int j = j0; j < s.x1; j += step) {
                const int t0 = (j < s.it.st ? j : j + s.it.skip) * kKeys;
                const bool cut = t0 + kKeys - 1 > tile_first ||
                                 (a.window > 0 && t0 <= tile_last - a.window && t0 + kKeys > snk);
                // the row's bounds inside this tile: columns [c_lo, c_hi) and [0, c_snk)
                const int c_hi = pos + 1 - t0, c_lo = lo - t0, c_snk = snk - t0;
#pragma unroll 1
                for (int b = 0; b < 2; ++b) {
                    const uint32_t t_sb = t_s + b * kHalf, p_bar = smem_u32(&sh.p_full[2 * wg + b]);
                    ok = warp_wait(smem_u32(&sh.s_full[2 * wg + b]), ns & 1, stop);
                    if (!ok) break;
                    if (!warp_live) {     // no row to serve: its products go nowhere
                        warp_arrive(p_bar);
                        continue;
                    }
                    tc_fence_after();
                    // By 32 columns: their maximum, then their exponentials against the reference. Only where the
                    // maximum has outrun the reference by more than the lag does the reference move up, and what is
                    // there in its units (the sum, this row's output, the first columns' probabilities) is scaled
                    // down. (Rolled by halves: the roles of this kernel run different code at the same time and
                    // share the instruction cache.)
                    float x[2][32];
                    tc_ld32(x[0], t_sb);
                    tc_ld32(x[1], t_sb + 32);
                    tc_wait_ld();
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float(&y)[32] = x[q];
                        if (__builtin_expect(cut, 0)) {
                            const int c1 = kHalf * b + 32 * q;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (c1 + i >= c_hi || (c1 + i < c_lo && c1 + i >= c_snk)) y[i] = -CUDART_INF_F;
                        }
                        float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                        for (int i = 0; i < 16; ++i) mx[i & 1] = fmaxf(mx[i & 1], fmaxf(y[2 * i], y[2 * i + 1]));
                        const float top = fmaxf(mx[0], mx[1]) * sl;
                        const bool grow = m == -CUDART_INF_F ? top > m : top > m + kLag;
                        if (__builtin_expect(__any_sync(kFull, grow), 0)) {
                            const float alpha = grow ? exp2_ftz(m - top) : 1.0f;     // 0 while m is -inf
                            if (grow) m = top;
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                l[i].x *= alpha;
                                l[i].y *= alpha;
                            }
                            if (q == 1) {
                                const uint32_t alpha2 = pack_h2(alpha, alpha);
                                float u[16];
                                uint32_t v[16];
                                tc_wait_st();
                                tc_ld16(u, t_sb);
                                tc_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) v[i] = hmul2(__float_as_uint(u[i]), alpha2);
                                tc_st16(t_sb, v);
                            }
                            if (j > j0 || b > 0) {     // once the products of the halves before are complete
                                ok = warp_wait(smem_u32(&sh.o_step[2 * wg + (b ^ 1)]), (ns + b - 1) & 1, stop);
                                if (!ok) break;
                                tc_fence_after();
#pragma unroll 1
                                for (int c = 0; c < kD / 16; ++c) {
                                    float u[16];
                                    uint32_t v[16];
                                    tc_ld16(u, t_o + 16 * c);
                                    tc_wait_ld();
#pragma unroll
                                    for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(u[i] * alpha);
                                    tc_st16(t_o + 16 * c, v);
                                }
                            }
                        }
                        const float mref = m == -CUDART_INF_F ? 0.0f : m;
                        const float2 sl2 = make_float2(sl, sl), mn2 = make_float2(-mref, -mref);
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 e = fma2(make_float2(y[2 * i], y[2 * i + 1]), sl2, mn2);
                            e.x = exp2_ftz(e.x);
                            e.y = exp2_ftz(e.y);
                            l[i & 1] = add2(l[i & 1], e);
                            p[i] = pack_h2(e.x, e.y);
                        }
                        tc_st16(t_sb + 16 * q, p);   // over scores that have been read
                    }
                    if (!ok) break;
                    tc_wait_st();
                    tc_fence_before();
                    warp_arrive(p_bar);
                }
                if (!ok) break;
                ++ns;
            }
            const bool any = j0 < s.x1;      // this warpgroup had tiles
            if (any) {
                ok = ok && warp_wait(smem_u32(&sh.o_step[2 * wg + 1]), (ns - 1) & 1, stop);
                if (!ok) break;
                tc_fence_after();
            }
            float sum = (l[0].x + l[0].y) + (l[1].x + l[1].y);
            float f0 = 1.0f, f1 = 0.0f;      // factors of the two states of a narrow segment
            bool both = false;
            if (narrow && s.x1 - s.x0 > 1) {
                if (wg == 1) {
                    // hand the state over; the output columns are read from TMEM by the other warpgroup
                    sh.hand_m[r] = m;
                    sh.hand_l[r] = sum;
                    tc_fence_before();
                    warp_arrive(smem_u32(&sh.hand_full));
                    ok = warp_wait(smem_u32(&sh.hand_empty), nh & 1, stop);
                    ++nh;
                    tc_fence_after();
                    continue;
                }
                ok = warp_wait(smem_u32(&sh.hand_full), nh & 1, stop);
                if (!ok) break;
                ++nh;
                tc_fence_after();
                both = true;
                const float m1 = sh.hand_m[r], l1 = sh.hand_l[r], mt = fmaxf(m, m1);
                if (mt != -CUDART_INF_F) {
                    f0 = exp2_ftz(m - mt);
                    f1 = exp2_ftz(m1 - mt);
                }
                sum = sum * f0 + l1 * f1;
                m = mt;
            } else if (narrow && wg == 1) {
                continue;
            }
            const bool whole = s.x0 == 0 && s.x1 == s.it.nt;
            if (whole) {
                const float inv = 1.0f / sum;
                f0 *= inv;
                f1 *= inv;
            }
            float* rec = whole ? nullptr : chunk_record(a, 2 * static_cast<int64_t>(c) + (s.x0 == 0), tile);
            if (warp_live) {
#pragma unroll 1
                for (int q = 0; q < kD / 32; ++q) {
                    float x[32], y[32];
                    tc_ld32(x, t_o + 32 * q);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) y[(i & 16) + span_channel<VB>(i & 15)] = x[i] * f0;
                    if (both) {
                        tc_ld32(x, t_o + kD + 32 * q);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            float& z = y[(i & 16) + span_channel<VB>(i & 15)];
                            z = fmaf(x[i], f1, z);
                        }
                    }
                    if (live && whole) {
                        store32<DT>(a.out, qrow, 32 * q, y);
                    } else if (live) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            reinterpret_cast<float4*>(rec)[(8 * q + i) * kRows + r] =
                                make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                    }
                    __syncwarp();
                }
            }
            if (both) {
                tc_fence_before();
                warp_arrive(smem_u32(&sh.hand_empty));
            }
            if (!whole && live) {
                rec[kRows * kD + r] = m;
                rec[kRows * kD + kRows + r] = sum;
            }
            if (!whole && s.x0 == 0 && tid == 0) {
                ChunkInfo f;
                f.b = s.it.b;
                f.row0 = s.it.row0;
                f.rows = s.it.rows;
                f.h = s.h;
                f.nseg = s.nseg;
                a.info[c] = f;
            }
            tc_fence_before();
        }
    } else if (warp < 16) {
        // ------------------------------------------------ keys (warps 8-11) and values (12-15)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOperandRegs));
        auto operands = [&](auto values) {
            constexpr bool VALUES = decltype(values)::value;
            constexpr int BITS = VALUES ? VB : KB;
            // warps 0 and 1 of the group take the first two subtiles of a tile, 2 and 3 the others; each warp has
            // half of the spans
            const int half = (warp >> 1) & 1, row_lo = lane & 7, span = (lane >> 3) + 4 * (warp & 1);
            uint64_t* full = VALUES ? sh.v_full : sh.k_full;
            uint64_t* empty = VALUES ? sh.v_empty : sh.k_empty;
            unsigned char* tiles = VALUES ? sv_tile : sk_tile;
            constexpr bool SPLIT = LO && !VALUES;      // a stage is half a tile, this warp pair's own
            const uint32_t a0 = SPLIT ? key_addr<LO>(row_lo, 2 * span) : op_addr(row_lo, 2 * span);
            const uint32_t a1 = SPLIT ? key_addr<LO>(row_lo, 2 * span + 1) : op_addr(row_lo, 2 * span + 1);
            auto stage = [&](uint32_t n) -> uint32_t { return SPLIT ? half : n % kKvStages; };
            auto use_of = [&](uint32_t n) -> uint32_t { return SPLIT ? n : n / kKvStages; };
            auto full_of = [&](uint32_t n) { return smem_u32(&full[SPLIT ? 2 * half + (n & 1) : n % kKvStages]); };
            auto place = [&](uint32_t st) { return tiles + st * kOpBytes + (SPLIT ? 0 : half * (2 * kTile * 128)); };
            // a lane's row of stored values to its two chunks; the rest of a stored f16 key is zero
            auto put = [&](unsigned char* to, const uint32_t (&o)[8]) {
                *reinterpret_cast<uint4*>(to + a0) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4*>(to + a1) = make_uint4(o[4], o[5], o[6], o[7]);
                if constexpr (SPLIT) {
                    *reinterpret_cast<uint4*>(to + a0 + KeyStage<LO>::kRest) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(to + a1 + KeyStage<LO>::kRest) = make_uint4(0, 0, 0, 0);
                }
            };
            const int gsh = a.G == 64 ? 6 : 5;
            uint32_t n = 0, raw0 = 0, raw_par = 0;    // tiles so far; the tile's first raw stage and its parity
            for (uint32_t si = 0; ok && seg_next(si); seg_done(si), ++si) {
                const ChunkSeg& s = sh.seg[si % kSegs];
                const kivi_seq& sq = a.seqs[s.it.b];
                const int np = static_cast<int>(n_packed(s.it.L, a.R, a.G));
                ChunkStored src;
                src.L = static_cast<int>(s.it.L);
                src.end = src.L + s.it.n;
                src.ring = a.R + a.G;
                src.res = static_cast<const uint16_t*>(VALUES ? sq.v_res : sq.k_res) + static_cast<int64_t>(s.h) * src.ring * kD;
                src.fresh = static_cast<const uint16_t*>(VALUES ? a.v_new[s.it.b] : a.k_new[s.it.b]) +
                            static_cast<int64_t>(s.h) * s.it.n * kD;
                const int x0 = s.x0, x1 = s.x1, lst = s.it.st, skip = s.it.skip;
                if (np <= (x0 < lst ? x0 : x0 + skip) * kKeys) {
                    // stored tokens only (a first chunk): as each row is stored, the row that follows it in the
                    // next subtile is loaded in its place
                    uint32_t x[4][8];
                    load_stored(src, (x0 < lst ? x0 : x0 + skip) * kKeys + 2 * half * kTile, row_lo, span, x);
                    for (int j = x0; j < x1; ++j, ++n) {
                        const uint32_t st = stage(n), use = use_of(n);
                        const int t0 = (j < lst ? j : j + skip) * kKeys + 2 * half * kTile;
                        const int t1 = (j + 1 < lst ? j + 1 : j + 1 + skip) * kKeys + 2 * half * kTile;   // in the next tile
                        if (use > 0) ok = warp_wait(smem_u32(&empty[st]), (use - 1) & 1, stop);
                        if (!ok) break;
                        unsigned char* dst = place(st);
#pragma unroll 1
                        for (int i = 0; i < 2; ++i, dst += kTile * 128) {
                            const int next = i == 0 ? t0 + kTile : j + 1 < x1 ? t1 : src.end;   // (rows from end on are zeros)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                uint32_t o[8];
                                pair_stored<BITS, DT>(x[k], o);
                                put(dst + 1024 * k, o);
                                load_row(src, next + row_lo + 8 * k, span, x[k]);
                            }
                        }
                        proxy_fence();
                        warp_arrive(full_of(n));
                    }
                    continue;
                }
                for (int j = x0; j < x1; ++j, ++n) {
                    const uint32_t st = stage(n), use = use_of(n);
                    const int t0 = (j < lst ? j : j + skip) * kKeys;
                    const int packed = np <= t0 ? 0 : np - t0 >= kKeys ? kKeys / kTile : (np - t0) / kTile;   // subtiles
                    auto wait_empty = [&]() {
                        if (use > 0) ok = warp_wait(smem_u32(&empty[st]), (use - 1) & 1, stop);
                    };
                    unsigned char* dst = place(st);
                    auto stored = [&](const uint32_t (&x)[4][8], unsigned char* to) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t o[8];
                            pair_stored<BITS, DT>(x[k], o);
                            put(to + 1024 * k, o);
                        }
                    };
                    if (2 * half < packed) {
                        const bool wrap = raw0 + half >= Raw::kStages;
                        const uint32_t slot = wrap ? raw0 + half - Raw::kStages : raw0 + half;
                        // the operand stage first: that it is free says that the tile before the last is done with, so
                        // the raw stage's use before this one is over and its parity tells (a warp whose half had no
                        // packed tokens for some tiles has not followed the stage's phases)
                        wait_empty();
                        if (!ok) break;
                        ok = warp_wait(smem_u32(&sh.raw_full[slot]), raw_par ^ wrap, stop);
                        if (!ok) break;
                        const unsigned char* from = raw_ring + slot * Raw::kBytes;
                        const int subs = packed - 2 * half < 2 ? 1 : 2;
#pragma unroll 1
                        for (int i = 0; i < subs; ++i) {
                            fill_packed<KB, VB, VALUES, LO>(from, gsh, row_lo, span, dst, a0, a1);
                            from += Raw::kSub;
                            dst += kTile * 128;
                        }
                        warp_arrive(smem_u32(&sh.raw_empty[slot]));
                        if (subs < 2) {     // the second subtile is stored tokens
                            uint32_t x[4][8];
                            load_stored(src, t0 + (2 * half + 1) * kTile, row_lo, span, x);
                            stored(x, dst);
                        }
                    } else {
                        uint32_t x[4][8];
                        load_stored(src, t0 + 2 * half * kTile, row_lo, span, x);
                        wait_empty();
                        if (!ok) break;
                        stored(x, dst);
                        load_stored(src, t0 + (2 * half + 1) * kTile, row_lo, span, x);
                        stored(x, dst + kTile * 128);
                    }
                    raw0 += (packed + 1) / 2;
                    if (raw0 >= Raw::kStages) {
                        raw0 -= Raw::kStages;
                        raw_par ^= 1;
                    }
                    proxy_fence();
                    warp_arrive(full_of(n));
                }
            }
        };
        if (warp < 12) operands(std::integral_constant<bool, false>{});
        else operands(std::integral_constant<bool, true>{});
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == 16 || warp == 19) {
            // ------------------------------------------------ tensor-core issue: warp 16 for softmax warpgroup 0, 19 for 1.
            // (The tensor core takes few products ahead, so a single issuing warp left it idle while it waited.) The
            // whole warp walks, one lane issues.
            const uint32_t t = warp == 16 ? 0 : 1;
            uint32_t n = 0, np = 0;   // key tiles and this warpgroup's probability tiles so far
            const uint32_t kb0 = smem_u32(sk_tile), vb0 = smem_u32(sv_tile), qb0 = smem_u32(sq_tile);
            const uint32_t d_s = __shfl_sync(kFull, tmem + t * kKeys, 0), d_o = __shfl_sync(kFull, tmem + 2 * kKeys + t * kD, 0);
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                ok = warp_wait(smem_u32(bar), parity, stop);
                return ok;
            };
            for (uint32_t si = 0; ok && seg_next(si); seg_done(si), ++si) {
                // Wide segments: this warpgroup (its row tile) takes every key tile; narrow ones: the warpgroups take
                // them in turn, and the one that takes a tile gives its stage back for both. Scores run one tile ahead:
                // S is free for the next scores after the products of the tile before.
                const ChunkSeg& s = sh.seg[si % kSegs];
                const uint32_t narrow = s.it.rows <= kRows, cnt = s.x1 - s.x0, step = 1 + narrow;
                // (Both warps wait for both warpgroups, in narrow segments too: then every key and value tile before is
                // done with, which the parities of their barriers rest on. A barrier for each slot of the ring, whose
                // slots are used again once every warp is done with them, so nobody can be two phases behind.)
                if (!wait(&sh.q_full[2 * (si % kSegs)], (si / kSegs) & 1)) break;
                if (!wait(&sh.q_full[2 * (si % kSegs) + 1], (si / kSegs) & 1)) break;
                const uint32_t q = __shfl_sync(kFull, desc_lo(qb0 + (narrow ? 0 : t) * kOpBytes, 16), 0);
                // halves of this warpgroup's tiles: half i is half i & 1 of its tile i >> 1, tile (i >> 1) step + narrow t
                // of the segment; scores run two halves ahead
                const uint32_t halves = 2 * ((cnt + narrow - narrow * t) / step);
#pragma unroll 1
                for (uint32_t i = 0; i < halves + 2; ++i) {
                    const uint32_t b = i & 1;
                    if (i >= 2) {          // products of half i - 2
                        const uint32_t u = n + ((i - 2) >> 1) * step + narrow * t, st = u % kKvStages;
                        if (!wait(&sh.v_full[st], (u / kKvStages) & 1) || !wait(&sh.p_full[2 * t + b], (np >> 1) & 1)) break;
                        ++np;
                        tc_fence_after();
                        // (broadcast, so that the compiler keeps the operands in uniform registers)
                        const uint32_t v = __shfl_sync(kFull, desc_lo(vb0 + st * kOpBytes + b * (kHalf * 128), kRows * 128), 0);
                        const uint32_t p = __shfl_sync(kFull, d_s + b * kHalf, 0), acc = __shfl_sync(kFull, i > 2 ? 1u : 0u, 0);
                        if (elect_one()) {
                            mma_ts(d_o, p, v, kIdescPV, acc);
#pragma unroll
                            for (uint32_t k = 1; k < kHalf / 16; ++k) mma_ts(d_o, p + 8 * k, v + k * (2048 >> 4), kIdescPV, 1);
                            tc_commit(smem_u32(&sh.o_step[2 * t + b]));
                            if (b) {
                                tc_commit(smem_u32(&sh.v_empty[st]));
                                if (narrow) tc_commit(smem_u32(&sh.v_empty[st]));
                            }
                        }
                    }
                    if (i < halves) {      // scores of half i
                        const uint32_t u = n + (i >> 1) * step + narrow * t, st = LO ? b : u % kKvStages;
                        if (!wait(&sh.k_full[LO ? 2 * b + (u & 1) : st], (u / 2) & 1)) break;
                        tc_fence_after();
                        const uint32_t k = __shfl_sync(kFull, desc_lo(kb0 + st * kOpBytes + (LO ? 0 : b * (kHalf * 128)), 16), 0);
                        const uint32_t d = __shfl_sync(kFull, d_s + b * kHalf, 0);
                        if (elect_one()) {
#pragma unroll
                            for (uint32_t c = 0; c < kD / 16; ++c) {
                                const uint32_t off = (c >> 2) * ((kRows * 128) >> 4) + (c & 3) * 2;
                                const uint32_t koff = (c >> 2) * (KeyStage<LO>::kBlock >> 4) + (c & 3) * 2;
                                mma_ss(d, q + off, k + koff, kIdescQK, c > 0);
                                if constexpr (LO) mma_ss(d, q + off, k + koff + (KeyStage<LO>::kRest >> 4), kIdescQK, 1);
                            }
                            tc_commit(smem_u32(&sh.s_full[2 * t + b]));
                            if (LO || b) {
                                tc_commit(smem_u32(&sh.k_empty[st]));
                                if (narrow) tc_commit(smem_u32(&sh.k_empty[st]));
                            }
                        }
                    }
                    __syncwarp();
                }
                n += cnt;
            }
        } else if (warp == 17) {
            // -------------------------------------------- raw packed tokens, 16 bytes a lane and copy. (Bulk copies of
            // the six buffers' runs, 256 to 1024 bytes each, made the kernel 3 % slower where memory counts: 64 x 32768
            // tokens, 4 new ones each.)
            uint32_t slot = 0, par = 0;
            bool full_turn = false;
            constexpr uint32_t kKcb = kTile * kD * KB / 8, kVcb = kTile * kD * VB / 8;    // codes of a subtile
            const int tpg = a.G / kTile;
            const uint32_t vmeta = kTile * (kD / a.G) * 2, vlanes = vmeta / 16;           // value scales (or zeros) of a subtile
            for (uint32_t si = 0; ok && seg_next(si); seg_done(si), ++si) {
                const ChunkSeg& s = sh.seg[si % kSegs];
                const kivi_seq& sq = a.seqs[s.it.b];
                // this lane's place in each buffer: codes at 16 lane, scales and zeros by half warps
                const unsigned char* kc = sq.k_codes + 16 * lane;
                const unsigned char* vc = sq.v_codes + 16 * lane;
                const unsigned char* km = reinterpret_cast<const unsigned char*>(lane < 16 ? sq.k_scale : sq.k_zero) + 16 * (lane & 15);
                const unsigned char* vm = reinterpret_cast<const unsigned char*>((lane & vlanes) == 0 ? sq.v_scale : sq.v_zero) +
                                          16 * (lane & (vlanes - 1));
                const bool paged = seq_paged(sq);
                const int32_t* table = sq.block_table;
                const int h = s.h, x1 = s.x1, st = s.it.st, skip = s.it.skip;
                const int tiles = static_cast<int>(n_packed(s.it.L, a.R, a.G) / kTile);   // packed subtiles
                const int64_t head = static_cast<int64_t>(h) * (sq.cap_tokens / a.G);     // contiguous: first group of the head
                // pages ahead: lane i holds the page of group page0 + i
                int page0 = -64, pages = 0;
                for (int j = s.x0; ok && j < x1; ++j) {
                    const int t0 = (j < st ? j : j + skip) * (kKeys / kTile);
                    for (int t = t0; t < t0 + kKeys / kTile && t < tiles; t += 2) {
                        if (full_turn) ok = warp_wait(smem_u32(&sh.raw_empty[slot]), par ^ 1, stop);
                        if (!ok) break;
                        unsigned char* dst = raw_ring + slot * Raw::kBytes;
                        const int subs = tiles - t < 2 ? 1 : 2;
#pragma unroll 1
                        for (int i = 0; i < subs; ++i, dst += Raw::kSub) {
                            const int group = tpg == 1 ? t + i : t >> 1;
                            int64_t at = head + group;                // the group's record
                            if (paged) {
                                if (group < page0 || group >= page0 + 32) {
                                    page0 = group;
                                    pages = (page0 + lane) * tpg < tiles ? __ldg(table + page0 + lane) : 0;
                                }
                                at = static_cast<int64_t>(__shfl_sync(kFull, pages, group - page0)) * a.H + h;
                            }
                            const int64_t rt = at * tpg + (tpg == 1 ? 0 : (t + i) & 1);   // the subtile's
#pragma unroll
                            for (uint32_t k = 0; k < kKcb; k += 512) cp_async16(dst + Raw::kKc + k + 16 * lane, kc + rt * kKcb + k);
                            cp_async16(dst + (lane < 16 ? Raw::kKs : Raw::kKz) + 16 * (lane & 15), km + at * (kD * 2));
#pragma unroll
                            for (uint32_t k = 0; k < kVcb; k += 512) cp_async16(dst + Raw::kVc + k + 16 * lane, vc + rt * kVcb + k);
                            if (lane < 2 * vlanes)
                                cp_async16(dst + ((lane & vlanes) == 0 ? Raw::kVs : Raw::kVz) + 16 * (lane & (vlanes - 1)), vm + rt * vmeta);
                        }
                        // this lane's arrival, once its copies have landed
                        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sh.raw_full[slot])) : "memory");
                        if (++slot == Raw::kStages) {
                            slot = 0;
                            par ^= 1;
                            full_turn = true;
                        }
                    }
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");   // nothing in flight when the CTA ends
        } else if (warp == 18 && lane == 0) {
            // -------------------------------------------- the walk over this CTA's share; x1 = 0 ends it
            ChunkWalk w;
            w.lo = sh.lo; w.hi = sh.hi; w.pos = sh.pos; w.idx = sh.idx; w.U = sh.U; w.C = sh.C; w.h = sh.h;
            bool more = true;
            for (uint32_t i = 0; more; ++i) {
                ChunkSeg s;
                more = chunk_next(a, w, s);
                if (!more) s.x0 = s.x1 = 0;
                if (i >= kSegs && !lane_wait(smem_u32(&sh.seg_empty[i % kSegs]), (i / kSegs - 1) & 1, stop)) break;
                sh.seg[i % kSegs] = s;
                mbar_arrive(smem_u32(&sh.seg_full[i % kSegs]));
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*stop != 0) {
        // a wait ran out: let the products in flight finish (with a limit) before the TMEM goes
        if (tid == 0) set_status(a.status, KIVI_ERR_CUDA);
        if ((warp == 16 || warp == 19) && lane == 0) {
            const uint32_t bar = smem_u32(&sh.warp_sum[warp]);
            mbar_init(bar, 1);
            tc_commit(bar);
            const long long t0 = clock64();
            while (!mbar_try(bar, 0) && clock64() - t0 < 4000000000LL) {}
        }
        __syncthreads();
    }
    if (warp == 16) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// Joins the records of the row tile pair that CTA blockIdx.x of the chunk kernel began and others
// went on with: blockIdx.y takes 32 of its rows. A record's max is -inf where its tiles
// showed the row nothing.
constexpr int kMergeRows = 32;
template <int DT>
__global__ void __launch_bounds__(256) chunk_merge_kernel(ChunkArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x;
    const ChunkInfo f = a.info[c];
    const int r0 = blockIdx.y * kMergeRows;
    if (f.nseg < 2 || r0 >= f.rows) return;
    const int g = a.Hq / a.H;
    for (int i = threadIdx.x; i < kMergeRows * (kD / 4); i += 256) {
        const int r = r0 + (i & (kMergeRows - 1)), quad = i / kMergeRows;
        if (r >= f.rows) continue;
        const int tile = r / kRows, rt = r % kRows;
        float m = -CUDART_INF_F, l = 0.0f;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int k = 0; k < f.nseg; ++k) {
            const float* rec = chunk_record(a, 2 * static_cast<int64_t>(c + k) + (k == 0), tile);
            const float mk = __ldcg(rec + kRows * kD + rt), lk = __ldcg(rec + kRows * kD + kRows + rt);
            const float4 xk = __ldcg(reinterpret_cast<const float4*>(rec) + quad * kRows + rt);
            if (mk == -CUDART_INF_F) continue;
            const float mn = fmaxf(m, mk), s0 = exp2f(m - mn), s1 = exp2f(mk - mn);
            l = l * s0 + lk * s1;
            x.x = x.x * s0 + xk.x * s1;
            x.y = x.y * s0 + xk.y * s1;
            x.z = x.z * s0 + xk.z * s1;
            x.w = x.w * s0 + xk.w * s1;
            m = mn;
        }
        const float inv = 1.0f / l;
        const int row = f.row0 + r, qi = row / g;
        const int64_t qrow = (static_cast<int64_t>(a.q_start[f.b]) + qi) * a.Hq + f.h * g + (row - qi * g);
        uint32_t w0, w1;
        if constexpr (DT == KIVI_F16) {
            w0 = pack_h2(x.x * inv, x.y * inv);
            w1 = pack_h2(x.z * inv, x.w * inv);
        } else {
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w0) : "f"(x.y * inv), "f"(x.x * inv));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w1) : "f"(x.w * inv), "f"(x.z * inv));
        }
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + qrow * kD + 4 * quad) = make_uint2(w0, w1);
    }
}

// SMs of the current device, at most kChunkMaxCtas (one CTA each). The first launch of an
// instantiation on a device raises its shared memory limit.
template <typename K>
int chunk_ctas(K kernel, int smem, std::atomic<int>* cache) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    const int have = cache[dev].load(std::memory_order_relaxed);
    if (have > 0) return have;
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    n = n > kChunkMaxCtas ? kChunkMaxCtas : n;
    cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

template <int KB, int VB, int DT>
cudaError_t launch_chunk_dt(ChunkArgs a, cudaStream_t stream) {
    static std::atomic<int> ctas[kMaxDevices];
    a.ctas = chunk_ctas(chunk_kernel<KB, VB, DT>, chunk_smem<KB, VB>(), ctas);
    if (a.ctas <= 0) return cudaErrorInvalidValue;
    chunk_kernel<KB, VB, DT><<<a.ctas, kChunkThreads, chunk_smem<KB, VB>(), stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.ctas, a.rec_tiles * kRows / kMergeRows);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, chunk_merge_kernel<DT>, a);
}

template <int KB, int VB>
cudaError_t launch_chunk_kv(const ChunkArgs& a, cudaStream_t stream) {
    return a.dtype == KIVI_F16 ? launch_chunk_dt<KB, VB, KIVI_F16>(a, stream)
                               : launch_chunk_dt<KB, VB, KIVI_BF16>(a, stream);
}

}  // namespace
}  // namespace kivi
