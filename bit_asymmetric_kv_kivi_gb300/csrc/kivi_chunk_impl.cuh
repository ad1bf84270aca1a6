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
//   warp 16          issues tcgen05.mma (kind::f16, M = N = 128): S = Q K^T from shared memory, O += P V
//                    with P from TMEM
// TMEM: S0, S1 (128 columns each, P over the first 64 of S), O0, O1. While the softmax of one row
// tile runs, the tensor core works on the other.
//
// Rounding: operands are f16 whatever the storage type. A dequantized token is rounded once,
// fma(c, s, z) to 11 bits, as an f16 cache would hold it; stored bf16 tokens with |x| <= 65504 are
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
#pragma once
#include "kivi_decode_impl.cuh"

namespace kivi {
namespace {

constexpr int kChunkSoftmaxWarps = 8;
constexpr int kChunkThreads = 17 * 32;
constexpr int kRows = 128;                // rows of a row tile
constexpr int kKeys = 128;                // tokens of a key tile
constexpr int kOpBytes = kRows * kD * 2;  // one 128 x 128 f16 operand tile
constexpr int kKvStages = 2;
constexpr int kUnitOverhead = 3;          // units charged per (row tile pair, kv head)
constexpr int kMinChunkUnits = 4;
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
// Waits for a phase; gives up (and tells the other roles) after about two seconds, so that no
// mistake in the schedule can hang the device.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* stop) {
    if (mbar_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try(bar, parity)) {
        if (*stop != 0) return false;
        if (clock64() - t0 > 4000000000LL) {
            *stop = 1;
            return false;
        }
    }
    return true;
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

// Operand tiles in shared memory: two blocks of 64 channels, each 128 rows of 128 bytes with the
// 16-byte chunks of a row XORed by its low three bits (the 128-byte swizzle).
__device__ __forceinline__ uint32_t op_addr(int row, int chunk) {   // chunk of 8 channels, 0 .. 15
    return static_cast<uint32_t>((chunk >> 3) * (kRows * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}
// Shared-memory descriptor, 128-byte swizzle. K-major (Q, K): rows of 8 every 1024 bytes. MN-major
// (V: channels contiguous): 64-channel blocks every kRows * 128 bytes, groups of 8 tokens every 1024.
__device__ __forceinline__ uint64_t op_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
           (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// f32 accumulator, f16 operands, N = M = 128; bit 16: B is MN-major
constexpr uint32_t kIdescQK = (1u << 4) | ((kKeys / 8) << 17) | ((kRows / 16) << 24);
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | ((kD / 8) << 17) | ((kRows / 16) << 24);

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc)) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc)) : "memory");
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

__device__ __forceinline__ ChunkItem chunk_item(const ChunkArgs& a, int64_t idx) {
    ChunkItem it;
    it.b = static_cast<int>(idx / a.pairs);
    const int64_t row0 = (idx - static_cast<int64_t>(it.b) * a.pairs) * (2 * kRows);
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

// A CTA's share of the row of units. Every role walks it by itself: next() yields the segments
// (a row tile pair of one kv head, listed key tiles [x0, x1)).
struct ChunkWalk {
    int64_t lo, hi, pos, idx;   // this CTA's units, first unit of item idx
    int64_t U;
    int C, h;
};
struct ChunkSeg {
    ChunkItem it;
    int h, x0, x1;
    int nseg;   // CTAs that share it
};

__device__ __forceinline__ bool chunk_next(const ChunkArgs& a, ChunkWalk& w, ChunkSeg& s) {
    const int64_t items = static_cast<int64_t>(a.nseq) * a.pairs;
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

struct ChunkShared {
    uint64_t k_full[kKvStages], k_empty[kKvStages], v_full[kKvStages], v_empty[kKvStages];
    uint64_t q_full[2], s_full[2], p_full[2], o_done[2];
    int64_t warp_sum[kChunkThreads / 32];
    int64_t lo, hi, pos, idx, U;
    int C, h;
    uint32_t tmem;
    int stop;
};
constexpr int kChunkSmem = 2 * kOpBytes + 2 * kKvStages * kOpBytes + 1024 + static_cast<int>(sizeof(ChunkShared));

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

// Where a sequence's tokens of one kv head lie.
struct ChunkSrc {
    const kivi_seq* sq;
    const uint16_t *res, *fresh;   // this head's ring and new tokens (keys or values)
    int64_t L, np, end;            // cached, packed, cached and new tokens
    int ring;
};

// One thread's part of a key (VALUES false) or value tile: rows lo8 + 8 rh + 16 k of each 32-token
// subtile, one 16-channel span, so that the eight lanes of a store phase hit eight rows
// (distinct banks under the swizzle).
template <int BITS, int DT, bool VALUES>
__device__ __forceinline__ void fill_tile(const ChunkArgs& a, const ChunkSrc& s, int h, int64_t t0, unsigned char* dst,
                                          int p) {
    const int row_lo = (p & 7) + 8 * (p >> 6), span = (p >> 3) & 7;
    constexpr int kRowBytes = kD * BITS / 8, kSpanBytes = 2 * BITS;
#pragma unroll 1
    for (int sub = 0; sub < kKeys / kTile; ++sub) {
        const int64_t tb = t0 + sub * kTile;
        uint32_t o[2][8];
        if (tb < s.np) {
            const GroupAddr g = tile_addr(*s.sq, a.H, h, tb / kTile, kD, a.kb, a.vb, a.G);
            uint32_t sc[8], zr[8];
            if constexpr (!VALUES) {
                uint32_t w[8];
                load8(w, g.ks + span * 16);
                pair_words<BITS>(w, sc);
                load8(w, g.kz + span * 16);
                pair_words<BITS>(w, zr);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int row = row_lo + 16 * k;
                const unsigned char* code = (VALUES ? g.vc : g.kc) + row * kRowBytes + span * kSpanBytes;
                uint32_t w[BITS / 2];
                if constexpr (BITS == 2) {
                    w[0] = __ldg(reinterpret_cast<const uint32_t*>(code));
                } else {
                    const uint2 x = __ldg(reinterpret_cast<const uint2*>(code));
                    w[0] = x.x;
                    w[1] = x.y;
                }
                uint32_t c[8];
                pair_codes<BITS>(w, c);
                if constexpr (VALUES) {
                    const int ng = kD / a.G, gr = span * 16 / a.G;
                    const uint32_t s1 = __ldg(g.vs + row * ng + gr), z1 = __ldg(g.vz + row * ng + gr);
                    const uint32_t s2 = prmt(s1, s1, 0x1010u), z2 = prmt(z1, z1, 0x1010u);
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[k][i] = hfma2(c[i], s2, z2);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[k][i] = hfma2(c[i], sc[i], zr[i]);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int64_t t = tb + row_lo + 16 * k;
                uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};   // rows behind the last token: zeros
                if (t < s.L) load8(w, s.res + (t % s.ring) * kD + span * 16);
                else if (t < s.end) load8(w, s.fresh + (t - s.L) * kD + span * 16);
                pair_stored<BITS, DT>(w, o[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int row = sub * kTile + row_lo + 16 * k;
            *reinterpret_cast<uint4*>(dst + op_addr(row, 2 * span)) = make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
            *reinterpret_cast<uint4*>(dst + op_addr(row, 2 * span + 1)) = make_uint4(o[k][4], o[k][5], o[k][6], o[k][7]);
        }
    }
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
    ChunkShared& sh = *reinterpret_cast<ChunkShared*>(sv_tile + kKvStages * kOpBytes);
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
            mbar_init(smem_u32(&sh.k_full[i]), 128);
            mbar_init(smem_u32(&sh.k_empty[i]), 1);
            mbar_init(smem_u32(&sh.v_full[i]), 128);
            mbar_init(smem_u32(&sh.v_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.q_full[i]), 128);
            mbar_init(smem_u32(&sh.s_full[i]), 1);
            mbar_init(smem_u32(&sh.p_full[i]), 128);
            mbar_init(smem_u32(&sh.o_done[i]), 1);
        }
        sh.stop = 0;
        sh.idx = INT64_MAX;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 16) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }

    // units of each thread's run of items, their exclusive prefix and the total
    const int64_t items = static_cast<int64_t>(a.nseq) * a.pairs;
    const int64_t per = (items + kChunkThreads - 1) / kChunkThreads;
    const int64_t i0 = tid * per < items ? tid * per : items, i1 = i0 + per < items ? i0 + per : items;
    int64_t mine = 0;
    for (int64_t i = i0; i < i1; ++i) mine += item_units(chunk_item(a, i)) * a.H;
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
            for (int64_t i = i0; i < i1; ++i) {
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
    ChunkWalk w;
    w.lo = sh.lo; w.hi = sh.hi; w.pos = sh.pos; w.idx = sh.idx; w.U = sh.U; w.C = sh.C; w.h = sh.h;
    ChunkSeg s;
    const uint32_t tmem = sh.tmem;

    if (warp < kChunkSoftmaxWarps) {
        // ------------------------------------------------ softmax of one row tile
        const int tile = warp >> 2, r = tid & 127;
        const uint32_t lane_off = static_cast<uint32_t>(warp & 3) << 21;     // this warp's 32 TMEM lanes
        const uint32_t t_s = tmem + lane_off + tile * kKeys, t_o = tmem + lane_off + 2 * kKeys + tile * kD;
        unsigned char* qt = sq_tile + tile * kOpBytes;
        uint32_t ns = 0, nq = 0;    // score tiles and segments so far
        bool ok = true;
        while (ok && chunk_next(a, w, s)) {
            if (tile * kRows >= s.it.rows) continue;   // this row tile is empty
            const int row = s.it.row0 + tile * kRows + r;
            const bool live = tile * kRows + r < s.it.rows;
            const int qi = row / g;
            const int64_t qrow = (static_cast<int64_t>(a.q_start[s.it.b]) + qi) * a.Hq + s.h * g + (row - qi * g);
            float sl;                                    // log2 units per score
            {
                // the row of Q, scaled by a power of two to |q| in (1/2, 1], in K's channel order
                const uint16_t* q = static_cast<const uint16_t*>(a.q) + qrow * kD;
                float mx = 0.0f;
#pragma unroll 2
                for (int sp = 0; sp < 8; ++sp) {
                    uint32_t x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                    if (live) load8(x, q + sp * 16);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        mx = fmaxf(mx, fmaxf(fabsf(widen<DT>(static_cast<uint16_t>(x[i]))),
                                             fabsf(widen<DT>(static_cast<uint16_t>(x[i] >> 16)))));
                }
                int e = 0;
                if (mx > 0.0f && a.scale_log2 != 0.0f) frexpf(mx, &e);
                const float pre = a.scale_log2 == 0.0f ? 0.0f : copysignf(ldexpf(1.0f, -e), a.scale_log2);
                sl = a.scale_log2 == 0.0f ? 1.0f : ldexpf(fabsf(a.scale_log2), e);
#pragma unroll 2
                for (int sp = 0; sp < 8; ++sp) {
                    uint32_t x[8] = {0, 0, 0, 0, 0, 0, 0, 0}, o[8];
                    if (live) load8(x, q + sp * 16);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int c0 = span_channel<KB>(2 * i), c1 = span_channel<KB>(2 * i + 1);
                        const float x0 = widen<DT>(static_cast<uint16_t>((c0 & 1) ? x[c0 >> 1] >> 16 : x[c0 >> 1]));
                        const float x1 = widen<DT>(static_cast<uint16_t>((c1 & 1) ? x[c1 >> 1] >> 16 : x[c1 >> 1]));
                        o[i] = pack_h2(x0 * pre, x1 * pre);
                    }
                    *reinterpret_cast<uint4*>(qt + op_addr(r, 2 * sp)) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4*>(qt + op_addr(r, 2 * sp + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
                }
                proxy_fence();
                mbar_arrive(smem_u32(&sh.q_full[tile]));
            }
            // tokens this row sees: [lo, pos] and [0, sinks)
            const int64_t pos = s.it.L + qi;
            const int64_t lo = a.window > 0 ? pos + 1 - a.window : 0;
            const int64_t snk = a.window > 0 ? a.sinks : 0;
            const int64_t tile_first = s.it.L + (s.it.row0 + tile * kRows) / g;   // position of the row tile's first query
            const int64_t tile_last = s.it.L + (s.it.row0 + tile * kRows + kRows - 1) / g;

            float m = -CUDART_INF_F, l = 0.0f;
            for (int j = s.x0; j < s.x1; ++j) {
                ok = __all_sync(kFull, mbar_wait(smem_u32(&sh.s_full[tile]), ns & 1, stop));
                if (!ok) break;
                ++ns;
                tc_fence_after();
                const int64_t t0 = static_cast<int64_t>(j < s.it.st ? j : j + s.it.skip) * kKeys;
                const bool cut = t0 + kKeys - 1 > tile_first ||
                                 (a.window > 0 && t0 <= tile_last - a.window && t0 + kKeys > a.sinks);
                // the row's bounds inside this tile: columns [c_lo, c_hi) and [0, c_snk)
                const int c_hi = static_cast<int>(pos + 1 - t0 < kKeys ? pos + 1 - t0 : kKeys);
                const int c_lo = static_cast<int>(lo - t0 > 0 ? (lo - t0 < kKeys ? lo - t0 : kKeys) : 0);
                const int c_snk = static_cast<int>(snk - t0 > 0 ? (snk - t0 < kKeys ? snk - t0 : kKeys) : 0);
                auto mask = [&](float (&x)[32], int c0) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c0 + i >= c_hi || (c0 + i < c_lo && c0 + i >= c_snk)) x[i] = -CUDART_INF_F;
                };
                float mx = -CUDART_INF_F;
#pragma unroll
                for (int q = 0; q < kKeys / 32; ++q) {
                    float x[32];
                    tc_ld32(x, t_s + 32 * q);
                    tc_wait_ld();
                    if (cut) mask(x, 32 * q);
#pragma unroll
                    for (int i = 0; i < 32; ++i) mx = fmaxf(mx, x[i]);
                }
                mx *= sl;
                const bool grow = mx > m + kLag || (m == -CUDART_INF_F && mx > m);
                if (__any_sync(kFull, grow)) {
                    const float mn = grow ? mx : m;
                    const float alpha = grow ? exp2_ftz(m - mn) : 1.0f;     // 0 while m is -inf
                    l *= alpha;
                    m = mn;
                    if (j > s.x0) {     // the products of the tiles before are complete (they precede these scores)
#pragma unroll 1
                        for (int q = 0; q < kD / 32; ++q) {
                            float x[32];
                            tc_ld32(x, t_o + 32 * q);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] *= alpha;
                            tc_st32(t_o + 32 * q, x);
                        }
                        tc_wait_st();
                    }
                }
                const float mref = m == -CUDART_INF_F ? 0.0f : m;
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int q = 0; q < kKeys / 32; ++q) {
                    float x[32];
                    tc_ld32(x, t_s + 32 * q);
                    tc_wait_ld();
                    if (cut) mask(x, 32 * q);
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float p0 = exp2_ftz(fmaf(x[2 * i], sl, -mref)), p1 = exp2_ftz(fmaf(x[2 * i + 1], sl, -mref));
                        sum[i & 3] += p0 + p1;
                        p[i] = pack_h2(p0, p1);
                    }
                    tc_st16(t_s + 16 * q, p);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tc_wait_st();
                tc_fence_before();
                mbar_arrive(smem_u32(&sh.p_full[tile]));
            }
            ok = ok && __all_sync(kFull, mbar_wait(smem_u32(&sh.o_done[tile]), nq & 1, stop));
            if (!ok) break;
            ++nq;
            tc_fence_after();
            const bool whole = s.x0 == 0 && s.x1 == s.it.nt;
            const float inv = whole ? 1.0f / l : 1.0f;
            float* rec = whole ? nullptr : chunk_record(a, 2 * static_cast<int64_t>(c) + (s.x0 == 0), tile);
#pragma unroll 1
            for (int q = 0; q < kD / 32; ++q) {
                float x[32], y[32];
                tc_ld32(x, t_o + 32 * q);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) y[(i & 16) + span_channel<VB>(i & 15)] = x[i] * inv;
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
            if (!whole && live) {
                rec[kRows * kD + r] = m;
                rec[kRows * kD + kRows + r] = l;
            }
            if (!whole && s.x0 == 0 && r == 0 && tile == 0) {
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
        const bool keys = warp < 12;
        const int p = tid & 127;
        uint64_t* full = keys ? sh.k_full : sh.v_full;
        uint64_t* empty = keys ? sh.k_empty : sh.v_empty;
        unsigned char* tiles = keys ? sk_tile : sv_tile;
        uint32_t n = 0;
        bool ok = true;
        while (ok && chunk_next(a, w, s)) {
            ChunkSrc src;
            const kivi_seq& sq = a.seqs[s.it.b];
            src.sq = &sq;
            src.L = s.it.L;
            src.np = n_packed(s.it.L, a.R, a.G);
            src.end = s.it.L + s.it.n;
            src.ring = a.R + a.G;
            src.res = static_cast<const uint16_t*>(keys ? sq.k_res : sq.v_res) + static_cast<int64_t>(s.h) * src.ring * kD;
            src.fresh = static_cast<const uint16_t*>(keys ? a.k_new[s.it.b] : a.v_new[s.it.b]) +
                        static_cast<int64_t>(s.h) * s.it.n * kD;
            for (int j = s.x0; j < s.x1; ++j, ++n) {
                const uint32_t st = n % kKvStages, use = n / kKvStages;
                if (use > 0 && !mbar_wait(smem_u32(&empty[st]), (use - 1) & 1, stop)) { ok = false; break; }
                const int64_t t0 = static_cast<int64_t>(j < s.it.st ? j : j + s.it.skip) * kKeys;
                if (keys) fill_tile<KB, DT, false>(a, src, s.h, t0, tiles + st * kOpBytes, p);
                else fill_tile<VB, DT, true>(a, src, s.h, t0, tiles + st * kOpBytes, p);
                proxy_fence();
                mbar_arrive(smem_u32(&full[st]));
            }
        }
    } else if (lane == 0) {
        // ------------------------------------------------ tensor-core issue
        uint32_t n = 0, np[2] = {0, 0}, nq[2] = {0, 0};   // key tiles, probability tiles, segments so far
        bool ok = true;
        const uint32_t kb0 = smem_u32(sk_tile), vb0 = smem_u32(sv_tile), qb0 = smem_u32(sq_tile);
        auto scores = [&](int t, uint32_t st) {
            const uint32_t q = qb0 + t * kOpBytes, k = kb0 + st * kOpBytes;
#pragma unroll
            for (int i = 0; i < kD / 16; ++i) {
                const uint32_t off = (i >> 2) * (kRows * 128) + (i & 3) * 32;
                mma_ss(tmem + t * kKeys, op_desc(q + off, 16, 1024), op_desc(k + off, 16, 1024), kIdescQK, i > 0);
            }
            tc_commit(smem_u32(&sh.s_full[t]));
        };
        while (ok && chunk_next(a, w, s)) {
            const int nt = s.it.rows > kRows ? 2 : 1, cnt = s.x1 - s.x0;
            for (int t = 0; t < nt && ok; ++t) {
                ok = mbar_wait(smem_u32(&sh.q_full[t]), nq[t] & 1, stop);
                ++nq[t];
            }
            ok = ok && mbar_wait(smem_u32(&sh.k_full[n % kKvStages]), (n / kKvStages) & 1, stop);
            if (!ok) break;
            tc_fence_after();
            for (int t = 0; t < nt; ++t) scores(t, n % kKvStages);
            tc_commit(smem_u32(&sh.k_empty[n % kKvStages]));
            for (int j = 0; j < cnt; ++j, ++n) {
                const uint32_t st = n % kKvStages, par = (n / kKvStages) & 1;
                const uint32_t st1 = (n + 1) % kKvStages, par1 = ((n + 1) / kKvStages) & 1;
                const bool more = j + 1 < cnt;
                ok = mbar_wait(smem_u32(&sh.v_full[st]), par, stop) &&
                     (!more || mbar_wait(smem_u32(&sh.k_full[st1]), par1, stop));
                for (int t = 0; t < nt && ok; ++t) {
                    ok = mbar_wait(smem_u32(&sh.p_full[t]), np[t] & 1, stop);
                    if (!ok) break;
                    ++np[t];
                    tc_fence_after();
                    const uint32_t v = vb0 + st * kOpBytes;
#pragma unroll
                    for (int i = 0; i < kKeys / 16; ++i)
                        mma_ts(tmem + 2 * kKeys + t * kD, tmem + t * kKeys + 8 * i, op_desc(v + i * 2048, kRows * 128, 1024),
                               kIdescPV, j > 0 || i > 0);
                    if (more) scores(t, st1);
                    else tc_commit(smem_u32(&sh.o_done[t]));
                }
                if (!ok) break;
                tc_commit(smem_u32(&sh.v_empty[st]));
                if (more) tc_commit(smem_u32(&sh.k_empty[st1]));
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        if (*stop != 0 && lane == 0) {
            // a wait ran out: let the products in flight finish (with a limit) before the TMEM goes
            set_status(a.status, KIVI_ERR_CUDA);
            mbar_init(smem_u32(&sh.warp_sum[0]), 1);
            tc_commit(smem_u32(&sh.warp_sum[0]));
            const long long t0 = clock64();
            while (!mbar_try(smem_u32(&sh.warp_sum[0]), 0) && clock64() - t0 < 4000000000LL) {}
        }
        __syncwarp();
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
int chunk_ctas(K kernel, std::atomic<int>* cache) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    const int have = cache[dev].load(std::memory_order_relaxed);
    if (have > 0) return have;
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kChunkSmem) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    n = n > kChunkMaxCtas ? kChunkMaxCtas : n;
    cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

template <int KB, int VB, int DT>
cudaError_t launch_chunk_dt(ChunkArgs a, cudaStream_t stream) {
    static std::atomic<int> ctas[kMaxDevices];
    a.ctas = chunk_ctas(chunk_kernel<KB, VB, DT>, ctas);
    if (a.ctas <= 0) return cudaErrorInvalidValue;
    chunk_kernel<KB, VB, DT><<<a.ctas, kChunkThreads, kChunkSmem, stream>>>(a);
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
