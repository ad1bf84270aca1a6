// Attention weights per packed group, and eviction of the groups of least weight.
//
// A decode call in its extended mode leaves, for every 32-token tile and query head h, the
// running maximum m and the sum s of 2^(x - m) over the tile's scores x (both as they stood
// when the tile was read), and per head the log2 sum E of all its exponentials. The weight
// that head h gave to the tile is then s 2^(m - E), so one pass over the cache serves the
// attention and the weights: 8 bytes per (tile, head) against the tile's keys and values.
//
// Eviction keeps whole groups (keys are quantized over the G tokens of a group, so a group is
// the smallest unit that can leave without quantizing again). group_select_kernel finds the
// kept ones by a radix select on the weights and closes the ranks of the weights and, in a
// paged cache, of the block table; evict_move_kernel moves a contiguous cache's groups and
// turns the residual rings, whose slots follow the positions.
//
// Measured (GB300, 64 sequences of 32768 tokens, 32 query heads on 8 kv heads): the weights add 15 us to
// an attention of 580 (16.8 MB of statistics against 1.64 GB of cache); cutting all 64 from 1020 to 512
// groups takes 28 us: 10 to select (latency of dependent passes, about the same for one short sequence) and 18 to
// turn 84 MB of rings (4.7 TB/s with the write).
#include "kivi_internal.cuh"

namespace kivi {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// ---------------------------------------------------------------- weights per group

constexpr int kWeightWarps = 8;
constexpr int kWeightGroups = 4;   // groups of a warp: their loads are in flight together

// One warp per (sequence, kWeightGroups groups): lanes over query heads, then a butterfly sum (a fixed
// order, so the result does not depend on timing). Launched behind the merge kernel as a
// programmatic dependent.
__global__ void __launch_bounds__(kWeightWarps * 32) group_weights_kernel(GroupWeightArgs a) {
    const int lane = threadIdx.x & 31, b = blockIdx.y;
    const int j0 = (blockIdx.x * kWeightWarps + (threadIdx.x >> 5)) * kWeightGroups;
    const int64_t L = a.kv_len[b];
    const bool bad = L < 0 || L > a.max_kv_len || n_packed(L, a.R, a.G) > a.seqs[b].cap_tokens;   // (status set by the decode kernel)
    const int tpg = a.G / kTile, tiles = bad ? 0 : static_cast<int>((L + kTile - 1) / kTile);
    asm volatile("griddepcontrol.wait;" ::: "memory");   // before anything an earlier kernel writes, weights included
    if (j0 >= a.stride) return;
    const float2* st = a.stats + (static_cast<int64_t>(b) * a.max_tiles + static_cast<int64_t>(j0) * tpg) * a.Hq;
    float w[kWeightGroups];
#pragma unroll
    for (int g = 0; g < kWeightGroups; ++g) w[g] = 0.0f;
    for (int h = lane; h < a.Hq; h += 32) {
        const float lse = a.lse[static_cast<int64_t>(b) * a.Hq + h];
#pragma unroll
        for (int i = 0; i < 2 * kWeightGroups; ++i) {   // tiles of these groups (half as many when G = 32)
            if (i < tpg * kWeightGroups && j0 * tpg + i < tiles) {
                const float2 x = st[static_cast<int64_t>(i) * a.Hq + h];
                const float y = x.y * exp2f(x.x - lse);
                w[i >> 1] += tpg == 2 ? y : 0.0f;
                if (i < kWeightGroups) w[i] += tpg == 1 ? y : 0.0f;
            }
        }
    }
#pragma unroll
    for (int g = 0; g < kWeightGroups; ++g) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) w[g] += __shfl_xor_sync(kAll, w[g], o);
    }
    if (lane < kWeightGroups && j0 + lane < a.stride) {
        const int j = j0 + lane;
        const int64_t at = static_cast<int64_t>(b) * a.stride + j;
        float v = w[0];
#pragma unroll
        for (int g = 1; g < kWeightGroups; ++g) v = lane == g ? w[g] : v;
        const bool held = static_cast<int64_t>(j) * a.G < L;
        const float before = a.in != nullptr && (bad || (held && a.decay != 0.0f)) ? a.in[at] : 0.0f;
        a.out[at] = bad ? before : !held ? 0.0f : a.decay != 0.0f ? fmaf(a.decay, before, v) : v;
    }
}

// ---------------------------------------------------------------- eviction

constexpr int kSelThreads = 512;
constexpr int kSelKeys = 8192;    // groups whose keys are kept in shared memory between the passes
constexpr int kSelWarps = kSelThreads / 32;

// Weights as unsigned numbers of the same order; NaN below everything, the zeros equal.
__device__ __forceinline__ uint32_t weight_key(float w) {
    const uint32_t u = __float_as_uint(w);
    if (w != w) return 0u;
    if (w == 0.0f) return 0x80000000u;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum over the CTA's threads of two 16-bit counts packed in one word; every
// thread gets its prefix and the total. s: kSelWarps words. Contains barriers.
__device__ __forceinline__ uint32_t scan_pair(uint32_t v, uint32_t* s, uint32_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s[warp] = incl;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
        const uint32_t x = s[w];
        before += w < warp ? x : 0;
        all += x;
    }
    __syncthreads();
    *total = all;
    return before + incl - v;
}

// One CTA per sequence. Of its ng packed groups the first `sink` and the last `recent` stay,
// and of the others the keep - sink - recent of largest weight, ties to the lower index.
//   1. radix select: four passes of 8 bits over the candidates' keys give the smallest kept
//      key and how many of the groups that have it stay;
//   2. one ordered walk closes the ranks of the kept groups in place: the walk reads a block of
//      entries before it writes any, and writes none past the block, so no entry is lost.
__global__ void __launch_bounds__(kSelThreads) group_select_kernel(EvictArgs a) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_keys[kSelKeys];
    __shared__ uint32_t s_scan[kSelWarps];
    __shared__ uint32_t s_key, s_need;
    const int tid = threadIdx.x, b = blockIdx.x;
    const int64_t L = a.kv_len[b];
    const kivi_seq& sq = a.seqs[b];
    const int64_t np = L < 0 ? 0 : n_packed(L, a.R, a.G);
    const bool bad = L < 0 || np > sq.cap_tokens || (L + a.G - 1) / a.G > a.stride;
    const int ng = bad ? 0 : static_cast<int>(np / a.G);
    const int m = ng > a.keep ? ng - a.keep : 0;
    if (m == 0) {
        if (tid == 0) {
            a.cut[2 * b] = 0;
            a.cut[2 * b + 1] = 0;
            if (bad) set_status(a.status, KIVI_ERR_LENGTH);
        }
        return;
    }
    float* w = a.weights + static_cast<int64_t>(b) * a.stride;
    int32_t* map = a.map + static_cast<int64_t>(b) * a.stride;
    const bool paged = seq_paged(sq);
    int32_t* table = const_cast<int32_t*>(sq.block_table);   // the caller's table, permuted in place
    const int c0 = a.sink, c1 = ng - a.recent;               // the candidates

    uint32_t key = 0, need = static_cast<uint32_t>(a.keep - a.sink - a.recent);
    if (need > 0) {
        // the need-th largest key among the candidates (their keys read from memory once, where they fit)
        const bool cached = c1 - c0 <= kSelKeys;
        if (cached)
            for (int j = c0 + tid; j < c1; j += kSelThreads) s_keys[j - c0] = weight_key(w[j]);
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            for (int j = c0 + tid; j < c1; j += kSelThreads) {
                const uint32_t k = cached ? s_keys[j - c0] : weight_key(w[j]);   // this thread's own entry
                if (shift == 24 || (k >> (shift + 8)) == (key >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1u);
            }
            __syncthreads();
            if (tid < 32) {
                // lane owns bins 255 - 8 lane ... 248 - 8 lane (descending)
                uint32_t n = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) n += hist[255 - 8 * tid - i];
                uint32_t incl = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(kAll, incl, o);
                    if (tid >= o) incl += y;
                }
                uint32_t above = incl - n;
                if (above < need && need <= incl) {
                    int bin = 255 - 8 * tid;
                    while (above + hist[bin] < need) above += hist[bin--];
                    s_key = key | (static_cast<uint32_t>(bin) << shift);
                    s_need = need - above;
                }
            }
            __syncthreads();
            key = s_key;
            need = s_need;
        }
    }
    const bool any = a.keep > a.sink + a.recent;   // whether any candidate stays

    int kept0 = 0, eq0 = 0;      // groups kept for sure, and groups at the smallest kept key, before this block
    int first = 0x7fffffff;      // first dropped group seen by this thread
    for (int base = 0; base < ng; base += kSelThreads) {
        const int j = base + tid;
        const bool in = j < ng;
        const float wj = in ? w[j] : 0.0f;
        const int32_t page = in && paged ? table[j] : 0;
        const bool held = in && (j < c0 || j >= c1);
        const uint32_t k = weight_key(wj);
        const bool sure = held || (in && any && k > key), eq = in && !held && any && k == key;
        uint32_t total;
        const uint32_t pre = scan_pair((sure ? 0x10000u : 0u) | (eq ? 1u : 0u), s_scan, &total);
        const int eqb = eq0 + static_cast<int>(pre & 0xffffu);
        const int rank = kept0 + static_cast<int>(pre >> 16) + (eqb < static_cast<int>(need) ? eqb : static_cast<int>(need));
        const bool kept = sure || (eq && eqb < static_cast<int>(need));
        if (kept) {
            w[rank] = wj;
            if (paged) table[rank] = page;
            else map[rank] = j;
        } else if (in) {
            if (paged) map[j - rank] = page;
            first = j < first ? j : first;
        }
        kept0 += static_cast<int>(total >> 16);
        eq0 += static_cast<int>(total & 0xffffu);
    }
    __syncthreads();
    // the first dropped group (groups before it keep their place)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const int y = __shfl_xor_sync(kAll, first, o);
        first = y < first ? y : first;
    }
    if ((tid & 31) == 0) s_scan[tid >> 5] = static_cast<uint32_t>(first);
    // freed pages follow the kept ones, ready for the groups to come
    if (paged)
        for (int e = tid; e < m; e += kSelThreads) table[a.keep + e] = map[e];
    // the weights of the groups that are not packed yet move down, zeros behind them
    for (int base = ng; base < a.stride + m; base += kSelThreads) {
        const int j = base + tid;
        const float x = j < a.stride ? w[j] : 0.0f;
        __syncthreads();
        if (j < a.stride + m) w[j - m] = x;
    }
    __syncthreads();
    if (tid == 0) {
        int f = 0x7fffffff;
        for (int i = 0; i < kSelWarps; ++i) f = static_cast<int>(s_scan[i]) < f ? static_cast<int>(s_scan[i]) : f;
        a.cut[2 * b] = m;
        a.cut[2 * b + 1] = f;
        a.kv_len[b] = static_cast<int32_t>(L - static_cast<int64_t>(m) * a.G);
    }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveBatch = 16;   // groups in flight per thread
constexpr int kTurnBatch = 10;   // ring rows in flight per thread
constexpr int kTurnSmem = 40 * 1024;

// Grid (tasks, kv heads, sequences). Tasks [0, 2 slices) turn one slice of 16-byte columns of
// the key or value ring by m G slots: the CTA reads its slice into shared memory, then
// writes every row to its new slot. The tasks behind them move a contiguous cache's groups:
// a thread owns one 16-byte column of the group record of one of the six buffers and walks
// the kept groups in order, kMoveBatch loads before their stores; rank r never passes its
// source, so no thread reads a column it has already overwritten, and threads share nothing.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictArgs a, int slice, int n_slices) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
    const int m = a.cut[2 * b];
    if (m == 0) return;
    const kivi_seq& sq = a.seqs[b];
    if (static_cast<int>(blockIdx.x) < 2 * n_slices) {
        const int ring = a.R + a.G;
        const int turn = static_cast<int>(static_cast<int64_t>(m) * a.G % ring);
        if (turn == 0) return;
        const int cols = a.D * 2 / 16;   // 16-byte columns of a row
        const int s0 = (blockIdx.x >> 1) * slice, w = cols - s0 < slice ? cols - s0 : slice;
        uint4* base = static_cast<uint4*>((blockIdx.x & 1) ? sq.v_res : sq.k_res) + static_cast<int64_t>(h) * ring * cols + s0;
        // (slice is a power of two that divides the block, so a thread stays in one column)
        uint4* buf = reinterpret_cast<uint4*>(smem);
        const int col = tid % slice, step = kMoveThreads / slice;
        if (col < w)
            for (int row = tid / slice; row < ring; row += step * kTurnBatch) {
                uint4 v[kTurnBatch];
#pragma unroll
                for (int i = 0; i < kTurnBatch; ++i)
                    if (row + i * step < ring) v[i] = base[static_cast<int64_t>(row + i * step) * cols + col];
#pragma unroll
                for (int i = 0; i < kTurnBatch; ++i)
                    if (row + i * step < ring) buf[(row + i * step) * slice + col] = v[i];
            }
        __syncthreads();
        if (col < w)
#pragma unroll 4
            for (int row = tid / slice; row < ring; row += step) {
                const int from = row + turn < ring ? row + turn : row + turn - ring;
                base[static_cast<int64_t>(row) * cols + col] = buf[from * slice + col];
            }
        return;
    }
    if (seq_paged(sq)) return;
    // bytes of one group of one kv head in each buffer, in kivi_seq order
    const int kcb = a.G * a.D * a.kb / 8, vcb = a.G * a.D * a.vb / 8, mb = a.D * 2;
    void* const bufs[6] = {sq.k_codes, sq.k_scale, sq.k_zero, sq.v_codes, sq.v_scale, sq.v_zero};
    const int sizes[6] = {kcb, mb, mb, vcb, mb, mb};
    int off = ((blockIdx.x - 2 * n_slices) * kMoveThreads + tid) * 16, size = 0;
    unsigned char* p = nullptr;
#pragma unroll
    for (int i = 0; i < 6; ++i) {
        if (p != nullptr) continue;
        if (off < sizes[i]) {
            p = static_cast<unsigned char*>(bufs[i]) + off;
            size = sizes[i];
        } else {
            off -= sizes[i];
        }
    }
    if (p == nullptr) return;
    p += static_cast<int64_t>(h) * (sq.cap_tokens / a.G) * size;
    const int32_t* map = a.map + static_cast<int64_t>(b) * a.stride;
    for (int r = a.cut[2 * b + 1]; r < a.keep; r += kMoveBatch) {
        uint4 v[kMoveBatch];
        const int n = a.keep - r < kMoveBatch ? a.keep - r : kMoveBatch;
#pragma unroll
        for (int i = 0; i < kMoveBatch; ++i)
            if (i < n) v[i] = *reinterpret_cast<const uint4*>(p + static_cast<int64_t>(map[r + i]) * size);
#pragma unroll
        for (int i = 0; i < kMoveBatch; ++i)
            if (i < n) *reinterpret_cast<uint4*>(p + static_cast<int64_t>(r + i) * size) = v[i];
    }
}

}  // namespace

cudaError_t launch_group_weights(const GroupWeightArgs& a, cudaStream_t stream) {
    constexpr int per = kWeightWarps * kWeightGroups;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.stride + per - 1) / per, a.nseq);
    cfg.blockDim = dim3(kWeightWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, group_weights_kernel, a);
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
    group_select_kernel<<<a.nseq, kSelThreads, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int ring = a.R + a.G, cols = a.D * 2 / 16;
    int slice = kTurnSmem / (ring * 16);
    while (slice & (slice - 1)) slice &= slice - 1;   // a power of two
    slice = slice < 1 ? 1 : slice > 32 ? 32 : slice;
    const int n_slices = (cols + slice - 1) / slice;
    const int smem = ring * slice * 16;
    if (smem > 48 * 1024) {
        e = cudaFuncSetAttribute(evict_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxTurnRing * 16);
        if (e != cudaSuccess) return e;
    }
    const int bytes = a.G * a.D * (a.kb + a.vb) / 8 + 8 * a.D;   // of one group of one kv head
    const int movers = (bytes / 16 + kMoveThreads - 1) / kMoveThreads;
    evict_move_kernel<<<dim3(2 * n_slices + movers, a.H, a.nseq), kMoveThreads, smem, stream>>>(a, slice, n_slices);
    return cudaGetLastError();
}

}  // namespace kivi
