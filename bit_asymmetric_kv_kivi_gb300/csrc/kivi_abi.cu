// The extern "C" boundary of the KIVI library: argument validation on the
// host, sizes and workspace planning, and the launches. Every entry point
// checks its arguments before anything is enqueued, so an invalid call
// launches nothing and returns an error code.
#include <math.h>
#include <string.h>

#include "kivi_internal.cuh"

namespace {

bool cfg_ok(const kivi_cfg* c) {
    if (c == nullptr) return false;
    if (c->k_bits != 2 && c->k_bits != 4) return false;
    if (c->v_bits != 2 && c->v_bits != 4) return false;
    if (c->group != 32 && c->group != 64) return false;
    if (c->residual <= 0 || c->residual % c->group != 0) return false;
    if (c->head_dim <= 0 || c->head_dim % c->group != 0 || c->head_dim > kivi::kMaxHeadDim) return false;
    if (c->num_kv_heads <= 0 || c->num_kv_heads > 65535) return false;
    if (c->num_q_heads <= 0 || c->num_q_heads % c->num_kv_heads != 0) return false;
    if (c->dtype != KIVI_F16 && c->dtype != KIVI_BF16) return false;
    return true;
}

kivi_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KIVI_OK : KIVI_ERR_CUDA; }

kivi_status codec_common(const kivi_cfg* cfg, int bits, int32_t n_streams, int32_t n_tokens, const void* x,
                         uint8_t* codes, uint16_t* scale, uint16_t* zero, kivi::CodecArgs* a) {
    if (!cfg_ok(cfg)) return KIVI_ERR_ARG;
    if (n_streams < 0 || n_tokens < 0 || n_streams > 65535) return KIVI_ERR_ARG;
    if (n_streams > 0 && n_tokens > 0 &&
        (x == nullptr || codes == nullptr || scale == nullptr || zero == nullptr))
        return KIVI_ERR_ARG;
    a->bits = bits;
    a->G = cfg->group;
    a->D = cfg->head_dim;
    a->dtype = cfg->dtype;
    a->n_streams = n_streams;
    a->n_tokens = n_tokens;
    a->x = x;
    a->codes = codes;
    a->scale = scale;
    a->zero = zero;
    return KIVI_OK;
}

}  // namespace

extern "C" {

kivi_status kivi_quant_keys(const kivi_cfg* cfg, int32_t n_streams, int32_t n_tokens, const void* x_dev,
                            uint8_t* codes_dev, uint16_t* scale_dev, uint16_t* zero_dev, void* stream) {
    kivi::CodecArgs a;
    const kivi_status st = codec_common(cfg, cfg ? cfg->k_bits : 0, n_streams, n_tokens, x_dev, codes_dev, scale_dev,
                                        zero_dev, &a);
    if (st != KIVI_OK) return st;
    if (n_tokens % cfg->group != 0) return KIVI_ERR_ARG;
    return from_cuda(kivi::launch_quant_keys(a, static_cast<cudaStream_t>(stream)));
}

kivi_status kivi_quant_values(const kivi_cfg* cfg, int32_t n_streams, int32_t n_tokens, const void* x_dev,
                              uint8_t* codes_dev, uint16_t* scale_dev, uint16_t* zero_dev, void* stream) {
    kivi::CodecArgs a;
    const kivi_status st = codec_common(cfg, cfg ? cfg->v_bits : 0, n_streams, n_tokens, x_dev, codes_dev, scale_dev,
                                        zero_dev, &a);
    if (st != KIVI_OK) return st;
    return from_cuda(kivi::launch_quant_values(a, static_cast<cudaStream_t>(stream)));
}

kivi_status kivi_append_flush(const kivi_cfg* cfg, int32_t nseq, const kivi_seq* seqs_dev, int32_t* kv_len_dev,
                              const void* const* k_new_dev, const void* const* v_new_dev,
                              const int32_t* n_new_dev, int32_t max_new, int32_t* status_dev, void* stream) {
    if (!cfg_ok(cfg)) return KIVI_ERR_ARG;
    if (nseq < 0 || nseq > 65535 || max_new < 0) return KIVI_ERR_ARG;
    if (nseq == 0) return KIVI_OK;
    if (seqs_dev == nullptr || kv_len_dev == nullptr || k_new_dev == nullptr || v_new_dev == nullptr ||
        n_new_dev == nullptr || status_dev == nullptr)
        return KIVI_ERR_ARG;
    kivi::AppendArgs a;
    a.kb = cfg->k_bits;
    a.vb = cfg->v_bits;
    a.G = cfg->group;
    a.D = cfg->head_dim;
    a.R = cfg->residual;
    a.H = cfg->num_kv_heads;
    a.dtype = cfg->dtype;
    a.nseq = nseq;
    a.max_new = max_new;
    a.seqs = seqs_dev;
    a.kv_len = kv_len_dev;
    a.k_new = k_new_dev;
    a.v_new = v_new_dev;
    a.n_new = n_new_dev;
    a.status = status_dev;
    return from_cuda(kivi::launch_append_flush(a, static_cast<cudaStream_t>(stream)));
}

size_t kivi_decode_workspace_bytes(const kivi_cfg* cfg, int32_t nseq, int32_t max_kv_len) {
    if (!cfg_ok(cfg) || nseq < 0 || max_kv_len < 0) return 0;
    int chunk, max_splits;
    size_t cb, pb;
    kivi::decode_plan(nseq, cfg->num_kv_heads, cfg->num_q_heads, cfg->head_dim, max_kv_len, &chunk,
                      &max_splits, &cb, &pb);
    return cb + pb;
}

kivi_status kivi_decode_attn(const kivi_cfg* cfg, int32_t nseq, const kivi_seq* seqs_dev,
                             const int32_t* kv_len_dev, const void* q_dev, float* out_dev, float softmax_scale,
                             int32_t max_kv_len, void* workspace_dev, size_t workspace_bytes,
                             int32_t* status_dev, void* stream) {
    if (!cfg_ok(cfg)) return KIVI_ERR_ARG;
    if (nseq < 0 || nseq > 65535 || max_kv_len < 0 || !isfinite(softmax_scale)) return KIVI_ERR_ARG;
    const int g = cfg->num_q_heads / cfg->num_kv_heads;
    if (cfg->head_dim != 128 || g > 32) return KIVI_ERR_UNSUPPORTED;
    if (nseq == 0) return KIVI_OK;
    if (seqs_dev == nullptr || kv_len_dev == nullptr || q_dev == nullptr || out_dev == nullptr)
        return KIVI_ERR_ARG;
    kivi::DecodeArgs a;
    size_t cb, pb;
    kivi::decode_plan(nseq, cfg->num_kv_heads, cfg->num_q_heads, cfg->head_dim, max_kv_len, &a.chunk,
                      &a.max_splits, &cb, &pb);
    if (workspace_dev == nullptr || workspace_bytes < cb + pb) return KIVI_ERR_WORKSPACE;
    a.kb = cfg->k_bits;
    a.vb = cfg->v_bits;
    a.G = cfg->group;
    a.D = cfg->head_dim;
    a.R = cfg->residual;
    a.Hq = cfg->num_q_heads;
    a.H = cfg->num_kv_heads;
    a.dtype = cfg->dtype;
    a.nseq = nseq;
    a.max_kv_len = max_kv_len;
    a.n_query = 0;
    a.seqs = seqs_dev;
    a.kv_len = kv_len_dev;
    a.q = q_dev;
    a.out = out_dev;
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    a.counters = static_cast<int32_t*>(workspace_dev);
    a.partials = reinterpret_cast<float*>(static_cast<char*>(workspace_dev) + cb);
    a.status = status_dev;
    return from_cuda(kivi::launch_decode(a, static_cast<cudaStream_t>(stream)));
}

// Multi-query calls that run on the persistent decode kernel: one query with a query group
// of 1, 2, 4 or 8 (decode attention; kv_len 0 stays a length error), several queries at a
// group of 4 or 8, and two queries at a group of 1 or 2 (one stream of the group's heads per
// query and kv head, each stopping at its query's causal end). Below four or eight (query,
// head) pairs per kv head that beat the multi-query kernel, whose shared unpack wins beyond.
static bool multi_is_decode(const kivi_cfg* cfg, int32_t n_query) {
    const int g = cfg->num_q_heads / cfg->num_kv_heads;
    return (n_query == 1 && (g == 1 || g == 2 || g == 4 || g == 8)) || (n_query > 1 && (g == 4 || g == 8)) ||
           (n_query == 2 && (g == 1 || g == 2));
}

static void multi_or_decode_plan(const kivi_cfg* cfg, int32_t nseq, int32_t n_query, int32_t max_kv_len, int* chunk,
                                 int* max_splits, size_t* cb, size_t* pb) {
    if (multi_is_decode(cfg, n_query) && n_query == 1) {
        kivi::decode_plan(nseq, cfg->num_kv_heads, cfg->num_q_heads, cfg->head_dim, max_kv_len, chunk, max_splits, cb,
                          pb);
    } else if (multi_is_decode(cfg, n_query)) {
        *chunk = 0;   // n_query streams of the group's heads per kv head
        *max_splits = 0;
        kivi::mma_plan(nseq, cfg->num_kv_heads, cfg->head_dim, cfg->num_q_heads / cfg->num_kv_heads, n_query, cb, pb);
    } else
        kivi::multi_plan(nseq, cfg->num_kv_heads, cfg->num_q_heads, cfg->head_dim, n_query, max_kv_len, chunk,
                         max_splits, cb, pb);
}

size_t kivi_decode_multi_workspace_bytes(const kivi_cfg* cfg, int32_t nseq, int32_t n_query, int32_t max_kv_len) {
    if (!cfg_ok(cfg) || nseq < 0 || max_kv_len < 0 || n_query < 1) return 0;
    int chunk, max_splits;
    size_t cb, pb;
    multi_or_decode_plan(cfg, nseq, n_query, max_kv_len, &chunk, &max_splits, &cb, &pb);
    return cb + pb;
}

kivi_status kivi_decode_multi_attn(const kivi_cfg* cfg, int32_t nseq, const kivi_seq* seqs_dev,
                                   const int32_t* kv_len_dev, int32_t n_query, const void* q_dev, float* out_dev,
                                   float softmax_scale, int32_t max_kv_len, void* workspace_dev,
                                   size_t workspace_bytes, int32_t* status_dev, void* stream) {
    if (!cfg_ok(cfg)) return KIVI_ERR_ARG;
    if (nseq < 0 || nseq > 65535 || max_kv_len < 0 || n_query < 1 || !isfinite(softmax_scale)) return KIVI_ERR_ARG;
    const int g = cfg->num_q_heads / cfg->num_kv_heads;
    if (cfg->head_dim != 128 || static_cast<int64_t>(n_query) * g > 32) return KIVI_ERR_UNSUPPORTED;
    if (nseq == 0) return KIVI_OK;
    if (seqs_dev == nullptr || kv_len_dev == nullptr || q_dev == nullptr || out_dev == nullptr)
        return KIVI_ERR_ARG;
    kivi::DecodeArgs a;
    size_t cb, pb;
    multi_or_decode_plan(cfg, nseq, n_query, max_kv_len, &a.chunk, &a.max_splits, &cb, &pb);
    if (workspace_dev == nullptr || workspace_bytes < cb + pb) return KIVI_ERR_WORKSPACE;
    a.kb = cfg->k_bits;
    a.vb = cfg->v_bits;
    a.G = cfg->group;
    a.D = cfg->head_dim;
    a.R = cfg->residual;
    a.Hq = cfg->num_q_heads;
    a.H = cfg->num_kv_heads;
    a.dtype = cfg->dtype;
    a.nseq = nseq;
    a.max_kv_len = max_kv_len;
    a.n_query = n_query;
    a.seqs = seqs_dev;
    a.kv_len = kv_len_dev;
    a.q = q_dev;
    a.out = out_dev;
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    a.counters = static_cast<int32_t*>(workspace_dev);
    a.partials = reinterpret_cast<float*>(static_cast<char*>(workspace_dev) + cb);
    a.status = status_dev;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return from_cuda(multi_is_decode(cfg, n_query) ? kivi::launch_decode(a, st) : kivi::launch_multi(a, st));
}

size_t kivi_decode_ext_workspace_bytes(const kivi_cfg* cfg, int32_t nseq, int32_t max_kv_len) {
    if (!cfg_ok(cfg) || nseq < 0 || max_kv_len < 0) return 0;
    const int g = cfg->num_q_heads / cfg->num_kv_heads;
    size_t cb, pb;
    kivi::mma_plan(nseq, cfg->num_kv_heads, cfg->head_dim, kivi::ext_heads(g), kivi::ext_parts(g), &cb, &pb);
    return cb + pb;
}

// 32-token tiles of the longest sequence, and the scratch bytes of their statistics and of
// the heads' log sums.
static size_t weight_tiles(int32_t max_kv_len) { return (static_cast<size_t>(max_kv_len) + kivi::kTile - 1) / kivi::kTile; }

size_t kivi_decode_weights_scratch_bytes(const kivi_cfg* cfg, int32_t nseq, int32_t max_kv_len) {
    if (!cfg_ok(cfg) || nseq < 0 || max_kv_len < 0) return 0;
    const size_t heads = static_cast<size_t>(nseq) * cfg->num_q_heads;
    return heads * weight_tiles(max_kv_len) * sizeof(float2) + heads * sizeof(float);
}

// Arguments and checks shared by the two extended decode calls.
static kivi_status ext_args(const kivi_cfg* cfg, int32_t nseq, const kivi_seq* seqs, const int32_t* kv_len,
                            const void* q, float* out, float softmax_scale, int32_t max_kv_len, void* ws,
                            size_t ws_bytes, int32_t* status, kivi::DecodeArgs* a) {
    if (!cfg_ok(cfg)) return KIVI_ERR_ARG;
    if (nseq < 0 || nseq > 65535 || max_kv_len < 0 || !isfinite(softmax_scale)) return KIVI_ERR_ARG;
    const int g = cfg->num_q_heads / cfg->num_kv_heads;
    if (cfg->head_dim != 128 || g > 32) return KIVI_ERR_UNSUPPORTED;
    if (nseq == 0) return KIVI_OK;
    if (seqs == nullptr || kv_len == nullptr || q == nullptr || out == nullptr) return KIVI_ERR_ARG;
    size_t cb, pb;
    kivi::mma_plan(nseq, cfg->num_kv_heads, cfg->head_dim, kivi::ext_heads(g), kivi::ext_parts(g), &cb, &pb);
    if (ws == nullptr || ws_bytes < cb + pb) return KIVI_ERR_WORKSPACE;
    a->chunk = a->max_splits = 0;
    a->kb = cfg->k_bits;
    a->vb = cfg->v_bits;
    a->G = cfg->group;
    a->D = cfg->head_dim;
    a->R = cfg->residual;
    a->Hq = cfg->num_q_heads;
    a->H = cfg->num_kv_heads;
    a->dtype = cfg->dtype;
    a->nseq = nseq;
    a->max_kv_len = max_kv_len;
    a->n_query = 0;
    a->n_part = kivi::ext_parts(g);
    a->seqs = seqs;
    a->kv_len = kv_len;
    a->q = q;
    a->out = out;
    a->scale_log2 = softmax_scale * 1.4426950408889634f;
    a->counters = static_cast<int32_t*>(ws);
    a->partials = reinterpret_cast<float*>(static_cast<char*>(ws) + cb);
    a->status = status;
    return KIVI_OK;
}

kivi_status kivi_decode_window_attn(const kivi_cfg* cfg, int32_t nseq, const kivi_seq* seqs_dev,
                                    const int32_t* kv_len_dev, const void* q_dev, float* out_dev,
                                    float softmax_scale, int32_t window, int32_t sinks, int32_t max_kv_len,
                                    void* workspace_dev, size_t workspace_bytes, int32_t* status_dev,
                                    void* stream) {
    if (window < 0 || sinks < 0) return KIVI_ERR_ARG;
    kivi::DecodeArgs a;
    const kivi_status st = ext_args(cfg, nseq, seqs_dev, kv_len_dev, q_dev, out_dev, softmax_scale, max_kv_len,
                                    workspace_dev, workspace_bytes, status_dev, &a);
    if (st != KIVI_OK || nseq == 0) return st;
    a.window = window;
    a.sinks = sinks;
    return from_cuda(kivi::launch_ext(a, static_cast<cudaStream_t>(stream)));
}

kivi_status kivi_decode_attn_weights(const kivi_cfg* cfg, int32_t nseq, const kivi_seq* seqs_dev,
                                     const int32_t* kv_len_dev, const void* q_dev, float* out_dev,
                                     const float* weights_in_dev, float* weights_out_dev, int32_t weights_stride,
                                     float decay, float softmax_scale, int32_t max_kv_len, void* workspace_dev,
                                     size_t workspace_bytes, void* scratch_dev, size_t scratch_bytes,
                                     int32_t* status_dev, void* stream) {
    kivi::DecodeArgs a;
    if (!cfg_ok(cfg) || weights_stride < 0 || !isfinite(decay)) return KIVI_ERR_ARG;
    if (static_cast<int64_t>(weights_stride) * cfg->group < max_kv_len) return KIVI_ERR_ARG;
    const kivi_status st = ext_args(cfg, nseq, seqs_dev, kv_len_dev, q_dev, out_dev, softmax_scale, max_kv_len,
                                    workspace_dev, workspace_bytes, status_dev, &a);
    if (st != KIVI_OK || nseq == 0) return st;
    if (weights_out_dev == nullptr && weights_stride > 0) return KIVI_ERR_ARG;
    if (scratch_dev == nullptr || scratch_bytes < kivi_decode_weights_scratch_bytes(cfg, nseq, max_kv_len))
        return KIVI_ERR_WORKSPACE;
    a.max_tiles = static_cast<int>(weight_tiles(max_kv_len));
    a.stats = static_cast<float2*>(scratch_dev);
    a.lse = reinterpret_cast<float*>(a.stats + static_cast<size_t>(nseq) * a.max_tiles * a.Hq);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = kivi::launch_ext(a, s);
    if (e != cudaSuccess || weights_stride == 0) return from_cuda(e);
    kivi::GroupWeightArgs w;
    w.G = a.G;
    w.R = a.R;
    w.Hq = a.Hq;
    w.nseq = nseq;
    w.max_kv_len = max_kv_len;
    w.max_tiles = a.max_tiles;
    w.stride = weights_stride;
    w.seqs = seqs_dev;
    w.kv_len = kv_len_dev;
    w.stats = a.stats;
    w.lse = a.lse;
    w.in = weights_in_dev;
    w.out = weights_out_dev;
    w.decay = decay;
    return from_cuda(kivi::launch_group_weights(w, s));
}

size_t kivi_chunk_scratch_bytes(const kivi_cfg* cfg, int32_t nseq, int32_t max_new) {
    if (!cfg_ok(cfg) || nseq < 0 || max_new < 0) return 0;
    int pairs, tiles;
    size_t rec;
    kivi::chunk_plan(cfg->num_q_heads, cfg->num_kv_heads, max_new, &pairs, &tiles, &rec);
    return rec + kivi::kChunkMaxCtas * sizeof(kivi::ChunkInfo);
}

kivi_status kivi_chunk_attn(const kivi_cfg* cfg, int32_t nseq, const kivi_seq* seqs_dev, const int32_t* kv_len_dev,
                            const void* const* k_new_dev, const void* const* v_new_dev, const int32_t* n_new_dev,
                            int32_t max_new, const void* q_dev, const int32_t* q_start_dev, void* out_dev,
                            float softmax_scale, int32_t window, int32_t sinks, int32_t max_kv_len,
                            void* scratch_dev, size_t scratch_bytes, int32_t* status_dev, void* stream) {
    if (!cfg_ok(cfg)) return KIVI_ERR_ARG;
    if (nseq < 0 || nseq > 65535 || max_new < 0 || max_kv_len < 0 || window < 0 || sinks < 0 || !isfinite(softmax_scale))
        return KIVI_ERR_ARG;
    const int64_t g = cfg->num_q_heads / cfg->num_kv_heads;
    if (cfg->head_dim != 128 || g * max_new > INT32_MAX - 256 || static_cast<int64_t>(max_kv_len) + max_new > INT32_MAX - 256)
        return KIVI_ERR_UNSUPPORTED;
    if (nseq == 0 || max_new == 0) return KIVI_OK;
    if (seqs_dev == nullptr || kv_len_dev == nullptr || k_new_dev == nullptr || v_new_dev == nullptr ||
        n_new_dev == nullptr || q_dev == nullptr || q_start_dev == nullptr || out_dev == nullptr)
        return KIVI_ERR_ARG;
    if (scratch_dev == nullptr || scratch_bytes < kivi_chunk_scratch_bytes(cfg, nseq, max_new)) return KIVI_ERR_WORKSPACE;
    kivi::ChunkArgs a;
    size_t rec;
    kivi::chunk_plan(cfg->num_q_heads, cfg->num_kv_heads, max_new, &a.pairs, &a.rec_tiles, &rec);
    if (static_cast<int64_t>(a.pairs) * nseq > INT32_MAX) return KIVI_ERR_UNSUPPORTED;
    a.kb = cfg->k_bits;
    a.vb = cfg->v_bits;
    a.G = cfg->group;
    a.R = cfg->residual;
    a.Hq = cfg->num_q_heads;
    a.H = cfg->num_kv_heads;
    a.dtype = cfg->dtype;
    a.nseq = nseq;
    a.max_new = max_new;
    a.max_kv_len = max_kv_len;
    a.window = static_cast<int64_t>(window) >= static_cast<int64_t>(max_kv_len) + max_new ? 0 : window;   // hides nothing
    a.sinks = sinks;
    a.ctas = 0;
    a.seqs = seqs_dev;
    a.kv_len = kv_len_dev;
    a.k_new = k_new_dev;
    a.v_new = v_new_dev;
    a.n_new = n_new_dev;
    a.q_start = q_start_dev;
    a.q = q_dev;
    a.out = out_dev;
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    a.records = static_cast<float*>(scratch_dev);
    a.info = reinterpret_cast<kivi::ChunkInfo*>(static_cast<char*>(scratch_dev) + rec);
    a.status = status_dev;
    return from_cuda(kivi::launch_chunk(a, static_cast<cudaStream_t>(stream)));
}

size_t kivi_evict_scratch_bytes(int32_t nseq, int32_t weights_stride) {
    if (nseq < 0 || weights_stride < 0) return 0;
    return static_cast<size_t>(nseq) * (static_cast<size_t>(weights_stride) + 2) * sizeof(int32_t);
}

kivi_status kivi_evict_groups(const kivi_cfg* cfg, int32_t nseq, const kivi_seq* seqs_dev, int32_t* kv_len_dev,
                              float* weights_dev, int32_t weights_stride, int32_t keep_groups, int32_t sink_groups,
                              int32_t recent_groups, void* scratch_dev, size_t scratch_bytes, int32_t* status_dev,
                              void* stream) {
    if (!cfg_ok(cfg)) return KIVI_ERR_ARG;
    if (nseq < 0 || nseq > 65535 || weights_stride < 0 || keep_groups < 0 || sink_groups < 0 || recent_groups < 0)
        return KIVI_ERR_ARG;
    if (static_cast<int64_t>(sink_groups) + recent_groups > keep_groups) return KIVI_ERR_ARG;
    if (static_cast<int64_t>(cfg->residual) + cfg->group > kivi::kMaxTurnRing) return KIVI_ERR_UNSUPPORTED;
    if (nseq == 0) return KIVI_OK;
    if (seqs_dev == nullptr || kv_len_dev == nullptr || status_dev == nullptr ||
        (weights_dev == nullptr && weights_stride > 0))
        return KIVI_ERR_ARG;
    if (scratch_dev == nullptr || scratch_bytes < kivi_evict_scratch_bytes(nseq, weights_stride))
        return KIVI_ERR_WORKSPACE;
    kivi::EvictArgs a;
    a.kb = cfg->k_bits;
    a.vb = cfg->v_bits;
    a.G = cfg->group;
    a.D = cfg->head_dim;
    a.R = cfg->residual;
    a.H = cfg->num_kv_heads;
    a.nseq = nseq;
    a.stride = weights_stride;
    a.keep = keep_groups;
    a.sink = sink_groups;
    a.recent = recent_groups;
    a.seqs = seqs_dev;
    a.kv_len = kv_len_dev;
    a.weights = weights_dev;
    a.cut = static_cast<int32_t*>(scratch_dev);
    a.map = a.cut + 2 * static_cast<size_t>(nseq);
    a.status = status_dev;
    return from_cuda(kivi::launch_evict(a, static_cast<cudaStream_t>(stream)));
}

kivi_status kivi_seq_buffer_bytes(const kivi_cfg* cfg, int32_t cap_tokens, size_t bytes_out[8]) {
    if (!cfg_ok(cfg) || cap_tokens < 0 || cap_tokens % cfg->group != 0 || bytes_out == nullptr) return KIVI_ERR_ARG;
    const size_t H = cfg->num_kv_heads, D = cfg->head_dim, cap = cap_tokens, G = cfg->group;
    const size_t esz = 2;  // fp16 and bf16
    const size_t kcodes = H * cap * D * cfg->k_bits / 8, vcodes = H * cap * D * cfg->v_bits / 8;
    const size_t kmeta = H * (cap / G) * D * 2;
    const size_t vmeta = H * cap * (D / G) * 2;
    const size_t ring = H * (cfg->residual + G) * D * esz;
    const size_t sizes[8] = {kcodes, kmeta, kmeta, vcodes, vmeta, vmeta, ring, ring};
    memcpy(bytes_out, sizes, sizeof(sizes));
    return KIVI_OK;
}

int64_t kivi_seq_bytes(const kivi_cfg* cfg, int32_t cap_tokens) {
    size_t b[8];
    if (kivi_seq_buffer_bytes(cfg, cap_tokens, b) != KIVI_OK) return -1;
    int64_t total = 0;
    for (int i = 0; i < 8; ++i) total += static_cast<int64_t>(b[i]);
    return total;
}

int64_t kivi_kv_bytes_plain(int32_t layers, int32_t num_kv_heads, int32_t head_dim, int32_t bits, int64_t tokens,
                            int64_t batch) {
    if (bits != 2 && bits != 4 && bits != 8 && bits != 16) return -1;
    if (layers < 0 || num_kv_heads < 0 || head_dim < 0 || tokens < 0 || batch < 0) return -1;
    // bits of one token of one layer (K and V), then bytes: every factor is checked against
    // overflow before it is applied
    const int64_t lim = INT64_MAX;
    int64_t v = 2 * static_cast<int64_t>(num_kv_heads) * head_dim * bits;   // < 2^49
    const int64_t f[3] = {layers, tokens, batch};
    for (int i = 0; i < 3; ++i) {
        if (f[i] != 0 && v > lim / f[i]) return -1;
        v *= f[i];
    }
    return v / 8;
}

int64_t kivi_n_packed(const kivi_cfg* cfg, int64_t kv_len) {
    if (!cfg_ok(cfg) || kv_len < 0) return -1;
    return kivi::n_packed(kv_len, cfg->residual, cfg->group);
}

const char* kivi_status_string(int32_t status) {
    switch (status) {
        case KIVI_OK: return "ok";
        case KIVI_ERR_ARG: return "invalid argument or configuration";
        case KIVI_ERR_UNSUPPORTED: return "configuration not supported by this library";
        case KIVI_ERR_CAPACITY: return "append exceeds the packed capacity of a sequence";
        case KIVI_ERR_WORKSPACE: return "workspace missing or too small";
        case KIVI_ERR_CUDA: return "CUDA launch or runtime error";
        case KIVI_ERR_LENGTH: return "sequence length or new-token count out of range";
        default: return "unknown status";
    }
}

int32_t kivi_abi_version(void) { return KIVI_ABI_VERSION; }

}  // extern "C"
