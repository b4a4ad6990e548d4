// extern "C" entry points of prompt attention, shared-prefix attention and the
// cache write / read calls (declared in include/hpc_decode.h): host-side argument
// checks, then the launches in tile_plan.cu, tile_attn.cu, tile_combine.cu and
// kv.cu. Nothing here allocates or synchronises, except hpc_tile_read_error.
#include "kv.cuh"
#include "tile.cuh"

using namespace hpc;

namespace {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline hpc_status launched(cudaError_t e) {
    if (e == cudaErrorInvalidValue) return HPC_ERR_INVALID_ARG;
    return e == cudaSuccess ? HPC_OK : HPC_ERR_CUDA;
}

bool seqs_ok(int num_seqs, int num_ctas) {
    return num_seqs >= 1 && num_seqs <= HPC_MAX_BATCH && num_ctas >= 1 && num_ctas <= HPC_MAX_TILE_CTAS;
}

bool heads_ok(int num_kv_heads) { return num_kv_heads >= 1 && num_kv_heads <= HPC_MAX_KV_HEADS; }

// Tile numbers over all heads stay in int32.
bool tokens_ok(int num_tokens, int num_seqs, int num_kv_heads) {
    return num_tokens >= 0 && ((long long)num_tokens / kTileCta + num_seqs) * num_kv_heads < 2147483647LL;
}

// Tiles of 64 tokens on pairs of CTAs, or of 32 on single ones, by the average of query
// tokens per sequence (the lengths are on the device): pairs from 64 on for prompts over bf16
// caches, above 96 for prompts over e4m3 caches and for prefix groups. A pair halves the
// copies and the shared memory traffic of a row, a single CTA wastes fewer rows on the last
// tile of a sequence, so neither wins everywhere. us, tile 32 / 64 (prompts: whole calls at
// 64/8 heads; prefixes: the attention alone):
//   8 prompts of 4096 keys   new tokens  32       48       64       80       96       112      128      512
//     bf16                              52 / 55  71 / 62  76 / 65 101 / 96 102 / 97 126 / 104 129 / 104 386 / 325
//     e4m3                              54 / 65  80 / 78  85 / 80 111 / 121 116 / 122 142 / 133 147 / 134 474 / 426
//   30 whole prompts, lengths log-uniform, average about 36, 70, 105, 140
//     bf16                              25 / 28  34 / 36  51 / 50  65 / 62
//     e4m3                              35 / 33  50 / 45  73 / 62  94 / 79
//   pieces beside single tokens: 4 x 512 and 28 (average 65), 4 x 512 and 12 (129), 2048 and 30 (67),
//   2048 and 15 (129), 2 x 1024 and 20 (94)
//     bf16                             491 / 453 418 / 392 375 / 413 337 / 355 348 / 350
//     e4m3                             553 / 614 509 / 526 497 / 564 453 / 480 433 / 471
//   a prefix of 8192           requests  64       80       96       112      128      160      192
//     bf16                              22 / 22  25 / 28  27 / 29  32 / 30  32 / 30  37 / 38  41 / 39
//     e4m3                              26 / 25  32 / 36  32 / 36  38 / 38  39 / 38  46 / 49  52 / 51
// Up to 96 rows a second 64-token tile is half empty, which costs e4m3 tiles and short walks
// more than the copies: hence 96 there, between whole prompts (for which pairs win earlier)
// and mixes with single tokens (for which they win later).
int auto_tile(int mode, bool fp8, int num_tokens, int num_seqs) {
    const bool pairs = mode == kModePrefill && !fp8 ? num_tokens >= 64LL * num_seqs : num_tokens > 96LL * num_seqs;
    return pairs ? kTilePair : kTileCta;
}

// Checks of a planner's call; fills the header and the launch's arguments.
hpc_status plan_common(const int32_t* d_starts, const int32_t* d_lens, int num_seqs, int num_tokens, int num_kv_heads,
                       int table_stride, int num_ctas, int min_blocks, int tile_tokens, int mode, int q_len,
                       hpc_tile_plan* plan, TilePlanArgs* args) {
    if (!d_starts || !d_lens || !plan || !plan->buf || !aligned(plan->buf, 16) || min_blocks < 0 || table_stride < 1)
        return HPC_ERR_INVALID_ARG;
    if (!seqs_ok(num_seqs, num_ctas) || !heads_ok(num_kv_heads) || !tokens_ok(num_tokens, num_seqs, num_kv_heads))
        return HPC_ERR_INVALID_ARG;
    if (tile_tokens != 0 && tile_tokens != kTileCta && tile_tokens != kTilePair) return HPC_ERR_INVALID_ARG;
    if (plan->bytes < hpc_tile_plan_bytes(num_seqs, num_ctas)) return HPC_ERR_WORKSPACE_TOO_SMALL;
    if (tile_tokens == 0) tile_tokens = auto_tile(mode, false, num_tokens, num_seqs);
    if (num_ctas == 1) tile_tokens = kTileCta;
    plan->num_seqs = num_seqs;
    plan->num_tokens = num_tokens;
    plan->num_kv_heads = num_kv_heads;
    plan->num_workers = tile_tokens == kTilePair ? num_ctas / 2 : num_ctas;
    plan->tile_tokens = tile_tokens;
    plan->mode = mode;
    plan->q_len = q_len;
    plan->table_stride = table_stride;
    const long long max_len = (long long)table_stride * kChunk;
    *args = TilePlanArgs{d_starts, d_lens, num_seqs, num_tokens, num_kv_heads, plan->num_workers, min_blocks,
                         max_len > kMaxKeys ? kMaxKeys : (int)max_len, mode, q_len, tile_tokens, plan->buf};
    return HPC_OK;
}

hpc_status prefix_plan_fill(const int32_t* d_group_starts, const int32_t* d_prefix_lens, int num_groups, int batch, int q_len,
                            int num_kv_heads, int prefix_table_stride, int num_ctas, int min_blocks_per_cta, int tile_tokens,
                            hpc_tile_plan* plan, TilePlanArgs* args) {
    if (batch < 1 || batch > HPC_MAX_BATCH || q_len < 1 || q_len > HPC_MAX_Q_LEN) return HPC_ERR_INVALID_ARG;
    return plan_common(d_group_starts, d_prefix_lens, num_groups, batch * q_len, num_kv_heads, prefix_table_stride, num_ctas,
                       min_blocks_per_cta, tile_tokens, kModePrefix, q_len, plan, args);
}

hpc_status plan_check(const hpc_tile_plan* plan, int mode, int num_kv_heads) {
    if (!plan || !plan->buf || plan->mode != mode || plan->num_kv_heads != num_kv_heads) return HPC_ERR_INVALID_ARG;
    if (plan->tile_tokens != kTileCta && plan->tile_tokens != kTilePair) return HPC_ERR_INVALID_ARG;
    if (!seqs_ok(plan->num_seqs, plan->num_workers) || plan->bytes < hpc_tile_plan_bytes(plan->num_seqs, plan->num_workers))
        return HPC_ERR_INVALID_ARG;
    return HPC_OK;
}

hpc_status shape_check(int num_q_heads, int num_kv_heads, int head_dim, int page_size) {
    if (num_q_heads < 1 || !heads_ok(num_kv_heads)) return HPC_ERR_INVALID_ARG;
    if (head_dim != kHeadDim || page_size != kChunk || num_q_heads != kGroup * num_kv_heads) return HPC_ERR_UNSUPPORTED;
    return HPC_OK;
}

hpc_status cache_check(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale, int kv_dtype,
                       int num_pages, int num_kv_heads) {
    if (kv_dtype != HPC_KV_BF16 && kv_dtype != HPC_KV_FP8_E4M3) return HPC_ERR_UNSUPPORTED;
    const bool fp8 = kv_dtype == HPC_KV_FP8_E4M3;
    if (!k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return HPC_ERR_INVALID_ARG;
    if (fp8 && (!k_scale || !v_scale || !aligned(k_scale, 16) || !aligned(v_scale, 16))) return HPC_ERR_INVALID_ARG;
    // token and scale-row coordinates, one page past the pool included
    if (num_pages < 1 || ((long long)num_pages + 1) * kChunk > 2147483647LL ||
        ((long long)num_pages + 1) * num_kv_heads > 2147483647LL)
        return HPC_ERR_INVALID_ARG;
    return HPC_OK;
}

hpc_status attn_common(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                       const float* v_scale, int kv_dtype, int num_pages, const int32_t* table, int table_stride,
                       int num_q_heads, int num_kv_heads, int head_dim, int page_size, const hpc_tile_plan* plan, int mode,
                       float* split_o, float* split_lse, void* out, float* out_lse, void* stream) {
    hpc_status st = shape_check(num_q_heads, num_kv_heads, head_dim, page_size);
    if (st != HPC_OK) return st;
    if ((st = cache_check(k_cache, v_cache, k_scale, v_scale, kv_dtype, num_pages, num_kv_heads)) != HPC_OK) return st;
    if ((st = plan_check(plan, mode, num_kv_heads)) != HPC_OK) return st;
    if (!table || table_stride != plan->table_stride) return HPC_ERR_INVALID_ARG;
    if (!split_o || !split_lse || !aligned(split_o, 16)) return HPC_ERR_INVALID_ARG;
    if (plan->num_tokens == 0) return HPC_OK;  // q and out have no rows, and may be null
    if (!q || !aligned(q, 16)) return HPC_ERR_INVALID_ARG;
    if (mode == kModePrefill && (!out || !aligned(out, 16))) return HPC_ERR_INVALID_ARG;
    const bool fp8 = kv_dtype == HPC_KV_FP8_E4M3;
    TileAttnArgs a;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = fp8 ? k_scale : nullptr;
    a.v_scale = fp8 ? v_scale : nullptr;
    a.fp8 = fp8;
    a.num_pages = num_pages;
    a.page_table = table;
    a.pt_stride = table_stride;
    a.S = plan->num_seqs;
    a.num_tokens = plan->num_tokens;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.plan = plan->buf;
    a.num_workers = plan->num_workers;
    a.tile_tokens = plan->tile_tokens;
    a.mode = mode;
    a.q_len = plan->q_len;
    a.split_o = split_o;
    a.split_lse = split_lse;
    a.out = out;
    a.out_lse = out_lse;
    return launched(launch_tile_attn(a, static_cast<cudaStream_t>(stream)));
}

inline size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

// Workspaces of the one-call forms: the maps first, then the split rows.
struct PrefillSpace {
    size_t plan, split_o, split_lse, total;
    PrefillSpace(int batch, int num_ctas) {
        const size_t rows = hpc_prefill_split_rows(num_ctas);
        plan = 0;
        split_o = align_up(hpc_tile_plan_bytes(batch, num_ctas));
        split_lse = split_o + align_up(rows * kHeadDim * sizeof(float));
        total = split_lse + align_up(rows * sizeof(float));
    }
};

struct PrefixSpace {
    size_t prefix_plan, plan, prefix_o, prefix_lse, split_o, split_lse, total;
    PrefixSpace(int groups, int batch, int q_len, int num_kv_heads, int prefix_ctas, int ctas) {
        const size_t pr = hpc_prefix_split_rows(groups, batch, q_len, num_kv_heads, prefix_ctas);
        const size_t sr = hpc_decode_split_capacity(batch, num_kv_heads, ctas) * q_len * kGroup;
        prefix_plan = 0;
        plan = align_up(hpc_tile_plan_bytes(groups, prefix_ctas));
        prefix_o = plan + align_up(hpc_decode_plan_bytes(batch, num_kv_heads, ctas));
        prefix_lse = prefix_o + align_up(pr * kHeadDim * sizeof(float));
        split_o = prefix_lse + align_up(pr * sizeof(float));
        split_lse = split_o + align_up(sr * kHeadDim * sizeof(float));
        total = split_lse + align_up(sr * sizeof(float));
    }
};

}  // namespace

extern "C" {

size_t hpc_tile_plan_bytes(int num_seqs, int num_ctas) {
    if (!seqs_ok(num_seqs, num_ctas)) return 0;
    return (size_t)tile_layout(num_seqs, num_ctas).total_ints * sizeof(int32_t);
}

int hpc_tile_default_num_ctas(void) { return tile_default_ctas(); }

size_t hpc_prefill_split_rows(int num_ctas) {
    if (!seqs_ok(1, num_ctas)) return 0;
    return (size_t)2 * num_ctas * kTileCta * kGroup;  // the same for half as many pairs
}

size_t hpc_prefix_split_rows(int num_groups, int batch, int q_len, int num_kv_heads, int num_ctas) {
    if (!seqs_ok(num_groups, num_ctas) || batch < 1 || batch > HPC_MAX_BATCH || q_len < 1 || q_len > HPC_MAX_Q_LEN ||
        !heads_ok(num_kv_heads))
        return 0;
    // every group has at most one tile that is not full, of 64 tokens at most
    const long long tiles = ((long long)batch * q_len / kTileCta + 2LL * num_groups) * num_kv_heads;
    return (size_t)(tiles + num_ctas) * kTileCta * kGroup;
}

hpc_status hpc_prefill_plan(const int32_t* d_q_starts, const int32_t* d_seq_lens, int batch, int num_tokens,
                            int num_kv_heads, int page_table_stride, int num_ctas, int min_blocks_per_cta,
                            int tile_tokens, hpc_tile_plan* plan, void* stream) {
    TilePlanArgs a;
    const hpc_status st = plan_common(d_q_starts, d_seq_lens, batch, num_tokens, num_kv_heads, page_table_stride, num_ctas,
                                      min_blocks_per_cta, tile_tokens, kModePrefill, 1, plan, &a);
    return st != HPC_OK ? st : launched(launch_tile_plan(a, static_cast<cudaStream_t>(stream)));
}

hpc_status hpc_prefix_plan(const int32_t* d_group_starts, const int32_t* d_prefix_lens, int num_groups, int batch,
                           int q_len, int num_kv_heads, int prefix_table_stride, int num_ctas, int min_blocks_per_cta,
                           int tile_tokens, hpc_tile_plan* plan, void* stream) {
    TilePlanArgs a;
    const hpc_status st = prefix_plan_fill(d_group_starts, d_prefix_lens, num_groups, batch, q_len, num_kv_heads,
                                           prefix_table_stride, num_ctas, min_blocks_per_cta, tile_tokens, plan, &a);
    return st != HPC_OK ? st : launched(launch_tile_plan(a, static_cast<cudaStream_t>(stream)));
}

hpc_status hpc_prefill_attn(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                            const float* v_scale, int kv_dtype, int num_pages, const int32_t* page_table,
                            int page_table_stride, int num_q_heads, int num_kv_heads, int head_dim, int page_size,
                            const hpc_tile_plan* plan, float* split_o, float* split_lse, void* out, float* out_lse,
                            void* stream) {
    return attn_common(q, k_cache, v_cache, k_scale, v_scale, kv_dtype, num_pages, page_table, page_table_stride,
                       num_q_heads, num_kv_heads, head_dim, page_size, plan, kModePrefill, split_o, split_lse, out,
                       out_lse, stream);
}

hpc_status hpc_prefill_combine(const hpc_tile_plan* plan, const float* split_o, const float* split_lse, void* out,
                               float* out_lse, int num_q_heads, int num_kv_heads, int head_dim, void* stream) {
    hpc_status st = shape_check(num_q_heads, num_kv_heads, head_dim, kChunk);
    if (st != HPC_OK) return st;
    if ((st = plan_check(plan, kModePrefill, num_kv_heads)) != HPC_OK) return st;
    if (!split_o || !split_lse || !aligned(split_o, 16)) return HPC_ERR_INVALID_ARG;
    if (plan->num_tokens == 0) return HPC_OK;
    if (!out || !aligned(out, 16)) return HPC_ERR_INVALID_ARG;
    return launched(launch_prefill_combine(plan->buf, plan->num_seqs, plan->num_tokens, num_q_heads, plan->num_workers, plan->tile_tokens, split_o, split_lse,
                                           out, out_lse, static_cast<cudaStream_t>(stream)));
}

hpc_status hpc_prefix_attn(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                           const float* v_scale, int kv_dtype, int num_pages, const int32_t* prefix_table,
                           int prefix_table_stride, int num_q_heads, int num_kv_heads, int head_dim, int page_size,
                           const hpc_tile_plan* plan, float* split_o, float* split_lse, void* stream) {
    return attn_common(q, k_cache, v_cache, k_scale, v_scale, kv_dtype, num_pages, prefix_table, prefix_table_stride,
                       num_q_heads, num_kv_heads, head_dim, page_size, plan, kModePrefix, split_o, split_lse, nullptr,
                       nullptr, stream);
}

hpc_status hpc_prefix_combine(const hpc_tile_plan* prefix_plan, const float* prefix_o, const float* prefix_lse,
                              const hpc_plan* plan, const float* split_o, const float* split_lse, void* out,
                              float* out_lse, int batch, int q_len, int num_q_heads, int num_kv_heads, int head_dim,
                              void* stream) {
    hpc_status st = shape_check(num_q_heads, num_kv_heads, head_dim, kChunk);
    if (st != HPC_OK) return st;
    if ((st = plan_check(prefix_plan, kModePrefix, num_kv_heads)) != HPC_OK) return st;
    if (q_len < 1 || q_len > HPC_MAX_Q_LEN || q_len != prefix_plan->q_len) return HPC_ERR_INVALID_ARG;
    if (batch < 1 || (long long)batch * q_len != prefix_plan->num_tokens) return HPC_ERR_INVALID_ARG;
    if (!plan || !plan->buf || plan->batch != batch || plan->num_kv_heads != num_kv_heads || plan->num_ctas < 1 ||
        plan->bytes < hpc_decode_plan_bytes(batch, num_kv_heads, plan->num_ctas))
        return HPC_ERR_INVALID_ARG;
    if (!prefix_o || !prefix_lse || !split_o || !split_lse || !out || !aligned(prefix_o, 16) || !aligned(split_o, 16) ||
        !aligned(out, 8))
        return HPC_ERR_INVALID_ARG;
    return launched(launch_prefix_combine(prefix_plan->buf, prefix_plan->num_seqs, prefix_plan->num_workers, prefix_plan->tile_tokens, prefix_o,
                                          prefix_lse, plan->buf, plan->num_ctas, split_o, split_lse,
                                          static_cast<__nv_bfloat16*>(out), out_lse, batch, num_q_heads, num_kv_heads,
                                          q_len, static_cast<cudaStream_t>(stream)));
}

size_t hpc_prefill_workspace_bytes(int batch, int num_ctas) {
    if (!seqs_ok(batch, num_ctas)) return 0;
    return PrefillSpace(batch, num_ctas).total;
}

hpc_status hpc_prefill(const void* q, const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                       int kv_dtype, int num_pages, const int32_t* page_table, int page_table_stride,
                       const int32_t* q_starts, const int32_t* seq_lens, int batch, int num_tokens, int num_q_heads,
                       int num_kv_heads, int head_dim, int page_size, int num_ctas, int min_blocks_per_cta,
                       int tile_tokens, void* workspace, size_t workspace_bytes, hpc_tile_plan* plan, void* out,
                       float* out_lse, void* stream) {
    if (!plan || !workspace || !aligned(workspace, 256) || !seqs_ok(batch, num_ctas)) return HPC_ERR_INVALID_ARG;
    const PrefillSpace w(batch, num_ctas);
    if (workspace_bytes < w.total) return HPC_ERR_WORKSPACE_TOO_SMALL;
    // every check of the attention call comes before the first launch
    hpc_status st = shape_check(num_q_heads, num_kv_heads, head_dim, page_size);
    if (st != HPC_OK) return st;
    if ((st = cache_check(k_cache, v_cache, k_scale, v_scale, kv_dtype, num_pages, num_kv_heads)) != HPC_OK) return st;
    if (!page_table) return HPC_ERR_INVALID_ARG;
    if (num_tokens != 0 && (!q || !aligned(q, 16) || !out || !aligned(out, 16))) return HPC_ERR_INVALID_ARG;
    if (tile_tokens == 0 && num_tokens >= 0) tile_tokens = auto_tile(kModePrefill, kv_dtype == HPC_KV_FP8_E4M3, num_tokens, batch);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    plan->buf = reinterpret_cast<int32_t*>(ws + w.plan);
    plan->bytes = hpc_tile_plan_bytes(batch, num_ctas);
    if ((st = hpc_prefill_plan(q_starts, seq_lens, batch, num_tokens, num_kv_heads, page_table_stride, num_ctas,
                               min_blocks_per_cta, tile_tokens, plan, stream)) != HPC_OK)
        return st;
    float* so = reinterpret_cast<float*>(ws + w.split_o);
    float* sl = reinterpret_cast<float*>(ws + w.split_lse);
    if ((st = hpc_prefill_attn(q, k_cache, v_cache, k_scale, v_scale, kv_dtype, num_pages, page_table, page_table_stride,
                               num_q_heads, num_kv_heads, head_dim, page_size, plan, so, sl, out, out_lse, stream)) != HPC_OK)
        return st;
    return hpc_prefill_combine(plan, so, sl, out, out_lse, num_q_heads, num_kv_heads, head_dim, stream);
}

size_t hpc_decode_shared_prefix_workspace_bytes(int num_groups, int batch, int q_len, int num_kv_heads,
                                                int prefix_num_ctas, int num_ctas) {
    if (!seqs_ok(num_groups, prefix_num_ctas) || !heads_ok(num_kv_heads) || batch < 1 || batch > HPC_MAX_BATCH ||
        q_len < 1 || q_len > HPC_MAX_Q_LEN || num_ctas < 1 || num_ctas > HPC_MAX_CTAS)
        return 0;
    return PrefixSpace(num_groups, batch, q_len, num_kv_heads, prefix_num_ctas, num_ctas).total;
}

hpc_status hpc_decode_shared_prefix(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                    const float* v_scale, int kv_dtype, int num_pages, const int32_t* page_table,
                                    int page_table_stride, const int32_t* seq_lens, const int32_t* prefix_table,
                                    int prefix_table_stride, const int32_t* prefix_lens, const int32_t* group_starts,
                                    int num_groups, int batch, int q_len, int num_q_heads, int num_kv_heads, int head_dim,
                                    int page_size, int num_ctas, int min_chunks_per_cta, int prefix_num_ctas,
                                    int min_blocks_per_cta, int tile_tokens, void* workspace, size_t workspace_bytes,
                                    hpc_tile_plan* prefix_plan, hpc_plan* plan, void* out, float* out_lse, void* stream) {
    if (!prefix_plan || !plan || !workspace || !aligned(workspace, 256)) return HPC_ERR_INVALID_ARG;
    const size_t need = hpc_decode_shared_prefix_workspace_bytes(num_groups, batch, q_len, num_kv_heads, prefix_num_ctas, num_ctas);
    if (need == 0) return HPC_ERR_INVALID_ARG;
    if (workspace_bytes < need) return HPC_ERR_WORKSPACE_TOO_SMALL;
    // every check of the chained calls comes before the first launch
    hpc_status st = cache_check(k_cache, v_cache, k_scale, v_scale, kv_dtype, num_pages, num_kv_heads);
    if (st != HPC_OK) return st;
    if ((st = step_args_check(q, k_cache, v_cache, k_scale, v_scale, kv_dtype, num_pages, page_table, page_table_stride,
                              seq_lens, batch, num_q_heads, num_kv_heads, head_dim, page_size, num_ctas, min_chunks_per_cta,
                              out)) != HPC_OK)
        return st;
    if (!prefix_table) return HPC_ERR_INVALID_ARG;
    const PrefixSpace w(num_groups, batch, q_len, num_kv_heads, prefix_num_ctas, num_ctas);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    prefix_plan->buf = reinterpret_cast<int32_t*>(ws + w.prefix_plan);
    prefix_plan->bytes = hpc_tile_plan_bytes(num_groups, prefix_num_ctas);
    plan->buf = reinterpret_cast<int32_t*>(ws + w.plan);
    plan->bytes = hpc_decode_plan_bytes(batch, num_kv_heads, num_ctas);
    float* po = reinterpret_cast<float*>(ws + w.prefix_o);
    float* pl = reinterpret_cast<float*>(ws + w.prefix_lse);
    float* so = reinterpret_cast<float*>(ws + w.split_o);
    float* sl = reinterpret_cast<float*>(ws + w.split_lse);
    TilePlanArgs ta;
    if ((st = prefix_plan_fill(group_starts, prefix_lens, num_groups, batch, q_len, num_kv_heads, prefix_table_stride,
                               prefix_num_ctas, min_blocks_per_cta, tile_tokens, prefix_plan, &ta)) != HPC_OK)
        return st;
    if ((st = decode_plan_fill(seq_lens, batch, num_kv_heads, num_ctas, min_chunks_per_cta, plan)) != HPC_OK) return st;
    if ((st = launched(launch_both_plans(ta, seq_lens, batch, num_kv_heads, num_ctas, min_chunks_per_cta, plan->buf,
                                         static_cast<cudaStream_t>(stream)))) != HPC_OK)
        return st;
    if ((st = hpc_prefix_attn(q, k_cache, v_cache, k_scale, v_scale, kv_dtype, num_pages, prefix_table, prefix_table_stride,
                              num_q_heads, num_kv_heads, head_dim, page_size, prefix_plan, po, pl, stream)) != HPC_OK)
        return st;
    if ((st = hpc_decode_attn_multi(q, q_len, k_cache, v_cache, k_scale, v_scale, kv_dtype, num_pages, page_table,
                                    page_table_stride, seq_lens, batch, num_q_heads, num_kv_heads, head_dim, page_size, plan,
                                    so, sl, stream)) != HPC_OK)
        return st;
    return hpc_prefix_combine(prefix_plan, po, pl, plan, so, sl, out, out_lse, batch, q_len, num_q_heads, num_kv_heads,
                              head_dim, stream);
}

hpc_status hpc_kv_write(const void* k, const void* v, long long k_token_stride, long long v_token_stride,
                        const int32_t* slot_mapping, int num_tokens, int num_kv_heads, int head_dim, int page_size,
                        void* k_cache, void* v_cache, float* k_scale, float* v_scale, int kv_dtype, int num_pages,
                        int* d_error_word, void* stream) {
    if (head_dim != kHeadDim || page_size != kChunk) return HPC_ERR_UNSUPPORTED;
    if (num_tokens < 0 || !heads_ok(num_kv_heads)) return HPC_ERR_INVALID_ARG;
    hpc_status st = cache_check(k_cache, v_cache, k_scale, v_scale, kv_dtype, num_pages, num_kv_heads);
    if (st != HPC_OK) return st;
    // rows of 16-byte pieces; a stride shorter than a token's heads would be a mistake
    const long long row = (long long)num_kv_heads * kHeadDim;
    if (k_token_stride < row || v_token_stride < row || k_token_stride % 8 != 0 || v_token_stride % 8 != 0)
        return HPC_ERR_INVALID_ARG;
    if (num_tokens == 0) return HPC_OK;  // the rows' pointers may be null then
    if (!k || !v || !slot_mapping || !aligned(k, 16) || !aligned(v, 16)) return HPC_ERR_INVALID_ARG;
    KvWriteArgs a;
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.k_stride = k_token_stride;
    a.v_stride = v_token_stride;
    a.slots = slot_mapping;
    a.num_tokens = num_tokens;
    a.num_kv_heads = num_kv_heads;
    a.num_pages = num_pages;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.err = d_error_word;
    return launched(launch_kv_write(a, kv_dtype == HPC_KV_FP8_E4M3, static_cast<cudaStream_t>(stream)));
}

hpc_status hpc_kv_read(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale, int kv_dtype,
                       int num_pages, const int32_t* page_table, int page_table_stride, const int32_t* first,
                       const int32_t* out_starts, int batch, int num_rows, int num_kv_heads, int head_dim, int page_size,
                       void* k_out, void* v_out, int* d_error_word, void* stream) {
    if (head_dim != kHeadDim || page_size != kChunk) return HPC_ERR_UNSUPPORTED;
    if (batch < 1 || batch > HPC_MAX_BATCH || num_rows < 0 || !heads_ok(num_kv_heads) || page_table_stride < 1)
        return HPC_ERR_INVALID_ARG;
    hpc_status st = cache_check(k_cache, v_cache, k_scale, v_scale, kv_dtype, num_pages, num_kv_heads);
    if (st != HPC_OK) return st;
    if (!page_table || !out_starts) return HPC_ERR_INVALID_ARG;
    if (num_rows == 0) return HPC_OK;
    if (!k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16)) return HPC_ERR_INVALID_ARG;
    KvReadArgs a;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.page_table = page_table;
    a.pt_stride = page_table_stride;
    a.first = first;
    a.out_starts = out_starts;
    a.batch = batch;
    a.num_rows = num_rows;
    a.num_kv_heads = num_kv_heads;
    a.num_pages = num_pages;
    a.k_out = static_cast<__nv_bfloat16*>(k_out);
    a.v_out = static_cast<__nv_bfloat16*>(v_out);
    a.err = d_error_word;
    return launched(launch_kv_read(a, kv_dtype == HPC_KV_FP8_E4M3, static_cast<cudaStream_t>(stream)));
}

hpc_status hpc_tile_read_error(const hpc_tile_plan* plan, int* device_error_word) {
    if (!plan || !plan->buf || !device_error_word) return HPC_ERR_INVALID_ARG;
    if (cudaDeviceSynchronize() != cudaSuccess) return HPC_ERR_CUDA;
    int w = 0;
    if (cudaMemcpy(&w, plan->buf + kTError, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return HPC_ERR_CUDA;
    *device_error_word = w;
    return w ? HPC_ERR_DEVICE_CHECK : HPC_OK;
}

}  // extern "C"
