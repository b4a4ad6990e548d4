// extern "C" entry points of the decode loop between two attention steps: attention weights
// of cached tokens, selection, compaction, verification of drafted tokens (declared in
// include/hpc_decode.h). Host-side argument checks, then one launch each; nothing here
// allocates or synchronises.
#include "loop.cuh"
#include "tile.cuh"

using namespace hpc;

namespace {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline hpc_status launched(cudaError_t e) {
    if (e == cudaErrorInvalidValue) return HPC_ERR_INVALID_ARG;
    return e == cudaSuccess ? HPC_OK : HPC_ERR_CUDA;
}

// An int32 array of a call. What one block writes while another still reads it, or writes it
// too, has no answer: such arrays must not overlap.
struct Words {
    const int32_t* p;
    long long n;
    bool overlaps(const Words& o) const {
        if (!p || !o.p || n < 1 || o.n < 1) return false;
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
        return a < b ? b - a < (uintptr_t)n * 4 : a - b < (uintptr_t)o.n * 4;
    }
};

bool batch_ok(int batch, int num_kv_heads) {
    return batch >= 1 && batch <= HPC_MAX_BATCH && num_kv_heads >= 1 && num_kv_heads <= HPC_MAX_KV_HEADS;
}

hpc_status pages_check(int kv_dtype, int num_pages, int num_kv_heads) {
    if (kv_dtype != HPC_KV_BF16 && kv_dtype != HPC_KV_FP8_E4M3) return HPC_ERR_UNSUPPORTED;
    // token and scale-row coordinates, one page past the pool included
    if (num_pages < 1 || ((long long)num_pages + 1) * kChunk > 2147483647LL ||
        ((long long)num_pages + 1) * num_kv_heads > 2147483647LL)
        return HPC_ERR_INVALID_ARG;
    return HPC_OK;
}

}  // namespace

extern "C" {

hpc_status hpc_attn_weights(const void* q, const void* k_cache, const float* k_scale, int kv_dtype, int num_pages,
                            const int32_t* page_table, int page_table_stride, const int32_t* q_starts,
                            const int32_t* seq_lens, const int32_t* row_counts, int window, const float* lse, int batch,
                            int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int page_size, float decay,
                            float* weights, long long weights_stride, int* d_error_word, void* stream) {
    if (num_q_heads < 1 || !batch_ok(batch, num_kv_heads)) return HPC_ERR_INVALID_ARG;
    if (head_dim != kHeadDim || page_size != kChunk || num_q_heads != kGroup * num_kv_heads) return HPC_ERR_UNSUPPORTED;
    const hpc_status st = pages_check(kv_dtype, num_pages, num_kv_heads);
    if (st != HPC_OK) return st;
    const bool fp8 = kv_dtype == HPC_KV_FP8_E4M3;
    if (!k_cache || !aligned(k_cache, 16) || (fp8 && (!k_scale || !aligned(k_scale, 16)))) return HPC_ERR_INVALID_ARG;
    if (!page_table || page_table_stride < 1 || page_table_stride > (1 << 24)) return HPC_ERR_INVALID_ARG;  // up to 2^30 tokens
    if (!seq_lens || !weights || window < 0 || num_tokens < 0) return HPC_ERR_INVALID_ARG;
    if (!(decay >= 0.f && decay <= 1.f)) return HPC_ERR_INVALID_ARG;
    if (weights_stride < (long long)page_table_stride * kChunk) return HPC_ERR_INVALID_ARG;
    if (!q_starts && num_tokens % batch != 0) return HPC_ERR_INVALID_ARG;
    if (num_tokens == 0) return HPC_OK;  // no sequence has rows
    if (!q || !aligned(q, 16) || !lse) return HPC_ERR_INVALID_ARG;
    AttnWeightsArgs a;
    a.q = q;
    a.k_cache = k_cache;
    a.k_scale = fp8 ? k_scale : nullptr;
    a.fp8 = fp8;
    a.num_pages = num_pages;
    a.page_table = page_table;
    a.pt_stride = page_table_stride;
    a.q_starts = q_starts;
    a.rows_per_seq = num_tokens / batch;
    a.seq_lens = seq_lens;
    a.counts = row_counts;
    a.window = window;
    a.lse = lse;
    a.batch = batch;
    a.num_tokens = num_tokens;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.decay = decay;
    a.weights = weights;
    a.w_stride = weights_stride;
    a.err = d_error_word;
    return launched(launch_attn_weights(a, static_cast<cudaStream_t>(stream)));
}

hpc_status hpc_kv_select(const float* weights, long long weights_stride, const int32_t* seq_lens, int batch,
                         int num_kv_heads, int budget, int num_first, int num_recent, int32_t* keep, int32_t* keep_lens,
                         int* d_error_word, void* stream) {
    if (!batch_ok(batch, num_kv_heads) || !weights || !seq_lens || !keep || !keep_lens) return HPC_ERR_INVALID_ARG;
    if (weights_stride < 1 || weights_stride > (1LL << 30) || budget < 1 || budget > (1 << 30)) return HPC_ERR_INVALID_ARG;
    if (num_first < 0 || num_recent < 0 || (long long)num_first + num_recent > budget) return HPC_ERR_INVALID_ARG;
    // (every head's CTAs read the lengths)
    const Words lens{seq_lens, batch}, kept{keep_lens, batch}, all{keep, (long long)batch * num_kv_heads * budget};
    if (kept.overlaps(lens) || all.overlaps(lens) || all.overlaps(kept)) return HPC_ERR_INVALID_ARG;
    const KvSelectArgs a{weights, weights_stride, seq_lens, batch, num_kv_heads, budget, num_first, num_recent, keep, keep_lens,
                         d_error_word};
    return launched(launch_kv_select(a, static_cast<cudaStream_t>(stream)));
}

hpc_status hpc_kv_compact(void* k_cache, void* v_cache, float* k_scale, float* v_scale, int kv_dtype, int num_pages,
                          const int32_t* page_table, int page_table_stride, const int32_t* keep, int keep_stride,
                          const int32_t* keep_lens, const int32_t* new_table, int new_table_stride, int batch,
                          int num_kv_heads, int head_dim, int page_size, const float* weights, long long weights_stride,
                          float* new_weights, long long new_weights_stride, int* d_error_word, void* stream) {
    if (head_dim != kHeadDim || page_size != kChunk) return HPC_ERR_UNSUPPORTED;
    if (!batch_ok(batch, num_kv_heads)) return HPC_ERR_INVALID_ARG;
    const hpc_status st = pages_check(kv_dtype, num_pages, num_kv_heads);
    if (st != HPC_OK) return st;
    const bool fp8 = kv_dtype == HPC_KV_FP8_E4M3;
    if (!k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return HPC_ERR_INVALID_ARG;
    if (fp8 && (!k_scale || !v_scale)) return HPC_ERR_INVALID_ARG;
    if (!page_table || page_table_stride < 1 || !keep || keep_stride < 1 || !keep_lens || !new_table || new_table_stride < 1)
        return HPC_ERR_INVALID_ARG;
    if (keep_stride > (1 << 30) || !weights != !new_weights) return HPC_ERR_INVALID_ARG;
    if (weights) {
        const long long room = (long long)new_table_stride * kChunk;
        if (weights_stride < (long long)page_table_stride * kChunk || weights == new_weights) return HPC_ERR_INVALID_ARG;
        if (new_weights_stride < (keep_stride < room ? keep_stride : room)) return HPC_ERR_INVALID_ARG;
    }
    KvCompactArgs a;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.num_pages = num_pages;
    a.page_table = page_table;
    a.pt_stride = page_table_stride;
    a.keep = keep;
    a.keep_stride = keep_stride;
    a.keep_lens = keep_lens;
    a.dst_table = new_table;
    a.dst_stride = new_table_stride;
    a.batch = batch;
    a.num_kv_heads = num_kv_heads;
    a.weights = weights;
    a.w_stride = weights_stride;
    a.weights_out = new_weights;
    a.w_out_stride = new_weights_stride;
    a.err = d_error_word;
    return launched(launch_kv_compact(a, fp8, static_cast<cudaStream_t>(stream)));
}

hpc_status hpc_verify_drafts(const void* target_probs, long long target_stride, const void* draft_probs,
                             long long draft_stride, int probs_dtype, const int32_t* draft_tokens,
                             const int32_t* draft_counts, const float* accept_rand, const float* sample_rand, int batch,
                             int num_drafts, int vocab, int32_t* num_accepted, int32_t* tokens, const int32_t* seq_lens,
                             int32_t* kept_lens, int* d_error_word, void* stream) {
    if (batch < 1 || batch > HPC_MAX_BATCH || num_drafts < 0 || num_drafts > HPC_MAX_DRAFTS || vocab < 1) return HPC_ERR_INVALID_ARG;
    if (probs_dtype != HPC_PROBS_F32 && probs_dtype != HPC_PROBS_BF16) return HPC_ERR_UNSUPPORTED;
    const size_t size = probs_dtype == HPC_PROBS_BF16 ? 2 : 4;
    if (!target_probs || !aligned(target_probs, size) || target_stride < vocab) return HPC_ERR_INVALID_ARG;
    if (num_drafts > 0) {
        if (draft_probs && (!aligned(draft_probs, size) || draft_stride < vocab)) return HPC_ERR_INVALID_ARG;
        if (!draft_tokens || !accept_rand) return HPC_ERR_INVALID_ARG;
    }
    if (!sample_rand || !num_accepted || !tokens || (kept_lens && !seq_lens)) return HPC_ERR_INVALID_ARG;
    // All of a request's CTAs read its count and its drafts; its lengths the one that writes the new ones.
    const Words drafted{draft_tokens, (long long)batch * num_drafts}, counts{draft_counts, batch}, lens{kept_lens ? seq_lens : nullptr, batch};
    const Words acc{num_accepted, batch}, kept{kept_lens, batch}, out{tokens, (long long)batch * (num_drafts + 1)};
    if (acc.overlaps(drafted) || acc.overlaps(counts) || acc.overlaps(lens) || acc.overlaps(kept) || acc.overlaps(out))
        return HPC_ERR_INVALID_ARG;
    if (kept.overlaps(drafted) || kept.overlaps(counts) || kept.overlaps(out) || (kept.overlaps(lens) && kept_lens != seq_lens))
        return HPC_ERR_INVALID_ARG;
    if (out.overlaps(counts) || out.overlaps(lens)) return HPC_ERR_INVALID_ARG;
    // One request's tokens may take the place of its drafts: what is written there before they are read is what was there.
    if (out.overlaps(drafted) && (batch > 1 || tokens != draft_tokens)) return HPC_ERR_INVALID_ARG;
    VerifyArgs a;
    a.target = target_probs;
    a.target_stride = target_stride;
    a.draft = num_drafts > 0 ? draft_probs : nullptr;
    a.draft_stride = draft_stride;
    a.drafted = draft_tokens;
    a.counts = draft_counts;
    a.accept_rand = accept_rand;
    a.sample_rand = sample_rand;
    a.batch = batch;
    a.drafts = num_drafts;
    a.vocab = vocab;
    a.accepted = num_accepted;
    a.tokens = tokens;
    a.seq_lens = seq_lens;
    a.kept_lens = kept_lens;
    a.err = d_error_word;
    return launched(launch_verify(a, probs_dtype == HPC_PROBS_BF16, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
