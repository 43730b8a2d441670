// extern "C" entry points of libspecverify.so: argument checks, workspace
// sizing and error reporting around the kernels' launchers.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <string>

#include "sv_internal.h"

namespace {

thread_local std::string g_last_error;
std::atomic<int> g_wait_tries{sv::kWaitTries};

sv_status fail(sv_status s, const std::string& msg) {
  g_last_error = msg;
  // a launch that failed leaves its error for the next cudaGetLastError(), which would be a good call's
  if (s == SV_ERR_CUDA) (void)cudaGetLastError();
  return s;
}

constexpr int kMaxK = 20;
constexpr long long kMaxItems = 0x7fffffffLL / 16;  // items per call: the grid is items x <= 16 CTAs
constexpr int kMaxSeqs = 1 << 30;                   // one thread per sequence
constexpr int kMaxRows = 1 << 30;                   // rows of an attention or linear call

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

extern "C" {

int sv_version(void) { return 100; }

size_t sv_workspace_size(int B, int K, int V, sv_dtype dt) {
  if (B < 1 || K < 0 || K > kMaxK || V < 1 || (dt != SV_F32 && dt != SV_BF16)) return 0;
  return sv::verify_workspace_bytes(B, K);
}

size_t sv_lmhead_workspace_size(int M, int H) {
  if (M < 1 || H < 1) return 0;
  return sv::lmhead_workspace_bytes(M, H);
}

// Host-checkable arguments of the three verify entry points; fills *L with
// everything but the workspace.
static sv_status verify_args(const void* target_logits, int64_t target_seq_stride,
                             int64_t target_pos_stride, const void* draft_logits,
                             int64_t draft_seq_stride, int64_t draft_pos_stride, sv_dtype dtype,
                             int B, int K, int V, const int32_t* draft_tokens,
                             const int32_t* k_per_row, const float* temperature, float top_p,
                             const float* uniforms, const uint8_t* mode, int32_t* out_tokens,
                             int32_t* n_accepted, float* diag, void* stream,
                             sv::VerifyLaunch* L) {
  if (dtype != SV_F32 && dtype != SV_BF16) return fail(SV_ERR_DTYPE, "dtype must be SV_F32 or SV_BF16");
  if (B < 1 || K < 0 || K > kMaxK || V < 1)
    return fail(SV_ERR_SHAPE, "need B >= 1, 0 <= K <= 20, V >= 1");
  // one cluster of up to 16 CTAs per (sequence, position): the grid must fit 2^31 - 1 blocks
  if ((long long)B * (K + 1) > kMaxItems)
    return fail(SV_ERR_SHAPE, "B * (K + 1) must be at most 134217727");
  if (!target_logits || !uniforms || !out_tokens || !n_accepted)
    return fail(SV_ERR_ARG, "target_logits, uniforms, out_tokens and n_accepted are required");
  if (K > 0 && !draft_tokens) return fail(SV_ERR_ARG, "draft_tokens is required when K > 0");
  if (K > 0 && !draft_logits && !mode)
    return fail(SV_ERR_ARG, "draft_logits may be NULL only when every row is greedy (mode given)");
  if (!(top_p > 0.0f && top_p <= 1.0f)) return fail(SV_ERR_ARG, "top_p must be in (0, 1]");
  const int es = dtype == SV_BF16 ? 2 : 4;
  if (!aligned(target_logits, es) || (draft_logits && !aligned(draft_logits, es)))
    return fail(SV_ERR_ARG, "logit pointers must be aligned to their element size");
  const long long Vl = V;
  const long long ts = target_seq_stride ? target_seq_stride : (long long)(K + 1) * Vl;
  const long long tp = target_pos_stride ? target_pos_stride : Vl;
  const long long ds = draft_seq_stride ? draft_seq_stride : (long long)K * Vl;
  const long long dp = draft_pos_stride ? draft_pos_stride : Vl;
  if (ts < 0 || tp < 0 || ds < 0 || dp < 0) return fail(SV_ERR_SHAPE, "strides must be >= 0");
  if (tp < Vl && K > 0) return fail(SV_ERR_SHAPE, "target position stride is smaller than V");
  if (dp < Vl && K > 1) return fail(SV_ERR_SHAPE, "draft position stride is smaller than V");
  L->target = target_logits;
  L->t_seq = ts;
  L->t_pos = tp;
  L->draft = draft_logits;
  L->d_seq = ds;
  L->d_pos = dp;
  L->dtype = dtype;
  L->B = B;
  L->K = K;
  L->V = V;
  L->tokens = draft_tokens;
  L->kpr = k_per_row;
  L->temp = temperature;
  L->top_p = top_p;
  L->unif = uniforms;
  L->mode = mode;
  L->out = out_tokens;
  L->nacc = n_accepted;
  L->diag = diag;
  L->workspace = nullptr;
  L->stream = stream;
  return SV_OK;
}

static sv_status spec_verify_impl(const void* target_logits, int64_t target_seq_stride,
                                  int64_t target_pos_stride, const void* draft_logits,
                                  int64_t draft_seq_stride, int64_t draft_pos_stride,
                                  sv_dtype dtype, int B, int K, int V, const int32_t* draft_tokens,
                                  const int32_t* k_per_row, const float* temperature, float top_p,
                                  const float* uniforms, const uint8_t* mode, int32_t* out_tokens,
                                  int32_t* n_accepted, float* diag, void* workspace,
                                  size_t workspace_bytes, void* stream, int topp_draft) {
  sv::VerifyLaunch L;
  const sv_status a = verify_args(target_logits, target_seq_stride, target_pos_stride,
                                  draft_logits, draft_seq_stride, draft_pos_stride, dtype, B, K,
                                  V, draft_tokens, k_per_row, temperature, top_p, uniforms, mode,
                                  out_tokens, n_accepted, diag, stream, &L);
  if (a != SV_OK) return a;
  if (!workspace || !aligned(workspace, 256))
    return fail(SV_ERR_WORKSPACE, "workspace must be non-NULL and 256-byte aligned");
  if (workspace_bytes < sv::verify_workspace_bytes(B, K))
    return fail(SV_ERR_WORKSPACE, "workspace smaller than sv_workspace_size()");
  L.workspace = workspace;
  L.topp_draft = topp_draft;
  std::string err;
  int s = sv::verify_launch(L, &err);
  if (s != SV_OK) return fail(static_cast<sv_status>(s), err);
  return SV_OK;
}

sv_status sv_spec_verify(const void* target_logits, int64_t target_seq_stride,
                         int64_t target_pos_stride, const void* draft_logits,
                         int64_t draft_seq_stride, int64_t draft_pos_stride, sv_dtype dtype,
                         int B, int K, int V, const int32_t* draft_tokens,
                         const int32_t* k_per_row, const float* temperature, float top_p,
                         const float* uniforms, const uint8_t* mode, int32_t* out_tokens,
                         int32_t* n_accepted, float* diag, void* workspace,
                         size_t workspace_bytes, void* stream) {
  return spec_verify_impl(target_logits, target_seq_stride, target_pos_stride, draft_logits,
                          draft_seq_stride, draft_pos_stride, dtype, B, K, V, draft_tokens,
                          k_per_row, temperature, top_p, uniforms, mode, out_tokens, n_accepted,
                          diag, workspace, workspace_bytes, stream, 1);
}

sv_status sv_spec_verify_target_topp(const void* target_logits, int64_t target_seq_stride,
                                     int64_t target_pos_stride, const void* draft_logits,
                                     int64_t draft_seq_stride, int64_t draft_pos_stride,
                                     sv_dtype dtype, int B, int K, int V,
                                     const int32_t* draft_tokens, const int32_t* k_per_row,
                                     const float* temperature, float top_p, const float* uniforms,
                                     const uint8_t* mode, int32_t* out_tokens, int32_t* n_accepted,
                                     float* diag, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  return spec_verify_impl(target_logits, target_seq_stride, target_pos_stride, draft_logits,
                          draft_seq_stride, draft_pos_stride, dtype, B, K, V, draft_tokens,
                          k_per_row, temperature, top_p, uniforms, mode, out_tokens, n_accepted,
                          diag, workspace, workspace_bytes, stream, 0);
}

sv_status sv_spec_verify_noalloc(const void* target_logits, int64_t target_seq_stride,
                                 int64_t target_pos_stride, const void* draft_logits,
                                 int64_t draft_seq_stride, int64_t draft_pos_stride,
                                 sv_dtype dtype, int B, int K, int V, const int32_t* draft_tokens,
                                 const int32_t* k_per_row, const float* temperature, float top_p,
                                 const float* uniforms, const uint8_t* mode, int32_t* out_tokens,
                                 int32_t* n_accepted, float* diag, void* stream) {
  sv::VerifyLaunch L;
  const sv_status a = verify_args(target_logits, target_seq_stride, target_pos_stride,
                                  draft_logits, draft_seq_stride, draft_pos_stride, dtype, B, K,
                                  V, draft_tokens, k_per_row, temperature, top_p, uniforms, mode,
                                  out_tokens, n_accepted, diag, stream, &L);
  if (a != SV_OK) return a;
  std::string err;
  int s = sv::verify_launch_noalloc(L, &err);
  if (s != SV_OK) return fail(static_cast<sv_status>(s), err);
  return SV_OK;
}

sv_status sv_kv_commit(int32_t* seq_lens, const int32_t* n_accepted, const int32_t* capacity,
                       const int32_t* k_per_row, int B, int K, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (B < 1 || B > kMaxSeqs) return fail(SV_ERR_SHAPE, "need 1 <= B <= 2^30");
  if (!seq_lens || !n_accepted) return fail(SV_ERR_ARG, "seq_lens and n_accepted are required");
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < 256)
    return fail(SV_ERR_WORKSPACE, "workspace must be non-NULL, 256-byte aligned, >= 256 bytes");
  std::string err;
  int s = sv::commit_launch(seq_lens, n_accepted, capacity, k_per_row, B, K,
                            static_cast<uint32_t*>(workspace), stream, &err);
  if (s != SV_OK) return fail(static_cast<sv_status>(s), err);
  return SV_OK;
}

sv_status sv_kv_commit_paged(int32_t* seq_lens, const int32_t* n_accepted,
                             const int32_t* k_per_row, int32_t* block_table, int max_pages,
                             int page_size, int32_t* free_pages, int32_t* free_top,
                             int free_capacity, int B, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (B < 1 || B > kMaxSeqs || max_pages < 1 || page_size < 1 || free_capacity < 0)
    return fail(SV_ERR_SHAPE, "need 1 <= B <= 2^30, max_pages >= 1, page_size >= 1, free_capacity >= 0");
  // lengths and page counts are int32 on the device: a full table plus one page must fit
  if ((long long)max_pages * page_size + page_size > 0x7fffffffLL)
    return fail(SV_ERR_SHAPE, "(max_pages + 1) * page_size must fit in int32");
  if (!seq_lens || !n_accepted || !k_per_row || !block_table || !free_pages || !free_top)
    return fail(SV_ERR_ARG, "every array argument is required");
  if (!workspace || workspace_bytes < 16 || !aligned(workspace, 16))
    return fail(SV_ERR_WORKSPACE, "workspace must be non-NULL, 16-byte aligned and >= 16 bytes");
  std::string err;
  const int s = sv::paged_commit_launch(seq_lens, n_accepted, k_per_row, block_table, max_pages,
                                        page_size, free_pages, free_top, free_capacity, B,
                                        static_cast<uint32_t*>(workspace), stream, &err);
  if (s != SV_OK) return fail(static_cast<sv_status>(s), err);
  return SV_OK;
}

size_t sv_dynk_state_size(int B) { return B < 1 || B > kMaxSeqs ? 0 : sv::dynk_state_bytes(B); }

sv_status sv_dynk_init(void* state, int B, int k0, void* stream) {
  if (B < 1 || B > kMaxSeqs) return fail(SV_ERR_SHAPE, "need 1 <= B <= 2^30");
  if (!state || !aligned(state, 16)) return fail(SV_ERR_ARG, "state must be non-NULL and 16-byte aligned");
  std::string err;
  const int s = sv::dynk_init_launch(state, B, k0, stream, &err);
  if (s != SV_OK) return fail(static_cast<sv_status>(s), err);
  return SV_OK;
}

sv_status sv_dynk_update(void* state, int B, const int32_t* n_accepted, const int32_t* k_used,
                         const int32_t* cap, int32_t* k_next, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (B < 1 || B > kMaxSeqs) return fail(SV_ERR_SHAPE, "need 1 <= B <= 2^30");
  if (!state || !aligned(state, 16)) return fail(SV_ERR_ARG, "state must be non-NULL and 16-byte aligned");
  if (!n_accepted || !k_used || !k_next) return fail(SV_ERR_ARG, "n_accepted, k_used and k_next are required");
  if (!workspace || workspace_bytes < 4 || !aligned(workspace, 4))
    return fail(SV_ERR_WORKSPACE, "workspace (its flag word) must be non-NULL, aligned, >= 4 bytes");
  std::string err;
  const int s = sv::dynk_update_launch(state, B, n_accepted, k_used, cap, k_next,
                                       static_cast<uint32_t*>(workspace), stream, &err);
  if (s != SV_OK) return fail(static_cast<sv_status>(s), err);
  return SV_OK;
}

size_t sv_draft_sample_workspace_size(void) { return 256; }

sv_status sv_draft_sample(const void* draft_logits, int64_t seq_stride, int64_t pos_stride,
                          sv_dtype dtype, int B, int K, int V, const int32_t* k_per_row,
                          const float* temperature, float top_p, const float* uniforms,
                          const uint8_t* mode, int32_t* out_tokens, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return fail(SV_ERR_DTYPE, "dtype must be SV_F32 or SV_BF16");
  if (B < 1 || K < 1 || V < 1) return fail(SV_ERR_SHAPE, "need B >= 1, K >= 1, V >= 1");
  if ((long long)B * K > kMaxItems) return fail(SV_ERR_SHAPE, "B * K must be at most 134217727");
  if (!draft_logits || !uniforms || !out_tokens)
    return fail(SV_ERR_ARG, "draft_logits, uniforms and out_tokens are required");
  if (!(top_p > 0.0f && top_p <= 1.0f)) return fail(SV_ERR_ARG, "top_p must be in (0, 1]");
  const int es = dtype == SV_BF16 ? 2 : 4;
  if (!aligned(draft_logits, es)) return fail(SV_ERR_ARG, "logits must be aligned to their element size");
  const long long Vl = V;
  const long long ss = seq_stride ? seq_stride : (long long)K * Vl;
  const long long ps = pos_stride ? pos_stride : Vl;
  if (ss < 0 || ps < 0) return fail(SV_ERR_SHAPE, "strides must be >= 0");
  if (ps < Vl && K > 1) return fail(SV_ERR_SHAPE, "position stride is smaller than V");
  if (!workspace || !aligned(workspace, 256))
    return fail(SV_ERR_WORKSPACE, "workspace must be non-NULL and 256-byte aligned");
  if (workspace_bytes < sv_draft_sample_workspace_size())
    return fail(SV_ERR_WORKSPACE, "workspace smaller than sv_draft_sample_workspace_size()");
  sv::SampleLaunch L;
  L.logits = draft_logits;
  L.l_seq = ss;
  L.l_pos = ps;
  L.dtype = dtype;
  L.B = B;
  L.K = K;
  L.V = V;
  L.kpr = k_per_row;
  L.temp = temperature;
  L.top_p = top_p;
  L.unif = uniforms;
  L.mode = mode;
  L.out = out_tokens;
  L.workspace = workspace;
  L.stream = stream;
  std::string err;
  const int s = sv::sample_launch(L, &err);
  if (s != SV_OK) return fail(static_cast<sv_status>(s), err);
  return SV_OK;
}

sv_status sv_lmhead_rmsnorm(const void* hidden, const void* norm_w, float eps, const void* W,
                            void* logits, sv_dtype out_dtype, int M, int H, int V,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (out_dtype != SV_F32 && out_dtype != SV_BF16) return fail(SV_ERR_DTYPE, "bad out_dtype");
  if (M < 1 || H < 64 || H % 64 != 0 || V < 16 || V % 16 != 0)
    return fail(SV_ERR_SHAPE, "need M >= 1, H % 64 == 0, V % 16 == 0");
  if (!hidden || !norm_w || !W || !logits) return fail(SV_ERR_ARG, "null pointer");
  if (!(eps >= 0.0f)) return fail(SV_ERR_ARG, "eps must be >= 0");
  if (!aligned(hidden, 16) || !aligned(W, 16) || !aligned(logits, 16) || !aligned(norm_w, 2))
    return fail(SV_ERR_ARG, "hidden, W and logits must be 16-byte aligned");
  if (!workspace || !aligned(workspace, 256))
    return fail(SV_ERR_WORKSPACE, "workspace must be non-NULL and 256-byte aligned");
  if (workspace_bytes < sv::lmhead_workspace_bytes(M, H))
    return fail(SV_ERR_WORKSPACE, "workspace smaller than sv_lmhead_workspace_size()");
  std::string err;
  int s = sv::lmhead_launch(hidden, norm_w, eps, W, logits, out_dtype, M, H, V, workspace,
                            workspace_bytes, stream, &err);
  if (s != SV_OK) return fail(static_cast<sv_status>(s), err);
  return SV_OK;
}

// Shapes of the attention call, for its workspace too; NULL if they are in range.
static const char* attention_shape(int B, int K, int Hq, int Hkv, int D, long long prefix_len,
                                   long long max_own) {
  if (B < 1 || K < 0 || K > kMaxK || Hq < 1 || Hkv < 1 || prefix_len < 0 || max_own < 1)
    return "need B >= 1, 0 <= K <= 20, Hq >= 1, Hkv >= 1, prefix_len >= 0";
  if (D != 64 && D != 128) return "D must be 64 or 128";
  if (Hq % Hkv != 0 || Hq / Hkv > 64) return "Hq must be a multiple of Hkv, at most 64 times";
  if ((long long)B * (K + 1) > kMaxRows / Hq) return "B * (K + 1) * Hq must be at most 2^30";
  if (prefix_len + max_own > 0x7fffffffLL - 4096) return "prefix_len + max_pages * page_size must fit in int32";
  return nullptr;
}

size_t sv_prefix_attention_workspace_size(int B, int K, int Hq, int Hkv, int D, int prefix_len,
                                          int max_own_len) {
  if (attention_shape(B, K, Hq, Hkv, D, prefix_len, max_own_len)) return 0;
  return sv::attention_workspace_bytes(B, K, Hq, Hkv, D, prefix_len, max_own_len);
}

sv_status sv_prefix_attention(const void* q, int64_t q_seq_stride, int64_t q_pos_stride,
                              int64_t q_head_stride, const void* k_pool, const void* v_pool,
                              int64_t page_stride, int64_t token_stride, int64_t head_stride,
                              int num_pages, int page_size, const int32_t* prefix_pages,
                              int prefix_len, const int32_t* block_table, int max_pages,
                              const int32_t* seq_lens, const int32_t* k_per_row, float scale,
                              void* out, int64_t out_seq_stride, int64_t out_pos_stride,
                              int64_t out_head_stride, float* lse, sv_dtype dtype, int B, int K,
                              int Hq, int Hkv, int D, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (dtype != SV_BF16) return fail(SV_ERR_DTYPE, "dtype must be SV_BF16");
  if (max_pages < 1 || page_size < 1 || num_pages < 1)
    return fail(SV_ERR_SHAPE, "need max_pages >= 1, page_size >= 1, num_pages >= 1");
  const long long own = (long long)max_pages * page_size;
  if (const char* why = attention_shape(B, K, Hq, Hkv, D, prefix_len, own)) return fail(SV_ERR_SHAPE, why);
  if (!q || !k_pool || !v_pool || !block_table || !seq_lens || !out)
    return fail(SV_ERR_ARG, "q, k_pool, v_pool, block_table, seq_lens and out are required");
  if (prefix_len > 0 && !prefix_pages) return fail(SV_ERR_ARG, "prefix_pages is required when prefix_len > 0");
  // (its product with log2(e) is what the kernel uses)
  if (!(scale >= -0x1p127f && scale <= 0x1p127f)) return fail(SV_ERR_ARG, "scale must be within +-2^127");
  if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(out, 16))
    return fail(SV_ERR_ARG, "q, k_pool, v_pool and out must be 16-byte aligned");
  if (!aligned(lse, 4) || !aligned(prefix_pages, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(k_per_row, 4))
    return fail(SV_ERR_ARG, "lse and the index arrays must be aligned to their element size");
  sv::AttentionLaunch L;
  L.q = q;
  L.q_head = q_head_stride ? q_head_stride : D;
  L.q_pos = q_pos_stride ? q_pos_stride : (long long)Hq * D;
  L.q_seq = q_seq_stride ? q_seq_stride : (long long)(K + 1) * Hq * D;
  L.k = k_pool;
  L.v = v_pool;
  L.head = head_stride ? head_stride : D;
  L.token = token_stride ? token_stride : (long long)Hkv * D;
  L.page = page_stride ? page_stride : (long long)page_size * Hkv * D;
  L.out = out;
  L.o_head = out_head_stride ? out_head_stride : D;
  L.o_pos = out_pos_stride ? out_pos_stride : (long long)Hq * D;
  L.o_seq = out_seq_stride ? out_seq_stride : (long long)(K + 1) * Hq * D;
  for (long long s : {L.q_head, L.q_pos, L.q_seq, L.head, L.token, L.page, L.o_head, L.o_pos, L.o_seq})
    if (s < 0 || s % 8 != 0) return fail(SV_ERR_SHAPE, "strides must be >= 0 and multiples of 8 elements");
  if (L.o_head < D && Hq > 1) return fail(SV_ERR_SHAPE, "out head stride is smaller than D");
  L.num_pages = num_pages;
  L.page_size = page_size;
  L.prefix_pages = prefix_pages;
  L.prefix_len = prefix_len;
  L.table = block_table;
  L.max_pages = max_pages;
  L.lens = seq_lens;
  L.kpr = k_per_row;
  L.scale = scale;
  L.lse = lse;
  L.B = B;
  L.K = K;
  L.Hq = Hq;
  L.Hkv = Hkv;
  L.D = D;
  L.wait_tries = g_wait_tries.load(std::memory_order_relaxed);
  if (!workspace || !aligned(workspace, 256))
    return fail(SV_ERR_WORKSPACE, "workspace must be non-NULL and 256-byte aligned");
  if (workspace_bytes < sv::attention_workspace_bytes(B, K, Hq, Hkv, D, prefix_len, (int)own))
    return fail(SV_ERR_WORKSPACE, "workspace smaller than sv_prefix_attention_workspace_size()");
  L.workspace = workspace;
  L.stream = stream;
  std::string err;
  const int s = sv::attention_launch(L, &err);
  if (s != SV_OK) return fail(static_cast<sv_status>(s), err);
  return SV_OK;
}

sv_status sv_rmsnorm_residual(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                              const void* norm_w, float eps, void* residual_out, int64_t ldro,
                              sv_dtype dtype, void* out, int64_t ldo, sv_dtype out_dtype,
                              float* out_scale, int M, int H, void* stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return fail(SV_ERR_DTYPE, "dtype must be SV_F32 or SV_BF16");
  if (out_dtype != SV_BF16 && out_dtype != SV_E4M3)
    return fail(SV_ERR_DTYPE, "out_dtype must be SV_BF16 or SV_E4M3");
  if (M < 1 || H < 1) return fail(SV_ERR_SHAPE, "need M >= 1, H >= 1");
  if (!x || !norm_w || !out) return fail(SV_ERR_ARG, "x, norm_w and out are required");
  if (out_dtype == SV_E4M3 && !out_scale) return fail(SV_ERR_ARG, "out_scale is required for SV_E4M3");
  if (!(eps >= 0.0f)) return fail(SV_ERR_ARG, "eps must be >= 0");
  const size_t es = dtype == SV_BF16 ? 2 : 4;
  if (!aligned(x, es) || !aligned(residual, es) || !aligned(residual_out, es) || !aligned(norm_w, 2) ||
      !aligned(out, out_dtype == SV_BF16 ? 2 : 1) || !aligned(out_scale, 4))
    return fail(SV_ERR_ARG, "pointers must be aligned to their element size");
  sv::NormLaunch L;
  L.x = x;
  L.ldx = ldx ? ldx : H;
  L.residual = residual;
  L.ldr = ldr ? ldr : H;
  L.w = norm_w;
  L.eps = eps;
  L.residual_out = residual_out;
  L.ldro = ldro ? ldro : H;
  L.dtype = dtype;
  L.out = out;
  L.ldo = ldo ? ldo : H;
  L.out_dtype = out_dtype;
  L.out_scale = out_scale;
  L.M = M;
  L.H = H;
  L.stream = stream;
  L.wait_tries = g_wait_tries.load(std::memory_order_relaxed);
  if (L.ldx < H || L.ldr < H || L.ldro < H || L.ldo < H)
    return fail(SV_ERR_SHAPE, "row strides must be 0 or at least H");
  if ((residual_out == x && L.ldro != L.ldx) || (residual && residual_out == residual && L.ldro != L.ldr))
    return fail(SV_ERR_ARG, "residual_out over an input needs that input's row stride");
  if (out == x || (residual && out == residual) || out == residual_out)
    return fail(SV_ERR_ARG, "out must not be x, residual or residual_out");
  std::string err;
  const int s = sv::norm_launch(L, &err);
  if (s != SV_OK) return fail(static_cast<sv_status>(s), err);
  return SV_OK;
}

size_t sv_linear_workspace_size(int M, int N, int K) { return M < 1 || N < 1 || K < 1 ? 0 : 256; }

sv_status sv_linear(const void* x, int64_t ldx, const float* x_scale, const void* W, int64_t ldw,
                    const float* w_scale, sv_dtype in_dtype, const void* bias,
                    const void* residual, int64_t ldr, int act, void* out, int64_t ldo,
                    sv_dtype out_dtype, int M, int N, int K, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (in_dtype != SV_BF16 && in_dtype != SV_E4M3)
    return fail(SV_ERR_DTYPE, "in_dtype must be SV_BF16 or SV_E4M3");
  if (out_dtype != SV_F32 && out_dtype != SV_BF16)
    return fail(SV_ERR_DTYPE, "out_dtype must be SV_F32 or SV_BF16");
  if (M < 1 || N < 1 || K < 1 || M > kMaxRows || N > kMaxRows || K > kMaxRows)
    return fail(SV_ERR_SHAPE, "need M, N and K in 1 .. 2^30");
  if (act < SV_ACT_NONE || act > SV_ACT_GELU_TANH) return fail(SV_ERR_ARG, "unknown activation");
  if (!x || !W || !out) return fail(SV_ERR_ARG, "x, W and out are required");
  const int es = in_dtype == SV_BF16 ? 2 : 1, os = out_dtype == SV_BF16 ? 2 : 4;
  if (!aligned(x, 16) || !aligned(W, 16)) return fail(SV_ERR_ARG, "x and W must be 16-byte aligned");
  if (!aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 2) || !aligned(residual, os) ||
      !aligned(out, os))
    return fail(SV_ERR_ARG, "pointers must be aligned to their element size");
  sv::LinearLaunch L;
  L.x = x;
  L.ldx = ldx ? ldx : K;
  L.x_scale = x_scale;
  L.W = W;
  L.ldw = ldw ? ldw : K;
  L.w_scale = w_scale;
  L.in_dtype = in_dtype;
  L.bias = bias;
  L.residual = residual;
  L.ldr = ldr ? ldr : N;
  L.act = act;
  L.out = out;
  L.ldo = ldo ? ldo : N;
  L.out_dtype = out_dtype;
  L.M = M;
  L.N = N;
  L.K = K;
  if (L.ldx < K || L.ldw < K || L.ldr < N || L.ldo < N)
    return fail(SV_ERR_SHAPE, "row strides must be 0 or at least the row's length");
  // the tensor-map limits of the operand copies
  if (L.ldx * es % 16 != 0 || L.ldw * es % 16 != 0 || L.ldx >= (1LL << 38) || L.ldw >= (1LL << 38))
    return fail(SV_ERR_SHAPE, "row strides of x and W must be multiples of 16 bytes below 2^38 elements");
  if (residual == out && L.ldr != L.ldo) return fail(SV_ERR_ARG, "residual over out needs its row stride");
  if (out == x || out == W) return fail(SV_ERR_ARG, "out must not be x or W");
  if (!workspace || !aligned(workspace, 256))
    return fail(SV_ERR_WORKSPACE, "workspace must be non-NULL and 256-byte aligned");
  if (workspace_bytes < sv_linear_workspace_size(M, N, K))
    return fail(SV_ERR_WORKSPACE, "workspace smaller than sv_linear_workspace_size()");
  L.flags = static_cast<uint32_t*>(workspace);
  L.stream = stream;
  L.wait_tries = g_wait_tries.load(std::memory_order_relaxed);
  std::string err;
  const int s = sv::linear_launch(L, &err);
  if (s != SV_OK) return fail(static_cast<sv_status>(s), err);
  return SV_OK;
}

// Geometry of a 4-bit cache and of a call's tokens; NULL if it is in range.
static const char* kv4_shape(int num_pages, int page_size, int max_pages, int B, int Hkv, int D) {
  if (B < 1 || Hkv < 1 || num_pages < 1 || page_size < 1 || max_pages < 1)
    return "need B, Hkv, num_pages, page_size and max_pages >= 1";
  if (D != 64 && D != 128) return "D must be 64 or 128";
  if ((long long)max_pages * page_size > 0x7fffffffLL - 4096) return "max_pages * page_size must be at most 2^31 - 4096";
  if (sv_kv4_page_bytes(Hkv, D, page_size) == 0) return "a page must be below 2^31 bytes";
  return nullptr;
}

size_t sv_kv4_page_bytes(int Hkv, int D, int page_size) {
  if (Hkv < 1 || (D != 64 && D != 128) || page_size < 1) return 0;
  const size_t head = sv::kv4_head_bytes(D, page_size);
  return head > 0x7fffffff / (size_t)Hkv ? 0 : head * Hkv;
}

static sv_status kv4_rows(const void* k_in, const void* v_in, void* k_out, void* v_out, int64_t seq_stride,
                          int64_t pos_stride, int64_t head_stride, sv_dtype dtype, const void* pool, int num_pages,
                          int page_size, const int32_t* block_table, int max_pages, const int32_t* starts,
                          const int32_t* n_per_row, int B, int T, int Hkv, int D, void* workspace,
                          size_t workspace_bytes, void* stream, bool append) {
  if (dtype != SV_BF16 && (append || dtype != SV_F32))
    return fail(SV_ERR_DTYPE, append ? "dtype must be SV_BF16" : "dtype must be SV_BF16 or SV_F32");
  if (T < 1) return fail(SV_ERR_SHAPE, "need T >= 1");
  if (const char* why = kv4_shape(num_pages, page_size, max_pages, B, Hkv, D)) return fail(SV_ERR_SHAPE, why);
  if ((long long)B * T > (1LL << 40) / Hkv) return fail(SV_ERR_SHAPE, "B * T * Hkv must be at most 2^40");
  const void* k = append ? k_in : k_out;
  const void* v = append ? v_in : v_out;
  if (!k || !v || !pool || !block_table || !starts)
    return fail(SV_ERR_ARG, "keys, values, pool, block_table and starts are required");
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(pool, 16))
    return fail(SV_ERR_ARG, "keys, values and pool must be 16-byte aligned");
  if (!aligned(block_table, 4) || !aligned(starts, 4) || !aligned(n_per_row, 4))
    return fail(SV_ERR_ARG, "the index arrays must be aligned to their element size");
  sv::Kv4RowsLaunch L;
  L.c = {const_cast<void*>(pool), num_pages, page_size, block_table, max_pages, Hkv};
  L.k_in = k_in;
  L.v_in = v_in;
  L.k_out = k_out;
  L.v_out = v_out;
  L.head = head_stride ? head_stride : D;
  L.pos = pos_stride ? pos_stride : (long long)Hkv * D;
  L.seq = seq_stride ? seq_stride : (long long)T * Hkv * D;
  for (long long s : {L.head, L.pos, L.seq})
    if (s < 0 || s % 8 != 0) return fail(SV_ERR_SHAPE, "strides must be >= 0 and multiples of 8 elements");
  if (!append && ((Hkv > 1 && L.head < D) || k_out == v_out))
    return fail(SV_ERR_SHAPE, "outputs must not overlap");
  L.dtype = dtype;
  L.starts = starts;
  L.n_per_row = n_per_row;
  L.B = B;
  L.T = T;
  L.D = D;
  if (!workspace || !aligned(workspace, 4) || workspace_bytes < 4)
    return fail(SV_ERR_WORKSPACE, "workspace (its flag word) must be non-NULL, aligned, >= 4 bytes");
  L.flags = static_cast<uint32_t*>(workspace);
  L.stream = stream;
  std::string err;
  const int s = sv::kv4_rows_launch(L, &err);
  if (s != SV_OK) return fail(static_cast<sv_status>(s), err);
  return SV_OK;
}

sv_status sv_kv4_append(const void* k, const void* v, int64_t seq_stride, int64_t pos_stride, int64_t head_stride,
                        sv_dtype dtype, void* pool, int num_pages, int page_size, const int32_t* block_table,
                        int max_pages, const int32_t* starts, const int32_t* n_per_row, int B, int T, int Hkv, int D,
                        void* workspace, size_t workspace_bytes, void* stream) {
  return kv4_rows(k, v, nullptr, nullptr, seq_stride, pos_stride, head_stride, dtype, pool, num_pages, page_size,
                  block_table, max_pages, starts, n_per_row, B, T, Hkv, D, workspace, workspace_bytes, stream, true);
}

sv_status sv_kv4_read(const void* pool, int num_pages, int page_size, const int32_t* block_table, int max_pages,
                      const int32_t* starts, const int32_t* n_per_row, void* k_out, void* v_out, int64_t seq_stride,
                      int64_t pos_stride, int64_t head_stride, sv_dtype dtype, int B, int T, int Hkv, int D,
                      void* workspace, size_t workspace_bytes, void* stream) {
  return kv4_rows(nullptr, nullptr, k_out, v_out, seq_stride, pos_stride, head_stride, dtype, pool, num_pages,
                  page_size, block_table, max_pages, starts, n_per_row, B, T, Hkv, D, workspace, workspace_bytes,
                  stream, false);
}

static const char* kv4_attention_shape(int B, int K, int Hq, int Hkv, int D) {
  return attention_shape(B, K, Hq, Hkv, D, 0, 1);
}

size_t sv_kv4_attention_workspace_size(int B, int K, int Hq, int Hkv, int D) {
  return kv4_attention_shape(B, K, Hq, Hkv, D) ? 0 : sv::kv4_attention_workspace_bytes(K, Hq, Hkv, D);
}

sv_status sv_kv4_attention(const void* q, int64_t q_seq_stride, int64_t q_pos_stride, int64_t q_head_stride,
                           const void* pool, int num_pages, int page_size, const int32_t* block_table, int max_pages,
                           const int32_t* seq_lens, const int32_t* k_per_row, int window, int sinks, float scale,
                           void* out, int64_t out_seq_stride, int64_t out_pos_stride, int64_t out_head_stride,
                           float* lse, sv_dtype dtype, int B, int K, int Hq, int Hkv, int D, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (dtype != SV_BF16) return fail(SV_ERR_DTYPE, "dtype must be SV_BF16");
  if (const char* why = kv4_attention_shape(B, K, Hq, Hkv, D)) return fail(SV_ERR_SHAPE, why);
  if (const char* why = kv4_shape(num_pages, page_size, max_pages, B, Hkv, D)) return fail(SV_ERR_SHAPE, why);
  if (window < 0 || sinks < 0) return fail(SV_ERR_SHAPE, "window and sinks must be >= 0");
  if (!q || !pool || !block_table || !seq_lens || !out)
    return fail(SV_ERR_ARG, "q, pool, block_table, seq_lens and out are required");
  if (!(scale > -0x1p64f && scale < 0x1p64f)) return fail(SV_ERR_ARG, "scale must be within +-2^64");
  if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(out, 16))
    return fail(SV_ERR_ARG, "q, pool and out must be 16-byte aligned");
  if (!aligned(lse, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(k_per_row, 4))
    return fail(SV_ERR_ARG, "lse and the index arrays must be aligned to their element size");
  sv::Kv4AttentionLaunch L;
  L.c = {const_cast<void*>(pool), num_pages, page_size, block_table, max_pages, Hkv};
  L.q = q;
  L.q_head = q_head_stride ? q_head_stride : D;
  L.q_pos = q_pos_stride ? q_pos_stride : (long long)Hq * D;
  L.q_seq = q_seq_stride ? q_seq_stride : (long long)(K + 1) * Hq * D;
  L.out = out;
  L.o_head = out_head_stride ? out_head_stride : D;
  L.o_pos = out_pos_stride ? out_pos_stride : (long long)Hq * D;
  L.o_seq = out_seq_stride ? out_seq_stride : (long long)(K + 1) * Hq * D;
  for (long long s : {L.q_head, L.q_pos, L.q_seq, L.o_head, L.o_pos, L.o_seq})
    if (s < 0 || s % 8 != 0) return fail(SV_ERR_SHAPE, "strides must be >= 0 and multiples of 8 elements");
  if (L.o_head < D && Hq > 1) return fail(SV_ERR_SHAPE, "out head stride is smaller than D");
  L.lens = seq_lens;
  L.kpr = k_per_row;
  L.window = window;
  L.sinks = sinks;
  L.scale = scale;
  L.lse = lse;
  L.B = B;
  L.K = K;
  L.Hq = Hq;
  L.D = D;
  if (!workspace || !aligned(workspace, 256))
    return fail(SV_ERR_WORKSPACE, "workspace must be non-NULL and 256-byte aligned");
  if (workspace_bytes < sv::kv4_attention_workspace_bytes(K, Hq, Hkv, D))
    return fail(SV_ERR_WORKSPACE, "workspace smaller than sv_kv4_attention_workspace_size()");
  L.workspace = workspace;
  L.wait_tries = g_wait_tries.load(std::memory_order_relaxed);
  L.stream = stream;
  std::string err;
  const int s = sv::kv4_attention_launch(L, &err);
  if (s != SV_OK) return fail(static_cast<sv_status>(s), err);
  return SV_OK;
}

size_t sv_linear_w4_workspace_size(int M, int N, int K) {
  if (M < 1 || N < 1 || K < 1 || M > kMaxRows || N > kMaxRows || K > kMaxRows) return 0;
  return sv::linear_w4_workspace_bytes(M, N, K);
}

sv_status sv_linear_w4(const void* x, int64_t ldx, const void* W, int64_t ldw, const void* scales,
                       const uint8_t* zeros, int group, const void* bias, const void* residual, int64_t ldr, int act,
                       void* out, int64_t ldo, sv_dtype out_dtype, int M, int N, int K, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (out_dtype != SV_BF16 && out_dtype != SV_F32) return fail(SV_ERR_DTYPE, "out_dtype must be SV_BF16 or SV_F32");
  if (M < 1 || N < 1 || K < 1 || M > kMaxRows || N > kMaxRows || K > kMaxRows)
    return fail(SV_ERR_SHAPE, "M, N and K must be in 1 .. 2^30");
  if (group != 32 && group != 64 && group != 128) return fail(SV_ERR_SHAPE, "group must be 32, 64 or 128");
  if (K % group != 0) return fail(SV_ERR_SHAPE, "K must be a multiple of group");
  if ((long long)N * (K / group) > 0x7fffffffLL) return fail(SV_ERR_SHAPE, "N * K / group must be below 2^31");
  if (act < SV_ACT_NONE || act > SV_ACT_GELU_TANH) return fail(SV_ERR_ARG, "unknown activation");
  if (!x || !W || !scales || !out) return fail(SV_ERR_ARG, "x, W, scales and out are required");
  const int os = out_dtype == SV_BF16 ? 2 : 4;
  if (!aligned(x, 16) || !aligned(W, 16)) return fail(SV_ERR_ARG, "x and W must be 16-byte aligned");
  if (!aligned(scales, 2) || !aligned(bias, 2) || !aligned(residual, os) || !aligned(out, os))
    return fail(SV_ERR_ARG, "pointers must be aligned to their element size");
  sv::LinearW4Launch L;
  L.x = x;
  L.ldx = ldx ? ldx : K;
  L.W = W;
  L.ldw = ldw ? ldw : K / 2;
  L.scales = scales;
  L.zeros = zeros;
  L.group = group;
  L.bias = bias;
  L.residual = residual;
  L.ldr = ldr ? ldr : N;
  L.act = act;
  L.out = out;
  L.ldo = ldo ? ldo : N;
  L.out_dtype = out_dtype;
  L.M = M;
  L.N = N;
  L.K = K;
  if (L.ldx < K || L.ldw < K / 2 || L.ldr < N || L.ldo < N)
    return fail(SV_ERR_SHAPE, "row strides must be 0 or at least the row's length");
  // the tensor-map limits of the operand copies
  if (L.ldx % 8 != 0 || L.ldw % 16 != 0 || L.ldx >= (1LL << 38) || L.ldw >= (1LL << 38))
    return fail(SV_ERR_SHAPE, "row strides of x and W must be multiples of 16 bytes below 2^38 elements");
  if (residual == out && L.ldr != L.ldo) return fail(SV_ERR_ARG, "residual over out needs its row stride");
  if (out == x || out == W) return fail(SV_ERR_ARG, "out must not be x or W");
  if (!workspace || !aligned(workspace, 256))
    return fail(SV_ERR_WORKSPACE, "workspace must be non-NULL and 256-byte aligned");
  if (workspace_bytes < sv::linear_w4_workspace_bytes(M, N, K))
    return fail(SV_ERR_WORKSPACE, "workspace smaller than sv_linear_w4_workspace_size()");
  L.workspace = workspace;
  L.wait_tries = g_wait_tries.load(std::memory_order_relaxed);
  L.stream = stream;
  std::string err;
  const int s = sv::linear_w4_launch(L, &err);
  if (s != SV_OK) return fail(static_cast<sv_status>(s), err);
  return SV_OK;
}

constexpr int kMaxCopies = 1 << 24;  // copies of a call; sequences of a block table

size_t sv_kv_pages_workspace_size(int num_pages, int n) {
  return num_pages < 1 || num_pages > kMaxRows || n < 0 || n > kMaxCopies ? 0 : sv::kv_pages_workspace_bytes(num_pages, n);
}

static sv_status pages_args(void* const* pools, const int64_t* page_bytes, int num_pools, int num_pages, int n,
                            void* workspace, size_t workspace_bytes, sv::PagePools* p) {
  if (num_pages < 1 || num_pages > kMaxRows) return fail(SV_ERR_SHAPE, "num_pages must be in 1 .. 2^30");
  if (p) {
    if (num_pools < 1 || num_pools > sv::kMaxPools) return fail(SV_ERR_SHAPE, "num_pools must be in 1 .. 256");
    if (!pools || !page_bytes) return fail(SV_ERR_ARG, "pools and page_bytes are required");
    p->n = num_pools;
    for (int i = 0; i < num_pools; ++i) {
      if (!pools[i] || !aligned(pools[i], 16)) return fail(SV_ERR_ARG, "every pool must be non-NULL and 16-byte aligned");
      if (page_bytes[i] < 16 || page_bytes[i] % 16 != 0 || page_bytes[i] > 0x7fffffffLL)
        return fail(SV_ERR_SHAPE, "page_bytes must be a multiple of 16 below 2^31");
      p->base[i] = static_cast<uint8_t*>(pools[i]);
      p->bytes[i] = page_bytes[i];
    }
  }
  if (!workspace || !aligned(workspace, 16))
    return fail(SV_ERR_WORKSPACE, "workspace must be non-NULL and 16-byte aligned");
  if (workspace_bytes < sv::kv_pages_workspace_bytes(num_pages, n))
    return fail(SV_ERR_WORKSPACE, "workspace smaller than sv_kv_pages_workspace_size()");
  return SV_OK;
}

static sv_status table_args(const int32_t* block_table, int max_pages, int page_size, int B) {
  if (B < 1 || B > kMaxCopies || max_pages < 1 || page_size < 1)
    return fail(SV_ERR_SHAPE, "need 1 <= B <= 2^24, max_pages >= 1, page_size >= 1");
  if ((long long)max_pages * page_size + page_size > 0x7fffffffLL)
    return fail(SV_ERR_SHAPE, "(max_pages + 1) * page_size must fit in int32");
  if (!block_table || !aligned(block_table, 4)) return fail(SV_ERR_ARG, "block_table is required and must be aligned");
  return SV_OK;
}

static bool index_array(const void* p) { return p && aligned(p, 4); }

sv_status sv_kv_copy_pages(void* const* pools, const int64_t* page_bytes, int num_pools, int num_pages,
                           const int32_t* src, const int32_t* dst, int n, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (n < 1 || n > kMaxCopies) return fail(SV_ERR_SHAPE, "n must be in 1 .. 2^24");
  sv::PagePools p;
  const sv_status a = pages_args(pools, page_bytes, num_pools, num_pages, n, workspace, workspace_bytes, &p);
  if (a != SV_OK) return a;
  if (!index_array(src) || !index_array(dst)) return fail(SV_ERR_ARG, "src and dst are required and must be aligned");
  std::string err;
  const int s = sv::kv_copy_launch(p, num_pages, src, dst, n, workspace, stream, &err);
  return s == SV_OK ? SV_OK : fail(static_cast<sv_status>(s), err);
}

sv_status sv_kv_fork(void* const* pools, const int64_t* page_bytes, int num_pools, int num_pages, int page_size,
                     int32_t* block_table, int max_pages, int32_t* seq_lens, int32_t* shares,
                     const int32_t* free_pages, int32_t* free_top, const int32_t* src, const int32_t* dst, int F,
                     int B, void* workspace, size_t workspace_bytes, void* stream) {
  if (F < 1 || F > sv::kMaxForks) return fail(SV_ERR_SHAPE, "F must be in 1 .. 4096");
  sv_status a = table_args(block_table, max_pages, page_size, B);
  if (a != SV_OK) return a;
  sv::PagePools p;
  a = pages_args(pools, page_bytes, num_pools, num_pages, F, workspace, workspace_bytes, &p);
  if (a != SV_OK) return a;
  for (const void* v : {(const void*)seq_lens, (const void*)shares, (const void*)free_pages, (const void*)free_top,
                        (const void*)src, (const void*)dst})
    if (!index_array(v)) return fail(SV_ERR_ARG, "every array argument is required and must be aligned");
  std::string err;
  const int s = sv::kv_fork_launch(p, num_pages, page_size, block_table, max_pages, seq_lens, shares, free_pages,
                                   free_top, src, dst, F, B, workspace, stream, &err);
  return s == SV_OK ? SV_OK : fail(static_cast<sv_status>(s), err);
}

sv_status sv_kv_free(int32_t* block_table, int max_pages, int32_t* seq_lens, int32_t* shares, int num_pages,
                     int32_t* free_pages, int32_t* free_top, int free_capacity, const int32_t* seqs, int n, int B,
                     void* workspace, size_t workspace_bytes, void* stream) {
  if (n < 1 || n > sv::kMaxForks) return fail(SV_ERR_SHAPE, "n must be in 1 .. 4096");
  sv_status a = table_args(block_table, max_pages, 1, B);
  if (a != SV_OK) return a;
  a = pages_args(nullptr, nullptr, 0, num_pages, n, workspace, workspace_bytes, nullptr);
  if (a != SV_OK) return a;
  if (free_capacity < num_pages) return fail(SV_ERR_SHAPE, "free_capacity must be at least num_pages");
  for (const void* v : {(const void*)seq_lens, (const void*)shares, (const void*)free_pages, (const void*)free_top,
                        (const void*)seqs})
    if (!index_array(v)) return fail(SV_ERR_ARG, "every array argument is required and must be aligned");
  std::string err;
  const int s = sv::kv_free_launch(block_table, max_pages, seq_lens, shares, num_pages, free_pages, free_top,
                                   free_capacity, seqs, n, B, workspace, stream, &err);
  return s == SV_OK ? SV_OK : fail(static_cast<sv_status>(s), err);
}

sv_status sv_kv_compact(void* const* pools, const int64_t* page_bytes, int num_pools, int num_pages,
                        int32_t* block_table, int max_pages, int B, int32_t* prefix_pages, int prefix_count,
                        int32_t* shares, int32_t* free_pages, int32_t* free_top, int free_capacity, void* workspace,
                        size_t workspace_bytes, void* stream) {
  sv_status a = table_args(block_table, max_pages, 1, B);
  if (a != SV_OK) return a;
  sv::PagePools p;
  a = pages_args(pools, page_bytes, num_pools, num_pages, 0, workspace, workspace_bytes, &p);
  if (a != SV_OK) return a;
  if (free_capacity < num_pages) return fail(SV_ERR_SHAPE, "free_capacity must be at least num_pages");
  if (prefix_count < 0 || (prefix_count > 0 && !index_array(prefix_pages)))
    return fail(SV_ERR_ARG, "prefix_pages is required when prefix_count > 0 and must be aligned");
  for (const void* v : {(const void*)shares, (const void*)free_pages, (const void*)free_top})
    if (!index_array(v)) return fail(SV_ERR_ARG, "every array argument is required and must be aligned");
  std::string err;
  const int s = sv::kv_compact_launch(p, num_pages, block_table, max_pages, B, prefix_pages, prefix_count, shares,
                                      free_pages, free_top, workspace, stream, &err);
  return s == SV_OK ? SV_OK : fail(static_cast<sv_status>(s), err);
}

sv_status sv_read_device_flags(const void* workspace, uint32_t* flags_host, void* stream) {
  if (!workspace || !flags_host) return fail(SV_ERR_ARG, "null pointer");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(flags_host, workspace, sizeof(uint32_t), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return fail(SV_ERR_CUDA, std::string("reading flags: ") + cudaGetErrorString(e));
  if (*flags_host == 0) return SV_OK;
  if (*flags_host & SV_FLAG_TIMEOUT) return fail(SV_ERR_TIMEOUT, "a bounded device wait ran out");
  return fail(SV_ERR_DEVICE_FLAG, "device flag word is non-zero");
}

const char* sv_last_error(void) { return g_last_error.c_str(); }

void sv_internal_wait_tries(int tries) { g_wait_tries.store(tries < 0 ? sv::kWaitTries : tries); }

}  // extern "C"
