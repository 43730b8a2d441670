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
