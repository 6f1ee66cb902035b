// serve_capi.cu -- the C ABI of the serving operators: argument checks,
// workspace carving and launches.
#include <cfloat>
#include <cmath>

#include "internal.h"

using namespace moe;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Workspace of the paged calls: the error word first, then the attention's
// parts of cut units (two a CTA, see paged_attn.cu): what they are of, (m, l)
// [rows][2] and outputs [rows][128] of the padded rows.
struct PagedLayout {
  size_t hdr, rec, part_o, part_ml, total;
};

int padded_rows(int n) { return n <= 16 ? 16 : n <= 32 ? 32 : 64; }

PagedLayout paged_layout(int rows) {
  PagedLayout L{};
  size_t off = 0;
  auto take = [&](size_t b) {
    size_t r = off;
    off = align256(off + b);
    return r;
  };
  L.hdr = take(256);
  L.rec = take(sizeof(PagedPart) * 2 * kPagedMaxCtas);
  L.part_ml = take(sizeof(float) * 2 * kPagedMaxCtas * 2 * padded_rows(rows));
  L.part_o = take(sizeof(float) * (size_t)kPagedMaxCtas * 2 * padded_rows(rows) * 128);
  L.total = off;
  return L;
}

moe_status check_heads(int max_rows, int nq, int nkv) {
  if (max_rows < 1 || nq < 1 || nkv < 1) return MOE_ERR_INVALID_ARG;
  if (max_rows > MOE_MAX_ROWS || nq % nkv != 0 || max_rows * (nq / nkv) > 64) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

// The checks shared by the paged calls; fills `p`.
moe_status paged_rows(const moe_paged_kv* kv, int n_rows, const int32_t* row_start, void* ws, PagedRows* p) {
  if (!kv || n_rows < 0 || !row_start || !ws) return MOE_ERR_INVALID_ARG;
  if (!kv->kpages || !kv->vpages || !kv->table || !kv->kv_len) return MOE_ERR_INVALID_ARG;
  if (kv->n_pages < 1 || kv->nkv < 1 || kv->n_seqs < 1 || kv->max_pages < 1) return MOE_ERR_INVALID_ARG;
  if (kv->head_dim != 128 || kv->n_seqs > kPagedMaxSeqs) return MOE_ERR_UNSUPPORTED_SHAPE;
  int lps = 4;
  while (lps < 7 && (1 << lps) != kv->page_size) ++lps;
  if ((1 << lps) != kv->page_size) return MOE_ERR_UNSUPPORTED_SHAPE;
  if ((long long)kv->n_pages * kv->nkv >= (1LL << 31) >> lps) return MOE_ERR_UNSUPPORTED_SHAPE;
  if ((long long)kv->max_pages << lps >= 1LL << 31) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(kv->kpages) || !aligned16(kv->vpages) || !aligned16(ws)) return MOE_ERR_MISALIGNED;
  if (!aligned4(kv->table) || !aligned4(kv->kv_len) || !aligned4(row_start)) return MOE_ERR_MISALIGNED;
  p->kp = kv->kpages;
  p->vp = kv->vpages;
  p->table = kv->table;
  p->kv_len = kv->kv_len;
  p->start = row_start;
  p->n_pages = kv->n_pages;
  p->lps = lps;
  p->nkv = kv->nkv;
  p->n_seqs = kv->n_seqs;
  p->max_pages = kv->max_pages;
  p->T = n_rows;
  p->err = static_cast<int*>(ws);
  return MOE_OK;
}

// A row-strided bf16 matrix of `width` columns (no rows: anything).
moe_status check_rows(const void* p, int64_t stride, int n_rows, int width) {
  if (n_rows == 0) return MOE_OK;
  if (!p) return MOE_ERR_INVALID_ARG;
  if (!aligned16(p) || stride % 8 != 0) return MOE_ERR_MISALIGNED;
  if (n_rows > 1 && stride < width) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

struct LogitLayout {
  size_t hdr, ticket, part_v, part_i, total;
};

moe_status check_logits(int R, int V) {
  if (R < 1 || V < 1) return MOE_ERR_INVALID_ARG;
  if (R > 4096 || V > 1 << 24) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

LogitLayout logit_layout(int R, int V) {
  LogitLayout L{};
  size_t off = 0;
  auto take = [&](size_t b) {
    size_t r = off;
    off = align256(off + b);
    return r;
  };
  const size_t tiles = ((size_t)V + 7 + 1023) / 1024;  // at the smallest tile
  L.hdr = take(256);
  L.ticket = take(sizeof(unsigned) * 4096);  // at one place for every R: a call leaves zeros here only
  L.part_v = take(sizeof(float) * R * tiles);
  L.part_i = take(sizeof(int) * R * tiles);
  L.total = off;
  return L;
}

}  // namespace

extern "C" {

size_t moe_paged_workspace_size(int max_rows, int nq, int nkv) {
  if (check_heads(max_rows, nq, nkv) != MOE_OK) return 0;
  return paged_layout(max_rows * (nq / nkv)).total;
}

moe_status moe_paged_kv_append(const moe_paged_kv* kv, const uint16_t* q, int64_t q_stride, const uint16_t* k_new,
                               int64_t k_stride, const uint16_t* v_new, int64_t v_stride, int n_rows, int nq,
                               const int32_t* row_start, const moe_attn_pos* pos, uint16_t* q_out,
                               int64_t q_out_stride, void* ws, size_t ws_bytes, void* stream) {
  PagedAppendArgs a{};
  moe_status st = paged_rows(kv, n_rows, row_start, ws, &a.p);
  if (st != MOE_OK) return st;
  if (!q != !q_out || (q && nq < 1)) return MOE_ERR_INVALID_ARG;
  if (nq > 1024 || kv->nkv > 1024) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (pos) {
    moe_attn_pos rotary = *pos;
    rotary.window = 0;  // a window is the attention's
    if ((st = check_pos(&rotary)) != MOE_OK) return st;
  }
  if ((st = check_rows(k_new, k_stride, n_rows, kv->nkv * 128)) != MOE_OK ||
      (st = check_rows(v_new, v_stride, n_rows, kv->nkv * 128)) != MOE_OK)
    return st;
  if (q && ((st = check_rows(q, q_stride, n_rows, nq * 128)) != MOE_OK ||
            (st = check_rows(q_out, q_out_stride, n_rows, nq * 128)) != MOE_OK))
    return st;
  if (q == q_out && q && q_stride != q_out_stride && n_rows > 1) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < 256) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (n_rows == 0) return MOE_OK;
  a.q = q;
  a.k = k_new;
  a.v = v_new;
  a.qo = q_out;
  a.qs = q_stride;
  a.ks = k_stride;
  a.vs = v_stride;
  a.qos = q_out_stride;
  a.nq = nq;
  double temp;
  if (pos && pos->rotary_dim > 0) {
    a.rd = pos->rotary_dim;
    rope_freqs(*pos, a.freq, &temp);
  }
  return launch_paged_append(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_paged_attention(const moe_paged_kv* kv, const uint16_t* q, int64_t q_stride, int n_rows, int max_rows,
                               int nq, const int32_t* row_start, const moe_paged_scores* scores, uint16_t* o,
                               int64_t o_stride, float* lse, void* ws, size_t ws_bytes, void* stream) {
  PagedAttnParams A{};
  PagedAttnArgs& a = A.a;
  moe_status st = paged_rows(kv, n_rows, row_start, ws, &a.p);
  if (st != MOE_OK) return st;
  if ((st = check_heads(max_rows, nq, kv->nkv)) != MOE_OK) return st;
  if ((st = check_rows(q, q_stride, n_rows, nq * 128)) != MOE_OK ||
      (st = check_rows(o, o_stride, n_rows, nq * 128)) != MOE_OK)
    return st;
  if (q == o && q_stride != o_stride && n_rows > 1) return MOE_ERR_INVALID_ARG;
  if (!aligned4(lse)) return MOE_ERR_MISALIGNED;
  const moe_paged_scores none{};
  if (!scores) scores = &none;
  constexpr float most = 0x1p126f;  // times log2 e it is finite
  if (scores->window < 0 || !(scores->scale >= 0.f && scores->scale <= most) ||
      !(scores->softcap >= 0.f && scores->softcap <= most))
    return MOE_ERR_INVALID_ARG;
  if (!aligned4(scores->slopes) || !aligned4(scores->first) || !aligned4(scores->prefix)) return MOE_ERR_MISALIGNED;
  const PagedLayout L = paged_layout(max_rows * (nq / kv->nkv));
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (n_rows == 0) return MOE_OK;
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.qs = q_stride;
  a.os = o_stride;
  a.nq = nq;
  a.group = nq / kv->nkv;
  a.max_rows = max_rows;
  a.window = scores->window;
  const double log2e = 1.4426950408889634, scale = scores->scale > 0.f ? scores->scale : 1.0 / std::sqrt(128.0);
  a.scale_log2 = (float)(scale * log2e);
  a.cap_in = 0.f;
  if (scores->softcap > 0.f)  // as far as FP32 goes (not 0 or infinite: 0 times infinity)
    a.cap_in = (float)std::fmin(std::fmax(2.0 * log2e * scale / scores->softcap, FLT_MIN), FLT_MAX);
  a.cap_log2 = (float)(scores->softcap * log2e);
  a.plain = !(scores->softcap > 0.f) && !scores->slopes;
  a.slopes = scores->slopes;
  a.first = scores->first;
  a.prefix = scores->prefix;
  char* b = static_cast<char*>(ws);
  A.rec = reinterpret_cast<PagedPart*>(b + L.rec);
  A.part_ml = reinterpret_cast<float*>(b + L.part_ml);
  A.part_o = reinterpret_cast<float*>(b + L.part_o);
  A.wait_ns = wait_limit_ns();
  const int64_t rows = (int64_t)kv->n_pages * kv->nkv * kv->page_size;
  const int box = kv->page_size < 64 ? kv->page_size : 64;
  const int halves = paged_attention_tc(a) ? 1 : 2;
  if (!encode_page_map(&A.km, kv->kpages, rows, box, halves) || !encode_page_map(&A.vm, kv->vpages, rows, box, halves))
    return MOE_ERR_CUDA;
  return launch_paged_attention(A, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_logits_workspace_size(int R, int V) {
  if (check_logits(R, V) != MOE_OK) return 0;
  return logit_layout(R, V).total;
}

moe_status moe_logits_constrain(const void* logits, int type, int64_t stride, int R, int V,
                                const moe_logit_rules* rules, void* out, int64_t out_stride, int32_t* tok,
                                float* best, void* ws, size_t ws_bytes, void* stream) {
  moe_status st = check_logits(R, V);
  if (st != MOE_OK) return st;
  if (!logits || !ws || (!out && !tok && !best) || (type != MOE_LOGITS_F32 && type != MOE_LOGITS_BF16))
    return MOE_ERR_INVALID_ARG;
  if (R > 1 && (stride < V || (out && out_stride < V))) return MOE_ERR_INVALID_ARG;
  if (out == logits && R > 1 && stride != out_stride) return MOE_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(out) || !aligned16(ws)) return MOE_ERR_MISALIGNED;
  if (!aligned4(tok) || !aligned4(best)) return MOE_ERR_MISALIGNED;
  LogitArgs a{};
  if (rules) {
    a.rules = *rules;
    if (!rules->tokens != !rules->begin || !rules->tokens != !rules->end || rules->n_tokens < 0)
      return MOE_ERR_INVALID_ARG;
    if ((rules->bias && (!rules->bias_row || rules->n_bias < 1)) ||
        (rules->allow && (!rules->allow_row || rules->n_allow < 1)))
      return MOE_ERR_INVALID_ARG;
    const void* ptrs[] = {rules->tokens, rules->begin, rules->end, rules->repetition, rules->presence,
                          rules->frequency, rules->bias, rules->bias_row, rules->allow, rules->allow_row};
    for (const void* p : ptrs)
      if (!aligned4(p)) return MOE_ERR_MISALIGNED;
  }
  const LogitLayout L = logit_layout(R, V);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  char* b = static_cast<char*>(ws);
  a.x = logits;
  a.out = out;
  a.xs = stride;
  a.os = out_stride;
  a.bf16 = type == MOE_LOGITS_BF16;
  a.R = R;
  a.V = V;
  a.tok = tok;
  a.best = best;
  a.err = reinterpret_cast<int*>(b + L.hdr);
  a.ticket = reinterpret_cast<unsigned*>(b + L.ticket);
  a.part_v = reinterpret_cast<float*>(b + L.part_v);
  a.part_i = reinterpret_cast<int*>(b + L.part_i);
  return launch_logits(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
