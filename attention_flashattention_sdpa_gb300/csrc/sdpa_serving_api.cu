// sdpa_serving_api.cu — C entry points of the rotary positions, the paged cache and the attention
// over it: argument checks on the host, then one or two launches.  As everywhere in this library
// nothing is allocated or synchronised, and what is not supported is refused with a message.
#include <cmath>
#include <cstdio>
#include <cstring>

#include "../../include/sdpa.h"
#include "sdpa_internal.h"

namespace {

using sdpa::api_fail;

#define SDPA_REFUSE(st, ...) return static_cast<sdpa_status_t>(api_fail(st, __VA_ARGS__))
#define SDPA_TRY(call)                                        \
  do {                                                        \
    const sdpa_status_t st_ = (call);                         \
    if (st_ != SDPA_OK) return st_;                           \
  } while (0)

constexpr int64_t kMaxLen = int64_t(1) << 30;   // tokens of a sequence: positions stay well inside 32 bits

bool is16(int dt) { return dt == SDPA_DTYPE_F16 || dt == SDPA_DTYPE_BF16; }

sdpa_status_t view(const char* name, const void* ptr, const sdpa_strides_t& st, int b, int h, int s, int d, int es) {
  return static_cast<sdpa_status_t>(sdpa::api_check_view(name, ptr, {st.b, st.h, st.s, st.d}, b, h, s, d, es));
}

void strides3(int64_t (&to)[3], const sdpa_strides_t& st, int es = 1) {
  to[0] = st.b * es;
  to[1] = st.h * es;
  to[2] = st.s * es;
}

bool same_strides(const sdpa_strides_t& a, const sdpa_strides_t& b) { return a.b == b.b && a.h == b.h && a.s == b.s; }

// What a rotation needs besides its rows (shared by sdpa_rope_* and sdpa_cache_write).
sdpa_status_t check_turn(const sdpa_rope_t* p, int d) {
  if (p->rot < 2 || p->rot > d || p->rot % 2 != 0)
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "rot must be even and in 2..%d, got %d", d, p->rot);
  if (p->interleaved != 0 && p->interleaved != 1)
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "interleaved must be 0 or 1, got %d", p->interleaved);
  if (!std::isfinite(p->attn_factor)) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "attn_factor must be finite");
  if (p->table == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "table: null pointer");
  if (reinterpret_cast<uintptr_t>(p->table) % 8) SDPA_REFUSE(SDPA_ERR_LAYOUT, "table must be 8-byte aligned");
  if (reinterpret_cast<uintptr_t>(p->positions) % 4) SDPA_REFUSE(SDPA_ERR_LAYOUT, "positions must be 4-byte aligned");
  if (p->positions_stride < 0) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "positions_stride must not be negative");
  return SDPA_OK;
}

sdpa::RopeArgs turn_of(const sdpa_rope_t* p, int sign) {
  sdpa::RopeArgs r;
  r.table = p->table;
  r.positions = p->positions;
  r.positions_stride = p->positions_stride;
  r.rot = p->rot;
  r.interleaved = p->interleaved;
  r.sign = sign;
  r.factor = p->attn_factor;
  return r;
}

sdpa_status_t rope(const sdpa_rope_t* p, const void* q, const void* k, void* q_out, void* k_out, int sign,
                   void* stream_, const char* what) {
  if (p == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "rope descriptor is NULL");
  if (p->b < 1 || p->h_q < 1 || p->h_k < 0 || p->s < 1)
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "sizes must be >= 1 (b=%d h_q=%d h_k=%d s=%d)", p->b, p->h_q, p->h_k, p->s);
  if (p->d < 8 || p->d > 512 || p->d % 8 != 0)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "head dim %d not supported (a multiple of 8, 8..512)", p->d);
  if (!is16(p->dtype)) SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "rotary positions take F16 or BF16 (dtype %d)", p->dtype);
  SDPA_TRY(check_turn(p, p->d));
  SDPA_TRY(view("q", q, p->q, p->b, p->h_q, p->s, p->d, 2));
  SDPA_TRY(view("q_out", q_out, p->q_out, p->b, p->h_q, p->s, p->d, 2));
  if (p->h_k > 0) {
    SDPA_TRY(view("k", k, p->k, p->b, p->h_k, p->s, p->d, 2));
    SDPA_TRY(view("k_out", k_out, p->k_out, p->b, p->h_k, p->s, p->d, 2));
  }
  if ((q == q_out && !same_strides(p->q, p->q_out)) || (p->h_k > 0 && k == k_out && !same_strides(p->k, p->k_out)))
    SDPA_REFUSE(SDPA_ERR_LAYOUT, "an output that is its input must have its strides");
  sdpa::RopeParams prm;
  memset(&prm, 0, sizeof(prm));
  prm.r = turn_of(p, sign);
  prm.in[0] = q;
  prm.in[1] = k;
  prm.out[0] = q_out;
  prm.out[1] = k_out;
  strides3(prm.in_st[0], p->q);
  strides3(prm.in_st[1], p->k);
  strides3(prm.out_st[0], p->q_out);
  strides3(prm.out_st[1], p->k_out);
  prm.in_place[0] = q == q_out;
  prm.in_place[1] = k == k_out;
  prm.b = p->b;
  prm.s = p->s;
  prm.d = p->d;
  prm.h_q = p->h_q;
  prm.h_all = p->h_q + p->h_k;
  if (sdpa::api_log_level() >= 1)
    fprintf(stderr, "[sdpa] %s b=%d h_q=%d h_k=%d s=%d d=%d rot=%d dt=%d\n", what, p->b, p->h_q, p->h_k, p->s, p->d,
            p->rot, p->dtype);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e = sdpa::launch_rope(prm, p->dtype, sdpa::api_num_sms(), stream);
  return static_cast<sdpa_status_t>(sdpa::api_finish(e, stream, what));
}

sdpa_status_t check_cache(const sdpa_cache_t* c) {
  if (c == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "cache descriptor is NULL");
  if (c->num_pages < 1 || c->h_kv < 1 || c->b < 1 || c->max_pages < 1 || c->page_size < 1)
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "cache sizes must be >= 1 (num_pages=%d page_size=%d h_kv=%d b=%d max_pages=%d)",
                c->num_pages, c->page_size, c->h_kv, c->b, c->max_pages);
  if (c->page_size % 16 != 0)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "page_size %d not supported (a multiple of 16)", c->page_size);
  if (c->d != 64 && c->d != 128 && c->d != 256)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "head dim %d not supported (64, 128 or 256)", c->d);
  if (!is16(c->dtype) && c->dtype != SDPA_DTYPE_E4M3)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "a cache holds F16, BF16 or E4M3 (dtype %d)", c->dtype);
  const int es = c->dtype == SDPA_DTYPE_E4M3 ? 1 : 2;
  SDPA_TRY(view("k cache", c->k, c->k_strides, c->num_pages, c->h_kv, c->page_size, c->d, es));
  SDPA_TRY(view("v cache", c->v, c->v_strides, c->num_pages, c->h_kv, c->page_size, c->d, es));
  if (c->dtype == SDPA_DTYPE_E4M3) {
    if (!c->k_scale || !c->v_scale) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "an E4M3 cache needs k_scale and v_scale");
    if (reinterpret_cast<uintptr_t>(c->k_scale) % 16 || reinterpret_cast<uintptr_t>(c->v_scale) % 16)
      SDPA_REFUSE(SDPA_ERR_LAYOUT, "k_scale and v_scale must be 16-byte aligned");
  } else if (c->k_scale || c->v_scale) {
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "a 16-bit cache takes no k_scale and v_scale");
  }
  if (!c->page_table || !c->seq_lens_kv)
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "page_table and seq_lens_kv must not be NULL");
  if (reinterpret_cast<uintptr_t>(c->page_table) % 4 || reinterpret_cast<uintptr_t>(c->seq_lens_kv) % 4)
    SDPA_REFUSE(SDPA_ERR_LAYOUT, "page_table and seq_lens_kv must be 4-byte aligned");
  if (c->b > 1 && c->page_table_stride < c->max_pages)
    SDPA_REFUSE(SDPA_ERR_LAYOUT, "page_table_stride below max_pages");
  return SDPA_OK;
}

sdpa::CacheArgs cache_args(const sdpa_cache_t* c) {
  const int es = c->dtype == SDPA_DTYPE_E4M3 ? 1 : 2;
  sdpa::CacheArgs a;
  memset(&a, 0, sizeof(a));
  a.k = static_cast<uint8_t*>(c->k);
  a.v = static_cast<uint8_t*>(c->v);
  strides3(a.k_st, c->k_strides, es);
  strides3(a.v_st, c->v_strides, es);
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.page_table = c->page_table;
  a.page_table_stride = c->page_table_stride;
  a.seq_lens_kv = c->seq_lens_kv;
  a.num_pages = c->num_pages;
  a.page_size = c->page_size;
  a.h_kv = c->h_kv;
  a.b = c->b;
  a.max_pages = c->max_pages;
  const int64_t cap = static_cast<int64_t>(c->max_pages) * c->page_size;
  a.max_len = static_cast<int>(cap < kMaxLen ? cap : kMaxLen);
  return a;
}

sdpa_status_t check_rows(const sdpa_cache_t* c, const sdpa_cache_rows_t* r, const void* k, const void* v) {
  SDPA_TRY(check_cache(c));
  if (r == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "rows descriptor is NULL");
  if (r->s < 1) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "sizes must be >= 1 (s=%d)", r->s);
  if (!is16(r->dtype)) SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "rows are F16 or BF16 (dtype %d)", r->dtype);
  if (c->dtype != SDPA_DTYPE_E4M3 && r->dtype != c->dtype)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "a 16-bit cache takes and gives rows of its own dtype (%d, rows %d)", c->dtype, r->dtype);
  SDPA_TRY(view("k", k, r->k, c->b, c->h_kv, r->s, c->d, 2));
  SDPA_TRY(view("v", v, r->v, c->b, c->h_kv, r->s, c->d, 2));
  return SDPA_OK;
}

sdpa::CacheRowsParams rows_params(const sdpa_cache_t* c, const sdpa_cache_rows_t* r, const void* k, const void* v) {
  sdpa::CacheRowsParams prm;
  memset(&prm, 0, sizeof(prm));
  prm.c = cache_args(c);
  prm.k = const_cast<void*>(k);
  prm.v = const_cast<void*>(v);
  strides3(prm.k_st, r->k);
  strides3(prm.v_st, r->v);
  prm.s = r->s;
  prm.d = c->d;
  return prm;
}

// Sizes and options of an attention call (all that its workspace depends on).
sdpa_status_t check_decode_sizes(const sdpa_cache_t* c, const sdpa_decode_t* p) {
  SDPA_TRY(check_cache(c));
  if (p == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "decode descriptor is NULL");
  if (p->h_q < 1 || p->s_q < 1) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "sizes must be >= 1 (h_q=%d s_q=%d)", p->h_q, p->s_q);
  if (p->h_q % c->h_kv != 0)
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "h_q (%d) must be a multiple of h_kv (%d)", p->h_q, c->h_kv);
  if (!is16(p->dtype)) SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "Q and O are F16 or BF16 (dtype %d)", p->dtype);
  if (c->dtype != SDPA_DTYPE_E4M3 && p->dtype != c->dtype)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "over a 16-bit cache Q and O have its dtype (%d, Q %d)", c->dtype, p->dtype);
  if (p->causal == 1)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "attention over a cache takes causal = 0 or 2 (bottom-right), not top-left");
  if (p->causal != 0 && p->causal != 2)
    SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "causal must be 0 (none) or 2 (bottom-right), got %d", p->causal);
  if (p->tree_mask && p->causal != 0)
    SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "a tree mask says itself what a row sees: causal must be 0");
  if (reinterpret_cast<uintptr_t>(p->tree_mask) % 4 || reinterpret_cast<uintptr_t>(p->seq_lens_q) % 4)
    SDPA_REFUSE(SDPA_ERR_LAYOUT, "tree_mask and seq_lens_q must be 4-byte aligned");
  if (p->tree_mask_stride < 0) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "tree_mask_stride must not be negative");
  if (!std::isfinite(p->attn_scale)) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "attn_scale must be finite");
  const int64_t rows = static_cast<int64_t>(p->s_q) * (p->h_q / c->h_kv);
  if (rows * c->b * c->h_kv >= (int64_t(1) << 31)) SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "b*h_q*s_q too large");
  return SDPA_OK;
}

sdpa::DecodeParams decode_params(const sdpa_cache_t* c, const sdpa_decode_t* p) {
  sdpa::DecodeParams prm;
  memset(&prm, 0, sizeof(prm));
  prm.c = cache_args(c);
  strides3(prm.q_st, p->q);
  strides3(prm.o_st, p->o);
  prm.seq_lens_q = p->seq_lens_q;
  prm.tree_mask = p->tree_mask;
  prm.tree_mask_stride = p->tree_mask_stride;
  prm.tree_words = (p->s_q + 31) / 32;
  prm.causal = p->causal;
  prm.h_q = p->h_q;
  prm.s_q = p->s_q;
  prm.group = p->h_q / c->h_kv;
  prm.rows = p->s_q * prm.group;
  prm.scale_log2 = p->attn_scale * 1.4426950408889634f;
  sdpa::decode_plan(&prm, c->d, c->dtype, sdpa::api_num_sms());
  return prm;
}

}  // namespace

extern "C" {

sdpa_status_t sdpa_rope_table(const sdpa_rope_table_t* cfg, int64_t* table, float* attn_factor) {
  if (cfg == nullptr || table == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "cfg and table must not be NULL");
  if (cfg->rot < 2 || cfg->rot % 2 != 0) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "rot must be even and >= 2, got %d", cfg->rot);
  const int n = cfg->rot / 2;
  double base = cfg->base;
  if (cfg->inv_freq == nullptr) {
    if (cfg->scaling < 0 || cfg->scaling > 3)
      SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "scaling must be 0 (none), 1 (linear), 2 (NTK) or 3 (by parts), got %d", cfg->scaling);
    if (!(base > 0) || !std::isfinite(base)) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "base must be positive and finite");
    if (cfg->scaling != 0 && !(cfg->factor >= 1 && std::isfinite(cfg->factor)))
      SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "factor must be >= 1 and finite");
    if (cfg->scaling == 2) {
      if (cfg->rot == 2) SDPA_REFUSE(SDPA_ERR_UNSUPPORTED, "NTK scaling needs rot > 2");
      base *= std::pow(cfg->factor, cfg->rot / (cfg->rot - 2.0));
    }
    if (cfg->scaling == 3 &&
        !(cfg->original_context > 0 && cfg->beta_fast > cfg->beta_slow && std::isfinite(cfg->original_context) &&
          std::isfinite(cfg->beta_fast) && std::isfinite(cfg->beta_slow)))
      SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "scaling by parts needs original_context > 0 and beta_fast > beta_slow");
  } else {
    for (int i = 0; i < n; ++i)
      if (!std::isfinite(cfg->inv_freq[i])) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "inv_freq[%d] must be finite", i);
  }
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  for (int i = 0; i < n; ++i) {
    double f = 0;
    if (cfg->inv_freq) {
      f = cfg->inv_freq[i];
    } else {
      f = std::pow(base, -2.0 * i / cfg->rot);
      if (cfg->scaling == 1) f /= cfg->factor;
      if (cfg->scaling == 3) {
        const double r = cfg->original_context * f / kTwoPi;
        double g = (r - cfg->beta_slow) / (cfg->beta_fast - cfg->beta_slow);
        g = g < 0 ? 0 : g > 1 ? 1 : g;
        f = f * g + f / cfg->factor * (1 - g);
      }
    }
    double turns = f / kTwoPi;
    turns -= std::floor(turns);                        // [0, 1], 1 where a tiny negative was rounded
    const double hi = std::floor(turns * 4294967296.0);
    const double lo = std::nearbyint((turns * 4294967296.0 - hi) * 4294967296.0);   // 2^32 carries
    table[i] = static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(lo));
  }
  if (attn_factor)
    *attn_factor = cfg->inv_freq == nullptr && cfg->scaling == 3 ? static_cast<float>(0.1 * std::log(cfg->factor) + 1.0) : 1.f;
  return static_cast<sdpa_status_t>(sdpa::api_ok());
}

sdpa_status_t sdpa_rope_fwd(const sdpa_rope_t* p, const void* q, const void* k, void* q_out, void* k_out, void* stream) {
  return rope(p, q, k, q_out, k_out, 1, stream, "sdpa_rope_fwd");
}

sdpa_status_t sdpa_rope_bwd(const sdpa_rope_t* p, const void* dq_out, const void* dk_out, void* dq, void* dk, void* stream) {
  return rope(p, dq_out, dk_out, dq, dk, -1, stream, "sdpa_rope_bwd");
}

sdpa_status_t sdpa_cache_write(const sdpa_cache_t* c, const sdpa_cache_rows_t* r, const void* k, const void* v,
                               void* stream_) {
  SDPA_TRY(check_rows(c, r, k, v));
  if (reinterpret_cast<uintptr_t>(r->seq_lens_q) % 4) SDPA_REFUSE(SDPA_ERR_LAYOUT, "seq_lens_q must be 4-byte aligned");
  if (r->rope) SDPA_TRY(check_turn(r->rope, c->d));
  sdpa::CacheRowsParams prm = rows_params(c, r, k, v);
  prm.seq_lens_q = r->seq_lens_q;
  prm.rope = r->rope != nullptr;
  if (r->rope) prm.r = turn_of(r->rope, 1);
  if (sdpa::api_log_level() >= 1)
    fprintf(stderr, "[sdpa] cache_write b=%d h_kv=%d s=%d d=%d dt=%d cache=%d rot=%d\n", c->b, c->h_kv, r->s, c->d,
            r->dtype, c->dtype, r->rope ? r->rope->rot : 0);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e = sdpa::launch_cache_write(prm, r->dtype, c->dtype, sdpa::api_num_sms(), stream);
  return static_cast<sdpa_status_t>(sdpa::api_finish(e, stream, "sdpa_cache_write"));
}

sdpa_status_t sdpa_cache_read(const sdpa_cache_t* c, const sdpa_cache_rows_t* r, void* k, void* v, void* stream_) {
  SDPA_TRY(check_rows(c, r, k, v));
  sdpa::CacheRowsParams prm = rows_params(c, r, k, v);
  if (sdpa::api_log_level() >= 1)
    fprintf(stderr, "[sdpa] cache_read b=%d h_kv=%d s=%d d=%d dt=%d cache=%d\n", c->b, c->h_kv, r->s, c->d, r->dtype, c->dtype);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e = sdpa::launch_cache_read(prm, r->dtype, c->dtype, stream);
  return static_cast<sdpa_status_t>(sdpa::api_finish(e, stream, "sdpa_cache_read"));
}

sdpa_status_t sdpa_decode_workspace_size(const sdpa_cache_t* c, const sdpa_decode_t* p, size_t* bytes) {
  if (bytes == nullptr) SDPA_REFUSE(SDPA_ERR_INVALID_ARG, "bytes is NULL");
  SDPA_TRY(check_decode_sizes(c, p));
  *bytes = sdpa::decode_workspace_bytes(decode_params(c, p), c->d, nullptr);
  return static_cast<sdpa_status_t>(sdpa::api_ok());
}

sdpa_status_t sdpa_decode(const sdpa_cache_t* c, const sdpa_decode_t* p, const void* q, void* o, float* lse,
                          void* workspace, size_t workspace_bytes, void* stream_) {
  SDPA_TRY(check_decode_sizes(c, p));
  SDPA_TRY(view("q", q, p->q, c->b, p->h_q, p->s_q, c->d, 2));
  SDPA_TRY(view("o", o, p->o, c->b, p->h_q, p->s_q, c->d, 2));
  if (reinterpret_cast<uintptr_t>(lse) % 4) SDPA_REFUSE(SDPA_ERR_LAYOUT, "lse must be 4-byte aligned");
  sdpa::DecodeParams prm = decode_params(c, p);
  size_t ml = 0;
  const size_t need = sdpa::decode_workspace_bytes(prm, c->d, &ml);
  if (workspace == nullptr || workspace_bytes < need)
    SDPA_REFUSE(SDPA_ERR_WORKSPACE, "workspace of %zu bytes required, %zu given%s", need, workspace_bytes,
                workspace ? "" : " (NULL)");
  if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
    SDPA_REFUSE(SDPA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  prm.q = q;
  prm.o = o;
  prm.lse = lse;
  prm.part_o = static_cast<float*>(workspace);
  prm.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ml);
  if (sdpa::api_log_level() >= 1)
    fprintf(stderr, "[sdpa] decode b=%d h_q=%d h_kv=%d s_q=%d d=%d dt=%d cache=%d page=%d block=%d ctas=%d ws=%zu\n", c->b, p->h_q,
            c->h_kv, p->s_q, c->d, p->dtype, c->dtype, c->page_size, prm.tile_rows, prm.ctas, need);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e;
  if (prm.wide) {
    CUtensorMap tm_k, tm_v;
    const int box = sdpa::decode_wide_box(c->page_size);
    const sdpa_strides_t &ks = c->k_strides, &vs = c->v_strides;
    SDPA_TRY(static_cast<sdpa_status_t>(sdpa::api_make_map(&tm_k, "k cache", c->k, {ks.b, ks.h, ks.s, ks.d}, c->num_pages,
                                                           c->h_kv, c->page_size, c->d, c->dtype, box)));
    SDPA_TRY(static_cast<sdpa_status_t>(sdpa::api_make_map(&tm_v, "v cache", c->v, {vs.b, vs.h, vs.s, vs.d}, c->num_pages,
                                                           c->h_kv, c->page_size, c->d, c->dtype, box)));
    e = sdpa::launch_decode_wide(prm, tm_k, tm_v, sdpa::api_wait_limit(), c->d, p->dtype, c->dtype, stream);
  } else {
    e = sdpa::launch_decode(prm, c->d, p->dtype, c->dtype, stream);
  }
  return static_cast<sdpa_status_t>(sdpa::api_finish(e, stream, "sdpa_decode"));
}

size_t sdpa_serving_struct_size(int which) {
  switch (which) {
    case 0: return sizeof(sdpa_rope_table_t);
    case 1: return sizeof(sdpa_rope_t);
    case 2: return sizeof(sdpa_cache_t);
    case 3: return sizeof(sdpa_cache_rows_t);
    case 4: return sizeof(sdpa_decode_t);
    default: return 0;
  }
}

}  // extern "C"
