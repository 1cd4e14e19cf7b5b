// dq_abi.cpp -- the C-ABI of libdq: argument checks, table upload, workspace
// sizing and kernel launches. Every entry point catches C++ exceptions and
// reports a DQ_ERR_* code; nothing here allocates per call except
// dq_build_tables.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <new>
#include <vector>

#include "dq_internal.h"

struct dq_tables {
  dq_config cfg{};
  int device = -1;
  int sm_count = 0;
  dqi::StreamDesign k, v;
  std::vector<int8_t> signs;
  void *d_block = nullptr;
  dqi::DevTables *d_tabs = nullptr;
  uint32_t *d_sign_bits = nullptr;
};

namespace {

thread_local int g_last_cuda = 0;

int cuda_fail(cudaError_t e) {
  g_last_cuda = static_cast<int>(e);
  cudaGetLastError();  // (a call's error is not held against the next one, whose launches ask for the last error)
  return DQ_ERR_CUDA;
}

// Same device as the tables? (Device pointers from another device would be
// read through peer mappings at best; refuse instead.)
int check_device(const dq_tables *t) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  return dev == t->device ? DQ_OK : DQ_ERR_DEVICE;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// IEEE binary32 -> binary16, round to nearest even (overflow to infinity).
uint16_t f32_to_f16_rn(float f) {
  uint32_t x;
  std::memcpy(&x, &f, 4);
  const uint32_t sign = (x >> 16) & 0x8000u;
  x &= 0x7FFFFFFFu;
  if (x >= 0x7F800000u) return static_cast<uint16_t>(sign | (x > 0x7F800000u ? 0x7E00u : 0x7C00u));
  if (x >= 0x477FF000u) return static_cast<uint16_t>(sign | 0x7C00u);  // rounds to >= 65520
  if (x < 0x38800000u) {  // below 2^-14: subnormal half, units of 2^-24
    float a;
    std::memcpy(&a, &x, 4);
    return static_cast<uint16_t>(sign | static_cast<uint32_t>(std::nearbyint(static_cast<double>(a) * 16777216.0)));
  }
  uint32_t h = ((((x >> 23) - 127u + 15u) << 10) | ((x & 0x7FFFFFu) >> 13));
  const uint32_t rem = x & 0x1FFFu;
  if (rem > 0x1000u || (rem == 0x1000u && (h & 1u))) ++h;
  return static_cast<uint16_t>(sign | h);
}

double f16_to_double(uint16_t h) {
  const int e = (h >> 10) & 0x1F;
  const int m = h & 0x3FF;
  double v = e == 0 ? std::ldexp(static_cast<double>(m), -24) : std::ldexp(1024.0 + m, e - 25);
  return (h & 0x8000u) ? -v : v;
}

// Scale kappa in [1, 2) (steps of 2^-16) that minimises the largest relative
// error of fp16(kappa * level) over the non-zero levels; the smallest such
// kappa on ties. (The error only grows with each level: a candidate is
// dropped once it is no better than the best so far.)
void choose_tile_scale(const dqi::StreamDesign &d, dqi::DevStream *s) {
  double best_err = INFINITY;
  double best_k = 1.0;
  for (int j = 0; j < 65536; ++j) {
    const double kappa = 1.0 + j / 65536.0;
    double err = 0.0;
    for (int i = 0; i < d.n_levels && err < best_err; ++i) {
      const double y = static_cast<double>(d.levels[i]);
      if (y == 0.0) continue;
      const double h = f16_to_double(f32_to_f16_rn(static_cast<float>(kappa * y)));
      err = std::max(err, std::fabs(h - kappa * y) / std::fabs(kappa * y));
    }
    if (err < best_err) {
      best_err = err;
      best_k = kappa;
    }
  }
  s->tile_scale = static_cast<float>(best_k);
  s->tile_rel_err = static_cast<float>(best_err);
  for (int i = 0; i < dqi::kMaxLevels; ++i) {
    s->level16[i] = 0u;
    if (i >= d.n_levels) continue;
    const double y = best_k * static_cast<double>(d.levels[i]);
    const uint16_t hi = f32_to_f16_rn(static_cast<float>(y));
    const uint16_t lo = f32_to_f16_rn(static_cast<float>(y - f16_to_double(hi)));
    s->level16[i] = static_cast<uint32_t>(hi) | static_cast<uint32_t>(lo) << 16;
  }
}

// Scale kappa in [1, 2) (steps of 2^-16) for the prefill score operand:
// minimises sum_s f_s |fp16(kappa y_s) / kappa - y_s|, the expected absolute
// error of a coordinate's level, so the frequent inner levels are the exact
// ones; the smallest such kappa on ties.
void choose_score_scale(const dqi::StreamDesign &d, dqi::DevStream *s) {
  double best_err = INFINITY;
  double best_k = 1.0;
  for (int j = 0; j < 65536; ++j) {
    const double kappa = 1.0 + j / 65536.0;
    double err = 0.0;
    for (int i = 0; i < d.n_levels && err < best_err; ++i) {
      const double y = static_cast<double>(d.levels[i]);
      const double h = f16_to_double(f32_to_f16_rn(static_cast<float>(kappa * y)));
      err += static_cast<double>(d.freq[i]) * std::fabs(h / kappa - y);
    }
    if (err < best_err) {
      best_err = err;
      best_k = kappa;
    }
  }
  double worst = 0.0;
  for (int i = 0; i < dqi::kMaxLevels; ++i) {
    s->score16[i] = 0u;
    if (i >= d.n_levels) continue;
    const double y = static_cast<double>(d.levels[i]);
    s->score16[i] = f32_to_f16_rn(static_cast<float>(best_k * y));
    if (y != 0.0) worst = std::max(worst, std::fabs(f16_to_double(static_cast<uint16_t>(s->score16[i])) - best_k * y) /
                                              std::fabs(best_k * y));
  }
  s->score_scale = static_cast<float>(best_k);
  s->score_err = static_cast<float>(worst);
}

void fill_dev_stream(const dqi::StreamDesign &d, dqi::DevStream *s) {
  std::memset(s, 0, sizeof(*s));
  for (int sym = 0; sym < d.n_levels; ++sym)
    for (uint32_t slot = d.cum[sym]; slot < d.cum[sym + 1]; ++slot)
      s->lut[slot] = (slot - d.cum[sym]) | (static_cast<uint32_t>(sym) << 11) | (d.freq[sym] << 20);
  for (int i = 0; i < dqi::kMaxLevels; ++i) {
    s->levels[i] = i < d.n_levels ? d.levels[i] : 0.0f;
    s->thresholds[i] = d.thresholds[i];
    s->cost[i] = i < d.n_levels ? d.cost[i] : INFINITY;
    s->freq[i] = i < d.n_levels ? d.freq[i] : 0u;
    s->cum[i] = i < d.n_levels ? d.cum[i] : dqi::kM;
  }
  choose_tile_scale(d, s);
  choose_score_scale(d, s);
  s->n_levels = d.n_levels;
  s->container_bytes = d.container_bytes;
  s->payload_bytes = d.payload_bytes;
}

// A symbol with f < 16 can make one coding step move two bytes.
bool has_small_freq(const dqi::StreamDesign &d) {
  for (int s = 0; s < d.n_levels; ++s)
    if (d.freq[s] < 16) return true;
  return false;
}

const dqi::StreamDesign *stream_of(const dq_tables *t, int kind) {
  if (!t) return nullptr;
  if (kind == DQ_STREAM_K) return &t->k;
  if (kind == DQ_STREAM_V) return &t->v;
  return nullptr;
}

// Workspace of dq_decode_attention: the token-group prefix sums, then one
// partial-state slot per (b, h) segment of a warp's range. Slot (b Hkv + h) +
// warp is unique, so B Hkv + (total warps) slots cover every case.
struct WsLayout {
  int grid = 0;
  int64_t total_warps = 0;
  size_t prefix_off = 0, o_off = 0, ml_off = 0, total = 0;
};

// Pages of a row in the bookkeeping calls: its tokens are counted in int32.
constexpr int64_t kMaxTablePages = int64_t(1) << 26;

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

WsLayout ws_layout(const dq_tables *t, int B, int Hkv, int G) {
  WsLayout w;
  const int nw = dqi::decode_warps_per_cta(G, t->k.container_bytes, t->v.container_bytes);
  if (nw <= 0) return w;
  w.grid = t->sm_count;
  w.total_warps = static_cast<int64_t>(w.grid) * nw;
  const size_t slots = static_cast<size_t>(B) * Hkv + static_cast<size_t>(w.total_warps);
  w.prefix_off = 0;
  w.o_off = round256((static_cast<size_t>(B) + 1) * sizeof(int64_t));
  w.ml_off = w.o_off + round256(slots * G * dqi::kD * sizeof(float));
  w.total = w.ml_off + slots * G * 2 * sizeof(float);
  return w;
}

}  // namespace

extern "C" {

void dq_config_default(dq_config *cfg) {
  if (!cfg) return;
  std::memset(cfg, 0, sizeof(*cfg));
  cfg->head_dim = 128;
  cfg->k_levels = 8;
  cfg->v_levels = 6;
  cfg->prob_bits = 12;
  cfg->k_bits_per_value = 2.26f;
  cfg->v_bits_per_value = 2.26f;
  cfg->n_kv_heads = 8;
  cfg->sign_seed = 0;
}

const char *dq_error_string(int status) {
  switch (status) {
    case DQ_OK: return "ok";
    case DQ_ERR_NULL: return "a required pointer is NULL";
    case DQ_ERR_CONFIG: return "invalid configuration (head_dim, prob_bits or level counts)";
    case DQ_ERR_BUDGET: return "container too small (or too large) for the level design";
    case DQ_ERR_SHAPE: return "invalid shape argument";
    case DQ_ERR_WORKSPACE: return "workspace too small";
    case DQ_ERR_ALIGN: return "misaligned pointer or T_cap not a multiple of 16";
    case DQ_ERR_DTYPE: return "unknown dtype";
    case DQ_ERR_CUDA: return "CUDA runtime error (see dq_last_cuda_error)";
    case DQ_ERR_DEVICE: return "not an sm_100 device or not the device of the tables";
    default: return "unknown status";
  }
}

int dq_last_cuda_error(void) { return g_last_cuda; }

// Host-only design of one stream (no device needed); arrays of 8 (9 for cum).
int dq_design_stream(int32_t n_levels, int32_t container_bytes, double rate_offset,
                     float *levels, float *thresholds, uint32_t *freq, uint32_t *cum,
                     float *cost, double *lambda, double *entropy, double *mse) {
  try {
    dqi::StreamDesign d;
    int rc = dqi::design_stream(n_levels, container_bytes, rate_offset, &d);
    if (rc != DQ_OK) return rc;
    for (int i = 0; i < dqi::kMaxLevels; ++i) {
      if (levels) levels[i] = i < n_levels ? d.levels[i] : 0.0f;
      if (thresholds && i < dqi::kMaxLevels - 1) thresholds[i] = d.thresholds[i];
      if (freq) freq[i] = d.freq[i];
      if (cost) cost[i] = i < n_levels ? d.cost[i] : 0.0f;
    }
    if (cum)
      for (int i = 0; i <= dqi::kMaxLevels; ++i) cum[i] = i <= n_levels ? d.cum[i] : dqi::kM;
    if (lambda) *lambda = d.lambda;
    if (entropy) *entropy = d.entropy;
    if (mse) *mse = d.mse;
    return DQ_OK;
  } catch (...) {
    return DQ_ERR_CONFIG;
  }
}

int dq_build_tables(const dq_config *cfg, dq_tables **out) {
  if (!cfg || !out) return DQ_ERR_NULL;
  *out = nullptr;
  if (cfg->head_dim != dqi::kD || cfg->prob_bits != dqi::kProbBits || cfg->n_kv_heads < 1 ||
      cfg->n_kv_heads > 4096 || (cfg->drift_mode != 0 && cfg->drift_mode != 1))
    return DQ_ERR_CONFIG;
  dq_tables *t = nullptr;
  try {
    t = new dq_tables();
    t->cfg = *cfg;
    const int ck = cfg->k_container_bytes ? cfg->k_container_bytes
                                          : dqi::container_bytes_for(cfg->k_bits_per_value);
    const int cv = cfg->v_container_bytes ? cfg->v_container_bytes
                                          : dqi::container_bytes_for(cfg->v_bits_per_value);
    int rc = dqi::design_stream(cfg->k_levels, ck, cfg->k_rate_offset, &t->k);
    if (rc == DQ_OK) rc = dqi::design_stream(cfg->v_levels, cv, cfg->v_rate_offset, &t->v);
    if (rc != DQ_OK) {
      delete t;
      return rc;
    }
    t->signs.resize(static_cast<size_t>(cfg->n_kv_heads) * dqi::kD);
    dqi::rotation_signs(cfg->sign_seed, cfg->n_kv_heads, t->signs.data());

    cudaError_t e = cudaGetDevice(&t->device);
    if (e != cudaSuccess) { delete t; return cuda_fail(e); }
    cudaDeviceProp prop;
    e = cudaGetDeviceProperties(&prop, t->device);
    if (e != cudaSuccess) { delete t; return cuda_fail(e); }
    if (prop.major != 10) { delete t; return DQ_ERR_DEVICE; }
    t->sm_count = prop.multiProcessorCount;

    std::vector<uint8_t> host(sizeof(dqi::DevTables) + t->signs.size() / 8);
    auto *dt = reinterpret_cast<dqi::DevTables *>(host.data());
    fill_dev_stream(t->k, &dt->k);
    fill_dev_stream(t->v, &dt->v);
    auto *bits = reinterpret_cast<uint32_t *>(host.data() + sizeof(dqi::DevTables));
    for (int h = 0; h < cfg->n_kv_heads; ++h)
      for (int w = 0; w < 4; ++w) {
        uint32_t word = 0;
        for (int l = 0; l < 32; ++l)
          if (t->signs[h * dqi::kD + w * 32 + l] < 0) word |= 1u << l;
        bits[h * 4 + w] = word;
      }
    e = cudaMalloc(&t->d_block, host.size());
    if (e != cudaSuccess) { delete t; return cuda_fail(e); }
    e = cudaMemcpy(t->d_block, host.data(), host.size(), cudaMemcpyHostToDevice);
    if (e != cudaSuccess) { cudaFree(t->d_block); delete t; return cuda_fail(e); }
    t->d_tabs = reinterpret_cast<dqi::DevTables *>(t->d_block);
    t->d_sign_bits = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(t->d_block) + sizeof(dqi::DevTables));
    *out = t;
    return DQ_OK;
  } catch (const std::bad_alloc &) {
    delete t;
    return DQ_ERR_CONFIG;
  } catch (...) {
    delete t;
    return DQ_ERR_CONFIG;
  }
}

void dq_free_tables(dq_tables *t) {
  if (!t) return;
  if (t->d_block) cudaFree(t->d_block);
  delete t;
}

int dq_get_stream_table(const dq_tables *t, int stream_kind, int32_t *n_levels,
                        int32_t *container_bytes, float *levels, float *thresholds,
                        uint32_t *freq, uint32_t *cum, float *cost) {
  const dqi::StreamDesign *d = stream_of(t, stream_kind);
  if (!d) return t ? DQ_ERR_CONFIG : DQ_ERR_NULL;
  if (n_levels) *n_levels = d->n_levels;
  if (container_bytes) *container_bytes = d->container_bytes;
  for (int i = 0; i < dqi::kMaxLevels; ++i) {
    if (levels) levels[i] = i < d->n_levels ? d->levels[i] : 0.0f;
    if (thresholds && i < dqi::kMaxLevels - 1) thresholds[i] = d->thresholds[i];
    if (freq) freq[i] = d->freq[i];
    if (cost) cost[i] = i < d->n_levels ? d->cost[i] : 0.0f;
  }
  if (cum)
    for (int i = 0; i <= dqi::kMaxLevels; ++i) cum[i] = i <= d->n_levels ? d->cum[i] : dqi::kM;
  return DQ_OK;
}

int dq_get_stream_design(const dq_tables *t, int stream_kind, double *lambda, double *entropy,
                         double *rate, double *mse, int32_t *is_lloyd_max) {
  const dqi::StreamDesign *d = stream_of(t, stream_kind);
  if (!d) return t ? DQ_ERR_CONFIG : DQ_ERR_NULL;
  if (lambda) *lambda = d->lambda;
  if (entropy) *entropy = d->entropy;
  if (rate) *rate = d->rate;
  if (mse) *mse = d->mse;
  if (is_lloyd_max) *is_lloyd_max = d->lloyd_max ? 1 : 0;
  return DQ_OK;
}

int dq_get_signs(const dq_tables *t, int8_t *signs) {
  if (!t || !signs) return DQ_ERR_NULL;
  std::memcpy(signs, t->signs.data(), t->signs.size());
  return DQ_OK;
}

size_t dq_append_workspace_bytes(const dq_tables *t, int B, int Hkv, int n_new) {
  if (!t || B < 0 || Hkv < 1 || n_new < 0) return 0;
  return dqi::append_workspace_bytes(static_cast<int64_t>(B) * Hkv * n_new);
}

int dq_append_kv(const dq_tables *t, const void *k, const void *v, int dtype, int B, int Hkv,
                 int n_new, const int32_t *d_start_pos, uint8_t *d_kcache, uint8_t *d_vcache,
                 int64_t T_cap, dq_stats *d_stats, void *stream) {
  return dq_append_kv_ws(t, k, v, dtype, B, Hkv, n_new, d_start_pos, d_kcache, d_vcache, T_cap, nullptr, 0,
                         d_stats, stream);
}

static int check_page_table(const int32_t *d_page_table, int64_t num_pages, int64_t max_pages) {
  if (!d_page_table) return DQ_ERR_NULL;
  if (num_pages < 1 || max_pages < 1 || max_pages > (int64_t(1) << 40) || num_pages > (int64_t(1) << 31))
    return DQ_ERR_SHAPE;
  return aligned(d_page_table, 4) ? DQ_OK : DQ_ERR_ALIGN;
}

// Shared by dq_append_kv_ws (page_table NULL) and dq_append_kv_paged.
static int append_core(const dq_tables *t, const void *k, const void *v, int dtype, int B, int Hkv, int n_new,
                       const int32_t *d_start_pos, uint8_t *d_kcache, uint8_t *d_vcache, int64_t T_cap,
                       void *d_workspace, size_t ws_bytes, dq_stats *d_stats, void *stream,
                       const int32_t *page_table, int64_t max_pages, int64_t num_pages) {
  try {
    if (!t || !k || !v || !d_start_pos || !d_kcache || !d_vcache) return DQ_ERR_NULL;
    if (dtype != DQ_F32 && dtype != DQ_BF16) return DQ_ERR_DTYPE;
    if (B < 0 || n_new < 0 || T_cap < 0 || Hkv != t->cfg.n_kv_heads) return DQ_ERR_SHAPE;
    if (!aligned(k, 16) || !aligned(v, 16) || T_cap % 32) return DQ_ERR_ALIGN;
    int rc = check_device(t);
    if (rc != DQ_OK) return rc;
    if (B == 0 || n_new == 0) return DQ_OK;
    dqi::AppendArgs a{};
    a.tabs = t->d_tabs;
    a.sign_bits = t->d_sign_bits;
    a.k = k;
    a.v = v;
    a.dtype = dtype;
    a.B = B;
    a.Hkv = Hkv;
    a.n_new = n_new;
    a.start_pos = d_start_pos;
    a.kcache = d_kcache;
    a.vcache = d_vcache;
    a.T_cap = T_cap;
    a.ck = t->k.container_bytes;
    a.cv = t->v.container_bytes;
    a.nk = t->k.n_levels;
    a.nv = t->v.n_levels;
    a.drift_mode = t->cfg.drift_mode;
    a.two_k = has_small_freq(t->k);
    a.two_v = has_small_freq(t->v);
    a.stats = d_stats;
    const int64_t nvec = static_cast<int64_t>(B) * Hkv * n_new;
    if (d_workspace) {
      if (!aligned(d_workspace, 16)) return DQ_ERR_ALIGN;
      if (ws_bytes < dqi::append_workspace_bytes(nvec)) return DQ_ERR_WORKSPACE;
      a.drift_count = static_cast<uint32_t *>(d_workspace);
      a.drift_list = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(d_workspace) + 256);
      a.list_cap = nvec;
    }
    a.page_table = page_table;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    int e = dqi::launch_append(a, stream);
    return e == 0 ? DQ_OK : cuda_fail(static_cast<cudaError_t>(e));
  } catch (...) {
    return DQ_ERR_CUDA;
  }
}

int dq_append_kv_ws(const dq_tables *t, const void *k, const void *v, int dtype, int B, int Hkv, int n_new,
                    const int32_t *d_start_pos, uint8_t *d_kcache, uint8_t *d_vcache, int64_t T_cap,
                    void *d_workspace, size_t ws_bytes, dq_stats *d_stats, void *stream) {
  return append_core(t, k, v, dtype, B, Hkv, n_new, d_start_pos, d_kcache, d_vcache, T_cap, d_workspace, ws_bytes,
                     d_stats, stream, nullptr, 0, 0);
}

int dq_append_kv_paged(const dq_tables *t, const void *k, const void *v, int dtype, int B, int Hkv, int n_new,
                       const int32_t *d_start_pos, uint8_t *d_kpool, uint8_t *d_vpool, int64_t num_pages,
                       const int32_t *d_page_table, int64_t max_pages, void *d_workspace, size_t ws_bytes,
                       dq_stats *d_stats, void *stream) {
  const int rc = check_page_table(d_page_table, num_pages, max_pages);
  if (rc != DQ_OK) return rc;
  return append_core(t, k, v, dtype, B, Hkv, n_new, d_start_pos, d_kpool, d_vpool, 32 * max_pages, d_workspace,
                     ws_bytes, d_stats, stream, d_page_table, max_pages, num_pages);
}

size_t dq_decode_workspace_bytes(const dq_tables *t, int B, int Hq, int Hkv, int64_t T_max) {
  if (!t || B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || T_max < 0) return 0;
  return ws_layout(t, B, Hkv, Hq / Hkv).total;
}

// Window arguments: at least the query's own token is visible, and scores are
// masked before they are scaled (an infinite scale would give NaN weights).
static int check_window(int64_t window, int64_t sinks, float sm_scale) {
  return window < 1 || sinks < 0 || !(sm_scale > 0.0f) || std::isinf(sm_scale) ? DQ_ERR_SHAPE : DQ_OK;
}

// Shared by the dq_decode_attention calls (page_table NULL: contiguous cache;
// window 0: none).
static int decode_core(const dq_tables *t, const void *q, int q_dtype, const uint8_t *d_kcache,
                       const uint8_t *d_vcache, const int32_t *d_seq_lens, int B, int Hq, int Hkv,
                       int64_t T_cap, int64_t T_max, float sm_scale, void *out, int out_dtype,
                       void *d_workspace, size_t ws_bytes, dq_stats *d_stats, void *stream,
                       const int32_t *page_table, int64_t max_pages, int64_t num_pages, int64_t window = 0,
                       int64_t sinks = 0) {
  try {
    if (!t || !q || !d_kcache || !d_vcache || !d_seq_lens || !out || !d_workspace) return DQ_ERR_NULL;
    if ((q_dtype != DQ_F32 && q_dtype != DQ_BF16) || (out_dtype != DQ_F32 && out_dtype != DQ_BF16))
      return DQ_ERR_DTYPE;
    if (B < 0 || Hkv != t->cfg.n_kv_heads || Hq < Hkv || Hq % Hkv) return DQ_ERR_SHAPE;
    const int G = Hq / Hkv;
    if (G != 1 && G != 2 && G != 4 && G != 8) return DQ_ERR_SHAPE;
    if (T_cap < 0 || T_max < 0 || T_max > T_cap) return DQ_ERR_SHAPE;
    if (T_cap % 32 || !aligned(d_kcache, 16) || !aligned(d_vcache, 16) || !aligned(d_workspace, 16) ||
        !aligned(q, 4) || !aligned(out, 4))
      return DQ_ERR_ALIGN;
    if (!std::isfinite(sm_scale)) return DQ_ERR_SHAPE;
    const WsLayout wl = ws_layout(t, B, Hkv, G);
    if (wl.total == 0) return DQ_ERR_SHAPE;
    if (ws_bytes < wl.total) return DQ_ERR_WORKSPACE;
    int rc = check_device(t);
    if (rc != DQ_OK) return rc;
    if (B == 0) return DQ_OK;
    dqi::DecodeArgs a{};
    a.tabs = t->d_tabs;
    a.sign_bits = t->d_sign_bits;
    a.q = q;
    a.q_dtype = q_dtype;
    a.kcache = d_kcache;
    a.vcache = d_vcache;
    a.seq_lens = d_seq_lens;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = G;
    a.T_cap = T_cap;
    a.T_max = T_max;
    a.sm_scale = sm_scale;
    a.out = out;
    a.out_dtype = out_dtype;
    uint8_t *ws = static_cast<uint8_t *>(d_workspace);
    a.prefix = reinterpret_cast<int64_t *>(ws + wl.prefix_off);
    a.ws_o = reinterpret_cast<float *>(ws + wl.o_off);
    a.ws_ml = reinterpret_cast<float *>(ws + wl.ml_off);
    a.grid = wl.grid;
    a.total_warps = wl.total_warps;
    a.ck = t->k.container_bytes;
    a.cv = t->v.container_bytes;
    a.two_k = has_small_freq(t->k);
    a.two_v = has_small_freq(t->v);
    a.stats = d_stats;
    a.page_table = page_table;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    // (A window of T_cap tokens or more hides nothing; at least 1 keeps the windowed kernel.)
    a.window = window > 0 ? std::max<int64_t>(1, std::min(window, T_cap)) : 0;
    a.sinks = std::min(sinks, T_cap);
    int e = dqi::launch_decode_attention(a, stream);
    return e == 0 ? DQ_OK : cuda_fail(static_cast<cudaError_t>(e));
  } catch (...) {
    return DQ_ERR_CUDA;
  }
}

int dq_decode_attention(const dq_tables *t, const void *q, int q_dtype, const uint8_t *d_kcache,
                        const uint8_t *d_vcache, const int32_t *d_seq_lens, int B, int Hq, int Hkv,
                        int64_t T_cap, int64_t T_max, float sm_scale, void *out, int out_dtype,
                        void *d_workspace, size_t ws_bytes, dq_stats *d_stats, void *stream) {
  return decode_core(t, q, q_dtype, d_kcache, d_vcache, d_seq_lens, B, Hq, Hkv, T_cap, T_max, sm_scale, out,
                     out_dtype, d_workspace, ws_bytes, d_stats, stream, nullptr, 0, 0);
}

int dq_decode_attention_paged(const dq_tables *t, const void *q, int q_dtype, const uint8_t *d_kpool,
                              const uint8_t *d_vpool, int64_t num_pages, const int32_t *d_page_table,
                              int64_t max_pages, const int32_t *d_seq_lens, int B, int Hq, int Hkv,
                              int64_t T_max, float sm_scale, void *out, int out_dtype, void *d_workspace,
                              size_t ws_bytes, dq_stats *d_stats, void *stream) {
  const int rc = check_page_table(d_page_table, num_pages, max_pages);
  if (rc != DQ_OK) return rc;
  return decode_core(t, q, q_dtype, d_kpool, d_vpool, d_seq_lens, B, Hq, Hkv, 32 * max_pages, T_max, sm_scale,
                     out, out_dtype, d_workspace, ws_bytes, d_stats, stream, d_page_table, max_pages, num_pages);
}

int dq_decode_attention_window(const dq_tables *t, const void *q, int q_dtype, const uint8_t *d_kcache,
                               const uint8_t *d_vcache, const int32_t *d_seq_lens, int B, int Hq, int Hkv,
                               int64_t T_cap, int64_t T_max, int64_t window, int64_t sinks, float sm_scale,
                               void *out, int out_dtype, void *d_workspace, size_t ws_bytes, dq_stats *d_stats,
                               void *stream) {
  const int rc = check_window(window, sinks, sm_scale);
  if (rc != DQ_OK) return rc;
  return decode_core(t, q, q_dtype, d_kcache, d_vcache, d_seq_lens, B, Hq, Hkv, T_cap, T_max, sm_scale, out,
                     out_dtype, d_workspace, ws_bytes, d_stats, stream, nullptr, 0, 0, window, sinks);
}

int dq_decode_attention_window_paged(const dq_tables *t, const void *q, int q_dtype, const uint8_t *d_kpool,
                                     const uint8_t *d_vpool, int64_t num_pages, const int32_t *d_page_table,
                                     int64_t max_pages, const int32_t *d_seq_lens, int B, int Hq, int Hkv,
                                     int64_t T_max, int64_t window, int64_t sinks, float sm_scale, void *out,
                                     int out_dtype, void *d_workspace, size_t ws_bytes, dq_stats *d_stats,
                                     void *stream) {
  int rc = check_page_table(d_page_table, num_pages, max_pages);
  if (rc == DQ_OK) rc = check_window(window, sinks, sm_scale);
  if (rc != DQ_OK) return rc;
  return decode_core(t, q, q_dtype, d_kpool, d_vpool, d_seq_lens, B, Hq, Hkv, 32 * max_pages, T_max, sm_scale, out,
                     out_dtype, d_workspace, ws_bytes, d_stats, stream, d_page_table, max_pages, num_pages, window,
                     sinks);
}

// Bytes of one (b, KV head) row of the prefill workspace.
static size_t prefill_row_bytes(int64_t T_cap, int n_q, int64_t window, int64_t sinks) {
  return static_cast<size_t>(dqi::prefill_row_slots(T_cap, n_q, window, sinks)) * dqi::prefill_slot_bytes();
}

static int prefill_core(const dq_tables *t, const void *q, int q_dtype, const uint8_t *d_kcache,
                        const uint8_t *d_vcache, const int32_t *d_q_start, int B, int n_q, int Hq, int Hkv,
                        int64_t T_cap, float sm_scale, void *out, int out_dtype, void *d_workspace,
                        size_t ws_bytes, dq_stats *d_stats, void *stream, const int32_t *page_table,
                        int64_t max_pages, int64_t num_pages, int64_t window = 0, int64_t sinks = 0) {
  try {
    if (!t || !q || !d_kcache || !d_vcache || !d_q_start || !out || !d_workspace) return DQ_ERR_NULL;
    if ((q_dtype != DQ_F32 && q_dtype != DQ_BF16) || (out_dtype != DQ_F32 && out_dtype != DQ_BF16))
      return DQ_ERR_DTYPE;
    if (B < 0 || n_q < 0 || Hkv != t->cfg.n_kv_heads || Hq < Hkv || Hq % Hkv) return DQ_ERR_SHAPE;
    const int G = Hq / Hkv;
    if (G != 1 && G != 2 && G != 4 && G != 8) return DQ_ERR_SHAPE;
    if (T_cap < 0) return DQ_ERR_SHAPE;
    if (T_cap % 32 || !aligned(d_kcache, 16) || !aligned(d_vcache, 16) || !aligned(q, 4) || !aligned(out, 4) ||
        !aligned(d_q_start, 4) || !aligned(d_workspace, 16))
      return DQ_ERR_ALIGN;
    if (!std::isfinite(sm_scale)) return DQ_ERR_SHAPE;
    if (!dqi::prefill_supported(t->k.container_bytes, t->v.container_bytes)) return DQ_ERR_SHAPE;
    // The workspace holds the decoded tiles of a wave of (b, KV head) rows:
    // at least one row; a smaller workspace than the whole batch's runs the
    // call in several waves.
    const int64_t rows = static_cast<int64_t>(B) * Hkv;
    // (A window of T_cap tokens or more hides nothing; at least 1 keeps the windowed kernels.)
    window = window > 0 ? std::max<int64_t>(1, std::min(window, T_cap)) : 0;
    sinks = std::min(sinks, T_cap);
    const size_t row_bytes = prefill_row_bytes(T_cap, n_q, window, sinks);
    if (T_cap > 0 && ws_bytes < row_bytes) return DQ_ERR_WORKSPACE;
    const int64_t per_wave = row_bytes ? std::min<int64_t>(rows, static_cast<int64_t>(ws_bytes / row_bytes)) : rows;
    if (per_wave > 0 && dqi::prefill_grid(per_wave, G, n_q) > 0x7FFFFFFF) return DQ_ERR_SHAPE;
    int rc = check_device(t);
    if (rc != DQ_OK) return rc;
    if (B == 0 || n_q == 0 || T_cap == 0) {
      if (B > 0 && n_q > 0) {  // no cache: every row is outside it, out = 0
        const size_t n = static_cast<size_t>(B) * n_q * Hq * dqi::kD * (out_dtype == DQ_F32 ? 4 : 2);
        cudaError_t e = cudaMemsetAsync(out, 0, n, static_cast<cudaStream_t>(stream));
        if (e != cudaSuccess) return cuda_fail(e);
      }
      return DQ_OK;
    }
    dqi::PrefillArgs a{};
    a.tabs = t->d_tabs;
    a.sign_bits = t->d_sign_bits;
    a.q = q;
    a.q_dtype = q_dtype;
    a.kcache = d_kcache;
    a.vcache = d_vcache;
    a.q_start = d_q_start;
    a.B = B;
    a.n_q = n_q;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = G;
    a.T_cap = T_cap;
    a.sm_scale = sm_scale;
    a.out = out;
    a.out_dtype = out_dtype;
    a.ck = t->k.container_bytes;
    a.cv = t->v.container_bytes;
    a.two_k = has_small_freq(t->k);
    a.two_v = has_small_freq(t->v);
    a.tiles = static_cast<uint8_t *>(d_workspace);
    a.nslots = dqi::prefill_ring_slots();
    a.window = window;
    a.sinks = sinks;
    a.row_slots = dqi::prefill_row_slots(T_cap, n_q, window, sinks);
    a.stats = d_stats;
    a.page_table = page_table;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    for (int64_t bh0 = 0; bh0 < rows; bh0 += per_wave) {
      a.bh0 = bh0;
      a.nbh = std::min<int64_t>(per_wave, rows - bh0);
      const int64_t groups = a.nbh * std::min<int64_t>(T_cap / 32, a.row_slots * 4);
      a.tile_grid = static_cast<int>(std::min<int64_t>(t->sm_count, window > 0 ? groups : (groups + 19) / 20));
      int e = dqi::launch_prefill_attention(a, stream);
      if (e != 0) return cuda_fail(static_cast<cudaError_t>(e));
    }
    return DQ_OK;
  } catch (...) {
    return DQ_ERR_CUDA;
  }
}

size_t dq_prefill_workspace_bytes(const dq_tables *t, int B, int Hkv, int64_t T_cap) {
  if (!t || B < 0 || Hkv < 1 || T_cap < 0 || T_cap % 32) return 0;
  return std::max<size_t>(16, static_cast<size_t>(B) * Hkv * prefill_row_bytes(T_cap, 0, 0, 0));
}

size_t dq_prefill_window_workspace_bytes(const dq_tables *t, int B, int Hkv, int64_t T_cap, int n_q, int64_t window,
                                         int64_t sinks) {
  if (!t || B < 0 || Hkv < 1 || T_cap < 0 || T_cap % 32 || n_q < 0 || window < 1 || sinks < 0) return 0;
  window = std::max<int64_t>(1, std::min(window, T_cap));
  return std::max<size_t>(16, static_cast<size_t>(B) * Hkv * prefill_row_bytes(T_cap, n_q, window, std::min(sinks, T_cap)));
}

int dq_prefill_attention(const dq_tables *t, const void *q, int q_dtype, const uint8_t *d_kcache,
                         const uint8_t *d_vcache, const int32_t *d_q_start, int B, int n_q, int Hq, int Hkv,
                         int64_t T_cap, float sm_scale, void *out, int out_dtype, void *d_workspace,
                         size_t ws_bytes, dq_stats *d_stats, void *stream) {
  return prefill_core(t, q, q_dtype, d_kcache, d_vcache, d_q_start, B, n_q, Hq, Hkv, T_cap, sm_scale, out,
                      out_dtype, d_workspace, ws_bytes, d_stats, stream, nullptr, 0, 0);
}

int dq_prefill_attention_paged(const dq_tables *t, const void *q, int q_dtype, const uint8_t *d_kpool,
                               const uint8_t *d_vpool, int64_t num_pages, const int32_t *d_page_table,
                               int64_t max_pages, const int32_t *d_q_start, int B, int n_q, int Hq, int Hkv,
                               float sm_scale, void *out, int out_dtype, void *d_workspace, size_t ws_bytes,
                               dq_stats *d_stats, void *stream) {
  const int rc = check_page_table(d_page_table, num_pages, max_pages);
  if (rc != DQ_OK) return rc;
  return prefill_core(t, q, q_dtype, d_kpool, d_vpool, d_q_start, B, n_q, Hq, Hkv, 32 * max_pages, sm_scale, out,
                      out_dtype, d_workspace, ws_bytes, d_stats, stream, d_page_table, max_pages, num_pages);
}

int dq_prefill_attention_window(const dq_tables *t, const void *q, int q_dtype, const uint8_t *d_kcache,
                                const uint8_t *d_vcache, const int32_t *d_q_start, int B, int n_q, int Hq, int Hkv,
                                int64_t T_cap, int64_t window, int64_t sinks, float sm_scale, void *out,
                                int out_dtype, void *d_workspace, size_t ws_bytes, dq_stats *d_stats, void *stream) {
  const int rc = check_window(window, sinks, sm_scale);
  if (rc != DQ_OK) return rc;
  return prefill_core(t, q, q_dtype, d_kcache, d_vcache, d_q_start, B, n_q, Hq, Hkv, T_cap, sm_scale, out, out_dtype,
                      d_workspace, ws_bytes, d_stats, stream, nullptr, 0, 0, window, sinks);
}

int dq_prefill_attention_window_paged(const dq_tables *t, const void *q, int q_dtype, const uint8_t *d_kpool,
                                      const uint8_t *d_vpool, int64_t num_pages, const int32_t *d_page_table,
                                      int64_t max_pages, const int32_t *d_q_start, int B, int n_q, int Hq, int Hkv,
                                      int64_t window, int64_t sinks, float sm_scale, void *out, int out_dtype,
                                      void *d_workspace, size_t ws_bytes, dq_stats *d_stats, void *stream) {
  int rc = check_page_table(d_page_table, num_pages, max_pages);
  if (rc == DQ_OK) rc = check_window(window, sinks, sm_scale);
  if (rc != DQ_OK) return rc;
  return prefill_core(t, q, q_dtype, d_kpool, d_vpool, d_q_start, B, n_q, Hq, Hkv, 32 * max_pages, sm_scale, out,
                      out_dtype, d_workspace, ws_bytes, d_stats, stream, d_page_table, max_pages, num_pages, window,
                      sinks);
}

size_t dq_pages_workspace_bytes(const dq_tables *t, int64_t num_pages, int B, int64_t max_pages) {
  if (!t || num_pages < 1 || num_pages > 0x7FFFFFFF || B < 0 || max_pages < 1 || max_pages > kMaxTablePages) return 0;
  return dqi::pages_layout(num_pages, B, max_pages).total;
}

// An array of the bookkeeping calls.
struct Span {
  const void *p;
  int64_t bytes;
};
static bool share_bytes(const Span &a, const Span &b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.bytes > 0 && b.bytes > 0 && x < y + static_cast<uintptr_t>(b.bytes) &&
         y < x + static_cast<uintptr_t>(a.bytes);
}
// The kernels read their inputs again after they have begun to write: an
// output shares no byte with an input or with another output, but for the
// first `own` of them, which may be the input of the same index itself.
static int check_apart(std::initializer_list<Span> in, std::initializer_list<Span> out, size_t own) {
  for (size_t o = 0; o < out.size(); ++o) {
    const Span &x = out.begin()[o];
    for (size_t i = 0; i < in.size(); ++i)
      if (share_bytes(x, in.begin()[i]) && !(i == o && i < own && x.p == in.begin()[i].p)) return DQ_ERR_SHAPE;
    for (size_t i = 0; i < o; ++i)
      if (share_bytes(x, out.begin()[i])) return DQ_ERR_SHAPE;
  }
  return DQ_OK;
}
// Bytes of int32 arrays (0 for sizes that pages_args refuses) and of the workspace that is used.
static int64_t int_bytes(int64_t rows, int64_t each) {
  return rows > 0 && rows <= 0x7FFFFFFF && each > 0 && each <= 2 * kMaxTablePages ? 4 * rows * each : 0;
}
static int64_t used_bytes(int64_t num_pages, int64_t max_pages, int B, size_t ws_bytes) {
  if (num_pages < 1 || num_pages > 0x7FFFFFFF || max_pages < 1 || max_pages > kMaxTablePages || B < 0) return 0;
  return static_cast<int64_t>(std::min(ws_bytes, dqi::pages_layout(num_pages, B, max_pages).total));
}

// Checks and arguments that the bookkeeping calls share; rows of the old and
// the new table. Arrays of no rows may be NULL.
static int pages_args(const dq_tables *t, int64_t num_pages, int64_t max_pages, const int32_t *d_refs,
                      const int32_t *d_table, int B_in, int32_t *d_refs_out, int32_t *d_table_out, int B_out,
                      int32_t *d_counts, void *d_workspace, size_t ws_bytes, dqi::PagesArgs *a) {
  if (!t || !d_refs || !d_refs_out || !d_counts || !d_workspace || (B_in > 0 && !d_table) || (B_out > 0 && !d_table_out))
    return DQ_ERR_NULL;
  if (num_pages < 1 || num_pages > 0x7FFFFFFF || max_pages < 1 || max_pages > kMaxTablePages || B_in < 0 || B_out < 0)
    return DQ_ERR_SHAPE;
  if (!aligned(d_refs, 4) || !aligned(d_table, 4) || !aligned(d_refs_out, 4) || !aligned(d_table_out, 4) ||
      !aligned(d_counts, 4) || !aligned(d_workspace, 16))
    return DQ_ERR_ALIGN;
  const dqi::PagesLayout l = dqi::pages_layout(num_pages, std::max(B_in, B_out), max_pages);
  if (ws_bytes < l.total) return DQ_ERR_WORKSPACE;
  const int rc = check_device(t);
  if (rc != DQ_OK) return rc;
  uint8_t *ws = static_cast<uint8_t *>(d_workspace);
  auto at = [&](size_t off) { return reinterpret_cast<int32_t *>(ws + off); };
  *a = dqi::PagesArgs{};
  a->num_pages = num_pages;
  a->max_pages = max_pages;
  a->B_in = B_in;
  a->B_out = B_out;
  a->refs_in = d_refs;
  a->table_in = d_table;
  a->refs_out = d_refs_out;
  a->table_out = d_table_out;
  a->counts = d_counts;
  a->list = at(l.list);
  a->item_need = at(l.need);
  a->item_lo = at(l.lo);
  a->item_hi = at(l.hi);
  a->map = a->children = at(l.map);
  a->movers = a->first = at(l.movers);
  return DQ_OK;
}

int dq_pages_advance(const dq_tables *t, int64_t num_pages, const int32_t *d_refs, const int32_t *d_page_table,
                     int64_t max_pages, const int32_t *d_lens, const int32_t *d_n_new, int B, int64_t window,
                     int64_t sinks, int32_t *d_refs_out, int32_t *d_page_table_out, int32_t *d_lens_out,
                     dq_page_counts *d_counts, void *d_workspace, size_t ws_bytes, void *stream) {
  try {
    if (B > 0 && (!d_lens || !d_n_new || !d_lens_out)) return DQ_ERR_NULL;
    if (window < 0 || sinks < 0) return DQ_ERR_SHAPE;
    if (!aligned(d_lens, 4) || !aligned(d_n_new, 4) || !aligned(d_lens_out, 4)) return DQ_ERR_ALIGN;
    const int64_t refs = int_bytes(num_pages, 1), rows = int_bytes(B, 1), table = int_bytes(B, max_pages);
    // (n_new may be lens_out: a row's number is read by the thread that then writes its length.)
    int rc = check_apart({{d_refs, refs}, {d_page_table, table}, {d_lens, rows}, {d_n_new, d_n_new == d_lens_out ? 0 : rows}},
                         {{d_refs_out, refs}, {d_page_table_out, table}, {d_lens_out, rows}, {d_counts, sizeof(dq_page_counts)},
                          {d_workspace, used_bytes(num_pages, max_pages, B, ws_bytes)}},
                         3);
    if (rc != DQ_OK) return rc;
    dqi::PagesArgs a;
    rc = pages_args(t, num_pages, max_pages, d_refs, d_page_table, B, d_refs_out, d_page_table_out, B,
                    reinterpret_cast<int32_t *>(d_counts), d_workspace, ws_bytes, &a);
    if (rc != DQ_OK) return rc;
    a.lens_in = d_lens;
    a.step = d_n_new;
    a.lens_out = d_lens_out;
    a.window = std::min<int64_t>(window, int64_t(1) << 40);  // (any length is below)
    a.sinks = std::min<int64_t>(sinks, int64_t(1) << 40);
    const int e = dqi::launch_pages_advance(a, t->sm_count, stream);
    return e == 0 ? DQ_OK : cuda_fail(static_cast<cudaError_t>(e));
  } catch (...) {
    return DQ_ERR_CUDA;
  }
}

int dq_pages_fork(const dq_tables *t, int64_t num_pages, const int32_t *d_refs, const int32_t *d_page_table,
                  int64_t max_pages, const int32_t *d_lens, int B_in, const int32_t *d_parent, int B_out,
                  int32_t *d_refs_out, int32_t *d_page_table_out, int32_t *d_lens_out, int32_t *d_pairs,
                  dq_page_counts *d_counts, void *d_workspace, size_t ws_bytes, void *stream) {
  try {
    if ((B_in > 0 && !d_lens) || (B_out > 0 && (!d_parent || !d_lens_out || !d_pairs))) return DQ_ERR_NULL;
    if (!aligned(d_lens, 4) || !aligned(d_parent, 4) || !aligned(d_lens_out, 4) || !aligned(d_pairs, 4))
      return DQ_ERR_ALIGN;
    const int64_t refs = int_bytes(num_pages, 1), rows = int_bytes(B_out, 1);
    int rc = check_apart({{d_refs, refs}, {d_page_table, int_bytes(B_in, max_pages)}, {d_lens, int_bytes(B_in, 1)}, {d_parent, rows}},
                         {{d_refs_out, refs}, {d_page_table_out, int_bytes(B_out, max_pages)}, {d_lens_out, rows},
                          {d_pairs, int_bytes(B_out, 2)}, {d_counts, sizeof(dq_page_counts)},
                          {d_workspace, used_bytes(num_pages, max_pages, std::max(B_in, B_out), ws_bytes)}},
                         0);
    if (rc != DQ_OK) return rc;
    dqi::PagesArgs a;
    rc = pages_args(t, num_pages, max_pages, d_refs, d_page_table, B_in, d_refs_out, d_page_table_out, B_out,
                    reinterpret_cast<int32_t *>(d_counts), d_workspace, ws_bytes, &a);
    if (rc != DQ_OK) return rc;
    a.lens_in = d_lens;
    a.step = d_parent;
    a.lens_out = d_lens_out;
    a.pairs = d_pairs;
    const int e = dqi::launch_pages_fork(a, stream);
    return e == 0 ? DQ_OK : cuda_fail(static_cast<cudaError_t>(e));
  } catch (...) {
    return DQ_ERR_CUDA;
  }
}

int dq_pages_compact(const dq_tables *t, int64_t num_pages, const int32_t *d_refs, const int32_t *d_page_table,
                     int64_t max_pages, int B, int32_t *d_refs_out, int32_t *d_page_table_out, int32_t *d_pairs,
                     dq_page_counts *d_counts, void *d_workspace, size_t ws_bytes, void *stream) {
  try {
    if (!d_pairs) return DQ_ERR_NULL;
    if (!aligned(d_pairs, 4)) return DQ_ERR_ALIGN;
    const int64_t refs = int_bytes(num_pages, 1), table = int_bytes(B, max_pages);
    int rc = check_apart({{d_refs, refs}, {d_page_table, table}},
                         {{d_refs_out, refs}, {d_page_table_out, table}, {d_pairs, int_bytes(std::max<int64_t>(1, num_pages / 2), 2)},
                          {d_counts, sizeof(dq_page_counts)}, {d_workspace, used_bytes(num_pages, max_pages, B, ws_bytes)}},
                         2);
    if (rc != DQ_OK) return rc;
    dqi::PagesArgs a;
    rc = pages_args(t, num_pages, max_pages, d_refs, d_page_table, B, d_refs_out, d_page_table_out, B,
                    reinterpret_cast<int32_t *>(d_counts), d_workspace, ws_bytes, &a);
    if (rc != DQ_OK) return rc;
    a.pairs = d_pairs;
    const int e = dqi::launch_pages_compact(a, stream);
    return e == 0 ? DQ_OK : cuda_fail(static_cast<cudaError_t>(e));
  } catch (...) {
    return DQ_ERR_CUDA;
  }
}

int dq_pages_copy(const dq_tables *t, uint8_t *d_kpool, uint8_t *d_vpool, int64_t num_pages, int64_t n_layers,
                  int64_t k_layer_stride, int64_t v_layer_stride, const int32_t *d_pairs, int64_t max_pairs,
                  const dq_page_counts *d_counts, dq_stats *d_stats, void *stream) {
  try {
    if (!t || !d_kpool || !d_vpool || (max_pairs > 0 && !d_pairs)) return DQ_ERR_NULL;
    if (num_pages < 1 || num_pages > (int64_t(1) << 31) || n_layers < 0 || n_layers > (1 << 20) || max_pairs < 0 ||
        max_pairs > (int64_t(1) << 31))
      return DQ_ERR_SHAPE;
    if (!aligned(d_kpool, 16) || !aligned(d_vpool, 16) || k_layer_stride % 16 || v_layer_stride % 16 ||
        !aligned(d_pairs, 4) || !aligned(d_counts, 4))
      return DQ_ERR_ALIGN;
    const int rc = check_device(t);
    if (rc != DQ_OK) return rc;
    if (n_layers == 0 || max_pairs == 0) return DQ_OK;
    dqi::CopyArgs a{};
    a.kpool = d_kpool;
    a.vpool = d_vpool;
    a.num_pages = num_pages;
    a.n_layers = n_layers;
    a.k_stride = k_layer_stride;
    a.v_stride = v_layer_stride;
    a.k_bytes = static_cast<int64_t>(t->cfg.n_kv_heads) * 32 * t->k.container_bytes;
    a.v_bytes = static_cast<int64_t>(t->cfg.n_kv_heads) * 32 * t->v.container_bytes;
    a.pairs = d_pairs;
    a.max_pairs = max_pairs;
    a.counts = reinterpret_cast<const int32_t *>(d_counts);
    a.stats = d_stats;
    const int e = dqi::launch_pages_copy(a, t->sm_count, stream);
    return e == 0 ? DQ_OK : cuda_fail(static_cast<cudaError_t>(e));
  } catch (...) {
    return DQ_ERR_CUDA;
  }
}

int dq_decode_symbols(const dq_tables *t, const uint8_t *d_cache, int stream_kind,
                      int64_t n_containers, uint8_t *d_syms, uint16_t *d_norm16, int32_t *d_status,
                      dq_stats *d_stats, void *stream) {
  try {
    if (!t || !d_cache || !d_syms || !d_norm16) return DQ_ERR_NULL;
    if (stream_kind != DQ_STREAM_K && stream_kind != DQ_STREAM_V) return DQ_ERR_CONFIG;
    if (n_containers < 0) return DQ_ERR_SHAPE;
    if (!aligned(d_cache, 4)) return DQ_ERR_ALIGN;
    int rc = check_device(t);
    if (rc != DQ_OK) return rc;
    if (n_containers == 0) return DQ_OK;
    dqi::SymbolsArgs a{};
    a.tab = stream_kind == DQ_STREAM_K ? &t->d_tabs->k : &t->d_tabs->v;
    a.cache = d_cache;
    a.n = n_containers;
    a.c = stream_kind == DQ_STREAM_K ? t->k.container_bytes : t->v.container_bytes;
    a.syms = d_syms;
    a.norm16 = d_norm16;
    a.status = d_status;
    a.stats = d_stats;
    int e = dqi::launch_decode_symbols(a, stream);
    return e == 0 ? DQ_OK : cuda_fail(static_cast<cudaError_t>(e));
  } catch (...) {
    return DQ_ERR_CUDA;
  }
}

}  // extern "C"
