// Host side of the C ABI declared in include/ditango.h: argument checks,
// the kernels' geometry, TMA tensor maps and launches.  No device memory is
// allocated here.
#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>

#include <nvtx3/nvToolsExt.h>

#include "common.cuh"

namespace ditango {
cudaError_t launch_attn_partial(const DevGeom &g, const CUtensorMap &tq, const CUtensorMap &tk,
                                const CUtensorMap &tv, const int *fresh_list, const int *counts,
                                float scale, void *out_O, float *out_lse, int out_by_slot,
                                int state_bf16, unsigned char *out_valid, float *drift_rows,
                                int *dev_status, long long wait_limit_ns, int num_sms,
                                int *work_counter, cudaStream_t stream);
int attn_key_tile(int d);
size_t plan_workspace_bytes(const DevGeom &g);
cudaError_t launch_plan(const DevGeom &g, const float *cache_lse, const unsigned char *cache_valid,
                        int band_k, int target, int anchor, signed char *plan_out, int *fresh_list,
                        int *counts, float *score_out, void *workspace, cudaStream_t stream,
                        const float *drift_rows, float *w_hold, float *age, float *delta,
                        unsigned char *local_ok, int refresh_w, int mass_given);
cudaError_t launch_merge(const DevGeom &g, const signed char *plan, const void *part_O,
                         const float *part_lse, void *cache_O, float *cache_lse,
                         unsigned char *cache_valid, int writeback, int state_bf16, void *out,
                         int out_is_fp32, long long osb, long long osh, long long osn,
                         float *out_lse, float *mass_partials, cudaStream_t stream);
cudaError_t launch_cache_update(const DevGeom &g, const signed char *plan, const void *part_O,
                                const float *part_lse, void *cache_O, float *cache_lse,
                                unsigned char *cache_valid, int state_bf16, int num_sms,
                                cudaStream_t stream);
cudaError_t launch_cache_compose(const DevGeom &fine, const DevGeom &coarse, const void *fine_O,
                                 const float *fine_lse, const unsigned char *fine_valid,
                                 void *coarse_O, float *coarse_lse, unsigned char *coarse_valid,
                                 int state_bf16, cudaStream_t stream);
cudaError_t launch_bounded_wait_selftest(long long limit_ns, int *dev_status,
                                         cudaStream_t stream);
cudaError_t launch_block_tables(int R, int max_blocks, int max_tokens, int n_pages, const int *ctx_len,
                                const int *new_len, const int *free_pages, int n_free, int *block_table,
                                int *kv_len, int *q_off, long long *slot_map, int *pages_used,
                                int *dev_status, int num_sms, cudaStream_t stream);
cudaError_t launch_kv4_rows(bool write, long long T, int Hkv, int d, int n_pages, const uint16_t *K,
                            const uint16_t *V, uint16_t *Ko, uint16_t *Vo, const int64_t *k_strides,
                            const int64_t *v_strides, const long long *slots, uint8_t *data,
                            int *dev_status, int num_sms, cudaStream_t stream);
cudaError_t launch_kv4_summary(int R, int Hkv, int d, int max_blocks, int n_pages, const int *ctx_len,
                               const int *kv_len, const int *block_table, const uint8_t *data,
                               signed char *codes, float *scale, int *dev_status, cudaStream_t stream);
size_t kv4_attn_workspace_bytes(int d);
cudaError_t launch_kv4_attn(int R, int H, int Hkv, int d, int T, int max_q, int max_blocks, int n_pages,
                            const uint16_t *Q, const int64_t *q_strides, const int *q_off,
                            const int *kv_len, const int *block_table, const uint8_t *data,
                            const int *sel, const int *sel_count, int max_sel, float scale, int causal,
                            void *out, int out_fp32, const int64_t *out_strides, float *out_lse,
                            const int64_t *lse_strides, void *workspace, int *dev_status,
                            long long wait_limit_ns, int num_sms, cudaStream_t stream);
cudaError_t launch_block_summary(int B, int H, int N, int d, int block, const uint16_t *x,
                                 const int64_t *s, const int *len, signed char *codes, float *scale,
                                 float *mean, cudaStream_t stream);
cudaError_t launch_block_summaries(int B, int H, int Hkv, int Nq, int Nk, int d, const uint16_t *Q,
                                   const int64_t *qst, const uint16_t *K, const int64_t *kst, const int *k_len,
                                   signed char *q_codes, float *q_scale, signed char *k_codes, float *k_scale,
                                   float *k_mean, cudaStream_t stream);
int select_max_blocks();
bool select_by_heads(int n_q, int G, int n_k);
cudaError_t launch_block_select(int B, int H, int Hkv, int n_q, int n_k, int d, int k, int band, int sink,
                                int room, int own, const signed char *qc, const float *qs,
                                const signed char *kc, const float *ks, const int *block_table,
                                int n_pages, const int *k_len, int *sel_out, int *count,
                                int *dev_status, const uint16_t *q, const int64_t *q_strides,
                                cudaStream_t stream);
cudaError_t launch_block_attn(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, int B,
                              int H, int Hkv, int Nq, int Nk, int d, const int *sel, const int *count,
                              int room, const int *k_len, float scale, void *out, int out_fp32,
                              const long long *os, float *out_lse, const long long *ls,
                              int *dev_status, long long wait_limit_ns, int num_sms,
                              cudaStream_t stream);
cudaError_t attn_check_status(int *out, bool reset);
cudaError_t merge_check_status(int *out, bool reset);
}  // namespace ditango

using namespace ditango;

namespace {

// An NVTX range over one entry point (shown by profilers; without one
// attached a push/pop costs a few nanoseconds).
struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

// Process-wide limit of every device wait; set from any host thread.
std::atomic<long long> g_wait_limit_ns{1000000000LL};

// Build the kernels' geometry; returns DITANGO_OK or the reason it cannot.
ditango_status make_geom(const ditango_geom *in, DevGeom *out) {
  if (!in) return DITANGO_ERR_INVALID;
  if (in->B < 1 || in->H < 1 || in->N < 1 || in->P < 1 || in->d < 1) return DITANGO_ERR_INVALID;
  if (in->P > kMaxP) return DITANGO_ERR_UNSUPPORTED;
  if (!(in->d == 64 || in->d == 96 || in->d == 128)) return DITANGO_ERR_UNSUPPORTED;
  if ((long long)in->B * in->H > 65535) return DITANGO_ERR_UNSUPPORTED;  // grid.z of the merge
  if (!in->part_off) return DITANGO_ERR_INVALID;
  if (in->part_off[0] != 0 || in->part_off[in->P] != in->N) return DITANGO_ERR_INVALID;
  for (int p = 0; p < in->P; ++p)
    if (in->part_off[p + 1] <= in->part_off[p]) return DITANGO_ERR_INVALID;
  if (in->F < 0 || in->F > kMaxP) return in->F < 0 ? DITANGO_ERR_INVALID : DITANGO_ERR_UNSUPPORTED;
  // frames of the first and the last token of every partition
  int f_lo[kMaxP], f_hi[kMaxP];
  if (in->F > 0) {
    if (!in->frame_off || !in->frame_mask) return DITANGO_ERR_INVALID;
    if (in->frame_off[0] != 0 || in->frame_off[in->F] != in->N) return DITANGO_ERR_INVALID;
    for (int f = 0; f < in->F; ++f)
      if (in->frame_off[f + 1] <= in->frame_off[f]) return DITANGO_ERR_INVALID;
    for (int p = 0, f = 0; p < in->P; ++p) {
      while (in->frame_off[f + 1] <= in->part_off[p]) ++f;
      f_lo[p] = f;
      int e = f;
      while (in->frame_off[e + 1] < in->part_off[p + 1]) ++e;
      f_hi[p] = e;
    }
  }
  DevGeom g;
  std::memset(&g, 0, sizeof(g));
  g.B = in->B;
  g.H = in->H;
  g.N = in->N;
  g.d = in->d;
  g.P = in->P;
  g.BH = in->B * in->H;
  int lmax = 0;
  for (int p = 0; p <= in->P; ++p) g.part_off[p] = in->part_off[p];
  for (int p = 0; p < in->P; ++p) {
    int L = in->part_off[p + 1] - in->part_off[p];
    if (L > lmax) lmax = L;
  }
  g.Lmax = lmax;
  // KV groups: runs of adjacent partitions (one per partition without groups)
  if (in->G < 0 || in->G > in->P) return DITANGO_ERR_INVALID;
  if (in->G == 0) {
    g.G = in->P;
    for (int c = 0; c <= in->P; ++c) g.group_off[c] = c;
  } else {
    if (!in->group_off || in->group_off[0] != 0 || in->group_off[in->G] != in->P)
      return DITANGO_ERR_INVALID;
    for (int c = 0; c < in->G; ++c)
      if (in->group_off[c + 1] <= in->group_off[c]) return DITANGO_ERR_INVALID;
    g.G = in->G;
    for (int c = 0; c <= in->G; ++c) g.group_off[c] = in->group_off[c];
  }
  for (int c = 0; c < g.G; ++c)
    for (int j = g.group_off[c]; j < g.group_off[c + 1]; ++j) g.part_group[j] = (signed char)c;
  // Pair (i, j) is active when some token of partition i may attend some
  // token of partition j.  When a partition straddles frames, an active
  // pair can also hold token pairs the mask forbids: the kernels then mask
  // those logits one by one (token_mask).
  g.F = in->F;
  g.token_mask = 0;
  if (in->F > 0) {
    for (int f = 0; f <= in->F; ++f) g.frame_off[f] = in->frame_off[f];
    for (int f = 0; f < in->F; ++f) {
      unsigned long long a = 0;
      for (int f2 = 0; f2 < in->F; ++f2)
        if (in->frame_mask[f * in->F + f2]) a |= 1ull << f2;
      g.frame_allow[f] = a;
    }
  }
  for (int i = 0; i < in->P; ++i) {
    unsigned long long m = 0;
    for (int j = 0; j < in->P; ++j) {
      if (in->F == 0) {
        m |= 1ull << j;
        continue;
      }
      const unsigned long long kf = bit_range(f_lo[j], f_hi[j] + 1);   // key frames of j
      bool any = false, all = true;
      for (int f = f_lo[i]; f <= f_hi[i]; ++f) {
        const unsigned long long hit = g.frame_allow[f] & kf;
        any = any || hit != 0ull;
        all = all && hit == kf;
      }
      if (any) {
        m |= 1ull << j;
        if (!all) g.token_mask = 1;
      }
    }
    g.pair_mask[i] = m;
  }
  int slot = 0;
  for (int i = 0; i < in->P; ++i) {
    g.row_start[i] = slot;
    unsigned long long m = 0;
    for (int c = 0; c < g.G; ++c)
      if (unit_pairs(g, i, c)) {
        m |= 1ull << c;
        ++slot;
      }
    g.row_mask[i] = m;
  }
  g.row_start[in->P] = slot;
  g.n_active = slot;
  g.multi_run = 0;
  for (int i = 0; i < in->P; ++i)
    for (int c = 0; c < g.G; ++c) {
      const unsigned long long b = unit_pairs(g, i, c);
      if (!b) continue;
      const unsigned long long sh = b >> __builtin_ctzll(b);
      if (sh & (sh + 1ull)) g.multi_run = 1;   // a gap between active partitions
    }
  *out = g;
  return DITANGO_OK;
}

// Fresh-unit count of a plan: max(|band|, floor(budget * active + 1e-9)).
int plan_target(DevGeom *dg, int band_k, double budget) {
  int n_band = 0;
  for (int i = 0; i < dg->P; ++i)
    for (int c = 0; c < dg->G; ++c)
      if (((dg->row_mask[i] >> c) & 1ull) && unit_in_band(*dg, i, c, band_k)) ++n_band;
  int target = (int)std::floor(budget * (double)dg->n_active + 1e-9);
  if (target < n_band) target = n_band;
  if (target > dg->n_active) target = dg->n_active;
  dg->n_band = n_band;
  return target;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool strides_ok(const int64_t s[3]) {
  for (int k = 0; k < 3; ++k)
    if (s[k] <= 0 || ((s[k] * 2) % 16) != 0 || s[k] * 2 >= (1LL << 40)) return false;
  return true;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, []() {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 4-D map over a bf16 [B, H, N, d] tensor (d contiguous), box 64 columns x
// box_rows rows, 128-byte swizzle; columns past d and rows past N read as zero.
bool make_qkv_map(CUtensorMap *m, const void *base, const DevGeom &g, const int64_t s[3],
                  unsigned box_rows) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  cuuint64_t dims[4] = {(cuuint64_t)g.d, (cuuint64_t)g.N, (cuuint64_t)g.H, (cuuint64_t)g.B};
  cuuint64_t strides[3] = {(cuuint64_t)(s[2] * 2), (cuuint64_t)(s[1] * 2), (cuuint64_t)(s[0] * 2)};
  cuuint32_t box[4] = {64, box_rows, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

int num_sms_current() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) != cudaSuccess) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
  return n;
}

ditango_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return DITANGO_OK;
  (void)cudaGetLastError();
  return DITANGO_ERR_CUDA;
}

}  // namespace

extern "C" {

int32_t ditango_version(void) { return 10400; }

const char *ditango_status_string(int32_t s) {
  switch (s) {
    case DITANGO_OK: return "ok";
    case DITANGO_ERR_INVALID: return "invalid argument";
    case DITANGO_ERR_UNSUPPORTED: return "unsupported shape";
    case DITANGO_ERR_CUDA: return "CUDA error";
    case DITANGO_ERR_TIMEOUT: return "device wait timed out";
    case DITANGO_ERR_BOUNDS: return "device input out of range";
    default: return "unknown status";
  }
}

ditango_status ditango_check_geom(const ditango_geom *g) {
  DevGeom dg;
  return make_geom(g, &dg);
}

int64_t ditango_num_active(const ditango_geom *g) {
  DevGeom dg;
  if (make_geom(g, &dg) != DITANGO_OK) return -1;
  return dg.n_active;
}

int64_t ditango_state_rows(const ditango_geom *g) {
  DevGeom dg;
  if (make_geom(g, &dg) != DITANGO_OK) return -1;
  return dg.Lmax;
}

ditango_status ditango_slot_table(const ditango_geom *g, int32_t *slot_out) {
  DevGeom dg;
  ditango_status st = make_geom(g, &dg);
  if (st != DITANGO_OK) return st;
  if (!slot_out) return DITANGO_ERR_INVALID;
  for (int i = 0; i < dg.P; ++i)
    for (int c = 0; c < dg.G; ++c)
      slot_out[i * dg.G + c] = ((dg.row_mask[i] >> c) & 1ull) ? slot_of(dg, i, c) : -1;
  return DITANGO_OK;
}

size_t ditango_plan_workspace_size(const ditango_geom *g) {
  DevGeom dg;
  if (make_geom(g, &dg) != DITANGO_OK) return 0;
  return plan_workspace_bytes(dg);
}

size_t ditango_workspace_size(const ditango_geom *g) { return ditango_plan_workspace_size(g); }

ditango_status ditango_plan(const ditango_geom *g, const float *cache_lse,
                            const uint8_t *cache_valid, int32_t band_k, double budget,
                            int32_t anchor, int8_t *plan, int32_t *fresh_list, int32_t *counts,
                            float *score_out, void *workspace, size_t workspace_bytes,
                            ditango_stream stream) {
  NvtxRange nvtx_range("ditango_plan");
  DevGeom dg;
  ditango_status st = make_geom(g, &dg);
  if (st != DITANGO_OK) return st;
  if (!plan || !fresh_list || !counts) return DITANGO_ERR_INVALID;
  if (!anchor) {
    if (!cache_lse || band_k < 0 || !(budget >= 0.0 && budget <= 1.0)) return DITANGO_ERR_INVALID;
    if (!workspace || workspace_bytes < plan_workspace_bytes(dg)) return DITANGO_ERR_INVALID;
  }
  const int target = plan_target(&dg, band_k, budget);
  return cuda_status(launch_plan(dg, cache_lse, cache_valid, band_k, target, anchor ? 1 : 0,
                                 reinterpret_cast<signed char *>(plan), fresh_list, counts,
                                 score_out, workspace, static_cast<cudaStream_t>(stream), nullptr,
                                 nullptr, nullptr, nullptr, nullptr, 0, 0));
}

ditango_status ditango_plan_from_mass(const ditango_geom *g, float *mass_partials,
                                     size_t mass_bytes, const uint8_t *cache_valid,
                                     int32_t band_k, double budget, int8_t *plan,
                                     int32_t *fresh_list, int32_t *counts, float *score_out,
                                     ditango_stream stream) {
  NvtxRange nvtx_range("ditango_plan_from_mass");
  DevGeom dg;
  ditango_status st = make_geom(g, &dg);
  if (st != DITANGO_OK) return st;
  if (!plan || !fresh_list || !counts || !mass_partials) return DITANGO_ERR_INVALID;
  if (band_k < 0 || !(budget >= 0.0 && budget <= 1.0)) return DITANGO_ERR_INVALID;
  if (mass_bytes < plan_workspace_bytes(dg)) return DITANGO_ERR_INVALID;
  const int target = plan_target(&dg, band_k, budget);
  return cuda_status(launch_plan(dg, nullptr, cache_valid, band_k, target, 0,
                                 reinterpret_cast<signed char *>(plan), fresh_list, counts,
                                 score_out, mass_partials,
                                 static_cast<cudaStream_t>(stream), nullptr, nullptr, nullptr,
                                 nullptr, nullptr, 0, 1));
}

ditango_status ditango_plan_error(const ditango_geom *g, const float *cache_lse,
                                  const uint8_t *cache_valid, int32_t band_k, double budget,
                                  int32_t anchor, int32_t refresh_w,
                                  const ditango_error_state *es, int8_t *plan,
                                  int32_t *fresh_list, int32_t *counts, float *score_out,
                                  void *workspace, size_t workspace_bytes,
                                  ditango_stream stream) {
  NvtxRange nvtx_range("ditango_plan_error");
  DevGeom dg;
  ditango_status st = make_geom(g, &dg);
  if (st != DITANGO_OK) return st;
  if (!plan || !fresh_list || !counts || !es) return DITANGO_ERR_INVALID;
  if (!es->w || !es->age || !es->delta || !es->local_ok) return DITANGO_ERR_INVALID;
  if (!anchor) {
    if (!es->drift_rows || band_k < 0 || !(budget >= 0.0 && budget <= 1.0))
      return DITANGO_ERR_INVALID;
    if (refresh_w && !cache_lse) return DITANGO_ERR_INVALID;
    if (!workspace || workspace_bytes < plan_workspace_bytes(dg)) return DITANGO_ERR_INVALID;
  }
  const int target = plan_target(&dg, band_k, budget);
  return cuda_status(launch_plan(dg, cache_lse, cache_valid, band_k, target, anchor ? 1 : 0,
                                 reinterpret_cast<signed char *>(plan), fresh_list, counts,
                                 score_out, workspace, static_cast<cudaStream_t>(stream),
                                 es->drift_rows, es->w, es->age, es->delta, es->local_ok,
                                 refresh_w ? 1 : 0, 0));
}

ditango_status ditango_attn_partial(const ditango_geom *g, const uint16_t *Q, const uint16_t *K,
                                    const uint16_t *V, const int32_t *fresh_list,
                                    const int32_t *counts, float scale, void *out_O,
                                    float *out_lse, int32_t out_by_slot, int32_t state_bf16,
                                    uint8_t *out_valid, float *drift_rows, int32_t *dev_status,
                                    int32_t *work_counter, ditango_stream stream) {
  NvtxRange nvtx_range("ditango_attn_partial");
  DevGeom dg;
  ditango_status st = make_geom(g, &dg);
  if (st != DITANGO_OK) return st;
  if (!Q || !K || !V || !fresh_list || !counts || !out_O || !out_lse) return DITANGO_ERR_INVALID;
  if (drift_rows && !out_by_slot) return DITANGO_ERR_INVALID;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(out_O))
    return DITANGO_ERR_INVALID;
  if (work_counter && (reinterpret_cast<uintptr_t>(work_counter) & 7u)) return DITANGO_ERR_INVALID;
  // the stride of a dimension of size 1 is never used (frameworks report 0
  // or anything for it): give it the packed value
  int64_t qs[3], ks[3], vs[3];
  for (int k = 0; k < 3; ++k) {
    qs[k] = g->q_strides[k];
    ks[k] = g->k_strides[k];
    vs[k] = g->v_strides[k];
  }
  for (int64_t *s : {qs, ks, vs}) {
    if (dg.N == 1) s[2] = dg.d;
    if (dg.H == 1) s[1] = s[2] * dg.N;
    if (dg.B == 1) s[0] = s[1] * dg.H;
  }
  if (!strides_ok(qs) || !strides_ok(ks) || !strides_ok(vs)) return DITANGO_ERR_INVALID;
  if (!(scale >= 0.f) || !std::isfinite(scale)) return DITANGO_ERR_INVALID;
  if (scale == 0.f) scale = 1.f / std::sqrt((float)dg.d);
  CUtensorMap tq, tk, tv;
  // Q in 128-row tiles, K and V in the kernel's key tiles (96 keys at d = 96, else 128)
  const unsigned bn = (unsigned)attn_key_tile(dg.d);
  if (!make_qkv_map(&tq, Q, dg, qs, 128) || !make_qkv_map(&tk, K, dg, ks, bn) ||
      !make_qkv_map(&tv, V, dg, vs, bn))
    return DITANGO_ERR_CUDA;
  return cuda_status(launch_attn_partial(dg, tq, tk, tv, fresh_list, counts, scale, out_O, out_lse,
                                         out_by_slot ? 1 : 0, state_bf16 ? 1 : 0, out_valid,
                                         drift_rows, dev_status, g_wait_limit_ns.load(),
                                         num_sms_current(), work_counter,
                                         static_cast<cudaStream_t>(stream)));
}

ditango_status ditango_merge(const ditango_geom *g, const int8_t *plan, const void *part_O,
                             const float *part_lse, void *cache_O, float *cache_lse,
                             uint8_t *cache_valid, int32_t writeback, int32_t state_bf16,
                             void *out, int32_t out_is_fp32, const int64_t *out_strides,
                             float *out_lse, float *mass_partials, ditango_stream stream) {
  NvtxRange nvtx_range("ditango_merge");
  DevGeom dg;
  ditango_status st = make_geom(g, &dg);
  if (st != DITANGO_OK) return st;
  if (!plan || !out) return DITANGO_ERR_INVALID;
  if ((part_O == nullptr) != (part_lse == nullptr)) return DITANGO_ERR_INVALID;
  if ((cache_O == nullptr) != (cache_lse == nullptr)) return DITANGO_ERR_INVALID;
  if (part_O == nullptr && cache_O == nullptr) return DITANGO_ERR_INVALID;
  if (writeback && part_O && !cache_O) return DITANGO_ERR_INVALID;
  // the merge moves state rows in 16-byte groups
  if ((part_O && !aligned16(part_O)) || (cache_O && !aligned16(cache_O))) return DITANGO_ERR_INVALID;
  long long osb = (long long)dg.H * dg.N * dg.d, osh = (long long)dg.N * dg.d, osn = dg.d;
  if (out_strides) {
    osb = out_strides[0];
    osh = out_strides[1];
    osn = out_strides[2];
    if (osb <= 0 || osh <= 0 || osn <= 0) return DITANGO_ERR_INVALID;
  }
  const int esz = out_is_fp32 ? 4 : 2;
  if ((osb * esz) % 16 || (osh * esz) % 16 || (osn * esz) % 16 ||
      (reinterpret_cast<uintptr_t>(out) % (out_is_fp32 ? 16 : 8)))
    return DITANGO_ERR_INVALID;
  return cuda_status(launch_merge(dg, reinterpret_cast<const signed char *>(plan), part_O,
                                  part_lse, cache_O, cache_lse, cache_valid,
                                  (writeback && part_O) ? 1 : 0, state_bf16 ? 1 : 0, out,
                                  out_is_fp32 ? 1 : 0, osb, osh, osn, out_lse, mass_partials,
                                  static_cast<cudaStream_t>(stream)));
}

ditango_status ditango_cache_update(const ditango_geom *g, const int8_t *plan,
                                    const void *part_O, const float *part_lse, void *cache_O,
                                    float *cache_lse, uint8_t *cache_valid, int32_t state_bf16,
                                    ditango_stream stream) {
  NvtxRange nvtx_range("ditango_cache_update");
  DevGeom dg;
  ditango_status st = make_geom(g, &dg);
  if (st != DITANGO_OK) return st;
  if (!plan || !part_O || !part_lse || !cache_O || !cache_lse) return DITANGO_ERR_INVALID;
  return cuda_status(launch_cache_update(dg, reinterpret_cast<const signed char *>(plan), part_O,
                                         part_lse, cache_O, cache_lse, cache_valid,
                                         state_bf16 ? 1 : 0, num_sms_current(),
                                         static_cast<cudaStream_t>(stream)));
}

ditango_status ditango_cache_compose(const ditango_geom *fine, const ditango_geom *coarse,
                                     const void *fine_O, const float *fine_lse,
                                     const uint8_t *fine_valid, void *coarse_O,
                                     float *coarse_lse, uint8_t *coarse_valid,
                                     int32_t state_bf16, ditango_stream stream) {
  NvtxRange nvtx_range("ditango_cache_compose");
  DevGeom gf, gc;
  ditango_status st = make_geom(fine, &gf);
  if (st != DITANGO_OK) return st;
  st = make_geom(coarse, &gc);
  if (st != DITANGO_OK) return st;
  // same attention call, only the KV grouping differs
  if (gf.B != gc.B || gf.H != gc.H || gf.N != gc.N || gf.d != gc.d || gf.P != gc.P)
    return DITANGO_ERR_INVALID;
  for (int p = 0; p <= gf.P; ++p)
    if (gf.part_off[p] != gc.part_off[p]) return DITANGO_ERR_INVALID;
  for (int i = 0; i < gf.P; ++i)
    if (gf.pair_mask[i] != gc.pair_mask[i]) return DITANGO_ERR_INVALID;
  // every coarse group boundary is a fine group boundary
  for (int C = 0, c = 0; C <= gc.G; ++C) {
    while (c <= gf.G && gf.group_off[c] < gc.group_off[C]) ++c;
    if (c > gf.G || gf.group_off[c] != gc.group_off[C]) return DITANGO_ERR_INVALID;
  }
  if (!fine_O || !fine_lse || !coarse_O || !coarse_lse) return DITANGO_ERR_INVALID;
  const size_t align = state_bf16 ? 8 : 16;
  if (reinterpret_cast<uintptr_t>(fine_O) % align || reinterpret_cast<uintptr_t>(coarse_O) % align)
    return DITANGO_ERR_INVALID;
  // the two state buffers must not overlap
  const size_t rows = (size_t)gf.BH * gf.Lmax;
  const size_t es = state_bf16 ? 2 : 4;
  const char *f0 = static_cast<const char *>(fine_O), *f1 = f0 + (size_t)gf.n_active * rows * gf.d * es;
  const char *c0 = static_cast<const char *>(coarse_O), *c1 = c0 + (size_t)gc.n_active * rows * gc.d * es;
  if (f0 < c1 && c0 < f1) return DITANGO_ERR_INVALID;
  const float *fl0 = fine_lse, *fl1 = fine_lse + (size_t)gf.n_active * rows;
  const float *cl0 = coarse_lse, *cl1 = coarse_lse + (size_t)gc.n_active * rows;
  if (fl0 < cl1 && cl0 < fl1) return DITANGO_ERR_INVALID;
  return cuda_status(launch_cache_compose(gf, gc, fine_O, fine_lse, fine_valid, coarse_O,
                                          coarse_lse, coarse_valid, state_bf16 ? 1 : 0,
                                          static_cast<cudaStream_t>(stream)));
}

void ditango_set_wait_limit_ns(int64_t ns) { g_wait_limit_ns.store(ns > 0 ? ns : 1); }

int32_t ditango_checked_build(void) {
#ifdef DITANGO_CHECK
  return 1;
#else
  return 0;
#endif
}

ditango_status ditango_check_status(int32_t *status_out, int32_t reset) {
  if (!status_out) return DITANGO_ERR_INVALID;
  int a = 0, m = 0;
  cudaError_t e = attn_check_status(&a, reset != 0);
  if (e == cudaSuccess) e = merge_check_status(&m, reset != 0);
  if (e != cudaSuccess) return cuda_status(e);
  *status_out = a != 0 ? a : m;
  return DITANGO_OK;
}

ditango_status ditango_selftest_bounded_wait(int64_t limit_ns, int32_t *dev_status,
                                             ditango_stream stream) {
  if (!dev_status || limit_ns <= 0) return DITANGO_ERR_INVALID;
  return cuda_status(
      launch_bounded_wait_selftest(limit_ns, dev_status, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Allocation-free plan.
//
// Some callers cannot allocate device memory at all: code that runs inside a
// memory arena owned by someone else, a serving process whose allocator is
// frozen after start-up, or a host that must never call cudaMalloc between
// denoising steps.  They still pass their own inputs and outputs, but the
// plan's scratch (the mass block sums and their means) lives here, in a fixed device
// array of this library of kNoAllocPlanScratchBytes.  Every GPU that loads
// the library holds that array until the process exits (or until its context
// is destroyed).
//
// The array's host-side name is not a device address: its address is asked
// of the runtime with the device current, and cached per device together
// with the unique ID of the context it belongs to.  A new context on the
// device (after cudaDeviceReset, say) has a new ID, and the address is then
// looked up again instead of reusing one that points into freed memory.
namespace {
constexpr size_t kNoAllocPlanScratchBytes = size_t(4) << 20;  // 4 MiB
constexpr int kNoAllocMaxDevices = 64;

struct NoAllocScratch {
  unsigned long long ctx_id;  // context the address belongs to
  void *ptr;                  // null: not looked up in that context yet
};
std::mutex g_noalloc_mu;
NoAllocScratch g_noalloc_scratch[kNoAllocMaxDevices] = {};

typedef CUresult (*CtxGetCurrentFn)(CUcontext *);
typedef CUresult (*CtxGetIdFn)(CUcontext, unsigned long long *);

// Unique ID (for the life of the process) of the calling thread's current
// context; false when no context is current or the driver has no such call.
bool current_context_id(unsigned long long *id) {
  static CtxGetCurrentFn get_current = nullptr;
  static CtxGetIdFn get_id = nullptr;
  static std::once_flag once;
  std::call_once(once, []() {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_current = reinterpret_cast<CtxGetCurrentFn>(p);
    p = nullptr;
    if (cudaGetDriverEntryPoint("cuCtxGetId", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<CtxGetIdFn>(p);
  });
  CUcontext ctx = nullptr;
  if (!get_current || !get_id || get_current(&ctx) != CUDA_SUCCESS || ctx == nullptr) return false;
  return get_id(ctx, id) == CUDA_SUCCESS;
}
}  // namespace

static __device__ __align__(256) unsigned char g_plan_scratch[kNoAllocPlanScratchBytes];

extern "C" ditango_status ditango_plan_noalloc(const ditango_geom *g, const float *cache_lse,
                                               const uint8_t *cache_valid, int32_t band_k,
                                               double budget, int32_t anchor, int8_t *plan,
                                               int32_t *fresh_list, int32_t *counts,
                                               float *score_out, ditango_stream stream) {
  NvtxRange nvtx_range("ditango_plan_noalloc");
  DevGeom dg;
  ditango_status st = make_geom(g, &dg);
  if (st != DITANGO_OK) return st;
  if (!plan || !fresh_list || !counts) return DITANGO_ERR_INVALID;
  if (!anchor) {
    if (!cache_lse || band_k < 0 || !(budget >= 0.0 && budget <= 1.0)) return DITANGO_ERR_INVALID;
    if (plan_workspace_bytes(dg) > kNoAllocPlanScratchBytes) return DITANGO_ERR_UNSUPPORTED;
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cuda_status(cudaErrorInvalidDevice);
  if (dev < 0 || dev >= kNoAllocMaxDevices) return DITANGO_ERR_UNSUPPORTED;
  void *scratch = nullptr;
  {
    // with this device current: the cached address if it belongs to the
    // current context, else ask the runtime for it (the first ask in a
    // context also makes the primary context current on this thread)
    std::lock_guard<std::mutex> lock(g_noalloc_mu);
    NoAllocScratch &e = g_noalloc_scratch[dev];
    unsigned long long id = 0;
    bool have_id = current_context_id(&id);
    if (have_id && e.ptr != nullptr && e.ctx_id == id) {
      scratch = e.ptr;
    } else {
      void *p = nullptr;
      cudaError_t err = cudaGetSymbolAddress(&p, g_plan_scratch);
      if (err != cudaSuccess || p == nullptr)
        return cuda_status(err == cudaSuccess ? cudaErrorUnknown : err);
      if (!have_id) have_id = current_context_id(&id);
      e.ptr = have_id ? p : nullptr;   // without a context ID: look it up every call
      e.ctx_id = have_id ? id : 0;
      scratch = p;
    }
  }
  const int target = plan_target(&dg, band_k, budget);
  return cuda_status(launch_plan(dg, cache_lse, cache_valid, band_k, target, anchor ? 1 : 0,
                                 reinterpret_cast<signed char *>(plan), fresh_list, counts,
                                 score_out, scratch, static_cast<cudaStream_t>(stream), nullptr,
                                 nullptr, nullptr, nullptr, nullptr, 0, 0));
}

// ---------------------------------------------------------------------------
// The 4-bit history and the selected-block operators
namespace {

constexpr int kMaxRequests = 4096;                        // shared memory of the tables kernel
constexpr int kMaxTableBlocks = 0x7fffffff / DITANGO_PAGE;  // token places of a request fit 31 bits

bool dim_ok(int d) { return d == 64 || d == 96 || d == 128; }

bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na && nb && x < y + nb && y < x + na;
}

ditango_status check_kv4(const ditango_kv4 *c) {
  if (!c || !c->data || c->n_pages < 1 || c->Hkv < 1 || c->d < 1 || !aligned16(c->data))
    return DITANGO_ERR_INVALID;
  if (!dim_ok(c->d) || c->Hkv > 65535) return DITANGO_ERR_UNSUPPORTED;
  return DITANGO_OK;
}

// (token, head) strides in elements; the stride of a dimension of size 1 is
// not used and gets the packed value.
bool row_strides(const int64_t *s, long long T, int H, int d, int multiple, int64_t out[2]) {
  out[0] = s ? s[0] : (int64_t)H * d;
  out[1] = s ? s[1] : d;
  if (H == 1) out[1] = d;
  if (T == 1) out[0] = (int64_t)H * (out[1] > 0 ? out[1] : d);
  for (int k = 0; k < 2; ++k)
    if (out[k] <= 0 || out[k] % multiple || out[k] >= (1LL << 40)) return false;
  return true;
}

// (b, h, n) strides in elements, likewise.
bool block_strides(const int64_t *s, int B, int H, int N, int d, int64_t out[3]) {
  out[2] = N == 1 ? d : s[2];
  out[1] = H == 1 ? out[2] * N : s[1];
  out[0] = B == 1 ? out[1] * H : s[0];
  return strides_ok(out);
}

// The forced band's indices fit 31 bits, and the lists hold what is always taken.
ditango_status check_select(int n_k, int k, int band, int sink, int own, int max_sel) {
  if (k < 0 || sink < 0 || band < -1 || own < 0 || max_sel < 1) return DITANGO_ERR_INVALID;
  const long long near = band < 0 ? 0 : (own > 0 ? own : 1) + 2LL * band;
  long long must = sink + near;
  if (must < k) must = k;
  if (must > n_k) must = n_k;
  if (max_sel < must) return DITANGO_ERR_INVALID;
  if (n_k > select_max_blocks() || band > (1 << 24) || own > 1024) return DITANGO_ERR_UNSUPPORTED;
  return DITANGO_OK;
}

ditango_status kv4_rows(bool write, const ditango_kv4 *c, int64_t T, const uint16_t *K, const uint16_t *V,
                        uint16_t *Ko, uint16_t *Vo, const int64_t *ks, const int64_t *vs,
                        const int64_t *slots, int32_t *dev_status, ditango_stream stream) {
  const ditango_status st = check_kv4(c);
  if (st != DITANGO_OK) return st;
  const void *k = write ? (const void *)K : (const void *)Ko, *v = write ? (const void *)V : (const void *)Vo;
  if (T < 0 || !ks || !vs) return DITANGO_ERR_INVALID;
  if (T == 0) return DITANGO_OK;
  if (!k || !v || !slots || !aligned16(k) || !aligned16(v)) return DITANGO_ERR_INVALID;
  if (T > ((1LL << 27) - 1) / c->Hkv) return DITANGO_ERR_UNSUPPORTED;   // the kernels' 32-bit row numbers
  int64_t kst[2], vst[2];
  if (!row_strides(ks, T, c->Hkv, c->d, 8, kst) || !row_strides(vs, T, c->Hkv, c->d, 8, vst))
    return DITANGO_ERR_INVALID;
  return cuda_status(launch_kv4_rows(write, T, c->Hkv, c->d, c->n_pages, K, V, Ko, Vo, kst, vst,
                                     reinterpret_cast<const long long *>(slots), c->data, dev_status,
                                     num_sms_current(), static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

ditango_status ditango_block_tables(int32_t R, int32_t max_blocks, int32_t max_tokens, int32_t n_pages,
                                    const int32_t *ctx_len, const int32_t *new_len,
                                    const int32_t *free_pages, int32_t n_free, int32_t *block_table,
                                    int32_t *kv_len, int32_t *q_off, int64_t *slot_map,
                                    int32_t *pages_used, int32_t *dev_status, ditango_stream stream) {
  NvtxRange nvtx_range("ditango_block_tables");
  if (R < 1 || max_blocks < 1 || max_tokens < 1 || n_pages < 1 || n_free < 0) return DITANGO_ERR_INVALID;
  if (!ctx_len || !new_len || (n_free > 0 && !free_pages) || !block_table || !kv_len || !q_off ||
      !slot_map || !pages_used)
    return DITANGO_ERR_INVALID;
  if (R > kMaxRequests || max_blocks > kMaxTableBlocks) return DITANGO_ERR_UNSUPPORTED;
  // the blocks read every input while others already write: no output may
  // lie on an input or on another output
  struct Span { const void *p; size_t n; };
  const size_t r4 = (size_t)R * 4;
  const Span in[3] = {{ctx_len, r4}, {new_len, r4}, {free_pages, (size_t)n_free * 4}};
  const Span out[5] = {{block_table, r4 * max_blocks}, {kv_len, r4}, {q_off, r4 + 4},
                       {slot_map, (size_t)max_tokens * 8}, {pages_used, 4}};
  for (int a = 0; a < 5; ++a) {
    for (const Span &s : in)
      if (overlap(out[a].p, out[a].n, s.p, s.n)) return DITANGO_ERR_INVALID;
    for (int b = 0; b < a; ++b)
      if (overlap(out[a].p, out[a].n, out[b].p, out[b].n)) return DITANGO_ERR_INVALID;
  }
  return cuda_status(launch_block_tables(R, max_blocks, max_tokens, n_pages, ctx_len, new_len, free_pages,
                                         n_free, block_table, kv_len, q_off,
                                         reinterpret_cast<long long *>(slot_map), pages_used, dev_status,
                                         num_sms_current(), static_cast<cudaStream_t>(stream)));
}

ditango_status ditango_kv4_write(const ditango_kv4 *c, int64_t T, const uint16_t *K, const uint16_t *V,
                                 const int64_t k_strides[2], const int64_t v_strides[2],
                                 const int64_t *slot_map, int32_t *dev_status, ditango_stream stream) {
  NvtxRange nvtx_range("ditango_kv4_write");
  return kv4_rows(true, c, T, K, V, nullptr, nullptr, k_strides, v_strides, slot_map, dev_status, stream);
}

ditango_status ditango_kv4_read(const ditango_kv4 *c, int64_t T, uint16_t *K, uint16_t *V,
                                const int64_t k_strides[2], const int64_t v_strides[2],
                                const int64_t *slot_map, int32_t *dev_status, ditango_stream stream) {
  NvtxRange nvtx_range("ditango_kv4_read");
  return kv4_rows(false, c, T, nullptr, nullptr, K, V, k_strides, v_strides, slot_map, dev_status, stream);
}

ditango_status ditango_kv4_summary(const ditango_kv4 *c, int32_t R, int32_t max_blocks,
                                   const int32_t *ctx_len, const int32_t *kv_len,
                                   const int32_t *block_table, int8_t *sum_codes, float *sum_scale,
                                   int32_t *dev_status, ditango_stream stream) {
  NvtxRange nvtx_range("ditango_kv4_summary");
  const ditango_status st = check_kv4(c);
  if (st != DITANGO_OK) return st;
  if (R < 1 || max_blocks < 1 || !ctx_len || !kv_len || !block_table || !sum_codes || !sum_scale)
    return DITANGO_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(sum_codes) & 7u) return DITANGO_ERR_INVALID;
  if (R > kMaxRequests || max_blocks > kMaxTableBlocks) return DITANGO_ERR_UNSUPPORTED;
  return cuda_status(launch_kv4_summary(R, c->Hkv, c->d, max_blocks, c->n_pages, ctx_len, kv_len,
                                        block_table, c->data, reinterpret_cast<signed char *>(sum_codes),
                                        sum_scale, dev_status, static_cast<cudaStream_t>(stream)));
}

ditango_status ditango_kv4_select(const ditango_kv4 *c, int32_t R, int32_t H, int32_t max_blocks, int32_t k,
                                  int32_t band, int32_t sink, int32_t max_sel, const uint16_t *Q,
                                  const int64_t q_strides[2], const int8_t *sum_codes, const float *sum_scale,
                                  const int32_t *block_table, const int32_t *kv_len, int8_t *q_codes,
                                  float *q_scale, int32_t *sel, int32_t *sel_count, int32_t *dev_status,
                                  ditango_stream stream) {
  NvtxRange nvtx_range("ditango_kv4_select");
  ditango_status st = check_kv4(c);
  if (st != DITANGO_OK) return st;
  if (R < 1 || H < 1 || H % c->Hkv || max_blocks < 1) return DITANGO_ERR_INVALID;
  if (!Q || !q_strides || !sum_codes || !sum_scale || !block_table || !kv_len || !q_codes || !q_scale || !sel ||
      !sel_count || !aligned16(Q))
    return DITANGO_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(q_codes) & 7u) || (reinterpret_cast<uintptr_t>(sum_codes) & 7u))
    return DITANGO_ERR_INVALID;
  st = check_select(max_blocks, k, band, sink, 0, max_sel);
  if (st != DITANGO_OK) return st;
  if (R > kMaxRequests || H > 65535) return DITANGO_ERR_UNSUPPORTED;
  int64_t qs[2];
  if (!row_strides(q_strides, R, H, c->d, 8, qs)) return DITANGO_ERR_INVALID;
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  // the queries' codes are formed by the selection itself where it takes all
  // heads of a key head at once, else by a launch of their own
  const bool fused = select_by_heads(1, H / c->Hkv, max_blocks);
  if (!fused) {
    const int64_t s3[3] = {qs[0], qs[1], c->d};
    const cudaError_t e = launch_block_summary(R, H, 1, c->d, DITANGO_PAGE, Q, s3, nullptr,
                                               reinterpret_cast<signed char *>(q_codes), q_scale, nullptr, on);
    if (e != cudaSuccess) return cuda_status(e);
  }
  return cuda_status(launch_block_select(R, H, c->Hkv, 1, max_blocks, c->d, k, band, sink, max_sel, 0,
                                         reinterpret_cast<const signed char *>(q_codes), q_scale,
                                         reinterpret_cast<const signed char *>(sum_codes), sum_scale, block_table,
                                         c->n_pages, kv_len, sel, sel_count, dev_status, fused ? Q : nullptr, qs, on));
}

size_t ditango_kv4_attn_workspace_size(int32_t d) { return dim_ok(d) ? kv4_attn_workspace_bytes(d) : 0; }

ditango_status ditango_kv4_attn(const ditango_kv4 *c, int32_t R, int32_t H, int32_t T, int32_t max_q,
                                int32_t max_blocks, const uint16_t *Q, const int64_t q_strides[2],
                                const int32_t *q_off, const int32_t *kv_len, const int32_t *block_table,
                                const int32_t *sel, const int32_t *sel_count, int32_t max_sel, float scale,
                                int32_t causal, void *out, int32_t out_is_fp32, const int64_t *out_strides,
                                float *out_lse, const int64_t *lse_strides, void *workspace,
                                size_t workspace_bytes, int32_t *dev_status, ditango_stream stream) {
  NvtxRange nvtx_range("ditango_kv4_attn");
  const ditango_status st = check_kv4(c);
  if (st != DITANGO_OK) return st;
  if (R < 1 || H < 1 || H % c->Hkv || T < 0 || max_q < (T > 0 ? 1 : 0) || max_blocks < 1) return DITANGO_ERR_INVALID;
  if (!q_strides || !q_off || !kv_len || !block_table) return DITANGO_ERR_INVALID;
  if ((sel == nullptr) != (sel_count == nullptr) || (sel && max_sel < 1)) return DITANGO_ERR_INVALID;
  if (!(scale >= 0.f) || !std::isfinite(scale)) return DITANGO_ERR_INVALID;
  if (R > kMaxRequests || max_blocks > kMaxTableBlocks || H > 65535) return DITANGO_ERR_UNSUPPORTED;
  if (T == 0) return DITANGO_OK;
  if (!Q || !out || Q == out || !workspace || !aligned16(Q) || !aligned16(workspace))
    return DITANGO_ERR_INVALID;
  if (workspace_bytes < kv4_attn_workspace_bytes(c->d)) return DITANGO_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(out) % (out_is_fp32 ? 16 : 8)) return DITANGO_ERR_INVALID;
  int64_t qs[2], os[2], ls[2] = {H, 1};
  if (!row_strides(q_strides, T, H, c->d, 8, qs) || !row_strides(out_strides, T, H, c->d, 4, os))
    return DITANGO_ERR_INVALID;
  if (lse_strides) {
    ls[0] = lse_strides[0];
    ls[1] = lse_strides[1];
    if ((T > 1 && ls[0] <= 0) || (H > 1 && ls[1] <= 0)) return DITANGO_ERR_INVALID;
  }
  if (scale == 0.f) scale = 1.f / std::sqrt((float)c->d);
  return cuda_status(launch_kv4_attn(R, H, c->Hkv, c->d, T, max_q, max_blocks, c->n_pages, Q, qs, q_off,
                                     kv_len, block_table, c->data, sel, sel_count, max_sel, scale,
                                     causal ? 1 : 0, out, out_is_fp32 ? 1 : 0, os, out_lse, ls, workspace,
                                     dev_status, g_wait_limit_ns.load(), num_sms_current(),
                                     static_cast<cudaStream_t>(stream)));
}

ditango_status ditango_block_summary(int32_t B, int32_t H, int32_t N, int32_t d, int32_t block,
                                     const uint16_t *x, const int64_t strides[3], const int32_t *len,
                                     int8_t *codes, float *scale, float *mean, ditango_stream stream) {
  NvtxRange nvtx_range("ditango_block_summary");
  if (B < 1 || H < 1 || N < 1 || d < 1 || !x || !strides || !codes || !scale || !aligned16(x))
    return DITANGO_ERR_INVALID;
  if (block != DITANGO_PAGE && block != DITANGO_QBLOCK) return DITANGO_ERR_INVALID;
  if (!dim_ok(d) || B > 65535 || H > 65535) return DITANGO_ERR_UNSUPPORTED;
  int64_t s[3];
  if (!block_strides(strides, B, H, N, d, s)) return DITANGO_ERR_INVALID;
  return cuda_status(launch_block_summary(B, H, N, d, block, x, s, len, reinterpret_cast<signed char *>(codes),
                                          scale, mean, static_cast<cudaStream_t>(stream)));
}

ditango_status ditango_block_summaries(int32_t B, int32_t H, int32_t Hkv, int32_t Nq, int32_t Nk, int32_t d,
                                       const uint16_t *Q, const int64_t q_strides[3], const uint16_t *K,
                                       const int64_t k_strides[3], const int32_t *k_len, int8_t *q_codes,
                                       float *q_scale, int8_t *k_codes, float *k_scale, float *k_mean,
                                       ditango_stream stream) {
  NvtxRange nvtx_range("ditango_block_summaries");
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv || Nq < 1 || Nk < 1 || d < 1) return DITANGO_ERR_INVALID;
  if (!Q || !K || !q_strides || !k_strides || !q_codes || !q_scale || !k_codes || !k_scale ||
      !aligned16(Q) || !aligned16(K))
    return DITANGO_ERR_INVALID;
  if (!dim_ok(d) || B > 65535 || (long long)H + Hkv > 65535) return DITANGO_ERR_UNSUPPORTED;
  int64_t qs[3], ks[3];
  if (!block_strides(q_strides, B, H, Nq, d, qs) || !block_strides(k_strides, B, Hkv, Nk, d, ks))
    return DITANGO_ERR_INVALID;
  return cuda_status(launch_block_summaries(B, H, Hkv, Nq, Nk, d, Q, qs, K, ks, k_len,
                                            reinterpret_cast<signed char *>(q_codes), q_scale,
                                            reinterpret_cast<signed char *>(k_codes), k_scale, k_mean,
                                            static_cast<cudaStream_t>(stream)));
}

ditango_status ditango_block_select(int32_t B, int32_t H, int32_t Hkv, int32_t n_q, int32_t n_k, int32_t d,
                                    int32_t k, int32_t band, int32_t sink, int32_t own_blocks,
                                    int32_t max_sel, const int8_t *q_codes, const float *q_scale,
                                    const int8_t *k_codes, const float *k_scale, const int32_t *block_table,
                                    int32_t n_pages, const int32_t *k_len, int32_t *sel,
                                    int32_t *sel_count, int32_t *dev_status, ditango_stream stream) {
  NvtxRange nvtx_range("ditango_block_select");
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv || n_q < 1 || n_k < 1 || d < 1) return DITANGO_ERR_INVALID;
  if (!q_codes || !q_scale || !k_codes || !k_scale || !sel || !sel_count) return DITANGO_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(q_codes) & 7u) || (reinterpret_cast<uintptr_t>(k_codes) & 7u))
    return DITANGO_ERR_INVALID;
  if (block_table && n_pages < 1) return DITANGO_ERR_INVALID;
  const ditango_status st = check_select(n_k, k, band, sink, own_blocks, max_sel);
  if (st != DITANGO_OK) return st;
  if (!dim_ok(d) || B > 65535 || Hkv > 65535 || (long long)n_q * own_blocks > (1 << 30))
    return DITANGO_ERR_UNSUPPORTED;
  return cuda_status(launch_block_select(B, H, Hkv, n_q, n_k, d, k, band, sink, max_sel, own_blocks,
                                         reinterpret_cast<const signed char *>(q_codes), q_scale,
                                         reinterpret_cast<const signed char *>(k_codes), k_scale, block_table,
                                         n_pages, k_len, sel, sel_count, dev_status, nullptr, nullptr,
                                         static_cast<cudaStream_t>(stream)));
}

ditango_status ditango_block_attn(int32_t B, int32_t H, int32_t Hkv, int32_t Nq, int32_t Nk, int32_t d,
                                  const uint16_t *Q, const uint16_t *K, const uint16_t *V,
                                  const int64_t q_strides[3], const int64_t k_strides[3],
                                  const int64_t v_strides[3], const int32_t *sel, const int32_t *sel_count,
                                  int32_t max_sel, const int32_t *k_len, float scale, void *out,
                                  int32_t out_is_fp32, const int64_t *out_strides, float *out_lse,
                                  int32_t *dev_status, ditango_stream stream) {
  return ditango_block_attn_strided(B, H, Hkv, Nq, Nk, d, Q, K, V, q_strides, k_strides, v_strides, sel,
                                    sel_count, max_sel, k_len, scale, out, out_is_fp32, out_strides, out_lse,
                                    nullptr, dev_status, stream);
}

ditango_status ditango_block_attn_strided(int32_t B, int32_t H, int32_t Hkv, int32_t Nq, int32_t Nk, int32_t d,
                                          const uint16_t *Q, const uint16_t *K, const uint16_t *V,
                                          const int64_t q_strides[3], const int64_t k_strides[3],
                                          const int64_t v_strides[3], const int32_t *sel,
                                          const int32_t *sel_count, int32_t max_sel, const int32_t *k_len,
                                          float scale, void *out, int32_t out_is_fp32,
                                          const int64_t *out_strides, float *out_lse,
                                          const int64_t *lse_strides, int32_t *dev_status,
                                          ditango_stream stream) {
  NvtxRange nvtx_range("ditango_block_attn");
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv || Nq < 1 || Nk < 1 || d < 1 || max_sel < 1)
    return DITANGO_ERR_INVALID;
  if (!Q || !K || !V || !q_strides || !k_strides || !v_strides || !sel || !sel_count || !out)
    return DITANGO_ERR_INVALID;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(out)) return DITANGO_ERR_INVALID;
  if (out == Q || out == K || out == V) return DITANGO_ERR_INVALID;
  if (!(scale >= 0.f) || !std::isfinite(scale)) return DITANGO_ERR_INVALID;
  if (!dim_ok(d) || B > 65535 || H > 65535) return DITANGO_ERR_UNSUPPORTED;
  DevGeom gq, gk;
  std::memset(&gq, 0, sizeof(gq));
  gq.B = B;
  gq.H = H;
  gq.N = Nq;
  gq.d = d;
  gk = gq;
  gk.H = Hkv;
  gk.N = Nk;
  int64_t qs[3], ks[3], vs[3];
  long long os[3] = {(long long)H * Nq * d, (long long)Nq * d, d};
  for (int a = 0; a < 3; ++a) {
    qs[a] = q_strides[a];
    ks[a] = k_strides[a];
    vs[a] = v_strides[a];
    if (out_strides) os[a] = out_strides[a];
  }
  auto pack = [&](auto *s, int heads, int n) {
    if (n == 1) s[2] = d;
    if (heads == 1) s[1] = s[2] * n;
    if (B == 1) s[0] = s[1] * heads;
  };
  pack(qs, H, Nq);
  pack(ks, Hkv, Nk);
  pack(vs, Hkv, Nk);
  pack(os, H, Nq);
  if (!strides_ok(qs) || !strides_ok(ks) || !strides_ok(vs)) return DITANGO_ERR_INVALID;
  const int esz = out_is_fp32 ? 4 : 2;
  for (int a = 0; a < 3; ++a)
    if (os[a] <= 0 || (os[a] * esz) % 16) return DITANGO_ERR_INVALID;
  long long ls[3] = {(long long)H * Nq, Nq, 1};
  if (lse_strides) {
    const int size[3] = {B, H, Nq};
    for (int a = 0; a < 3; ++a) {
      ls[a] = lse_strides[a];
      if (size[a] > 1 && ls[a] <= 0) return DITANGO_ERR_INVALID;
    }
  }
  if (scale == 0.f) scale = 1.f / std::sqrt((float)d);
  CUtensorMap tq, tk, tv;
  if (!make_qkv_map(&tq, Q, gq, qs, DITANGO_QBLOCK) || !make_qkv_map(&tk, K, gk, ks, DITANGO_PAGE) ||
      !make_qkv_map(&tv, V, gk, vs, DITANGO_PAGE))
    return DITANGO_ERR_CUDA;
  return cuda_status(launch_block_attn(tq, tk, tv, B, H, Hkv, Nq, Nk, d, sel, sel_count, max_sel, k_len,
                                       scale, out, out_is_fp32 ? 1 : 0, os, out_lse, ls, dev_status,
                                       g_wait_limit_ns.load(), num_sms_current(),
                                       static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
