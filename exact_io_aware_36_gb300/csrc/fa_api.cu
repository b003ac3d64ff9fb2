// fa_api.cu -- the C ABI of libfa (declared in include/fa.h): argument
// checks, workspace sizing, the per-device status word and dispatch to the
// kernels.  Every check runs before any launch; nothing here allocates
// device memory.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <functional>
#include <mutex>
#include <queue>
#include <vector>

#include "fa_host_util.h"
#include "fa_internal.h"

namespace {

__device__ unsigned int g_fa_status;   // per-device status word

constexpr int kMaxDevices = 64;

unsigned int* status_ptr() {
  static unsigned int* ptrs[kMaxDevices] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!ptrs[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_fa_status) != cudaSuccess) return nullptr;
    ptrs[dev] = static_cast<unsigned int*>(p);
  }
  return ptrs[dev];
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

// Shared size checks of fa_fwd / fa_bwd.  Fills T.
fa_status check_sizes(int B, int Hq, int Hkv, int N, int d, float scale,
                      const int32_t* cu_seqlens, long long total_tokens, fa_dtype dtype,
                      bool backward, long long* T) {
  if (B < 0 || N < 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || total_tokens < 0) return FA_ERR_SHAPE;
  if (Hq % Hkv != 0) return FA_ERR_SHAPE;
  if (dtype != FA_BF16 && dtype != FA_FP32) return FA_ERR_UNSUPPORTED;
  if (backward && dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (dtype == FA_BF16 && d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (dtype == FA_FP32 && d > 128) return FA_ERR_UNSUPPORTED;
  if (!(scale > 0.f) || !isfinite(scale)) return FA_ERR_UNSUPPORTED;
  if (B > 65535 || Hq > 65535) return FA_ERR_UNSUPPORTED;
  // 1-D grids of (blocks per sequence) x heads x sequences must fit 2^31 - 1
  if ((long long)((N + 127) / 128) * Hq * B >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  const long long dense = (long long)B * N;
  if (cu_seqlens == nullptr) {
    if (total_tokens != 0 && total_tokens != dense) return FA_ERR_SHAPE;
    *T = dense;
  } else {
    *T = total_tokens;
  }
  // token coordinates are 32-bit in the TMA descriptors and the kernels
  if (*T >= (1ll << 31) || (long long)N >= (1ll << 30)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Window argument -> band width: < 0 means none; a band that reaches back
// over the whole longest sequence (window >= N - 1) masks nothing beyond the
// causal mask, so it is run as unbanded.
int band_width(int window, int N) { return (window < 0 || window >= N - 1) ? fa::kNoWindow : window; }

fa::AttnParams base_params(int B, int Hq, int Hkv, int N, int d, float scale, int causal,
                           int window, const int32_t* cu_seqlens, long long T,
                           const float* alibi) {
  fa::AttnParams p = {};
  p.window = band_width(window, N);
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.N = N;
  p.d = d;
  p.T = T;
  p.group = Hq / Hkv;
  p.causal = causal ? 1 : 0;
  p.scale = scale;
  p.scale_log2 = scale * fa::kLog2e;
  p.cu_seqlens = cu_seqlens;
  p.alibi = alibi;
  return p;
}

}  // namespace

extern "C" {

int fa_version(void) { return 10000; }

const char* fa_status_string(fa_status s) {
  switch (s) {
    case FA_OK: return "ok";
    case FA_ERR_NULL: return "a required pointer is NULL";
    case FA_ERR_SHAPE: return "invalid or inconsistent sizes";
    case FA_ERR_UNSUPPORTED: return "unsupported configuration (head dim, dtype or scale)";
    case FA_ERR_ALIGN: return "a bf16 tensor is not 16-byte aligned";
    case FA_ERR_WORKSPACE: return "workspace missing or too small";
    case FA_ERR_CUDA: return "CUDA runtime or launch error";
    case FA_ERR_DEVICE_TIMEOUT: return "device pipeline wait exceeded its time limit";
    case FA_ERR_CU_SEQLENS: return "cu_seqlens malformed or a sequence longer than N";
    case FA_ERR_PAGE: return "a page outside the pool, or pages whose copies clash";
    case FA_ERR_POSITION: return "a position outside the table of angles";
  }
  return "unknown status";
}

fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                 int Hkv, int N, int d, float scale, int causal, int window,
                 const int32_t* cu_seqlens, long long total_tokens, const float* alibi_slopes,
                 fa_dtype dtype, fa_dtype o_dtype, void* stream) {
  long long T = 0;
  fa_status st = check_sizes(B, Hq, Hkv, N, d, scale, cu_seqlens, total_tokens, dtype, false, &T);
  if (st != FA_OK) return st;
  if (window >= 0 && !causal) return FA_ERR_UNSUPPORTED;
  if (o_dtype != FA_FP32 && !(o_dtype == FA_BF16 && dtype == FA_BF16)) return FA_ERR_UNSUPPORTED;
  if (!q || !k || !v || !o || !lse) return FA_ERR_NULL;
  if (dtype == FA_BF16 && (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)))
    return FA_ERR_ALIGN;
  if (dtype == FA_FP32 && ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) |
                            reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(o)) & 3u))
    return FA_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_ALIGN;
  if (T == 0 || B == 0 || N == 0) return FA_OK;
  fa::AttnParams p = base_params(B, Hq, Hkv, N, d, scale, causal, window, cu_seqlens, T,
                                 alibi_slopes);
  p.q = q;
  p.k = k;
  p.v = v;
  p.o = o;
  p.lse = lse;
  p.o_f32 = o_dtype == FA_FP32;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  const int e = dtype == FA_FP32 ? fa::launch_fwd_fp32(p, stream) : fa::launch_fwd_bf16(p, stream);
  return e == 0 ? FA_OK : FA_ERR_CUDA;
}

size_t fa_bwd_workspace_size(int B, int Hq, int N, int d, long long total_tokens) {
  if (B < 0 || Hq <= 0 || N < 0 || d <= 0 || total_tokens < 0) return 0;
  const long long T = total_tokens > 0 ? total_tokens : (long long)B * N;
  return round256((size_t)Hq * T * sizeof(float)) + round256((size_t)Hq * T * d * sizeof(float)) + 256;
}

// Largest number of parts the dK/dV work of a GQA group may be split into:
// 2 when the group splits evenly, else 1 (no split).  (Four parts were
// measured no faster than two on the GQA workload, B=2 Hq=32 Hkv=4 N=8192,
// while their sum costs twice as much.)
static int gqa_split_max(int Hq, int Hkv) {
  const int group = Hkv > 0 ? Hq / Hkv : 0;
  return (group >= 2 && group % 2 == 0) ? 2 : 1;
}

// How many parts to split each dense batch's dK/dV work items into (1 or
// 2).  The kernel's SMs take items largest first as they finish; with few,
// large items (a long causal sequence and few kv heads) the last ones leave
// SMs idle.  For each allowed split this simulates that list schedule over
// the items' step counts (a step is 64 queries of one head against the key
// tile), estimates the time as its longest SM in steps, plus the stage that
// adds the parts up (reads 2 x split fp32 tensors [T, Hkv, d]), and keeps
// the fastest.  Results are cached per shape.  Packed batches, whose
// lengths the host does not see, are not split.
static int dkdv_split(int B, int Hq, int Hkv, int N, int d, int causal, int window) {
  const int smax = gqa_split_max(Hq, Hkv);
  if (smax == 1) return 1;
  int nsm = 0;
  if (fa::sm_count(&nsm) != 0 || nsm <= 0) return 1;
  struct Entry { int B, Hq, Hkv, N, d, causal, window, nsm, split; };
  static Entry cache[16];
  static int ncache = 0;
  static std::mutex mu;
  {
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < ncache; ++i) {
      const Entry& e = cache[i];
      if (e.B == B && e.Hq == Hq && e.Hkv == Hkv && e.N == N && e.d == d && e.causal == causal &&
          e.window == window && e.nsm == nsm)
        return e.split;
    }
  }
  const int group = Hq / Hkv;
  const long long nkt = (N + 127) / 128, nqt_all = (N + 63) / 64;
  std::vector<long long> per_kt((size_t)nkt);
  for (long long kt = 0; kt < nkt; ++kt) {
    const long long qt0 = causal ? 2 * kt : 0;
    long long qt_end = nqt_all;
    if (causal && window != fa::kNoWindow)
      qt_end = std::min(nqt_all, (kt * 128 + 127 + window) / 64 + 1);
    per_kt[(size_t)kt] = std::max(0ll, qt_end - qt0);
  }
  std::sort(per_kt.begin(), per_kt.end(), std::greater<long long>());
  const double step_s = 1.6e-6 * d / 128.0;         // measured per-step time of one SM
  const double bytes_per_s = 6.0e12;                // HBM rate of the adding stage
  int best = 1;
  double best_t = 0.0;
  for (int split = 1; split <= smax; split *= 2) {
    std::priority_queue<long long, std::vector<long long>, std::greater<long long>> load;
    for (int i = 0; i < nsm; ++i) load.push(0);
    const long long per_item = (long long)B * Hkv * split;
    for (long long steps : per_kt)
      for (long long i = 0; i < per_item; ++i) {
        const long long x = load.top();
        load.pop();
        load.push(x + steps * group / split);
      }
    long long makespan = 0;
    while (!load.empty()) { makespan = load.top(); load.pop(); }
    double t = makespan * step_s;
    if (split > 1) t += (double)split * 2 * B * N * Hkv * d * 4 / bytes_per_s;
    if (split == 1 || t < best_t) {
      best = split;
      best_t = t;
    }
  }
  std::lock_guard<std::mutex> lock(mu);
  cache[ncache < 16 ? ncache++ : (B + N) % 16] = Entry{B, Hq, Hkv, N, d, causal, window, nsm, best};
  return best;
}

size_t fa_bwd_workspace_size_gqa(int B, int Hq, int Hkv, int N, int d, long long total_tokens) {
  const size_t base = fa_bwd_workspace_size(B, Hq, N, d, total_tokens);
  if (base == 0 || Hkv <= 0 || Hq % Hkv != 0) return 0;
  const int split = gqa_split_max(Hq, Hkv);
  if (split == 1) return base;
  const long long T = total_tokens > 0 ? total_tokens : (long long)B * N;
  return base + round256((size_t)split * 2 * T * Hkv * d * sizeof(float));
}

}  // extern "C"

namespace fa {

fa_status bwd_check_args(const void* q, const void* k, const void* v, const void* o,
                         const void* dO, const float* lse, const void* dq, const void* dk,
                         const void* dv, int B, int Hq, int Hkv, int N, int d, float scale,
                         int causal, int window, const int32_t* cu_seqlens,
                         long long total_tokens, fa_dtype dtype, fa_dtype o_dtype,
                         int deterministic, long long* T) {
  fa_status st = check_sizes(B, Hq, Hkv, N, d, scale, cu_seqlens, total_tokens, dtype, true, T);
  if (st != FA_OK) return st;
  if (o_dtype != FA_FP32 && o_dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (window >= 0 && !causal) return FA_ERR_UNSUPPORTED;
  if (deterministic != 0 && deterministic != 1) return FA_ERR_UNSUPPORTED;
  if (!q || !k || !v || !o || !dO || !lse || !dq || !dk || !dv) return FA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dO) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(lse))
    return FA_ERR_ALIGN;
  if (B == 0 || N == 0) *T = 0;
  return FA_OK;
}

}  // namespace fa

extern "C" {

static fa_status bwd_impl(int stage, const void* q, const void* k, const void* v, const void* o,
                          const void* dO, const float* lse, void* dq, void* dk, void* dv, int B,
                          int Hq, int Hkv, int N, int d, float scale, int causal, int window,
                          const int32_t* cu_seqlens, long long total_tokens,
                          const float* alibi_slopes, fa_dtype dtype, fa_dtype o_dtype,
                          int deterministic, void* workspace, size_t workspace_bytes,
                          void* stream) {
  if (stage < -1 || stage > 2) return FA_ERR_UNSUPPORTED;
  long long T = 0;
  fa_status st = fa::bwd_check_args(q, k, v, o, dO, lse, dq, dk, dv, B, Hq, Hkv, N, d, scale,
                                    causal, window, cu_seqlens, total_tokens, dtype, o_dtype,
                                    deterministic, &T);
  if (st != FA_OK) return st;
  if (T == 0) return FA_OK;
  const size_t need = fa_bwd_workspace_size(B, Hq, N, d, T);
  if (!workspace || workspace_bytes < need) return FA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_ALIGN;
  fa::AttnParams p = base_params(B, Hq, Hkv, N, d, scale, causal, window, cu_seqlens, T,
                                 alibi_slopes);
  p.deterministic = deterministic;
  p.q = q;
  p.k = k;
  p.v = v;
  p.o = const_cast<void*>(o);
  p.lse = const_cast<float*>(lse);
  p.o_f32 = o_dtype == FA_FP32;
  p.dO = dO;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.D = static_cast<float*>(workspace);
  p.dq_acc = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                      round256((size_t)Hq * T * sizeof(float)));
  p.work_ctr = reinterpret_cast<int*>(static_cast<char*>(workspace) + round256((size_t)Hq * T * sizeof(float)) +
                                      round256((size_t)Hq * T * d * sizeof(float)));
  // A workspace of fa_bwd_workspace_size_gqa bytes also holds per-part dK /
  // dV sums, which lets the dK/dV kernel split each GQA group's work.
  p.kv_split = 1;
  if (!cu_seqlens && gqa_split_max(Hq, Hkv) > 1 &&
      workspace_bytes >= fa_bwd_workspace_size_gqa(B, Hq, Hkv, N, d, 0)) {
    p.kv_split = dkdv_split(B, Hq, Hkv, N, d, causal, p.window);
    p.dkv_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + need);
  }
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  const int e = fa::launch_bwd_bf16(p, stream, stage);
  return e == 0 ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO,
                 const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N,
                 int d, float scale, int causal, int window, const int32_t* cu_seqlens,
                 long long total_tokens, const float* alibi_slopes, fa_dtype dtype,
                 fa_dtype o_dtype, int deterministic, void* workspace, size_t workspace_bytes,
                 void* stream) {
  return bwd_impl(-1, q, k, v, o, dO, lse, dq, dk, dv, B, Hq, Hkv, N, d, scale, causal, window,
                  cu_seqlens, total_tokens, alibi_slopes, dtype, o_dtype, deterministic,
                  workspace, workspace_bytes, stream);
}

fa_status fa_bwd_stage(int stage, const void* q, const void* k, const void* v, const void* o,
                       const void* dO, const float* lse, void* dq, void* dk, void* dv, int B,
                       int Hq, int Hkv, int N, int d, float scale, int causal, int window,
                       const int32_t* cu_seqlens, long long total_tokens,
                       const float* alibi_slopes, fa_dtype dtype, fa_dtype o_dtype,
                       int deterministic, void* workspace, size_t workspace_bytes,
                       void* stream) {
  if (stage < 0 || stage > 2) return FA_ERR_UNSUPPORTED;
  return bwd_impl(stage, q, k, v, o, dO, lse, dq, dk, dv, B, Hq, Hkv, N, d, scale, causal,
                  window, cu_seqlens, total_tokens, alibi_slopes, dtype, o_dtype, deterministic,
                  workspace, workspace_bytes, stream);
}

// Decode: sizes valid and supported?  Fills the derived sizes.
static fa_status decode_sizes(int B, int Hq, int Hkv, int S_max, int q_len, int d, int* R,
                              int* chunk, int* nsplit) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || S_max < 0 || q_len <= 0 || d <= 0) return FA_ERR_SHAPE;
  if (Hq % Hkv != 0) return FA_ERR_SHAPE;
  if (B > 0 && q_len > S_max) return FA_ERR_SHAPE;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  const long long rows = (long long)(Hq / Hkv) * q_len;
  if (rows > fa::kDecodeMaxRows) return FA_ERR_UNSUPPORTED;
  if ((long long)B * S_max >= (1ll << 31) || (long long)B * q_len * Hq >= (1ll << 31))
    return FA_ERR_UNSUPPORTED;
  *R = (int)rows;
  *chunk = fa::decode_chunk(B, Hkv, S_max);
  *nsplit = S_max > 0 ? (S_max + *chunk - 1) / *chunk : 0;
  return FA_OK;
}

size_t fa_decode_workspace_size(int B, int Hq, int Hkv, int S_max, int q_len, int d) {
  int R = 0, chunk = 0, nsplit = 0;
  if (decode_sizes(B, Hq, Hkv, S_max, q_len, d, &R, &chunk, &nsplit) != FA_OK) return 0;
  const size_t units = (size_t)B * Hkv * nsplit;
  return round256(units * R * d * sizeof(float)) + round256(units * R * 3 * sizeof(float));
}

fa_status fa_decode(const void* q, const void* k_cache, const void* v_cache,
                    const int32_t* cache_seqlens, void* o, float* lse, int B, int Hq, int Hkv,
                    int S_max, int q_len, int d, float scale, int window,
                    const float* alibi_slopes, fa_dtype o_dtype, void* workspace,
                    size_t workspace_bytes, void* stream) {
  int R = 0, chunk = 0, nsplit = 0;
  fa_status st = decode_sizes(B, Hq, Hkv, S_max, q_len, d, &R, &chunk, &nsplit);
  if (st != FA_OK) return st;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_UNSUPPORTED;
  if (o_dtype != FA_FP32 && o_dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (!q || !k_cache || !v_cache || !o || !lse) return FA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o))
    return FA_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_ALIGN;
  if (B == 0) return FA_OK;
  const size_t need = fa_decode_workspace_size(B, Hq, Hkv, S_max, q_len, d);
  if (!workspace || workspace_bytes < need) return FA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_ALIGN;
  fa::DecodeParams p = {};
  p.q = q;
  p.k = k_cache;
  p.v = v_cache;
  p.o = o;
  p.lse = lse;
  p.seqlens = cache_seqlens;
  p.alibi = alibi_slopes;
  const size_t units = (size_t)B * Hkv * nsplit;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                       round256(units * R * d * sizeof(float)));
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.S_max = S_max;
  p.q_len = q_len;
  p.d = d;
  p.group = Hq / Hkv;
  p.R = R;
  p.chunk = chunk;
  p.nsplit = nsplit;
  p.window = band_width(window, S_max);
  p.o_f32 = o_dtype == FA_FP32;
  p.scale = scale;
  p.scale_log2 = scale * fa::kLog2e;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  const int e = fa::launch_decode_bf16(p, stream);
  return e == 0 ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_fp8_layout_get(int B, int Hq, int Hkv, int N, int d, long long total_tokens,
                            fa_fp8_layout* out) {
  if (!out) return FA_ERR_NULL;
  if (B < 0 || N < 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || total_tokens < 0) return FA_ERR_SHAPE;
  if (Hq % Hkv != 0) return FA_ERR_SHAPE;
  if (d != 128) return FA_ERR_UNSUPPORTED;
  const long long T = total_tokens > 0 ? total_tokens : (long long)B * N;
  const long long nblk = ((long long)N + 127) / 128;
  const long long vt = (long long)B * nblk * 128;      // keys per transposed V row
  // token and key coordinates are 32-bit in the TMA descriptors
  if (T >= (1ll << 31) || vt >= (1ll << 31) || (long long)N >= (1ll << 30)) return FA_ERR_UNSUPPORTED;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = round256(off + bytes);
    return at;
  };
  out->q8 = take((size_t)T * Hq * 128);
  out->k8 = take((size_t)T * Hkv * 128);
  out->v8t = take((size_t)Hkv * 128 * vt);
  out->q_scale = take(sizeof(float) * Hq * B * nblk);
  out->k_scale = take(sizeof(float) * Hkv * B * nblk);
  out->v_scale = take(sizeof(float) * Hkv * B * nblk);
  out->v_scale_max = take(sizeof(float) * Hkv);
  out->total = off;
  out->nblk = (int)nblk;
  return FA_OK;
}

fa_status fa_fp8_quantize(const void* q, const void* k, const void* v, const float* signs,
                          int B, int Hq, int Hkv, int N, int d, const int32_t* cu_seqlens,
                          long long total_tokens, void* fp8_buf, size_t fp8_bytes, void* stream) {
  long long T = 0;
  fa_status st = check_sizes(B, Hq, Hkv, N, d, 1.0f, cu_seqlens, total_tokens, FA_BF16, false, &T);
  if (st != FA_OK) return st;
  if (d != 128) return FA_ERR_UNSUPPORTED;
  if (!q || !k || !v || !signs) return FA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v)) return FA_ERR_ALIGN;
  if (T == 0 || B == 0 || N == 0) return FA_OK;
  fa_fp8_layout lay;
  st = fa_fp8_layout_get(B, Hq, Hkv, N, d, cu_seqlens ? T : 0, &lay);
  if (st != FA_OK) return st;
  if (!fp8_buf || fp8_bytes < lay.total) return FA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(fp8_buf) & 255u) != 0) return FA_ERR_ALIGN;
  char* base = static_cast<char*>(fp8_buf);
  fa::QuantParams p = {};
  p.q = q;
  p.k = k;
  p.v = v;
  p.signs = signs;
  p.cu_seqlens = cu_seqlens;
  p.q8 = reinterpret_cast<uint8_t*>(base + lay.q8);
  p.k8 = reinterpret_cast<uint8_t*>(base + lay.k8);
  p.v8t = reinterpret_cast<uint8_t*>(base + lay.v8t);
  p.q_scale = reinterpret_cast<float*>(base + lay.q_scale);
  p.k_scale = reinterpret_cast<float*>(base + lay.k_scale);
  p.v_scale = reinterpret_cast<float*>(base + lay.v_scale);
  p.v_smax = reinterpret_cast<float*>(base + lay.v_scale_max);
  p.T = T;
  p.vt_stride = (long long)B * lay.nblk * 128;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.N = N;
  p.nblk = lay.nblk;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  return fa::launch_fp8_quantize(p, stream) == 0 ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_fwd_fp8(const void* fp8_buf, size_t fp8_bytes, void* o, float* lse, int B, int Hq,
                     int Hkv, int N, int d, float scale, int causal, int window,
                     const int32_t* cu_seqlens, long long total_tokens,
                     const float* alibi_slopes, fa_dtype o_dtype, void* stream) {
  long long T = 0;
  fa_status st = check_sizes(B, Hq, Hkv, N, d, scale, cu_seqlens, total_tokens, FA_BF16, false, &T);
  if (st != FA_OK) return st;
  if (d != 128) return FA_ERR_UNSUPPORTED;
  if (window >= 0 && !causal) return FA_ERR_UNSUPPORTED;
  if (o_dtype != FA_FP32 && o_dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (!fp8_buf || !o || !lse) return FA_ERR_NULL;
  if (!aligned16(o) || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(fp8_buf) & 255u) != 0) return FA_ERR_ALIGN;
  if (T == 0 || B == 0 || N == 0) return FA_OK;
  fa_fp8_layout lay;
  st = fa_fp8_layout_get(B, Hq, Hkv, N, d, cu_seqlens ? T : 0, &lay);
  if (st != FA_OK) return st;
  if (fp8_bytes < lay.total) return FA_ERR_WORKSPACE;
  const char* base = static_cast<const char*>(fp8_buf);
  fa::AttnParams p = base_params(B, Hq, Hkv, N, d, scale, causal, window, cu_seqlens, T,
                                 alibi_slopes);
  p.q = base + lay.q8;
  p.k = base + lay.k8;
  p.v = base + lay.v8t;
  p.q_scale = reinterpret_cast<const float*>(base + lay.q_scale);
  p.k_scale = reinterpret_cast<const float*>(base + lay.k_scale);
  p.v_scale = reinterpret_cast<const float*>(base + lay.v_scale);
  p.v_smax = reinterpret_cast<const float*>(base + lay.v_scale_max);
  p.nblk = lay.nblk;
  p.vt_stride = (long long)B * lay.nblk * 128;
  p.o = o;
  p.lse = lse;
  p.o_f32 = o_dtype == FA_FP32;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  return fa::launch_fwd_fp8(p, stream) == 0 ? FA_OK : FA_ERR_CUDA;
}

// Checks of the sizes, weights and angles of the norm and rotation calls, and
// their places in p (everything but q, k, v and the outputs).
static fa_status norm_rope_args(fa::NormRopeParams* p, const float* q_weight, const float* k_weight,
                                float eps, const float* cos, const float* sin, long long T, int Hq,
                                int Hkv, int d, int rot_dim, int max_pos, int interleaved) {
  if (T < 0 || Hq < 0 || Hkv < 0 || Hq + (long long)Hkv == 0 || d <= 0 || rot_dim < 0 || rot_dim > d || max_pos < 0)
    return FA_ERR_SHAPE;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (rot_dim % 16 != 0 || (interleaved != 0 && interleaved != 1)) return FA_ERR_UNSUPPORTED;
  if (Hq > 65535 || Hkv > 65535 || T >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return FA_ERR_UNSUPPORTED;
  if (!q_weight != !k_weight) return FA_ERR_NULL;
  if (rot_dim && (!cos || !sin)) return FA_ERR_NULL;
  if (!aligned16(q_weight) || !aligned16(k_weight)) return FA_ERR_ALIGN;
  if (rot_dim && (!aligned16(cos) || !aligned16(sin))) return FA_ERR_ALIGN;
  p->q_weight = q_weight;
  p->k_weight = k_weight;
  p->eps = eps;
  p->cos = cos;
  p->sin = sin;
  p->T = T;
  p->Hq = Hq;
  p->Hkv = Hkv;
  p->d = d;
  p->rot = rot_dim;
  p->max_pos = max_pos;
  p->interleaved = interleaved;
  return FA_OK;
}

// One [T, H, d] tensor given by its token stride: FA_OK if H heads fit the
// stride and the rows are 16-byte aligned (a tensor without elements passes).
static fa_status check_rows(const void* x, long long stride, long long T, int H, int d, int esize) {
  if (H == 0 || T == 0) return FA_OK;
  if (!x) return FA_ERR_NULL;
  if (T > 1 && stride < (long long)H * d) return FA_ERR_SHAPE;
  if (!aligned16(x) || (stride * esize) % 16 != 0) return FA_ERR_ALIGN;
  return FA_OK;
}

// Sizes of a cache in pages, and their places in p.
static fa_status page_args(fa::NormRopeParams* p, int B, int N, int page_size, int num_pages, int max_pages) {
  if (B < 0 || N < 0 || num_pages < 0 || max_pages < 0 || page_size <= 0) return FA_ERR_SHAPE;
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0) return FA_ERR_UNSUPPORTED;
  // slots and positions are 32-bit in the kernels
  if ((long long)num_pages * page_size >= (1ll << 31) || (long long)max_pages * page_size >= (1ll << 30))
    return FA_ERR_UNSUPPORTED;
  p->B = B;
  p->N = N;
  p->page_size = page_size;
  p->page_shift = 0;
  while ((1 << p->page_shift) < page_size) ++p->page_shift;
  p->num_pages = num_pages;
  p->max_pages = max_pages;
  return FA_OK;
}

fa_status fa_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out,
                          long long q_stride, long long k_stride, const float* q_weight,
                          const float* k_weight, float eps, const float* cos, const float* sin,
                          const int32_t* positions, long long T, int Hq, int Hkv, int d,
                          int rot_dim, int max_pos, int interleaved, fa_dtype dtype, void* stream) {
  fa::NormRopeParams p = {};
  fa_status st = norm_rope_args(&p, q_weight, k_weight, eps, cos, sin, T, Hq, Hkv, d, rot_dim, max_pos, interleaved);
  if (st != FA_OK) return st;
  if (dtype != FA_BF16 && dtype != FA_FP32) return FA_ERR_UNSUPPORTED;
  if (!q_weight && rot_dim == 0) return FA_ERR_UNSUPPORTED;
  const int esize = dtype == FA_FP32 ? 4 : 2;
  if ((st = check_rows(q, q_stride, T, Hq, d, esize)) != FA_OK) return st;
  if ((st = check_rows(k, k_stride, T, Hkv, d, esize)) != FA_OK) return st;
  if ((st = check_rows(q_out, (long long)Hq * d, T, Hq, d, esize)) != FA_OK) return st;
  if ((st = check_rows(k_out, (long long)Hkv * d, T, Hkv, d, esize)) != FA_OK) return st;
  if (rot_dim && !positions) return FA_ERR_NULL;
  if (T == 0) return FA_OK;
  p.q = q;
  p.k = k;
  p.q_out = q_out;
  p.k_out = k_out;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.positions = positions;
  p.f32 = dtype == FA_FP32;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  return fa::launch_norm_rope(p, stream) == 0 ? FA_OK : FA_ERR_CUDA;
}

size_t fa_qk_norm_rope_bwd_workspace_size(int d) {
  return d > 0 ? round256((size_t)fa::kNormRopeBwdBlocks * 2 * d * sizeof(float)) : 0;
}

fa_status fa_qk_norm_rope_bwd(const void* q, const void* k, const void* dq_out,
                              const void* dk_out, long long q_stride, long long k_stride,
                              const float* q_weight, const float* k_weight, float eps,
                              const float* cos, const float* sin, const int32_t* positions,
                              void* dq, void* dk, long long dq_stride, long long dk_stride,
                              float* dq_weight, float* dk_weight, long long T, int Hq, int Hkv,
                              int d, int rot_dim, int max_pos, int interleaved, fa_dtype dtype,
                              void* workspace, size_t workspace_bytes, void* stream) {
  fa::NormRopeParams p = {};
  fa_status st = norm_rope_args(&p, q_weight, k_weight, eps, cos, sin, T, Hq, Hkv, d, rot_dim, max_pos, interleaved);
  if (st != FA_OK) return st;
  if (dtype != FA_BF16 && dtype != FA_FP32) return FA_ERR_UNSUPPORTED;
  if (!q_weight && rot_dim == 0) return FA_ERR_UNSUPPORTED;
  const int esize = dtype == FA_FP32 ? 4 : 2;
  if ((st = check_rows(q, q_stride, T, Hq, d, esize)) != FA_OK) return st;
  if ((st = check_rows(k, k_stride, T, Hkv, d, esize)) != FA_OK) return st;
  if ((st = check_rows(dq_out, (long long)Hq * d, T, Hq, d, esize)) != FA_OK) return st;
  if ((st = check_rows(dk_out, (long long)Hkv * d, T, Hkv, d, esize)) != FA_OK) return st;
  if ((st = check_rows(dq, dq_stride, T, Hq, d, esize)) != FA_OK) return st;
  if ((st = check_rows(dk, dk_stride, T, Hkv, d, esize)) != FA_OK) return st;
  if (rot_dim && !positions) return FA_ERR_NULL;
  if (q_weight) {
    if (!dq_weight || !dk_weight) return FA_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(dq_weight) | reinterpret_cast<uintptr_t>(dk_weight)) & 3u) return FA_ERR_ALIGN;
    if (!workspace || workspace_bytes < fa_qk_norm_rope_bwd_workspace_size(d)) return FA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_ALIGN;
  }
  if (T == 0) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (q_weight && (cudaMemsetAsync(dq_weight, 0, d * sizeof(float), s) != cudaSuccess ||
                     cudaMemsetAsync(dk_weight, 0, d * sizeof(float), s) != cudaSuccess))
      return FA_ERR_CUDA;
    return FA_OK;
  }
  p.q = q;
  p.k = k;
  p.dq_out = dq_out;
  p.dk_out = dk_out;
  p.dq = dq;
  p.dk = dk;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.dq_stride = dq_stride;
  p.dk_stride = dk_stride;
  p.dq_weight = dq_weight;
  p.dk_weight = dk_weight;
  p.dw_part = static_cast<float*>(workspace);
  p.positions = positions;
  p.f32 = dtype == FA_FP32;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  return fa::launch_norm_rope_bwd(p, stream) == 0 ? FA_OK : FA_ERR_CUDA;
}

// fa_cache_append (no q, no norm, no rotation) and fa_qk_norm_rope_append; with
// `scales`, {of the key pages, of the value pages}, into pages of e4m3 codes.
static fa_status append_impl(fa::NormRopeParams& p, void* const* scales, const void* q, const void* k, const void* v,
                             void* q_out, void* k_pages, void* v_pages, long long q_stride,
                             long long k_stride, long long v_stride, const int32_t* block_table,
                             const int32_t* cache_seqlens, const int32_t* cu_seqlens, int B, int N,
                             long long total_tokens, int page_size, int num_pages, int max_pages,
                             void* stream) {
  if (p.Hkv == 0) return FA_ERR_SHAPE;
  fa_status st = page_args(&p, B, N, page_size, num_pages, max_pages);
  if (st != FA_OK) return st;
  const long long dense = (long long)B * N;
  if (!cu_seqlens && total_tokens != 0 && total_tokens != dense) return FA_ERR_SHAPE;
  if (!cu_seqlens && dense >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  p.T = cu_seqlens ? total_tokens : dense;
  if ((st = check_rows(q, q_stride, p.T, p.Hq, p.d, 2)) != FA_OK) return st;
  if ((st = check_rows(q_out, (long long)p.Hq * p.d, p.T, p.Hq, p.d, 2)) != FA_OK) return st;
  if ((st = check_rows(k, k_stride, p.T, p.Hkv, p.d, 2)) != FA_OK) return st;
  if ((st = check_rows(v, v_stride, p.T, p.Hkv, p.d, 2)) != FA_OK) return st;
  if (p.T == 0 || B == 0) return FA_OK;      // N = 0 with tokens: the kernel finds whose they are
  if (!k_pages || !v_pages || !block_table || !cache_seqlens) return FA_ERR_NULL;
  if (scales && (!scales[0] || !scales[1])) return FA_ERR_NULL;
  if (!aligned16(k_pages) || !aligned16(v_pages)) return FA_ERR_ALIGN;
  if (scales && (!aligned16(scales[0]) || !aligned16(scales[1]))) return FA_ERR_ALIGN;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.k_out = k_pages;
  p.v_out = v_pages;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.block_table = block_table;
  p.cache_seqlens = cache_seqlens;
  p.cu_seqlens = cu_seqlens;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  if (scales) {
    fa::QuantAppendParams qp = {};
    qp.n = p;
    qp.k_scales = static_cast<uint8_t*>(scales[0]);
    qp.v_scales = static_cast<uint8_t*>(scales[1]);
    return fa::launch_append_fp8(qp, p.Hq > 0, stream) == 0 ? FA_OK : FA_ERR_CUDA;
  }
  return fa::launch_norm_rope_pages(p, stream) == 0 ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_cache_append(const void* k, const void* v, void* k_pages, void* v_pages,
                          long long k_stride, long long v_stride, const int32_t* block_table,
                          const int32_t* cache_seqlens, const int32_t* cu_seqlens, int B, int Hkv,
                          int N, int d, long long total_tokens, int page_size, int num_pages,
                          int max_pages, void* stream) {
  fa::NormRopeParams p = {};
  const fa_status st = norm_rope_args(&p, nullptr, nullptr, 0.f, nullptr, nullptr, total_tokens, 0, Hkv, d, 0, 0, 0);
  if (st != FA_OK) return st;
  return append_impl(p, nullptr, nullptr, k, v, nullptr, k_pages, v_pages, 0, k_stride, v_stride, block_table,
                     cache_seqlens, cu_seqlens, B, N, total_tokens, page_size, num_pages, max_pages, stream);
}

fa_status fa_qk_norm_rope_append(const void* q, const void* k, const void* v, void* q_out,
                                 void* k_pages, void* v_pages, long long q_stride,
                                 long long k_stride, long long v_stride, const float* q_weight,
                                 const float* k_weight, float eps, const float* cos,
                                 const float* sin, const int32_t* block_table,
                                 const int32_t* cache_seqlens, const int32_t* cu_seqlens, int B,
                                 int Hq, int Hkv, int N, int d, long long total_tokens,
                                 int rot_dim, int max_pos, int interleaved, int page_size,
                                 int num_pages, int max_pages, void* stream) {
  fa::NormRopeParams p = {};
  const fa_status st = norm_rope_args(&p, q_weight, k_weight, eps, cos, sin, total_tokens, Hq, Hkv, d, rot_dim, max_pos, interleaved);
  if (st != FA_OK) return st;
  if (Hq == 0) return FA_ERR_SHAPE;
  if (!q_weight && rot_dim == 0) return FA_ERR_UNSUPPORTED;
  return append_impl(p, nullptr, q, k, v, q_out, k_pages, v_pages, q_stride, k_stride, v_stride, block_table,
                     cache_seqlens, cu_seqlens, B, N, total_tokens, page_size, num_pages, max_pages, stream);
}

fa_status fa_cache_append_fp8(const void* k, const void* v, void* k_pages, void* v_pages,
                              void* k_scales, void* v_scales, long long k_stride,
                              long long v_stride, const int32_t* block_table,
                              const int32_t* cache_seqlens, const int32_t* cu_seqlens, int B,
                              int Hkv, int N, int d, long long total_tokens, int page_size,
                              int num_pages, int max_pages, void* stream) {
  fa::NormRopeParams p = {};
  void* const scales[2] = {k_scales, v_scales};
  const fa_status st = norm_rope_args(&p, nullptr, nullptr, 0.f, nullptr, nullptr, total_tokens, 0, Hkv, d, 0, 0, 0);
  if (st != FA_OK) return st;
  return append_impl(p, scales, nullptr, k, v, nullptr, k_pages, v_pages, 0, k_stride, v_stride, block_table,
                     cache_seqlens, cu_seqlens, B, N, total_tokens, page_size, num_pages, max_pages, stream);
}

fa_status fa_qk_norm_rope_append_fp8(const void* q, const void* k, const void* v, void* q_out,
                                     void* k_pages, void* v_pages, void* k_scales,
                                     void* v_scales, long long q_stride, long long k_stride,
                                     long long v_stride, const float* q_weight,
                                     const float* k_weight, float eps, const float* cos,
                                     const float* sin, const int32_t* block_table,
                                     const int32_t* cache_seqlens, const int32_t* cu_seqlens,
                                     int B, int Hq, int Hkv, int N, int d,
                                     long long total_tokens, int rot_dim, int max_pos,
                                     int interleaved, int page_size, int num_pages,
                                     int max_pages, void* stream) {
  fa::NormRopeParams p = {};
  void* const scales[2] = {k_scales, v_scales};
  const fa_status st = norm_rope_args(&p, q_weight, k_weight, eps, cos, sin, total_tokens, Hq, Hkv, d, rot_dim, max_pos, interleaved);
  if (st != FA_OK) return st;
  if (Hq == 0) return FA_ERR_SHAPE;
  if (!q_weight && rot_dim == 0) return FA_ERR_UNSUPPORTED;
  return append_impl(p, scales, q, k, v, q_out, k_pages, v_pages, q_stride, k_stride, v_stride, block_table,
                     cache_seqlens, cu_seqlens, B, N, total_tokens, page_size, num_pages, max_pages, stream);
}

// Rows of the largest item of the paged forward: two tiles of 128 / group
// tokens, times the group's heads.
static long long paged_part_rows(int group, int N) { return (long long)std::min(2 * (128 / group), N) * group; }

// Workspace for parts of up to `part_rows` rows, and its places in p.
static size_t paged_parts(fa::PagedParams* p, char* ws, long long part_rows, int d) {
  const size_t rows = 2 * (size_t)fa::kPagedCtas * part_rows;
  const size_t o = round256(rows * d * sizeof(float)), ml = round256(rows * 4 * sizeof(float));
  if (p) {
    p->part_rows = (int)part_rows;
    p->part_o = reinterpret_cast<float*>(ws);
    p->part_ml = reinterpret_cast<float*>(ws + o);
    p->part_meta = reinterpret_cast<int4*>(ws + o + ml);
  }
  return o + ml + round256(2 * fa::kPagedCtas * sizeof(int4));
}

size_t fa_fwd_paged_workspace_size(int Hq, int Hkv, int N, int d) {
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || Hq / Hkv > 128 || N < 0 || d <= 0) return 0;
  return paged_parts(nullptr, nullptr, paged_part_rows(Hq / Hkv, N), d);
}

// Over codes, sequences of up to this many rows per kv head go to the kernel for
// few rows: 32 where no sequence brings more (then it is the call's only one),
// else what one token of each brings, in eights; 0 with larger groups.
static int paged_few_rows(int group, int N) {
  const long long rows = (long long)N * group <= 32 ? (long long)N * group : group;
  return rows <= 32 ? (int)std::max(1ll, (rows + 7) / 8) * 8 : 0;
}

static long long paged_few_part_rows(int group, int N) { return (long long)std::min(paged_few_rows(group, N) / group, N) * group; }

// q as codes: both parts, and the rows' exponents.
static size_t paged_codes(fa::PagedParams* p, char* ws, long long T, int Hq, int d) {
  const size_t codes = round256((size_t)2 * T * Hq * d);
  if (p) {
    p->q_codes = reinterpret_cast<uint8_t*>(ws);
    p->q_exps = reinterpret_cast<int*>(ws + codes);
  }
  return codes + round256((size_t)T * Hq * sizeof(int));
}

size_t fa_fwd_paged_fp8_workspace_size(int Hq, int Hkv, int N, int d, long long total_tokens) {
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || Hq / Hkv > 128 || N < 0 || d <= 0 || total_tokens < 0) return 0;
  const int group = Hq / Hkv, few = paged_few_rows(group, N);
  size_t n = 0;
  if (few) n += paged_parts(nullptr, nullptr, paged_few_part_rows(group, N), d);
  if ((long long)N * group > few)
    n += paged_parts(nullptr, nullptr, paged_part_rows(group, N), d) + paged_codes(nullptr, nullptr, total_tokens, Hq, d);
  return n;
}

// fa_fwd_paged, and with `scales` ({of the keys, of the values}) fa_fwd_paged_fp8.
static fa_status paged_impl(const void* q, const void* k_pages, const void* v_pages,
                            const void* const* scales, const int32_t* block_table,
                            const int32_t* cache_seqlens, const int32_t* cu_seqlens, void* o,
                            float* lse, int B, int Hq, int Hkv, int N, int d,
                            long long total_tokens, int page_size, int num_pages, int max_pages,
                            float scale, int causal, int window, const float* alibi_slopes,
                            fa_dtype o_dtype, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (Hq <= 0 || Hkv <= 0 || d <= 0 || total_tokens < 0) return FA_ERR_SHAPE;
  if (Hq % Hkv != 0) return FA_ERR_SHAPE;
  fa::NormRopeParams sizes = {};
  fa_status st = page_args(&sizes, B, N, page_size, num_pages, max_pages);
  if (st != FA_OK) return st;
  const long long dense = (long long)B * N;
  if (!cu_seqlens && total_tokens != 0 && total_tokens != dense) return FA_ERR_SHAPE;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (Hq / Hkv > 128 || Hq > 65535 || B > fa::kPagedMaxBatch) return FA_ERR_UNSUPPORTED;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_UNSUPPORTED;
  if (causal != 0 && causal != 1) return FA_ERR_UNSUPPORTED;
  if (!causal && (window >= 0 || alibi_slopes)) return FA_ERR_UNSUPPORTED;
  if (o_dtype != FA_FP32 && o_dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  const long long T = cu_seqlens ? total_tokens : dense;
  if (T >= (1ll << (scales ? 30 : 31)) || N >= (1 << 30)) return FA_ERR_UNSUPPORTED;   // (codes: q twice)
  if (T == 0 || B == 0) return FA_OK;        // N = 0 with tokens: the kernel finds whose they are
  if (num_pages == 0) return FA_ERR_SHAPE;
  if (!q || !k_pages || !v_pages || !block_table || !cache_seqlens || !o || !lse) return FA_ERR_NULL;
  if (scales && (!scales[0] || !scales[1])) return FA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages)) return FA_ERR_ALIGN;
  if (scales && (!aligned16(scales[0]) || !aligned16(scales[1]))) return FA_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(o) & 31u) != 0) return FA_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_ALIGN;
  const size_t need = scales ? fa_fwd_paged_fp8_workspace_size(Hq, Hkv, N, d, T) : fa_fwd_paged_workspace_size(Hq, Hkv, N, d);
  if (!workspace || workspace_bytes < need) return FA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_ALIGN;
  fa::PagedParams p = {};
  p.q = q;
  p.k = k_pages;
  p.v = v_pages;
  p.o = o;
  p.lse = lse;
  p.block_table = block_table;
  p.cache_seqlens = cache_seqlens;
  p.cu_seqlens = cu_seqlens;
  p.alibi = alibi_slopes;
  p.T = T;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.N = N;
  p.d = d;
  p.group = Hq / Hkv;
  p.tpt = 128 / p.group;
  char* ws = static_cast<char*>(workspace);
  if (!scales) paged_parts(&p, ws, paged_part_rows(p.group, N), d);
  // lanes that add up a sequence's q blocks: enough for the longest chunk
  const int blocks = (N + 2 * p.tpt - 1) / (2 * p.tpt);
  p.plan_lanes = 1;
  while (p.plan_lanes < 32 && p.plan_lanes < blocks) p.plan_lanes *= 2;
  p.page_size = page_size;
  p.page_shift = sizes.page_shift;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.causal = causal;
  const long long reach = (long long)max_pages * page_size;
  p.window = window < 0 || window >= reach - 1 ? fa::kNoWindow : window;
  p.o_f32 = o_dtype == FA_FP32;
  p.scale = scale;
  p.scale_log2 = scale * fa::kLog2e;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  if (scales) {
    p.k_scales = static_cast<const uint8_t*>(scales[0]);
    p.v_scales = static_cast<const uint8_t*>(scales[1]);
    p.few_rows = paged_few_rows(p.group, N);
    fa::PagedParams few = p;
    few.few = 1;
    if (p.few_rows) {
      few.tpt = p.few_rows / p.group;
      few.plan_lanes = 1;
      ws += paged_parts(&few, ws, paged_few_part_rows(p.group, N), d);
    } else {
      few.B = 0;
    }
    if ((long long)N * p.group > p.few_rows) {
      ws += paged_parts(&p, ws, paged_part_rows(p.group, N), d);
      paged_codes(&p, ws, T, Hq, d);
    } else {
      p.B = 0;
    }
    return fa::launch_fwd_paged_fp8(few, p, stream) == 0 ? FA_OK : FA_ERR_CUDA;
  }
  return fa::launch_fwd_paged(p, stream) == 0 ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_fwd_paged(const void* q, const void* k_pages, const void* v_pages,
                       const int32_t* block_table, const int32_t* cache_seqlens,
                       const int32_t* cu_seqlens, void* o, float* lse, int B, int Hq, int Hkv,
                       int N, int d, long long total_tokens, int page_size, int num_pages,
                       int max_pages, float scale, int causal, int window,
                       const float* alibi_slopes, fa_dtype o_dtype, void* workspace,
                       size_t workspace_bytes, void* stream) {
  return paged_impl(q, k_pages, v_pages, nullptr, block_table, cache_seqlens, cu_seqlens, o, lse, B,
                    Hq, Hkv, N, d, total_tokens, page_size, num_pages, max_pages, scale, causal,
                    window, alibi_slopes, o_dtype, workspace, workspace_bytes, stream);
}

fa_status fa_fwd_paged_fp8(const void* q, const void* k_pages, const void* v_pages,
                           const void* k_scales, const void* v_scales, const int32_t* block_table,
                           const int32_t* cache_seqlens, const int32_t* cu_seqlens, void* o,
                           float* lse, int B, int Hq, int Hkv, int N, int d,
                           long long total_tokens, int page_size, int num_pages, int max_pages,
                           float scale, int causal, int window, const float* alibi_slopes,
                           fa_dtype o_dtype, void* workspace, size_t workspace_bytes,
                           void* stream) {
  const void* const scales[2] = {k_scales, v_scales};
  return paged_impl(q, k_pages, v_pages, scales, block_table, cache_seqlens, cu_seqlens, o, lse, B,
                    Hq, Hkv, N, d, total_tokens, page_size, num_pages, max_pages, scale, causal,
                    window, alibi_slopes, o_dtype, workspace, workspace_bytes, stream);
}

// fa_cache_copy, and with `scales` ({of the keys, of the values}) fa_cache_copy_fp8.
static fa_status copy_impl(void* k_pages, void* v_pages, void* const* scales, const int32_t* src,
                           const int32_t* dst, int n, int num_pages, int page_size, int Hkv, int d,
                           void* stream) {
  if (n < 0 || Hkv <= 0 || d <= 0) return FA_ERR_SHAPE;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  // every block looks through all n pairs
  if (Hkv > 65535 || n > fa::kCopyMaxPairs) return FA_ERR_UNSUPPORTED;
  fa::NormRopeParams sizes = {};
  const fa_status st = page_args(&sizes, 0, 0, page_size, num_pages, 0);
  if (st != FA_OK) return st;
  if (n == 0) return FA_OK;
  if (!k_pages || !v_pages || !src || !dst) return FA_ERR_NULL;
  if (scales && (!scales[0] || !scales[1])) return FA_ERR_NULL;
  if (!aligned16(k_pages) || !aligned16(v_pages)) return FA_ERR_ALIGN;
  if (scales && (!aligned16(scales[0]) || !aligned16(scales[1]))) return FA_ERR_ALIGN;
  fa::CachePagesCopy p = {};
  p.k = k_pages;
  p.v = v_pages;
  if (scales) {
    p.k_scales = static_cast<uint8_t*>(scales[0]);
    p.v_scales = static_cast<uint8_t*>(scales[1]);
  }
  p.src = src;
  p.dst = dst;
  p.n = n;
  p.num_pages = num_pages;
  p.page_bytes = (long long)page_size * Hkv * d * (scales ? 1 : 2);
  p.scale_bytes = page_size / 16 * Hkv;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  return fa::launch_copy_pages(p, stream) == 0 ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_cache_copy(void* k_pages, void* v_pages, const int32_t* src, const int32_t* dst,
                        int n, int num_pages, int page_size, int Hkv, int d, void* stream) {
  return copy_impl(k_pages, v_pages, nullptr, src, dst, n, num_pages, page_size, Hkv, d, stream);
}

fa_status fa_cache_copy_fp8(void* k_pages, void* v_pages, void* k_scales, void* v_scales,
                            const int32_t* src, const int32_t* dst, int n, int num_pages,
                            int page_size, int Hkv, int d, void* stream) {
  void* const scales[2] = {k_scales, v_scales};
  return copy_impl(k_pages, v_pages, scales, src, dst, n, num_pages, page_size, Hkv, d, stream);
}

fa_status fa_selftest_wait_timeout(unsigned long long limit_ns, void* stream) {
  if (limit_ns == 0 || limit_ns > 10000000000ull) return FA_ERR_UNSUPPORTED;
  unsigned int* status = status_ptr();
  if (!status) return FA_ERR_CUDA;
  return fa::launch_selftest_wait(status, limit_ns, stream) == 0 ? FA_OK : FA_ERR_CUDA;
}

int fa_bwd_dkdv_split(int B, int Hq, int Hkv, int N, int d, int causal, int window,
                      const int32_t* cu_seqlens, size_t workspace_bytes) {
  if (B <= 0 || N <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return 1;
  if (cu_seqlens || gqa_split_max(Hq, Hkv) == 1) return 1;
  if (workspace_bytes < fa_bwd_workspace_size_gqa(B, Hq, Hkv, N, d, 0)) return 1;
  return dkdv_split(B, Hq, Hkv, N, d, causal ? 1 : 0, band_width(window, N));
}

void fa_host_cache_stats(unsigned long long* tmaps_encoded, unsigned long long* tmaps_reused,
                         unsigned long long* smem_attrs_set) {
  fa::host_cache_stats(tmaps_encoded, tmaps_reused, smem_attrs_set);
}

fa_status fa_check_device_error(void* stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return FA_ERR_CUDA;
  unsigned int* p = status_ptr();
  if (!p) return FA_ERR_CUDA;
  unsigned int v = 0;
  if (cudaMemcpy(&v, p, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return FA_ERR_CUDA;
  if (v != 0 && cudaMemset(p, 0, sizeof(v)) != cudaSuccess) return FA_ERR_CUDA;
  return static_cast<fa_status>(v);
}

}  // extern "C"
