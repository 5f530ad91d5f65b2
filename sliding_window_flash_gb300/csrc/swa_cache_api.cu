// swa_cache_api.cu — the C ABI of include/swa_cache.h: argument checks and launches of the cache
// calls and of the key weights.
#include <climits>
#include <cmath>
#include <cstdint>

#include "swa_cache_kernels.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr long long kIndexLimit = 1ll << 31;
constexpr long long kSlotLimit = 1ll << 30;  // of a sequence's table

// Slots in 30 bits (the kernels add to them), blocks (page, head) and table entries in 31; element
// offsets are 64-bit.
bool sizes_fit(int B, int Hkv, int max_pages, int page) {
  return static_cast<long long>(max_pages) * page < kSlotLimit &&
         static_cast<long long>(B) * Hkv < kIndexLimit && B <= 65535 && Hkv <= 65535;
}

// Query rows of an attention call in 31 bits (B <= 65535, T <= 64: no overflow here).
bool rows_fit(int B, int Hq, int T) { return static_cast<long long>(B) * Hq * T < kIndexLimit; }

// A window reaching past every slot changes nothing; clamping keeps the offsets in range.
int slots_seen(int window, int max_pages, int page) {
  const int slots = max_pages * page;
  return window < slots ? window : slots;
}

// Sinks that a window leaves to be seen: none where it hides nothing, and no more than there are slots.
int sinks_seen(int window, int sinks, int max_pages, int page) {
  const int slots = max_pages * page;
  return window >= slots ? 0 : sinks < slots ? sinks : slots;
}

// Query rows of a sequence and kv head that a call with a shared prefix takes.
constexpr int kSharedRows = 65536;

// Slots that are walked once for all sequences: a single sequence shares them with nobody.
int prefix_slots(int B, int shared, int page) { return B > 1 ? shared * page : 0; }

// The checks every cache call makes of the cache, its table and lengths.
swa_status check_cache(const swa_cache* c, const int* table, int max_pages, const int* lens, int B) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !table || !lens)
    return SWA_ERR_INVALID_ARG;
  if (c->pages < 1 || c->Hkv < 1 || max_pages < 1 || B < 1) return SWA_ERR_INVALID_ARG;
  if (c->page != 32 && c->page != 64 && c->page != 128) return SWA_ERR_UNSUPPORTED;
  if (c->D != 64 && c->D != 128 && c->D != 256) return SWA_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->pages) * c->Hkv >= kIndexLimit ||
      !sizes_fit(B, c->Hkv, max_pages, c->page))
    return SWA_ERR_INVALID_ARG;
  // What is read an element at a time needs an element's alignment only, here and in the calls below.
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) ||
      !aligned(c->v_scale, 4) || !aligned(c->weight, 16) || !aligned(table, 4) || !aligned(lens, 4))
    return SWA_ERR_MISALIGNED;
  return SWA_OK;
}

swa::CacheView view(const swa_cache* c, const int* table, int max_pages, const int* lens,
                    const int* new_lens, int B, int T, unsigned* err) {
  swa::CacheView v;
  v.k = static_cast<uint8_t*>(c->k);
  v.v = static_cast<uint8_t*>(c->v);
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  v.weight = c->weight;
  v.pages = c->pages;
  v.Hkv = c->Hkv;
  v.page = c->page;
  v.D = c->D;
  v.table = table;
  v.max_pages = max_pages;
  v.lens = lens;
  v.new_lens = new_lens;
  v.B = B;
  v.T = T;
  v.err = err;
  return v;
}

swa_status check_key_weights(int B, int Hq, int Hkv, int Lq, int Lk, int D, int window, int causal,
                             float scale) {
  if (causal != 0 && causal != 1) return SWA_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Lq < 1 || Lk < Lq || window < 1)
    return SWA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return SWA_ERR_INVALID_ARG;
  if (D != 64 && D != 128 && D != 256) return SWA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * Hq * Lq >= kIndexLimit ||
      static_cast<long long>(B) * Hkv * Lk >= kIndexLimit ||
      static_cast<long long>(B) * Hkv * ((static_cast<long long>(Lk) + 255) / 256) >= kIndexLimit / 2)
    return SWA_ERR_INVALID_ARG;
  return SWA_OK;
}

swa::Problem key_weights_problem(int B, int Hq, int Hkv, int Lq, int Lk, int D, int window,
                                 int sinks, int causal, float scale, int f16, unsigned* err) {
  swa::Problem pb;
  pb.B = B;
  pb.Hq = Hq;
  pb.Hkv = Hkv;
  pb.D = D;
  const int W = window < Lk ? window : Lk;
  pb.span.Lq = Lq;
  pb.span.Lk = Lk;
  pb.span.off = Lk - Lq;
  pb.span.dmin = causal ? 0 : -(W - 1);
  pb.span.dmax = W - 1;
  pb.scale = scale;
  pb.err = err;
  pb.f16 = f16;
  pb.sinks = W == Lk ? 0 : sinks < Lk ? sinks : Lk;
  return pb;
}

}  // namespace

extern "C" {

swa_status swa_cache_append(const swa_cache* cache, const int* table, int max_pages,
                            const int* lens, const int* new_lens, const void* k, const void* v,
                            const float* weight, int B, int T, int dtype, cudaStream_t stream) {
  swa_status st = check_cache(cache, table, max_pages, lens, B);
  if (st != SWA_OK) return st;
  if (!k || !v || T < 1 || dtype < SWA_BF16 || dtype > SWA_FP32) return SWA_ERR_INVALID_ARG;
  if (weight && !cache->weight) return SWA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * cache->Hkv * T >= kIndexLimit) return SWA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(weight, 4) || !aligned(new_lens, 4))
    return SWA_ERR_MISALIGNED;
  unsigned* err = nullptr;
  if ((st = swa::device_error_word(&err)) != SWA_OK) return st;
  const swa::CacheView c = view(cache, table, max_pages, lens, new_lens, B, T, err);
  return swa::launch_cache_append(c, k, v, weight, dtype, stream) == cudaSuccess ? SWA_OK
                                                                                 : SWA_ERR_CUDA;
}

size_t swa_cache_attn_shared_workspace_bytes(int B, int Hq, int Hkv, int T, int D, int max_pages,
                                             int page, int window, int sinks, int shared,
                                             int accumulate) {
  if (sinks < 0 || shared < 0 || shared > max_pages || (shared > 0 && accumulate) || B < 1 || Hq < 1 ||
      Hkv < 1 || Hq % Hkv != 0 || T < 1 || T > swa::kMaxCacheQueries || max_pages < 1 || window < 1 ||
      (D != 64 && D != 128 && D != 256) || (page != 32 && page != 64 && page != 128) ||
      !sizes_fit(B, Hkv, max_pages, page) || !rows_fit(B, Hq, T) ||
      (shared > 0 && Hq / Hkv * T > kSharedRows))
    return 0;
  return swa::cache_attn_workspace_bytes(B, Hq, Hkv, T, D, max_pages, page,
                                         slots_seen(window, max_pages, page),
                                         sinks_seen(window, sinks, max_pages, page),
                                         prefix_slots(B, shared, page), accumulate);
}

size_t swa_cache_attn_sinks_workspace_bytes(int B, int Hq, int Hkv, int T, int D, int max_pages,
                                            int page, int window, int sinks, int accumulate) {
  return swa_cache_attn_shared_workspace_bytes(B, Hq, Hkv, T, D, max_pages, page, window, sinks, 0,
                                               accumulate);
}

size_t swa_cache_attn_window_workspace_bytes(int B, int Hq, int Hkv, int T, int D, int max_pages,
                                             int page, int window, int accumulate) {
  return swa_cache_attn_sinks_workspace_bytes(B, Hq, Hkv, T, D, max_pages, page, window, 0, accumulate);
}

size_t swa_cache_attn_workspace_bytes(int B, int Hq, int Hkv, int T, int D, int max_pages,
                                      int page, int accumulate) {
  return swa_cache_attn_window_workspace_bytes(B, Hq, Hkv, T, D, max_pages, page, INT_MAX, accumulate);
}

swa_status swa_cache_attn(const swa_cache* cache, const int* table, int max_pages,
                          const int* lens, const int* new_lens, const void* q, void* o, float* lse,
                          int B, int Hq, int T, int window, float scale, int accumulate, int dtype,
                          void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return swa_cache_attn_sinks(cache, table, max_pages, lens, new_lens, q, o, lse, B, Hq, T, window, 0,
                              scale, accumulate, dtype, workspace, workspace_bytes, stream);
}

swa_status swa_cache_attn_sinks(const swa_cache* cache, const int* table, int max_pages,
                                const int* lens, const int* new_lens, const void* q, void* o,
                                float* lse, int B, int Hq, int T, int window, int sinks, float scale,
                                int accumulate, int dtype, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream) {
  return swa_cache_attn_shared(cache, table, max_pages, lens, new_lens, q, o, lse, B, Hq, T, window,
                               sinks, 0, scale, accumulate, dtype, workspace, workspace_bytes, stream);
}

swa_status swa_cache_attn_shared(const swa_cache* cache, const int* table, int max_pages,
                                 const int* lens, const int* new_lens, const void* q, void* o,
                                 float* lse, int B, int Hq, int T, int window, int sinks, int shared,
                                 float scale, int accumulate, int dtype, void* workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
  swa_status st = check_cache(cache, table, max_pages, lens, B);
  if (st != SWA_OK) return st;
  if (!q || !o || !lse || Hq < 1 || Hq % cache->Hkv != 0 || window < 1) return SWA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return SWA_ERR_INVALID_ARG;
  if (T < 1 || T > swa::kMaxCacheQueries || (accumulate != 0 && accumulate != 1) ||
      (dtype != SWA_BF16 && dtype != SWA_FP16))
    return SWA_ERR_INVALID_ARG;
  if (accumulate && !cache->weight) return SWA_ERR_INVALID_ARG;
  if (sinks < 0 || !rows_fit(B, Hq, T)) return SWA_ERR_INVALID_ARG;
  if (shared < 0 || shared > max_pages || (shared > 0 && accumulate) ||
      (shared > 0 && Hq / cache->Hkv * T > kSharedRows))
    return SWA_ERR_INVALID_ARG;
  const size_t need = swa_cache_attn_shared_workspace_bytes(
      B, Hq, cache->Hkv, T, cache->D, max_pages, cache->page, window, sinks, shared, accumulate);
  if (need != 0 && (!workspace || workspace_bytes < need)) return SWA_ERR_WORKSPACE;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 16) ||
      !aligned(new_lens, 4))
    return SWA_ERR_MISALIGNED;
  unsigned* err = nullptr;
  if ((st = swa::device_error_word(&err)) != SWA_OK) return st;
  const swa::CacheView c = view(cache, table, max_pages, lens, new_lens, B, T, err);
  swa::CacheAttnArgs a;
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.Hq = Hq;
  a.window = slots_seen(window, max_pages, cache->page);
  a.sinks = sinks_seen(window, sinks, max_pages, cache->page);
  a.base = prefix_slots(B, shared, cache->page);
  a.scale = scale;
  a.accumulate = accumulate;
  a.dtype = dtype;
  a.workspace = workspace;
  return swa::launch_cache_attn(c, a, stream) == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

swa_status swa_cache_evict(const swa_cache* cache, const int* table, int max_pages,
                           const int* lens, const int* dst_table, int dst_pages, int budget,
                           int recent, int* kept, int* lens_out, int B, cudaStream_t stream) {
  swa_status st = check_cache(cache, table, max_pages, lens, B);
  if (st != SWA_OK) return st;
  if (!cache->weight || !dst_table || !kept || !lens_out) return SWA_ERR_INVALID_ARG;
  if (dst_pages < 1 || budget < 1 || recent < 0 || recent > budget ||
      static_cast<long long>(dst_pages) * cache->page < budget ||
      static_cast<long long>(dst_pages) * cache->page >= kSlotLimit)
    return SWA_ERR_INVALID_ARG;
  if (!aligned(dst_table, 4) || !aligned(kept, 4) || !aligned(lens_out, 4))
    return SWA_ERR_MISALIGNED;
  if (dst_table == table) return SWA_ERR_INVALID_ARG;  // the pages read would be written
  unsigned* err = nullptr;
  if ((st = swa::device_error_word(&err)) != SWA_OK) return st;
  const swa::CacheView c = view(cache, table, max_pages, lens, nullptr, B, 0, err);
  swa::CacheEvictArgs a;
  a.dst_table = dst_table;
  a.dst_pages = dst_pages;
  a.budget = budget;
  a.recent = recent;
  a.kept = kept;
  a.lens_out = lens_out;
  return swa::launch_cache_evict(c, a, stream) == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

size_t swa_attn_key_weights_workspace_bytes(int B, int Hq, int Hkv, int Lq, int Lk, int D,
                                            int window, int causal) {
  return swa_attn_key_weights_sinks_workspace_bytes(B, Hq, Hkv, Lq, Lk, D, window, 0, causal);
}

size_t swa_attn_key_weights_sinks_workspace_bytes(int B, int Hq, int Hkv, int Lq, int Lk, int D,
                                                  int window, int sinks, int causal) {
  if (sinks < 0 || check_key_weights(B, Hq, Hkv, Lq, Lk, D, window, causal, 1.f) != SWA_OK) return 0;
  return swa::key_weights_workspace_bytes(
      key_weights_problem(B, Hq, Hkv, Lq, Lk, D, window, sinks, causal, 1.f, 0, nullptr));
}

swa_status swa_attn_key_weights(const void* q, const void* k, const float* lse, float* w, int B,
                                int Hq, int Hkv, int Lq, int Lk, int D, int window, int causal,
                                float scale, int dtype, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream) {
  return swa_attn_key_weights_sinks(q, k, lse, w, B, Hq, Hkv, Lq, Lk, D, window, 0, causal, scale, dtype,
                                    workspace, workspace_bytes, stream);
}

swa_status swa_attn_key_weights_sinks(const void* q, const void* k, const float* lse, float* w, int B,
                                      int Hq, int Hkv, int Lq, int Lk, int D, int window, int sinks,
                                      int causal, float scale, int dtype, void* workspace,
                                      size_t workspace_bytes, cudaStream_t stream) {
  if (!q || !k || !lse || !w || (dtype != SWA_BF16 && dtype != SWA_FP16) || sinks < 0)
    return SWA_ERR_INVALID_ARG;
  swa_status st = check_key_weights(B, Hq, Hkv, Lq, Lk, D, window, causal, scale);
  if (st != SWA_OK) return st;
  swa::Problem pb = key_weights_problem(B, Hq, Hkv, Lq, Lk, D, window, sinks, causal, scale,
                                        dtype == SWA_FP16, nullptr);
  const size_t need = swa::key_weights_workspace_bytes(pb);
  if (need != 0 && (!workspace || workspace_bytes < need)) return SWA_ERR_WORKSPACE;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(lse, 4) || !aligned(w, 4) ||
      !aligned(workspace, 16))
    return SWA_ERR_MISALIGNED;
  if ((st = swa::device_error_word(&pb.err)) != SWA_OK) return st;
  return swa::launch_key_weights(pb, q, k, lse, w, workspace, stream) == cudaSuccess
             ? SWA_OK
             : SWA_ERR_CUDA;
}

}  // extern "C"
