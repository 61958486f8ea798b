// C-ABI of the bdlm library: argument validation, the per-device workspace, TMA tensor
// maps and kernel launches.  See include/bdlm.h for the contract of each entry point.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>
#include <vector>

#include "../../include/bdlm.h"
#include "cache_ops.h"
#include "kernels.h"
#include "workspace.h"

namespace {

using bdlm::AttnPlan;
using bdlm::CommitPlan;
using bdlm::LmHeadPlan;
using bdlm::Workspace;

constexpr int kMaxDevices = 64;

struct DeviceState {
  bool checked = false;
  bool supported = false;
  int num_sms = 0;
  int* err = nullptr;            // device error word
  Workspace attn_cnt;            // attention scheduler counters (zero between calls)
  Workspace data;                // split / commit partials, gathered rows, sequence order
  Workspace aux;                 // prompt-block prefix lengths of a prefill
  std::vector<void*> retired;    // smaller workspaces that callers' graphs may hold
};

std::mutex g_mu;
DeviceState g_dev[kMaxDevices];
// Bumped whenever a workspace is reallocated or freed: CUDA graphs that captured the old
// buffers are re-captured before their next launch.
unsigned g_workspace_gen = 0;
// This thread is capturing the round loop's own graph, which such a bump has captured again.
thread_local bool t_own_capture = false;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;

// cudaMalloc whose failure is told by the return value alone: the runtime's last error is cleared, or
// the next call that asks for it after a launch would report this one's failure as its own.
bool device_alloc(void** ptr, size_t bytes) {
  if (cudaMalloc(ptr, bytes) == cudaSuccess) return true;
  cudaGetLastError();
  *ptr = nullptr;
  return false;
}

// Whether `stream` is being captured (the legacy default stream cannot be): nothing may be allocated
// then, nor the device waited for, which would end the capture.
int is_capturing(bdlm_stream stream, bool* yes) {
  *yes = false;
  if (!stream || stream == static_cast<bdlm_stream>(cudaStreamLegacy)) return BDLM_OK;
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &cs) != cudaSuccess)
    return BDLM_ERR_CUDA;
  *yes = cs != cudaStreamCaptureStatusNone;
  return BDLM_OK;
}

// The current device's state.  The first call sets up its error word, and is refused with
// BDLM_ERR_NOMEM while `stream` is being captured.
int current_device(DeviceState** st, bdlm_stream stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return BDLM_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return BDLM_ERR_UNSUPPORTED;
  DeviceState& s = g_dev[dev];
  if (!s.checked) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return BDLM_ERR_CUDA;
    s.supported = (major == 10 && minor == 3);
    s.num_sms = sms;
    if (s.supported && !s.err) {
      bool captured;
      const int rc = is_capturing(stream, &captured);
      if (rc) return rc;
      if (captured) return BDLM_ERR_NOMEM;
      void* err = nullptr;
      if (!device_alloc(&err, 256)) return BDLM_ERR_NOMEM;
      if (cudaMemset(err, 0, 256) != cudaSuccess ||
          cudaStreamSynchronize(nullptr) != cudaSuccess) {
        cudaFree(err);
        return BDLM_ERR_CUDA;
      }
      s.err = static_cast<int*>(err);
    }
    s.checked = true;
  }
  if (!s.supported) return BDLM_ERR_UNSUPPORTED;
  *st = &s;
  return BDLM_OK;
}

// A device's memory, as bdlm::grow takes it.
struct DeviceMemory {
  DeviceState* st;
  bool wait() { return cudaDeviceSynchronize() == cudaSuccess; }
  bool alloc(void** ptr, size_t bytes) { return device_alloc(ptr, bytes); }
  void free(void* ptr) { cudaFree(ptr); }
  bool zero(void* ptr, size_t bytes) {   // waits: the caller's stream may not wait for it
    return cudaMemset(ptr, 0, bytes) == cudaSuccess && cudaStreamSynchronize(nullptr) == cudaSuccess;
  }
  bool retire(void* ptr) {
    try {
      st->retired.push_back(ptr);
      return true;
    } catch (...) {   // no host memory for the list
      return false;
    }
  }
};

// Makes a workspace (zero-initialised where `zero`) hold `need` bytes, for work on `stream`.  Nothing
// can be allocated while `stream` is being captured: growth is refused with BDLM_ERR_NOMEM then,
// which leaves the capture valid.
int ensure(DeviceState* st, Workspace& w, size_t need, bool zero, bdlm_stream stream) {
  bool captured;
  const int rc = is_capturing(stream, &captured);
  if (rc) return rc;
  if (need <= w.cap) {
    if (captured && !t_own_capture) w.in_graph = true;
    return BDLM_OK;
  }
  if (captured) return BDLM_ERR_NOMEM;
  ++g_workspace_gen;
  return bdlm::grow(w, need, zero, DeviceMemory{st});
}

int get_encoder() {
  if (g_encode) return BDLM_OK;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                       &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess || fn == nullptr)
    return BDLM_ERR_CUDA;
  g_encode = reinterpret_cast<EncodeTiledFn>(fn);
  return BDLM_OK;
}

// bf16 tensor map, 128-byte swizzle; dims/strides innermost first, strides in bytes.
int encode(CUtensorMap* tm, const void* base, int rank, const cuuint64_t* dims,
           const cuuint64_t* strides, const cuuint32_t* box) {
  cuuint32_t es[5] = {1, 1, 1, 1, 1};
  CUresult r = g_encode(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base),
                        dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BDLM_OK : BDLM_ERR_INVALID;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Arguments of a commit rule: the threshold rule wants 0 <= threshold <= 1, the entropy rule a
// finite budget >= 0 (in `threshold`), the others k >= 1.
bool rule_ok(int rule, int k, float threshold) {
  switch (rule) {
    case BDLM_COMMIT_THRESHOLD: return threshold >= 0.f && threshold <= 1.f;
    case BDLM_COMMIT_ENTROPY_BOUNDED: return threshold >= 0.f && isfinite(threshold);
    case BDLM_COMMIT_TOPK:
    case BDLM_COMMIT_SEQUENTIAL:
    case BDLM_COMMIT_ANTI_SEQUENTIAL: return k >= 1;
    default: return false;
  }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace of the fused LM head + commit: gathered rows | partials | scored-row list | count.
struct LmCommitLayout {
  size_t off_part, off_act, off_n, total;
};
LmCommitLayout lm_commit_layout(const bdlm::LmConfPlan& plan, int rows) {
  LmCommitLayout l;
  l.off_part = align256(plan.gather_bytes);
  l.off_act = l.off_part + align256(plan.part_bytes);
  l.off_n = l.off_act + align256(static_cast<size_t>(rows) * sizeof(int32_t));
  l.total = l.off_n + 256;
  return l;
}

int reserve_attention(DeviceState* st, const bdlm_attn_desc& d, bool head_tables, AttnPlan* plan,
                      bdlm_stream stream);
int attention_impl(DeviceState* st, const bdlm_attn_desc& d, const bdlm_bf16* q,
                   const bdlm_bf16* k_pages, const bdlm_bf16* v_pages, const int32_t* page_table,
                   const int32_t* prefix_lens, bdlm_bf16* out, bdlm_stream stream,
                   int table_div, int mask_block = 0,
                   const bdlm::BlockKvWrite* kv_write = nullptr,
                   const bdlm::AttnExt* ext = nullptr);

}  // namespace

extern "C" {

const char* bdlm_status_string(int status) {
  switch (status) {
    case BDLM_OK: return "ok";
    case BDLM_ERR_INVALID: return "invalid argument";
    case BDLM_ERR_CUDA: return "CUDA error";
    case BDLM_ERR_UNSUPPORTED: return "unsupported device or shape";
    case BDLM_ERR_NOMEM: return "workspace allocation failed";
    default: return "unknown status";
  }
}

int bdlm_device_error(int* bits_out) {
  if (!bits_out) return BDLM_ERR_INVALID;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return BDLM_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return BDLM_ERR_UNSUPPORTED;
  if (cudaDeviceSynchronize() != cudaSuccess) return BDLM_ERR_CUDA;
  int v = 0;
  {
    // the workspace's word exists once an allocating call has run on this device
    std::lock_guard<std::mutex> lk(g_mu);
    const DeviceState& s = g_dev[dev];
    if (s.err) {
      if (cudaMemcpy(&v, s.err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
        return BDLM_ERR_CUDA;
      if (cudaMemset(s.err, 0, sizeof(int)) != cudaSuccess) return BDLM_ERR_CUDA;
    }
  }
  int w = 0;
  const int rc = bdlm::noalloc_take_error(dev, &w);  // bdlm_confidence_commit_noalloc's word
  if (rc) return rc;
  *bits_out = v | w;
  return BDLM_OK;
}

int bdlm_selftest_wait_timeout(int limit_us, bdlm_stream stream) {
  if (limit_us < 1 || limit_us > 2000000) return BDLM_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  const int rc = current_device(&st, stream);
  if (rc) return rc;
  const cudaError_t e = bdlm::launch_wait_timeout(
      st->err, static_cast<unsigned long long>(limit_us) * 1000ull,
      static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? BDLM_OK : BDLM_ERR_CUDA;
}

int bdlm_release(void) {
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  int rc = current_device(&st, nullptr);
  if (rc) return rc;
  if (cudaDeviceSynchronize() != cudaSuccess) return BDLM_ERR_CUDA;
  ++g_workspace_gen;
  for (Workspace* w : {&st->attn_cnt, &st->data, &st->aux}) {
    cudaFree(w->ptr);
    *w = Workspace{};
  }
  for (void* p : st->retired) cudaFree(p);
  st->retired.clear();
  return BDLM_OK;
}

int bdlm_confidence_commit(const bdlm_bf16* logits, const uint8_t* mask, int B, int L, int V,
                           float threshold, float temperature, int32_t* tok_out,
                           float* conf_out, uint8_t* commit_out, bdlm_stream stream) {
  return bdlm_confidence_commit_rule(logits, mask, B, L, V, BDLM_COMMIT_THRESHOLD, 1, threshold,
                                     temperature, tok_out, conf_out, nullptr, commit_out, stream);
}

int bdlm_confidence_commit_rule(const bdlm_bf16* logits, const uint8_t* mask, int B, int L, int V,
                                int rule, int k, float threshold, float temperature,
                                int32_t* tok_out, float* conf_out, float* entropy_out,
                                uint8_t* commit_out, bdlm_stream stream) {
  if (B < 0 || L < 1 || L > 64 || V < 1) return BDLM_ERR_INVALID;
  if (!(temperature > 0.f) || !isfinite(temperature)) return BDLM_ERR_INVALID;
  if (!rule_ok(rule, k, threshold)) return BDLM_ERR_INVALID;
  if (B == 0) return BDLM_OK;
  if (!logits || !mask || !tok_out || !conf_out || !commit_out) return BDLM_ERR_INVALID;
  if (static_cast<long long>(B) * L > 0x7FFFFFFFll) return BDLM_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  int rc = current_device(&st, stream);
  if (rc) return rc;
  const CommitPlan plan = bdlm::plan_commit(B, L, V, st->num_sms);
  if (plan.total_items > 0x7FFFFFFFll) return BDLM_ERR_INVALID;
  rc = ensure(st, st->data, plan.part_bytes, false, stream);
  if (rc) return rc;
  cudaError_t e = bdlm::launch_commit(logits, mask, B, L, V, threshold, temperature, tok_out,
                                      conf_out, entropy_out, commit_out, plan,
                                      static_cast<bdlm::CommitPartial*>(st->data.ptr), st->err,
                                      static_cast<cudaStream_t>(stream), rule, k);
  return e == cudaSuccess ? BDLM_OK : BDLM_ERR_CUDA;
}

int bdlm_apply_commit(uint8_t* mask, const uint8_t* commit, int n, bdlm_stream stream) {
  if (n < 0) return BDLM_ERR_INVALID;
  if (n == 0) return BDLM_OK;
  if (!mask || !commit) return BDLM_ERR_INVALID;
  cudaError_t e = bdlm::launch_apply_commit(mask, commit, n, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? BDLM_OK : BDLM_ERR_CUDA;
}

int bdlm_block_attention(const bdlm_attn_desc* desc, const bdlm_bf16* q,
                         const bdlm_bf16* k_pages, const bdlm_bf16* v_pages,
                         const int32_t* page_table, const int32_t* prefix_lens, int L,
                         bdlm_bf16* out, bdlm_stream stream) {
  if (!desc) return BDLM_ERR_INVALID;
  const bdlm_attn_desc d = *desc;
  if (d.B < 0 || L != d.L || d.L < 1 || d.L > 64 || d.Hq < 1 || d.Hkv < 1 ||
      d.Hq % d.Hkv != 0 || d.Hq / d.Hkv > 16 || d.D != 128 || d.page_size != 16 ||
      d.max_pages_per_seq < 1 || d.num_pages < 1 || !isfinite(d.sm_scale))
    return BDLM_ERR_INVALID;
  if (d.B == 0) return BDLM_OK;
  if (!q || !k_pages || !v_pages || !page_table || !prefix_lens || !out) return BDLM_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out))
    return BDLM_ERR_INVALID;
  if (static_cast<long long>(d.B) * d.L * d.Hq > 0x7FFFFFFFll ||
      static_cast<long long>(d.B) * d.max_pages_per_seq > 0x7FFFFFFFll ||
      static_cast<long long>(d.max_pages_per_seq) * d.page_size > 0x7FFFFFFFll)
    return BDLM_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  int rc = current_device(&st, stream);
  if (rc) return rc;
  return attention_impl(st, d, q, k_pages, v_pages, page_table, prefix_lens, out, stream, 1);
}

int bdlm_block_attention_kv(const bdlm_attn_desc* desc, const bdlm_bf16* q,
                            const bdlm_bf16* k_new, const bdlm_bf16* v_new, bdlm_bf16* k_pages,
                            bdlm_bf16* v_pages, const int32_t* page_table,
                            const int32_t* prefix_lens, int L, bdlm_bf16* out,
                            bdlm_stream stream) {
  if (!desc) return BDLM_ERR_INVALID;
  const bdlm_attn_desc d = *desc;
  if (d.B < 0 || L != d.L || d.L < 1 || d.L > 64 || d.Hq < 1 || d.Hkv < 1 ||
      d.Hq % d.Hkv != 0 || d.Hq / d.Hkv > 16 || d.D != 128 || d.page_size != 16 ||
      d.max_pages_per_seq < 1 || d.num_pages < 1 || !isfinite(d.sm_scale))
    return BDLM_ERR_INVALID;
  if (d.B == 0) return BDLM_OK;
  if (!q || !k_new || !v_new || !k_pages || !v_pages || !page_table || !prefix_lens || !out)
    return BDLM_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pages) ||
      !aligned16(v_pages) || !aligned16(out))
    return BDLM_ERR_INVALID;
  if (static_cast<long long>(d.B) * d.L * d.Hq > 0x7FFFFFFFll ||
      static_cast<long long>(d.B) * d.max_pages_per_seq > 0x7FFFFFFFll ||
      static_cast<long long>(d.max_pages_per_seq) * d.page_size > 0x7FFFFFFFll)
    return BDLM_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  int rc = current_device(&st, stream);
  if (rc) return rc;
  const bdlm::BlockKvWrite kw{k_new, v_new, k_pages, v_pages};
  return attention_impl(st, d, q, k_pages, v_pages, page_table, prefix_lens, out, stream, 1, 0,
                        &kw);
}

int bdlm_prefill_attention(const bdlm_attn_desc* desc, int prompt_len, const bdlm_bf16* q,
                           const bdlm_bf16* k_new, const bdlm_bf16* v_new, bdlm_bf16* k_pages,
                           bdlm_bf16* v_pages, const int32_t* page_table,
                           const int32_t* prefix_lens, bdlm_bf16* out, bdlm_stream stream) {
  if (!desc) return BDLM_ERR_INVALID;
  const bdlm_attn_desc d = *desc;
  if (d.B < 0 || d.L < 1 || d.L > 64 || d.Hq < 1 || d.Hkv < 1 || d.Hq % d.Hkv != 0 ||
      d.Hq / d.Hkv > 16 || d.D != 128 || d.page_size != 16 || d.max_pages_per_seq < 1 ||
      d.num_pages < 1 || !isfinite(d.sm_scale))
    return BDLM_ERR_INVALID;
  if (prompt_len < 1 || prompt_len % d.L != 0) return BDLM_ERR_INVALID;
  if (d.B == 0) return BDLM_OK;
  if (!q || !k_new || !v_new || !k_pages || !v_pages || !page_table || !prefix_lens || !out)
    return BDLM_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pages) ||
      !aligned16(v_pages) || !aligned16(out))
    return BDLM_ERR_INVALID;
  // Queries go to the attention in chunks of Lq positions (a multiple of L dividing the prompt,
  // Lq * G <= 256 query rows per KV head, the most one attention item takes) with the
  // block-causal mask inside a chunk, so each chunk reads the K/V before it once; chunks of
  // one block (Lq = L) need no mask.  Narrow chunks (Lq * G <= 32 rows) stay one block per
  // attention sequence.
  const int G = d.Hq / d.Hkv;
  int Lq = d.L;
  for (int c = d.L; c * G <= 256 && c <= prompt_len; c += d.L)
    if (prompt_len % c == 0) Lq = c;
  if (Lq * G <= 32) Lq = d.L;
  const int nb = prompt_len / Lq;
  if (static_cast<long long>(d.B) * prompt_len * d.Hq > 0x7FFFFFFFll ||
      static_cast<long long>(d.B) * d.max_pages_per_seq > 0x7FFFFFFFll ||
      static_cast<long long>(d.max_pages_per_seq) * d.page_size > 0x7FFFFFFFll)
    return BDLM_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  int rc = current_device(&st, stream);
  if (rc) return rc;
  rc = ensure(st, st->aux, static_cast<size_t>(d.B) * nb * sizeof(int32_t), false, stream);
  if (rc) return rc;
  bdlm_attn_desc dv = d;
  dv.B = d.B * nb;
  dv.L = Lq;
  AttnPlan plan;   // before anything is launched: a refused call writes nothing
  if ((rc = reserve_attention(st, dv, false, &plan, stream))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // the prompt's K/V into the cache, then one attention sequence per chunk of Lq queries
  if (bdlm::launch_write_block_kv(k_new, v_new, k_pages, v_pages, page_table, prefix_lens, d.B,
                                  prompt_len, d.Hkv, d.max_pages_per_seq, d.num_pages, st->err,
                                  s) != cudaSuccess)
    return BDLM_ERR_CUDA;
  int32_t* pre = static_cast<int32_t*>(st->aux.ptr);
  if (bdlm::launch_prompt_prefix(prefix_lens, d.B, nb, Lq, pre, s) != cudaSuccess)
    return BDLM_ERR_CUDA;
  return attention_impl(st, dv, q, k_pages, v_pages, page_table, pre, out, stream, nb,
                        Lq > d.L ? d.L : 0);
}
}  // extern "C"

namespace {

// Plans the attention and sizes its workspaces.
int reserve_attention(DeviceState* st, const bdlm_attn_desc& d, bool head_tables, AttnPlan* plan,
                      bdlm_stream stream) {
  *plan = bdlm::plan_attention(d.B, d.L, d.Hq, d.Hkv, d.max_pages_per_seq, d.page_size,
                               st->num_sms);
  if (plan->n_mma == 0) return BDLM_ERR_UNSUPPORTED;
  if (head_tables) bdlm::plan_even_lists(*plan, d.B, d.Hkv, d.max_pages_per_seq, st->num_sms);
  const int rc = ensure(st, st->attn_cnt, plan->cnt_bytes, true, stream);
  return rc ? rc : ensure(st, st->data, plan->part_bytes, false, stream);
}

// Block attention of d.B sequences (the caller holds g_mu and has validated d); sequence b
// uses page-table row b / table_div; mask_block > 0 makes each sequence's queries
// block-causal in blocks of mask_block.
int attention_impl(DeviceState* st, const bdlm_attn_desc& d, const bdlm_bf16* q,
                   const bdlm_bf16* k_pages, const bdlm_bf16* v_pages, const int32_t* page_table,
                   const int32_t* prefix_lens, bdlm_bf16* out, bdlm_stream stream,
                   int table_div, int mask_block, const bdlm::BlockKvWrite* kv_write,
                   const bdlm::AttnExt* ext) {
  int rc = get_encoder();
  if (rc) return rc;
  AttnPlan plan;
  if ((rc = reserve_attention(st, d, ext && ext->head_tables, &plan, stream))) return rc;
  // q viewed as [B*L rows][Hq heads][D]; box = 64 dims x G heads x lsub rows
  CUtensorMap tm_q, tm_k, tm_v;
  {
    cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(d.Hq), static_cast<cuuint64_t>(d.B) * d.L};
    cuuint64_t strides[2] = {256, static_cast<cuuint64_t>(d.Hq) * 256};
    cuuint32_t box[3] = {64, static_cast<cuuint32_t>(plan.G), static_cast<cuuint32_t>(plan.lsub)};
    if ((rc = encode(&tm_q, q, 3, dims, strides, box))) return rc;
  }
  {
    // pools viewed as [num_pages][page_size][Hkv][D]; box = 64 dims x 1 head x 16 slots
    cuuint64_t dims[4] = {128, static_cast<cuuint64_t>(d.Hkv), 16,
                          static_cast<cuuint64_t>(d.num_pages)};
    cuuint64_t strides[3] = {256, static_cast<cuuint64_t>(d.Hkv) * 256,
                             static_cast<cuuint64_t>(d.Hkv) * 256 * 16};
    cuuint32_t box[4] = {64, 1, 16, 1};
    if ((rc = encode(&tm_k, k_pages, 4, dims, strides, box))) return rc;
    if ((rc = encode(&tm_v, v_pages, 4, dims, strides, box))) return rc;
  }
  const float scale = d.sm_scale > 0.f ? d.sm_scale : 1.0f / sqrtf(128.0f);
  cudaError_t e = bdlm::launch_attention_ext(tm_q, tm_k, tm_v, page_table, prefix_lens, out, d.B,
                                             d.L, d.Hq, d.Hkv, d.max_pages_per_seq, d.num_pages,
                                             scale, plan, static_cast<float*>(st->data.ptr),
                                             static_cast<int*>(st->attn_cnt.ptr), st->err, st->num_sms,
                                             static_cast<cudaStream_t>(stream), table_div,
                                             mask_block, kv_write, ext);
  return e == cudaSuccess ? BDLM_OK : BDLM_ERR_CUDA;
}

// The LM head planned for n_active rows; n_active_dev (may be null) holds the count the
// kernels use, read on the device (at most n_active).
int lm_head_impl(const bdlm_bf16* hidden, const bdlm_bf16* w, const int32_t* active_idx,
                 int n_active, const int32_t* n_active_dev, int n_rows, int H, int V,
                 bdlm_bf16* logits, bdlm_stream stream) {
  if (n_active < 0 || n_rows < 0 || H < 8 || V < 8 || H % 8 != 0 || V % 8 != 0 ||
      n_active > n_rows)
    return BDLM_ERR_INVALID;
  if (n_active == 0) return BDLM_OK;
  if (!hidden || !w || !active_idx || !logits) return BDLM_ERR_INVALID;
  if (!aligned16(hidden) || !aligned16(w)) return BDLM_ERR_INVALID;
  if (static_cast<long long>(n_rows) * V > (1ll << 40)) return BDLM_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  int rc = current_device(&st, stream);
  if (rc) return rc;
  if ((rc = get_encoder())) return rc;
  const LmHeadPlan plan = bdlm::plan_lm_head(n_active, H, V, st->num_sms);
  rc = ensure(st, st->data, plan.gather_bytes, false, stream);
  if (rc) return rc;
  uint16_t* gathered = static_cast<uint16_t*>(st->data.ptr);
  CUtensorMap tm_w, tm_h;
  {
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(V)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(H) * 2};
    cuuint32_t box[2] = {64, 128};
    if ((rc = encode(&tm_w, w, 2, dims, strides, box))) return rc;
  }
  {
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(n_active)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(H) * 2};
    cuuint32_t box[2] = {64, static_cast<cuuint32_t>(plan.bn)};
    if ((rc = encode(&tm_h, gathered, 2, dims, strides, box))) return rc;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = bdlm::launch_gather_rows(hidden, active_idx, n_active, n_active_dev, n_rows, H,
                                           gathered, st->err, s);
  if (e != cudaSuccess) return BDLM_ERR_CUDA;
  e = bdlm::launch_lm_head(tm_w, tm_h, active_idx, n_active, n_active_dev, n_rows, H, V, logits,
                           plan, st->err, s);
  return e == cudaSuccess ? BDLM_OK : BDLM_ERR_CUDA;
}

}  // namespace

extern "C" {

int bdlm_lm_head(const bdlm_bf16* hidden, const bdlm_bf16* w, const int32_t* active_idx,
                 int n_active, int n_rows, int H, int V, bdlm_bf16* logits, bdlm_stream stream) {
  return lm_head_impl(hidden, w, active_idx, n_active, nullptr, n_rows, H, V, logits, stream);
}

int bdlm_lm_head_device_count(const bdlm_bf16* hidden, const bdlm_bf16* w,
                              const int32_t* active_idx, const int32_t* n_active_dev,
                              int max_active, int n_rows, int H, int V, bdlm_bf16* logits,
                              bdlm_stream stream) {
  if (!n_active_dev) return BDLM_ERR_INVALID;
  return lm_head_impl(hidden, w, active_idx, max_active, n_active_dev, n_rows, H, V, logits,
                      stream);
}

int bdlm_active_rows(const uint8_t* mask, const uint8_t* denoising, int B, int L,
                     int32_t* active_idx, int32_t* n_active_dev, bdlm_stream stream) {
  if (B < 0 || L < 1 || L > 64 || static_cast<long long>(B) * L > 0x7FFFFFFFll)
    return BDLM_ERR_INVALID;
  if (!mask || !active_idx || !n_active_dev) return BDLM_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  int rc = current_device(&st, stream);
  if (rc) return rc;
  cudaError_t e = bdlm::launch_active_rows(mask, denoising, B, L, active_idx, n_active_dev,
                                           static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? BDLM_OK : BDLM_ERR_CUDA;
}

int bdlm_write_block_kv(const bdlm_attn_desc* desc, const bdlm_bf16* k_new,
                        const bdlm_bf16* v_new, bdlm_bf16* k_pages, bdlm_bf16* v_pages,
                        const int32_t* page_table, const int32_t* prefix_lens, bdlm_stream stream) {
  if (!desc) return BDLM_ERR_INVALID;
  const bdlm_attn_desc d = *desc;
  if (d.B < 0 || d.L < 1 || d.L > 64 || d.Hkv < 1 || d.D != 128 || d.page_size != 16 ||
      d.max_pages_per_seq < 1 || d.num_pages < 1)
    return BDLM_ERR_INVALID;
  if (d.B == 0) return BDLM_OK;
  if (!k_new || !v_new || !k_pages || !v_pages || !page_table || !prefix_lens)
    return BDLM_ERR_INVALID;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pages) || !aligned16(v_pages))
    return BDLM_ERR_INVALID;
  if (static_cast<long long>(d.B) * d.L * d.Hkv > 0x7FFFFFFFll ||
      static_cast<long long>(d.B) * d.max_pages_per_seq > 0x7FFFFFFFll)
    return BDLM_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  int rc = current_device(&st, stream);
  if (rc) return rc;
  cudaError_t e = bdlm::launch_write_block_kv(k_new, v_new, k_pages, v_pages, page_table,
                                              prefix_lens, d.B, d.L, d.Hkv, d.max_pages_per_seq,
                                              d.num_pages, st->err,
                                              static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? BDLM_OK : BDLM_ERR_CUDA;
}

int bdlm_lm_head_commit(const bdlm_bf16* hidden, const bdlm_bf16* w, const uint8_t* mask,
                        const uint8_t* denoising, int B, int L, int H, int V, int rule, int k,
                        float threshold, float temperature, int32_t* tok_out, float* conf_out,
                        float* entropy_out, uint8_t* commit_out, bdlm_bf16* logits,
                        bdlm_stream stream) {
  if (B < 0 || L < 1 || L > 64 || H < 8 || V < 8 || H % 8 != 0 || V % 8 != 0)
    return BDLM_ERR_INVALID;
  if (!(temperature > 0.f) || !isfinite(temperature)) return BDLM_ERR_INVALID;
  if (!rule_ok(rule, k, threshold)) return BDLM_ERR_INVALID;
  if (B == 0) return BDLM_OK;
  if (!hidden || !w || !mask || !tok_out || !conf_out || !commit_out) return BDLM_ERR_INVALID;
  if (!aligned16(hidden) || !aligned16(w) || (logits && !aligned16(logits)))
    return BDLM_ERR_INVALID;
  const long long R = static_cast<long long>(B) * L;
  if (R > 0x7FFFFFFFll || R * V > (1ll << 40)) return BDLM_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  int rc = current_device(&st, stream);
  if (rc) return rc;
  if ((rc = get_encoder())) return rc;
  const int rows = static_cast<int>(R);
  const bdlm::LmConfPlan plan = bdlm::plan_lm_conf(rows, H, V, st->num_sms);
  if (plan.max_row_tiles > plan.units) return BDLM_ERR_UNSUPPORTED;
  const LmCommitLayout lay = lm_commit_layout(plan, rows);
  rc = ensure(st, st->data, lay.total, false, stream);
  if (rc) return rc;
  uint8_t* base = static_cast<uint8_t*>(st->data.ptr);
  uint16_t* gathered = reinterpret_cast<uint16_t*>(base);
  bdlm::CommitPartial* part = reinterpret_cast<bdlm::CommitPartial*>(base + lay.off_part);
  int32_t* act = reinterpret_cast<int32_t*>(base + lay.off_act);
  int32_t* n_act = reinterpret_cast<int32_t*>(base + lay.off_n);
  CUtensorMap tm_w, tm_h;
  {
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(V)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(H) * 2};
    cuuint32_t box[2] = {64, 128};
    if ((rc = encode(&tm_w, w, 2, dims, strides, box))) return rc;
  }
  {
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(H) * 2};
    cuuint32_t box[2] = {64, 128};
    if ((rc = encode(&tm_h, gathered, 2, dims, strides, box))) return rc;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = bdlm::launch_scored_gather(hidden, mask, denoising, B, L, H, gathered, act,
                                             n_act, s);
  if (e == cudaSuccess)
    e = bdlm::launch_lm_conf(tm_w, tm_h, act, n_act, rows, rows, H, V, temperature, logits, part,
                             plan, st->err, s,
                             entropy_out != nullptr || rule == BDLM_COMMIT_ENTROPY_BOUNDED);
  if (e == cudaSuccess)
    e = bdlm::launch_lm_commit_finalize(mask, denoising, B, L, part, plan, temperature, rule, k,
                                        threshold, tok_out, conf_out, entropy_out, commit_out, s);
  return e == cudaSuccess ? BDLM_OK : BDLM_ERR_CUDA;
}

}  // extern "C"

// ------------------------------------------------------------------ part of the cache
namespace {

// The limits of block attention's descriptor that depend on no pointer.
bool attn_desc_ok(const bdlm_attn_desc& d) {
  return d.B >= 0 && d.L >= 1 && d.L <= 64 && d.Hq >= 1 && d.Hkv >= 1 && d.Hq % d.Hkv == 0 &&
         d.Hq / d.Hkv <= 16 && d.D == 128 && d.page_size == 16 && d.max_pages_per_seq >= 1 &&
         d.num_pages >= 1 && isfinite(d.sm_scale) &&
         static_cast<long long>(d.B) * d.L * d.Hq <= 0x7FFFFFFFll &&
         static_cast<long long>(d.B) * d.max_pages_per_seq <= 0x7FFFFFFFll &&
         static_cast<long long>(d.max_pages_per_seq) * d.page_size <= 0x7FFFFFFFll;
}

// The same for calls that read no queries (L, Hq and sm_scale unused).
bool cache_desc_ok(const bdlm_attn_desc& d) {
  return d.B >= 0 && d.Hkv >= 1 && d.D == 128 && d.page_size == 16 && d.max_pages_per_seq >= 1 &&
         d.num_pages >= 1 && static_cast<long long>(d.B) * d.Hkv <= 0x7FFFFFFFll &&
         static_cast<long long>(d.B) * d.max_pages_per_seq <= 0x7FFFFFFFll &&
         static_cast<long long>(d.max_pages_per_seq) * d.page_size <= 0x7FFFFFFFll;
}

// The kernels that walk a sequence's tokens count them, and a few thousand past its end, in 32 bits.
constexpr int kMaxTokens = 1 << 30;
bool too_many_tokens(const bdlm_attn_desc& d) { return d.max_pages_per_seq > kMaxTokens / 16; }

// Moves of n tokens a list to other pages are one launch, a CTA for eight runs of 32.
bool too_many_moves(const bdlm_attn_desc& d, int n) {
  const long long runs = (static_cast<long long>(n) + 31) / 32;
  return static_cast<long long>(d.B) * d.Hkv * runs > 8 * 0x7FFFFFFFll;
}

bdlm::KeyParams key_params(const bdlm_attn_desc& d, const int32_t* page_table,
                           const int32_t* prefix_lens, int* err) {
  bdlm::KeyParams p = {};
  p.page_table = page_table;
  p.prefix_lens = prefix_lens;
  p.B = d.B;
  p.L = d.L;
  p.Hq = d.Hq;
  p.Hkv = d.Hkv;
  p.G = d.Hq / d.Hkv;
  p.max_pages = d.max_pages_per_seq;
  p.num_pages = d.num_pages;
  p.err = err;
  return p;
}

// Queries of nl block positions and of the query heads that share a KV head, 64 dims a box.
int encode_key_q(CUtensorMap* tm, const bdlm_bf16* q, const bdlm_attn_desc& d, int nl) {
  const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(d.Hq), static_cast<cuuint64_t>(d.B) * d.L};
  const cuuint64_t strides[2] = {256, static_cast<cuuint64_t>(d.Hq) * 256};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(d.Hq / d.Hkv), static_cast<cuuint32_t>(nl)};
  return encode(tm, q, 3, dims, strides, box);
}

}  // namespace

extern "C" {

int bdlm_tree_attention(const bdlm_attn_desc* desc, const bdlm_bf16* q, const bdlm_bf16* k_pages,
                        const bdlm_bf16* v_pages, const int32_t* page_table,
                        const int32_t* prefix_lens, const uint64_t* tree_mask, bdlm_bf16* out,
                        float* lse, bdlm_stream stream) {
  if (!desc || !attn_desc_ok(*desc)) return BDLM_ERR_INVALID;
  const bdlm_attn_desc d = *desc;
  if (d.B == 0) return BDLM_OK;
  if (!q || !k_pages || !v_pages || !page_table || !prefix_lens || !out) return BDLM_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(tree_mask) & 7) != 0)
    return BDLM_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  int rc = current_device(&st, stream);
  if (rc) return rc;
  bdlm::AttnExt ext;
  ext.tree = true;
  ext.tree_mask = tree_mask;
  ext.lse = lse;
  return attention_impl(st, d, q, k_pages, v_pages, page_table, prefix_lens, out, stream, 1, 0,
                        nullptr, &ext);
}

int bdlm_page_bounds(const bdlm_attn_desc* desc, const bdlm_bf16* k_pages,
                     const int32_t* page_table, const int32_t* from_lens, const int32_t* to_lens,
                     bdlm_bf16* bounds, bdlm_stream stream) {
  if (!desc || !cache_desc_ok(*desc)) return BDLM_ERR_INVALID;
  const bdlm_attn_desc d = *desc;
  if (too_many_tokens(d)) return BDLM_ERR_UNSUPPORTED;
  if (d.B == 0) return BDLM_OK;
  if (!k_pages || !page_table || !to_lens || !bounds || !aligned16(k_pages) || !aligned16(bounds))
    return BDLM_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  int rc = current_device(&st, stream);
  if (rc) return rc;
  return bdlm::launch_page_bounds(k_pages, page_table, from_lens, to_lens, d.B, d.Hkv,
                                  d.max_pages_per_seq, d.num_pages, st->num_sms, bounds, st->err,
                                  static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? BDLM_OK
             : BDLM_ERR_CUDA;
}

int bdlm_select_pages(const bdlm_attn_desc* desc, const bdlm_bf16* q, const bdlm_bf16* bounds,
                      const int32_t* page_table, const int32_t* prefix_lens, int group,
                      int n_select, int sel_cols, int32_t* sel_table, int32_t* sel_lens,
                      bdlm_stream stream) {
  if (!desc || !attn_desc_ok(*desc)) return BDLM_ERR_INVALID;
  const bdlm_attn_desc d = *desc;
  if (group < 1 || d.L % group != 0 || n_select < 0 ||
      sel_cols < static_cast<long long>(n_select) + (d.L + 30) / 16)
    return BDLM_ERR_INVALID;
  const int G = d.Hq / d.Hkv, groups = d.L / group;
  const long long lists = static_cast<long long>(d.B) * groups * d.Hkv;
  if (lists > 0x7FFFFFFFll) return BDLM_ERR_INVALID;
  if (group * G > bdlm::key_rows_max() || d.max_pages_per_seq > bdlm::kSelectMaxPages ||
      static_cast<long long>(d.num_pages) * d.Hkv > 0x3FFFFFFFll)   // (rows of bounds: 32 bits)
    return BDLM_ERR_UNSUPPORTED;
  if (d.B == 0) return BDLM_OK;
  if (!q || !bounds || !page_table || !prefix_lens || !sel_table || !sel_lens ||
      !aligned16(q) || !aligned16(bounds))
    return BDLM_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  int rc = current_device(&st, stream);
  if (rc) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int max_tiles = (d.max_pages_per_seq + bdlm::kKeyTile - 1) / bdlm::kKeyTile;
  bdlm::SelectParams sp{q, bounds, page_table, prefix_lens, nullptr, nullptr, nullptr,
                        d.B, d.L, d.Hq, d.Hkv, G, d.max_pages_per_seq, d.num_pages, group,
                        groups, max_tiles, n_select, sel_cols,
                        sel_table, sel_lens, st->err};
  if (!bdlm::select_scores_itself(static_cast<int>(lists), d.max_pages_per_seq, group * G,
                                  st->num_sms)) {
    // workspace: near ties' exact scores | scores | magnitudes
    const size_t score_bytes =
        align256(static_cast<size_t>(lists) * d.max_pages_per_seq * sizeof(float));
    const size_t amax_bytes =
        static_cast<size_t>(d.B) * d.Hkv * max_tiles * bdlm::kAmaxPerTile * sizeof(float);
    rc = ensure(st, st->data, 3 * score_bytes + amax_bytes, false, stream);
    if (rc) return rc;
    bdlm::KeyParams p = key_params(d, page_table, prefix_lens, st->err);
    p.max_tiles = max_tiles;
    p.q = q;
    p.bounds = bounds;
    p.scores = reinterpret_cast<float*>(static_cast<uint8_t*>(st->data.ptr) + 2 * score_bytes);
    p.amax = reinterpret_cast<float*>(static_cast<uint8_t*>(st->data.ptr) + 3 * score_bytes);
    p.group = group;
    p.groups = groups;
    p.width = group * G;
    // a launch scores whole groups of up to 256 query rows per KV head
    int per = bdlm::key_rows_max() / (group * G) * group;
    if (per > d.L) per = d.L;
    CUtensorMap tm_q = {}, tm_bounds = {};
    if (per * G > bdlm::kDirectRows) {
      if ((rc = get_encoder())) return rc;
      const cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(d.num_pages) * d.Hkv * 2};
      const cuuint64_t strides[1] = {256};
      const cuuint32_t box[2] = {64, 1};
      if ((rc = encode(&tm_bounds, bounds, 2, dims, strides, box))) return rc;
    }
    for (p.l0 = 0; p.l0 < d.L; p.l0 += per) {
      const int nl = d.L - p.l0 < per ? d.L - p.l0 : per;
      p.rows = nl * G;
      if (p.rows > bdlm::kDirectRows && (rc = encode_key_q(&tm_q, q, d, nl))) return rc;
      if (bdlm::launch_page_scores(tm_q, tm_bounds, p, st->num_sms, s) != cudaSuccess)
        return BDLM_ERR_CUDA;
    }
    sp.scores = p.scores;
    sp.amax = p.amax;
    sp.exact = static_cast<unsigned long long*>(st->data.ptr);
  }
  return bdlm::launch_select_pages(sp, st->num_sms, s) == cudaSuccess ? BDLM_OK : BDLM_ERR_CUDA;
}

int bdlm_sparse_attention(const bdlm_attn_desc* desc, const bdlm_bf16* q, const bdlm_bf16* k_pages,
                          const bdlm_bf16* v_pages, int group, int sel_cols,
                          const int32_t* sel_table, const int32_t* sel_lens, bdlm_bf16* out,
                          bdlm_stream stream) {
  if (!desc || !attn_desc_ok(*desc)) return BDLM_ERR_INVALID;
  bdlm_attn_desc d = *desc;
  if (group < 1 || d.L % group != 0 || sel_cols < 1) return BDLM_ERR_INVALID;
  if (d.B == 0) return BDLM_OK;
  if (!q || !k_pages || !v_pages || !sel_table || !sel_lens || !out || !aligned16(q) ||
      !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out))
    return BDLM_ERR_INVALID;
  // every query group is an attention sequence with a page list per KV head
  d.B *= d.L / group;
  d.L = group;
  d.max_pages_per_seq = sel_cols;
  if (!attn_desc_ok(d)) return BDLM_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  int rc = current_device(&st, stream);
  if (rc) return rc;
  bdlm::AttnExt ext;
  ext.head_tables = true;
  return attention_impl(st, d, q, k_pages, v_pages, sel_table, sel_lens, out, stream, 1, 0,
                        nullptr, &ext);
}

int bdlm_attention_weights(const bdlm_attn_desc* desc, const bdlm_bf16* q,
                           const bdlm_bf16* k_pages, const int32_t* page_table,
                           const int32_t* prefix_lens, const float* lse, float decay,
                           float* weights, bdlm_stream stream) {
  if (!desc || !attn_desc_ok(*desc) || !isfinite(decay)) return BDLM_ERR_INVALID;
  const bdlm_attn_desc d = *desc;
  if (too_many_tokens(d)) return BDLM_ERR_UNSUPPORTED;
  if (d.sm_scale > 0.f && d.sm_scale < 0x1p-64f) return BDLM_ERR_UNSUPPORTED;   // lse / sm_scale
  if (d.B == 0) return BDLM_OK;
  if (!q || !k_pages || !page_table || !prefix_lens || !lse || !weights || !aligned16(q) ||
      !aligned16(k_pages))
    return BDLM_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  int rc = current_device(&st, stream);
  if (rc) return rc;
  if ((rc = get_encoder())) return rc;
  const int G = d.Hq / d.Hkv;
  int per = bdlm::key_rows_max() / G;   // block positions of one launch
  if (per > d.L) per = d.L;
  CUtensorMap tm_q, tm_k;
  {
    cuuint64_t dims[4] = {128, static_cast<cuuint64_t>(d.Hkv), 16,
                          static_cast<cuuint64_t>(d.num_pages)};
    cuuint64_t strides[3] = {256, static_cast<cuuint64_t>(d.Hkv) * 256,
                             static_cast<cuuint64_t>(d.Hkv) * 256 * 16};
    cuuint32_t box[4] = {64, 1, 16, 1};
    if ((rc = encode(&tm_k, k_pages, 4, dims, strides, box))) return rc;
  }
  bdlm::KeyParams p = key_params(d, page_table, prefix_lens, st->err);
  p.max_tiles = static_cast<int>((static_cast<long long>(d.max_pages_per_seq) * d.page_size +
                                  bdlm::kKeyTile - 1) / bdlm::kKeyTile);
  p.lse = lse;
  p.weights = weights;
  p.decay = decay;
  p.scale_log2 = (d.sm_scale > 0.f ? d.sm_scale : 1.0f / sqrtf(128.0f)) * 1.4426950408889634f;
  // more than 256 query rows per KV head: one launch per 256, each adding to the one before
  for (p.l0 = 0; p.l0 < d.L; p.l0 += per) {
    const int nl = d.L - p.l0 < per ? d.L - p.l0 : per;
    p.rows = nl * G;
    if ((rc = encode_key_q(&tm_q, q, d, nl))) return rc;
    if (bdlm::launch_attention_weights(tm_q, tm_k, p, st->num_sms,
                                       static_cast<cudaStream_t>(stream)) != cudaSuccess)
      return BDLM_ERR_CUDA;
    p.decay = 1.f;
  }
  return BDLM_OK;
}

int bdlm_evict_kv(const bdlm_attn_desc* desc, bdlm_bf16* k_pages, bdlm_bf16* v_pages,
                  const int32_t* page_table, const int32_t* lens, const float* weights, int keep,
                  int recent, const int32_t* to_table, float* to_weights, int32_t* kept,
                  int32_t* new_lens, bdlm_stream stream) {
  if (!desc || !cache_desc_ok(*desc)) return BDLM_ERR_INVALID;
  const bdlm_attn_desc d = *desc;
  if (keep < 1 || keep > static_cast<long long>(d.max_pages_per_seq) * d.page_size || recent < 0 ||
      recent > keep)
    return BDLM_ERR_INVALID;
  if (too_many_tokens(d) || (to_table != page_table && too_many_moves(d, keep)))
    return BDLM_ERR_UNSUPPORTED;
  if (d.B == 0) return BDLM_OK;
  if (!k_pages || !v_pages || !page_table || !lens || !weights || !to_table || !to_weights ||
      !kept || !new_lens || lens == new_lens || !aligned16(k_pages) || !aligned16(v_pages))
    return BDLM_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  int rc = current_device(&st, stream);
  if (rc) return rc;
  const bdlm::EvictParams p{lens, weights, to_weights, kept, new_lens, d.B, d.Hkv,
                            d.max_pages_per_seq, keep, recent, st->err};
  const bdlm::CompactParams m{k_pages, v_pages, page_table, to_table, nullptr, kept, new_lens,
                              d.B, d.Hkv, d.Hkv, d.max_pages_per_seq, d.num_pages, keep, st->err};
  return bdlm::launch_evict(p, m, st->num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? BDLM_OK
             : BDLM_ERR_CUDA;
}

int bdlm_compact_kv(const bdlm_attn_desc* desc, bdlm_bf16* k_pages, bdlm_bf16* v_pages,
                    const int32_t* page_table, const int32_t* base_lens, const int32_t* idx,
                    int heads, int n_max, const int32_t* counts, const int32_t* to_table,
                    bdlm_stream stream) {
  if (!desc || !cache_desc_ok(*desc)) return BDLM_ERR_INVALID;
  const bdlm_attn_desc d = *desc;
  if ((heads != 1 && heads != d.Hkv) || n_max < 0) return BDLM_ERR_INVALID;
  if (too_many_tokens(d) || n_max > kMaxTokens ||
      (to_table != page_table && too_many_moves(d, n_max)))
    return BDLM_ERR_UNSUPPORTED;
  if (d.B == 0 || n_max == 0) return BDLM_OK;
  if (!k_pages || !v_pages || !page_table || !idx || !counts || !to_table || !aligned16(k_pages) ||
      !aligned16(v_pages))
    return BDLM_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  int rc = current_device(&st, stream);
  if (rc) return rc;
  const bdlm::CompactParams p{k_pages, v_pages, page_table, to_table, base_lens, idx, counts,
                              d.B, d.Hkv, heads, d.max_pages_per_seq, d.num_pages, n_max, st->err};
  return bdlm::launch_compact(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? BDLM_OK
                                                                                  : BDLM_ERR_CUDA;
}

}  // extern "C"

// ------------------------------------------------------------------ device-side round loop
struct bdlm_round_loop {
  bdlm_round_loop_desc d;
  int device = 0;
  void* scratch = nullptr;
  bdlm_bf16 *q_w = nullptr, *k_w = nullptr, *v_w = nullptr, *h_w = nullptr;
  bdlm_bf16* attn_out = nullptr;
  int32_t* tok = nullptr;
  float* conf = nullptr;
  uint8_t* com = nullptr;
  int* step = nullptr;
  cudaStream_t cap = nullptr;
  cudaGraph_t graph = nullptr;
  cudaGraphExec_t exec = nullptr;
  unsigned gen = 0;
};

namespace {

// Sizes the library workspaces for one round of the loop (nothing may be allocated while the
// round is being captured, nor while `stream` is).
int reserve_round(const bdlm_round_loop_desc& d, bdlm_stream stream) {
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState* st = nullptr;
  int rc = current_device(&st, stream);
  if (rc) return rc;
  const bdlm_attn_desc& a = d.attn;
  const AttnPlan ap = bdlm::plan_attention(a.B, a.L, a.Hq, a.Hkv, a.max_pages_per_seq,
                                           a.page_size, st->num_sms);
  if (ap.n_mma == 0) return BDLM_ERR_UNSUPPORTED;
  const int R = a.B * a.L;
  const bdlm::LmConfPlan cp = bdlm::plan_lm_conf(R, d.H, d.V, st->num_sms);
  if (cp.max_row_tiles > cp.units) return BDLM_ERR_UNSUPPORTED;
  size_t data = ap.part_bytes;
  const size_t fused = lm_commit_layout(cp, R).total;
  if (fused > data) data = fused;
  if ((rc = ensure(st, st->attn_cnt, ap.cnt_bytes, true, stream))) return rc;
  if ((rc = ensure(st, st->data, data, false, stream))) return rc;
  return get_encoder();
}

void drop_graph(bdlm_round_loop* lp) {
  if (lp->exec) cudaGraphExecDestroy(lp->exec);
  if (lp->graph) cudaGraphDestroy(lp->graph);
  lp->exec = nullptr;
  lp->graph = nullptr;
}

// Builds the graph: step counter := 0, then WHILE(condition) { one round }.  It will be launched on
// `stream`.
int capture_round_loop(bdlm_round_loop* lp, bdlm_stream stream) {
  const bdlm_round_loop_desc& d = lp->d;
  const bdlm_attn_desc& a = d.attn;
  const int R = a.B * a.L;
  int rc = reserve_round(d, stream);
  if (rc) return rc;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    lp->gen = g_workspace_gen;
  }
  drop_graph(lp);
  if (cudaGraphCreate(&lp->graph, 0) != cudaSuccess) return BDLM_ERR_CUDA;
  cudaMemsetParams ms = {};
  ms.dst = lp->step;
  ms.value = 0;
  ms.elementSize = 4;
  ms.width = 1;
  ms.height = 1;
  cudaGraphNode_t init;
  if (cudaGraphAddMemsetNode(&init, lp->graph, nullptr, 0, &ms) != cudaSuccess) return BDLM_ERR_CUDA;
  cudaGraphConditionalHandle handle;
  if (cudaGraphConditionalHandleCreate(&handle, lp->graph, 1, cudaGraphCondAssignDefault) !=
      cudaSuccess)
    return BDLM_ERR_CUDA;
  cudaGraphNodeParams np = {};
  np.type = cudaGraphNodeTypeConditional;
  np.conditional.handle = handle;
  np.conditional.type = cudaGraphCondTypeWhile;
  np.conditional.size = 1;
  cudaGraphNode_t loop;
  if (cudaGraphAddNode(&loop, lp->graph, &init, nullptr, 1, &np) != cudaSuccess) return BDLM_ERR_CUDA;
  cudaGraph_t body = np.conditional.phGraph_out[0];
  if (cudaStreamBeginCaptureToGraph(lp->cap, body, nullptr, nullptr, 0,
                                    cudaStreamCaptureModeThreadLocal) != cudaSuccess)
    return BDLM_ERR_CUDA;
  bdlm_stream s = lp->cap;
  bdlm::StepCopy c = {};
  c.src[0] = reinterpret_cast<const uint4*>(d.q_steps);
  c.dst[0] = reinterpret_cast<uint4*>(lp->q_w);
  c.n_vec[0] = static_cast<long long>(R) * a.Hq * a.D * 2 / 16;
  c.src[1] = reinterpret_cast<const uint4*>(d.k_new_steps);
  c.dst[1] = reinterpret_cast<uint4*>(lp->k_w);
  c.n_vec[1] = static_cast<long long>(R) * a.Hkv * a.D * 2 / 16;
  c.src[2] = reinterpret_cast<const uint4*>(d.v_new_steps);
  c.dst[2] = reinterpret_cast<uint4*>(lp->v_w);
  c.n_vec[2] = c.n_vec[1];
  c.src[3] = reinterpret_cast<const uint4*>(d.hidden_steps);
  c.dst[3] = reinterpret_cast<uint4*>(lp->h_w);
  c.n_vec[3] = static_cast<long long>(R) * d.H * 2 / 16;
  int r2 = BDLM_OK;
  t_own_capture = true;
  if (bdlm::launch_select_step(c, lp->step, d.steps, lp->cap) != cudaSuccess) r2 = BDLM_ERR_CUDA;
  if (!r2) r2 = bdlm_block_attention_kv(&a, lp->q_w, lp->k_w, lp->v_w, d.k_pages, d.v_pages,
                                        d.page_table, d.prefix_lens, a.L, lp->attn_out, s);
  if (!r2) r2 = bdlm_lm_head_commit(lp->h_w, d.w, d.mask, d.denoising, a.B, a.L, d.H, d.V, d.rule,
                                    d.k, d.threshold, d.temperature, lp->tok, lp->conf, nullptr,
                                    lp->com, nullptr, s);
  if (!r2 && bdlm::launch_record_step(lp->step, d.steps, R, lp->tok, lp->conf, lp->com,
                                      d.tok_steps, d.conf_steps, d.commit_steps,
                                      reinterpret_cast<const uint4*>(lp->attn_out),
                                      reinterpret_cast<uint4*>(d.attn_out_steps),
                                      static_cast<long long>(R) * a.Hq * a.D * 2 / 16,
                                      lp->cap) != cudaSuccess)
    r2 = BDLM_ERR_CUDA;
  if (!r2) r2 = bdlm_apply_commit(d.mask, lp->com, R, s);
  if (!r2 && bdlm::launch_loop_condition(handle, d.mask, R, lp->step, d.steps, d.steps_done,
                                         lp->cap) != cudaSuccess)
    r2 = BDLM_ERR_CUDA;
  t_own_capture = false;
  cudaGraph_t captured = nullptr;
  const cudaError_t ec = cudaStreamEndCapture(lp->cap, &captured);
  if (r2) return r2;
  if (ec != cudaSuccess) return BDLM_ERR_CUDA;
  if (cudaGraphInstantiate(&lp->exec, lp->graph, 0) != cudaSuccess) return BDLM_ERR_CUDA;
  return BDLM_OK;
}

}  // namespace

extern "C" {

int bdlm_round_loop_create(const bdlm_round_loop_desc* desc, bdlm_round_loop** out) {
  if (!desc || !out) return BDLM_ERR_INVALID;
  *out = nullptr;
  const bdlm_round_loop_desc& d = *desc;
  const bdlm_attn_desc& a = d.attn;
  if (a.B < 1 || a.L < 1 || a.L > 64 || a.Hq < 1 || a.Hkv < 1 || a.Hq % a.Hkv != 0 ||
      a.D != 128 || a.page_size != 16 || a.max_pages_per_seq < 1 || a.num_pages < 1)
    return BDLM_ERR_INVALID;
  if (d.steps < 1 || d.H < 8 || d.H % 8 != 0 || d.V < 8 || d.V % 8 != 0) return BDLM_ERR_INVALID;
  if (!rule_ok(d.rule, d.k, d.threshold)) return BDLM_ERR_INVALID;
  if (!(d.temperature > 0.f) || !isfinite(d.temperature)) return BDLM_ERR_INVALID;
  if (!d.q_steps || !d.k_new_steps || !d.v_new_steps || !d.hidden_steps || !d.k_pages ||
      !d.v_pages || !d.page_table || !d.prefix_lens || !d.w || !d.mask || !d.tok_steps ||
      !d.conf_steps || !d.commit_steps || !d.steps_done)
    return BDLM_ERR_INVALID;
  if (d.attn_out_steps && !aligned16(d.attn_out_steps)) return BDLM_ERR_INVALID;
  const long long R = static_cast<long long>(a.B) * a.L;
  if (R * a.Hq > 0x7FFFFFFFll || R * d.V > (1ll << 40)) return BDLM_ERR_INVALID;
  auto* lp = new bdlm_round_loop();
  lp->d = d;
  cudaGetDevice(&lp->device);
  // owned scratch: one step's inputs, the attention output, this step's tok/conf/commit and
  // the step counter (the logits never leave the fused LM head)
  const size_t q_b = align256(R * a.Hq * a.D * 2), kv_b = align256(R * a.Hkv * a.D * 2);
  const size_t h_b = align256(R * d.H * 2);
  const size_t r4 = align256(R * 4), r1 = align256(R);
  const size_t total = 2 * q_b + 2 * kv_b + h_b + 2 * r4 + r1 + 256;
  if (!device_alloc(&lp->scratch, total)) {
    delete lp;
    return BDLM_ERR_NOMEM;
  }
  uint8_t* p = static_cast<uint8_t*>(lp->scratch);
  lp->q_w = reinterpret_cast<bdlm_bf16*>(p);      p += q_b;
  lp->attn_out = reinterpret_cast<bdlm_bf16*>(p); p += q_b;
  lp->k_w = reinterpret_cast<bdlm_bf16*>(p);      p += kv_b;
  lp->v_w = reinterpret_cast<bdlm_bf16*>(p);      p += kv_b;
  lp->h_w = reinterpret_cast<bdlm_bf16*>(p);      p += h_b;
  lp->tok = reinterpret_cast<int32_t*>(p);        p += r4;
  lp->conf = reinterpret_cast<float*>(p);         p += r4;
  lp->com = p;                                    p += r1;
  lp->step = reinterpret_cast<int*>(p);
  if (cudaStreamCreateWithFlags(&lp->cap, cudaStreamNonBlocking) != cudaSuccess) {
    cudaFree(lp->scratch);
    delete lp;
    return BDLM_ERR_CUDA;
  }
  const int rc = capture_round_loop(lp, nullptr);
  if (rc) {
    bdlm_round_loop_destroy(lp);
    return rc;
  }
  *out = lp;
  return BDLM_OK;
}

int bdlm_round_loop_launch(bdlm_round_loop* loop, bdlm_stream stream) {
  if (!loop) return BDLM_ERR_INVALID;
  unsigned gen = 0;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    gen = g_workspace_gen;
  }
  if (gen != loop->gen || !loop->exec) {
    const int rc = capture_round_loop(loop, stream);  // a workspace moved since the capture
    if (rc) return rc;
  }
  bool captured;
  const int rc = is_capturing(stream, &captured);
  if (rc) return rc;
  if (captured) {   // the caller's graph will hold what the loop's does
    std::lock_guard<std::mutex> lk(g_mu);
    g_dev[loop->device].attn_cnt.in_graph = g_dev[loop->device].data.in_graph = true;
  }
  return cudaGraphLaunch(loop->exec, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? BDLM_OK
             : BDLM_ERR_CUDA;
}

int bdlm_round_loop_destroy(bdlm_round_loop* loop) {
  if (!loop) return BDLM_OK;
  drop_graph(loop);
  if (loop->cap) cudaStreamDestroy(loop->cap);
  if (loop->scratch) cudaFree(loop->scratch);
  delete loop;
  return BDLM_OK;
}

}  // extern "C"
