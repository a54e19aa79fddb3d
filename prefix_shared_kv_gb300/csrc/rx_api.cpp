// C-ABI of the library: argument checks, the host work planners, the radix cache and the token
// accounting.  Device work is in the .cu files; this file launches nothing itself.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <limits>
#include <memory>
#include <numeric>
#include <queue>
#include <string>
#include <unordered_map>
#include <vector>

#include "rx_internal.h"

using namespace rx;

namespace {

thread_local std::string g_err;

rx_status fail(rx_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_err = buf;
  return st;
}

rx_status cuda_fail(int e, const char* what) {
  return fail(RX_ERR_CUDA, "%s: %s", what, cudaGetErrorString((cudaError_t)e));
}

// A planner's result; no C++ exception leaves a C entry (the plan may then be of no kind, or the one
// it was).
template <class F>
rx_status no_throw(F&& plan) {
  try {
    return plan();
  } catch (const std::exception& e) {
    return fail(RX_ERR_WORKSPACE, "the plan does not fit the host's memory (%s)", e.what());
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

rx_status check_desc(const rx_kv_desc* d, bool need_table) {
  if (!d) return fail(RX_ERR_INVALID, "desc is NULL");
  if (d->head_dim != kHeadDim) return fail(RX_ERR_UNSUPPORTED, "head_dim %d != 128", d->head_dim);
  if (d->num_kv_heads <= 0 || d->num_q_heads <= 0)
    return fail(RX_ERR_INVALID, "head counts must be positive");
  if (d->num_q_heads % d->num_kv_heads)
    return fail(RX_ERR_UNSUPPORTED, "num_q_heads %% num_kv_heads != 0");
  const int gq = d->num_q_heads / d->num_kv_heads;
  if (gq != 1 && gq != 2 && gq != 4 && gq != 8)
    return fail(RX_ERR_UNSUPPORTED, "head ratio %d not in {1,2,4,8}", gq);
  if (d->num_kv_heads > 256) return fail(RX_ERR_UNSUPPORTED, "num_kv_heads > 256");
  if (d->pool_size <= 0 || d->pool_size > (int64_t)INT32_MAX)
    return fail(RX_ERR_INVALID, "pool_size must be in [1, 2^31)");
  if (!(d->softmax_scale > 0.f) || !std::isfinite(d->softmax_scale))
    return fail(RX_ERR_INVALID, "softmax_scale must be finite and > 0");
  if (need_table) {
    if (!d->req_to_token) return fail(RX_ERR_INVALID, "req_to_token is NULL");
    if (d->req_to_token_rows <= 0 || d->req_to_token_stride <= 0 ||
        d->req_to_token_stride > (int64_t)INT32_MAX || d->req_to_token_rows > (int64_t)INT32_MAX)
      return fail(RX_ERR_INVALID, "bad req_to_token shape");
  }
  return RX_OK;
}

// SMs of the current device (plans are sized for it); 152 when no device can be asked
int device_sms() {
  static std::atomic<int> cached[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 152;
  }
  if ((n = cached[dev].load()) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0) {
    cached[dev].store(n);
    return n;
  }
  cudaGetLastError();
  return 152;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

// ---------------------------------------------------------------------------------------------
// Plans
// ---------------------------------------------------------------------------------------------
struct rx_plan {
  int kind = 0;  // 0 = empty, 1 = extend, 2 = decode
  int32_t ext_kernel = RX_EXTEND_TILES;  // the kernel extend plans built from now on run on
  int32_t kv_next = RX_KV_BF16;          // the pool type plans built from now on are for
  int32_t kv_type = RX_KV_BF16;          // the pool type the built plan is for
  std::vector<uint8_t> blob;  // header + tables, uploaded verbatim
  size_t ws_bytes = 0;
  int64_t key_reads = 0;  // (key, KV head) rows of the pool the kernels read
  double q8_us = 0;       // decode plans for the 8-bit pool: the planner's estimate of a call
  int32_t hq = 0, hkv = 0;
  int64_t rows = 0, stride = 0, pool = 0;
  const int32_t* table = nullptr;
  // rx_plan_upload stages the blob in pinned host memory so that the copy is asynchronous for the
  // host too; `staged` records the copy, and the buffer is reused only once it has completed
  mutable void* pinned = nullptr;
  mutable size_t pinned_bytes = 0;
  mutable cudaEvent_t staged = nullptr;
  mutable int staged_dev = -1;
  mutable bool staged_pending = false;
  // decode: the second stream on which a call runs its mma.sync units beside the tensor-core
  // units, with its fork / join events; created on first use, on that call's device, and owned by
  // the plan (so callers with plans of their own never serialise on a shared stream)
  mutable cudaStream_t aux = nullptr;
  mutable cudaEvent_t aux_fork = nullptr, aux_join = nullptr;
  mutable int aux_dev = -1;
  void drop_aux() const {
    if (aux_fork) cudaEventDestroy(aux_fork);
    if (aux_join) cudaEventDestroy(aux_join);
    if (aux) cudaStreamDestroy(aux);
    aux = nullptr;
    aux_fork = aux_join = nullptr;
    aux_dev = -1;
  }
  ~rx_plan() {
    if (staged) {
      if (staged_pending) cudaEventSynchronize(staged);
      cudaEventDestroy(staged);
    }
    if (pinned) cudaFreeHost(pinned);
    drop_aux();
  }
  PlanHeader hdr() const {
    PlanHeader h;
    std::memcpy(&h, blob.data(), sizeof h);
    return h;
  }
};

namespace {

// Steps of the tensor-core attention kernel over a segment of n keys, and an item's cost in
// fourteenths of a two-tile step.  The weights are a least-squares fit of the per-CTA times of
// the extend, radix-mixed (tree and one-level), chunked-prefill and paged workloads (globaltimer
// at each CTA's entry and exit, 760 CTAs): a two-tile step 1.03 µs, a one-tile step 0.81 µs, and
// 4.9 µs per item beyond its steps (its query tiles in, its rows out, the pipelines' refill).
int32_t attn_steps(int64_t n) { return (int32_t)((n + kAttnKeys - 1) / kAttnKeys); }
int64_t attn_cost(const ExtItem& it) { return (int64_t)it.n_steps * (it.n_tok[1] > 0 ? 14 : 11); }
constexpr int64_t kItemCost = 66;

// 8-bit pool: an item's last `steps` steps, given to CTA `to`.
struct Cut {
  int32_t item, steps, to;
};
// A cut costs its two pieces' partial rows about two steps, and the plan a merge (5 us, and what it
// takes to write and read the rows), in the units of attn_cost.  The figures were fitted over 60 random
// batches: five groups of six requests with 1 to 9 new tokens on 5,169, 16 heads, 145 us without
// cuts, 123 with; five groups of nine with up to 1,365 on 986, one head, 86 and 65; a chunk of 2,048
// new tokens on 5,120, 32/8 heads, 229 and 232: not cut.
constexpr int64_t kCutCost = 28, kMergeCost = 75, kMergeRowsPerCost = 160;
constexpr int32_t kLeastPiece = 4;  // steps

// Cuts by which every list ends at `end` or before: each that ends later gives the end of its longest
// item to the one with most room.  False when that does not do.
bool cut_lists(const std::vector<ExtItem>& items, const std::vector<std::vector<int32_t>>& lists,
               const std::vector<int64_t>& load, int64_t end, std::vector<Cut>& cuts) {
  cuts.clear();
  std::priority_queue<std::pair<int64_t, int32_t>> room;
  std::vector<std::pair<int64_t, int32_t>> late;
  for (int32_t k = 0; k < (int32_t)load.size(); ++k)
    if (load[k] > end)
      late.push_back({load[k] - end, k});
    else
      room.push({end - load[k], k});
  std::sort(late.begin(), late.end(), std::greater<std::pair<int64_t, int32_t>>());
  for (const auto& l : late) {
    int32_t longest = lists[l.second][0];
    for (int32_t i : lists[l.second])
      if (items[i].n_steps > items[longest].n_steps) longest = i;
    const ExtItem& it = items[longest];
    const int64_t step = it.n_tok[1] > 0 ? 14 : 11;
    const int32_t n =
        (int32_t)std::max<int64_t>(kLeastPiece, (l.first + kCutCost + step - 1) / step);
    if (it.n_steps - n < kLeastPiece || room.empty()) return false;
    const auto to = room.top();
    const int64_t left = to.first - (n * step + kItemCost + kCutCost);
    if (left < 0) return false;
    room.pop();
    room.push({left, to.second});
    cuts.push_back({longest, n, to.second});
  }
  return true;
}

// SMs of the calling thread's current GPU, the number of per-CTA lists an extend plan for the
// one-SM kernel makes; a GB300's 152 where no GPU can be asked (plans are host work).
int32_t plan_sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0)
    return n;
  (void)cudaGetLastError();
  return 152;
}
// On the SM-pair kernel an item takes steps of kPairKeys keys per segment and costs its steps
// whether or not it has a second tile (the other CTA gathers and multiplies anyway).
int32_t pair_steps(int64_t n) { return (int32_t)((n + kPairKeys - 1) / kPairKeys); }
constexpr int64_t kPairCostClass = 2;  // two steps

template <typename T>
void put(std::vector<uint8_t>& blob, int64_t off, const std::vector<T>& v) {
  if (!v.empty()) std::memcpy(blob.data() + off, v.data(), v.size() * sizeof(T));
}

void remember_desc(rx_plan* p, const rx_kv_desc* d) {
  p->kv_type = p->kv_next;
  p->hq = d->num_q_heads;
  p->hkv = d->num_kv_heads;
  p->rows = d->req_to_token_rows;
  p->stride = d->req_to_token_stride;
  p->pool = d->pool_size;
  p->table = d->req_to_token;
}

// The pointers of an 8-bit pool.
rx_status check_kv_q8(const rx_kv_q8* kv) {
  if (!kv) return fail(RX_ERR_INVALID, "kv is NULL");
  if (!kv->k_code || !kv->v_code || !kv->k_scale || !kv->v_scale)
    return fail(RX_ERR_INVALID, "NULL code or scale pointer");
  if (!aligned16(kv->k_code) || !aligned16(kv->v_code) || !aligned16(kv->k_scale) ||
      !aligned16(kv->v_scale))
    return fail(RX_ERR_INVALID, "codes and scales must be 16-byte aligned");
  return RX_OK;
}

// Whether a built plan's attention call has rows; without any it enqueues nothing and takes no tensors.
bool has_rows(const PlanHeader& h) { return h.n_items > 0 || (h.kind == 2 && h.batch > 0); }

rx_status check_plan_use(const rx_plan* p, int kind, int32_t kv_type, const rx_kv_desc* d,
                         const void* k,
                         const void* v, const void* q, const void* o, const void* lse,
                         const void* ws, size_t ws_bytes) {
  if (!p) return fail(RX_ERR_INVALID, "plan is NULL");
  if (p->kind != kind)
    return fail(RX_ERR_INVALID, "plan was built for %s", p->kind == 1 ? "extend" : p->kind == 2 ? "decode" : "nothing");
  if (p->kv_type != kv_type)
    return fail(RX_ERR_INVALID, "plan was built for a %s pool (rx_plan_set_kv_type)",
                p->kv_type == RX_KV_E4M3 ? "8-bit" : "bf16");
  rx_status st = check_desc(d, true);
  if (st) return st;
  if (d->num_q_heads != p->hq || d->num_kv_heads != p->hkv || d->req_to_token_rows != p->rows ||
      d->req_to_token_stride != p->stride || d->pool_size != p->pool)
    return fail(RX_ERR_INVALID, "descriptor differs from the one the plan was built with");
  if (has_rows(p->hdr())) {
    if (!k || !v || !q || !o || !lse) return fail(RX_ERR_INVALID, "NULL tensor pointer");
    if (!aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(o) || !aligned16(lse))
      return fail(RX_ERR_INVALID, "tensors must be 16-byte aligned");
  }
  if (!ws) return fail(RX_ERR_WORKSPACE, "workspace is NULL");
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return fail(RX_ERR_INVALID, "workspace must be 256-byte aligned");
  if (ws_bytes < p->ws_bytes)
    return fail(RX_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed", ws_bytes, p->ws_bytes);
  return RX_OK;
}

// check_plan_use for a call over an 8-bit pool.
rx_status check_plan_use_q8(const rx_plan* p, int kind, const rx_kv_desc* d, const rx_kv_q8* kv,
                            const void* q, const void* o, const void* lse, const void* ws,
                            size_t ws_bytes) {
  const bool no_rows = p && p->kind == kind && !has_rows(p->hdr());
  const rx_status st = no_rows ? RX_OK : check_kv_q8(kv);
  if (st) return st;
  return check_plan_use(p, kind, RX_KV_E4M3, d, kv ? kv->k_code : nullptr,
                        kv ? kv->v_code : nullptr, q, o, lse, ws, ws_bytes);
}

}  // namespace

rx_status rx::set_error(rx_status st, const char* msg) { return fail(st, "%s", msg); }

rx_status rx::plan_aux_stream(const rx_plan* plan, AuxStream* out) {
  out->stream = out->fork = out->join = nullptr;
  const PlanHeader h = plan->hdr();
  if (!(h.n_xitems > 0 && h.n_items > 0)) return RX_OK;  // one kernel: no second stream
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e) return cuda_fail(e, "decode: current device");
  if (plan->aux && plan->aux_dev != dev) plan->drop_aux();  // streams belong to one device
  if (!plan->aux) {
    e = cudaStreamCreateWithFlags(&plan->aux, cudaStreamNonBlocking);
    if (!e) e = cudaEventCreateWithFlags(&plan->aux_fork, cudaEventDisableTiming);
    if (!e) e = cudaEventCreateWithFlags(&plan->aux_join, cudaEventDisableTiming);
    if (e) {
      plan->drop_aux();
      return cuda_fail(e, "decode: second stream");
    }
    plan->aux_dev = dev;
  }
  out->stream = plan->aux;
  out->fork = plan->aux_fork;
  out->join = plan->aux_join;
  return RX_OK;
}

rx_status rx::plan_for_noalloc(const rx_plan* plan, const rx_kv_desc* desc, const void* k,
                               const void* v, const void* q, const void* o, const void* lse,
                               const void* scratch, size_t scratch_bytes, PlanHeader* hdr) {
  if (plan && plan->kind == 2 && plan->ws_bytes > scratch_bytes)
    return fail(RX_ERR_WORKSPACE,
                "rx_decode_attn_noalloc: the plan needs %zu bytes of scratch, the library holds "
                "%zu; use rx_decode_attn with a workspace for batches this large",
                plan->ws_bytes, scratch_bytes);
  rx_status st = check_plan_use(plan, 2, RX_KV_BF16, desc, k, v, q, o, lse, scratch,
                                scratch_bytes);
  if (st) return st;
  *hdr = plan->hdr();
  return RX_OK;
}

extern "C" {

const char* rx_status_string(int s) {
  switch (s) {
    case RX_OK: return "ok";
    case RX_ERR_INVALID: return "invalid argument";
    case RX_ERR_RANGE: return "out of range";
    case RX_ERR_UNSUPPORTED: return "unsupported shape";
    case RX_ERR_CUDA: return "CUDA error";
    case RX_ERR_TIMEOUT: return "device wait timed out";
    case RX_ERR_WORKSPACE: return "workspace too small";
    default: return "unknown status";
  }
}

const char* rx_last_error(void) { return g_err.c_str(); }

rx_status rx_store_kv(const rx_kv_desc* desc, void* k_pool, void* v_pool, const void* k_new,
                      const void* v_new, const int32_t* slots, int64_t num_tokens,
                      rx_stream_t stream) {
  rx_status st = check_desc(desc, false);
  if (st) return st;
  if (num_tokens < 0) return fail(RX_ERR_INVALID, "num_tokens < 0");
  if (num_tokens == 0) return RX_OK;
  if (!k_pool || !v_pool || !k_new || !v_new || !slots)
    return fail(RX_ERR_INVALID, "NULL pointer");
  if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(k_new) || !aligned16(v_new))
    return fail(RX_ERR_INVALID, "K/V pointers must be 16-byte aligned");
  if (num_tokens > (int64_t)INT32_MAX) return fail(RX_ERR_RANGE, "num_tokens >= 2^31");
  const int e = launch_store_kv(desc, k_pool, v_pool, k_new, v_new, slots, num_tokens, stream);
  return e ? cuda_fail(e, "store_kv launch") : RX_OK;
}

rx_status rx_store_kv_q8(const rx_kv_desc* desc, const rx_kv_q8* kv, const void* k_new,
                         const void* v_new, const int32_t* slots, int64_t num_tokens,
                         rx_stream_t stream) {
  rx_status st = check_desc(desc, false);
  if (st) return st;
  if (num_tokens < 0) return fail(RX_ERR_INVALID, "num_tokens < 0");
  if (num_tokens == 0) return RX_OK;
  st = check_kv_q8(kv);
  if (st) return st;
  if (!k_new || !v_new || !slots) return fail(RX_ERR_INVALID, "NULL pointer");
  if (!aligned16(k_new) || !aligned16(v_new))
    return fail(RX_ERR_INVALID, "K/V pointers must be 16-byte aligned");
  if (num_tokens > (int64_t)INT32_MAX) return fail(RX_ERR_RANGE, "num_tokens >= 2^31");
  const int e = launch_store_kv_q8(desc, kv, k_new, v_new, slots, num_tokens, stream);
  return e ? cuda_fail(e, "store_kv_q8 launch") : RX_OK;
}

rx_status rx_load_kv_q8(const rx_kv_desc* desc, const rx_kv_q8* kv, const int32_t* slots,
                        int64_t num_tokens, void* k_out, void* v_out, rx_stream_t stream) {
  rx_status st = check_desc(desc, false);
  if (st) return st;
  if (num_tokens < 0) return fail(RX_ERR_INVALID, "num_tokens < 0");
  if (num_tokens == 0) return RX_OK;
  st = check_kv_q8(kv);
  if (st) return st;
  if (!k_out || !v_out || !slots) return fail(RX_ERR_INVALID, "NULL pointer");
  if (!aligned16(k_out) || !aligned16(v_out))
    return fail(RX_ERR_INVALID, "K/V pointers must be 16-byte aligned");
  if (num_tokens > (int64_t)INT32_MAX) return fail(RX_ERR_RANGE, "num_tokens >= 2^31");
  const int e = launch_load_kv_q8(desc, kv, slots, num_tokens, k_out, v_out, stream);
  return e ? cuda_fail(e, "load_kv_q8 launch") : RX_OK;
}

rx_status rx_plan_create(rx_plan** out) {
  if (!out) return fail(RX_ERR_INVALID, "out is NULL");
  *out = new rx_plan();
  return RX_OK;
}

void rx_plan_destroy(rx_plan* plan) { delete plan; }

rx_status rx_plan_set_extend_kernel(rx_plan* plan, int32_t kernel) {
  if (!plan) return fail(RX_ERR_INVALID, "plan is NULL");
  if (kernel != RX_EXTEND_TILES && kernel != RX_EXTEND_PAIR)
    return fail(RX_ERR_INVALID, "unknown extend kernel");
  plan->ext_kernel = kernel;
  return RX_OK;
}

rx_status rx_plan_set_kv_type(rx_plan* plan, int32_t kv_type) {
  if (!plan) return fail(RX_ERR_INVALID, "plan is NULL");
  if (kv_type != RX_KV_BF16 && kv_type != RX_KV_E4M3)
    return fail(RX_ERR_INVALID, "unknown pool type");
  plan->kv_next = kv_type;
  return RX_OK;
}

rx_status rx_plan_key_reads(const rx_plan* plan, int64_t* rows) {
  if (!plan || !rows) return fail(RX_ERR_INVALID, "NULL argument");
  if (!plan->kind) return fail(RX_ERR_INVALID, "plan has not been built");
  *rows = plan->key_reads;
  return RX_OK;
}

rx_status rx_plan_rows(const rx_plan* plan, int64_t* rows) {
  if (!plan || !rows) return fail(RX_ERR_INVALID, "NULL argument");
  if (!plan->kind) return fail(RX_ERR_INVALID, "plan has not been built");
  const PlanHeader h = plan->hdr();
  *rows = h.kind == 1 ? h.n_rows : h.batch;  // extend: one row per new token
  return RX_OK;
}

rx_status rx_plan_launches(const rx_plan* plan, int32_t* launches) {
  if (!plan || !launches) return fail(RX_ERR_INVALID, "NULL argument");
  if (!plan->kind) return fail(RX_ERR_INVALID, "plan has not been built");
  const PlanHeader h = plan->hdr();
  // the same conditions the launchers test: extend -- the tensor-core kernel when there are
  // items; decode -- the tensor-core kernel for its shared-prefix units, the mma.sync partial
  // kernel for the others, and the merge whenever there are requests
  // (an extend over an 8-bit pool expands the plan's keys in a kernel of its own first, and merges
  // when its tiles' keys are split, or runs as a decode of its few new tokens)
  *launches = h.kind == 1 ? (h.n_items > 0) * (1 + (h.kv_type == RX_KV_E4M3) +
                                                   (h.n_part_rows > 0))
                              : (h.n_xitems > 0) * (1 + (h.kv_type == RX_KV_E4M3)) + (h.n_wide > 0) + (h.n_items > 0) + (h.batch > 0);
  return RX_OK;
}

rx_status rx_plan_workspace_size(const rx_plan* plan, size_t* bytes) {
  if (!plan || !bytes) return fail(RX_ERR_INVALID, "NULL argument");
  if (!plan->kind) return fail(RX_ERR_INVALID, "plan has not been built");
  *bytes = plan->ws_bytes;
  return RX_OK;
}

rx_status rx_plan_upload(const rx_plan* plan, void* workspace, size_t workspace_bytes,
                         rx_stream_t stream) {
  if (!plan || !plan->kind) return fail(RX_ERR_INVALID, "plan has not been built");
  if (!workspace) return fail(RX_ERR_WORKSPACE, "workspace is NULL");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(RX_ERR_INVALID, "workspace must be 256-byte aligned");
  if (workspace_bytes < plan->ws_bytes)
    return fail(RX_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed", workspace_bytes,
                plan->ws_bytes);
  // the previous upload's copy out of the staging buffer must be done before it is overwritten
  cudaError_t e = cudaSuccess;
  if (plan->staged_pending) {
    e = cudaEventSynchronize(plan->staged);
    if (e) return cuda_fail(e, "plan upload");
    plan->staged_pending = false;
  }
  const size_t n = plan->blob.size();
  if (plan->pinned_bytes < n) {
    if (plan->pinned) cudaFreeHost(plan->pinned);
    plan->pinned = nullptr;
    plan->pinned_bytes = 0;
    e = cudaHostAlloc(&plan->pinned, n, cudaHostAllocPortable);
    if (e) return cuda_fail(e, "plan upload: pinned staging buffer");
    plan->pinned_bytes = n;
  }
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e) return cuda_fail(e, "plan upload");
  if (plan->staged && plan->staged_dev != dev) {  // events belong to one device
    cudaEventDestroy(plan->staged);
    plan->staged = nullptr;
  }
  if (!plan->staged) {
    e = cudaEventCreateWithFlags(&plan->staged, cudaEventDisableTiming);
    if (e) return cuda_fail(e, "plan upload");
    plan->staged_dev = dev;
  }
  std::memcpy(plan->pinned, plan->blob.data(), n);
  e = cudaMemcpyAsync(workspace, plan->pinned, n, cudaMemcpyHostToDevice, (cudaStream_t)stream);
  if (e) return cuda_fail(e, "plan upload");
  e = cudaEventRecord(plan->staged, (cudaStream_t)stream);
  if (e) return cuda_fail(e, "plan upload");
  plan->staged_pending = true;
  return RX_OK;
}

// ---------------------------------------------------------------------------------------------
// Validates a group forest: parents listed first, a prefix at least as long as its parent's.
rx_status check_tree(int32_t num_groups, const int32_t* group_prefix_len,
                     const int32_t* group_parent) {
  for (int g = 0; g < num_groups; ++g) {
    if (group_prefix_len[g] < 0) return fail(RX_ERR_RANGE, "group_prefix_len[%d] < 0", g);
    if (!group_parent) continue;
    const int pa = group_parent[g];
    if (pa < -1 || pa >= g)
      return fail(RX_ERR_RANGE, "group_parent[%d] = %d: parents must be listed first", g, pa);
    if (pa >= 0 && group_prefix_len[pa] > group_prefix_len[g])
      return fail(RX_ERR_RANGE, "group_prefix_len[%d] < its parent's", g);
  }
  return RX_OK;
}

// Decode planner.  Work units: (group node, member tile, chunk of the node's own keys) -- a node's
// members are all requests of its subtree -- and (request, chunk of its keys past its deepest
// group's prefix); each unit becomes one item per KV-head block.  Chunk
// lengths aim at about three items' worth of bytes per SM so a longest-first launch order
// balances; partial rows are allocated per unit over all KV heads.
// ---------------------------------------------------------------------------------------------
rx_status rx_decode_plan(rx_plan* plan, const rx_kv_desc* desc, int32_t batch,
                         const int32_t* req_idx, const int32_t* seq_len,
                         const int32_t* group_of_req, int32_t num_groups,
                         const int32_t* group_prefix_len) {
  return rx_decode_plan_tree(plan, desc, batch, req_idx, seq_len, group_of_req, num_groups,
                             group_prefix_len, nullptr);
}

static rx_status decode_plan_tree(rx_plan* plan, const rx_kv_desc* desc, int32_t batch,
                                  const int32_t* req_idx, const int32_t* seq_len,
                                  const int32_t* group_of_req, int32_t num_groups,
                                  const int32_t* group_prefix_len, const int32_t* group_parent);

rx_status rx_decode_plan_tree(rx_plan* plan, const rx_kv_desc* desc, int32_t batch,
                              const int32_t* req_idx, const int32_t* seq_len,
                              const int32_t* group_of_req, int32_t num_groups,
                              const int32_t* group_prefix_len, const int32_t* group_parent) {
  return no_throw([&] {
    return decode_plan_tree(plan, desc, batch, req_idx, seq_len, group_of_req, num_groups,
                            group_prefix_len, group_parent);
  });
}

static rx_status decode_plan_tree(rx_plan* plan, const rx_kv_desc* desc, int32_t batch,
                                  const int32_t* req_idx, const int32_t* seq_len,
                                  const int32_t* group_of_req, int32_t num_groups,
                                  const int32_t* group_prefix_len, const int32_t* group_parent) {
  if (!plan) return fail(RX_ERR_INVALID, "plan is NULL");
  rx_status st = check_desc(desc, true);
  if (st) return st;
  if (batch < 0 || num_groups < 0) return fail(RX_ERR_INVALID, "negative batch or group count");
  if (batch > 0 && (!req_idx || !seq_len)) return fail(RX_ERR_INVALID, "NULL length array");
  if (num_groups > 0 && !group_prefix_len) return fail(RX_ERR_INVALID, "group_prefix_len NULL");
  st = check_tree(num_groups, group_prefix_len, group_parent);
  if (st) return st;
  const int hkv = desc->num_kv_heads, gq = desc->num_q_heads / hkv;
  auto parent = [&](int g) { return group_parent ? group_parent[g] : -1; };
  std::vector<int> grp(batch, -1);
  for (int b = 0; b < batch; ++b) {
    if (req_idx[b] < 0 || req_idx[b] >= desc->req_to_token_rows)
      return fail(RX_ERR_RANGE, "req_idx[%d] = %d outside the table", b, req_idx[b]);
    if (seq_len[b] < 1 || seq_len[b] > desc->req_to_token_stride)
      return fail(RX_ERR_RANGE, "seq_len[%d] = %d outside [1, stride]", b, seq_len[b]);
    if (group_of_req) {
      const int g = group_of_req[b];
      if (g < -1 || g >= num_groups) return fail(RX_ERR_RANGE, "group_of_req[%d] = %d", b, g);
      if (g >= 0) {
        if (group_prefix_len[g] < 0 || group_prefix_len[g] > seq_len[b])
          return fail(RX_ERR_RANGE, "group_prefix_len[%d] = %d exceeds seq_len of member %d", g,
                      group_prefix_len[g], b);
        grp[b] = g;
      }
    }
  }
  // a node's members: every request of its subtree (batch order)
  std::vector<std::vector<int>> members(num_groups);
  for (int b = 0; b < batch; ++b)
    for (int g = grp[b]; g >= 0; g = parent(g)) members[g].push_back(b);
  auto node_lo = [&](int g) { return parent(g) >= 0 ? group_prefix_len[parent(g)] : 0; };

  struct Unit {
    int kind, kv_row, k_begin, k_end, row_begin, n_tok;
    int64_t part;
  };
  std::vector<Unit> units;
  std::vector<int32_t> rows;
  std::vector<std::vector<DecMergeRef>> refs(batch);
  int64_t npart = 0;
  // 8-bit pools have kinds, head blocks and splits of their own (see kQ8WarpKeys): kind 2 is wide
  const bool q8 = plan->kv_next == RX_KV_E4M3;
  const int q8_hb = 1 << q8_head_block_log2(hkv), q8_whb = std::max(1, q8_hb / 2);
  const int max_tok = (q8 ? kQ8MaxWideRows : 64) / gq;
  auto kind_of_rows = [&](int r) {
    return q8 ? (r > kQ8MaxRows ? 2 : r > 8) : r <= 16 ? 0 : (r <= 32 ? 1 : 2);
  };
  // by kind: heads a block, partial results a unit, keys of a pipeline stage (looked up per item and
  // per comparison of the sorts below)
  const int hbs[3] = {q8 ? q8_hb : 8, q8 ? q8_hb : 4, q8 ? q8_whb : 2};
  const int splits[3] = {q8 ? 8 / hbs[0] : 1, q8 ? 8 / hbs[1] : 1, q8 ? 4 / hbs[2] : 1};
  const int stages_keys[3] = {q8 ? splits[0] * kQ8WarpKeys : kDecRows / hbs[0],
                              q8 ? splits[1] * kQ8WarpKeys : kDecRows / hbs[1],
                              q8 ? splits[2] * kQ8WarpKeys : kDecRows / hbs[2]};
  auto hb_of = [&](int kind) { return hbs[kind]; };
  auto splits_of = [&](int kind) { return splits[kind]; };
  auto stage_keys = [&](int kind) { return stages_keys[kind]; };

  // The units' keys: a shared prefix for a tile of its members, then each request's own.
  struct Span {
    int kind, n_rows, len;
  };
  std::vector<Span> spans;  // 8-bit pool: for the choice of the items' length
  // bytes of K+V per key for one KV head
  const double key_bytes = 2.0 * kHeadDim * 2;
  double total = 0;
  for (int g = 0; g < num_groups; ++g)
    if (!members[g].empty() && group_prefix_len[g] > node_lo(g)) {
      const int len = group_prefix_len[g] - node_lo(g);
      total += (double)len * hkv * key_bytes * ((members[g].size() + max_tok - 1) / max_tok);
      const bool tiles = (int64_t)members[g].size() * gq >= kQ8TileRows;  // not items of these forms
      for (size_t t0 = 0; q8 && !tiles && t0 < members[g].size(); t0 += max_tok) {
        const int r = (int)std::min<size_t>(max_tok, members[g].size() - t0) * gq;
        spans.push_back({kind_of_rows(r), r, len});
      }
    }
  for (int b = 0; b < batch; ++b) {
    const int len = seq_len[b] - (grp[b] >= 0 ? group_prefix_len[grp[b]] : 0);
    total += (double)len * hkv * key_bytes;
    if (q8 && len > 0) spans.push_back({0, gq, len});
  }
  // bytes of K/V per mma.sync item: about three items per SM, but no item under 1 MiB (smaller
  // ones spend more on their own start and partial write-out than on the read)
  const int sms = device_sms();
  const double target = std::min(4.0 * 1048576, std::max(1048576.0, total / (3.0 * sms)));

  // 8-bit pool: stages per item, for the narrow and the wide items.  An item costs, beyond its
  // stages, its start (1.5 stages) and its partial rows (written, read by the merge, and what that
  // disturbs: 3 passes), in stages of copy time.  Shorter items even the lists out (and fill the GPU
  // when there is little work), longer ones pay less per item: of a few lengths the one with the
  // shortest longest list is taken, the longest of equals.  The two figures were fitted over a
  // hundred random batches: a start of 0.5 stages and 2 passes read 16 x 16 requests on 2,000-token
  // prefixes in 153 us instead of 155, but 126 requests of up to 542 tokens in 33.8 instead of 26.3.
  int q8_stages[2] = {1, 1};
  int64_t q8_longest[2] = {0, 0};
  auto item_cost = [&](int kind, int n_rows, int stages) {  // in hundredths of a stage
    const int hb = hb_of(kind), rows_stage = kind == 2 ? 128 : 256;
    return 100ll * stages + 150 + 100ll * 3 * n_rows * hb * kHeadDim * 4 / (rows_stage * 264);
  };
  for (int wide = 0; q8 && wide < 2; ++wide) {
    int64_t stages = 0;
    auto of = [&](const Span& u) { return (u.kind == 2) == (wide == 1); };
    for (const Span& u : spans)
      if (of(u))
        stages += (int64_t)((u.len + stage_keys(u.kind) - 1) / stage_keys(u.kind)) *
                  (hkv / hb_of(u.kind));
    int64_t best = INT64_MAX;
    for (int per : {1, 2, 3, 4, 6, 8, 12}) {  // items per SM
      const int64_t n = std::max<int64_t>(1, (stages + (int64_t)per * sms - 1) / ((int64_t)per * sms));
      if (per > 1 && n < 2) break;
      std::vector<int64_t> costs;
      int64_t sum = 0;
      for (const Span& u : spans) {
        if (!of(u)) continue;
        const int64_t st = (u.len + stage_keys(u.kind) - 1) / stage_keys(u.kind);
        const int64_t parts = (st + n - 1) / n;
        for (int64_t i = 0; i < parts; ++i) {
          const int64_t c = item_cost(u.kind, u.n_rows, (int)((st + parts - 1) / parts));
          for (int h = 0; h < hkv / hb_of(u.kind); ++h) costs.push_back(c);
          sum += c * (hkv / hb_of(u.kind));
        }
      }
      int64_t longest = sum / sms;
      if (costs.size() <= (size_t)16 * sms) {  // (more items even out by themselves)
        std::sort(costs.begin(), costs.end(), std::greater<int64_t>());
        std::priority_queue<int64_t, std::vector<int64_t>, std::greater<int64_t>> ends;
        for (int k = 0; k < sms; ++k) ends.push(0);
        for (int64_t c : costs) {
          const int64_t e = ends.top() + c;
          ends.pop();
          ends.push(e);
          longest = std::max(longest, e);
        }
      }
      if (longest < best) {
        best = longest;
        q8_longest[wide] = longest;
        q8_stages[wide] = (int)std::min<int64_t>(n, 1 << 16);
      }
    }
  }
  auto chunks = [&](int len, int kind, std::vector<std::pair<int, int>>& out) {
    const int hb = std::min(hb_of(kind), hkv);
    const int nk = stage_keys(kind);
    int max_keys = (int)(target / (hb * key_bytes));
    max_keys = q8 ? q8_stages[kind == 2] * nk
                  : std::max(64, std::min(kDecMaxKeysPerItem, max_keys));
    const int n = (len + max_keys - 1) / max_keys;
    int c = (len + n - 1) / n;
    c = (c + nk - 1) / nk * nk;
    if (!q8) c = std::min(c, kDecMaxKeysPerItem);
    out.clear();
    for (int k = 0; k < len; k += c) out.push_back({k, std::min(len, k + c)});
  };
  std::vector<std::pair<int, int>> ch;
  // The references of one request to a unit of `len` keys: one partial per split that has keys.
  auto refer = [&](int b, int kind, int64_t part, int len, int n_rows, int row) {
    refs[b].push_back({(int32_t)part, n_rows, row, 0});
    for (int k = 1; k < splits_of(kind) && k * kQ8WarpKeys < len; ++k)
      refs[b].push_back({(int32_t)(part + (int64_t)k * hkv * n_rows), n_rows, row, 0});
  };

  // Shared-prefix units whose stacked query rows reach 32 per KV head run on the tensor-core
  // attention kernel (128 / gq requests per tile, two tiles per item, one KV head per item, about
  // 2048-key chunks); the rest on the mma.sync kernel above.
  const bool tc_ok = (int64_t)desc->pool_size * hkv < (int64_t)INT32_MAX;
  const int tc_tok = 128 / gq;
  std::vector<ExtItem> xitems;
  std::vector<ExtRow> xrows;
  std::vector<ExtSeg> xsegs;
  std::vector<Q8Tile> tiles8;  // 8-bit pool: the tiles of their keys, in the segments' order
  int64_t key_reads = 0;
  // The tile items' longest list when list-scheduled, costliest first, with chunks of `keys` keys, in
  // the units of attn_cost.
  auto tiles_end = [&](int keys) {
    std::vector<int64_t> costs;
    for (int g = 0; g < num_groups; ++g) {
      const int64_t tiles = ((int64_t)members[g].size() + tc_tok - 1) / tc_tok;
      const int len = group_prefix_len[g] - node_lo(g);
      if ((int64_t)members[g].size() * gq < kQ8TileRows || len <= 0) continue;
      const int n = (len + keys - 1) / keys;
      const int64_t steps = attn_steps((len + n - 1) / n);
      for (int64_t i = 0; i < tiles; i += 2)
        costs.insert(costs.end(), (size_t)n * hkv,
                     steps * (i + 1 < tiles ? 14 : 11) + kItemCost + kCutCost);
    }
    std::sort(costs.begin(), costs.end(), std::greater<int64_t>());
    std::priority_queue<int64_t, std::vector<int64_t>, std::greater<int64_t>> ends;
    for (int k = 0; k < sms; ++k) ends.push(0);
    int64_t longest = 0;
    for (int64_t c : costs) {
      const int64_t e = ends.top() + c;
      ends.pop();
      ends.push(e);
      longest = std::max(longest, e);
    }
    return longest;
  };
  // 8-bit pool: the chunks' length by the earliest end (seven groups of 152 rows on 2,309 keys, 40/5
  // heads, 35 items of 2,048: 89 us, 69 in shorter chunks; over 40 random batches with such groups 20 %
  // less on the average, none slower)
  int tile_keys = 2048;
  if (q8) {
    int64_t best = tiles_end(tile_keys);
    for (int keys : {1536, 1024, 768, 512, 384, 256}) {
      const int64_t end = tiles_end(keys);
      if (end < best) {
        best = end;
        tile_keys = keys;
      }
    }
  }
  for (int g = 0; g < num_groups; ++g) {
    const int lo = node_lo(g), hi = group_prefix_len[g];
    const auto& mem = members[g];
    if (mem.empty() || hi <= lo) continue;
    const int64_t tc_rows = (int64_t)mem.size() * gq;
    if (q8 ? tc_rows >= kQ8TileRows : tc_ok && tc_rows >= 32) {
      struct XTile {
        int row_begin, n_tok, t0;
      };
      std::vector<XTile> tiles;
      for (size_t t0 = 0; t0 < mem.size(); t0 += tc_tok) {
        const int n_tok = (int)std::min<size_t>(tc_tok, mem.size() - t0);
        tiles.push_back({(int)xrows.size(), n_tok, (int)t0});
        for (int i = 0; i < n_tok; ++i)
          xrows.push_back({mem[t0 + i], INT32_MAX, mem[t0 + i], 0});
      }
      const int n_ch = q8 ? (hi - lo + tile_keys - 1) / tile_keys
                          : std::max(1, (hi - lo + 1024) / 2048);
      const int clen = ((hi - lo + n_ch - 1) / n_ch + 63) / 64 * 64;
      for (int c0 = lo; c0 < hi; c0 += clen) {
        const int c1 = std::min(hi, c0 + clen);
        const int seg = (int)xsegs.size();
        xsegs.push_back({q8 ? (int32_t)tiles8.size() : req_idx[mem[0]], c0, c1, -1});
        for (int k = c0; q8 && k < c1; k += kAttnKeys)
          tiles8.push_back({req_idx[mem[0]], k, std::min(kAttnKeys, c1 - k), 0});
        std::vector<int64_t> part(tiles.size());
        for (size_t k = 0; k < tiles.size(); ++k) {
          part[k] = npart;
          npart += (int64_t)hkv * tiles[k].n_tok * gq;
          for (int i = 0; i < tiles[k].n_tok; ++i)
            refs[mem[tiles[k].t0 + i]].push_back(
                {(int32_t)part[k], tiles[k].n_tok * gq, i * gq, 0});
        }
        for (size_t k = 0; k < tiles.size(); k += 2) {
          const bool pair = k + 1 < tiles.size();
          for (int h = 0; h < hkv; ++h) {
            ExtItem it;
            it.row_begin[0] = tiles[k].row_begin;
            it.n_tok[0] = tiles[k].n_tok;
            it.row_begin[1] = pair ? tiles[k + 1].row_begin : 0;
            it.n_tok[1] = pair ? tiles[k + 1].n_tok : 0;
            it.seg_begin = seg;
            it.n_seg = 1;
            it.kv_head = h;
            it.n_steps = attn_steps(c1 - c0);
            it.part[0] = (int32_t)(part[k] + (int64_t)h * tiles[k].n_tok * gq);
            it.part[1] = pair ? (int32_t)(part[k + 1] + (int64_t)h * tiles[k + 1].n_tok * gq) : 0;
            xitems.push_back(it);
          }
          if (!q8 || k == 0) key_reads += (int64_t)(c1 - c0) * hkv;  // (expanded once)
        }
      }
      continue;
    }
    for (size_t t0 = 0; t0 < mem.size(); t0 += max_tok) {
      const int n_tok = (int)std::min<size_t>(max_tok, mem.size() - t0);
      const int kind = kind_of_rows(n_tok * gq);
      const int row_begin = (int)rows.size();
      for (int i = 0; i < n_tok; ++i) rows.push_back(mem[t0 + i]);
      chunks(hi - lo, kind, ch);
      for (auto& c : ch) {
        const int64_t part = npart;
        npart += (int64_t)splits_of(kind) * hkv * n_tok * gq;
        units.push_back(
            {kind, req_idx[mem[t0]], lo + c.first, lo + c.second, row_begin, n_tok, part});
        for (int i = 0; i < n_tok; ++i)
          refer(mem[t0 + i], kind, part, c.second - c.first, n_tok * gq, i * gq);
      }
    }
  }
  for (int b = 0; b < batch; ++b) {
    const int k0 = grp[b] >= 0 ? group_prefix_len[grp[b]] : 0;
    if (seq_len[b] <= k0) continue;
    const int row_begin = (int)rows.size();
    rows.push_back(b);
    chunks(seq_len[b] - k0, 0, ch);
    for (auto& c : ch) {
      const int64_t part = npart;
      npart += (int64_t)splits_of(0) * hkv * gq;
      units.push_back({0, req_idx[b], k0 + c.first, k0 + c.second, row_begin, 1, part});
      refer(b, 0, part, c.second - c.first, gq, 0);
    }
  }
  if (npart > (int64_t)INT32_MAX || (int64_t)tiles8.size() * hkv > (int64_t)INT32_MAX)
    return fail(RX_ERR_RANGE, "plan too large");

  std::vector<DecItem> items, wide;
  for (const Unit& u : units) {
    const int hb = hb_of(u.kind);
    for (int h = 0; h * hb < hkv; ++h)
      (q8 && u.kind == 2 ? wide : items)
          .push_back({u.kind, h, u.kv_row, u.k_begin, u.k_end, u.row_begin, u.n_tok,
                      (int32_t)u.part});
    key_reads += (int64_t)(u.k_end - u.k_begin) * hkv;
  }
  auto cost = [&](const DecItem& it) {  // 8-bit pool
    return (double)item_cost(it.kind, it.n_tok * gq,
                             (it.k_end - it.k_begin + stage_keys(it.kind) - 1) /
                                 stage_keys(it.kind));
  };
  auto by_cost = [&](const DecItem& a, const DecItem& b) { return cost(a) > cost(b); };
  // bf16 pool: by keys times heads
  auto by_rows = [&](const DecItem& a, const DecItem& b) {
    return (int64_t)(a.k_end - a.k_begin) * std::min(hbs[a.kind], hkv) >
           (int64_t)(b.k_end - b.k_begin) * std::min(hbs[b.kind], hkv);
  };
  if (q8) {
    std::stable_sort(items.begin(), items.end(), by_cost);
    std::stable_sort(wide.begin(), wide.end(), by_cost);
  } else {
    std::stable_sort(items.begin(), items.end(), by_rows);
  }

  // 8-bit pool: one list per CTA, each item (costliest first) to the list that is shortest so
  // far; the table is stored list by list
  auto deal = [&](std::vector<DecItem>& all, std::vector<int32_t>& begin) {
    if (all.empty()) return;
    const int32_t G = (int32_t)std::min<int64_t>(sms, (int64_t)all.size());
    using Slot = std::pair<double, int32_t>;  // (length of the list, CTA)
    std::priority_queue<Slot, std::vector<Slot>, std::greater<Slot>> free_at;
    for (int32_t k = 0; k < G; ++k) free_at.push({0., k});
    std::vector<std::vector<DecItem>> lists(G);
    for (const DecItem& it : all) {
      const Slot s = free_at.top();
      free_at.pop();
      lists[s.second].push_back(it);
      free_at.push({s.first + cost(it), s.second});
    }
    all.clear();
    begin.push_back(0);
    for (const auto& l : lists) {
      all.insert(all.end(), l.begin(), l.end());
      begin.push_back((int32_t)all.size());
    }
  };
  std::vector<int32_t> cta_begin, wide_begin;
  if (q8) {
    deal(items, cta_begin);
    deal(wide, wide_begin);
  }

  std::stable_sort(xitems.begin(), xitems.end(), [](const ExtItem& a, const ExtItem& b) {
    return attn_cost(a) > attn_cost(b);
  });

  std::vector<int32_t> midx(batch + 1, 0);
  std::vector<DecMergeRef> mref;
  for (int b = 0; b < batch; ++b) {
    midx[b] = (int32_t)mref.size();
    mref.insert(mref.end(), refs[b].begin(), refs[b].end());
  }
  midx[batch] = (int32_t)mref.size();
  int32_t max_refs = 0;
  for (int b = 0; b < batch; ++b) max_refs = std::max(max_refs, midx[b + 1] - midx[b]);

  PlanHeader h;
  std::memset(&h, 0, sizeof h);
  h.magic = kPlanMagic;
  h.kind = 2;
  h.kv_type = plan->kv_next;
  h.n_items = (int32_t)items.size();
  h.num_q_heads = desc->num_q_heads;
  h.num_kv_heads = hkv;
  h.batch = batch;
  h.n_rows = (int32_t)rows.size();
  size_t off = align256(sizeof(PlanHeader));
  h.off_items = off; off = align256(off + items.size() * sizeof(DecItem));
  h.off_rows = off; off = align256(off + rows.size() * 4);
  h.off_segs = off;
  h.off_merge_idx = off; off = align256(off + midx.size() * 4);
  h.off_merge = off; off = align256(off + mref.size() * sizeof(DecMergeRef));
  h.off_xitems = off; off = align256(off + xitems.size() * sizeof(ExtItem));
  h.off_xrows = off; off = align256(off + xrows.size() * sizeof(ExtRow));
  h.off_xsegs = off; off = align256(off + xsegs.size() * sizeof(ExtSeg));
  h.n_xitems = (int32_t)xitems.size();
  h.off_cta = off; off = align256(off + cta_begin.size() * sizeof(int32_t));
  h.n_ctas = cta_begin.empty() ? 0 : (int32_t)cta_begin.size() - 1;
  h.off_q8_tiles = off; off = align256(off + tiles8.size() * sizeof(Q8Tile));
  h.n_q8_tiles = (int32_t)tiles8.size();
  h.off_wide = off; off = align256(off + wide.size() * sizeof(DecItem));
  h.off_wide_cta = off; off = align256(off + wide_begin.size() * sizeof(int32_t));
  h.n_wide = (int32_t)wide.size();
  h.n_wide_ctas = wide_begin.empty() ? 0 : (int32_t)wide_begin.size() - 1;
  h.max_refs = max_refs;
  h.n_sms = sms;
  const size_t tables = off;
  h.off_part_o = off; off = align256(off + (size_t)npart * kHeadDim * 4);
  h.off_part_lse = off; off = align256(off + (size_t)npart * 4);
  h.n_part_rows = npart;
  h.off_q8_stage = off; off = align256(off + tiles8.size() * (size_t)hkv * kQ8BlockBytes);
  h.total_bytes = off;
  plan->blob.assign(tables, 0);
  std::memcpy(plan->blob.data(), &h, sizeof h);
  put(plan->blob, h.off_items, items);
  put(plan->blob, h.off_rows, rows);
  put(plan->blob, h.off_merge_idx, midx);
  put(plan->blob, h.off_merge, mref);
  put(plan->blob, h.off_xitems, xitems);
  put(plan->blob, h.off_xrows, xrows);
  put(plan->blob, h.off_xsegs, xsegs);
  put(plan->blob, h.off_cta, cta_begin);
  put(plan->blob, h.off_q8_tiles, tiles8);
  put(plan->blob, h.off_wide, wide);
  put(plan->blob, h.off_wide_cta, wide_begin);
  // a narrow stage takes 1.7 us (67 KB at the rate of an SM), a wide one 2.1 (its arithmetic)
  plan->q8_us = 0.017 * q8_longest[0] + 0.021 * q8_longest[1];
  plan->ws_bytes = off;
  plan->key_reads = key_reads;
  plan->kind = 2;
  remember_desc(plan, desc);
  return RX_OK;
}

rx_status rx_decode_attn(const rx_plan* plan, const rx_kv_desc* desc, const void* k_pool,
                         const void* v_pool, const void* q, void* o, float* lse,
                         void* workspace, size_t workspace_bytes, rx_stream_t stream) {
  rx_status st = check_plan_use(plan, 2, RX_KV_BF16, desc, k_pool, v_pool, q, o, lse, workspace,
                                workspace_bytes);
  if (st) return st;
  const PlanHeader h = plan->hdr();
  AuxStream aux;
  st = plan_aux_stream(plan, &aux);
  if (st) return st;
  const int e = launch_decode(desc, &h, k_pool, v_pool, q, o, lse, workspace, stream, &aux);
  return e ? cuda_fail(e, "decode launch") : RX_OK;
}

rx_status rx_decode_attn_q8(const rx_plan* plan, const rx_kv_desc* desc, const rx_kv_q8* kv,
                            const void* q, void* o, float* lse, void* workspace,
                            size_t workspace_bytes, rx_stream_t stream) {
  const rx_status st =
      check_plan_use_q8(plan, 2, desc, kv, q, o, lse, workspace, workspace_bytes);
  if (st) return st;
  const PlanHeader h = plan->hdr();
  if (!has_rows(h)) return RX_OK;
  const int e = launch_decode_q8(desc, &h, kv, q, o, lse, workspace, stream);
  return e ? cuda_fail(e, "decode launch") : RX_OK;
}

// ---------------------------------------------------------------------------------------------
// Extend planner.  The new tokens of a group's members are packed, member after member, into
// tiles of 128 / gq tokens (128 query rows per KV head).  A tile's segments: the shared prefix
// (read from the first member's row, visible to all rows) and, per member present, its keys from
// the group prefix up to its last row's causal limit.  Ungrouped requests get tiles of their own.
// One item per (tile, KV head).
// ---------------------------------------------------------------------------------------------
rx_status rx_extend_plan(rx_plan* plan, const rx_kv_desc* desc, int32_t batch,
                         const int32_t* req_idx, const int32_t* prefix_len,
                         const int32_t* extend_len, const int32_t* group_of_req,
                         int32_t num_groups, const int32_t* group_prefix_len) {
  return rx_extend_plan_tree(plan, desc, batch, req_idx, prefix_len, extend_len, group_of_req,
                             num_groups, group_prefix_len, nullptr);
}

static rx_status extend_plan_tree(rx_plan* plan, const rx_kv_desc* desc, int32_t batch,
                                  const int32_t* req_idx, const int32_t* prefix_len,
                                  const int32_t* extend_len, const int32_t* group_of_req,
                                  int32_t num_groups, const int32_t* group_prefix_len,
                                  const int32_t* group_parent);

rx_status rx_extend_plan_tree(rx_plan* plan, const rx_kv_desc* desc, int32_t batch,
                              const int32_t* req_idx, const int32_t* prefix_len,
                              const int32_t* extend_len, const int32_t* group_of_req,
                              int32_t num_groups, const int32_t* group_prefix_len,
                              const int32_t* group_parent) {
  return no_throw([&] {
    return extend_plan_tree(plan, desc, batch, req_idx, prefix_len, extend_len, group_of_req,
                            num_groups, group_prefix_len, group_parent);
  });
}

// 8-bit pool: extends of at most this many new tokens, in all and of a request, are also planned as a
// decode, and the plan with the lower estimate is taken.  The estimates miss by up to a quarter and no
// margin is asked for, so where both are close the slower may win (16 requests of one or two new tokens
// in pairs on 5,715, 48/12 heads: 36.8 us, expanded and on tiles 172; 10 of up to 17 on 715, 12/12
// heads: 17.0 and 14.8, on tiles).
constexpr int64_t kFewTokens = 2048;
constexpr int32_t kFewPerRequest = 32;
// A step's keys in the expansion (read, and written), and what an extend's launches take beyond a
// decode's.
constexpr double kQ8ExpandBytes = kAttnKeys * 264. + kQ8BlockBytes, kQ8ExtendUs = 1.;

// The decode plan of an extend's new tokens: each a request of its own with the keys up to itself; a
// request's cached keys are a node that its tokens share.
static rx_status few_tokens_plan(rx_plan* plan, const rx_kv_desc* desc, int32_t batch,
                                 const int32_t* req_idx, const int32_t* prefix_len,
                                 const int32_t* extend_len, const std::vector<int>& grp,
                                 int32_t num_groups, const int32_t* group_prefix_len,
                                 const int32_t* group_parent) {
  std::vector<int32_t> row, len, node, node_len, parent;
  for (int32_t g = 0; g < num_groups; ++g) {
    node_len.push_back(group_prefix_len[g]);
    parent.push_back(group_parent ? group_parent[g] : -1);
  }
  for (int32_t b = 0; b < batch; ++b) {
    int32_t at = grp[b];
    if (extend_len[b] > 1 && prefix_len[b] > (at >= 0 ? node_len[at] : 0)) {
      node_len.push_back(prefix_len[b]);
      parent.push_back(at);
      at = (int32_t)node_len.size() - 1;
    }
    for (int32_t i = 0; i < extend_len[b]; ++i) {
      row.push_back(req_idx[b]);
      len.push_back(prefix_len[b] + i + 1);
      node.push_back(at);
    }
  }
  return decode_plan_tree(plan, desc, (int32_t)row.size(), row.data(), len.data(), node.data(),
                          (int32_t)node_len.size(), node_len.data(), parent.data());
}

static rx_status extend_plan_tree(rx_plan* plan, const rx_kv_desc* desc, int32_t batch,
                                  const int32_t* req_idx, const int32_t* prefix_len,
                                  const int32_t* extend_len, const int32_t* group_of_req,
                                  int32_t num_groups, const int32_t* group_prefix_len,
                                  const int32_t* group_parent) {
  if (!plan) return fail(RX_ERR_INVALID, "plan is NULL");
  rx_status st = check_desc(desc, true);
  if (st) return st;
  if (batch < 0 || num_groups < 0) return fail(RX_ERR_INVALID, "negative batch or group count");
  if (batch > 0 && (!req_idx || !prefix_len || !extend_len))
    return fail(RX_ERR_INVALID, "NULL length array");
  if (num_groups > 0 && !group_prefix_len) return fail(RX_ERR_INVALID, "group_prefix_len NULL");
  st = check_tree(num_groups, group_prefix_len, group_parent);
  if (st) return st;
  if (plan->kv_next == RX_KV_E4M3 && plan->ext_kernel == RX_EXTEND_PAIR)
    return fail(RX_ERR_UNSUPPORTED, "the SM-pair extend kernel reads bf16 pools only");
  const int hkv = desc->num_kv_heads, gq = desc->num_q_heads / hkv;
  std::vector<int64_t> cu(batch + 1, 0);
  std::vector<int> grp(batch, -1);
  for (int b = 0; b < batch; ++b) {
    if (req_idx[b] < 0 || req_idx[b] >= desc->req_to_token_rows)
      return fail(RX_ERR_RANGE, "req_idx[%d] = %d outside the table", b, req_idx[b]);
    if (prefix_len[b] < 0 || extend_len[b] < 0)
      return fail(RX_ERR_INVALID, "negative length for request %d", b);
    if ((int64_t)prefix_len[b] + extend_len[b] > desc->req_to_token_stride)
      return fail(RX_ERR_RANGE, "prefix_len + extend_len of request %d exceeds the stride", b);
    cu[b + 1] = cu[b] + extend_len[b];
    if (group_of_req) {
      const int g = group_of_req[b];
      if (g < -1 || g >= num_groups) return fail(RX_ERR_RANGE, "group_of_req[%d] = %d", b, g);
      if (g >= 0) {
        if (group_prefix_len[g] < 0 || group_prefix_len[g] > prefix_len[b])
          return fail(RX_ERR_RANGE, "group_prefix_len[%d] = %d exceeds prefix_len of member %d",
                      g, group_prefix_len[g], b);
        grp[b] = g;
      }
    }
  }
  if (cu[batch] > (int64_t)INT32_MAX) return fail(RX_ERR_RANGE, "sum of extend_len >= 2^31");
  const int tile_tok = 128 / gq;

  std::vector<ExtRow> rows;
  std::vector<ExtSeg> segs;
  struct Tile {
    int row_begin, n_tok;
    std::vector<ExtSeg> segs;  // shared prefix (owner -1) first, then one per member present
    double cost;
  };
  // A unit is a group (all its tiles read the same prefix KV) or a lone request.
  struct Unit {
    std::vector<Tile> tiles;
    double cost = 0;
  };
  std::vector<Unit> units;

  auto emit_unit = [&](const std::vector<int>& reqs, int gp) {
    Unit un;
    const int first_row = (int)rows.size();
    for (int r : reqs)
      for (int i = 0; i < extend_len[r]; ++i)
        rows.push_back({(int32_t)(cu[r] + i), prefix_len[r] + i + 1, r, 0});
    const int n = (int)rows.size() - first_row;
    for (int t0 = 0; t0 < n; t0 += tile_tok) {
      const int nt = std::min(tile_tok, n - t0);
      Tile tl{first_row + t0, nt, {}, 0.0};
      if (gp > 0) {
        tl.segs.push_back({req_idx[reqs[0]], 0, gp, -1});
        tl.cost += (double)gp;
      }
      int i = 0;
      while (i < nt) {
        const int owner = rows[first_row + t0 + i].owner;
        int j = i;
        while (j + 1 < nt && rows[first_row + t0 + j + 1].owner == owner) ++j;
        const int kend = rows[first_row + t0 + j].kmax;  // last row's causal limit
        if (kend > gp) {
          tl.segs.push_back({req_idx[owner], gp, kend, owner});
          tl.cost += (double)(kend - gp);
        }
        i = j + 1;
      }
      un.cost += tl.cost;
      un.tiles.push_back(std::move(tl));
    }
    std::stable_sort(un.tiles.begin(), un.tiles.end(),
                     [](const Tile& a, const Tile& b) { return a.cost > b.cost; });
    units.push_back(std::move(un));
  };

  // A request's new rows go with the deepest group on its path that holds at least two requests
  // with new tokens (rows that share the most keys share tiles); the tile's shared segment is
  // that group's whole prefix, which is contiguous in every member's row.
  std::vector<int> with_new(num_groups, 0);
  for (int b = 0; b < batch; ++b)
    if (extend_len[b] > 0)
      for (int g = grp[b]; g >= 0; g = group_parent ? group_parent[g] : -1) ++with_new[g];
  std::vector<std::vector<int>> members(num_groups);
  for (int b = 0; b < batch; ++b) {
    if (extend_len[b] <= 0 || grp[b] < 0) continue;
    int g = grp[b];
    while (g >= 0 && with_new[g] < 2) g = group_parent ? group_parent[g] : -1;
    if (g >= 0)
      members[g].push_back(b);
    else
      grp[b] = -1;  // alone on its path: a unit of its own below
  }
  for (int g = 0; g < num_groups; ++g) {
    if (members[g].empty()) continue;
    if (group_prefix_len[g] > 0) {
      emit_unit(members[g], group_prefix_len[g]);
    } else {
      for (int b : members[g]) emit_unit(std::vector<int>{b}, 0);
    }
  }
  for (int b = 0; b < batch; ++b)
    if (grp[b] < 0 && extend_len[b] > 0) emit_unit(std::vector<int>{b}, 0);

  // 8-bit pool: each distinct segment (table row, first key) gets tiles of kAttnKeys keys, as many
  // as its longest use needs; the segments of the items then refer to their first tile.
  const bool q8 = plan->kv_next == RX_KV_E4M3;
  std::vector<Q8Tile> tiles8;
  std::unordered_map<int64_t, std::pair<int32_t, int32_t>> stage;  // -> (longest end, first tile)
  auto stage_of = [&](const ExtSeg& sg) -> std::pair<int32_t, int32_t>& {
    return stage[(int64_t)sg.kv_row << 32 | (uint32_t)sg.k_begin];
  };
  if (q8) {
    for (const Unit& un : units)
      for (const Tile& tl : un.tiles)
        for (const ExtSeg& sg : tl.segs)
          stage_of(sg) = {std::max(stage_of(sg).first, sg.k_end), -1};
    for (const Unit& un : units)
      for (const Tile& tl : un.tiles)
        for (const ExtSeg& sg : tl.segs) {
          auto& w = stage_of(sg);
          if (w.second >= 0) continue;
          if ((int64_t)tiles8.size() + attn_steps(w.first - sg.k_begin) > (int64_t)INT32_MAX / 2)
            return fail(RX_ERR_RANGE, "plan too large");
          w.second = (int32_t)tiles8.size();
          for (int k = sg.k_begin; k < w.first; k += kAttnKeys)
            tiles8.push_back({sg.kv_row, k, std::min(kAttnKeys, w.first - k), 0});
        }
  }
  // Pair consecutive tiles of a unit (similar cost after the sort) into one item; the pair walks
  // the union of the two segment lists (same owner: the longer range).  An odd last tile is
  // paired with an empty one.
  struct Pair {
    int a, b;  // tile indices, b = -1 for none
    int seg_begin, n_seg;
  };
  std::vector<std::vector<Pair>> pairs(units.size());
  for (size_t k = 0; k < units.size(); ++k) {
    const auto& tiles = units[k].tiles;
    for (size_t i = 0; i < tiles.size(); i += 2) {
      Pair pr{(int)i, i + 1 < tiles.size() ? (int)i + 1 : -1, (int)segs.size(), 0};
      std::vector<ExtSeg> u = tiles[i].segs;
      if (pr.b >= 0)
        for (const ExtSeg& sg : tiles[pr.b].segs) {
          bool merged = false;
          for (ExtSeg& x : u)
            if (x.owner == sg.owner && x.kv_row == sg.kv_row && x.k_begin == sg.k_begin) {
              x.k_end = std::max(x.k_end, sg.k_end);
              merged = true;
              break;
            }
          if (!merged) u.push_back(sg);
        }
      segs.insert(segs.end(), u.begin(), u.end());
      pr.n_seg = (int)u.size();
      pairs[k].push_back(pr);
    }
  }

  // 8-bit pool: when the pairs of tiles would leave SMs without work, the steps of each pair, or of
  // each tile by itself, are split over as many items as there are SMs for; such items leave partial
  // rows, which a merge combines.  (In the units of attn_cost: writing a tile's partial rows costs
  // about a step, the merge about 3 us and its reads.  Pairs pass over the keys half as often, single
  // tiles leave half as many partial rows: 155 new tokens on 8,049 in three groups, 64/16 heads, 96
  // tiles: by tiles 190 us, by pairs 122; 129 on 4,007 in two, 24/3 heads: 29.7 and 33.1.)
  struct Work {
    int32_t row_begin[2], n_tok[2];
    std::vector<ExtSeg> segs;
    int32_t n_steps;
  };
  std::vector<Work> works;  // of the split
  int32_t split_steps = 0;  // a split item's, 0: no split
  if (q8) {
    const int64_t sms = plan_sm_count();
    auto works_of = [&](bool by_pairs) {
      std::vector<Work> all;
      for (size_t k = 0; k < units.size(); ++k) {
        const auto& tiles = units[k].tiles;
        auto add = [&](int a, int b, std::vector<ExtSeg> sg) {
          Work w{{tiles[a].row_begin, b >= 0 ? tiles[b].row_begin : 0},
                 {tiles[a].n_tok, b >= 0 ? tiles[b].n_tok : 0}, std::move(sg), 0};
          for (const ExtSeg& x : w.segs) w.n_steps += attn_steps(x.k_end - x.k_begin);
          all.push_back(std::move(w));
        };
        if (by_pairs)
          for (const Pair& pr : pairs[k])
            add(pr.a, pr.b, {segs.begin() + pr.seg_begin, segs.begin() + pr.seg_begin + pr.n_seg});
        else
          for (size_t i = 0; i < tiles.size(); ++i) add((int)i, -1, tiles[i].segs);
      }
      return all;
    };
    int64_t n_pairs = 0, longest = 0;
    for (const auto& u : pairs) n_pairs += (int64_t)u.size() * hkv;
    if (n_pairs > 0 && n_pairs < sms) {
      int64_t best = INT64_MAX;
      for (int by_pairs = 1; by_pairs >= 0; --by_pairs) {
        std::vector<Work> all = works_of(by_pairs);
        if ((int64_t)all.size() * hkv > sms) continue;
        int64_t total = 0, most = 0;
        for (const Work& w : all) {
          total += (int64_t)w.n_steps * hkv;
          most = std::max<int64_t>(most, w.n_steps);
        }
        if (by_pairs) longest = 14 * most;
        auto count = [&](int64_t steps) {
          int64_t n = 0;
          for (const Work& w : all) n += (w.n_steps + steps - 1) / steps * hkv;
          return n;
        };
        int64_t c = std::max<int64_t>(2, (total + sms - 1) / sms);
        while (c < most && count(c) > sms) ++c;
        int64_t partials = 0;
        for (const Work& w : all)
          partials += (w.n_steps + c - 1) / c * (w.n_tok[0] + w.n_tok[1]) * gq * hkv;
        const int64_t cost =
            (by_pairs ? 14 * c + 28 : 11 * c + 14) + partials / (2 * kMergeRowsPerCost);
        if (c < most && cost < best && cost + 41 < longest) {
          best = cost;
          split_steps = (int32_t)c;
          works = std::move(all);
        }
      }
    }
  }

  // Launch order: largest unit first (longest-processing-time first across units); inside a
  // unit, KV head outer and pairs inner (for the one-SM kernel then sorted, stably, costliest
  // first), so the tiles that read the same prefix K/V run in the same wave and hit in L2.
  std::vector<size_t> order(units.size());
  std::iota(order.begin(), order.end(), 0);
  std::stable_sort(order.begin(), order.end(),
                   [&](size_t a, size_t b) { return units[a].cost > units[b].cost; });
  std::vector<ExtItem> items;
  const bool pair_kernel = plan->ext_kernel == RX_EXTEND_PAIR;
  int64_t key_reads = 0;
  for (size_t k : order)
    for (const Pair& pr : pairs[k])
      for (int i = 0; i < pr.n_seg; ++i)
        key_reads += (int64_t)(segs[pr.seg_begin + i].k_end - segs[pr.seg_begin + i].k_begin) * hkv;
  for (size_t k : order) {
    const size_t unit_first = items.size();
    for (int h = 0; h < hkv; ++h)
      for (const Pair& pr : pairs[k]) {
        const Tile& ta = units[k].tiles[pr.a];
        ExtItem it;
        it.row_begin[0] = ta.row_begin;
        it.n_tok[0] = ta.n_tok;
        it.row_begin[1] = pr.b >= 0 ? units[k].tiles[pr.b].row_begin : 0;
        it.n_tok[1] = pr.b >= 0 ? units[k].tiles[pr.b].n_tok : 0;
        it.seg_begin = pr.seg_begin;
        it.n_seg = pr.n_seg;
        it.kv_head = h;
        it.n_steps = 0;
        for (int i = 0; i < pr.n_seg; ++i) {
          const int64_t n = segs[pr.seg_begin + i].k_end - segs[pr.seg_begin + i].k_begin;
          it.n_steps += pair_kernel ? pair_steps(n) : attn_steps(n);
        }
        items.push_back(it);
      }
    // inside a unit the costliest items first (a long causal tile reads all the keys before it)
    if (!pair_kernel)
      std::stable_sort(items.begin() + unit_first, items.end(),
                       [](const ExtItem& a, const ExtItem& b) {
                         return attn_cost(a) > attn_cost(b);
                       });
  }
  // The items refer to the expanded tiles, or, split, are made anew.
  std::vector<std::vector<DecMergeRef>> refs(split_steps ? cu[batch] : 0);
  int64_t npart = 0;
  if (q8 && !split_steps) {
    for (ExtSeg& sg : segs) sg.kv_row = stage_of(sg).second;
  } else if (q8) {
    items.clear();
    segs.clear();
    for (const Work& w : works) {
      const int32_t parts = (w.n_steps + split_steps - 1) / split_steps;
      const int32_t per = (w.n_steps + parts - 1) / parts;
      size_t at = 0;
      int32_t k0 = w.segs[0].k_begin;
      while (at < w.segs.size()) {
        ExtItem it;
        std::memset(&it, 0, sizeof it);
        it.seg_begin = (int32_t)segs.size();
        for (int32_t left = per; left > 0 && at < w.segs.size();) {
          const ExtSeg& sg = w.segs[at];
          const int32_t n = std::min(left, attn_steps(sg.k_end - k0));
          const int32_t end = std::min(sg.k_end, k0 + n * kAttnKeys);
          segs.push_back({stage_of(sg).second + (k0 - sg.k_begin) / kAttnKeys, k0, end, sg.owner});
          it.n_steps += n;
          left -= n;
          k0 = end;
          if (k0 >= sg.k_end && ++at < w.segs.size()) k0 = w.segs[at].k_begin;
        }
        it.n_seg = (int32_t)segs.size() - it.seg_begin;
        const int64_t first = npart;
        for (int x = 0; x < 2; ++x) {
          it.row_begin[x] = w.row_begin[x];
          it.n_tok[x] = w.n_tok[x];
          // the rows that see one of the item's keys take its partial result
          for (int i = 0; i < w.n_tok[x]; ++i) {
            const ExtRow& row = rows[w.row_begin[x] + i];
            bool sees = false;
            for (int j = 0; j < it.n_seg && !sees; ++j) {
              const ExtSeg& sg = segs[it.seg_begin + j];
              sees = (sg.owner < 0 || sg.owner == row.owner) && sg.k_begin < row.kmax;
            }
            if (sees)
              refs[row.q_row].push_back({(int32_t)npart, w.n_tok[x] * gq, i * gq, 0});
          }
          npart += (int64_t)hkv * w.n_tok[x] * gq;
          if (npart > (int64_t)INT32_MAX) return fail(RX_ERR_RANGE, "plan too large");
        }
        for (int h = 0; h < hkv; ++h) {
          it.kv_head = h;
          it.part[0] = (int32_t)(first + (int64_t)h * w.n_tok[0] * gq);
          it.part[1] = (int32_t)(first + (int64_t)(hkv * w.n_tok[0] + h * w.n_tok[1]) * gq);
          items.push_back(it);
        }
      }
    }
  }
  if (q8) {
    key_reads = 0;  // the pool is read by the expansion only
    for (const Q8Tile& t : tiles8) key_reads += (int64_t)t.n_keys * hkv;
  }
  std::vector<int32_t> midx;
  std::vector<DecMergeRef> mref;
  std::vector<MergeRow> merge_rows;
  int32_t max_refs = 0;
  int64_t ends_at = 0;  // of the longest list, in the units of attn_cost
  if (split_steps) {
    midx.push_back(0);
    for (const auto& r : refs) {
      mref.insert(mref.end(), r.begin(), r.end());
      midx.push_back((int32_t)mref.size());
      max_refs = std::max(max_refs, (int32_t)r.size());
    }
  }
  if (items.size() > (size_t)INT32_MAX) return fail(RX_ERR_RANGE, "plan too large");
  std::vector<int32_t> cta_begin;
  if (pair_kernel) {
    // The pair kernel deals the list to its clusters in rounds (snake order): sorted by falling
    // cost, every cluster gets a similar total.  The sort is by cost classes two steps wide and
    // keeps the planned order (a unit's KV heads and tiles together) inside a class.
    std::stable_sort(items.begin(), items.end(), [](const ExtItem& a, const ExtItem& b) {
      return a.n_steps / kPairCostClass > b.n_steps / kPairCostClass;
    });
  } else if (!items.empty()) {
    // One list per CTA, made by list scheduling in the planned order (largest unit first; in a
    // unit, costliest item first): each item goes to the CTA whose list ends first under
    // the cost model.  A CTA runs its list in order, so items next to each other in the planned
    // order start at about the same time on different SMs -- the tiles of one unit read its
    // prefix and its causal keys while they are in L2 -- and the lists end at about the same
    // time.  The table is stored CTA by CTA.
    // (8-bit pool: a list for every SM, so that cut items can fill those without an item)
    const int32_t G = q8 && !split_steps
                          ? plan_sm_count()
                          : (int32_t)std::min<int64_t>(plan_sm_count(), (int64_t)items.size());
    using Slot = std::pair<int64_t, int32_t>;  // (end of the list, CTA)
    std::priority_queue<Slot, std::vector<Slot>, std::greater<Slot>> free_at;
    for (int32_t k = 0; k < G; ++k) free_at.push({0, k});
    std::vector<std::vector<int32_t>> lists(G);
    auto cost_of = [&](int32_t i) { return attn_cost(items[i]) + kItemCost; };
    for (size_t i = 0; i < items.size(); ++i) {
      const Slot s = free_at.top();
      free_at.pop();
      lists[s.second].push_back((int32_t)i);
      free_at.push({s.first + cost_of((int32_t)i), s.second});
    }
    // The lists' ends are left up to one item apart, and the last units' items are large (a
    // branch's 1,700-key tile, a long causal tile).  Balance them: while it lowers the larger of
    // the two, move from the longest list to the shortest the item whose cost best splits their
    // gap (appended at the end, so the longest list's other items only start earlier).
    std::vector<int64_t> load(G, 0);
    for (int32_t k = 0; k < G; ++k)
      for (int32_t i : lists[k]) load[k] += cost_of(i);
    for (int32_t round = 0; round < 8 * G; ++round) {
      const int32_t hi = (int32_t)(std::max_element(load.begin(), load.end()) - load.begin());
      const int32_t lo = (int32_t)(std::min_element(load.begin(), load.end()) - load.begin());
      const int64_t gap = load[hi] - load[lo];
      int64_t best_gain = 0;
      size_t best = 0;
      for (size_t j = 0; j < lists[hi].size(); ++j) {
        const int64_t c = cost_of(lists[hi][j]);
        const int64_t gain = std::min(c, gap - c);  // the longer list shortens by this much
        if (c < gap && gain > best_gain) {
          best_gain = gain;
          best = j;
        }
      }
      if (best_gain <= 0) break;
      const int32_t i = lists[hi][best];
      lists[hi].erase(lists[hi].begin() + (std::ptrdiff_t)best);
      lists[lo].push_back(i);
      load[hi] -= cost_of(i);
      load[lo] += cost_of(i);
    }
    ends_at = *std::max_element(load.begin(), load.end());
    // 8-bit pool: where the lists end apart all the same (a few items each), those that end late
    // give the last steps of their longest item to those that end early.  Both pieces of such an
    // item leave partial rows for a merge.
    if (q8 && !split_steps) {
      const int64_t before = ends_at;
      int64_t lo = 0;
      for (int64_t x : load) lo += x;
      lo /= G;  // no schedule ends before
      std::vector<Cut> cuts, best_cuts;
      int64_t after = before;
      while (after - lo > 1) {
        const int64_t end = lo + (after - lo) / 2;
        if (cut_lists(items, lists, load, end, cuts)) {
          after = end;
          best_cuts.swap(cuts);
        } else {
          lo = end;
        }
      }
      int64_t cut_rows = 0;
      for (const Cut& c : best_cuts)
        cut_rows += (int64_t)(items[c.item].n_tok[0] + items[c.item].n_tok[1]) * gq;
      if (before - after > kMergeCost + cut_rows / kMergeRowsPerCost &&
          npart + 2 * cut_rows <= (int64_t)INT32_MAX) {
        ends_at = after;
        for (ExtItem& it : items) it.part[0] = it.part[1] = -1;
        midx.push_back(0);
        for (const Cut& c : best_cuts) {
          ExtItem tail = items[c.item];
          ExtItem& head = items[c.item];
          // the tail's segments: a part of the one it starts in, and those behind
          int32_t at = head.seg_begin, skip = head.n_steps - c.steps;
          for (; skip >= attn_steps(segs[at].k_end - segs[at].k_begin); ++at)
            skip -= attn_steps(segs[at].k_end - segs[at].k_begin);
          const int32_t behind = head.seg_begin + head.n_seg;
          const int32_t shared = skip > 0;  // the segment at which both pieces take a part
          const int32_t first = (int32_t)segs.size();
          for (int32_t j = head.seg_begin; j < at + shared; ++j) segs.push_back(segs[j]);
          tail.seg_begin = (int32_t)segs.size();
          for (int32_t j = at; j < behind; ++j) segs.push_back(segs[j]);
          if (shared) {
            const int32_t k = segs[at].k_begin + skip * kAttnKeys;
            segs[tail.seg_begin - 1].k_end = k;
            segs[tail.seg_begin].k_begin = k;
            segs[tail.seg_begin].kv_row += skip;
          }
          head.seg_begin = first;
          head.n_seg = tail.seg_begin - first;
          head.n_steps -= c.steps;
          tail.n_seg = (int32_t)segs.size() - tail.seg_begin;
          tail.n_steps = c.steps;
          for (int x = 0; x < 2; ++x) {
            const int32_t n = head.n_tok[x];
            if (n == 0) continue;
            head.part[x] = (int32_t)npart;
            tail.part[x] = (int32_t)(npart + (int64_t)n * gq);
            for (int32_t i = 0; i < n; ++i) {
              mref.push_back({head.part[x] + i * gq, 0, 0, 0});
              mref.push_back({tail.part[x] + i * gq, 0, 0, 0});
              midx.push_back((int32_t)mref.size());
              merge_rows.push_back({rows[head.row_begin[x] + i].q_row, head.kv_head});
            }
            npart += 2 * (int64_t)n * gq;
          }
          max_refs = 2;
          lists[c.to].push_back((int32_t)items.size());
          items.push_back(tail);
        }
      }
    }
    std::vector<ExtItem> by_cta;
    by_cta.reserve(items.size());
    cta_begin.push_back(0);
    for (const auto& l : lists) {
      if (l.empty()) continue;
      for (int32_t i : l) by_cta.push_back(items[i]);
      cta_begin.push_back((int32_t)by_cta.size());
    }
    items.swap(by_cta);
  }

  // 8-bit pool: a few new tokens a request are a decode of as many rows, each with the keys up to its
  // own; the planner takes the plan that it expects to be faster.
  if (q8 && !items.empty() && cu[batch] <= kFewTokens &&
      *std::max_element(extend_len, extend_len + batch) <= kFewPerRequest) {
    const double expand_us = (double)tiles8.size() * hkv * kQ8ExpandBytes / 5e6;
    const double tiles_us =
        kQ8ExtendUs + expand_us + ends_at / 13.6 + (npart > 0 ? kMergeCost / 13.6 : 0.);
    rx_plan few;
    few.kv_next = RX_KV_E4M3;
    if (few_tokens_plan(&few, desc, batch, req_idx, prefix_len, extend_len, grp, num_groups,
                        group_prefix_len, group_parent) == RX_OK &&
        few.hdr().n_xitems == 0 && few.q8_us < tiles_us) {
      plan->blob.swap(few.blob);
      plan->ws_bytes = few.ws_bytes;
      plan->key_reads = few.key_reads;
      plan->kind = 1;
      remember_desc(plan, desc);
      return RX_OK;
    }
  }

  PlanHeader h;
  std::memset(&h, 0, sizeof h);
  h.magic = kPlanMagic;
  h.kind = 1;
  h.kv_type = plan->kv_next;
  h.ext_kernel = plan->ext_kernel;
  h.n_items = (int32_t)items.size();
  h.num_q_heads = desc->num_q_heads;
  h.num_kv_heads = hkv;
  h.batch = batch;
  h.n_rows = (int32_t)rows.size();
  size_t off = align256(sizeof(PlanHeader));
  h.off_items = off; off = align256(off + items.size() * sizeof(ExtItem));
  h.off_rows = off; off = align256(off + rows.size() * sizeof(ExtRow));
  h.off_segs = off; off = align256(off + segs.size() * sizeof(ExtSeg));
  h.off_cta = off; off = align256(off + cta_begin.size() * sizeof(int32_t));
  h.n_ctas = cta_begin.empty() ? 0 : (int32_t)cta_begin.size() - 1;
  h.off_q8_tiles = off; off = align256(off + tiles8.size() * sizeof(Q8Tile));
  h.n_q8_tiles = (int32_t)tiles8.size();
  h.off_merge_idx = off; off = align256(off + midx.size() * 4);
  h.off_merge = off; off = align256(off + mref.size() * sizeof(DecMergeRef));
  h.off_merge_rows = off; off = align256(off + merge_rows.size() * sizeof(MergeRow));
  h.n_merge_rows = (int64_t)merge_rows.size();
  h.max_refs = max_refs;
  h.n_sms = device_sms();
  plan->blob.assign(off, 0);
  h.off_part_o = off; off = align256(off + (size_t)npart * kHeadDim * 4);
  h.off_part_lse = off; off = align256(off + (size_t)npart * 4);
  h.n_part_rows = npart;
  h.off_q8_stage = off; off = align256(off + tiles8.size() * (size_t)hkv * kQ8BlockBytes);
  h.total_bytes = off;
  std::memcpy(plan->blob.data(), &h, sizeof h);
  put(plan->blob, h.off_items, items);
  put(plan->blob, h.off_rows, rows);
  put(plan->blob, h.off_segs, segs);
  put(plan->blob, h.off_cta, cta_begin);
  put(plan->blob, h.off_q8_tiles, tiles8);
  put(plan->blob, h.off_merge_idx, midx);
  put(plan->blob, h.off_merge, mref);
  put(plan->blob, h.off_merge_rows, merge_rows);
  plan->ws_bytes = off;
  plan->key_reads = key_reads;
  plan->kind = 1;
  remember_desc(plan, desc);
  return RX_OK;
}

rx_status rx_extend_attn(const rx_plan* plan, const rx_kv_desc* desc, const void* k_pool,
                         const void* v_pool, const void* q, void* o, float* lse,
                         void* workspace, size_t workspace_bytes, rx_stream_t stream) {
  rx_status st = check_plan_use(plan, 1, RX_KV_BF16, desc, k_pool, v_pool, q, o, lse, workspace,
                                workspace_bytes);
  if (st) return st;
  if (desc->pool_size * desc->num_kv_heads >= (int64_t)INT32_MAX)
    return fail(RX_ERR_UNSUPPORTED, "pool_size * num_kv_heads must be < 2^31 for extend");
  const PlanHeader h = plan->hdr();
  const int e = launch_extend(desc, &h, k_pool, v_pool, q, o, lse, workspace, stream);
  return e ? cuda_fail(e, "extend launch") : RX_OK;
}

rx_status rx_extend_attn_q8(const rx_plan* plan, const rx_kv_desc* desc, const rx_kv_q8* kv,
                            const void* q, void* o, float* lse, void* workspace,
                            size_t workspace_bytes, rx_stream_t stream) {
  const rx_status st =
      check_plan_use_q8(plan, 1, desc, kv, q, o, lse, workspace, workspace_bytes);
  if (st) return st;
  const PlanHeader h = plan->hdr();
  if (!has_rows(h)) return RX_OK;
  const int e = h.kind == 2 ? launch_decode_q8(desc, &h, kv, q, o, lse, workspace, stream)
                            : launch_extend_q8(desc, &h, kv, q, o, lse, workspace, stream);
  return e ? cuda_fail(e, "extend launch") : RX_OK;
}

rx_status rx_read_status(const void* workspace, int32_t* status, rx_stream_t stream) {
  if (!workspace || !status) return fail(RX_ERR_INVALID, "NULL argument");
  const char* w = static_cast<const char*>(workspace) + offsetof(PlanHeader, status);
  cudaError_t e = cudaMemcpyAsync(status, w, 4, cudaMemcpyDeviceToHost, (cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "status read");
  if (*status != 0) {
    e = cudaMemsetAsync(const_cast<char*>(w), 0, 4, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "status clear");
  }
  return RX_OK;
}

// ---------------------------------------------------------------------------------------------
// Validation of the contracts the attention calls trust (host copies of the tables).
// ---------------------------------------------------------------------------------------------
rx_status rx_check_slots(const int32_t* slots, int64_t n, int64_t pool_size, int64_t* bad) {
  if (bad) *bad = -1;
  if (n < 0 || pool_size <= 0) return fail(RX_ERR_INVALID, "negative count or empty pool");
  if (n > 0 && !slots) return fail(RX_ERR_INVALID, "slots is NULL");
  for (int64_t t = 0; t < n; ++t)
    if (slots[t] < 0 || slots[t] >= pool_size) {
      if (bad) *bad = t;
      return fail(RX_ERR_RANGE, "slots[%lld] = %d is outside the pool [0, %lld)", (long long)t,
                  slots[t], (long long)pool_size);
    }
  // (slot, index) pairs in order: within a run of one slot the first index is the original and
  // every later one a repeat; the earliest repeat over all runs is reported
  std::vector<std::pair<int32_t, int64_t>> by(n);
  for (int64_t t = 0; t < n; ++t) by[t] = {slots[t], t};
  std::sort(by.begin(), by.end());
  int64_t rep = -1, orig = -1, run = 0;  // run: start of the current slot's run
  for (int64_t i = 1; i < n; ++i) {
    if (by[i].first != by[i - 1].first) {
      run = i;
    } else if (i == run + 1 && (rep < 0 || by[i].second < rep)) {  // a run's first repeat
      rep = by[i].second;
      orig = by[run].second;
    }
  }
  if (rep >= 0) {
    if (bad) *bad = rep;
    return fail(RX_ERR_INVALID, "slots[%lld] = %d repeats slots[%lld]", (long long)rep,
                slots[rep], (long long)orig);
  }
  return RX_OK;
}

rx_status rx_check_tables(const int32_t* req_to_token, int64_t rows, int64_t stride,
                          int64_t pool_size, int32_t batch, const int32_t* req_idx,
                          const int32_t* key_len, const int32_t* group_of_req,
                          int32_t num_groups, const int32_t* group_prefix_len,
                          const int32_t* group_parent, int64_t* bad) {
  if (bad) *bad = -1;
  if (!req_to_token || rows <= 0 || stride <= 0 || pool_size <= 0 || batch < 0 ||
      num_groups < 0)
    return fail(RX_ERR_INVALID, "bad table shape, pool size or count");
  if (batch > 0 && (!req_idx || !key_len)) return fail(RX_ERR_INVALID, "NULL length array");
  if (num_groups > 0 && !group_prefix_len) return fail(RX_ERR_INVALID, "group_prefix_len NULL");
  rx_status st = check_tree(num_groups, group_prefix_len, group_parent);
  if (st) return st;
  auto parent = [&](int g) { return group_parent ? group_parent[g] : -1; };
  auto row = [&](int b) { return req_to_token + (int64_t)req_idx[b] * stride; };
  // lengths and slots of every request
  for (int b = 0; b < batch; ++b) {
    if (bad) *bad = b;
    if (req_idx[b] < 0 || req_idx[b] >= rows)
      return fail(RX_ERR_RANGE, "req_idx[%d] = %d outside the table", b, req_idx[b]);
    if (key_len[b] < 0 || key_len[b] > stride)
      return fail(RX_ERR_RANGE, "request %d reads %d keys, table rows hold %lld", b, key_len[b],
                  (long long)stride);
    const int g = group_of_req ? group_of_req[b] : -1;
    if (g < -1 || g >= num_groups) return fail(RX_ERR_RANGE, "group_of_req[%d] = %d", b, g);
    if (g >= 0 && group_prefix_len[g] > key_len[b])
      return fail(RX_ERR_RANGE, "request %d reads %d keys, fewer than its group's prefix %d", b,
                  key_len[b], group_prefix_len[g]);
    const int32_t* r = row(b);
    for (int j = 0; j < key_len[b]; ++j)
      if (r[j] < 0 || r[j] >= pool_size)
        return fail(RX_ERR_RANGE, "request %d: key %d has slot %d outside the pool", b, j, r[j]);
  }
  // Every request holds, for each group a on its path, the same entries as a's first request
  // (in batch order, over a's subtree) on a's own keys [prefix of a's parent, prefix of a).  By
  // induction down the path, every request of a's subtree then agrees with every other on
  // [0, prefix of a): the shared prefix the planners read once.
  std::vector<int> rep(num_groups, -1);
  for (int b = 0; b < batch; ++b) {
    const int g = group_of_req ? group_of_req[b] : -1;
    for (int a = g; a >= 0; a = parent(a))
      if (rep[a] < 0) rep[a] = b;
  }
  for (int b = 0; b < batch; ++b) {
    const int g = group_of_req ? group_of_req[b] : -1;
    for (int a = g; a >= 0; a = parent(a)) {
      const int lo = parent(a) >= 0 ? group_prefix_len[parent(a)] : 0;
      const int32_t *x = row(b), *y = row(rep[a]);
      for (int j = lo; j < group_prefix_len[a]; ++j)
        if (x[j] != y[j]) {
          if (bad) *bad = b;
          return fail(RX_ERR_INVALID,
                      "request %d, key %d: slot %d differs from slot %d of request %d, the "
                      "first of group %d (a shared prefix of %d keys)",
                      b, j, x[j], y[j], rep[a], a, group_prefix_len[a]);
        }
    }
  }
  if (bad) *bad = -1;
  return RX_OK;
}

}  // extern "C"
