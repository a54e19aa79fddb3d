// rx_decode_attn_q8: split-KV decode straight from the 8-bit pool.
//
// With codes kc, vc (e4m3) and scales ks, vs (fp32) of key j, and base-2 scores
//   s_j = scale log2(e) ks_j (q . kc_j):     o = sum_j 2^s_j vs_j vc_j / sum_j 2^s_j.
// The codes are exact in fp16, so both products run on the fp16 tensor cores with fp32 sums: a
// query row is brought to fp16 by a power of two that puts its largest magnitude in [2^14, 2^15)
// (what the conversion loses is below 2^-38 of that magnitude, and the power comes back in fp32).
// The second product's weights are 2^(s_j + log2 vs_j - m'), m' the running maximum of
// s_j + log2 vs_j: at most 1 whatever the scales are, so fp16 holds them to 2^-12 of their value
// down to 2^-14 of the largest term, and V's scale costs no product of its own.  The softmax's sum
// keeps its own running maximum of s_j.
//
// Work items are the bf16 decode's: a chunk of one table row's keys for up to eight KV heads and
// up to 16 stacked query rows (a shared prefix's members, or one request).  The queries are the
// narrow side of the products: S^T = Kc Q^T (16 keys x 8 rows a tile) and O^T = Vc^T P^T, so one
// request of a grouped-query model pads its rows to 8, not 16, and the codes, the wide operand,
// are converted once for all the query rows.
//   warps 0-7   one KV head each (where there are fewer than eight, the warps split a stage's keys
//               and each leaves a partial result of its own): 32 keys a stage, online softmax and
//               both products in registers.
//   warps 8-11  gather the codes by slot with 16-byte cp.async (chunks XOR-swizzled by row) and
//               the scales with 4-byte ones into a 3-stage ring that runs on across items; an
//               entry outside the pool is flagged and read as zeros.
// A persistent CTA per SM takes the items in snake order (they are sorted by falling cost).  Each
// item leaves normalised fp32 partial rows and base-2 log-sum-exps, which a second kernel merges.
// Waits are bounded; one that runs out records RX_ERR_TIMEOUT and every role leaves.
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>

#include "ptx.cuh"
#include "rx_internal.h"
#include "tc.cuh"

namespace rx {
namespace {

struct Params {
  const uint8_t* k_code;
  const uint8_t* v_code;
  const float* k_scale;
  const float* v_scale;
  const __nv_bfloat16* q;
  const int32_t* req_to_token;
  int64_t stride;
  int hq, hkv, gq;
  int hb_log2;  // heads of a block: 1 << hb_log2
  float scale_log2;
  const DecItem* items;
  const int32_t* rows;
  float* part_o;
  float* part_lse;
  int64_t pool_size;
  int32_t* status;
  int n_items;
};

constexpr int kWarps = 8;              // consumers
constexpr int kProducers = 128;        // threads
constexpr int kThreads = 32 * kWarps + kProducers;
constexpr int kWarpKeys = kQ8WarpKeys;  // keys a warp takes from a stage
constexpr int kRows = kWarps * kWarpKeys;        // (key, head) rows of K and of V per stage
constexpr int kHalf = kRows * kHeadDim;          // 32 KiB of codes
constexpr int kOffScale = 2 * kHalf;             // K scales, then V scales, of the rows
constexpr int kStageBytes = 2 * kHalf + 2 * kRows * 4;
constexpr int kStages = 3;
constexpr int kOffBar = kStages * kStageBytes;   // full[kStages], empty[kStages], abort
constexpr int kSmem = kOffBar + 2 * kStages * 8 + 16;
constexpr uint64_t kWaitNs = 2000000000ull;
static_assert(kSmem <= 227 * 1024, "shared memory budget");

__device__ __forceinline__ uint32_t row_off(int r, int c) {  // 16-byte chunk c of 128-byte row r
  return (uint32_t)(r * kHeadDim + ((c ^ (r & 7)) << 4));
}

// The k-th item of a CTA (snake order), -1 past the end.
__device__ __forceinline__ int item_at(const Params& p, int k) {
  const int G = gridDim.x;
  const int64_t i = (int64_t)k * G + ((k & 1) ? G - 1 - (int)blockIdx.x : (int)blockIdx.x);
  return i < p.n_items ? (int)i : -1;
}

__device__ __forceinline__ int checked(const Params& p, int slot) {
  if (slot < 0 || slot >= p.pool_size) {
    atomicCAS(p.status, 0, (int)RX_ERR_RANGE);
    return -1;
  }
  return slot;
}

__device__ __forceinline__ void arrive_on_copies(uint32_t mbar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(mbar) : "memory");
}

__device__ void producer(const Params& p, uint32_t base, volatile int* abort) {
  const int tid = threadIdx.x - 32 * kWarps;
  const int hb = 1 << p.hb_log2;
  const int nk = kRows >> p.hb_log2;  // keys of a stage
  const int c = tid & 7;
  constexpr int U = kRows * 8 / kProducers;  // 16-byte chunks of K (and of V) per thread and stage
  uint32_t g = 0;                            // stages filled so far
  for (int k = 0;; ++k) {
    const int idx = item_at(p, k);
    if (idx < 0) break;
    const DecItem it = p.items[idx];
    const int nkeys = it.k_end - it.k_begin;
    const int32_t* table = p.req_to_token + (int64_t)it.kv_row * p.stride + it.k_begin;
    const int head0 = it.head_block << p.hb_log2;
    auto slots_of = [&](int k0, int (&sl)[U], int (&ss)[2]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int key = k0 + ((u * (kProducers / 8) + (tid >> 3)) >> p.hb_log2);
        sl[u] = key < nkeys ? __ldg(table + key) : -2;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int key = k0 + ((u * kProducers + tid) >> p.hb_log2);
        ss[u] = key < nkeys ? __ldg(table + key) : -2;
      }
    };
    int sl[U], ss[2];
    slots_of(0, sl, ss);
    for (int k0 = 0; k0 < nkeys; k0 += nk, ++g) {
      const int st = g % kStages;
      const uint32_t full = base + kOffBar + 8 * st, empty = full + 8 * kStages;
      if (g >= kStages && !tc::mbar_wait(empty, (g / kStages - 1) & 1, abort, p.status, kWaitNs)) {
        cp_async_wait<0>();
        return;
      }
      const uint32_t kb = base + st * kStageBytes, vb = kb + kHalf, sb = kb + kOffScale;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = u * (kProducers / 8) + (tid >> 3);
        const int h = i & (hb - 1), key = i >> p.hb_log2;
        int s = sl[u];
        if (s != -2) s = checked(p, s);
        const bool ok = s >= 0;
        const int64_t off = ok ? ((int64_t)s * p.hkv + head0 + h) * kHeadDim + 16 * c : 0;
        // row of warp (key / 32) * hb + h: its 32 keys lie together
        const uint32_t so = row_off((((key >> 5) << p.hb_log2) + h) * kWarpKeys + (key & 31), c);
        cp_async16(kb + so, p.k_code + off, ok);
        cp_async16(vb + so, p.v_code + off, ok);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = u * kProducers + tid;
        const int h = i & (hb - 1), key = i >> p.hb_log2;
        const int s = ss[u];
        const bool ok = s >= 0 && s < p.pool_size;
        const int64_t off = ok ? (int64_t)s * p.hkv + head0 + h : 0;
        const uint32_t r = (((key >> 5) << p.hb_log2) + h) * kWarpKeys + (key & 31);
        cp_async4(sb + 4 * r, p.k_scale + off, ok);
        cp_async4(sb + 4 * (kRows + r), p.v_scale + off, ok);
      }
      arrive_on_copies(full);
      if (k0 + nk < nkeys) slots_of(k0 + nk, sl, ss);
    }
  }
  cp_async_wait<0>();
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One item on a consumer warp: NT tiles of 8 query rows.  Returns false when a wait gave up.
template <int NT>
__device__ bool run_item(const Params& p, const DecItem& it, uint32_t base, const uint8_t* smem,
                         uint32_t& gs, volatile int* abort) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int head = (it.head_block << p.hb_log2) + (warp & ((1 << p.hb_log2) - 1));
  const int split = warp >> p.hb_log2;
  const int nk = kRows >> p.hb_log2;
  const int nkeys = it.k_end - it.k_begin;
  const int rows = it.n_tok * p.gq;

  // Query fragments: position 2c + e of a 16-wide step holds d = 16 step + 4c + e, and 8 + 2c + e
  // holds 16 step + 4c + 2 + e, as the conversion of four neighbouring codes leaves K.
  uint32_t qf[8][NT][2];
  float qs[NT][2];  // scale_log2 and the row's power of two, for the columns 2c and 2c + 1
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = 8 * n + g;
    uint2 x[8];
    uint32_t m = 0;
    if (r < rows) {
      const __nv_bfloat16* src =
          p.q + ((int64_t)__ldg(p.rows + it.row_begin + r / p.gq) * p.hq + head * p.gq + r % p.gq) *
                    kHeadDim + 4 * c;
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = __ldg(reinterpret_cast<const uint2*>(src + 16 * k));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = make_uint2(0, 0);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      m = __vmaxu2(m, __vmaxu2(x[k].x & 0x7fff7fffu, x[k].y & 0x7fff7fffu));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    // biased exponent of the row's largest magnitude; a row below 2^-87 keeps 2^-87's power
    const int e = max((int)(max(m & 0xffffu, m >> 16) >> 7), 40);
    const float up = __uint_as_float((uint32_t)(268 - e) << 23);
    const float down = __uint_as_float((uint32_t)(e - 14) << 23);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      qf[k][n][0] = pack_f16(__uint_as_float(x[k].x << 16) * up,
                             __uint_as_float(x[k].x & 0xffff0000u) * up);
      qf[k][n][1] = pack_f16(__uint_as_float(x[k].y << 16) * up,
                             __uint_as_float(x[k].y & 0xffff0000u) * up);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
      qs[n][j] = __shfl_sync(0xffffffffu, down, 4 * (2 * c + j)) * p.scale_log2;
  }

  float o[8][NT][4];
  float m1[NT][2], m2[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      m1[n][j] = m2[n][j] = -CUDART_INF_F;
      l[n][j] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
  }

  for (int k0 = 0; k0 < nkeys; k0 += nk, ++gs) {
    const int st = gs % kStages;
    const uint32_t full = base + kOffBar + 8 * st;
    const bool ok = tc::mbar_wait(full, (gs / kStages) & 1, abort, p.status, kWaitNs);
    if (__any_sync(0xffffffffu, !ok)) return false;
    const int left = nkeys - k0 - split * kWarpKeys;  // keys of this warp in the stage
    if (left > 0) {
      const uint32_t kb = base + st * kStageBytes + warp * kWarpKeys * kHeadDim;
      const uint32_t vb = kb + kHalf;
      const float* sc = reinterpret_cast<const float*>(smem + st * kStageBytes + kOffScale) +
                        warp * kWarpKeys;
      float s[2][NT][4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n) s[t][n][0] = s[t][n][1] = s[t][n][2] = s[t][n][3] = 0.f;
#pragma unroll
      for (int k2 = 0; k2 < 4; ++k2)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          uint32_t x[4];
          const int r = 16 * t + (lane & 15);
          ldsm_x4(kb + row_off(r, 2 * k2 + (lane >> 4)), x[0], x[1], x[2], x[3]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a[4] = {e4m3x2_to_f16x2(x[2 * h]), e4m3x2_to_f16x2(x[2 * h + 1]),
                                   e4m3x2_hi_to_f16x2(x[2 * h]), e4m3x2_hi_to_f16x2(x[2 * h + 1])};
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_16816_f16(s[t][n], a, qf[2 * k2 + h][n][0], qf[2 * k2 + h][n][1]);
          }
        }
      // scales, masks, the two running maxima (columns 2c + j; keys 16 t + 8 h + g)
      float lv[2][2];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = 16 * t + 8 * h + g;
          const float ks = sc[key];
          lv[t][h] = lg2(sc[kRows + key]);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              s[t][n][2 * h + j] =
                  key < left ? s[t][n][2 * h + j] * ks * qs[n][j] : -CUDART_INF_F;
        }
      uint32_t pt[2][NT][2];  // P^T: columns are query rows, two keys a register
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float a2[2], p2[2][2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x1 = fmaxf(fmaxf(s[0][n][j], s[0][n][2 + j]), fmaxf(s[1][n][j], s[1][n][2 + j]));
          float x2 = fmaxf(fmaxf(s[0][n][j] + lv[0][0], s[0][n][2 + j] + lv[0][1]),
                           fmaxf(s[1][n][j] + lv[1][0], s[1][n][2 + j] + lv[1][1]));
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
            x2 = fmaxf(x2, __shfl_xor_sync(0xffffffffu, x2, off));
          }
          x1 = fmaxf(x1, m1[n][j]);
          x2 = fmaxf(x2, m2[n][j]);
          // no finite score yet: any finite reference serves
          const float r1 = x1 == -CUDART_INF_F ? 0.f : x1, r2 = x2 == -CUDART_INF_F ? 0.f : x2;
          const float a1 = fast_exp2(m1[n][j] - r1);
          a2[j] = fast_exp2(m2[n][j] - r2);
          m1[n][j] = x1;
          m2[n][j] = x2;
          float sum = 0.f;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float v = s[t][n][2 * h + j];
              sum += fast_exp2(v - r1);
              p2[t][h][j] = fast_exp2(v + lv[t][h] - r2);
            }
          l[n][j] = l[n][j] * a1 + sum;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) pt[t][n][h] = movm_t(pack_f16(p2[t][h][0], p2[t][h][1]));
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][n][e] *= a2[e & 1];
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i2 = 0; i2 < 4; ++i2) {
          uint32_t x[4];
          const int r = 16 * t + (lane & 15);
          ldsm_x4_t(vb + row_off(r, 2 * i2 + (lane >> 4)), x[0], x[1], x[2], x[3]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // bytes (key, d), (key, d+1), (key+1, d), (key+1, d+1) -> the two keys of d, of d+1
            const uint32_t y0 = __byte_perm(x[2 * h], 0, 0x3120);
            const uint32_t y1 = __byte_perm(x[2 * h + 1], 0, 0x3120);
            const uint32_t a[4] = {e4m3x2_to_f16x2(y0), e4m3x2_hi_to_f16x2(y0),
                                   e4m3x2_to_f16x2(y1), e4m3x2_hi_to_f16x2(y1)};
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_16816_f16(o[2 * i2 + h][n], a, pt[t][n][0], pt[t][n][1]);
          }
        }
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(full + 8 * kStages);
  }

  // partial rows: split, KV head, row.  A split without keys has none (the merge knows).
  if (split * kWarpKeys >= nkeys) return true;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
        l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], off);
      const int r = 8 * n + 2 * c + j;
      if (r >= rows) continue;
      const bool none = l[n][j] == 0.f;
      // (m1 = -inf with a sum: NaN scores only, and the sum says so)
      const float r1 = m1[n][j] == -CUDART_INF_F ? 0.f : m1[n][j];
      const float f = none ? 0.f : fast_exp2(m2[n][j] - r1) / l[n][j];
      const int64_t row = (int64_t)it.part + ((int64_t)split * p.hkv + head) * rows + r;
      float* dst = p.part_o + row * kHeadDim + 2 * g;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<float2*>(dst + 16 * i) = make_float2(o[i][n][j] * f, o[i][n][2 + j] * f);
      if (g == 0) p.part_lse[row] = none ? -CUDART_INF_F : r1 + __log2f(l[n][j]);
    }
  }
  return true;
}

__global__ void __launch_bounds__(kThreads, 1) decode_q8_kernel(const Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + kOffBar + 2 * kStages * 8);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(base + kOffBar + 8 * i, kProducers);
      tc::mbar_init(base + kOffBar + 8 * (kStages + i), kWarps);
    }
    *abort = 0;
  }
  __syncthreads();
  if (threadIdx.x >= 32 * kWarps) {
    producer(p, base, abort);
    return;
  }
  uint32_t gs = 0;
  for (int k = 0;; ++k) {
    const int idx = item_at(p, k);
    if (idx < 0) return;
    const DecItem it = p.items[idx];
    const bool ok = it.kind == 0 ? run_item<1>(p, it, base, smem, gs, abort)
                                 : run_item<2>(p, it, base, smem, gs, abort);
    if (!ok) return;
  }
}

// One warp per (request, query head); lane owns 4 of the 128 columns.  lse = log2 sum 2^lse_i,
// o = sum 2^(lse_i - lse) o_i; a partial whose log-sum-exp is NaN makes both NaN.
constexpr int kMergeWarps = 8;
__global__ void __launch_bounds__(32 * kMergeWarps) merge_q8_kernel(
    const float* __restrict__ part_o, const float* __restrict__ part_lse,
    const int32_t* __restrict__ merge_idx, const DecMergeRef* __restrict__ refs, int batch, int hq,
    int gq, __nv_bfloat16* __restrict__ o, float* __restrict__ lse) {
  const int64_t task = (int64_t)blockIdx.x * kMergeWarps + threadIdx.x / 32;
  if (task >= (int64_t)batch * hq) return;
  const int lane = threadIdx.x % 32;
  const int b = (int)(task / hq), h = (int)(task % hq);
  const int hk = h / gq, g = h % gq;
  const int r_begin = merge_idx[b], r_end = merge_idx[b + 1];
  float mx = -CUDART_INF_F, tot = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  // per chunk of 32 partials the lanes fetch one reference and log-sum-exp each, so every weight is
  // known before any row is read and the row reads are independent of one another
  for (int c0 = r_begin; c0 < r_end; c0 += 32) {
    const int i = c0 + lane;
    int64_t idx = 0;
    float li = -CUDART_INF_F;
    if (i < r_end) {
      const DecMergeRef rf = refs[i];
      idx = (int64_t)rf.part + (int64_t)hk * rf.rows_real + rf.row + g;
      li = part_lse[idx];
    }
    float cm = li;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, off));
    const float m_new = fmaxf(mx, cm);
    const float ref = m_new == -CUDART_INF_F ? 0.f : m_new;
    const float a = fast_exp2(mx - ref);  // exp2(-inf) = 0
    const float w = li == -CUDART_INF_F ? 0.f : fast_exp2(li - ref);
    float ws = w;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, off);
    tot = tot * a + ws;
    acc.x *= a;
    acc.y *= a;
    acc.z *= a;
    acc.w *= a;
    mx = m_new;
    const int cnt = min(32, r_end - c0);
#pragma unroll 4
    for (int j = 0; j < cnt; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const int64_t ij = __shfl_sync(0xffffffffu, idx, j);
      if (wj == 0.f) continue;  // the same for the whole warp
      const float4 v = *reinterpret_cast<const float4*>(part_o + ij * kHeadDim + lane * 4);
      acc.x += wj * v.x;
      acc.y += wj * v.y;
      acc.z += wj * v.z;
      acc.w += wj * v.w;
    }
  }
  const float inv = tot == 0.f ? 0.f : 1.f / tot;
  const uint2 packed =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  *reinterpret_cast<uint2*>(o + ((int64_t)b * hq + h) * kHeadDim + lane * 4) = packed;
  if (lane == 0)
    lse[(int64_t)b * hq + h] =
        tot == 0.f ? -CUDART_INF_F
                   : ((mx == -CUDART_INF_F ? 0.f : mx) + __log2f(tot)) * 0.69314718055994530942f;
}

}  // namespace

int launch_decode_q8(const rx_kv_desc* d, const PlanHeader* h, const rx_kv_q8* kv, const void* q,
                     void* o, float* lse, void* ws, void* stream) {
  // kernel attributes belong to the current device: set once per device (bit d of the mask)
  static std::atomic<uint64_t> attr_set{0};
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return (int)e;
  if (dev < 0 || dev >= 64) return (int)cudaErrorInvalidDevice;
  if (!((attr_set.load() >> dev) & 1)) {
    e = cudaFuncSetAttribute(decode_q8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return (int)e;
    attr_set.fetch_or(1ull << dev);
  }
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return (int)e;
  uint8_t* base = static_cast<uint8_t*>(ws);
  Params p;
  p.k_code = static_cast<const uint8_t*>(kv->k_code);
  p.v_code = static_cast<const uint8_t*>(kv->v_code);
  p.k_scale = kv->k_scale;
  p.v_scale = kv->v_scale;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.req_to_token = d->req_to_token;
  p.stride = d->req_to_token_stride;
  p.hq = d->num_q_heads;
  p.hkv = d->num_kv_heads;
  p.gq = d->num_q_heads / d->num_kv_heads;
  p.hb_log2 = q8_head_block_log2(d->num_kv_heads);
  p.scale_log2 = d->softmax_scale * 1.4426950408889634f;
  p.items = reinterpret_cast<const DecItem*>(base + h->off_items);
  p.rows = reinterpret_cast<const int32_t*>(base + h->off_rows);
  p.part_o = reinterpret_cast<float*>(base + h->off_part_o);
  p.part_lse = reinterpret_cast<float*>(base + h->off_part_lse);
  p.pool_size = d->pool_size;
  p.status = reinterpret_cast<int32_t*>(base + offsetof(PlanHeader, status));
  p.n_items = h->n_items;
  cudaStream_t s = (cudaStream_t)stream;
  if (h->n_items > 0) {
    const int grid = h->n_items < sms ? h->n_items : sms;
    decode_q8_kernel<<<grid, kThreads, kSmem, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return (int)e;
  }
  if (h->batch > 0) {
    const int64_t tasks = (int64_t)h->batch * p.hq;
    merge_q8_kernel<<<(unsigned)((tasks + kMergeWarps - 1) / kMergeWarps), 32 * kMergeWarps, 0,
                      s>>>(p.part_o, p.part_lse,
                           reinterpret_cast<const int32_t*>(base + h->off_merge_idx),
                           reinterpret_cast<const DecMergeRef*>(base + h->off_merge), h->batch,
                           p.hq, p.gq, static_cast<__nv_bfloat16*>(o), lse);
  }
  return (int)cudaGetLastError();
}

}  // namespace rx
