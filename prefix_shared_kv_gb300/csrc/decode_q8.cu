// rx_decode_attn_q8: split-KV decode straight from the 8-bit pool.
//
// With codes kc, vc (e4m3) and scales ks, vs (fp32) of key j, and base-2 scores
//   s_j = scale log2(e) ks_j (q . kc_j):     o = sum_j 2^s_j vs_j vc_j / sum_j 2^s_j.
// The codes are exact in fp16, so both products run on the fp16 tensor cores with fp32 sums.  A
// warp's query rows are brought to fp16 by a common power of two, taken back in fp32, which puts
// their largest magnitude H in [2^14, 2^15): what the conversion loses of an element is below
// 2^-39 H, less than the fp32 sums of the row of H lose.  Rows of 2^20 or more, beside which that would
// tell on another request's scores, have no part in it (unless all are that large, and within
// 2^16): a warp computes them in fp32 by themselves when it is done with the others.
// With p_j = 2^(s_j - m), m a running reference of the row, the sum takes p_j and the
// second product's weights are p_j vs_j c, c a power of two of the row that keeps their magnitude at
// 2^8 or less whatever the scales (of either sign) are: fp16 holds them to 2^-11 of their value down to 2^-14, and to
// 2^-25 below.  m and c only move (and O is only rescaled) when some p_j or weight of the warp's
// passes 2^8, which one vote per step decides; until then a step needs no maximum across lanes.
//
// Work items are the bf16 decode's: a chunk of one table row's keys for a block of KV heads and
// some stacked query rows (a shared prefix's members, or one request).  The queries are the narrow
// side of the products: S^T = Kc Q^T (16 keys x 8 rows a tile) and O^T = Vc^T P^T, so one request
// of a grouped-query model pads its rows to 8, not 16, and the codes, the wide operand, are
// converted once for all the query rows of a warp.
//   warps 0-7   one KV head each: 32 keys a stage, softmax and both products in registers.  Where a
//               block has fewer heads than there are warps for it, the warps split the stage's keys
//               and each leaves a partial result of its own.
//   warps 8-11  gather the codes by slot with 16-byte cp.async (chunks XOR-swizzled by row) and the
//               scales with 4-byte ones into a ring that runs on across items; an entry outside the
//               pool is flagged and read as zeros.
// Two forms.  Narrow items have up to 16 rows: eight heads a block, queries in registers, three
// stages.  Wide ones have up to 64: a head's rows go to two warps (32 each), four heads a block;
// the O tile alone takes 128 registers, so the queries lie in shared memory as fragments and the
// producers hand registers to the consumers.  (On 16 x 16 requests with 64 rows per KV head and
// 16,000 shared keys, whole call: 278 us; 16-key steps, which halve the independent products, 294
// us; 224 or 216 registers for the consumers, with spills, 288 and 306 us; the references in shared
// memory instead of spills, 284 us.)
// (A shared prefix of more than 128 rows is not run here: its keys are expanded as for an
// extend, which moves three times their bytes, and the tensor-core tile kernel takes 256 rows at a
// time.)
// A persistent CTA per SM runs the list of items that the planner gave it.  Each item leaves
// normalised fp32 partial rows and base-2 log-sum-exps, which a last kernel merges.  The kernels are
// chained by programmatic dependent launch: the narrow one starts as SMs come free of the wide
// one, and the merge waits for both.
// Waits are bounded; one that runs out records RX_ERR_TIMEOUT and every role leaves.
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>

#include "pdl.cuh"
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
  float scale_log2;
  const DecItem* items;
  const int32_t* rows;
  float* part_o;
  float* part_lse;
  int64_t pool_size;
  int32_t* status;
  const int32_t* cta_begin;  // per-CTA item lists: [gridDim.x + 1] starts
  bool after_wide;           // the wide kernel was launched before this (narrow) one
};

constexpr int kWarps = 8;        // consumers
constexpr int kProducers = 128;  // threads
constexpr int kThreads = 32 * kWarps + kProducers;
// Registers: the launch's 168 a thread; the wide form moves them to its consumers.
constexpr int kRegsLaunch = 168, kRegsConsumer = 232, kRegsProducer = 40;
static_assert(2 * kRegsConsumer + kRegsProducer == 3 * kRegsLaunch, "register split");
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kUnset = -3.402823466e38f;  // a reference no score has moved yet: the lowest float

// HB = 1 << HBL KV heads a block.
template <bool WIDE, int HBL>
struct Form {
  static constexpr int HB = 1 << HBL;
  static constexpr int kRowWarps = WIDE ? 2 : 1;               // warps that share a head's rows
  static constexpr int kRows = kWarps / kRowWarps * kQ8WarpKeys;  // (key, head) rows of a stage
  static constexpr int NK = kRows / HB;                        // keys of a stage
  static constexpr int kStages = WIDE ? 4 : 3;
  static constexpr int kHalf = kRows * kHeadDim;               // codes of K, then of V
  static constexpr int kOffScale = 2 * kHalf;                  // K scales, then V scales, [key][head]
  static constexpr int kStageBytes = 2 * kHalf + 2 * kRows * 4;
  static constexpr int kOffBar = kStages * kStageBytes;        // full[], empty[], abort
  static constexpr int kOffQ = kOffBar + 2 * kStages * 8 + 64 - (2 * kStages * 8) % 64;
  static constexpr int kQWarp = 8 * 4 * 32 * 8;                // a warp's query fragments (wide)
  static constexpr int kSmem = kOffQ + (WIDE ? kWarps * kQWarp : 0);
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(NK % 32 == 0, "a stage holds whole groups of 32 keys");
};

__device__ __forceinline__ uint32_t row_off(int r, int c) {  // 16-byte chunk c of 128-byte row r
  return (uint32_t)(r * kHeadDim + ((c ^ (r & 7)) << 4));
}

// The k-th item of the CTA's list, -1 past its end.
__device__ __forceinline__ int item_at(const Params& p, int k) {
  const int i = __ldg(&p.cta_begin[blockIdx.x]) + k;
  return i < __ldg(&p.cta_begin[blockIdx.x + 1]) ? i : -1;
}

__device__ __forceinline__ void arrive_on_copies(uint32_t mbar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(mbar) : "memory");
}

// Producer warp w of four.  Flat row f = key * HB + head of a stage takes eight lanes, so an
// instruction copies four rows (512 contiguous bytes where a block has four heads or more), and the
// warps take every fourth instruction.  A lane holds the table entries of keys lane, lane + 32, ...
// of the stage, fetched a stage ahead and checked once; the copies take them by shuffle.
template <bool WIDE, int HBL>
__device__ void producer(const Params& p, uint32_t base, volatile int* abort) {
  using F = Form<WIDE, HBL>;
  constexpr int HB = F::HB, NK = F::NK, S = NK / 32;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - kWarps;
  const int c = lane & 7, sub = lane >> 3;
  uint32_t g = 0;  // stages filled so far
  for (int k = 0;; ++k) {
    const int idx = item_at(p, k);
    if (idx < 0) break;
    const DecItem it = p.items[idx];
    const int nkeys = it.k_end - it.k_begin;
    const int32_t* table = p.req_to_token + (int64_t)it.kv_row * p.stride + it.k_begin;
    const int head0 = it.head_block * HB;
    int nxt[S];
    auto fetch = [&](int k0) {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int key = k0 + 32 * i + lane;
        nxt[i] = key < nkeys ? __ldg(table + key) : -1;
      }
    };
    fetch(0);
    for (int k0 = 0; k0 < nkeys; k0 += NK, ++g) {
      const int st = g % F::kStages;
      const uint32_t full = base + F::kOffBar + 8 * st, empty = full + 8 * F::kStages;
      int sl[S];
#pragma unroll
      for (int i = 0; i < S; ++i) {
        sl[i] = nxt[i];
        if (sl[i] < 0 || sl[i] >= p.pool_size) {  // a key's: flagged, and read as zeros
          if (k0 + 32 * i + lane < nkeys) atomicCAS(p.status, 0, (int)RX_ERR_RANGE);
          sl[i] = -1;
        }
      }
      if (k0 + NK < nkeys) fetch(k0 + NK);
      const bool ok = g < F::kStages ||
                      tc::mbar_wait(empty, (g / F::kStages - 1) & 1, abort, p.status, kWaitNs);
      if (__any_sync(0xffffffffu, !ok)) {
        cp_async_wait<0>();
        return;
      }
      const uint32_t kb = base + st * F::kStageBytes, vb = kb + F::kHalf, sb = kb + F::kOffScale;
#pragma unroll
      for (int i = 0; i < F::kRows / 16; ++i) {
        const int f = 16 * i + 4 * w + sub;
        const int key = f >> HBL, h = f & (HB - 1);
        // (16 i .. 16 i + 15 lie in one run of 32 keys: the register is known here)
        const int slot = __shfl_sync(0xffffffffu, sl[(16 * i) >> (HBL + 5)], key & 31);
        const int64_t off =
            slot >= 0 ? ((int64_t)slot * p.hkv + head0 + h) * kHeadDim + 16 * c : 0;
        const uint32_t so = row_off(((key >> 5) * HB + h) * kQ8WarpKeys + (key & 31), c);
        cp_async16(kb + so, p.k_code + off, slot >= 0);
        cp_async16(vb + so, p.v_code + off, slot >= 0);
      }
#pragma unroll
      for (int i = 0; i < F::kRows / 128; ++i) {  // scales, [key][head]
        const int f = 128 * i + 32 * w + lane;
        const int key = f >> HBL, h = f & (HB - 1);
        int slot = 0;
#pragma unroll
        for (int j = 0; j < S; ++j) {
          const int x = __shfl_sync(0xffffffffu, sl[j], key & 31);
          if (j == key >> 5) slot = x;
        }
        const int64_t off = slot >= 0 ? (int64_t)slot * p.hkv + head0 + h : 0;
        cp_async4(sb + 4 * f, p.k_scale + off, slot >= 0);
        cp_async4(sb + 4 * (F::kRows + f), p.v_scale + off, slot >= 0);
      }
      arrive_on_copies(full);
    }
  }
  cp_async_wait<0>();
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The partial result of one query row over the warp's keys of an item, in fp32, without the ring: a
// lane takes a key's score, then four of the 128 columns.
template <bool WIDE, int HBL>
__device__ void run_far_row(const Params& p, const DecItem& it, int head, int split, int rows,
                            int r) {
  using F = Form<WIDE, HBL>;
  const int lane = threadIdx.x & 31;
  const int nkeys = it.k_end - it.k_begin;
  const int32_t* table = p.req_to_token + (int64_t)it.kv_row * p.stride + it.k_begin;
  const uint4* q = reinterpret_cast<const uint4*>(
      p.q + ((int64_t)__ldg(p.rows + it.row_begin + r / p.gq) * p.hq + head * p.gq + r % p.gq) *
                kHeadDim);
  float m = -CUDART_INF_F, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k0 = split * kQ8WarpKeys; k0 < nkeys; k0 += F::NK) {
    const bool live = k0 + lane < nkeys;
    int slot = live ? __ldg(table + k0 + lane) : -1;
    if (slot >= p.pool_size) slot = -1;  // (flagged by the producer; zeros)
    const int64_t row = (int64_t)slot * p.hkv + head;
    float s = 0.f, vs = 0.f;
    if (slot >= 0) {
      vs = __ldg(p.v_scale + row);
#pragma unroll 1
      for (int c = 0; c < 16; ++c) {
        const uint2 k = __ldg(reinterpret_cast<const uint2*>(p.k_code + row * kHeadDim) + c);
        const uint4 x = __ldg(q + c);
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = e4m3x2_to_f32((i < 2 ? k.x : k.y) >> (16 * (i & 1)));
          s += f.x * __uint_as_float(xs[i] << 16) + f.y * __uint_as_float(xs[i] & 0xffff0000u);
        }
      }
      s *= __ldg(p.k_scale + row) * p.scale_log2;
    }
    if (!live) s = -CUDART_INF_F;
    float x = s;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
    const float m_new = fmaxf(m, x), ref = m_new == -CUDART_INF_F ? 0.f : m_new;
    const float a = fast_exp2(m - ref), e = fast_exp2(s - ref), w = e * vs;
    m = m_new;
    l = l * a + e;  // this lane's keys
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= a;
#pragma unroll 1
    for (int j = 0; j < 32; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const int sj = __shfl_sync(0xffffffffu, slot, j);
      if (sj < 0) continue;
      const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(
                                   p.v_code + ((int64_t)sj * p.hkv + head) * kHeadDim) + lane);
      const float2 f0 = e4m3x2_to_f32(v), f1 = e4m3x2_to_f32(v >> 16);
      o[0] += wj * f0.x;
      o[1] += wj * f0.y;
      o[2] += wj * f1.x;
      o[3] += wj * f1.y;
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  const float f = l == 0.f ? 0.f : 1.f / l;
  const int64_t prow = (int64_t)it.part + ((int64_t)split * p.hkv + head) * rows + r;
  *reinterpret_cast<float4*>(p.part_o + prow * kHeadDim + 4 * lane) =
      make_float4(o[0] * f, o[1] * f, o[2] * f, o[3] * f);
  if (lane == 0)
    p.part_lse[prow] =
        l == 0.f ? -CUDART_INF_F : (m == -CUDART_INF_F ? 0.f : m) + __log2f(l);
}

// One item on a consumer warp: NT tiles of 8 query rows.  Returns false when a wait gave up.
template <int NT, bool WIDE, int HBL>
__device__ __forceinline__ bool run_item(const Params& p, const DecItem& it, uint32_t base,
                                         uint8_t* smem, uint32_t& gs, volatile int* abort) {
  using F = Form<WIDE, HBL>;
  constexpr int HB = F::HB, NK = F::NK;
  constexpr int KT = kQ8WarpKeys / 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int kw = warp % (kWarps / F::kRowWarps);  // the warp's 32-key run of a stage
  const int row0 = warp / (kWarps / F::kRowWarps) * (8 * NT);
  const int head = it.head_block * HB + (kw & (HB - 1));
  const int split = kw >> HBL;
  const int nkeys = it.k_end - it.k_begin;
  const int rows = it.n_tok * p.gq;

  // Query fragments: position 2c + e of a 16-wide step holds d = 16 step + 4c + e, and 8 + 2c + e
  // holds 16 step + 4c + 2 + e, as the conversion of four neighbouring codes leaves K.  The wide
  // form keeps them in shared memory, written and read by the same lane.
  uint2 qf[WIDE ? 1 : 8][WIDE ? 1 : NT];
  uint2* sq = reinterpret_cast<uint2*>(smem + F::kOffQ + warp * F::kQWarp) + lane;
  float qs;          // scale_log2 and the power of two
  uint32_t far = 0;  // rows computed apart
  {
    uint2 x[WIDE ? 1 : NT][8];
    int ex[NT];  // biased exponent of the row's largest magnitude (255: not finite)
    auto load = [&](int n, uint2 (&y)[8]) {
      const int r = row0 + 8 * n + g;
      const __nv_bfloat16* src =
          p.q + ((int64_t)(r < rows ? __ldg(p.rows + it.row_begin + r / p.gq) : 0) * p.hq +
                 head * p.gq + r % p.gq) * kHeadDim + 4 * c;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        y[k] = r < rows ? __ldg(reinterpret_cast<const uint2*>(src + 16 * k)) : make_uint2(0, 0);
    };
    int hi = 0, lo = 255;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint2(&y)[8] = x[WIDE ? 0 : n];
      load(n, y);
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        m = __vmaxu2(m, __vmaxu2(y[k].x & 0x7fff7fffu, y[k].y & 0x7fff7fffu));
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
      ex[n] = (int)(max(m & 0xffffu, m >> 16) >> 7);
      if (row0 + 8 * n + g < rows) {
        lo = min(lo, ex[n]);
        if (ex[n] < 127 + 20) hi = max(hi, ex[n]);
      }
    }
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (hi == 0) {  // zeros and subnormals, or large rows only
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = min(lo + 16, 254);
    }
    hi = max(hi, 40);
    const float up = __uint_as_float((uint32_t)(268 - hi) << 23);
    qs = __uint_as_float((uint32_t)(hi - 14) << 23) * p.scale_log2;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // (a row that is not finite stays: its scores are NaN in its own column)
      const bool apart = ex[n] > hi && ex[n] < 255;
      const uint32_t some = __ballot_sync(0xffffffffu, apart && c == 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) far |= (some >> (4 * i) & 1u) << (8 * n + i);
      uint2(&v)[8] = x[WIDE ? 0 : n];
      if constexpr (WIDE) load(n, v);  // (again, from the cache: fewer registers)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint2 y = make_uint2(pack_f16(__uint_as_float(v[k].x << 16) * up,
                                      __uint_as_float(v[k].x & 0xffff0000u) * up),
                             pack_f16(__uint_as_float(v[k].y << 16) * up,
                                      __uint_as_float(v[k].y & 0xffff0000u) * up));
        if (apart) y = make_uint2(0, 0);
        if constexpr (WIDE)
          sq[(k * NT + n) * 32] = y;
        else
          qf[k][n] = y;
      }
    }
  }

  float o[8][NT][4];
  // per column pair 2c, 2c + 1: -m, c, and this lane's part of the sum
  uint64_t nm[NT], cw[NT], l[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    nm[n] = f2_pack(-kUnset, -kUnset);
    cw[n] = l[n] = 0ull;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
  }

  for (int k0 = 0; k0 < nkeys; k0 += NK, ++gs) {
    const int st = gs % F::kStages;
    const uint32_t full = base + F::kOffBar + 8 * st;
    const bool ok = tc::mbar_wait(full, (gs / F::kStages) & 1, abort, p.status, kWaitNs);
    if (__any_sync(0xffffffffu, !ok)) return false;
    const int left = nkeys - k0 - split * kQ8WarpKeys;  // keys of this warp in the stage
    const uint32_t kb = base + st * F::kStageBytes + kw * kQ8WarpKeys * kHeadDim;
    const uint32_t vb = kb + F::kHalf;
    const float* sc = reinterpret_cast<const float*>(smem + st * F::kStageBytes + F::kOffScale) +
                      split * kQ8WarpKeys * HB + (kw & (HB - 1));
    if (left > 0) {
      float s[KT][NT][4];
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n) s[t][n][0] = s[t][n][1] = s[t][n][2] = s[t][n][3] = 0.f;
#pragma unroll
      for (int k2 = 0; k2 < 4; ++k2)
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          uint32_t x[4];
          const int r = 16 * t + (lane & 15);
          ldsm_x4(kb + row_off(r, 2 * k2 + (lane >> 4)), x[0], x[1], x[2], x[3]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a[4] = {e4m3x2_to_f16x2(x[2 * h]), e4m3x2_to_f16x2(x[2 * h + 1]),
                                   e4m3x2_hi_to_f16x2(x[2 * h]), e4m3x2_hi_to_f16x2(x[2 * h + 1])};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              uint2 y;
              if constexpr (WIDE)
                y = sq[((2 * k2 + h) * NT + n) * 32];
              else
                y = qf[2 * k2 + h][n];
              mma_16816_f16(s[t][n], a, y.x, y.y);
            }
          }
        }
      // scales of keys 16 t + 8 h + g; a key past the item's has score -inf and weight 0
      float kq[KT][2], vs[KT][2];
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = 16 * t + 8 * h + g;
          kq[t][h] = sc[key * HB] * qs;
          vs[t][h] = sc[F::kRows + key * HB];
        }
      if (left < kQ8WarpKeys) {
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (16 * t + 8 * h + g >= left) {
              kq[t][h] = 1.f;
#pragma unroll
              for (int n = 0; n < NT; ++n)
                s[t][n][2 * h] = s[t][n][2 * h + 1] = -CUDART_INF_F;
            }
      }
      uint32_t pt[KT][NT][2];  // P^T: columns are query rows, two keys a register
      uint64_t add[NT];
      auto weigh = [&]() {  // weights and sums under the present references; the largest magnitude
        float top = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          add[n] = 0ull;
#pragma unroll
          for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float e0, e1, w0, w1;
              f2_unpack(f2_fma(f2_pack(s[t][n][2 * h], s[t][n][2 * h + 1]),
                               f2_pack(kq[t][h], kq[t][h]), nm[n]), e0, e1);
              e0 = fast_exp2(e0);
              e1 = fast_exp2(e1);
              const uint64_t e = f2_pack(e0, e1);
              add[n] = f2_add(add[n], e);
              f2_unpack(f2_mul(f2_mul(e, f2_pack(vs[t][h], vs[t][h])), cw[n]), w0, w1);
              top = fmax3(top, e0, e1);
              top = fmax3(top, fabsf(w0), fabsf(w1));
              pt[t][n][h] = pack_f16(w0, w1);
            }
        }
        return top;
      };
      if (__any_sync(0xffffffffu, weigh() > 256.f)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float m[2], w[2], ls[2];
          f2_unpack(nm[n], m[0], m[1]);
          f2_unpack(cw[n], w[0], w[1]);
          f2_unpack(l[n], ls[0], ls[1]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float m_old = -m[j];
            const int ew = (int)(__float_as_uint(w[j]) >> 23) - 127;  // log2 c
            const float m2_old = w[j] == 0.f ? kUnset : m_old - (float)ew;
            float x1 = m_old, x2 = m2_old;
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float v = s[t][n][2 * h + j] * kq[t][h];
                x1 = fmaxf(x1, v);
                x2 = fmaxf(x2, v + lg2(fabsf(vs[t][h])));
              }
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
              x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
              x2 = fmaxf(x2, __shfl_xor_sync(0xffffffffu, x2, off));
            }
            // a column moves when it has to itself: another request's scores are no reason
            if (!(x1 > m_old + 8.f || x2 > m2_old + 8.f)) continue;
            // c = 2^en with weights of at most about 1.  The largest c while every V scale was 0 or
            // subnormal (lg2 flushes those): O is still 0, or as small as such scales make it, and
            // the first scale of any size either gives weights that fp16 holds or moves c.
            const int en = x2 == kUnset ? 126 : (int)rintf(fminf(fmaxf(x1 - x2, -126.f), 126.f));
            ls[j] *= fast_exp2(m_old - x1);
            const float a = w[j] == 0.f ? 0.f : fast_exp2(m_old - x1 + (float)(en - ew));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[i][n][j] *= a;
              o[i][n][2 + j] *= a;
            }
            m[j] = -x1;
            w[j] = __uint_as_float((uint32_t)(en + 127) << 23);
          }
          nm[n] = f2_pack(m[0], m[1]);
          cw[n] = f2_pack(w[0], w[1]);
          l[n] = f2_pack(ls[0], ls[1]);
        }
        weigh();
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        l[n] = f2_add(l[n], add[n]);
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) pt[t][n][h] = movm_t(pt[t][n][h]);
      }
#pragma unroll
      for (int t = 0; t < KT; ++t)
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
    if (lane == 0) tc::mbar_arrive(full + 8 * F::kStages);
  }

  // partial rows: split, KV head, row.  A split without keys has none (the merge knows).
  if (split * kQ8WarpKeys >= nkeys) return true;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float m[2], w[2], ls[2];
    f2_unpack(nm[n], m[0], m[1]);
    f2_unpack(cw[n], w[0], w[1]);
    f2_unpack(l[n], ls[0], ls[1]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) ls[j] += __shfl_xor_sync(0xffffffffu, ls[j], off);
      const int r = row0 + 8 * n + 2 * c + j;
      if (r >= rows || (far >> (8 * n + 2 * c + j) & 1u)) continue;
      const bool none = ls[j] == 0.f;
      const float f = none || w[j] == 0.f ? 0.f : 1.f / w[j] / ls[j];
      const int64_t row = (int64_t)it.part + ((int64_t)split * p.hkv + head) * rows + r;
      float* dst = p.part_o + row * kHeadDim + 2 * g;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<float2*>(dst + 16 * i) = make_float2(o[i][n][j] * f, o[i][n][2 + j] * f);
      if (g == 0) p.part_lse[row] = none ? -CUDART_INF_F : -m[j] + __log2f(ls[j]);
    }
  }
  for (; far; far &= far - 1)  // (the warp's lanes hold the same rows)
    run_far_row<WIDE, HBL>(p, it, head, split, rows, row0 + __ffs(far) - 1);
  return true;
}

template <bool WIDE, int HBL>
__global__ void __launch_bounds__(kThreads, 1) decode_q8_kernel(const Params p) {
  using F = Form<WIDE, HBL>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + F::kOffBar + 2 * F::kStages * 8);
  if (threadIdx.x == 0) {
    for (int i = 0; i < F::kStages; ++i) {
      tc::mbar_init(base + F::kOffBar + 8 * i, kProducers);
      tc::mbar_init(base + F::kOffBar + 8 * (F::kStages + i), kWarps);
    }
    *abort = 0;
  }
  __syncthreads();
  // (the plan is older than every kernel that this one may start beside; one request of 16,411 keys
  // 13.4 us instead of 13.7, 64 rows a head on 16,000 keys 280 instead of 285)
  if (const int first = item_at(p, 0); first >= 0)
    asm volatile("prefetch.global.L1 [%0];" ::"l"(p.items + first));
  // A narrow kernel behind a wide one starts beside it: the wide one's CTAs have all passed this
  // wait by then, so what came before the call is complete.
  if (WIDE || !p.after_wide) wait_for_predecessors();
  let_successors_start();
  if (threadIdx.x >= 32 * kWarps) {
    if constexpr (WIDE) tc::regs_dec<kRegsProducer>();
    producer<WIDE, HBL>(p, base, abort);
  } else {
    if constexpr (WIDE) tc::regs_inc<kRegsConsumer>();
    uint32_t gs = 0;
    for (int k = 0;; ++k) {
      const int idx = item_at(p, k);
      if (idx < 0) break;
      const DecItem it = p.items[idx];
      bool ok;
      if constexpr (WIDE)
        ok = run_item<4, WIDE, HBL>(p, it, base, smem, gs, abort);
      else
        ok = it.kind == 0 ? run_item<1, WIDE, HBL>(p, it, base, smem, gs, abort)
                          : run_item<2, WIDE, HBL>(p, it, base, smem, gs, abort);
      if (!ok) break;
    }
  }
  // the merge behind this kernel waits for this one only
  if constexpr (!WIDE)
    if (p.after_wide) wait_for_predecessors();
}

// W warps per (request, query head), W from the longest list of partials: warp w takes partials
// w, w + W, ... and a lane 4 of the 128 columns; the warps' sums meet in shared memory.
//   lse = log2 sum 2^lse_i,   o = sum 2^(lse_i - lse) o_i;
// a partial whose log-sum-exp is NaN makes both NaN.
// What bounds it is the latency of its reads, so a warp has kRows partial rows in flight: one after
// another (a branch on the weight around each read) the call on 16,411 keys of one request took
// 12.7 us instead of 11.3; the first references fetched beside the kernel before, 10.8.  Eight rows
// instead of four cost a warp with few partials 1 to 2 %.
constexpr int merge_warps(int w) { return w > 8 ? w : 8; }  // warps of a CTA
template <int W>
__global__ void __launch_bounds__(32 * merge_warps(W)) merge_q8_kernel(
    const float* __restrict__ part_o, const float* __restrict__ part_lse,
    const int32_t* __restrict__ merge_idx, const DecMergeRef* __restrict__ refs, int batch, int hq,
    int gq, const MergeRow* __restrict__ out, __nv_bfloat16* __restrict__ o,
    float* __restrict__ lse) {
  constexpr int kMergeWarps = merge_warps(W), kRows = W == 1 ? 4 : 8;
  __shared__ float4 s_acc[kMergeWarps][32];
  __shared__ float s_max[kMergeWarps], s_tot[kMergeWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, w = warp % W;
  const int64_t task = (int64_t)blockIdx.x * (kMergeWarps / W) + warp / W;
  // an entry of the merge index holds one row's partials, for all its query heads, or (out) those of
  // one KV head
  const int heads = out ? gq : hq;
  const bool live = task < (int64_t)batch * heads;
  const int b = live ? (int)(task / heads) : 0, h = live ? (int)(task % heads) : 0;
  const int hk = h / gq, g = h % gq;
  const int r_begin = merge_idx[b], n = live ? merge_idx[b + 1] - r_begin : 0;
  float mx = -CUDART_INF_F, tot = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  // (the plan was complete before the kernels of this call began, its partials are not)
  DecMergeRef first{0, 0, 0, 0};
  if (w + W * lane < n) first = refs[r_begin + w + W * lane];
  wait_for_predecessors();  // the partials are complete
  let_successors_start();
  // per chunk the lanes fetch one reference and log-sum-exp each, so every weight is known before
  // any row is read and the row reads are independent of one another
  for (int c0 = w; c0 < n; c0 += 32 * W) {
    const int i = c0 + W * lane;
    int64_t idx = 0;
    float li = -CUDART_INF_F;
    if (i < n) {
      const DecMergeRef rf = c0 == w ? first : refs[r_begin + i];
      idx = (int64_t)rf.part + (int64_t)hk * rf.rows_real + rf.row + g;
      li = part_lse[idx];
    }
    float cm = li;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, off));
    const float m_new = fmaxf(mx, cm);
    const float ref = m_new == -CUDART_INF_F ? 0.f : m_new;
    const float a = fast_exp2(mx - ref);  // exp2(-inf) = 0
    const float wi = li == -CUDART_INF_F ? 0.f : fast_exp2(li - ref);
    float ws = wi;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, off);
    tot = tot * a + ws;
    acc.x *= a;
    acc.y *= a;
    acc.z *= a;
    acc.w *= a;
    mx = m_new;
    // (behind the last partial the reads go to row 0; a row of weight zero may hold anything and is
    // not used)
    const int cnt = min(32, (n - c0 + W - 1) / W);
    for (int j0 = 0; j0 < cnt; j0 += kRows) {
      float wj[kRows];
      float4 v[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        wj[u] = __shfl_sync(0xffffffffu, wi, j0 + u);
        const int64_t ij = __shfl_sync(0xffffffffu, idx, j0 + u);
        v[u] = *reinterpret_cast<const float4*>(part_o + ij * kHeadDim + lane * 4);
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u)
        if (wj[u] != 0.f) {
          acc.x += wj[u] * v[u].x;
          acc.y += wj[u] * v[u].y;
          acc.z += wj[u] * v[u].z;
          acc.w += wj[u] * v[u].w;
        }
    }
  }
  if constexpr (W > 1) {
    s_acc[warp][lane] = acc;
    if (lane == 0) {
      s_max[warp] = mx;
      s_tot[warp] = tot;
    }
    __syncthreads();
    if (w != 0) return;
    float m = mx;
#pragma unroll
    for (int i = 1; i < W; ++i) m = fmaxf(m, s_max[warp + i]);
    const float ref = m == -CUDART_INF_F ? 0.f : m;
    tot = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float f = fast_exp2(s_max[warp + i] - ref);
      const float t = s_tot[warp + i];
      // (a warp of NaN scores only has the maximum -inf and a NaN sum)
      tot += s_max[warp + i] == -CUDART_INF_F ? t : t * f;
      const float4 v = s_acc[warp + i][lane];
      acc.x += v.x * f;
      acc.y += v.y * f;
      acc.z += v.z * f;
      acc.w += v.w * f;
    }
    mx = m;
  }
  if (!live) return;
  const float inv = tot == 0.f ? 0.f : 1.f / tot;
  const uint2 packed =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  int64_t row = (int64_t)b * hq + h;
  if (out) row = (int64_t)out[b].q_row * hq + out[b].kv_head * gq + g;
  *reinterpret_cast<uint2*>(o + row * kHeadDim + lane * 4) = packed;
  if (lane == 0)
    lse[row] =
        tot == 0.f ? -CUDART_INF_F
                   : ((mx == -CUDART_INF_F ? 0.f : mx) + __log2f(tot)) * 0.69314718055994530942f;
}

template <int W>
cudaError_t launch_merge(const uint8_t* base, const PlanHeader* h, int32_t n, int hq, int gq,
                         void* o, float* lse, cudaStream_t stream) {
  constexpr int kMergeWarps = merge_warps(W);
  const bool listed = h->n_merge_rows > 0;
  const int64_t tasks = (int64_t)n * (listed ? gq : hq);
  return launch_beside(merge_q8_kernel<W>,
                       dim3((unsigned)((tasks + kMergeWarps / W - 1) / (kMergeWarps / W))),
                       dim3(32 * kMergeWarps), 0, stream,
                       reinterpret_cast<const float*>(base + h->off_part_o),
                       reinterpret_cast<const float*>(base + h->off_part_lse),
                       reinterpret_cast<const int32_t*>(base + h->off_merge_idx),
                       reinterpret_cast<const DecMergeRef*>(base + h->off_merge), (int)n, hq, gq,
                       listed ? reinterpret_cast<const MergeRow*>(base + h->off_merge_rows)
                              : nullptr,
                       static_cast<__nv_bfloat16*>(o), lse);
}

template <bool WIDE, int HBL>
cudaError_t launch_partials(const Params& p, int grid, cudaStream_t stream) {
  // kernel attributes belong to the current device: set once per device (bit d of the mask)
  static std::atomic<uint64_t> attr_set{0};
  constexpr int kSmem = Form<WIDE, HBL>::kSmem;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!((attr_set.load() >> dev) & 1)) {
    // the wide form's register split balances only if every thread starts with kRegsLaunch (with
    // fewer the consumers would wait for registers that never come): any other build is refused
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, decode_q8_kernel<WIDE, HBL>);
    if (e != cudaSuccess) return e;
    if (WIDE && fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(decode_q8_kernel<WIDE, HBL>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    attr_set.fetch_or(1ull << dev);
  }
  return launch_beside(decode_q8_kernel<WIDE, HBL>, dim3(grid), dim3(kThreads), kSmem, stream, p);
}

}  // namespace

int launch_decode_q8(const rx_kv_desc* d, const PlanHeader* h, const rx_kv_q8* kv, const void* q,
                     void* o, float* lse, void* ws, void* stream) {
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
  p.scale_log2 = d->softmax_scale * 1.4426950408889634f;
  p.rows = reinterpret_cast<const int32_t*>(base + h->off_rows);
  p.part_o = reinterpret_cast<float*>(base + h->off_part_o);
  p.part_lse = reinterpret_cast<float*>(base + h->off_part_lse);
  p.pool_size = d->pool_size;
  p.status = reinterpret_cast<int32_t*>(base + offsetof(PlanHeader, status));
  cudaStream_t s = (cudaStream_t)stream;
  const int hbl = q8_head_block_log2(p.hkv);
  cudaError_t e = cudaSuccess;
  if (h->n_xitems > 0) {  // shared prefixes of very many rows
    uint8_t* stage = base + h->off_q8_stage;
    int x = launch_expand_q8(d, kv, reinterpret_cast<const Q8Tile*>(base + h->off_q8_tiles),
                             h->n_q8_tiles, stage, p.status, stream);
    if (!x)
      x = launch_tiles_q8(d, reinterpret_cast<const ExtItem*>(base + h->off_xitems),
                          reinterpret_cast<const ExtRow*>(base + h->off_xrows),
                          reinterpret_cast<const ExtSeg*>(base + h->off_xsegs), h->n_xitems, stage,
                          q, p.part_o, p.part_lse, p.status, stream);
    if (x) return x;
  }
  if (h->n_wide > 0) {
    p.items = reinterpret_cast<const DecItem*>(base + h->off_wide);
    p.cta_begin = reinterpret_cast<const int32_t*>(base + h->off_wide_cta);
    p.after_wide = false;
    e = hbl == 3   ? launch_partials<true, 2>(p, h->n_wide_ctas, s)
        : hbl == 2 ? launch_partials<true, 1>(p, h->n_wide_ctas, s)
                   : launch_partials<true, 0>(p, h->n_wide_ctas, s);
    if (e != cudaSuccess) return (int)e;
  }
  if (h->n_items > 0) {
    p.items = reinterpret_cast<const DecItem*>(base + h->off_items);
    p.cta_begin = reinterpret_cast<const int32_t*>(base + h->off_cta);
    p.after_wide = h->n_wide > 0;
    e = hbl == 3   ? launch_partials<false, 3>(p, h->n_ctas, s)
        : hbl == 2 ? launch_partials<false, 2>(p, h->n_ctas, s)
        : hbl == 1 ? launch_partials<false, 1>(p, h->n_ctas, s)
                   : launch_partials<false, 0>(p, h->n_ctas, s);
    if (e != cudaSuccess) return (int)e;
  }
  return h->batch > 0 ? launch_merge_q8(d, h, h->batch, o, lse, ws, stream) : 0;
}

int launch_merge_q8(const rx_kv_desc* d, const PlanHeader* h, int32_t n, void* o, float* lse,
                    void* ws, void* stream) {
  const uint8_t* base = static_cast<const uint8_t*>(ws);
  const int hq = d->num_q_heads, gq = hq / d->num_kv_heads;
  cudaStream_t s = (cudaStream_t)stream;
  if (h->n_merge_rows > 0) n = (int32_t)h->n_merge_rows;
  // One warp a row up to 8 partials, two up to 32, else eight; sixteen for no more rows than SMs (52
  // rows of some 130 partials: the call takes 12.6 us, with eight warps 14.5; 300 rows: 40.0 us, with
  // eight 38.0)
  const bool few = (int64_t)n * hq <= h->n_sms;
  return (int)(h->max_refs <= 8    ? launch_merge<1>(base, h, n, hq, gq, o, lse, s)
               : h->max_refs <= 32 ? launch_merge<2>(base, h, n, hq, gq, o, lse, s)
               : few               ? launch_merge<16>(base, h, n, hq, gq, o, lse, s)
                                   : launch_merge<8>(base, h, n, hq, gq, o, lse, s));
}

}  // namespace rx
