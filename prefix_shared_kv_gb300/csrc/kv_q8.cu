// rx_store_kv_q8 / rx_load_kv_q8: the 8-bit pool's scatter and gather.
//
// A row is the 128 values of one (token, KV head) of K or of V.  With a = max |x| over the row:
//   scale = max(a / 448, 2^-126),  code = e4m3(x * r),  r = 448 / a  (2^126 at the scale's floor),
// so the largest value takes the largest code, 448.  A code is within half an e4m3 step of x / scale
// but for the float32 roundings of scale, r and x r (together 3 x 2^-24 of the value): a value that
// close to a tie may go to either side of it.  448 is e4m3's largest value; the floor keeps scale and
// r normal numbers, for a row of zeros too.  Reading back is code * scale, rounded once to bf16.  A
// row with an infinity or a NaN has no such scale: its scale is NaN and its codes 0, so it reads as
// NaN.
//
// Both kernels move data: 256 + 132 bytes a row.  Eight lanes share a row, so that a lane's bf16 side
// is a 32-byte access (two of 16 where the tensor is not 32-byte aligned), its codes a 16-byte one,
// and a row's maximum takes three shuffles; K and V are the two halves of the grid's y axis, and a thread has the loads of all its rows in
// flight before the first is used.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pdl.cuh"
#include "ptx.cuh"
#include "rx_internal.h"

namespace rx {
namespace {

constexpr int kThreads = 256;
constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126

// Two fp32 values -> two e4m3 codes (round to nearest even, saturating), lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 32 bytes at once (the address 32-byte aligned), or as two halves.
template <bool B32>
__device__ __forceinline__ void ld32b(const uint4* p, uint4 (&x)[2]) {
  if constexpr (B32) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(x[0].x), "=r"(x[0].y), "=r"(x[0].z), "=r"(x[0].w), "=r"(x[1].x),
                   "=r"(x[1].y), "=r"(x[1].z), "=r"(x[1].w)
                 : "l"(p));
  } else {
    x[0] = __ldcs(p);
    x[1] = __ldcs(p + 1);
  }
}
template <bool B32>
__device__ __forceinline__ void st32b(uint4* p, const uint4 (&x)[2]) {
  if constexpr (B32) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0].x),
                 "r"(x[0].y), "r"(x[0].z), "r"(x[0].w), "r"(x[1].x), "r"(x[1].y), "r"(x[1].z),
                 "r"(x[1].w)
                 : "memory");
  } else {
    p[0] = x[0];
    p[1] = x[1];
  }
}

// A position in the flat list of rows, moved on by a fixed stride without divisions.
struct RowIter {
  int64_t row, token;
  int head;
  __device__ RowIter(int64_t r, int hkv) : row(r), token(r / hkv), head((int)(r - token * hkv)) {}
  __device__ void step(int64_t rows, int64_t tokens, int heads, int hkv) {
    row += rows;
    token += tokens;
    head += heads;
    if (head >= hkv) {
      head -= hkv;
      ++token;
    }
  }
};

template <int U, bool B32>
__global__ void __launch_bounds__(kThreads) store_q8_kernel(
    uint8_t* __restrict__ k_code, uint8_t* __restrict__ v_code, float* __restrict__ k_scale,
    float* __restrict__ v_scale, const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
    const int32_t* __restrict__ slots, int64_t n_rows, int hkv, int64_t pool_size) {
  const bool is_v = blockIdx.y != 0;
  const uint4* src = is_v ? v_new : k_new;
  uint8_t* code = is_v ? v_code : k_code;
  float* scale = is_v ? v_scale : k_scale;
  const int l = threadIdx.x & 7;  // lane of the row: values 16 l .. 16 l + 15
  const int64_t stride = (int64_t)gridDim.x * (kThreads / 8);
  const int64_t st_tokens = stride / hkv;
  const int st_heads = (int)(stride - st_tokens * hkv);
  RowIter it((int64_t)blockIdx.x * (kThreads / 8) + threadIdx.x / 8, hkv);
  wait_for_predecessors();
  let_successors_start();
  // the eight lanes of a row leave together; a warp's four rows may not, hence the group's mask
  const uint32_t group = 0xffu << (threadIdx.x & 24);
  while (it.row < n_rows) {
    uint4 x[U][2];
    int64_t dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      dst[u] = -1;
      x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
      if (it.row < n_rows) {
        const int64_t s = __ldg(slots + it.token);
        if (s >= 0 && s < pool_size) {
          dst[u] = s * hkv + it.head;
          ld32b<B32>(src + it.row * 16 + 2 * l, x[u]);
        }
      }
      it.step(stride, st_tokens, st_heads, hkv);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t w[8] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w,
                             x[u][1].x, x[u][1].y, x[u][1].z, x[u][1].w};
      // the order of bf16 magnitudes is that of their bits; an infinity or a NaN ends at 0x7f80
      // or above
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
#pragma unroll
      for (int off = 1; off < 8; off <<= 1) m = __vmaxu2(m, __shfl_xor_sync(group, m, off));
      const uint32_t top = max(m & 0xffffu, m >> 16);
      const float a = __uint_as_float(top << 16);
      const bool fine = top < 0x7f80u;
      const float sc = fmaxf(a / kE4m3Max, kMinScale);
      const float r = sc > kMinScale ? kE4m3Max / a : 1.f / kMinScale;
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = e4m3x2(bf_lo(w[2 * i]) * r, bf_hi(w[2 * i]) * r) |
               e4m3x2(bf_lo(w[2 * i + 1]) * r, bf_hi(w[2 * i + 1]) * r) << 16;
        if (!fine) c[i] = 0;
      }
      if (dst[u] >= 0) {
        *reinterpret_cast<uint4*>(code + dst[u] * kHeadDim + 16 * l) =
            make_uint4(c[0], c[1], c[2], c[3]);
        if (l == 0) scale[dst[u]] = fine ? sc : __uint_as_float(0x7fc00000u);
      }
    }
  }
}

template <int U, bool B32>
__global__ void __launch_bounds__(kThreads) load_q8_kernel(
    const uint8_t* __restrict__ k_code, const uint8_t* __restrict__ v_code,
    const float* __restrict__ k_scale, const float* __restrict__ v_scale,
    const int32_t* __restrict__ slots, uint4* __restrict__ k_out, uint4* __restrict__ v_out,
    int64_t n_rows, int hkv, int64_t pool_size) {
  const bool is_v = blockIdx.y != 0;
  const uint8_t* code = is_v ? v_code : k_code;
  const float* scale = is_v ? v_scale : k_scale;
  uint4* out = is_v ? v_out : k_out;
  const int l = threadIdx.x & 7;  // lane of the row: values 16 l .. 16 l + 15
  const int64_t stride = (int64_t)gridDim.x * (kThreads / 8);
  const int64_t st_tokens = stride / hkv;
  const int st_heads = (int)(stride - st_tokens * hkv);
  RowIter it((int64_t)blockIdx.x * (kThreads / 8) + threadIdx.x / 8, hkv);
  int64_t src[U];  // rows of the pool of the next U, -1: none, or outside the pool (zeros)
  auto fetch = [&]() {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      src[u] = -1;
      if (it.row < n_rows) {
        const int64_t s = __ldg(slots + it.token);
        if (s >= 0 && s < pool_size) src[u] = s * hkv + it.head;
      }
      it.step(stride, st_tokens, st_heads, hkv);
    }
  };
  int64_t first = it.row;
  wait_for_predecessors();
  let_successors_start();
  fetch();
  for (; first < n_rows; first += U * stride) {
    uint4 c[U];
    float sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      c[u] = make_uint4(0, 0, 0, 0);
      sc[u] = 0.f;
      if (src[u] >= 0) {
        c[u] = __ldg(reinterpret_cast<const uint4*>(code + src[u] * kHeadDim) + l);
        sc[u] = __ldg(scale + src[u]);
      }
    }
    fetch();  // the next rows' slots, behind this round's codes
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = first + u * stride;
      if (row >= n_rows) break;
      const uint32_t w[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
      uint32_t y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = e4m3x2_to_f32(i & 1 ? w[i >> 1] >> 16 : w[i >> 1]);
        y[i] = pack_bf16(f.x * sc[u], f.y * sc[u]);
      }
      const uint4 o[2] = {make_uint4(y[0], y[1], y[2], y[3]), make_uint4(y[4], y[5], y[6], y[7])};
      st32b<B32>(out + row * 16 + 2 * l, o);
    }
  }
}

// Four e4m3 codes -> four bf16 (exact).  A code's seven magnitude bits, put under the sign of a bf16
// four bits up, are the value times 2^-120 (the exponent biases are 7 and 127; subnormal codes give
// subnormal bf16 numbers): one product restores it.
__device__ __forceinline__ uint2 e4m3x4_to_bf16(uint32_t w) {
  const __nv_bfloat162 up = __halves2bfloat162(__ushort_as_bfloat16(0x7B80),
                                               __ushort_as_bfloat16(0x7B80));  // 2^120
  const uint32_t t[2] = {__byte_perm(w, 0, 0x1404), __byte_perm(w, 0, 0x3424)};
  uint32_t r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = ((t[i] >> 4) & 0x07f007f0u) | (t[i] & 0x80008000u);
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), up);
    r[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint2(r[0], r[1]);
}

// The expanded segments that the tensor-core extend kernel reads (layout at Q8Tile).  One CTA per
// tile of 64 keys and group of up to four KV heads: a lane turns 16 codes of a row of K and of V
// into two 16-byte chunks of the operand's image; a row's codes are read by eight neighbouring
// lanes, neighbouring heads of a key behind one another.  Moves 128 + 256 bytes a row.
// (Heads a CTA: 2, 4 and 8 within 1 %, 16 2 % slower on 32 heads.)
constexpr int kExpandHeads = 4;
__global__ void __launch_bounds__(kThreads) expand_q8_kernel(
    const uint8_t* __restrict__ k_code, const uint8_t* __restrict__ v_code,
    const float* __restrict__ k_scale, const float* __restrict__ v_scale,
    const int32_t* __restrict__ req_to_token, int64_t stride, int64_t pool_size, int hkv,
    float scale_log2, const Q8Tile* __restrict__ tiles, uint8_t* __restrict__ stage,
    int32_t* status) {
  __shared__ int32_t s_slot[kAttnKeys];
  __shared__ uint32_t s_special[kExpandHeads];
  const Q8Tile tile = tiles[blockIdx.x];
  const int head0 = blockIdx.y * kExpandHeads, nh = min(kExpandHeads, hkv - head0);
  wait_for_predecessors();
  if (threadIdx.x < kAttnKeys) {
    int s = -1;  // past the segment, or outside the pool (flagged): zeros
    if ((int)threadIdx.x < tile.n_keys) {
      s = __ldg(req_to_token + (int64_t)tile.kv_row * stride + tile.k_begin + threadIdx.x);
      if (s < 0 || s >= pool_size) {
        atomicCAS(status, 0, (int)RX_ERR_RANGE);
        s = -1;
      }
    }
    s_slot[threadIdx.x] = s;
  }
  if (threadIdx.x < kExpandHeads) s_special[threadIdx.x] = 0;
  __syncthreads();
  let_successors_start();
  uint8_t* blocks = stage + ((int64_t)blockIdx.x * hkv + head0) * kQ8BlockBytes;
  for (int i = threadIdx.x; i < kAttnKeys * nh; i += kThreads) {
    const int key = i / nh, h = i - key * nh;
    const int64_t row = (int64_t)s_slot[key] * hkv + head0 + h;
    const bool ok = s_slot[key] >= 0;
    float* sc = reinterpret_cast<float*>(blocks + (int64_t)h * kQ8BlockBytes + kQ8BlockV) -
                kAttnKeys + key;
    sc[0] = ok ? __ldg(k_scale + row) * scale_log2 : 0.f;
    const float v = ok ? __ldg(v_scale + row) : 0.f;
    sc[kQ8BlockV / 4] = v;
    if (!isfinite(v)) s_special[h] = 1;  // (every writer writes the same)
  }
  const int n = kAttnKeys * nh * 8;
  constexpr int U = 4;
  for (int i0 = threadIdx.x; i0 < n; i0 += U * kThreads) {
    uint4 x[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads;
      x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
      if (i < n) {
        const int f = i >> 3, key = f / nh, h = f - key * nh;
        const int slot = s_slot[key];
        if (slot >= 0) {
          const int64_t off = ((int64_t)slot * hkv + head0 + h) * kHeadDim + 16 * (i & 7);
          x[u][0] = __ldg(reinterpret_cast<const uint4*>(k_code + off));
          x[u][1] = __ldg(reinterpret_cast<const uint4*>(v_code + off));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= n) break;
      const int c = i & 7, f = i >> 3, key = f / nh, h = f - key * nh;
      // chunks 2c and 2c + 1 of the row: half c / 4, swizzled by the row's low three bits
      uint8_t* dst = blocks + (int64_t)h * kQ8BlockBytes + (c >> 2) * (kAttnKeys * 128) + key * 128;
      dst += (((2 * c) & 6) ^ (key & 6)) << 4;  // the two chunks' 32 bytes; an odd row swaps them
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint2 a = e4m3x4_to_bf16(x[u][v].x), b = e4m3x4_to_bf16(x[u][v].y);
        const uint2 e = e4m3x4_to_bf16(x[u][v].z), g = e4m3x4_to_bf16(x[u][v].w);
        const uint4 lo = make_uint4(a.x, a.y, b.x, b.y), hi = make_uint4(e.x, e.y, g.x, g.y);
        const uint4 y[2] = {key & 1 ? hi : lo, key & 1 ? lo : hi};
        st32b<true>(reinterpret_cast<uint4*>(dst + v * kQ8BlockV), y);
      }
    }
  }
  __syncthreads();
  if ((int)threadIdx.x < nh)
    *reinterpret_cast<uint32_t*>(blocks + (int64_t)threadIdx.x * kQ8BlockBytes + 2 * kQ8BlockV) =
        s_special[threadIdx.x];
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

// Launch shapes (GB300, K and V each).  Many rows: four a thread in flight and two CTAs per SM;
// 13,064 tokens x 32 heads stored take 53.5 us so, 54.9 with two rows a thread, 58.4 with four CTAs
// per SM; 32,003 x 32 read back 124.7 us, 129.6 with four CTAs, 126.6 with two rows and four CTAs.
// Few rows, up to what the GPU holds at once with one row per eight lanes (32 a CTA, four of an SM's
// eight CTAs for K and four for V): one, and as many CTAs as that makes; 40 tokens x 32 heads stored
// take 1.6 us so, 3.0 with four rows.
constexpr int kManyRows = 4, kManyCtas = 2;
bool few_rows(int64_t rows, int sms) { return rows <= (int64_t)sms * (2048 / kThreads / 2) * (kThreads / 8); }

// One x column per kThreads / 8 * u rows, at most `most`; y: K, V.
dim3 rows_grid(int64_t rows, int u, int64_t most) {
  const int64_t per = (int64_t)(kThreads / 8) * u, blocks = (rows + per - 1) / per;
  return dim3((unsigned)(blocks < most ? blocks : most), 2);
}

}  // namespace

int launch_store_kv_q8(const rx_kv_desc* d, const rx_kv_q8* kv, const void* k_new,
                       const void* v_new, const int32_t* slots, int64_t n, void* stream) {
  if (n == 0) return 0;
  const int64_t rows = n * d->num_kv_heads;
  const int sms = sm_count();
  if (sms == 0) return (int)cudaGetLastError();
  const bool b32 = ((reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) & 31) == 0;
  auto run = [&](auto kernel, int u) {
    return (int)launch_beside(
        kernel, rows_grid(rows, u, u == 1 ? rows : kManyCtas * sms), dim3(kThreads), 0,
        (cudaStream_t)stream, (uint8_t*)kv->k_code, (uint8_t*)kv->v_code, kv->k_scale, kv->v_scale,
        (const uint4*)k_new, (const uint4*)v_new, slots, rows, d->num_kv_heads, d->pool_size);
  };
  if (few_rows(rows, sms)) return b32 ? run(store_q8_kernel<1, true>, 1) : run(store_q8_kernel<1, false>, 1);
  return b32 ? run(store_q8_kernel<kManyRows, true>, kManyRows)
             : run(store_q8_kernel<kManyRows, false>, kManyRows);
}

int launch_load_kv_q8(const rx_kv_desc* d, const rx_kv_q8* kv, const int32_t* slots, int64_t n,
                      void* k_out, void* v_out, void* stream) {
  if (n == 0) return 0;
  const int64_t rows = n * d->num_kv_heads;
  const int sms = sm_count();
  if (sms == 0) return (int)cudaGetLastError();
  const bool b32 = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31) == 0;
  auto run = [&](auto kernel, int u) {
    return (int)launch_beside(
        kernel, rows_grid(rows, u, u == 1 ? rows : kManyCtas * sms), dim3(kThreads), 0,
        (cudaStream_t)stream, (const uint8_t*)kv->k_code, (const uint8_t*)kv->v_code, kv->k_scale,
        kv->v_scale, slots, (uint4*)k_out, (uint4*)v_out, rows, d->num_kv_heads, d->pool_size);
  };
  if (few_rows(rows, sms)) return b32 ? run(load_q8_kernel<1, true>, 1) : run(load_q8_kernel<1, false>, 1);
  return b32 ? run(load_q8_kernel<kManyRows, true>, kManyRows)
             : run(load_q8_kernel<kManyRows, false>, kManyRows);
}

int launch_expand_q8(const rx_kv_desc* d, const rx_kv_q8* kv, const Q8Tile* tiles, int32_t n_tiles,
                     void* stage, int32_t* status, void* stream) {
  const dim3 grid(n_tiles, (d->num_kv_heads + kExpandHeads - 1) / kExpandHeads);
  return (int)launch_beside(
      expand_q8_kernel, grid, dim3(kThreads), 0, (cudaStream_t)stream, (const uint8_t*)kv->k_code,
      (const uint8_t*)kv->v_code, kv->k_scale, kv->v_scale, d->req_to_token,
      d->req_to_token_stride, d->pool_size, d->num_kv_heads,
      d->softmax_scale * 1.4426950408889634f, tiles, (uint8_t*)stage, status);
}

}  // namespace rx
