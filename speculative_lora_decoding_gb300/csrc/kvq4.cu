// The paged KV cache held in 4 bits: quantising a pass's K and V rows as they
// are written, and reading positions back in bf16.
//
// Layout (include/mlora.h): codes [num_blocks, H, block_size, D/2] and scales
// [num_blocks, H, block_size, D/16]; a head's tokens of one page lie side by
// side.  For a group of 16 values with largest magnitude amax
//   scale = E4M3(amax / (6 unit)),   code = E2M1(v / (scale unit)),
// fp32 with IEEE division, so that the codes follow from the inputs alone.
//
// Both kernels are copies that change the format and are bound by HBM: a row
// of the pass (a position, with all heads of K and V) per slice of threads, a
// thread per group of 16: 32 bytes of bf16 on one side and 8 + 1 bytes on the
// other.  What a thread's group fixes (K or V, head, place in the row) stays
// the same from row to row, and a row's slot and values are asked for a row ahead.
//
// Measured, 8 requests of 4096 rows, 8 heads of 128: written in 31 us (0.82 of the
// copy bandwidth), all read back (behind up to 2000 positions) in 42 us (0.53); a
// third of what the instructions wait for is the conversions' pipe.
#include <climits>
#include <cmath>

#include "common.cuh"
#include "e2m1.cuh"
#include "launch.h"

namespace mlora {

constexpr int KV4_THREADS = 256;

// The slot (block, offset) of a position through a request's table as the
// index of head 0's row, (block * H) * block_size + offset; -1 outside.
__device__ __forceinline__ int kv4_slot(const Kv4 &c, int b, long long pos) {
  const long long j = pos >= 0 && pos <= INT32_MAX ? (long long)((uint32_t)pos / (uint32_t)c.block_size) : c.max_blocks;
  const int blk = j < c.max_blocks ? __ldg(c.block_table + (size_t)b * c.max_blocks + j) : -1;
  if (blk < 0 || blk >= c.num_blocks) return -1;
  return blk * c.H * c.block_size + (int)(pos - j * c.block_size);
}

// x / d for a code or a scale, r about 1 / d.  EXACT: IEEE division.  Otherwise
// the unit is a power of two.  Then x has 8 significant bits, a scale 4 and a
// border between two codes 3, or 6 unit has 2 and a border between two scales
// 5: a quotient that is not on a border is at least 2^-8 of it away, so x r,
// within 2^-21 of the quotient, rounded to 12 bits falls on the same side, or
// on the border itself.
template <bool EXACT>
__device__ __forceinline__ float kv4_ratio(float x, float d, float r) {
  if (EXACT) return __fdiv_rn(x, d);
  return __uint_as_float((__float_as_uint(x * r) + 0x800u) & 0xFFFFF000u);
}

// 1 / d within 2^-22, for d in the range of normal numbers.
__device__ __forceinline__ float rcp_approx(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return r;
}

// 32 bytes in one access (32-byte aligned).
__device__ __forceinline__ void ldg_32(const void *p, uint32_t (&w)[8]) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void stg_32(void *p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Slices of `lanes` threads, each with a row at a time.  VEC: every row of y
// starts on a 32-byte boundary.
template <bool VEC, bool EXACT>
__global__ void __launch_bounds__(KV4_THREADS) kv_write_q4_kernel(const Kv4Write a, int lanes) {
  grid_launch_dependents();
  grid_dependency_wait();  // y comes from the projection just before
  const int GD = a.c.D / Q4_GROUP, per = a.c.H * GD;
  const int slices = KV4_THREADS / lanes, slice = threadIdx.x / lanes, lane = threadIdx.x - slice * lanes;
  const int stride = gridDim.x * slices, m0 = blockIdx.x * slices + slice;
  auto slot_of = [&](int k) {  // of the walk's row k
    const long long m = m0 + (long long)k * stride;
    if (m >= a.M) return -1;
    const int b = (int)m / a.rows_per_req, t = (int)m - b * a.rows_per_req;
    const int L = __ldg(a.seq_len + b);
    if (L < 0) return -1;  // unused request slot
    const int slot = kv4_slot(a.c, b, (long long)L + a.t0 + t);
    if (slot < 0) raise_status(a.c.status, MLORA_DEV_BAD_SLOT);
    return slot;
  };
  // (whole warps: the last of them may have lanes without a group)
  for (int i = lane; (i & ~31) < 2 * per; i += lanes) {
    const bool mine = i < 2 * per;
    const int kv = i >= per, e = mine ? i - (kv ? per : 0) : 0, h = e / GD, g = e - h * GD;
    const float unit = (kv ? a.c.unit[1] : a.c.unit[0]), unit6 = 6.f * unit, inv6 = 1.f / unit6;
    const uint16_t *const y = a.y + (kv ? a.col[1] : a.col[0]) + e * Q4_GROUP;
    uint8_t *const codes = (kv ? a.c.codes[1] : a.c.codes[0]) + (size_t)h * a.c.block_size * (a.c.D / 2) + g * 8;
    uint8_t *const scales = (kv ? a.c.scales[1] : a.c.scales[0]) + (size_t)h * a.c.block_size * GD + g;
    auto fetch = [&](int row, uint32_t (&w)[8]) {
      if (row >= a.M) return;
      const uint16_t *src = y + (size_t)row * a.ld;
      if (VEC) {
        ldg_32(src, w);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = (uint32_t)src[2 * k] | ((uint32_t)src[2 * k + 1] << 16);
      }
    };
    uint32_t ahead[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    fetch(m0, ahead);
    // The slots of the warp's rows, 32 rows at a time: lane i looks up the i-th.
    int now = slot_of((int)(threadIdx.x & 31u)), first = 0;
    auto slot_at = [&](int k) {
      if (k - first >= 32) {
        first = k;
        now = slot_of(k + (int)(threadIdx.x & 31u));
      }
      return __shfl_sync(0xffffffffu, now, k - first);
    };
    for (int m = m0, k0 = 0; m < a.M; m += stride, ++k0) {
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = ahead[k];
      fetch(m + stride, ahead);
      const int slot = slot_at(k0);
      if (slot < 0 || !mine) continue;
      // The largest magnitude by its bits: a NaN's lie above every number's, so
      // a NaN anywhere in the group reaches the scale.
      uint32_t mx = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) mx = __vmaxu2(mx, w[k] & 0x7FFF7FFFu);
      mx = max(mx & 0xFFFFu, mx >> 16);
      const uint32_t sc =
          mx > 0x7F80u ? 0x7Fu : cvt_e4m3(kv4_ratio<EXACT>(__uint_as_float(mx << 16), unit6, inv6));
      const float s = e4m3_to_float(sc) * unit, r = EXACT ? 0.f : rcp_approx(s);
      uint2 c = make_uint2(0u, 0u);
      if (s != 0.f) {
        float v[8];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[2 * k] = kv4_ratio<EXACT>(__uint_as_float(w[4 * half + k] << 16), s, r);
            v[2 * k + 1] = kv4_ratio<EXACT>(__uint_as_float(w[4 * half + k] & 0xFFFF0000u), s, r);
          }
          (half ? c.y : c.x) = cvt_e2m1x8(v);
        }
      }
      *reinterpret_cast<uint2 *>(codes + (size_t)slot * (a.c.D / 2)) = c;
      scales[(size_t)slot * GD] = (uint8_t)sc;
    }
  }
}

template <bool VEC>
__global__ void __launch_bounds__(KV4_THREADS) kv_read_q4_kernel(const Kv4Read a, int lanes) {
  grid_launch_dependents();
  grid_dependency_wait();  // the cache may come from the write just before
  const int GD = a.c.D / Q4_GROUP, per = a.c.H * GD, M = a.c.B * a.rows;
  const int slices = KV4_THREADS / lanes, slice = threadIdx.x / lanes, lane = threadIdx.x - slice * lanes;
  const int stride = gridDim.x * slices, m0 = blockIdx.x * slices + slice;
  auto slot_of = [&](int k) {  // of the walk's row k
    const long long m = m0 + (long long)k * stride;
    if (m >= M) return -1;
    const int b = (int)m / a.rows, t = (int)m - b * a.rows;
    const int L = __ldg(a.start + b);
    const long long pos = (long long)L + t;
    if (L < 0 || pos >= __ldg(a.end + b)) return -1;
    const int slot = kv4_slot(a.c, b, pos);
    if (slot < 0) raise_status(a.c.status, MLORA_DEV_BAD_SLOT);
    return slot;
  };
  // (whole warps: the last of them may have lanes without a group)
  for (int i = lane; (i & ~31) < 2 * per; i += lanes) {
    const bool mine = i < 2 * per;
    const int kv = i >= per, e = mine ? i - (kv ? per : 0) : 0, h = e / GD, g = e - h * GD;
    const float unit = (kv ? a.c.unit[1] : a.c.unit[0]);
    const uint8_t *const codes = (kv ? a.c.codes[1] : a.c.codes[0]) + (size_t)h * a.c.block_size * (a.c.D / 2) + g * 8;
    const uint8_t *const scales = (kv ? a.c.scales[1] : a.c.scales[0]) + (size_t)h * a.c.block_size * GD + g;
    // The slots of the warp's rows, 32 rows at a time: lane i looks up the i-th.
    int now = slot_of((int)(threadIdx.x & 31u)), first = 0;
    auto slot_at = [&](int k) {
      if (k - first >= 32) {
        first = k;
        now = slot_of(k + (int)(threadIdx.x & 31u));
      }
      return __shfl_sync(0xffffffffu, now, k - first);
    };
    // A row's codes are asked for while the two before it are written.
    int slot[2];
    uint2 c[2];
    uint32_t sc[2];
    auto ask = [&](int k, int n) {
      slot[n] = slot_at(k);
      c[n] = make_uint2(0, 0);
      sc[n] = 0;
      if (slot[n] >= 0) {
        c[n] = __ldg(reinterpret_cast<const uint2 *>(codes + (size_t)slot[n] * (a.c.D / 2)));
        sc[n] = __ldg(scales + (size_t)slot[n] * GD);
      }
    };
    auto put = [&](long long m, int n) {
      if (m >= M || !mine) return;
      uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (slot[n] >= 0) {
        const float s = e4m3_to_float(sc[n]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t f[4];
          e2m1x8_to_f16(half ? c[n].y : c[n].x, f);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            // code * scale is exact; the product with unit is rounded to fp32
            // (exact for a power of two), then once to bf16.
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                : "=r"(w[4 * half + k])
                : "f"(f16_hi(f[k]) * s * unit), "f"(f16_lo(f[k]) * s * unit));
        }
      }
      uint4 *dst = reinterpret_cast<uint4 *>((kv ? a.out[1] : a.out[0]) + ((size_t)m * per + e) * Q4_GROUP);
      if (VEC) {
        stg_32(dst, w);
      } else {
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    };
    ask(0, 0);
    ask(1, 1);
    long long m = m0;
    for (int k = 0; m < M; k += 2, m += 2ll * stride) {
      put(m, 0);
      ask(k + 2, 0);
      put(m + stride, 1);
      ask(k + 3, 1);
    }
  }
}

// Threads to a row: a power of two, as many as its groups, 32 at least.
static int kv4_lanes(const Kv4 &c) {
  int lanes = 32;
  while (lanes < KV4_THREADS && lanes < 2 * c.H * (c.D / Q4_GROUP)) lanes *= 2;
  return lanes;
}

static unsigned kv4_grid(long long rows, int lanes, int num_sms) {
  const long long slices = KV4_THREADS / lanes, want = (rows + slices - 1) / slices, cap = (long long)num_sms * 8;
  return (unsigned)(want < cap ? want : cap);
}

cudaError_t launch_kv_write_q4(const Kv4Write &a, int num_sms, cudaStream_t s) {
  if (a.M <= 0) return cudaSuccess;
  const int lanes = kv4_lanes(a.c);
  const unsigned grid = kv4_grid(a.M, lanes, num_sms);
  const bool vec = a.ld % 16 == 0 && a.col[0] % 16 == 0 && a.col[1] % 16 == 0 && ((uintptr_t)a.y & 31u) == 0;
  // (1 / scale stays a normal number in this range)
  auto pow2 = [](float u) {
    int e;
    return std::frexp(u, &e) == 0.5f && e > -100 && e < 100;
  };
  const bool exact = !pow2(a.c.unit[0]) || !pow2(a.c.unit[1]);
  if (vec && !exact) return launch_pdl(kv_write_q4_kernel<true, false>, dim3(grid), dim3(KV4_THREADS), 0, s, a, lanes);
  if (vec) return launch_pdl(kv_write_q4_kernel<true, true>, dim3(grid), dim3(KV4_THREADS), 0, s, a, lanes);
  if (!exact) return launch_pdl(kv_write_q4_kernel<false, false>, dim3(grid), dim3(KV4_THREADS), 0, s, a, lanes);
  return launch_pdl(kv_write_q4_kernel<false, true>, dim3(grid), dim3(KV4_THREADS), 0, s, a, lanes);
}

cudaError_t launch_kv_read_q4(const Kv4Read &a, int num_sms, cudaStream_t s) {
  if (a.rows <= 0) return cudaSuccess;
  const int lanes = kv4_lanes(a.c);
  const unsigned grid = kv4_grid((long long)a.c.B * a.rows, lanes, num_sms);
  if ((((uintptr_t)a.out[0] | (uintptr_t)a.out[1]) & 31u) == 0)
    return launch_pdl(kv_read_q4_kernel<true>, dim3(grid), dim3(KV4_THREADS), 0, s, a, lanes);
  return launch_pdl(kv_read_q4_kernel<false>, dim3(grid), dim3(KV4_THREADS), 0, s, a, lanes);
}

}  // namespace mlora
