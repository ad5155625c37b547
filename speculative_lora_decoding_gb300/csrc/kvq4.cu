// The paged KV cache held in 4 bits: quantising a pass's K and V rows as they
// are written, and reading positions back in bf16.
//
// Layout (include/mlora.h): codes [num_blocks, H, block_size, D/2] and scales
// [num_blocks, H, block_size, D/16]; a head's tokens of one page lie side by
// side.  For a group of 16 values with largest magnitude amax
//   scale = E4M3(amax / (6 unit)),   code = E2M1(v / (scale unit)),
// fp32 with IEEE division, so that the codes follow from the inputs alone.
//
// Both kernels are copies that change the format: one thread per (row, K or V,
// head, group), 32 bytes of bf16 on one side and 8 + 1 bytes on the other, all
// of them contiguous across a warp within a head.
#include "common.cuh"
#include "e2m1.cuh"
#include "launch.h"

namespace mlora {

constexpr int KV4_THREADS = 256;

// The slot (block, offset) of a position through a request's table as the
// index of head 0's row, (block * H) * block_size + offset; -1 outside.
__device__ __forceinline__ long long kv4_slot(const Kv4 &c, int b, long long pos) {
  const long long j = pos / c.block_size;
  const int blk = pos >= 0 && j < c.max_blocks ? c.block_table[(size_t)b * c.max_blocks + j] : -1;
  if (blk < 0 || blk >= c.num_blocks) return -1;
  return (long long)blk * c.H * c.block_size + (pos - j * c.block_size);
}

// VEC: every row of y starts on a 16-byte boundary.
template <bool VEC>
__global__ void __launch_bounds__(KV4_THREADS) kv_write_q4_kernel(const Kv4Write a) {
  grid_launch_dependents();
  grid_dependency_wait();  // y comes from the projection just before
  const int GD = a.c.D / Q4_GROUP;
  const int per_row = 2 * a.c.H * GD;
  const long long n = (long long)a.M * per_row;
  for (long long i = (long long)blockIdx.x * KV4_THREADS + threadIdx.x; i < n; i += (long long)gridDim.x * KV4_THREADS) {
    const int m = (int)(i / per_row);
    int r = (int)(i - (long long)m * per_row);
    const int kv = r >= a.c.H * GD;
    r -= kv * a.c.H * GD;
    const int h = r / GD, g = r - h * GD;
    const int b = m / a.rows_per_req, t = m - b * a.rows_per_req;
    const int L = a.seq_len[b];
    if (L < 0) continue;  // unused request slot
    const long long slot = kv4_slot(a.c, b, (long long)L + a.t0 + t);
    if (slot < 0) {
      raise_status(a.c.status, MLORA_DEV_BAD_SLOT);
      continue;
    }
    const uint16_t *src = a.y + (size_t)m * a.ld + a.col[kv] + h * a.c.D + g * Q4_GROUP;
    uint32_t w[8];
    if (VEC) {
      const uint4 v0 = __ldg(reinterpret_cast<const uint4 *>(src));
      const uint4 v1 = __ldg(reinterpret_cast<const uint4 *>(src) + 1);
      w[0] = v0.x; w[1] = v0.y; w[2] = v0.z; w[3] = v0.w;
      w[4] = v1.x; w[5] = v1.y; w[6] = v1.z; w[7] = v1.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = (uint32_t)src[2 * e] | ((uint32_t)src[2 * e + 1] << 16);
    }
    // The largest magnitude by its bits: a NaN's lie above every number's, so
    // a NaN anywhere in the group reaches the scale.
    uint32_t mx = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = max(mx, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
    const float unit = a.c.unit[kv];
    const uint32_t sc = cvt_e4m3(__fdiv_rn(__uint_as_float(mx << 16), 6.f * unit));
    const float s = e4m3_to_float(sc) * unit;
    uint2 codes = make_uint2(0u, 0u);
    if (s != 0.f) {
      float v[8];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[2 * e] = __fdiv_rn(__uint_as_float(w[4 * half + e] << 16), s);
          v[2 * e + 1] = __fdiv_rn(__uint_as_float(w[4 * half + e] & 0xFFFF0000u), s);
        }
        (half ? codes.y : codes.x) = cvt_e2m1x8(v);
      }
    }
    const size_t row = (size_t)(slot + (long long)h * a.c.block_size);
    *reinterpret_cast<uint2 *>(a.c.codes[kv] + row * (a.c.D / 2) + g * 8) = codes;
    a.c.scales[kv][row * GD + g] = (uint8_t)sc;
  }
}

__global__ void __launch_bounds__(KV4_THREADS) kv_read_q4_kernel(const Kv4Read a) {
  grid_launch_dependents();
  grid_dependency_wait();  // the cache may come from the write just before
  const int GD = a.c.D / Q4_GROUP;
  const int per_row = a.c.H * GD;
  const long long per = (long long)a.c.B * a.rows * per_row, n = 2 * per;
  for (long long i = (long long)blockIdx.x * KV4_THREADS + threadIdx.x; i < n; i += (long long)gridDim.x * KV4_THREADS) {
    const int kv = i >= per;
    const long long o = i - (kv ? per : 0);
    const int m = (int)(o / per_row);
    const int r = (int)(o - (long long)m * per_row);
    const int h = r / GD, g = r - h * GD;
    const int b = m / a.rows, t = m - b * a.rows;
    const int L = a.start[b];
    const long long pos = (long long)L + t;
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    if (L >= 0 && pos < a.end[b]) {
      const long long slot = kv4_slot(a.c, b, pos);
      if (slot < 0) {
        raise_status(a.c.status, MLORA_DEV_BAD_SLOT);
      } else {
        const size_t row = (size_t)(slot + (long long)h * a.c.block_size);
        const uint2 codes = __ldg(reinterpret_cast<const uint2 *>(a.c.codes[kv] + row * (a.c.D / 2) + g * 8));
        const float s = e4m3_to_float(__ldg(a.c.scales[kv] + row * GD + g));
        const float unit = a.c.unit[kv];
        uint32_t w[8];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t f[4];
          e2m1x8_to_f16(half ? codes.y : codes.x, f);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            // code * scale is exact; the product with unit is rounded to fp32
            // (exact for a power of two), then once to bf16.
            w[4 * half + e] = (uint32_t)float_to_bf16_bits(f16_lo(f[e]) * s * unit) |
                              ((uint32_t)float_to_bf16_bits(f16_hi(f[e]) * s * unit) << 16);
        }
        lo = make_uint4(w[0], w[1], w[2], w[3]);
        hi = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
    uint4 *dst = reinterpret_cast<uint4 *>(a.out[kv] + (size_t)o * Q4_GROUP);
    dst[0] = lo;
    dst[1] = hi;
  }
}

static unsigned kv4_grid(long long n, int num_sms) {
  const long long want = (n + KV4_THREADS - 1) / KV4_THREADS, cap = (long long)num_sms * 8;
  return (unsigned)(want < cap ? want : cap);
}

cudaError_t launch_kv_write_q4(const Kv4Write &a, int num_sms, cudaStream_t s) {
  if (a.M <= 0) return cudaSuccess;
  const unsigned grid = kv4_grid((long long)a.M * 2 * a.c.H * (a.c.D / Q4_GROUP), num_sms);
  const bool vec = a.ld % 8 == 0 && a.col[0] % 8 == 0 && a.col[1] % 8 == 0 && ((uintptr_t)a.y & 15u) == 0;
  if (vec) return launch_pdl(kv_write_q4_kernel<true>, dim3(grid), dim3(KV4_THREADS), 0, s, a);
  return launch_pdl(kv_write_q4_kernel<false>, dim3(grid), dim3(KV4_THREADS), 0, s, a);
}

cudaError_t launch_kv_read_q4(const Kv4Read &a, int num_sms, cudaStream_t s) {
  if (a.rows <= 0) return cudaSuccess;
  const unsigned grid = kv4_grid(2ll * a.c.B * a.rows * a.c.H * (a.c.D / Q4_GROUP), num_sms);
  return launch_pdl(kv_read_q4_kernel, dim3(grid), dim3(KV4_THREADS), 0, s, a);
}

}  // namespace mlora
