// Writing rows into a 4-bit cache and reading them back.
//
// Four lanes share a group of 32 values, eight values (16 bytes of the 16-bit
// row, one 32-bit word of codes) each, so a warp covers eight groups and both
// sides of the copy are contiguous.  The group's minimum and maximum are a
// two-step butterfly over the four lanes.  Both kernels move each byte once
// and are bound by HBM (a few launches' worth of rows) or by the launch.
//
// The code of a value is the correctly rounded fp32 quotient (x - min) /
// scale, rounded to nearest even: the borders between codes, (k + 1/2) *
// scale, are exact in fp32, so a correctly rounded quotient never falls on
// the wrong side of one.
#include <cuda_runtime.h>

#include "kernels.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace gqa {
namespace {

using namespace q4;

constexpr int kThreads = 256;

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// What one lane works on: eight values of a group of one row.
struct Piece {
  int kv, b, h, t, g, d0;  // tensor (0 K, 1 V), entry, head, row, group, first value
};

// Piece x of the 2 * B * H * n rows, 4 * G lanes each; rows fastest in t.
__device__ __forceinline__ Piece piece_of(uint32_t x, const Q4RowsArgs& a, int G) {
  Piece p;
  const uint32_t lanes = 4u * static_cast<uint32_t>(G);
  uint32_t row = x / lanes;
  const uint32_t r = x - row * lanes;
  p.g = static_cast<int>(r >> 2);
  p.d0 = static_cast<int>(r) * 8;
  uint32_t y = row / static_cast<uint32_t>(a.n);
  p.t = static_cast<int>(row - y * static_cast<uint32_t>(a.n));
  row = y;
  y = row / static_cast<uint32_t>(a.H);
  p.h = static_cast<int>(row - y * static_cast<uint32_t>(a.H));
  p.kv = y >= static_cast<uint32_t>(a.B) ? 1 : 0;
  p.b = static_cast<int>(y) - p.kv * a.B;
  return p;
}

// Byte offset of row j of entry b, head h in a cache, or -1: a page outside the pool.
__device__ __forceinline__ int64_t record_at(const Q4RowsArgs& a, int kv, int b, int h, int64_t j) {
  const int64_t* s = a.cs[kv];
  if (a.bt == nullptr) return b * s[0] + h * s[1] + j * s[2];
  const int64_t page = a.bt[b * a.bt_stride + j / a.page_size];
  if (page < 0 || page >= a.num_pages) return -1;
  return page * s[0] + h * s[1] + (j % a.page_size) * s[2];
}

// New rows of entry b, or -1 where they do not fit.
__device__ __forceinline__ int count_of(const Q4RowsArgs& a, int b, int64_t len) {
  const int c = a.counts != nullptr ? a.counts[b] : a.n;
  if (c < 0 || c > a.n || len < 0 || len > a.cap - c) return -1;
  return c;
}

template <bool F16>
__global__ void __launch_bounds__(kThreads) gqa_q4_append_kernel(const Q4RowsArgs a,
                                                                 const uint32_t pieces) {
  griddep_launch_dependents();  // as in the 16-bit append
  const int G = groups_of(a.D);
  // Every lane of a group's four takes the same branches (pieces is a
  // multiple of 4, and so is the stride).
  for (uint32_t x = blockIdx.x * kThreads + threadIdx.x; x < pieces; x += gridDim.x * kThreads) {
    const Piece p = piece_of(x, a, G);
    const uint32_t quad = 0xFu << (lane_id() & 28u);
    const int64_t len = a.lens[p.b];
    const int count = count_of(a, p.b, len);
    if (count < 0) {
      if (p.kv == 0 && p.h == 0 && p.t == 0 && p.d0 == 0) atomicOr(a.err, kErrKvLength);
      continue;
    }
    if (p.t >= count) continue;
    const int64_t at = record_at(a, p.kv, p.b, p.h, len + p.t);
    if (at < 0) {
      if (p.kv == 0 && p.h == 0 && p.d0 == 0) atomicOr(a.err, kErrPage);
      continue;
    }
    const int64_t* rs = a.rs[p.kv];
    const uint16_t* src = a.rows[p.kv] + p.b * rs[0] + p.h * rs[1] + p.t * rs[2] + p.d0;
    const bool live = p.d0 < a.D;  // head_dim is a multiple of 8
    uint16_t v[8];
    if (live) {
      if (a.vec) {
        *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(src);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = src[i];
      }
    }
    float f[8];
    float lo = INFINITY, hi = -INFINITY;
    if (live) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] = to_f32<F16>(v[i]);
        lo = min_nan(lo, f[i]);
        hi = max_nan(hi, f[i]);
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      lo = min_nan(lo, __shfl_xor_sync(quad, lo, o));
      hi = max_nan(hi, __shfl_xor_sync(quad, hi, o));
    }
    // Not finite where the group holds a NaN or an infinity, or its spread overflows.
    const float spread = __fsub_rn(hi, lo);
    const bool finite = fabsf(spread) <= 3.402823466e38f;
    const uint32_t s16 = finite ? to_16<F16>(__fdiv_rn(spread, 15.f)) : 0x7FFFu;
    const uint32_t m16 = finite ? to_16<F16>(lo) : 0x7FFFu;
    const float s = to_f32<F16>(s16);
    uint32_t word = 0;
    if (live && finite && s > 0.f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float c = fminf(rintf(__fdiv_rn(__fsub_rn(f[i], lo), s)), 15.f);
        word |= static_cast<uint32_t>(c) << (4 * i);
      }
    }
    uint8_t* rec = a.cache[p.kv] + at;
    const int lane4 = (p.d0 >> 3) & 3;
    *reinterpret_cast<uint32_t*>(rec + kHeadBytes + 16 * p.g + 4 * lane4) = word;
    // The group's parameters, and zeros in the head's slots that no group has.
    if (lane4 == 0) *reinterpret_cast<uint32_t*>(rec + 4 * p.g) = s16 | (m16 << 16);
    if (p.g == 0 && lane4 >= G) *reinterpret_cast<uint32_t*>(rec + 4 * lane4) = 0u;
  }
  if (!a.advance) return;

  __shared__ int last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == gridDim.x - 1 ? 1 : 0;
  }
  __syncthreads();
  if (last) {
    // Every CTA has read the lengths it needed: advance them.
    __threadfence();
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
      const int64_t len = a.lens[b];
      const int count = count_of(a, b, len);
      if (count <= 0) continue;
      bool pages_ok = true;
      if (a.bt != nullptr)
        for (int64_t pg = len / a.page_size; pg <= (len + count - 1) / a.page_size; ++pg) {
          const int64_t page = a.bt[b * a.bt_stride + pg];
          pages_ok = pages_ok && page >= 0 && page < a.num_pages;
        }
      if (pages_ok) a.lens[b] = static_cast<int32_t>(len + count);
    }
    if (threadIdx.x == 0) atomicExch(a.ticket, 0u);
  }
}

template <bool F16>
__global__ void __launch_bounds__(kThreads) gqa_q4_read_kernel(const Q4RowsArgs a,
                                                               const uint32_t pieces) {
  const int G = groups_of(a.D);
  for (uint32_t x = blockIdx.x * kThreads + threadIdx.x; x < pieces; x += gridDim.x * kThreads) {
    const Piece p = piece_of(x, a, G);
    if (p.d0 >= a.D) continue;
    const bool first = p.kv == 0 && p.h == 0 && p.t == 0 && p.d0 == 0;
    int64_t len = a.cap;
    if (a.lens != nullptr) {
      len = a.lens[p.b];
      if (len < 0 || len > a.cap) {
        if (first) atomicOr(a.err, kErrKvLength);
        len = len < 0 ? 0 : a.cap;
      }
    }
    const int64_t start = a.starts != nullptr ? a.starts[p.b] : a.start;
    if (start < 0 && first) atomicOr(a.err, kErrKvLength);
    const int64_t j = start + p.t;
    uint32_t out[4] = {0u, 0u, 0u, 0u};
    if (start >= 0 && j < len) {
      const int64_t at = record_at(a, p.kv, p.b, p.h, j);
      if (at < 0) {
        if (p.kv == 0 && p.h == 0 && p.d0 == 0) atomicOr(a.err, kErrPage);
      } else {
        const uint8_t* rec = a.cache[p.kv] + at;
        const uint32_t par = *reinterpret_cast<const uint32_t*>(rec + 4 * p.g);
        const uint32_t word = *reinterpret_cast<const uint32_t*>(rec + kHeadBytes + p.d0 / 2);
        const float s = scale_of<F16>(par), m = min_of<F16>(par);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          out[i] = pack2<F16>(fmaf(s, static_cast<float>((word >> (8 * i)) & 15u), m),
                              fmaf(s, static_cast<float>((word >> (8 * i + 4)) & 15u), m));
      }
    }
    const int64_t* rs = a.rs[p.kv];
    uint16_t* dst = a.rows[p.kv] + p.b * rs[0] + p.h * rs[1] + p.t * rs[2] + p.d0;
    if (a.vec) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dst[2 * i] = static_cast<uint16_t>(out[i] & 0xFFFFu);
        dst[2 * i + 1] = static_cast<uint16_t>(out[i] >> 16);
      }
    }
  }
}

uint32_t pieces_of(const Q4RowsArgs& a) {
  return 2u * static_cast<uint32_t>(a.B) * static_cast<uint32_t>(a.H) *
         static_cast<uint32_t>(a.n) * 4u * static_cast<uint32_t>(groups_of(a.D));
}

unsigned grid_of(uint32_t pieces) {
  const uint32_t blocks = (pieces + kThreads - 1) / kThreads;
  return blocks < 148u * 32u ? blocks : 148u * 32u;
}

}  // namespace

int launch_q4_append(const Q4RowsArgs& a, bool f16, cudaStream_t stream) {
  const uint32_t pieces = pieces_of(a);
  if (f16)
    gqa_q4_append_kernel<true><<<grid_of(pieces), kThreads, 0, stream>>>(a, pieces);
  else
    gqa_q4_append_kernel<false><<<grid_of(pieces), kThreads, 0, stream>>>(a, pieces);
  return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

int launch_q4_read(const Q4RowsArgs& a, bool f16, cudaStream_t stream) {
  const uint32_t pieces = pieces_of(a);
  if (f16)
    gqa_q4_read_kernel<true><<<grid_of(pieces), kThreads, 0, stream>>>(a, pieces);
  else
    gqa_q4_read_kernel<false><<<grid_of(pieces), kThreads, 0, stream>>>(a, pieces);
  return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace gqa
