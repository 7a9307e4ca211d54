// Writing rows into a 4-bit cache and reading them back.
//
// Append: one thread takes one group of 32 values (four 16-byte loads in
// flight, 16 bytes of codes and 4 of parameters out), or, where that would
// leave most of the machine idle, four threads share one (eight values each, a
// two-step butterfly for minimum and maximum): 4 x 4096 tokens of 8 heads take
// 29 us one way and 61 us the other, 16 single tokens the other way round
// 0.6 us less.  Consecutive threads take the groups of a row, then rows, so
// that a warp's loads and stores cover whole sectors.
//
// The code of a value is rint((x - min) / scale).  A division per value would
// cost more than the rest: the quotient is taken as a product with the
// reciprocal, at most one code off, and the remainder (x - min) - code *
// scale, exact in one fused multiply-add, says where: only when it reaches
// half a scale.  (The borders (k + 1/2) * scale are exact in fp32, so that the
// rounded quotient, too, is on a border only if the remainder is half a scale:
// ties go to the even code either way.)
//
// Read back: a thread takes eight dims (a 32-bit word of codes, 16 bytes out)
// of kRows rows, their loads all in flight before the first is used; nothing
// but the row changes between them (no division per piece).
//
// Both move each byte once: bound by HBM for long prompts (8 x 8192 rows of 8
// heads are read back in 76 us, 71% of the copy rate), by the launch for single
// tokens (append and read of 16: 4.9 us).
#include <cuda_runtime.h>

#include "kernels.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace gqa {
namespace {

using namespace q4;

constexpr int kThreads = 256;
constexpr double kManyPieces = 148.0 * 2048 * 4;

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

// Larger / smaller of two packed 16-bit pairs; a NaN stays.
template <bool F16>
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y) {
  uint32_t r;
  if (F16)
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  else
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t min2(uint32_t x, uint32_t y) {
  uint32_t r;
  if (F16)
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  else
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// Codes of eight values (four packed words), as the nibbles of one word.
template <bool F16>
__device__ __forceinline__ uint32_t codes_of(const uint32_t (&w)[4], float lo, float s, float r,
                                             float half) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
  uint32_t word = 0;
  bool near = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = __fsub_rn(to_f32<F16>((i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu), lo);
    const float c = __fmaf_rn(d, r, kMagic);
    const float rest = __fmaf_rn(-__fsub_rn(c, kMagic), s, d);
    near = near || fabsf(rest) >= half;
    word += __float_as_uint(c) << (4 * i);
  }
  word -= 0x4B400000u * 0x11111111u;  // the magic number's bits of all eight
  if (near) {
    word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = __fsub_rn(to_f32<F16>((i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu), lo);
      const float c = __fmaf_rn(d, r, kMagic);
      const float rest = __fmaf_rn(-__fsub_rn(c, kMagic), s, d);
      uint32_t n = __float_as_uint(c) - 0x4B400000u;
      const bool odd = (n & 1u) != 0u;
      if (rest > half || (rest == half && odd)) ++n;
      if (rest < -half || (rest == -half && odd)) --n;
      word |= n << (4 * i);
    }
  }
  return word;
}

// The same by division, clamped: for subnormal scales, whose reciprocal may be
// infinite and which may be far below a fifteenth of the spread.
template <bool F16>
__device__ __forceinline__ uint32_t codes_by_division(const uint32_t (&w)[4], float lo, float s) {
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = to_f32<F16>((i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu);
    word |= static_cast<uint32_t>(fminf(rintf(__fdiv_rn(__fsub_rn(x, lo), s)), 15.f)) << (4 * i);
  }
  return word;
}

// LPG: threads that share a group (1 or 4).
template <bool F16, int G, int LPG>
__global__ void __launch_bounds__(kThreads) gqa_q4_append_kernel(const Q4RowsArgs a) {
  // A decode launched after this one as a programmatic dependent may start its
  // prologue now; this kernel itself may have started before its predecessor
  // ended, and touches memory only after it has.
  griddep_launch_dependents();
  griddep_wait();
  constexpr int L = G * LPG, K = 4 / LPG;         // threads of a row; eight-value words of a thread
  const int rows_per_block = blockDim.x / L;      // (G = 3: a few threads idle)
  const int g = threadIdx.x % L / LPG, part = threadIdx.x % LPG, slot = threadIdx.x / L;
  // Words of this thread that lie below head_dim.
  const int words = min(K, (a.D - g * kGroup) / 8 - part * K);
  const uint32_t quad = 0xFu << (lane_id() & 28u);
  const int kv = blockIdx.z;
  for (int bh = blockIdx.y; bh < a.B * a.H; bh += gridDim.y) {
    const int b = bh / a.H, h = bh - b * a.H;
    const int64_t len = a.lens[b];
    const int count = count_of(a, b, len);
    if (count < 0) {
      if (kv == 0 && h == 0 && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, kErrKvLength);
      continue;
    }
    if (slot >= rows_per_block) continue;
    const int64_t* rs = a.rs[kv];
    const uint16_t* src = a.rows[kv] + b * rs[0] + h * rs[1] + g * kGroup + part * K * 8;
    // (The threads of a group take the same branches.)
    for (int t = blockIdx.x * rows_per_block + slot; t < count; t += gridDim.x * rows_per_block) {
      uint32_t w[K][4];  // [eight values][packed pair]
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const uint16_t* from = src + t * rs[2] + 8 * k;
        if (k >= words) {  // past head_dim: repeat, so that minimum and maximum hold
#pragma unroll
          for (int i = 0; i < 4; ++i) w[k][i] = k > 0 ? w[0][i] : 0u;
        } else if (a.vec) {
          const uint4 x = __ldcs(reinterpret_cast<const uint4*>(from));
          w[k][0] = x.x;
          w[k][1] = x.y;
          w[k][2] = x.z;
          w[k][3] = x.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[k][i] = from[2 * i] | (static_cast<uint32_t>(from[2 * i + 1]) << 16);
        }
      }
      const int64_t at = record_at(a, kv, b, h, len + t);
      if (at < 0) {
        if (kv == 0 && h == 0 && g == 0 && part == 0) atomicOr(a.err, kErrPage);
        continue;
      }
      uint32_t lo2 = w[0][0], hi2 = w[0][0];
#pragma unroll
      for (int i = 1; i < 4 * K; ++i) {
        lo2 = min2<F16>(lo2, w[i >> 2][i & 3]);
        hi2 = max2<F16>(hi2, w[i >> 2][i & 3]);
      }
      float lo = min_nan(to_f32<F16>(lo2 & 0xFFFFu), to_f32<F16>(lo2 >> 16));
      float hi = max_nan(to_f32<F16>(hi2 & 0xFFFFu), to_f32<F16>(hi2 >> 16));
      if (LPG > 1) {
        if (words <= 0) {
          lo = INFINITY;
          hi = -INFINITY;
        }
#pragma unroll
        for (int o = 1; o < LPG; o <<= 1) {
          lo = min_nan(lo, __shfl_xor_sync(quad, lo, o));
          hi = max_nan(hi, __shfl_xor_sync(quad, hi, o));
        }
      }
      // Not finite where the group holds a NaN or an infinity, or its spread overflows.
      const float spread = __fsub_rn(hi, lo);
      const bool finite = fabsf(spread) <= 3.402823466e38f;
      const uint32_t s16 = finite ? to_16<F16>(__fdiv_rn(spread, 15.f)) : 0x7FFFu;
      const uint32_t m16 = finite ? to_16<F16>(lo) : 0x7FFFu;
      const float s = to_f32<F16>(s16);
      uint32_t code[K];
#pragma unroll
      for (int k = 0; k < K; ++k) code[k] = 0u;
      if (finite && s > 0.f) {
        if (s >= (F16 ? 6.103515625e-05f : 1.17549435e-38f)) {  // a normal number of the type
          const float r = __frcp_rn(s), half = 0.5f * s;
#pragma unroll
          for (int k = 0; k < K; ++k)
            if (k < words) code[k] = codes_of<F16>(w[k], lo, s, r, half);
        } else {
#pragma unroll
          for (int k = 0; k < K; ++k)
            if (k < words) code[k] = codes_by_division<F16>(w[k], lo, s);
        }
      }
      uint8_t* rec = a.cache[kv] + at;
      if (LPG == 1)
        *reinterpret_cast<uint4*>(rec + kHeadBytes + 16 * g) =
            make_uint4(code[0], code[K / 4], code[K / 2], code[K - 1]);
      else
        *reinterpret_cast<uint32_t*>(rec + kHeadBytes + 16 * g + 4 * part) = code[0];
      if (part == 0) *reinterpret_cast<uint32_t*>(rec + 4 * g) = s16 | (m16 << 16);
      if (part == 0 && g == G - 1)  // the head's slots that no group has
        for (int i = G; i < 4; ++i) *reinterpret_cast<uint32_t*>(rec + 4 * i) = 0u;
    }
  }
  if (!a.advance) return;

  __shared__ int last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == gridDim.x * gridDim.y * gridDim.z - 1 ? 1 : 0;
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

template <bool F16, int G, int kRows>
__global__ void __launch_bounds__(kThreads) gqa_q4_read_kernel(const Q4RowsArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int L = 4 * G;
  const int per_pass = blockDim.x / L;
  const int piece = threadIdx.x % L, slot = threadIdx.x / L;
  const int d0 = piece * 8, g = piece >> 2;
  if (slot >= per_pass || d0 >= a.D) return;
  const int kv = blockIdx.z;
  for (int bh = blockIdx.y; bh < a.B * a.H; bh += gridDim.y) {
    const int b = bh / a.H, h = bh - b * a.H;
    const bool first = kv == 0 && h == 0 && blockIdx.x == 0 && threadIdx.x == 0;
    int64_t len = a.cap;
    if (a.lens != nullptr) {
      len = a.lens[b];
      if (len < 0 || len > a.cap) {
        if (first) atomicOr(a.err, kErrKvLength);
        len = len < 0 ? 0 : a.cap;
      }
    }
    const int64_t start = a.starts != nullptr ? a.starts[b] : a.start;
    if (start < 0) {
      if (first) atomicOr(a.err, kErrKvLength);
      len = start;
    }
    const int64_t* rs = a.rs[kv];
    uint16_t* dst = a.rows[kv] + b * rs[0] + h * rs[1] + d0;
    const int step = per_pass * kRows;
    const int64_t left = len - start;  // rows that exist, `held` of them asked for
    int held = left < 0 ? 0 : left < a.n ? static_cast<int>(left) : a.n;
    int n = a.n, low = 0, from = 0;  // [low, held) are read, the rest of [from, n) is zeros
    if (a.leave_tail) {
      n = held;
      if (len + a.to < held) {
        held = len + a.to > 0 ? static_cast<int>(len + a.to) : 0;
        n = min(n, (held + 127) / 128 * 128);
      }
      if (len + a.from > 0) low = len + a.from < held ? static_cast<int>(len + a.from) : held;
      from = low / 128 * 128;
    }
    for (int t0 = from + blockIdx.x * step; t0 < n; t0 += gridDim.x * step) {
      uint32_t par[kRows], word[kRows];
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int t = t0 + k * per_pass + slot;
        par[k] = word[k] = 0u;  // reads as zeros
        if (t < low || t >= held) continue;
        const int64_t at = record_at(a, kv, b, h, start + t);
        if (at < 0) {
          if (kv == 0 && h == 0 && d0 == 0) atomicOr(a.err, kErrPage);
          continue;
        }
        const uint8_t* rec = a.cache[kv] + at;
        par[k] = *reinterpret_cast<const uint32_t*>(rec + 4 * g);
        word[k] = *reinterpret_cast<const uint32_t*>(rec + kHeadBytes + d0 / 2);
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int t = t0 + k * per_pass + slot;
        if (t >= n) continue;
        const float s = scale_of<F16>(par[k]), m = min_of<F16>(par[k]);
        uint32_t out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          out[i] = pack2<F16>(fmaf(s, static_cast<float>((word[k] >> (8 * i)) & 15u), m),
                              fmaf(s, static_cast<float>((word[k] >> (8 * i + 4)) & 15u), m));
        uint16_t* to = dst + t * rs[2];
        if (a.vec) {
          *reinterpret_cast<uint4*>(to) = make_uint4(out[0], out[1], out[2], out[3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            to[2 * i] = static_cast<uint16_t>(out[i] & 0xFFFFu);
            to[2 * i + 1] = static_cast<uint16_t>(out[i] >> 16);
          }
        }
      }
    }
  }
}

template <typename Kernel>
int launch_rows(Kernel kern, const Q4RowsArgs& a, int per_row, int rows, cudaStream_t stream) {
  // per_row threads for a row, `rows` rows in turn per thread; blocks of as
  // many threads as a short run of rows has work for.
  const int64_t want = (static_cast<int64_t>(a.n) * per_row + 31) / 32 * 32;
  const int threads = want < kThreads ? static_cast<int>(want) : kThreads;
  const int64_t step = static_cast<int64_t>(threads / per_row) * rows;
  const int64_t bh = static_cast<int64_t>(a.B) * a.H;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((a.n + step - 1) / step),
                     static_cast<unsigned>(bh < 32768 ? bh : 32768), 2);
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  return GQA_OK;
}

// Whether there are several eight-value pieces for every thread that fits the
// machine: then a thread takes several of them; fewer are spread wide.
bool many_rows(const Q4RowsArgs& a, int G) {
  return 2.0 * a.B * a.H * a.n * 4 * G >= kManyPieces;
}

template <bool F16, int G>
int append_g(const Q4RowsArgs& a, cudaStream_t stream) {
  return many_rows(a, G) ? launch_rows(gqa_q4_append_kernel<F16, G, 1>, a, G, 1, stream)
                         : launch_rows(gqa_q4_append_kernel<F16, G, 4>, a, 4 * G, 1, stream);
}

template <bool F16, int G>
int read_g(const Q4RowsArgs& a, cudaStream_t stream) {
  return many_rows(a, G) ? launch_rows(gqa_q4_read_kernel<F16, G, 4>, a, 4 * G, 4, stream)
                         : launch_rows(gqa_q4_read_kernel<F16, G, 1>, a, 4 * G, 1, stream);
}

}  // namespace

int launch_q4_append(const Q4RowsArgs& a, bool f16, cudaStream_t stream) {
  switch (groups_of(a.D)) {
    case 1: return f16 ? append_g<true, 1>(a, stream) : append_g<false, 1>(a, stream);
    case 2: return f16 ? append_g<true, 2>(a, stream) : append_g<false, 2>(a, stream);
    case 3: return f16 ? append_g<true, 3>(a, stream) : append_g<false, 3>(a, stream);
    default: return f16 ? append_g<true, 4>(a, stream) : append_g<false, 4>(a, stream);
  }
}

int launch_q4_read(const Q4RowsArgs& a, bool f16, cudaStream_t stream) {
  switch (groups_of(a.D)) {
    case 1: return f16 ? read_g<true, 1>(a, stream) : read_g<false, 1>(a, stream);
    case 2: return f16 ? read_g<true, 2>(a, stream) : read_g<false, 2>(a, stream);
    case 3: return f16 ? read_g<true, 3>(a, stream) : read_g<false, 3>(a, stream);
    default: return f16 ? read_g<true, 4>(a, stream) : read_g<false, 4>(a, stream);
  }
}

}  // namespace gqa
