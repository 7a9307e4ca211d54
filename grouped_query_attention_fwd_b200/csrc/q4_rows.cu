// Attention over 4-bit records on the CUDA cores: one warp per output row,
// four values of the head dimension per lane, online softmax in fp32.
#include <cuda_runtime.h>

#include "epilogue.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace gqa {
namespace {

using namespace q4;

template <bool F16>
__global__ void __launch_bounds__(256)
    gqa_q4_rows_kernel(const gqa_problem p, const uint16_t* __restrict__ q,
                       const uint8_t* __restrict__ k, const uint8_t* __restrict__ v,
                       const uint8_t* __restrict__ mask, uint16_t* __restrict__ out,
                       uint32_t* __restrict__ err, const float scale_log2) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= p.batch * p.heads_q * p.seq_q) return;
  const int64_t i = row % p.seq_q, h = row / p.seq_q % p.heads_q, b = row / p.seq_q / p.heads_q;
  const int64_t kv = h / (p.heads_q / p.heads_kv);
  const uint16_t* qr = q + b * p.q_stride[0] + h * p.q_stride[1] + i * p.q_stride[2];
  const uint8_t* mrow = mask ? mask + b * p.mask_stride[0] + i * p.mask_stride[1] : nullptr;
  const int d0 = lane * 4, g = lane >> 3;
  const bool live = d0 < p.head_dim;
  float qv[4] = {0.f, 0.f, 0.f, 0.f}, acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (live)
    for (int e = 0; e < 4; ++e) qv[e] = to_f32<F16>(qr[d0 + e]);
  int64_t len = p.seq_k;
  if (p.kv_lens != nullptr) {
    len = p.kv_lens[b];
    if (len < 0 || len > p.seq_k) {
      if (lane == 0) atomicOr(err, kErrKvLength);
      len = len < 0 ? 0 : p.seq_k;
    }
  }
  int64_t lo = 0, hi = len;
  if (p.causal) {
    const int64_t top = i + p.causal_offset + (len - p.seq_k);
    if (top + 1 < hi) hi = top + 1;
    if (p.window > 0 && top - p.window + 1 > 0) lo = top - p.window + 1;
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t j = lo; j < hi; ++j) {
    if (!mask_allows(mrow, j)) continue;
    int64_t ko, vo;
    if (p.block_table != nullptr) {
      const int64_t page = p.block_table[b * p.block_table_stride + j / p.page_size];
      const bool ok = page >= 0 && page < p.num_pages;
      if (!ok && lane == 0) atomicOr(err, kErrPage);
      ko = ok ? page * p.k_stride[0] + (j % p.page_size) * p.k_stride[2] : -1;
      vo = ok ? page * p.v_stride[0] + (j % p.page_size) * p.v_stride[2] : -1;
    } else {
      ko = b * p.k_stride[0] + j * p.k_stride[2];
      vo = b * p.v_stride[0] + j * p.v_stride[2];
    }
    float kx[4] = {0.f, 0.f, 0.f, 0.f}, vx[4] = {0.f, 0.f, 0.f, 0.f};
    if (live && ko >= 0) {
      const uint8_t* kr = k + ko + kv * p.k_stride[1];
      const uint8_t* vr = v + vo + kv * p.v_stride[1];
      const uint32_t kp = *reinterpret_cast<const uint32_t*>(kr + 4 * g);
      const uint32_t vp = *reinterpret_cast<const uint32_t*>(vr + 4 * g);
      const uint32_t kc = *reinterpret_cast<const uint16_t*>(kr + kHeadBytes + 2 * lane);
      const uint32_t vc = *reinterpret_cast<const uint16_t*>(vr + kHeadBytes + 2 * lane);
      for (int e = 0; e < 4; ++e) {
        kx[e] = fmaf(scale_of<F16>(kp), static_cast<float>((kc >> (4 * e)) & 15u), min_of<F16>(kp));
        vx[e] = fmaf(scale_of<F16>(vp), static_cast<float>((vc >> (4 * e)) & 15u), min_of<F16>(vp));
      }
    }
    float dot = 0.f;
    for (int e = 0; e < 4; ++e) dot = fmaf(qv[e], kx[e], dot);
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    const float t = dot * scale_log2;
    const float m_new = fmaxf(m, t);
    const float alpha = exp2f(m - m_new), w = exp2f(t - m_new);
    l = l * alpha + w;
    for (int e = 0; e < 4; ++e) acc[e] = fmaf(w, vx[e], acc[e] * alpha);
    m = m_new;
  }
  uint16_t* orow = out + b * p.o_stride[0] + h * p.o_stride[1] + i * p.o_stride[2];
  if (live)  // l == 0 (no visible key): NaN
    for (int e = 0; e < 4; ++e) orow[d0 + e] = static_cast<uint16_t>(to_16<F16>(acc[e] / l));
}

}  // namespace

int launch_q4_rows(const gqa_problem& p, const void* q, const uint8_t* k, const uint8_t* v,
                   const uint8_t* mask, void* out, uint32_t* err, cudaStream_t stream) {
  const int64_t blocks = (p.batch * p.heads_q * p.seq_q + 7) / 8;
  if (blocks > 0x7fffffff) return GQA_ERR_UNSUPPORTED;
  const float scale_log2 = static_cast<float>(static_cast<double>(p.scale) * 1.4426950408889634);
  auto kern = p.dtype == GQA_DTYPE_F16 ? gqa_q4_rows_kernel<true> : gqa_q4_rows_kernel<false>;
  kern<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
      p, static_cast<const uint16_t*>(q), k, v, p.has_mask ? mask : nullptr,
      static_cast<uint16_t*>(out), err, scale_log2);
  return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace gqa
