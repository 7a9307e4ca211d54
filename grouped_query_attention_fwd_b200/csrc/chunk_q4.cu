// Query blocks of more than a few rows over a 4-bit cache, on the 5th
// generation tensor cores.
//
// The decode kernel unpacks every record once per 8 rows; from about 16 rows
// per kv head on it is cheaper to unpack it once for 128.  A group here is one
// (entry, kv head, 128-row query tile), rows packed as in the prefill kernels
// (row r: head r / qpt of the kv head's group, query q0 + r % qpt); its 128-key
// tiles are split over CTAs like a decode's (few rows and long keys give too
// few groups to fill the machine), which leaves partial softmax states that a
// second launch merges.
//
//   records --TMA--> raw ring --8 warps--> K, V in 16 bits, 128-byte swizzle
//   S = Q K^T    tcgen05.mma, Q from TMEM (copied in once per group), K from
//                shared memory, S double-buffered in TMEM
//   P = 2^(S - m)  8 warps, two threads per row with half of the keys each,
//                  which trade their maxima; P over the first half of S
//   O += P V     tcgen05.mma, P from TMEM, V from shared memory, O in TMEM
//
// Unpacking: a pair of codes becomes 128 + c (bf16) or 1024 + c (fp16) by one
// AND-OR, c by one packed subtraction, and the rounded value scale * c + min by
// one packed fused multiply-add: one rounding to 16 bits per key and value
// element.  K's pairs are put in the dims' order (Q comes in it); V's stay as
// the nibbles of a word fall (0 4 1 5 2 6 3 7), which permutes O's columns,
// undone in registers at the end.  Values past a length are written as zeros.
//
// Bound: issue slots.  Per key tile an SM spends about 600 cycles of each
// scheduler on unpacking 32768 codes and 770 on 128 rows' softmax; the two
// products need about 1000 of the tensor core.
//
// Warp roles (640 threads, one CTA per SM):
//   warps 0-3   softmax of keys 0-63 of each tile, epilogue of half of O's
//               columns (thread t: row t)
//   warps 4-7   the same for keys 64-127 and the other half
//   warps 8-15  unpacking (thread: one key, half of the dims)
//   warp 16     TMA producer of Q tiles and records
//   warp 17     TMEM allocator and MMA issuer (warps 18, 19 idle)
// Every wait is bounded; a thread that gives up sets the abort flag and the
// error word, and every role leaves its loops.
#include <cuda_runtime.h>

#include "decode_sched.cuh"
#include "epilogue.cuh"
#include "kernels.h"
#include "prefill_common.cuh"
#include "ptx.cuh"
#include "q4.cuh"

namespace gqa {
namespace {

using namespace prefill;
using namespace q4;

constexpr int kThreads = kChunkThreads;
constexpr int kSoftmaxWarps = 8;
constexpr int kConvWarps = 8;
constexpr int kWarpLoad = 16;
constexpr int kWarpMMA = 17;
constexpr int HK = BN / 2;  // keys of a tile per softmax thread
// Registers of the five warpgroups (setmaxnreg): softmax twice, unpacking
// twice, the rest; together no more than the launch's 96 a thread.
constexpr int kLaunchRegs = 96;
constexpr int kSoftmaxRegs = 136, kConvRegs = 72, kIoRegs = 64;
static_assert(2 * kSoftmaxRegs + 2 * kConvRegs + kIoRegs <= 5 * kLaunchRegs, "register split");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 256, kQCol = 384;  // S buffers at 0 and 128

template <int D>
struct ChunkLayout {
  static constexpr int NG = D / kGroup;
  static constexpr int CH = D / 64;
  static constexpr int kChunkBytes = 128 * 128;
  static constexpr int kTile = CH * kChunkBytes;  // a 16-bit Q, K or V tile
  static constexpr int kPitch = record_bytes(D);
  static constexpr int kRaw = 2 * BN * kPitch;    // K and V records of a key tile
  static constexpr int kKOff = kTile;             // Q first
  static constexpr int kVOff = kKOff + 2 * kTile;
  static constexpr int kRawOff = kVOff + 2 * kTile;
  static int bytes(int stages, int ragged_batch) {
    return 1024 + kRawOff + stages * kRaw + (2 * stages + 20) * 8 + 32 + 2 * 2 * 128 * 4 +
           (ragged_batch > 0 ? ((8 * ragged_batch + 4 + 15) / 16) * 16 : 0);
  }
};

__device__ __forceinline__ uint32_t ld_shared(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint4 ld_shared4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ void st_shared4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

__device__ __forceinline__ uint32_t sub2(uint32_t x, uint32_t y, bool f16) {
  uint32_t r;
  if (f16)
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  else
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t fma2(uint32_t x, uint32_t y, uint32_t z, bool f16) {
  uint32_t r;
  if (f16)
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(z));
  else
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(z));
  return r;
}

// Values of a word's nibble pairs (i, i + 4), i = 0 .. 3.
template <bool F16>
__device__ __forceinline__ void values_of(uint32_t (&v)[4], uint32_t w, uint32_t scale2,
                                          uint32_t min2) {
  constexpr uint32_t kBias = F16 ? 0x64006400u : 0x43004300u;  // 1024, 128
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = fma2(sub2(((w >> (4 * i)) & 0x000F000Fu) | kBias, kBias, F16), scale2, min2, F16);
}

// One CTA's share of a group.
struct Share {
  Pair pr;
  Slot sl;
  int id;                // group
  int nt_beg, nt_end;    // its key tiles that the query tile can see
  bool opens;            // the group's first unit is in this range
  int c_lo, c_hi;        // CTAs that share the group
};

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    gqa_chunk_q4_kernel(const __grid_constant__ CUtensorMap tmq,
                        const __grid_constant__ CUtensorMap tmk,
                        const __grid_constant__ CUtensorMap tmv, const PrefillArgs a,
                        const ChunkArgs ca, const PagedKV pg) {
  using L = ChunkLayout<D>;
  constexpr int NG = L::NG, CH = L::CH, P = L::kPitch;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int R = ca.stages;
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + L::kRawOff + R * L::kRaw);
  uint64_t* raw_empty = raw_full + R;
  uint64_t* q_full = raw_empty + R;
  uint64_t* q_empty = q_full + 1;    // Q copied into TMEM
  uint64_t* k_full = q_empty + 1;    // [J & 1] K unpacked (8 warps)
  uint64_t* k_empty = k_full + 2;    // [J & 1] QK(J) done
  uint64_t* v_full = k_empty + 2;
  uint64_t* v_empty = v_full + 2;
  uint64_t* s_full = v_empty + 2;    // [J & 1] QK(J) done
  uint64_t* p_full = s_full + 2;     // [J & 1] P(J) written (8 warps)
  uint64_t* o_ready = p_full + 2;    // [J & 1] PV(J) done
  uint64_t* o_final = o_ready + 2;   // the share's last PV done
  uint64_t* o_free = o_final + 1;    // O read by the epilogue (8 warps)
  uint64_t* mma_done = o_free + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* xch = reinterpret_cast<float*>(tmem_slot + 4);  // [2][half][row]: what a row's threads trade
  int* len_s = reinterpret_cast<int*>(xch + 512);
  int* pre_s = len_s + a.B;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const bool ragged = a.lens != nullptr;
  const int gpb = a.Hkv * ca.m_tiles;

  if (threadIdx.x == 0) {
    for (int i = 0; i < R; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], kConvWarps);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], kConvWarps);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], kConvWarps);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kSoftmaxWarps);
      mbar_init(&o_ready[i], 1);
    }
    mbar_init(o_final, 1);
    mbar_init(o_free, kSoftmaxWarps);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // Q rows past qpt * g of a tile are never written by TMA: zero them once.
  for (int i = threadIdx.x; i < CH * (BM - ca.rows) * 8; i += kThreads) {
    const int c = i / ((BM - ca.rows) * 8), r = i % ((BM - ca.rows) * 8);
    reinterpret_cast<uint4*>(smem + c * L::kChunkBytes + ca.rows * 128)[r] =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  if (warp == kWarpMMA) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();
  if (ragged) {
    for (int b = threadIdx.x; b < a.B; b += kThreads) {
      int len = a.lens[b];
      if (len < 0 || len > a.Sk) {
        if (blockIdx.x == 0) atomicOr(a.err, kErrKvLength);
        len = len < 0 ? 0 : a.Sk;
      }
      len_s[b] = len;
    }
    __syncthreads();
    if (warp == 0) {
      // pre[b + 1] = sum over entries <= b of their places.
      int carry = 0;
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane;
        int v = 0;
        if (b < a.B)
          v = gpb * (ca.lead + decode_key_range(len_s[b], a.Sk, a.Sq, a.causal, a.causal_offset,
                                                a.window)
                                   .tiles);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int n = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += n;
        }
        if (b < a.B) pre_s[b + 1] = carry + v;
        carry += __shfl_sync(0xffffffffu, v, 31);
      }
      if (lane == 0) pre_s[0] = 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The places of the launch (`lead` empty ones before each group's units) in
  // equal ranges, one per CTA.
  Sched sc;
  sc.pre = ragged ? pre_s : nullptr;
  sc.len = ragged ? len_s : nullptr;
  sc.per_b = gpb * (ca.tiles + ca.lead);
  sc.gpb = gpb;
  sc.B = a.B;
  sc.total = ragged ? pre_s[a.B] : ca.places;
  sc.P = static_cast<int>(gridDim.x) < sc.total ? static_cast<int>(gridDim.x) : sc.total;
  const int cta = static_cast<int>(blockIdx.x);
  const int v_begin = cta < sc.P ? range_start(cta, sc.total, sc.P) : 0;
  const int v_end = cta < sc.P ? range_start(cta + 1, sc.total, sc.P) : 0;

  // Calls f(share) for every group that has units in the range, in order;
  // f returns false to stop.
  auto each_share = [&](auto&& f) {
    Cursor cu;
    for (int va = v_begin; va < v_end;) {
      if (cu.b < 0 || va >= cu.end) {
        cu.b = sc.batch_of(va);
        cu.beg = sc.start_of(cu.b);
        cu.kr = decode_key_range(sc.len ? sc.len[cu.b] : a.Sk, a.Sk, a.Sq, a.causal,
                                 a.causal_offset, a.window);
        cu.end = cu.beg + gpb * (cu.kr.tiles + ca.lead);
      }
      const int span = cu.kr.tiles + ca.lead;
      const int gi = (va - cu.beg) / span;
      const int beg = cu.beg + gi * span + ca.lead;  // the group's first unit
      const int t0 = max(va - beg, 0), t1 = min(v_end - beg, cu.kr.tiles);
      va = beg + cu.kr.tiles;
      if (t1 <= t0) return;  // the range ends in the group's lead
      Share s;
      s.pr.b = cu.b;
      s.pr.kv = gi / ca.m_tiles;
      s.pr.mt0 = gi % ca.m_tiles;
      s.pr.len = sc.len ? sc.len[cu.b] : a.Sk;
      s.sl = slot_of(s.pr, a, ca.qpt);
      s.id = cu.b * gpb + gi;
      s.nt_beg = max(cu.kr.t0 + t0, static_cast<int>(s.sl.key_lo / BN));
      s.nt_end = min(cu.kr.t0 + t1, static_cast<int>((s.sl.key_hi + BN - 1) / BN));
      if (s.nt_end < s.nt_beg) s.nt_end = s.nt_beg;
      s.opens = t0 == 0;
      s.c_lo = cta_of_unit(beg, sc.total, sc.P);
      s.c_hi = cta_of_unit(beg + cu.kr.tiles - 1, sc.total, sc.P);
      if (!f(s)) return;
    }
  };

  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIoRegs));
    if (warp == kWarpLoad) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        prefetch_tmap(&tmq);
        prefetch_tmap(&tmk);
        prefetch_tmap(&tmv);
      }
      uint32_t J = 0, nq = 0;
      int s = 0;
      uint32_t parity = 1;  // of the wait for a free stage (passes at once in round 0)
      auto wait = [&](uint64_t* bar, uint32_t par) {
        return __all_sync(0xffffffffu,
                          mbar_try_wait(bar, par) ||
                              mbar_wait(bar, par, abort_flag, a.err, kErrPrefillWait)) != 0;
      };
      each_share([&](const Share& sh) {
        if (sh.nt_end == sh.nt_beg) return true;
        if (nq > 0 && !wait(q_empty, (nq - 1) & 1u)) return false;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(ca.rows * 128 * CH));
          for (int c = 0; c < CH; ++c)
            tma_load_4d(smem + c * L::kChunkBytes, &tmq, q_full, c * 64, sh.sl.q0,
                        sh.pr.kv * a.g, sh.pr.b);
        }
        __syncwarp();
        ++nq;
        // Paged: lane i holds the page of half i % 2 (64 keys) of tile i / 2 of
        // a block of 16, read one block ahead of its use.
        auto page_of = [&](int nt) {
          const int key = nt * BN + (lane & 1) * 64;
          if (nt >= sh.nt_end || key >= sh.pr.len) return pg.num_pages;
          const int page = __ldg(pg.bt + sh.pr.b * pg.bt_stride + key / pg.page_size);
          if (page >= 0 && page < pg.num_pages) return page;
          atomicOr(a.err, kErrPage);
          return pg.num_pages;  // out of range: read as zeros
        };
        const bool paged = pg.bt != nullptr;
        int next_page = paged ? page_of(sh.nt_beg + (lane >> 1)) : 0;
        for (int n0 = sh.nt_beg; n0 < sh.nt_end; n0 += 16) {
          const int my_page = next_page;
          if (paged) next_page = page_of(n0 + 16 + (lane >> 1));
          for (int i = 0; i < 16 && n0 + i < sh.nt_end; ++i) {
            const int nt = n0 + i;
            const int p0 = __shfl_sync(0xffffffffu, my_page, 2 * i);
            const int p1 = __shfl_sync(0xffffffffu, my_page, 2 * i + 1);
            if (!wait(&raw_empty[s], parity)) return false;
            if (lane == 0) {
              uint8_t* dst = smem + L::kRawOff + s * L::kRaw;
              mbar_arrive_expect_tx(&raw_full[s], L::kRaw);
              if (paged) {
                const int r0 = nt * BN % pg.page_size, r1 = (nt * BN + 64) % pg.page_size;
                tma_load_4d(dst, &tmk, &raw_full[s], 0, r0, sh.pr.kv, p0);
                tma_load_4d(dst + 64 * P, &tmk, &raw_full[s], 0, r1, sh.pr.kv, p1);
                tma_load_4d(dst + BN * P, &tmv, &raw_full[s], 0, r0, sh.pr.kv, p0);
                tma_load_4d(dst + (BN + 64) * P, &tmv, &raw_full[s], 0, r1, sh.pr.kv, p1);
              } else {
                tma_load_4d(dst, &tmk, &raw_full[s], 0, nt * BN, sh.pr.kv, sh.pr.b);
                tma_load_4d(dst + BN * P, &tmv, &raw_full[s], 0, nt * BN, sh.pr.kv, sh.pr.b);
              }
            }
            __syncwarp();
            ++J;
            if (++s == R) {
              s = 0;
              parity ^= 1u;
            }
          }
        }
        return true;
      });
      // On an abort, the copies still in flight land before the CTA leaves.
      if (lane == 0 && *abort_flag) {
        for (uint32_t j = J > static_cast<uint32_t>(R) ? J - R : 0; j < J; ++j)
          mbar_wait_drain(&raw_full[j % R], (j / R) & 1u);
        if (nq > 0) mbar_wait_drain(q_full, (nq - 1) & 1u);
      }
    } else if (warp == kWarpMMA) {
      // ------------------------------------------------------------ MMA warp
      // Converged, one elected lane issues; the order on the tensor core is
      // QK(0), QK(1), PV(0), QK(2), PV(1), ... and operations of one thread
      // execute in issue order, so QK(j + 2) may overwrite P(j) after PV(j).
      constexpr uint32_t idesc_qk = F16 ? idesc_f16_f32(BM, BN, 0, 0) : idesc_bf16_f32(BM, BN, 0, 0);
      constexpr uint32_t idesc_pv = F16 ? idesc_f16_f32(BM, D, 0, 1) : idesc_bf16_f32(BM, D, 0, 1);
      const uint64_t dk0 = kmajor_desc(smem_u32(smem + L::kKOff));
      const uint64_t dv0 = mnmajor_desc(smem_u32(smem + L::kVOff), L::kChunkBytes);
      uint32_t Jq = 0, Jp = 0;  // tiles whose QK / PV have been issued
      uint32_t n_share = 0;
      auto wait = [&](uint64_t* bar, uint32_t par) {
        return __all_sync(0xffffffffu, mbar_wait_hot(bar, par, abort_flag, a.err,
                                                     kErrPrefillWait)) != 0;
      };
      auto issue_qk = [&]() {
        const uint32_t s = Jq & 1u;
        if (!wait(&k_full[s], (Jq >> 1) & 1u)) return false;
        tc_fence_after();
        const uint64_t dk = dk0 + s * (L::kTile >> 4);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t step = ((ks >> 2) * L::kChunkBytes + (ks & 3) * 32) >> 4;
            tc_mma_ts(tmem + s * BN, tmem + kQCol + ks * 8, dk + step, idesc_qk, ks > 0 ? 1u : 0u);
          }
          tc_commit(&s_full[s]);
          tc_commit(&k_empty[s]);
        }
        __syncwarp();
        ++Jq;
        return true;
      };
      auto issue_pv = [&](bool first, bool last) {
        const uint32_t s = Jp & 1u;
        if (!wait(&p_full[s], (Jp >> 1) & 1u) || !wait(&v_full[s], (Jp >> 1) & 1u)) return false;
        if (first && n_share > 0 && !wait(o_free, (n_share - 1) & 1u)) return false;
        tc_fence_after();
        const uint64_t dv = dv0 + s * (L::kTile >> 4);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < BN / 16; ++ks)
            tc_mma_ts(tmem + kOCol, tmem + s * BN + ks * 8, dv + ((ks * 16 * 128) >> 4), idesc_pv,
                      (!first || ks > 0) ? 1u : 0u);
          tc_commit(&o_ready[s]);
          tc_commit(&v_empty[s]);
          if (last) tc_commit(o_final);
        }
        __syncwarp();
        ++Jp;
        return true;
      };
      each_share([&](const Share& sh) {
        const int n = sh.nt_end - sh.nt_beg;
        if (n == 0) return true;
        // Q into TMEM; the copy follows the last share's QKs on the tensor core.
        if (!wait(q_full, n_share & 1u)) return false;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            tc_cp_128x256b(tmem + kQCol + ks * 8,
                           kmajor_desc(smem_u32(smem) + (ks >> 2) * L::kChunkBytes + (ks & 3) * 32));
          tc_commit(q_empty);
        }
        __syncwarp();
        for (int i = 0; i < 2 && i < n; ++i)
          if (!issue_qk()) return false;
        for (int i = 0; i < n; ++i) {
          if (!issue_pv(i == 0, i == n - 1)) return false;
          if (i + 2 < n && !issue_qk()) return false;
        }
        ++n_share;
        return true;
      });
      if (elect_one()) tc_commit(mma_done);
      __syncwarp();
      mbar_wait_drain(mma_done, 0);
    }
  } else if (warp >= 8) {
    // -------------------------------------------------------------- unpacking
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    // A thread takes one key and half of the dims: NG / 2 groups.  Eight
    // consecutive keys in a quarter-warp: neither the records' 80-byte rows
    // nor the swizzled 16-byte stores conflict.
    constexpr int G2 = NG / 2;
    const int ct = static_cast<int>(threadIdx.x) - 256;
    const int half = ct >> 7, key = ct & 127;
    // The row's 16-byte pieces in the swizzled tile: piece p at row_at ^ 16 p.
    const uint32_t row_at = smem_u32(smem) + (CH == 2 ? half * L::kChunkBytes : half * 64) +
                            key * 128;
    const uint32_t swz = static_cast<uint32_t>(key & 7) << 4;
    const uint32_t raw_at = smem_u32(smem) + L::kRawOff + key * P + half * G2 * 4;
    const uint32_t code_at = smem_u32(smem) + L::kRawOff + key * P + kHeadBytes + half * G2 * 16;
    uint32_t J = 0;
    int s = 0;
    uint32_t parity = 0;
    auto wait = [&](uint64_t* bar, uint32_t par) {
      return __all_sync(0xffffffffu, mbar_wait_hot(bar, par, abort_flag, a.err,
                                                   kErrPrefillWait)) != 0;
    };
    each_share([&](const Share& sh) {
      for (int nt = sh.nt_beg; nt < sh.nt_end; ++nt, ++J) {
        if (!wait(&raw_full[s], parity)) return false;
        const bool held = nt * BN + key < sh.pr.len;
        uint32_t par[2][G2];
        uint4 code[2][G2];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < G2; ++i) {
            par[x][i] = ld_shared(raw_at + s * L::kRaw + x * BN * P + i * 4);
            code[x][i] = ld_shared4(code_at + s * L::kRaw + x * BN * P + i * 16);
            if (!held) par[x][i] = 0u;  // past the length: zeros
          }
        __syncwarp();
        if (lane == 0) mbar_arrive(&raw_empty[s]);
        if (++s == R) {
          s = 0;
          parity ^= 1u;
        }
        const uint32_t buf = J & 1u;
#pragma unroll
        for (int x = 0; x < 2; ++x) {  // K, then V
          uint64_t* const empty = x == 0 ? &k_empty[buf] : &v_empty[buf];
          if (J >= 2 && !wait(empty, ((J >> 1) - 1) & 1u)) return false;
          const uint32_t to = row_at + (x == 0 ? L::kKOff : L::kVOff) + buf * L::kTile;
#pragma unroll
          for (int i = 0; i < G2; ++i) {
            const uint32_t scale2 = __byte_perm(par[x][i], 0u, 0x1010);
            const uint32_t min2 = __byte_perm(par[x][i], 0u, 0x3232);
            const uint32_t w[4] = {code[x][i].x, code[x][i].y, code[x][i].z, code[x][i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t v[4];
              values_of<F16>(v, w[j], scale2, min2);
              uint4 out;
              if (x == 0) {  // dims in order
                out.x = __byte_perm(v[0], v[1], 0x5410);
                out.y = __byte_perm(v[2], v[3], 0x5410);
                out.z = __byte_perm(v[0], v[1], 0x7632);
                out.w = __byte_perm(v[2], v[3], 0x7632);
              } else {       // as the nibbles fall
                out = make_uint4(v[0], v[1], v[2], v[3]);
              }
              // (half * 64 is a multiple of 64 and swz of 16: the XOR of the
              // piece's number stays inside the row's 128 bytes.)
              st_shared4((to + (i * 4 + j) * 16) ^ swz, out);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(x == 0 ? &k_full[buf] : &v_full[buf]);
        }
      }
      return true;
    });
  } else {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    constexpr int HD = D / 2;
    const int h = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t o_col = tmem + lane_base + kOCol + h * HD;
    const int hh = row / ca.qpt, qi = row % ca.qpt;
    const bool live = (warp & 3) * 32 < ca.rows;  // a warp without rows only keeps step
    uint32_t X = 0;  // values traded so far
    // Publish v, meet the row's other thread, return its value; `flag` becomes
    // the AND over the two warps.
    auto trade = [&](float v, bool& flag) {
      float* slot = xch + (X & 1u) * 256;
      slot[h * 128 + row] = v;
      flag = bar_and(1 + (warp & 3), 64, flag);
      const float other = slot[(h ^ 1) * 128 + row];
      ++X;
      return other;
    };
    uint32_t J = 0, n_share = 0;
    bool first_share = true;
    bool ok = true;  // nothing has failed; carried to the next trade, so that no
                     // warp is left alone at its named barrier
    each_share([&](const Share& sh) {
      const int q = sh.sl.q0 + qi;
      const bool row_valid = row < ca.rows && q < a.Sq;
      // Keys [row_lo, row_hi) that this row sees, and key tiles [all_beg,
      // all_end) that every row sees all of.
      int row_lo = 0, row_hi = sh.pr.len, all_beg = 0, all_end = sh.pr.len / BN;
      if (a.causal) {
        const int64_t off = pair_off(a, sh.pr);
        row_hi = static_cast<int>(imax64(0, imin64(row_hi, q + off + 1)));
        all_end = static_cast<int>(imax64(0, imin64(sh.pr.len, sh.sl.q0 + off + 1)) / BN);
        if (a.window > 0) {
          row_lo = static_cast<int>(imin64(row_hi, imax64(0, q + off - a.window + 1)));
          all_beg = static_cast<int>(
              imin64(all_end, (imax64(0, sh.sl.q_last + off - a.window + 1) + BN - 1) / BN));
        }
      }
      float m_ref = -INFINITY, l = 0.f;  // m_ref is the same in both threads of a row
      for (int nt = sh.nt_beg; nt < sh.nt_end; ++nt, ++J) {
        const uint32_t s_col = tmem + lane_base + (J & 1u) * BN;
        // (Warp-uniform: every TMEM access below is made by the whole warp.)
        bool okt = __all_sync(0xffffffffu,
                              ok && mbar_wait_hot(&s_full[J & 1u], (J >> 1) & 1u, abort_flag,
                                                  a.err, kErrPrefillWait));
        if (!live) {
          if (!okt) return false;
          if (lane == 0) mbar_arrive(&p_full[J & 1u]);
          continue;
        }
        // Wholly visible tiles work on raw scores and fold the scale into one
        // FMA per element; the others test each key.
        const bool fast = nt >= all_beg && nt < all_end && a.scale_log2 >= 0.f;
        uint32_t r[HK];
        float mx = -INFINITY;
        if (okt) {
          tc_fence_after();
          tmem_ld32(s_col + h * HK, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
          tmem_ld32(s_col + h * HK + 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
          tmem_ld_wait();
          if (!fast) {
            const int lo = row_lo - nt * BN - h * HK, hi = row_hi - nt * BN - h * HK;
#pragma unroll
            for (int c = 0; c < HK; ++c)
              r[c] = __float_as_uint(c >= lo && c < hi ? __uint_as_float(r[c]) * a.scale_log2
                                                       : -INFINITY);
          }
          float part[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) part[e] = -INFINITY;
#pragma unroll
          for (int c = 0; c < HK; c += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              part[e] = fmax3(part[e], __uint_as_float(r[c + e]), __uint_as_float(r[c + 4 + e]));
          mx = fmax3(part[0], part[1], fmaxf(part[2], part[3]));
          if (fast) mx *= a.scale_log2;
        }
        // Once traded, both halves of S are in registers: P may overwrite them.
        tc_fence_before();
        const float mx_other = trade(mx, okt);
        tc_fence_after();
        if (!okt) return false;
        const float m_new = fmaxf(m_ref, fmaxf(mx, mx_other));
        const bool grow = m_new > m_ref + kRescaleLog2;  // also for -inf -> finite
        const float alpha = grow ? fast_exp2(m_ref - m_new) : 1.f;
        const bool o_live = grow && nt > sh.nt_beg && m_ref != -INFINITY;
        if (grow) {
          l *= alpha;
          m_ref = m_new;
        }
        const float ref = exp_ref(m_ref);
        const float sc = fast ? a.scale_log2 : 1.f;
        const uint64_t sc2 = f2_pack(sc, sc), nref2 = f2_pack(-ref, -ref);
        uint64_t lp[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) lp[e] = 0;
#pragma unroll
        for (int c = 0; c < HK / 32; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int c0 = c * 32 + 2 * e;
            const uint64_t x = f2_fma(f2_pack(__uint_as_float(r[c0]), __uint_as_float(r[c0 + 1])),
                                      sc2, nref2);
            const float p0 = fast_exp2(f2_lo(x)), p1 = fast_exp2(f2_hi(x));
            lp[e & 3] = f2_add(lp[e & 3], f2_pack(p0, p1));
            pk[e] = pack2<F16>(p0, p1);
          }
          tmem_st16(s_col + h * (HK / 2) + c * 16, pk);
        }
        l += ((f2_lo(lp[0]) + f2_hi(lp[0])) + (f2_lo(lp[1]) + f2_hi(lp[1]))) +
             ((f2_lo(lp[2]) + f2_hi(lp[2])) + (f2_lo(lp[3]) + f2_hi(lp[3])));
        if (__any_sync(0xffffffffu, o_live)) {
          // O holds the earlier tiles' P V with the old reference: rescale this
          // half of it once the previous tile's PV has completed.
          if (__all_sync(0xffffffffu,
                         mbar_wait_hot(&o_ready[(J - 1) & 1u], ((J - 1) >> 1) & 1u, abort_flag,
                                       a.err, kErrPrefillWait))) {
            tc_fence_after();
            const float f = o_live ? alpha : 1.f;
#pragma unroll
            for (int c = 0; c < HD / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(o_col + c * 32, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(o_col + c * 32, *reinterpret_cast<uint32_t(*)[16]>(&o[0]));
              tmem_st16(o_col + c * 32 + 16, *reinterpret_cast<uint32_t(*)[16]>(&o[16]));
            }
          } else {
            ok = false;
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[J & 1u]);
      }
      // Epilogue: out, or this CTA's partial of a split group.
      const bool some = sh.nt_end > sh.nt_beg;
      const bool split = sh.c_lo != sh.c_hi;
      bool oke = __all_sync(0xffffffffu, ok && (!some || mbar_wait_hot(o_final, n_share & 1u,
                                                                       abort_flag, a.err,
                                                                       kErrPrefillWait)));
      float l_other = 0.f;
      if (live) l_other = trade(l, oke);
      if (!oke) return false;
      uint32_t r[HD];
      if (some && live) {
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < HD / 32; ++c)
          tmem_ld32(o_col + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&r[c * 32]));
        tmem_ld_wait();
        tc_fence_before();
      } else {
#pragma unroll
        for (int e = 0; e < HD; ++e) r[e] = 0u;
      }
      if (some) {
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);
        ++n_share;
      }
      const int slot = cta * 2 + (first_share ? 0 : 1);
      first_share = false;
      if (threadIdx.x == 0 && (!split || sh.opens))
        ca.info[sh.id] = split ? make_int2(slot, sh.c_hi - sh.c_lo + 1) : make_int2(0, 1);
      if (!row_valid) return true;
      // O's columns are the dims with each eight as V's nibbles fell.
      constexpr int kAt[8] = {0, 2, 4, 6, 1, 3, 5, 7};  // column of dim e of eight
      const float lsum = l + l_other;
      if (split) {
        const int64_t at = static_cast<int64_t>(slot) * BM + row;
        if (h == 0) ca.part_ml[at] = make_float2(m_ref, lsum);
        float* po = ca.part_o + at * D + h * HD;
#pragma unroll
        for (int d = 0; d < HD; d += 8)
#pragma unroll
          for (int e = 0; e < 8; e += 4)
            *reinterpret_cast<float4*>(po + d + e) =
                make_float4(__uint_as_float(r[d + kAt[e]]), __uint_as_float(r[d + kAt[e + 1]]),
                            __uint_as_float(r[d + kAt[e + 2]]), __uint_as_float(r[d + kAt[e + 3]]));
      } else {
        uint16_t* orow = a.out + sh.pr.b * a.os[0] +
                         static_cast<int64_t>(sh.pr.kv * a.g + hh) * a.os[1] +
                         static_cast<int64_t>(q) * a.os[2] + h * HD;
        const float inv = 1.f / lsum;  // no visible key: 0 * inf = NaN
#pragma unroll
        for (int d = 0; d < HD; d += 8) {
          if (h * HD + d >= a.Dv) break;
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = pack2<F16>(__uint_as_float(r[d + kAt[2 * e]]) * inv,
                              __uint_as_float(r[d + kAt[2 * e + 1]]) * inv);
          *reinterpret_cast<uint4*>(orow + d) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      return true;
    });
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMMA) tmem_dealloc(tmem, kTmemCols);
}

// Merge of the split groups' partials: a warp per row.
template <int D, bool F16>
__global__ void __launch_bounds__(256)
    gqa_chunk_q4_merge_kernel(const PrefillArgs a, const ChunkArgs ca) {
  griddep_launch_dependents();
  griddep_wait();
  const int id = blockIdx.x;
  const int2 info = ca.info[id];
  // (Anything else than slots of the launch: it was aborted before writing.)
  if (info.y <= 1 || info.x < 0 || info.y > ca.grid || info.x / 2 > ca.grid - info.y) return;
  const int lane = threadIdx.x & 31;
  const int gpb = a.Hkv * ca.m_tiles;
  const int b = id / gpb, gi = id % gpb;
  const int kv = gi / ca.m_tiles, mt = gi % ca.m_tiles;
  constexpr int kLanes = D / 4;  // lanes with a quad of the row
  const int d = lane % kLanes * 4;
  for (int row = blockIdx.y * 8 + (threadIdx.x >> 5); row < ca.rows; row += gridDim.y * 8) {
    const int q = mt * ca.qpt + row % ca.qpt;
    if (q >= a.Sq) continue;
    // Partial k: the opening CTA's slot, then the first slot of each next CTA.
    auto at = [&](int k) {
      return static_cast<int64_t>(k == 0 ? info.x : (info.x / 2 + k) * 2) * BM + row;
    };
    float M = -INFINITY;
    for (int k = lane; k < info.y; k += 32) M = fmaxf(M, ca.part_ml[at(k)].x);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, i));
    const float ref = exp_ref(M);
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < info.y; ++k) {
      const float2 ml = ca.part_ml[at(k)];
      const float4 o = *reinterpret_cast<const float4*>(ca.part_o + at(k) * D + d);
      const float w = fast_exp2(ml.x - ref);
      l = fmaf(w, ml.y, l);
      acc.x = fmaf(w, o.x, acc.x);
      acc.y = fmaf(w, o.y, acc.y);
      acc.z = fmaf(w, o.z, acc.z);
      acc.w = fmaf(w, o.w, acc.w);
    }
    if (lane < kLanes && d < a.Dv) {
      const float inv = 1.f / l;
      uint2 pk;
      pk.x = pack2<F16>(acc.x * inv, acc.y * inv);
      pk.y = pack2<F16>(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(a.out + b * a.os[0] +
                                static_cast<int64_t>(kv * a.g + row / ca.qpt) * a.os[1] +
                                static_cast<int64_t>(q) * a.os[2] + d) = pk;
    }
  }
}

template <int D, bool F16>
int launch_t(const ChunkShape& s, const PrefillArgs& a, const ChunkArgs& ca, const PagedKV& pg,
             const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv,
             cudaStream_t stream) {
  auto kern = gqa_chunk_q4_kernel<D, F16>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, s.smem_bytes) !=
      cudaSuccess) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  // The register split assumes the launch allocation it was sized for.
  cudaFuncAttributes fa{};
  if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess || fa.numRegs != kLaunchRegs) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(s.grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(s.smem_bytes);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, tmq, tmk, tmv, a, ca, pg) != cudaSuccess) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(s.groups), static_cast<unsigned>((s.rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  if (cudaLaunchKernelEx(&cfg, gqa_chunk_q4_merge_kernel<D, F16>, a, ca) != cudaSuccess) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  return GQA_OK;
}

}  // namespace

ChunkShape plan_chunk_q4(const gqa_problem& p, int sm_count) {
  ChunkShape s{};
  const int64_t g = p.heads_q / p.heads_kv;
  s.D = p.head_dim <= 64 ? 64 : 128;
  // Only as many query positions per tile as there are: the live rows then sit
  // in few warps.
  s.qpt = static_cast<int>(BM / g < p.seq_q ? BM / g : p.seq_q);
  s.rows = static_cast<int>(s.qpt * g);
  s.m_tiles = static_cast<int>((p.seq_q + s.qpt - 1) / s.qpt);
  s.tiles = p.kv_lens != nullptr
                ? static_cast<int>((p.seq_k + BN - 1) / BN)
                : decode_key_range(p.seq_k, p.seq_k, p.seq_q, p.causal, p.causal_offset, p.window)
                      .tiles;
  if (s.tiles < 1) s.tiles = 1;
  s.groups = p.batch * p.heads_kv * s.m_tiles;
  s.places = s.groups * (s.tiles + kQ4Lead);
  const int64_t real = s.groups * s.tiles;
  s.grid = static_cast<int>(real < sm_count ? real : sm_count);
  const int rb = p.kv_lens != nullptr ? static_cast<int>(p.batch) : 0;
  for (s.stages = s.D == 128 ? 3 : 6;; --s.stages) {
    s.smem_bytes = s.D == 128 ? ChunkLayout<128>::bytes(s.stages, rb)
                              : ChunkLayout<64>::bytes(s.stages, rb);
    if (s.smem_bytes <= kDecodeMaxSmem || s.stages <= 2) break;
  }
  // What the kernel does not take: masks, counts past 32 bits, and batches
  // whose lengths do not fit beside its tiles.
  s.fits = !p.has_mask && s.smem_bytes <= kDecodeMaxSmem &&
           s.places < (int64_t(1) << 31);
  s.info_offset = kScratchOffset;
  s.part_ml_offset = s.info_offset + (s.groups * 8 + 255) / 256 * 256;
  s.part_o_offset = s.part_ml_offset + static_cast<int64_t>(s.grid) * 2 * BM * 8;
  s.workspace_end = s.part_o_offset + static_cast<int64_t>(s.grid) * 2 * BM * s.D * 4;
  return s;
}

int launch_chunk_q4(const gqa_problem& p, const ChunkShape& s, const PrefillArgs& a, uint8_t* ws,
                    const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv,
                    cudaStream_t stream) {
  ChunkArgs ca{};
  ca.qpt = s.qpt;
  ca.rows = s.rows;
  ca.m_tiles = s.m_tiles;
  ca.tiles = s.tiles;
  ca.lead = kQ4Lead;
  ca.places = static_cast<int>(s.places);
  ca.stages = s.stages;
  ca.grid = s.grid;
  ca.info = reinterpret_cast<int2*>(ws + s.info_offset);
  ca.part_ml = reinterpret_cast<float2*>(ws + s.part_ml_offset);
  ca.part_o = reinterpret_cast<float*>(ws + s.part_o_offset);
  PagedKV pg{};
  pg.bt = p.block_table;
  pg.bt_stride = p.block_table_stride;
  pg.page_size = static_cast<int>(p.page_size);
  pg.num_pages = static_cast<int>(p.num_pages);
  const bool f16 = p.dtype == GQA_DTYPE_F16;
  if (s.D == 128)
    return f16 ? launch_t<128, true>(s, a, ca, pg, tmq, tmk, tmv, stream)
               : launch_t<128, false>(s, a, ca, pg, tmq, tmk, tmv, stream);
  return f16 ? launch_t<64, true>(s, a, ca, pg, tmq, tmk, tmv, stream)
             : launch_t<64, false>(s, a, ca, pg, tmq, tmk, tmv, stream);
}

}  // namespace gqa
