// Query blocks of more than a few rows over a 4-bit cache, on the 5th
// generation tensor cores.
//
// The decode kernel unpacks every record once per 8 rows; from about 16 rows
// per kv head on it is cheaper to unpack it once for 128 or 256.  A group here
// is one or two consecutive 128-row query tiles of one (entry, kv head), rows
// packed as in the prefill kernels (row r of a tile: head r / qpt of the kv
// head's group, query q0 + r % qpt); its 128-key tiles are split over CTAs like
// a decode's (few rows and long keys give too few groups to fill the machine),
// which leaves partial softmax states that a second launch merges.
//
//   records --TMA--> raw ring --8 warps--> K, V in 16 bits, 128-byte swizzle
//   S_X = Q K^T      tcgen05.mma, both from shared memory, S_X in TMEM
//   P_X = 2^(S - m)  a warpgroup per X, one thread per row; P_X over S_X
//   O_X += P_X V     tcgen05.mma, P_X from TMEM, V from shared memory, O_X in TMEM
//
// Two softmax states X = 0, 1 take turns, so that the tensor core works on one
// while a warpgroup turns the other's scores into P.  Job i of a share belongs
// to X = i % 2.  With two query tiles X is the tile and two jobs share a key
// tile; with one, X is the parity of the key tile, and the two states of a row
// are merged at the end of the share.  The MMA warp issues QK(0), QK(1), PV(0),
// QK(2), PV(1), ...: operations of one thread execute in issue order, so QK(i +
// 2) may overwrite P(i), and the commit that signals S(i + 2) also means that
// PV(i) is done and O_X may be rescaled.
//
// Unpacking: a pair of codes becomes 1024 + c (fp16) by one AND-OR, c by one
// packed subtraction, and the rounded value scale * c + min by one packed fused
// multiply-add: one rounding to 16 bits per key and value element, and P is
// rounded likewise.  K's pairs are put in the dims' order (Q comes in it); V's
// stay as the nibbles of a word fall (0 4 1 5 2 6 3 7), which permutes O's
// columns, undone in registers at the end.  Values of keys before the first or
// past the last that a row of the group can see are written as zeros, whatever
// their records hold.
//
// Operands: the products take two operands of one 16-bit type.  A bf16 cache is
// unpacked into fp16, which keeps 8 times as many bits (relative error against 64
// bits 0.0017, the result's own rounding, against 0.0036 with bf16 operands and
// P), its Q is brought to fp16 a share at a time, and P is fp16.  fp16 does not
// hold bf16's range: a CTA that meets records or queries past what would keep
// bf16's bits (see kUp) goes over its shares once more with bf16 operands, which
// costs the others a barrier and a flag.  An fp16 cache's values are rounded to
// fp16: 0.00044, the result's own rounding being 0.0002.
//
// Measured (8 entries of 32768 keys, 64/8 heads of 128, 32 queries, bf16): 305
// us, 900 TFLOP/s; a 128-key tile costs an SM 2.4 us with two query tiles and 1.8
// us with one (fp16 caches 2.3 and 1.6 us), of which the products need 1.1 us and
// 0.55 us.  Bound: the unpacking warps and the softmax, which share the issue
// slots.  With four unpacking warps of twice the work each it
// took a tenth longer (a tenth less without their arithmetic and stores, a
// sixth less without the softmax).  A whole S row per thread costs some spills
// at 168 registers; fewer cost more (152: 5% longer, 136: 38%).
//
// Warp roles (640 threads, one CTA per SM):
//   warps 0-3   softmax of X = 0 and its epilogue (thread t: row t)
//   warps 4-7   the same for X = 1
//   warps 8-15  unpacking (thread: one key, half of the dims)
//   warp 16     TMA producer of Q tiles and records
//   warp 17     TMEM allocator and MMA issuer (warps 18, 19 idle)
// The softmax warps also bring a bf16 cache's Q to fp16.
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
// Registers of the five warpgroups (setmaxnreg): softmax twice, unpacking
// twice, the rest; together no more than the launch's 96 a thread.
constexpr int kLaunchRegs = 96;
constexpr int kSoftmaxRegs = 168, kConvRegs = 48, kIoRegs = 48;
static_assert(2 * kSoftmaxRegs + 2 * kConvRegs + kIoRegs <= 5 * kLaunchRegs, "register split");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 256;  // S_X at 128 X, O_X at kOCol + 128 X

// bf16 records in fp16 operands: values are taken kUp times as large, which puts
// the middle of what fp16 holds where caches have their values.  They overflow
// from scales of 2^7 or minima of 2^11 on (patterns in bf16).  A value's, scale's
// and minimum's rounding is off by 2^-25 / kUp or 2^-12 of it: fewer bits than
// bf16's where a group of V's is below 2^-16 throughout (eight scales and the
// minimum are; groups of zeros may be), and, in the scores, where a row's
// |scale * q| passes 2^9.
// P is taken 2^kWeightLog2 times as large, as far as the reference that trails
// by 2^kRescaleLog2 lets fp16: weights keep 11 bits down to 2^-21 of the
// largest, and 8 down to 2^-24 (a row may leave most of its weight on a key
// whose values are zeros).  With bf16 operands, too: partials of a group meet.
constexpr float kWeightLog2 = 7.f;
static_assert(kWeightLog2 + kRescaleLog2 < 16.f, "P stays in fp16");
constexpr float kUp = 16.f;
constexpr uint32_t kUp2 = 0x41804180u;  // twice, in bf16
constexpr uint32_t kMostScale = (127 + 7) << 7, kMostMin = (127 + 11) << 7;
constexpr uint32_t kLeast = ((127 - 16 + 4) << 23) - 1;  // (kUp times the value's bits, less one)
constexpr float kMostToLog2 = 0x1p9f / (0x1p15f * kUp);

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;  // (of a NaN and a number, the number: fp16 has NaN, too)
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

template <int D>
struct ChunkLayout {
  static constexpr int NG = D / kGroup;
  static constexpr int CH = D / 64;
  static constexpr int kChunkBytes = 128 * 128;
  static constexpr int kTile = CH * kChunkBytes;  // a 16-bit Q, K or V tile
  static constexpr int kPitch = record_bytes(D);
  static constexpr int kRaw = BN * kPitch;        // K or V records of a key tile
  // Q tiles first, then K twice, V twice, the raw ring.
  __host__ __device__ static constexpr int k_off(int nq) { return nq * kTile; }
  __host__ __device__ static constexpr int v_off(int nq) { return (nq + 2) * kTile; }
  __host__ __device__ static constexpr int raw_off(int nq) { return (nq + 4) * kTile; }
  static int bytes(int nq, int stages, int ragged_batch) {
    return 1024 + raw_off(nq) + stages * kRaw + (2 * stages + 19) * 8 + 16 +
           (nq == 1 ? 2 * 2 * 128 * 8 : 0) +
           (ragged_batch > 0 ? ((8 * ragged_batch + 4 + 15) / 16) * 16 : 0);
  }
};

__device__ __forceinline__ uint32_t ld_shared(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_shared4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
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
  Pair pr;               // mt0: the first query tile
  int id;                // group
  int nt_beg, nt_end;    // its key tiles that the query tiles can see
  int key_beg, key_end;  // from the first key that one of their rows can see to past the last
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
  const int R = ca.stages, nq = ca.nq, sh = nq - 1;
  uint8_t* const raw = smem + L::raw_off(nq);
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(raw + R * L::kRaw);
  uint64_t* raw_empty = raw_full + R;
  uint64_t* q_full = raw_empty + R;
  uint64_t* q_empty = q_full + 1;    // the share's last QK done
  uint64_t* k_full = q_empty + 1;    // [u & 1] K unpacked (8 warps)
  uint64_t* k_empty = k_full + 2;    // [u & 1] the QKs of key tile u done
  uint64_t* v_full = k_empty + 2;
  uint64_t* v_empty = v_full + 2;
  uint64_t* s_full = v_empty + 2;    // [X] S_X done (and every earlier PV)
  uint64_t* p_full = s_full + 2;     // [X] P_X written (4 warps)
  uint64_t* o_final = p_full + 2;    // the share's last PV done
  uint64_t* o_free = o_final + 1;    // both O_X read by the epilogue (8 warps)
  uint64_t* mma_done = o_free + 1;
  uint64_t* q_ready = mma_done + 1;  // W: the share's Q in fp16 (8 warps)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_ready + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* redo = abort_flag + 1;  // fp16 operands would not do
  // With one query tile: [share & 1][X][row] (m, l), which a row's threads trade.
  float2* xch = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(q_full) + 19 * 8 + 16);
  int* len_s = reinterpret_cast<int*>(xch + (nq == 1 ? 512 : 0));
  int* pre_s = len_s + a.B;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const bool ragged = a.lens != nullptr;
  const int gpb = a.Hkv * ca.m_groups;

  auto init_barriers = [&] {
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
      mbar_init(&p_full[i], kSoftmaxWarps / 2);
    }
    mbar_init(o_final, 1);
    mbar_init(o_free, kSoftmaxWarps);
    mbar_init(mma_done, 1);
    mbar_init(q_ready, kSoftmaxWarps);
    fence_mbar_init();
  };
  if (threadIdx.x == 0) {
    init_barriers();
    *abort_flag = 0;
    *redo = 0;
  }
  // Q rows past qpt * g of a tile are never written by TMA: zero them once.
  for (int i = threadIdx.x; i < nq * CH * (BM - ca.rows) * 8; i += kThreads) {
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
      s.pr.kv = gi / ca.m_groups;
      s.pr.len = sc.len ? sc.len[cu.b] : a.Sk;
      s.id = cu.b * gpb + gi;
      // From the first key of the group's first query tile to the last of its last.
      s.pr.mt0 = min((gi % ca.m_groups + 1) * nq, ca.m_tiles) - 1;
      const Slot last = slot_of(s.pr, a, ca.qpt);
      s.pr.mt0 = gi % ca.m_groups * nq;
      const Slot first = nq == 1 ? last : slot_of(s.pr, a, ca.qpt);
      const int64_t lo = first.key_hi > first.key_lo ? first.key_lo : last.key_lo;
      const int64_t hi = last.key_hi > last.key_lo ? last.key_hi : first.key_hi;
      s.nt_beg = max(cu.kr.t0 + t0, static_cast<int>(lo / BN));
      s.nt_end = min(cu.kr.t0 + t1, static_cast<int>((hi + BN - 1) / BN));
      if (s.nt_end < s.nt_beg) s.nt_end = s.nt_beg;
      s.key_beg = static_cast<int>(lo);
      s.key_end = static_cast<int>(hi);
      s.opens = t0 == 0;
      s.c_lo = cta_of_unit(beg, sc.total, sc.P);
      s.c_hi = cta_of_unit(beg + cu.kr.tiles - 1, sc.total, sc.P);
      if (!f(s)) return;
    }
  };

  // Each role's work, as body(whether the operands are fp16): over all shares
  // with fp16 operands, and, where some of a bf16 cache's values turned out not
  // to fit, over all of them once more with bf16 ones.
  auto passes = [&](auto&& body) {
    body(BoolConst<true>{});
    if (F16) return;
    tc_fence_before();
    __syncthreads();  // every copy has landed, every product is done
    tc_fence_after();
    if (*redo == 0 || *abort_flag) return;
    if (threadIdx.x == 0) {
      for (uint64_t* b = raw_full; b <= q_ready; ++b) mbar_inval(b);
      init_barriers();
    }
    __syncthreads();
    body(BoolConst<false>{});
  };

  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIoRegs));
    if (warp == kWarpLoad) passes([&](auto) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        prefetch_tmap(&tmq);
        prefetch_tmap(&tmk);
        prefetch_tmap(&tmv);
      }
      uint32_t J = 0, n_share = 0;  // half tiles and shares loaded
      int s = 0;
      uint32_t parity = 1;  // of the wait for a free stage (passes at once in round 0)
      auto wait = [&](uint64_t* bar, uint32_t par) {
        return __all_sync(0xffffffffu,
                          mbar_try_wait(bar, par) ||
                              mbar_wait(bar, par, abort_flag, a.err, kErrPrefillWait)) != 0;
      };
      each_share([&](const Share& me) {
        if (me.nt_end == me.nt_beg) return true;
        // Paged: lane i holds the page of half i % 2 (64 keys) of tile i / 2 of
        // a block of 16, read one block ahead of its use.
        auto page_of = [&](int nt) {
          const int key = nt * BN + (lane & 1) * 64;
          if (nt >= me.nt_end || key >= me.pr.len) return pg.num_pages;
          // (From L2: an earlier kernel may have written it while this one was resident.)
          const int page = __ldcg(pg.bt + me.pr.b * pg.bt_stride + key / pg.page_size);
          if (page >= 0 && page < pg.num_pages) return page;
          atomicOr(a.err, kErrPage);
          return pg.num_pages;  // out of range: read as zeros
        };
        const bool paged = pg.bt != nullptr;
        int next_page = paged ? page_of(me.nt_beg + (lane >> 1)) : 0;
        for (int n0 = me.nt_beg; n0 < me.nt_end; n0 += 16) {
          const int my_page = next_page;
          if (paged) next_page = page_of(n0 + 16 + (lane >> 1));
          for (int i = 0; i < 16 && n0 + i < me.nt_end; ++i) {
            const int nt = n0 + i;
            const int p0 = __shfl_sync(0xffffffffu, my_page, 2 * i);
            const int p1 = __shfl_sync(0xffffffffu, my_page, 2 * i + 1);
            for (int x = 0; x < 2; ++x) {  // K, then V
              if (!wait(&raw_empty[s], parity)) return false;
              if (ca.withhold >= 0 && ca.withhold == me.id * ca.tiles + nt) return false;
              if (lane == 0) {
                const CUtensorMap* map = x == 0 ? &tmk : &tmv;
                uint8_t* dst = raw + s * L::kRaw;
                mbar_arrive_expect_tx(&raw_full[s], L::kRaw);
                if (paged) {
                  const int r0 = nt * BN % pg.page_size, r1 = (nt * BN + 64) % pg.page_size;
                  tma_load_4d(dst, map, &raw_full[s], 0, r0, me.pr.kv, p0);
                  tma_load_4d(dst + 64 * P, map, &raw_full[s], 0, r1, me.pr.kv, p1);
                } else {
                  tma_load_4d(dst, map, &raw_full[s], 0, nt * BN, me.pr.kv, me.pr.b);
                }
              }
              __syncwarp();
              ++J;
              if (++s == R) {
                s = 0;
                parity ^= 1u;
              }
            }
            if (nt > me.nt_beg) continue;
            // The share's Q, once the last share's QKs have read theirs; its
            // first key tile's records are on their way by then.
            if (n_share > 0 && !wait(q_empty, (n_share - 1) & 1u)) return false;
            if (lane == 0) {
              mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(nq * ca.rows * 128 * CH));
              for (int t = 0; t < nq; ++t)
                for (int c = 0; c < CH; ++c)
                  tma_load_4d(smem + t * L::kTile + c * L::kChunkBytes, &tmq, q_full, c * 64,
                              (me.pr.mt0 + t) * ca.qpt, me.pr.kv * a.g, me.pr.b);
            }
            __syncwarp();
            ++n_share;
          }
        }
        return true;
      });
      // On an abort, the copies still in flight land before the CTA leaves.
      if (lane == 0 && *abort_flag) {
        for (uint32_t j = J > static_cast<uint32_t>(R) ? J - R : 0; j < J; ++j)
          mbar_wait_drain(&raw_full[j % R], (j / R) & 1u);
        if (n_share > 0) mbar_wait_drain(q_full, (n_share - 1) & 1u);
      }
    });
    else if (warp == kWarpMMA) passes([&](auto half) {
      // ------------------------------------------------------------ MMA warp
      // Converged, one elected lane issues.
      constexpr bool H = decltype(half)::value, W = H && !F16;
      constexpr uint32_t idesc_qk = H ? idesc_f16_f32(BM, BN, 0, 0) : idesc_bf16_f32(BM, BN, 0, 0);
      constexpr uint32_t idesc_pv = H ? idesc_f16_f32(BM, D, 0, 1) : idesc_bf16_f32(BM, D, 0, 1);
      const uint64_t dq0 = kmajor_desc(smem_u32(smem));
      const uint64_t dk0 = kmajor_desc(smem_u32(smem + L::k_off(nq)));
      const uint64_t dv0 = mnmajor_desc(smem_u32(smem + L::v_off(nq)), L::kChunkBytes);
      uint32_t U = 0;               // key tiles of earlier shares
      uint32_t p_parity = 0;        // bit X: of the next wait for P_X
      uint32_t n_share = 0;
      auto wait = [&](uint64_t* bar, uint32_t par) {
        return __all_sync(0xffffffffu, mbar_wait_hot(bar, par, abort_flag, a.err,
                                                     kErrPrefillWait)) != 0;
      };
      // Job i of the share; its key tile's first and last job wait for and free it.
      auto issue_qk = [&](int i, bool last) {
        const uint32_t u = U + (i >> sh), X = i & 1u;
        if ((i & sh) == 0) {
          if (!wait(&k_full[u & 1u], (u >> 1) & 1u)) return false;
          tc_fence_after();
        }
        const uint64_t dq = dq0 + ((i & sh) * L::kTile >> 4);
        const uint64_t dk = dk0 + ((u & 1u) * L::kTile >> 4);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t step = ((ks >> 2) * L::kChunkBytes + (ks & 3) * 32) >> 4;
            tc_mma_ss(tmem + X * BN, dq + step, dk + step, idesc_qk, ks > 0 ? 1u : 0u);
          }
          tc_commit(&s_full[X]);
          if ((i & sh) == sh) tc_commit(&k_empty[u & 1u]);
          if (last) tc_commit(q_empty);
        }
        __syncwarp();
        return true;
      };
      auto issue_pv = [&](int i, bool last) {
        const uint32_t u = U + (i >> sh), X = i & 1u;
        if ((i & sh) == 0 && !wait(&v_full[u & 1u], (u >> 1) & 1u)) return false;
        if (!wait(&p_full[X], (p_parity >> X) & 1u)) return false;
        p_parity ^= 1u << X;
        if (i == 0 && n_share > 0 && !wait(o_free, (n_share - 1) & 1u)) return false;
        tc_fence_after();
        const uint64_t dv = dv0 + ((u & 1u) * L::kTile >> 4);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < BN / 16; ++ks)
            tc_mma_ts(tmem + kOCol + X * 128, tmem + X * BN + ks * 8, dv + ((ks * 16 * 128) >> 4),
                      idesc_pv, (i > 1 || ks > 0) ? 1u : 0u);
          if ((i & sh) == sh) tc_commit(&v_empty[u & 1u]);
          if (last) tc_commit(o_final);
        }
        __syncwarp();
        return true;
      };
      each_share([&](const Share& me) {
        const int n = (me.nt_end - me.nt_beg) << sh;
        if (n == 0) return true;
        if (!wait(W ? q_ready : q_full, n_share & 1u)) return false;
        tc_fence_after();
        for (int i = 0; i < 2 && i < n; ++i)
          if (!issue_qk(i, i == n - 1)) return false;
        for (int i = 0; i < n; ++i) {
          if (!issue_pv(i, i == n - 1)) return false;
          if (i + 2 < n && !issue_qk(i + 2, i + 2 == n - 1)) return false;
        }
        U += static_cast<uint32_t>(me.nt_end - me.nt_beg);
        ++n_share;
        return true;
      });
      if (elect_one()) tc_commit(mma_done);
      __syncwarp();
      mbar_wait_drain(mma_done, 0);
    });
    else passes([](auto) {});
  } else if (warp >= 8) {
    // -------------------------------------------------------------- unpacking
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    passes([&](auto half_type) {
      constexpr bool H = decltype(half_type)::value, W = H && !F16;
      // A thread takes one key and half of the dims: NG / 2 groups.  Eight
      // consecutive keys in a quarter-warp: neither the records' 16 (D / 32 +
      // 1)-byte rows nor the swizzled 16-byte stores conflict.
      constexpr int G2 = NG / 2;
      const int key = static_cast<int>(threadIdx.x) & 127;
      const int half = static_cast<int>(threadIdx.x - 256) >> 7;
      const uint32_t swz = static_cast<uint32_t>(key & 7) << 4;
      const uint32_t raw_at = smem_u32(raw) + key * P;
      const uint32_t row_at =
          smem_u32(smem) + (CH == 2 ? half * L::kChunkBytes : half * 64) + key * 128;
      const uint32_t k_at = row_at + L::k_off(nq), v_at = row_at + L::v_off(nq);
      uint32_t U = 0;  // key tiles unpacked
      int s = 0;
      uint32_t parity = 0;
      uint32_t most = 0u, least = ~0u;  // W: the records' parameters so far (see kMostScale)
      auto wait = [&](uint64_t* bar, uint32_t par) {
        return __all_sync(0xffffffffu, mbar_wait_hot(bar, par, abort_flag, a.err,
                                                     kErrPrefillWait)) != 0;
      };
      each_share([&](const Share& me) {
        for (int nt = me.nt_beg; nt < me.nt_end; ++nt, ++U) {
          const bool held = nt * BN + key >= me.key_beg && nt * BN + key < me.key_end;
          const uint32_t buf = U & 1u;
#pragma unroll
          for (int x = 0; x < 2; ++x) {  // K, then V
            if (!wait(&raw_full[s], parity)) return false;
            uint32_t par[G2];
            uint4 code[G2];
#pragma unroll
            for (int i = 0; i < G2; ++i) {
              par[i] = ld_shared(raw_at + s * L::kRaw + (half * G2 + i) * 4);
              code[i] = ld_shared4(raw_at + s * L::kRaw + kHeadBytes + (half * G2 + i) * 16);
            }
            // The stage goes back to the producer, whose next copy overwrites it.
            // Three things stand between the loads above and that copy: the loads
            // are generic accesses and the copy is one of the async proxy, which
            // the mbarrier alone does not order (the proxy fence); they are 32
            // lanes' and the arrival is lane 0's (__syncwarp, which a vote does not
            // replace); and the words are in registers (the branch, never taken).
            // Without the fence and the branch, results at head dim 128 changed
            // from call to call.
            uint32_t any = 0u;
#pragma unroll
            for (int i = 0; i < G2; ++i)
              any ^= par[i] ^ code[i].x ^ code[i].y ^ code[i].z ^ code[i].w;
            if (__any_sync(0xffffffffu, any == 0xA5A5A5A5u)) __nanosleep(0);
            fence_proxy_async_smem();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < G2; ++i)
              if (!held) par[i] = 0u;  // seen by no row: zeros, whatever is there
            if (lane == 0) mbar_arrive(&raw_empty[s]);
            if (++s == R) {
              s = 0;
              parity ^= 1u;
            }
            if (W) {
#pragma unroll
              for (int i = 0; i < G2; ++i) {
                most = max_bf16x2(most, par[i] & 0x7FFF7FFFu);
                const uint32_t up = mul_bf16x2(par[i], kUp2);
                const float scale = __uint_as_float(up << 16);
                const float low = __uint_as_float(up & 0xFFFF0000u);
                // (The bits less one, so that a group of zeros counts as large.)
                if (x == 1)
                  least = min(least, __float_as_uint(fmaxf(8.f * scale, fabsf(low))) - 1u);
                par[i] = pack_f16x2(scale, low);
              }
            }
            uint64_t* const empty = x == 0 ? &k_empty[buf] : &v_empty[buf];
            if (U >= 2 && !wait(empty, ((U >> 1) - 1) & 1u)) return false;
            const uint32_t to = (x == 0 ? k_at : v_at) + buf * L::kTile;
#pragma unroll
            for (int i = 0; i < G2; ++i) {
              const uint32_t scale2 = __byte_perm(par[i], 0u, 0x1010);
              const uint32_t min2 = __byte_perm(par[i], 0u, 0x3232);
              const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t v[4];
                values_of<H>(v, w[j], scale2, min2);
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
      if (W && ((most & 0xFFFFu) >= kMostScale || (most >> 16) >= kMostMin || least < kLeast))
        *redo = 1;
    });
  } else {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    passes([&](auto half) {
      constexpr bool H = decltype(half)::value, W = H && !F16;
      const int X = warp >> 2;
      const int row = (warp & 3) * 32 + lane;
      const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t s_col = tmem + lane_base + X * BN;
      const uint32_t o_col = tmem + lane_base + kOCol;  // O_0's
      const int hh = row / ca.qpt, qi = row % ca.qpt;
      const bool live = (warp & 3) * 32 < ca.rows;  // a warp without rows only keeps step
      uint32_t J = 0, n_share = 0, n_trade = 0;
      bool first_share = true;
      each_share([&](const Share& me) {
        Pair pr = me.pr;
        if (nq == 2) pr.mt0 += X;
        const Slot sl = slot_of(pr, a, ca.qpt);
        const int q = sl.q0 + qi;
        const bool row_valid = row < ca.rows && q < a.Sq;
        // Keys [row_lo, row_hi) that this row sees, and key tiles [all_beg,
        // all_end) that every row sees all of.
        int row_lo = 0, row_hi = pr.len, all_beg = 0, all_end = pr.len / BN;
        if (a.causal) {
          const int64_t off = pair_off(a, pr);
          row_hi = static_cast<int>(imax64(0, imin64(row_hi, q + off + 1)));
          all_end = static_cast<int>(imax64(0, imin64(pr.len, sl.q0 + off + 1)) / BN);
          if (a.window > 0) {
            row_lo = static_cast<int>(imin64(row_hi, imax64(0, q + off - a.window + 1)));
            all_beg = static_cast<int>(
                imin64(all_end, (imax64(0, sl.q_last + off - a.window + 1) + BN - 1) / BN));
          }
        }
        bool ok = true;
        // Base-2 scores per score of the products (W: without Q's and K's powers).
        float to_log2 = a.scale_log2;
        if (W && me.nt_end > me.nt_beg) {
          // The row of Q in fp16, times the power of two that brings its largest
          // element to [2^14, 2^15): exact down to 2^-28 of that.  With one query
          // tile a row's two threads, who both need the power, take half each.
          if (live) {
            ok = __all_sync(0xffffffffu, mbar_wait_hot(q_full, n_share & 1u, abort_flag, a.err,
                                                       kErrPrefillWait));
            const uint32_t q_at = smem_u32(smem) + (nq == 2 ? X * L::kTile : 0) + row * 128;
            const uint32_t swz = static_cast<uint32_t>(row & 7) << 4;
            auto piece = [&](int i) {
              return q_at + (i >> 3) * L::kChunkBytes + (((i & 7) << 4) ^ swz);
            };
            uint32_t big = 0u;
#pragma unroll
            for (int i = 0; i < 8 * CH; ++i) {
              const uint4 v = ld_shared4(piece(i));
              big = __vmaxu2(big, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                           __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
            }
            if (nq == 1) ok = bar_and(1 + (warp & 3), 64, ok);  // both have read the row
            const int top = static_cast<int>(max(big & 0xFFFFu, big >> 16) >> 7);
            const int e = top == 0 || top == 255 ? 0 : min(14 + 127 - top, 126);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            to_log2 *= __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * (1.f / kUp);
            if (top != 0 && !(fabsf(to_log2) <= kMostToLog2)) *redo = 1;
            const int i0 = nq == 1 ? X * 4 * CH : 0, i1 = nq == 1 ? i0 + 4 * CH : 8 * CH;
            for (int i = i0; i < i1; ++i) {
              uint4 v = ld_shared4(piece(i));
              uint32_t* w = &v.x;
#pragma unroll
              for (int x = 0; x < 4; ++x)
                w[x] = pack_f16x2(__uint_as_float(w[x] << 16) * up,
                                  __uint_as_float(w[x] & 0xFFFF0000u) * up);
              st_shared4(piece(i), v);
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(q_ready);
          if (!ok) return false;
        }
        float m_ref = -INFINITY, l = 0.f;
        bool begun = false;  // O_X holds something of this share
        for (int nt = me.nt_beg + (nq == 1 ? X : 0); nt < me.nt_end; nt += 3 - nq) {
          // (Warp-uniform: every TMEM access below is made by the whole warp.)
          ok = __all_sync(0xffffffffu,
                          mbar_wait_hot(&s_full[X], J & 1u, abort_flag, a.err, kErrPrefillWait));
          ++J;
          if (!ok) break;
          if (live) {
            // Wholly visible tiles work on raw scores and fold the scale into one
            // FMA per element; the others test each key.
            const bool fast = nt >= all_beg && nt < all_end && a.scale_log2 >= 0.f;
            uint32_t r[BN];
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < BN / 32; ++c)
              tmem_ld32(s_col + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&r[c * 32]));
            tmem_ld_wait();
            if (!fast) {
              const int lo = row_lo - nt * BN, hi = row_hi - nt * BN;
#pragma unroll
              for (int c = 0; c < BN; ++c)
                r[c] = __float_as_uint(c >= lo && c < hi ? __uint_as_float(r[c]) * to_log2
                                                         : -INFINITY);
            }
            float part[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) part[e] = -INFINITY;
#pragma unroll
            for (int c = 0; c < BN; c += 16)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                part[e] = fmax3(part[e], __uint_as_float(r[c + e]), __uint_as_float(r[c + 8 + e]));
            float mx = fmax3(fmax3(part[0], part[1], part[2]), fmax3(part[3], part[4], part[5]),
                             fmaxf(part[6], part[7]));
            if (fast) mx *= to_log2;
            const float m_new = fmaxf(m_ref, mx);
            const bool grow = m_new > m_ref + kRescaleLog2;  // also for -inf -> finite
            const float alpha = grow ? fast_exp2(m_ref - m_new) : 1.f;
            const bool o_live = grow && begun && m_ref != -INFINITY;
            if (grow) {
              l *= alpha;
              m_ref = m_new;
            }
            const float ref = exp_ref(m_ref);
            const float sc = fast ? to_log2 : 1.f;
            const float up = kWeightLog2 - ref;
            const uint64_t sc2 = f2_pack(sc, sc), nref2 = f2_pack(up, up);
            uint64_t lp[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) lp[e] = 0;
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) {
              uint32_t pk[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int c0 = c * 32 + 2 * e;
                const uint64_t x = f2_fma(
                    f2_pack(__uint_as_float(r[c0]), __uint_as_float(r[c0 + 1])), sc2, nref2);
                const float p0 = fast_exp2(f2_lo(x)), p1 = fast_exp2(f2_hi(x));
                lp[e & 3] = f2_add(lp[e & 3], f2_pack(p0, p1));
                pk[e] = pack2<H>(p0, p1);
              }
              tmem_st16(s_col + c * 16, pk);
            }
            l += ((f2_lo(lp[0]) + f2_hi(lp[0])) + (f2_lo(lp[1]) + f2_hi(lp[1]))) +
                 ((f2_lo(lp[2]) + f2_hi(lp[2])) + (f2_lo(lp[3]) + f2_hi(lp[3])));
            if (__any_sync(0xffffffffu, o_live)) {
              // O_X holds the earlier tiles' P V with the old reference; they are
              // done (S_X follows them) and the next PV_X waits for this P.
              const float f = o_live ? alpha : 1.f;
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(o_col + X * 128 + c * 32, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(o_col + X * 128 + c * 32, *reinterpret_cast<uint32_t(*)[16]>(&o[0]));
                tmem_st16(o_col + X * 128 + c * 32 + 16,
                          *reinterpret_cast<uint32_t(*)[16]>(&o[16]));
              }
            }
            begun = true;
            tmem_st_wait();
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[X]);
        }
        // Epilogue: out, or this CTA's partial of a split group.
        const bool some = me.nt_end > me.nt_beg;
        const bool split = me.c_lo != me.c_hi;
        ok = __all_sync(0xffffffffu,
                        ok && (!some || mbar_wait_hot(o_final, n_share & 1u, abort_flag, a.err,
                                                      kErrPrefillWait)));
        // Weights of O_0 and O_1 in this row's result.
        float w0 = X == 0 ? 1.f : 0.f, w1 = X == 0 ? 0.f : 1.f;
        if (nq == 1 && live) {
          // The row's two threads trade their states and take half of the columns
          // each.  (A warp that has failed meets its partner here once more.)
          float2* at = xch + (n_trade & 1u) * 256;
          ++n_trade;
          at[X * 128 + row] = make_float2(m_ref, l);
          ok = bar_and(1 + (warp & 3), 64, ok);
          const float2 other = at[(X ^ 1) * 128 + row];
          const float M = fmaxf(m_ref, other.x), ref = exp_ref(M);
          const float wm = fast_exp2(m_ref - ref), wo = fast_exp2(other.x - ref);
          l = wm * l + wo * other.y;
          m_ref = M;
          w0 = X == 0 ? wm : wo;
          w1 = X == 0 ? wo : wm;
        }
        if (!ok) return false;
        const int slot = cta * 2 + (first_share ? 0 : 1);
        first_share = false;
        if (threadIdx.x == 0 && (!split || me.opens))
          ca.info[me.id] = split ? make_int2(slot, me.c_hi - me.c_lo + 1) : make_int2(0, 1);
        // O_X exists if X had a tile in this share.
        const bool has0 = some && (nq == 1 || X == 0);
        const bool has1 = nq == 1 ? me.nt_end - me.nt_beg > 1 : some && X == 1;
        const int64_t pat = (static_cast<int64_t>(slot) * nq + (nq == 2 ? X : 0)) * BM + row;
        if (split && row_valid && (nq == 2 || X == 0)) ca.part_ml[pat] = make_float2(m_ref, l);
        const float inv = split ? 1.f : 1.f / l;  // no visible key: 0 * inf = NaN
        w0 *= W ? inv * (1.f / kUp) : inv;
        w1 *= W ? inv * (1.f / kUp) : inv;
        constexpr int kCols = D / 32;  // 32-column pieces
        const int c_beg = nq == 1 ? X * (kCols / 2) : 0;
        const int c_end = nq == 1 ? c_beg + kCols / 2 : kCols;
        for (int c = c_beg; c < c_end; ++c) {
          __syncwarp();  // (the TMEM loads below are the whole warp's)
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f * inv;
          if (live) {
            uint32_t r[32];
            tc_fence_after();
            if (has0) {
              tmem_ld32(o_col + c * 32, r);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(r[e]) * w0;
            }
            if (has1) {
              tmem_ld32(o_col + 128 + c * 32, r);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e)
                o[e] = has0 ? fmaf(__uint_as_float(r[e]), w1, o[e]) : __uint_as_float(r[e]) * w1;
            }
            tc_fence_before();
          }
          if (!row_valid) continue;
          // O's columns are the dims with each eight as V's nibbles fell.
          constexpr int kAt[8] = {0, 2, 4, 6, 1, 3, 5, 7};  // column of dim e of eight
          if (split) {
            float* po = ca.part_o + pat * D + c * 32;
#pragma unroll
            for (int d = 0; d < 32; d += 8)
#pragma unroll
              for (int e = 0; e < 8; e += 4)
                *reinterpret_cast<float4*>(po + d + e) =
                    make_float4(o[d + kAt[e]], o[d + kAt[e + 1]], o[d + kAt[e + 2]],
                                o[d + kAt[e + 3]]);
          } else {
            uint16_t* orow = a.out + pr.b * a.os[0] +
                             static_cast<int64_t>(pr.kv * a.g + hh) * a.os[1] +
                             static_cast<int64_t>(q) * a.os[2] + c * 32;
#pragma unroll
            for (int d = 0; d < 32; d += 8) {
              if (c * 32 + d >= a.Dv) break;
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack2<F16>(o[d + kAt[2 * e]], o[d + kAt[2 * e + 1]]);
              *reinterpret_cast<uint4*>(orow + d) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        if (some) {
          __syncwarp();
          if (lane == 0) mbar_arrive(o_free);
          ++n_share;
        }
        return true;
      });
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
  const int2 info = __ldcg(&ca.info[id]);  // (L2: resident before these were written)
  // (Anything else than slots of the launch: it was aborted before writing.)
  if (info.y <= 1 || info.x < 0 || info.y > ca.grid || info.x / 2 > ca.grid - info.y) return;
  const int lane = threadIdx.x & 31;
  const int gpb = a.Hkv * ca.m_groups;
  const int b = id / gpb, gi = id % gpb;
  const int kv = gi / ca.m_groups;
  constexpr int kLanes = D / 4;  // lanes with a quad of the row
  const int d = lane % kLanes * 4;
  for (int r = blockIdx.y * 8 + (threadIdx.x >> 5); r < ca.nq * ca.rows; r += gridDim.y * 8) {
    const int X = r >= ca.rows ? 1 : 0, row = r - X * ca.rows;
    const int q = (gi % ca.m_groups * ca.nq + X) * ca.qpt + row % ca.qpt;
    if (q >= a.Sq) continue;
    // Partial k: the opening CTA's slot, then the first slot of each next CTA.
    auto at = [&](int k) {
      return (static_cast<int64_t>(k == 0 ? info.x : (info.x / 2 + k) * 2) * ca.nq + X) * BM + row;
    };
    float M = -INFINITY;
    for (int k = lane; k < info.y; k += 32) M = fmaxf(M, __ldcg(&ca.part_ml[at(k)]).x);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, i));
    const float ref = exp_ref(M);
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < info.y; ++k) {
      const float2 ml = __ldcg(&ca.part_ml[at(k)]);
      const float4 o = __ldcg(reinterpret_cast<const float4*>(ca.part_o + at(k) * D + d));
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
  cfg.gridDim = dim3(static_cast<unsigned>(s.groups), static_cast<unsigned>((s.nq * s.rows + 7) / 8));
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
  // A pair of query tiles costs less than two alone (chunk_tile_ns): two at a
  // time are cheaper as soon as there are two, even where the last pair is half
  // empty.
  s.nq = s.m_tiles > 1 ? 2 : 1;
  s.m_groups = (s.m_tiles + s.nq - 1) / s.nq;
  s.groups = p.batch * p.heads_kv * s.m_groups;
  s.places = s.groups * (s.tiles + kChunkLead);
  const int64_t real = s.groups * s.tiles;
  s.grid = static_cast<int>(real < sm_count ? real : sm_count);
  const int rb = p.kv_lens != nullptr ? static_cast<int>(p.batch) : 0;
  for (s.stages = 8;; --s.stages) {
    s.smem_bytes = s.D == 128 ? ChunkLayout<128>::bytes(s.nq, s.stages, rb)
                              : ChunkLayout<64>::bytes(s.nq, s.stages, rb);
    if (s.smem_bytes <= kDecodeMaxSmem || s.stages <= 2) break;
  }
  // What the kernel does not take: masks, counts past 32 bits, and batches
  // whose lengths do not fit beside its tiles.
  s.fits = !p.has_mask && s.smem_bytes <= kDecodeMaxSmem &&
           s.places < (int64_t(1) << 31);
  s.info_offset = kScratchOffset;
  s.part_ml_offset = s.info_offset + (s.groups * 8 + 255) / 256 * 256;
  s.part_o_offset = s.part_ml_offset + static_cast<int64_t>(s.grid) * 2 * s.nq * BM * 8;
  s.workspace_end = s.part_o_offset + static_cast<int64_t>(s.grid) * 2 * s.nq * BM * s.D * 4;
  return s;
}

int launch_chunk_q4(const gqa_problem& p, const ChunkShape& s, const PrefillArgs& a, uint8_t* ws,
                    const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv,
                    cudaStream_t stream) {
  ChunkArgs ca{};
  ca.qpt = s.qpt;
  ca.rows = s.rows;
  ca.m_tiles = s.m_tiles;
  ca.nq = s.nq;
  ca.m_groups = s.m_groups;
  ca.tiles = s.tiles;
  ca.lead = kChunkLead;
  ca.places = static_cast<int>(s.places);
  ca.stages = s.stages;
  ca.grid = s.grid;
  ca.info = reinterpret_cast<int2*>(ws + s.info_offset);
  ca.part_ml = reinterpret_cast<float2*>(ws + s.part_ml_offset);
  ca.part_o = reinterpret_cast<float*>(ws + s.part_o_offset);
  uint64_t limit;  // (the kernel's waits keep theirs)
  decode_test_settings(&ca.withhold, &limit);
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
