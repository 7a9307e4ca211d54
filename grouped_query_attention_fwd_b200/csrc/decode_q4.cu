// Decode over a 4-bit cache: split-K attention that reads the records once.
//
// One token (or a short query block) attends to keys held as records: per
// group of 32 values a scale s, a minimum m and 4-bit codes c.  Nothing is
// expanded in memory, and no value is rounded to 16 bits on the way:
//
//   q . K_j   = sum_g  s_jg (q_g . c_jg) + m_jg sum(q_g)
//   out       = sum_j  (p_j s_jg) c_jg   +  sum_j p_j m_jg        per group g
//
// The two products over codes run on the tensor cores (warp-level MMAs: the
// operands come out of registers, where the codes are unpacked), everything
// with a scale or a minimum in fp32.
//
//  * Codes as operands: a nibble in bits 0-3 or 4-7 of a 16-bit half is, read
//    as bf16 or fp16, a subnormal (or first-binade) number, linear in the
//    code: c or 16 c times the type's smallest step.  One AND per two codes
//    makes an operand register, one shift per word brings the upper byte down:
//    5 instructions per 8 codes.  The 16 is undone in Q (its odd dims are
//    scaled by 1/16) or in the output rows.  Q is scaled by a power of two so
//    that the products stay inside fp32's normal range (bf16: 2^64; fp16: so
//    that each head's largest element is in [2^14, 2^15)).
//  * S^T = C_K Q^T with 16 keys of a chunk in M: a thread's 32-bit word of a
//    K record holds eight consecutive dims of one key, which are just the k
//    indices that its fragments want when Q uses the same order.  For V,
//    ldmatrix.trans of the 16-byte code blocks pairs the same halfword of two
//    keys in one register, the layout of V^T as the A operand.
//  * The weights p_j s_jg are rounded to fp16 (2^-11) as the B operand of
//    P V in both cache types.  So that they use fp16's range whatever the
//    scales, every row has a power of two per group of 32 dims on them, which
//    is taken off the group's outputs at the end and brings the row's largest
//    weight of the group so far to about 1: weights down to 2^-14 of it keep
//    their 11 bits, and each is off by at most 2^-25 of it.  (One power for
//    all groups, from each key's largest scale, is cheaper by a few percent and
//    wrong: a group of values 2^20 times smaller than its neighbours' comes out
//    4% off.)
//  * Both the exponent reference m and the powers are lazy.  They are taken
//    anew when a score passes m by more than 2^6 or a key's scale is more than
//    2^9 times what the group's power stands for, so that a weight stays below
//    2^15; one vote per chunk finds out.  m is a whole number: it moves by
//    powers of two, which the groups' powers take up, so that the products'
//    sums stay as they are.
//  * With an fp16 cache the rounded weights are also summed (a row of ones in
//    an MMA of its own) and eight of them taken off, so that the rounding
//    multiplies codes counted from the middle of the group's range, at most
//    half of it; bf16 outputs are rounded 8 times more coarsely than the
//    weights as it is.
//
// Reads 160 bytes per key of 128 dims against 512 in 16 bits.  Bound: issue
// slots of the unpacking and the softmax, then HBM: 16 entries of 32768 keys,
// 64/8 heads, take 147 us, 4.6 TB/s (103 us at the copy rate); 4096 keys, 32/8
// heads 24 us, half of it the ranges' ends.  At head dim 128 a thread wants a few
// more than its 168 registers: 100 to 210 bytes are spilled.  A stage is held
// until its words are used and fenced (handing it back once loaded took a twentieth
// less, but a load that has only been issued is no proof that it has come).  Work
// is cut into ranges of 128-key units as in the 16-bit decode; a producer warp
// streams K and V records with TMA into a ring, W consumer warps take 32-key
// chunks in turn, and each keeps a softmax state of its own until the group ends.
// 80-byte (48-byte) rows make every ldmatrix and parameter read free of bank
// conflicts without a swizzle.
#include <cuda_runtime.h>

#include "decode_sched.cuh"
#include "epilogue.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace gqa {
namespace {

using namespace q4;

// Loads of what an earlier kernel of the stream may have written (the mask and
// its bits, the block table, partials) go to L2: as a programmatic dependent
// this kernel can be resident before those writes, so that neither the
// non-coherent path nor a line in L1 is good for them.

constexpr int KT = kDecodeKeysPerTile;
// Powers of two that a score may pass the exponent reference by, and a value
// scale the row's largest weight of its group, before they are taken anew: their
// product has to stay in fp16 (2^15).
constexpr int kLazyLog2 = 6, kLazyScaleLog2 = 9;
constexpr uint32_t kPowerMost = 100;  // of a group: no weight yet
constexpr int kFastMerge = 4;              // contributors of a split group merged directly
constexpr int kBatch = 8;                  // partials loaded at a time by the other merge
// How many units longer than equal ranges the ranges may be that no two groups
// share, for ragged batches: what the changes of groups inside a range cost.
constexpr int kApartUnits = 6;

template <int NG>
struct Q4Layout {
  static constexpr int D = NG * kGroup;            // head_dim, padded
  static constexpr int HP = 8;                     // rows per pass: the columns of one MMA
  static constexpr int W = 11;                     // consumer warps: with the producer three per scheduler
  // 16-key MMA tiles a warp takes at a time: more of them share the waits,
  // votes and address arithmetic of a chunk (one takes a quarter longer), and
  // four, with 7 warps for their registers, gain nothing over two.
  static constexpr int kSub = 2;
  static constexpr int kChunk = 16 * kSub;         // keys of a chunk
  static constexpr int kChunks = KT / kChunk;
  static constexpr int kThreads = (W + 1) * 32;
  static_assert(kThreads == kQ4Threads, "the plan reports it");
  static constexpr int kPitch = record_bytes(D);   // bytes per record in shared memory
  static constexpr int kTile = KT * kPitch;        // K (or V) records of a unit
  static constexpr int kStage = 2 * kTile;
  static constexpr int kRow = D + 4;               // a row's O, then (m, l), padded (floats)
  static constexpr int kScratch = W * HP * kRow * 4;
  static constexpr int kQRows = HP * D * 2;        // Q rows of the range's second group
  static constexpr int kVis = HP * (KT / 32) * 4;  // a unit's mask bits of the pass's queries
  static int bytes(int stages, int ragged_batch) {
    return 128 /*alignment slack*/ + stages * (kStage + kVis) + kScratch + kQRows + (2 * stages + 2) * 8 +
           32 +
           (ragged_batch > 0 ? ((8 * ragged_batch + 4 + 15) / 16) * 16 : 0);
  }
};

// The lowest n bits (n below 0: none, above 31: all).
__device__ __forceinline__ uint32_t below(int n) {
  return n >= 32 ? ~0u : (n <= 0 ? 0u : (1u << n) - 1u);
}

// D = A B, no accumulator.
template <bool F16>
__device__ __forceinline__ void mma_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void ldmatrix_x2(uint32_t& r0, uint32_t& r1, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];"
               : "=r"(r0), "=r"(r1)
               : "r"(addr));
}

// 2^e, e in [-127, 127] (2^-127: 0), and the exponent of a power of two or of
// any other positive number, rounded down (below 2^-126: -127).
__device__ __forceinline__ float power_of_two(int e) {
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}
__device__ __forceinline__ int exponent_of(float x) {
  return static_cast<int>(__float_as_uint(x) >> 23) - 127;
}

// 2^e in the cache's type, rounded down where it has none: 0 or infinity.
template <bool F16>
__device__ __forceinline__ uint32_t type_power(int e) {
  constexpr int kBias = F16 ? 15 : 127, kBits = F16 ? 10 : 7;
  return static_cast<uint32_t>(min(max(e + kBias, 0), 2 * kBias + 1)) << kBits;
}

// Larger of two pairs of 16-bit numbers; of a NaN and a number, the number.
template <bool F16>
__device__ __forceinline__ uint32_t max_number(uint32_t x, uint32_t y) {
  uint32_t r;
  if (F16)
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  else
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// Record heads: NG words (scale | minimum << 16).
template <int NG>
__device__ __forceinline__ void load_params(uint32_t (&w)[NG], uint32_t addr) {
  if (NG == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[NG - 2]), "=r"(w[NG - 1])
                 : "r"(addr));
  else
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
}

// 32-bit words of one query's mask bits: whole 128-key units.
__host__ __device__ constexpr int64_t mask_words(int64_t Sk) { return (Sk + KT - 1) / KT * (KT / 32); }

constexpr int kMaskSpan = 1024;  // keys a warp packs at a time, a word per lane

// The mask as bits, one per key: [batch, seq_q] rows of mask_words.  The decode
// kernel needs each bit in up to eight heads' passes; read as bytes there, in
// its producer or its consumers, they cost it more than the records (8 x 6001
// keys, four queries: 100 and 55 us against 32 without a mask).
__global__ void __launch_bounds__(256)
    gqa_q4_mask_bits_kernel(const DecodeArgs a, uint32_t* bits) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t words = mask_words(a.Sk);
  const int64_t k0 = (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * kMaskSpan;
  if (k0 >= a.Sk) return;
  for (int64_t row = blockIdx.y; row < static_cast<int64_t>(a.B) * a.Sq; row += gridDim.y) {
    const int64_t b = row / a.Sq, i = row - b * a.Sq;
    const uint8_t* m = a.mask + b * a.ms[0] + i * a.ms[1];
    uint32_t mine = 0u;
#pragma unroll
    for (int w0 = 0; w0 < 32; w0 += 8) {
      uint8_t on[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const int64_t key = k0 + 32 * (w0 + w) + lane;
        on[w] = key < a.Sk ? __ldcg(m + key) : 0;
      }
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const uint32_t word = __ballot_sync(0xffffffffu, on[w] != 0);
        if (lane == w0 + w) mine = word;
      }
    }
    if (k0 / 32 + lane < words) bits[row * words + k0 / 32 + lane] = mine;
  }
}

// MQ: several query positions per kv head; row r = head * seq_q + query.
template <int NG, bool MQ, bool F16>
__global__ void __launch_bounds__(Q4Layout<NG>::kThreads, 1)
    gqa_decode_q4_kernel(const __grid_constant__ CUtensorMap tmk,
                         const __grid_constant__ CUtensorMap tmv, const DecodeArgs a,
                         const int tiles_per_group, const int passes, const int units,
                         const int stages, const int split, const int lead,
                         const uint32_t* mask_bits, uint32_t* counters) {
  using L = Q4Layout<NG>;
  constexpr int HP = L::HP, D = L::D, W = L::W, P = L::kPitch, R = L::kRow;
  constexpr int kSub = L::kSub, kChunk = L::kChunk, kChunks = L::kChunks;
  constexpr int NW = kSub / 2;  // 32-key words of a chunk's visibility

  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                             ~static_cast<uintptr_t>(127));
  float* scr = reinterpret_cast<float*>(ring + stages * L::kStage);
  uint16_t* q_next = reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(scr) + L::kScratch);
  uint32_t* vis_s = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(q_next) + L::kQRows);
  uint64_t* full = reinterpret_cast<uint64_t*>(vis_s + stages * (L::kVis / 4));
  uint64_t* empty = full + stages;
  uint64_t* q_full = empty + stages;     // the second group's Q rows landed
  uint64_t* scr_free = q_full + 1;       // the scratch's states have been merged
  volatile int* abort_flag = reinterpret_cast<volatile int*>(scr_free + 1);
  volatile int* last_flag = abort_flag + 1;
  volatile int* fast_flag = abort_flag + 2;  // the final split group is merged here directly
  // Ticket count of the final split group, read by the producer near the end
  // of the range (kNoPeek until then).
  volatile uint32_t* peek_count = reinterpret_cast<volatile uint32_t*>(abort_flag + 3);
  constexpr uint32_t kNoPeek = 0xFFFFFFFFu;
  int* flushed = const_cast<int*>(abort_flag) + 4;  // warps whose state of a mid group is in the scratch
  volatile int* mid_last = abort_flag + 5;  // the range's first group is this CTA's to merge
  volatile int* piece = abort_flag + 6;     // ragged, every group in ranges of its own: most units of one
  int* len_s = const_cast<int*>(abort_flag) + 8;
  int* pre_s = len_s + a.B;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const bool ragged = a.lens != nullptr;
  const int gpb = a.Hkv * passes;
  auto trace = [&]() { return a.trace + blockIdx.x * kDecodeTraceWords; };  // diagnostics
  const uint64_t t_entry = (a.trace != nullptr && threadIdx.x == 0) ? globaltimer_ns() : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kChunks);  // one arrival per chunk
    }
    mbar_init(q_full, 1);
    mbar_init(scr_free, 1);
    *abort_flag = 0;
    *fast_flag = 0;
    *peek_count = kNoPeek;
    *flushed = 0;
    *mid_last = 0;
    fence_mbar_init();
  }
  // Q rows past the group and dims past head_dim stay zero.
  for (int i = threadIdx.x; i < L::kQRows / 16; i += blockDim.x)
    reinterpret_cast<uint4*>(q_next)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  Sched sc;
  sc.pre = ragged ? pre_s : nullptr;
  sc.len = ragged ? len_s : nullptr;
  sc.per_b = gpb * (tiles_per_group + lead);
  sc.gpb = gpb;
  sc.B = a.B;
  // Nothing global that earlier work on the stream writes is read, and nothing
  // is written, before griddep_wait.  With lengths that is here, for every
  // thread; without, the cut into ranges needs no memory, and each role waits
  // right before its first access (the way there is long: cold instructions).
  if (ragged) {
    griddep_wait();
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
      int len = a.lens[b];
      if (len < 0 || len > a.Sk) {
        if (blockIdx.x == 0) atomicOr(a.err, kErrKvLength);
        len = len < 0 ? 0 : a.Sk;
      }
      len_s[b] = len;
    }
    __syncthreads();
    if (warp == 0) {
      auto tiles_of = [&](int b) {
        return decode_key_range(len_s[b], a.Sk, a.Sq, a.causal, a.causal_offset, a.window).tiles;
      };
      // Every group in ranges of its own (see below): the fewest units per
      // range with which they are no more than the CTAs.
      int units_of_piece = 0;
      const int grid = static_cast<int>(gridDim.x);
      if (a.B <= grid / gpb) {
        int most = 0, all = 0;
        for (int b = lane; b < a.B; b += 32) {
          const int t = tiles_of(b);
          most = max(most, t);
          all += t;
        }
        most = __reduce_max_sync(0xffffffffu, most);
        all = __reduce_add_sync(0xffffffffu, all);
        int lo = 1, hi = most;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          int n = 0;
          for (int b = lane; b < a.B; b += 32) n += (tiles_of(b) + mid - 1) / mid;
          n = __reduce_add_sync(0xffffffffu, n);
          if (n <= grid / gpb)
            hi = mid;
          else
            lo = mid + 1;
        }
        if (lo <= (all + lead * a.B) / (grid / gpb) + kApartUnits) units_of_piece = lo;
      }
      if (lane == 0) *piece = units_of_piece;
      // pre[b + 1] = sum over entries <= b of their places (or ranges).
      int carry = 0;
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane;
        int v = 0;
        if (b < a.B)
          v = gpb * (units_of_piece > 0 ? (tiles_of(b) + units_of_piece - 1) / units_of_piece
                                        : lead + tiles_of(b));
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
  __syncthreads();
  griddep_launch_dependents();
  if (a.trace != nullptr && threadIdx.x == 0) {
    for (int w = 0; w < kDecodeTraceWords; ++w) trace()[w] = 0;
    trace()[kTrEntry] = t_entry;
  }
  sc.total = ragged ? pre_s[a.B] : units;
  sc.P = static_cast<int>(gridDim.x) < sc.total ? static_cast<int>(gridDim.x) : sc.total;

  Cursor cu;
  // Address of row hl (a head, or a (head, query) pair) of kv head kv of entry b.
  auto q_row = [&](int b, int kv, int hl) {
    const int hh = MQ ? hl / a.Sq : hl, qi = MQ ? hl % a.Sq : 0;
    return a.q + b * a.qs[0] + static_cast<int64_t>(kv * a.g + hh) * a.qs[1] +
           static_cast<int64_t>(qi) * a.qs[2];
  };
  // Group (kv head and pass of one entry) of a place: its index in the launch,
  // the place of its first unit, its units, and the CTAs that share those.
  struct Group {
    int b, kv, pass, id, beg, tiles, c_lo, c_hi, rows;
  };
  auto group_of_entry = [&](int gi) {  // the cursor's entry
    Group g;
    g.id = cu.b * gpb + gi;
    g.b = cu.b;
    g.kv = gi / passes;
    g.pass = gi - g.kv * passes;
    g.tiles = cu.kr.tiles;
    g.rows = min(HP, a.rows - g.pass * HP);
    return g;
  };
  auto range_of_entry = [&](int b) {
    return decode_key_range(sc.len ? sc.len[b] : a.Sk, a.Sk, a.Sq, a.causal, a.causal_offset,
                            a.window);
  };
  // The units of a launch are cut into CTA ranges in one of two ways.
  //  apart: every group has ranges of its own, `split` of them (uniform), or
  //    as many as keep each within `piece` units (ragged).  No CTA changes
  //    groups.  A place is a unit of the CTA's own group.
  //  even: all groups lie end to end and are cut into equal ranges.  Every
  //    group has `lead` empty places (what a change of groups costs, in units)
  //    and then one per unit.
  const bool apart = ragged ? *piece > 0 : split > 0;
  auto id_at = [&](int place) {  // even: the group of a place; the cursor goes to its entry
    if (cu.b < 0 || place < cu.beg || place >= cu.end) {
      cu.b = sc.batch_of(place);
      cu.beg = sc.start_of(cu.b);
      cu.kr = range_of_entry(cu.b);
      cu.end = cu.beg + gpb * (cu.kr.tiles + lead);
    }
    return cu.b * gpb + (place - cu.beg) / (cu.kr.tiles + lead);
  };
  Group own{};  // apart: the CTA's group
  auto group_at = [&](int place) {
    if (apart) return own;
    const int id = id_at(place);
    Group g = group_of_entry(id - cu.b * gpb);
    g.beg = cu.beg + (id - cu.b * gpb) * (cu.kr.tiles + lead) + lead;
    g.c_lo = cta_of_unit(g.beg, sc.total, sc.P);
    g.c_hi = cta_of_unit(g.beg + g.tiles - 1, sc.total, sc.P);
    return g;
  };
  const int cta = static_cast<int>(blockIdx.x);
  int v_begin = 0, v_end = 0;  // this CTA's places
  if (cta < sc.P) {
    if (apart) {
      int gi, part, parts;
      if (ragged) {
        cu.b = sc.batch_of(cta);
        cu.kr = range_of_entry(cu.b);
        parts = (cu.kr.tiles + *piece - 1) / *piece;
        const int r = cta - sc.start_of(cu.b);
        gi = r / parts;
        part = r - gi * parts;
      } else {
        parts = split;
        const int id = cta / split;
        part = cta - id * split;
        cu.b = id / gpb;
        gi = id - cu.b * gpb;
        cu.kr = range_of_entry(cu.b);
      }
      own = group_of_entry(gi);
      own.beg = 0;
      own.c_lo = cta - part;
      own.c_hi = own.c_lo + parts - 1;
      v_begin = static_cast<int>(static_cast<int64_t>(part) * own.tiles / parts);
      v_end = static_cast<int>(static_cast<int64_t>(part + 1) * own.tiles / parts);
    } else {
      v_begin = range_start(cta, sc.total, sc.P);
      v_end = range_start(cta + 1, sc.total, sc.P);
      if (v_begin < v_end) {  // a range that ends in a group's lead has no unit of that group
        const Group g = group_at(v_end - 1);
        if (v_end <= g.beg) v_end = max(v_begin, g.beg - lead);
      }
    }
  }

  if (warp == W) {
    // ------------------------------------------------------------ producer
    // Group by group of the range, with everything that a unit's copies need
    // kept in counters: the producer shares its scheduler with consumers, and
    // a unit has to be on its way every ~800 cycles.  With a paged cache the
    // units go in blocks of 16: lane i holds the page of half i % 2 (64 keys)
    // of unit i / 2 of the block, read one block ahead of its use, so that the
    // table's latency stays off the path of the copies.
    constexpr int kBlock = 32 / (KT / kDecodePageBox);
    const bool paged = a.bt != nullptr;
    int it = 0, s = 0;          // units issued; stage of the next one
    uint32_t parity = 1;        // of the wait for a free stage (passes at once in round 0)
    bool ok = true, q_sent = false;
    if (lane == 0) {
      prefetch_tmap(&tmk);
      prefetch_tmap(&tmv);
    }
    for (int va = v_begin; va < v_end && ok;) {
      const Group grp = group_at(va);
      const int t0 = max(va - grp.beg, 0);               // units [t0, t1) of the group
      const int t1 = min(v_end - grp.beg, grp.tiles);
      const int kv = grp.kv, b = grp.b;
      // With a mask: this lane's query of the pass (they go in row order,
      // wrapping) and its bits.
      const uint32_t* my_bits = nullptr;
      if (a.has_mask && lane / (KT / 32) < (MQ ? min(a.Sq, HP) : 1)) {
        const int qi = MQ ? (grp.pass * HP + lane / (KT / 32)) % a.Sq : 0;
        my_bits = mask_bits + (static_cast<int64_t>(b) * a.Sq + qi) * mask_words(a.Sk) +
                  lane % (KT / 32);
      }
      int key0 = (t0 + cu.kr.t0) * KT;
      if (va == v_begin && !ragged) {
        // Contiguous caches: the first units start towards L2 before the grid
        // dependency resolves (earlier work may still be writing the cache;
        // these are hints, the copies below read what it wrote).
        if (!paged && lane < 2 && t0 + lane < t1) {
          tma_prefetch_4d(&tmk, 0, key0 + lane * KT, kv, b);
          tma_prefetch_4d(&tmv, 0, key0 + lane * KT, kv, b);
        }
        griddep_wait();
      }
      if (a.trace != nullptr && lane == 0 && va == v_begin) trace()[kTrReady] = globaltimer_ns();
      const int len = sc.len ? sc.len[b] : a.Sk;
      // Page and row of a 64-key box; one past the sequence's length takes
      // page num_pages, which is out of range: TMA fills it with zeros.
      auto page_of = [&](int key, bool wanted) {
        if (!wanted || key >= len) return a.num_pages;
        const int page = __ldcg(a.bt + b * a.bt_stride + key / a.page_size);
        if (page >= 0 && page < a.num_pages) return page;
        atomicOr(a.err, kErrPage);
        return a.num_pages;  // read as zeros
      };
      const int at = (lane >> 1) * KT + (lane & 1) * kDecodePageBox;
      int next_page = paged ? page_of(key0 + at, t0 + (lane >> 1) < t1) : 0;
      for (int u = t0; u < t1 && ok;) {
        const int my_page = next_page;
        const int my_row = paged ? (key0 + at) % a.page_size : 0;
        const int u_stop = min(u + kBlock, t1);
        if (paged) next_page = page_of(key0 + kBlock * KT + at, u + kBlock + (lane >> 1) < t1);
        for (int i = 0; u < u_stop; ++u, ++i, key0 += KT) {
          int page[2] = {0, 0}, row[2] = {0, 0};
          if (paged) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              page[h] = __shfl_sync(0xffffffffu, my_page, 2 * i + h);
              row[h] = __shfl_sync(0xffffffffu, my_row, 2 * i + h);
            }
          }
          // Mask bits of the unit's 128 keys, lane 4 i + w: query i of the pass,
          // keys 32 w .. + 31.  (Read before the wait for a free stage.)
          const uint32_t bits = my_bits != nullptr ? __ldcg(my_bits + key0 / 32) : 0u;
          // (Every lane waits: the warp stays converged.)
          ok = __all_sync(0xffffffffu, mbar_try_wait(&empty[s], parity) ||
                                           mbar_wait(&empty[s], parity, abort_flag, a.err,
                                                     kErrDecodeWait, a.wait_ns));
          if (ok && (apart ? grp.id * tiles_per_group : grp.beg - lead * (grp.id + 1)) + u ==
                        a.withhold_unit) {
            // Test of the bounded waits, as in the 16-bit decode: nothing more
            // is issued, and the consumers' wait for this unit runs out.
            const uint64_t t0 = globaltimer_ns();
            while (!*abort_flag && globaltimer_ns() - t0 < 4 * a.wait_ns) {
            }
            __syncwarp();
            ok = false;
          }
          if (!ok) break;
          if (a.has_mask) {
            vis_s[s * (L::kVis / 4) + lane] = bits;
            __syncwarp();  // (lane 0's arrival below releases them)
          }
          if (lane == 0) {
            uint8_t* st = ring + s * L::kStage;
            mbar_arrive_expect_tx(&full[s], L::kStage);
            if (paged) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint8_t* dst = st + h * kDecodePageBox * P;
                tma_load_4d(dst, &tmk, &full[s], 0, row[h], kv, page[h]);
                tma_load_4d(dst + L::kTile, &tmv, &full[s], 0, row[h], kv, page[h]);
              }
            } else {
              tma_load_4d(st, &tmk, &full[s], 0, key0, kv, b);
              tma_load_4d(st + L::kTile, &tmv, &full[s], 0, key0, kv, b);
            }
            if (a.trace != nullptr && it == 0) trace()[kTrFirstIssue] = globaltimer_ns();
          }
          __syncwarp();
          ++it;
          if (++s == stages) {
            s = 0;
            parity ^= 1u;
          }
        }
      }
      const int vb = grp.beg + t1;
      if (va == v_begin && vb < v_end && ok) {
        // The Q rows of the range's second group: at the change of groups
        // they would cost the consumers a round trip.  (The first group's
        // come while its first unit does; a range over more groups has short
        // ones, and the consumers fetch the others' when they get there.)
        const Group next = group_at(vb);
        if (lane == 0)
          mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(next.rows * a.Dv * 2));
        __syncwarp();
        if (lane < next.rows)
          bulk_load(q_next + lane * D, q_row(next.b, next.kv, next.pass * HP + lane),
                    static_cast<uint32_t>(a.Dv * 2), q_full);
        q_sent = true;
      }
      va = vb;
    }
    if (lane == 0) {
      if (a.trace != nullptr) trace()[kTrLastIssue] = globaltimer_ns();
      // Final group split over several CTAs: once the consumers are on the
      // range's last unit, read its ticket count for their final merge (the
      // fence makes the partials published before those tickets visible).
      if (!*abort_flag && v_begin < v_end) {
        const Group g = group_at(v_end - 1);
        if (g.c_lo != g.c_hi) {
          const int j = it - 2;  // second-to-last unit of the range
          if (j < 0 || mbar_wait(&empty[j % stages], static_cast<uint32_t>((j / stages) & 1),
                                 abort_flag, a.err, kErrDecodeWait, a.wait_ns)) {
            const uint32_t n = ld_relaxed_gpu(&counters[g.id]);
            fence_acq_rel_gpu();
            *peek_count = n;
          }
        }
      }
      // Unwind: no copy may still be landing in this CTA's shared memory.
      if (*abort_flag)
        for (int j = it > stages ? it - stages : 0; j < it; ++j)
          mbar_wait_drain(&full[j % stages], static_cast<uint32_t>((j / stages) & 1),
                          a.wait_ns / 4);
      if (*abort_flag && q_sent) mbar_wait_drain(q_full, 0, a.wait_ns / 4);
    }
  } else {
    // ------------------------------------------------------------ consumers
    const int c = lane & 3, r8 = lane >> 2;
    auto sync_consumers = [] { asm volatile("bar.sync 1, %0;" ::"n"(W * 32) : "memory"); };
    // Output row hr of a group's pass, dims 4 d4 .. + 3.
    auto write_out = [&](const Group& g, int hr, int d4, float lsum, const float4& acc) {
      if (4 * d4 >= a.Dv) return;
      const int row = g.pass * HP + hr;
      const int hh = MQ ? row / a.Sq : row, qi = MQ ? row % a.Sq : 0;
      const float inv = 1.f / lsum;  // no visible key: 0 * inf = NaN
      uint2 pk;
      pk.x = pack2<F16>(acc.x * inv, acc.y * inv);
      pk.y = pack2<F16>(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(a.out + g.b * a.os[0] +
                                static_cast<int64_t>(g.kv * a.g + hh) * a.os[1] +
                                static_cast<int64_t>(qi) * a.os[2] + 4 * d4) = pk;
    };
    // Partial slot of a CTA for a split group: only a range's first and last
    // group can be split, so there are two.
    auto slot_of = [&](int cta, int id) {
      if (apart) return cta * 2 * HP;
      return (cta * 2 + (id_at(range_start(cta, sc.total, sc.P)) == id ? 0 : 1)) * HP;
    };
    // All partials of a split group are published: their merge by the whole
    // consumer group, eight contributors' loads in flight at a time.
    auto merge_partials = [&](const Group& g) {
      const int n = g.c_hi - g.c_lo + 1;
      int* slot = reinterpret_cast<int*>(scr);
      for (int k = threadIdx.x; k < n; k += W * 32) slot[k] = slot_of(g.c_lo + k, g.id);
      sync_consumers();
      for (int i = threadIdx.x; i < g.rows * (D / 4); i += W * 32) {
        const int hr = i / (D / 4), d4 = i % (D / 4);
        float M = -INFINITY, lsum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = 0; k0 < n; k0 += kBatch) {
          float2 ml[kBatch];
          float4 ov[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            ml[k] = make_float2(-INFINITY, 0.f);
            ov[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k0 + k < n) {
              const int64_t at = slot[k0 + k] + hr;
              ml[k] = __ldcg(&a.part_ml[at]);
              ov[k] = __ldcg(reinterpret_cast<const float4*>(&a.part_o[at * D + 4 * d4]));
            }
          }
          float top = M;
#pragma unroll
          for (int k = 0; k < kBatch; ++k) top = fmaxf(top, ml[k].x);
          const float ref = exp_ref(top), old = fast_exp2(M - ref);
          M = top;
          lsum *= old;
          acc.x *= old;
          acc.y *= old;
          acc.z *= old;
          acc.w *= old;
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const float w = fast_exp2(ml[k].x - ref);
            lsum = fmaf(w, ml[k].y, lsum);
            acc.x = fmaf(w, ov[k].x, acc.x);
            acc.y = fmaf(w, ov[k].y, acc.y);
            acc.z = fmaf(w, ov[k].z, acc.z);
            acc.w = fmaf(w, ov[k].w, acc.w);
          }
        }
        write_out(g, hr, d4, lsum, acc);
      }
      if (threadIdx.x == 0) atomicExch(&counters[g.id], 0u);
      sync_consumers();
    };

    int n_flush = 0;           // groups whose states went through the scratch
    int v_second = v_end;      // where the range's second group begins
    int done = 0;              // units of the groups before
    for (int va = v_begin; va < v_end;) {
      // One group (kv head and pass of one entry): units [t0, t1) of it.
      const Group grp = group_at(va);
      const int t0 = max(va - grp.beg, 0);
      const int t1 = min(v_end - grp.beg, grp.tiles);
      const int vb = grp.beg + t1;
      const int kv = grp.kv, pass = grp.pass, b = grp.b;
      const int len = sc.len ? sc.len[b] : a.Sk;
      const KeyRange kr = cu.kr;
      if (va == v_begin) {
        v_second = vb;
        if (!ragged) griddep_wait();
      }
      // (A wait that gave up sets the abort flag: the arithmetic goes on with
      // whatever is there, the result is undefined.)
      const bool stashed = va == v_second;
      if (stashed) mbar_wait(q_full, 0, abort_flag, a.err, kErrDecodeWait, a.wait_ns);

      // Q as B fragments, thread (r8, c): row r8 of the pass, dims 32 t + 8 c
      // .. + 7; and the sums over each group's dims, the factors of the
      // minima, as two 16-bit parts: a record's head is the A operand of a
      // product of its own, and its scales meet zeros.
      uint32_t bq[NG][4], bm[2];
      float fac[2];         // what turns this thread's two rows' scores into base 2
      int vlo[2], vhi[2];   // their visible keys, without the mask
      {
        const int hl = pass * HP + r8;
        const uint16_t* qrow = stashed ? q_next + r8 * D : q_row(b, kv, hl);
        float f[NG][8];
        float amax = 0.f;
#pragma unroll
        for (int t = 0; t < NG; ++t) {
          uint4 x = make_uint4(0u, 0u, 0u, 0u);
          if (stashed || (hl < a.rows && 32 * t + 8 * c < a.Dv))
            x = *reinterpret_cast<const uint4*>(qrow + 32 * t + 8 * c);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[t][2 * i] = to_f32<F16>(w[i] & 0xFFFFu);
            f[t][2 * i + 1] = to_f32<F16>(w[i] >> 16);
            amax = fmaxf(amax, fmaxf(fabsf(f[t][2 * i]), fabsf(f[t][2 * i + 1])));
          }
        }
        // Power of two that Q is scaled by, and what the scores then lack
        // (the codes' own step is 2^-133 in bf16, 2^-24 in fp16).
        float up, back;
        if (F16) {
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
          const int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
          const int e = amax > 0.f && ex < 16 ? 14 - ex : 0;
          up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
          back = __uint_as_float(static_cast<uint32_t>(127 + 24 - e) << 23);
        } else {
          up = 0x1p64f;
          back = 0x1p69f;
        }
        float mine = 0.f;  // group c's sum
#pragma unroll
        for (int t = 0; t < NG; ++t) {
          float s = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) s += f[t][i];
          s += __shfl_xor_sync(0xffffffffu, s, 1);
          s += __shfl_xor_sync(0xffffffffu, s, 2);
          if (t == c) mine = s / back;  // a power of two: exact
          const float odd = up * 0.0625f;
          bq[t][0] = pack2<F16>(f[t][0] * up, f[t][4] * up);
          bq[t][1] = pack2<F16>(f[t][1] * odd, f[t][5] * odd);
          bq[t][2] = pack2<F16>(f[t][2] * up, f[t][6] * up);
          bq[t][3] = pack2<F16>(f[t][3] * odd, f[t][7] * odd);
        }
        const uint32_t high = to_16<F16>(mine);
        bm[0] = high << 16;
        bm[1] = to_16<F16>(mine - to_f32<F16>(high)) << 16;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          fac[e] = a.scale_log2 * __shfl_sync(0xffffffffu, back, (2 * c + e) * 4);
          vlo[e] = kr.lo;
          vhi[e] = kr.hi;
          if (MQ) {
            const int row = pass * HP + 2 * c + e;
            const int i = (row < a.rows ? row : 0) % a.Sq;
            const int64_t top = i + a.causal_offset + (len - a.Sk);  // query i's diagonal
            int64_t lo = 0, hi = len;
            if (a.causal) {
              hi = top + 1 < hi ? top + 1 : hi;
              if (a.window > 0 && top - a.window + 1 > 0) lo = top - a.window + 1;
            }
            vlo[e] = static_cast<int>(lo < len ? lo : len);
            vhi[e] = static_cast<int>(hi > 0 ? hi : 0);
          }
        }
      }
      // Keys that every query sees (without a mask): the first one's upper
      // limit, the last one's lower limit.
      int all_lo = kr.lo, all_hi = kr.hi;
      if (MQ && a.causal) {
        const int64_t top0 = a.causal_offset + (len - a.Sk);
        all_hi = static_cast<int>(top0 + 1 < 0 ? 0 : (top0 + 1 < len ? top0 + 1 : len));
        if (a.window > 0) {
          const int64_t lo = top0 + a.Sq - a.window;
          all_lo = static_cast<int>(lo < 0 ? 0 : (lo < len ? lo : len));
        }
      }
      // With a mask: where the bits of this thread's two rows' queries are.
      int vis_at[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        vis_at[e] = (!MQ ? 0 : (a.Sq < HP ? (2 * c + e) % a.Sq : 2 * c + e)) * (KT / 32);

      float o[NG][2][4];
      uint64_t corr[NG];  // of both rows
      float osum[4];  // fp16: lanes 4 t + c hold group t's summed weights
      uint64_t pow[NG];   // both rows' powers of two on the groups' weights, in o and osum
      uint32_t limit[NG / 2];  // value scales that they allow, two groups to a word
      // The exponent reference (running maximum), its negative with 0 for
      // -inf, the score above which it moves, and the sum of the weights.
      float m_ref[2], m_neg[2], m_top[2], l[2];
#pragma unroll
      for (int x = 0; x < 4; ++x) osum[x] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m_ref[e] = m_top[e] = -INFINITY;
        m_neg[e] = l[e] = 0.f;
#pragma unroll
        for (int t = 0; t < NG; ++t) {
          corr[t] = 0;
          pow[t] = f2_pack(0x1p100f, 0x1p100f);
          limit[t / 2] = 0u;
#pragma unroll
          for (int x = 0; x < 4; ++x) o[t][e][x] = 0.f;
        }
      }

      // Chunks of the CTA's range are numbered through; warp w takes those
      // that are w modulo W.
      const int x0 = done * kChunks, x1 = (done + t1 - t0) * kChunks;
      int x = x0 + (warp - x0 % W + W) % W;
      int s = (x / kChunks) % stages;
      uint32_t parity = static_cast<uint32_t>((x / kChunks) / stages) & 1u;
      for (int it = x / kChunks; x < x1; x += W) {
        for (; it < x / kChunks; ++it)
          if (++s == stages) {
            s = 0;
            parity ^= 1u;
          }
        const int chunk = x % kChunks;
        const int key0 = (t0 + kr.t0 + it - done) * KT + chunk * kChunk;
        const bool landed =
            mbar_try_wait(&full[s], parity) ||
            mbar_wait(&full[s], parity, abort_flag, a.err, kErrDecodeWait, a.wait_ns);
        if (a.trace != nullptr && x == 0 && lane == 0) trace()[kTrFirstLand] = globaltimer_ns();
        // Visible keys of the chunk, one bit each, where some are not: the
        // range of each row, and its query's mask bits.
        uint32_t vis[2][NW];
        bool whole = key0 >= all_lo && key0 + kChunk <= all_hi;
        bool none = key0 >= kr.hi || key0 + kChunk <= kr.lo;
        if (!none && (!whole || a.has_mask)) {
          const uint32_t* words = vis_s + s * (L::kVis / 4) + chunk * NW;
          uint32_t all = ~0u, any = 0u;
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int w = 0; w < NW; ++w) {
              vis[e][w] = below(vhi[e] - key0 - 32 * w) & ~below(vlo[e] - key0 - 32 * w);
              if (a.has_mask) vis[e][w] &= words[vis_at[e] + w];
              all &= vis[e][w];
              any |= vis[e][w];
            }
          whole = __all_sync(0xffffffffu, all == ~0u);
          none = !__any_sync(0xffffffffu, any != 0u);
        }
        // (A wait that gave up sets the abort flag: the arithmetic is skipped,
        // the walk goes on, so that all warps reach the same barriers.)
        if (!__all_sync(0xffffffffu, landed) || none) {
          if (lane == 0) mbar_arrive(&empty[s]);
          continue;
        }
        const uint32_t kb = smem_u32(ring + s * L::kStage) + chunk * kChunk * P;
        const uint32_t vb = kb + L::kTile;
        // ldmatrix row of this lane: 8-key halves, then groups.
        const uint32_t at =
            (((lane >> 3) & 1) * 8 + (lane & 7)) * P + kHeadBytes + (lane >> 4) * 16;

        float sv[kSub][4];  // scores: keys r8 (0, 1) and r8 + 8 (2, 3), rows 2 c + {0, 1}
#pragma unroll
        for (int j = 0; j < kSub; ++j) {
          const uint32_t kj = kb + j * 16 * P;
          uint32_t kw[NG][2], kp[2][NG], h0, h1;  // codes [group][key half], heads
#pragma unroll
          for (int t = 0; t < NG; t += 2)
            ldmatrix_x4(kw[t][0], kw[t][1], kw[t + 1][0], kw[t + 1][1], kj + at + t * 16);
          ldmatrix_x2(h0, h1, kj + (lane & 15) * P);
          load_params<NG>(kp[0], kj + r8 * P);
          load_params<NG>(kp[1], kj + (r8 + 8) * P);
          mma_zero<F16>(sv[j], h0, h1, h0, h1, bm[0], bm[1]);
#pragma unroll
          for (int t = 0; t < NG; ++t) {
            const uint32_t a8 = kw[t][0] >> 8, b8 = kw[t][1] >> 8;
            float acc[4];
            mma_zero<F16>(acc, kw[t][0] & 0x000F000Fu, kw[t][1] & 0x000F000Fu,
                          kw[t][0] & 0x00F000F0u, kw[t][1] & 0x00F000F0u, bq[t][0], bq[t][1]);
            mma_16816<F16>(acc, a8 & 0x000F000Fu, b8 & 0x000F000Fu, a8 & 0x00F000F0u,
                           b8 & 0x00F000F0u, bq[t][2], bq[t][3]);
#pragma unroll
            for (int y = 0; y < 4; ++y)
              sv[j][y] = fmaf(scale_of<F16>(kp[y >> 1][t]), acc[y], sv[j][y]);
          }
        }
        auto rest = [&](auto all_seen) {
          constexpr bool kWhole = decltype(all_seen)::value;
          // Scores in base 2 are sv * fac; with hidden keys the product is
          // taken first and replaced by -inf.
          bool raise = false;
          bool seen[kSub][4];
#pragma unroll
          for (int j = 0; j < kSub; ++j)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int e = y & 1;
              float& t = sv[j][y];
              seen[j][y] =
                  kWhole || ((vis[e][j >> 1] >> (r8 + 16 * (j & 1) + 8 * (y >> 1))) & 1u) != 0u;
              if (!kWhole) t = seen[j][y] ? t * fac[e] : -INFINITY;
              raise |= (kWhole ? t * fac[e] : t) > m_top[e];
            }
          // The largest scales of the values, against what the powers allow.
          {
            uint32_t most[NG];
#pragma unroll
            for (int j = 0; j < kSub; ++j)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t w[NG];
                load_params<NG>(w, vb + (j * 16 + 8 * k + r8) * P);
#pragma unroll
                for (int t = 0; t < NG; ++t)
                  most[t] = j + k == 0 ? w[t] : max_number<F16>(most[t], w[t]);
              }
#pragma unroll
            for (int t = 0; t < NG; t += 2)
              raise |= max_number<F16>(__byte_perm(most[t], most[t + 1], 0x5410), limit[t / 2]) !=
                       limit[t / 2];
          }
          if (__any_sync(0xffffffffu, raise)) {
            // The reference goes to the maximum, rounded up; l and corr follow by
            // alpha (0 for a row without a key so far).  Powers of two are kept as
            // the bits of their exponent.
            const bool begun =
                __any_sync(0xffffffffu, m_ref[0] > -INFINITY || m_ref[1] > -INFINITY);
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float f = kWhole ? fac[e] : 1.f;
              float mx = -INFINITY;
#pragma unroll
              for (int j = 0; j < kSub; ++j) mx = fmax3(mx, sv[j][e] * f, sv[j][2 + e] * f);
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
              const float m_new = ceilf(fmaxf(m_ref[e], mx));
              alpha[e] = power_of_two(static_cast<int>(fmaxf(m_ref[e] - m_new, -127.f)));
              m_neg[e] = -exp_ref(m_new);
              m_ref[e] = m_new;
              m_top[e] = m_new + float(kLazyLog2);
            }
            // This chunk's largest weight of each group, as bf16 pairs of rows.
            uint32_t most[NG];
#pragma unroll
            for (int j = 0; j < kSub; ++j)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t w[NG];
                load_params<NG>(w, vb + (j * 16 + 8 * k + r8) * P);
                float pe[2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  pe[e] = fast_exp2(fmaf(sv[j][2 * k + e], kWhole ? fac[e] : 1.f, m_neg[e]));
#pragma unroll
                for (int t = 0; t < NG; ++t) {
                  const float scale = scale_of<F16>(w[t]);
                  const uint64_t ww = f2_mul(f2_pack(pe[0], pe[1]), f2_pack(scale, scale));
                  const uint32_t x =
                      pack_bf16x2(kWhole || seen[j][2 * k] ? f2_lo(ww) : 0.f,
                                  kWhole || seen[j][2 * k + 1] ? f2_hi(ww) : 0.f);
                  most[t] = max_number<false>(j + k == 0 ? 0u : most[t], x);
                }
              }
#pragma unroll
            for (int i = 4; i < 32; i <<= 1)
#pragma unroll
              for (int t = 0; t < NG; ++t)
                most[t] = max_number<false>(most[t], __shfl_xor_sync(0xffffffffu, most[t], i));
            // The powers follow the reference, as far as the largest weight (and
            // 2^kPowerMost) allows, and o and osum what is left.
#pragma unroll
            for (int t = 0; t < NG; ++t) {
              uint32_t to[2], high = 0u;
              float by[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                constexpr uint32_t kOne = 127u << 23;
                const uint32_t old = __float_as_uint(e ? f2_hi(pow[t]) : f2_lo(pow[t]));
                const uint32_t back = old + kOne - __float_as_uint(alpha[e]);  // old / alpha
                const uint32_t weight = (e ? most[t] : most[t] << 16) & 0x7F800000u;
                to[e] = min(min(back, (127u + kPowerMost) << 23),
                            2u * kOne - min(weight, 253u << 23));
                by[e] = alpha[e] > 0.f && to[e] + kOne > back
                            ? __uint_as_float(to[e] + kOne - back)
                            : 0.f;
                if (m_ref[e] > -INFINITY) high = max(high, to[e]);
              }
              const uint32_t code =
                  type_power<F16>(kLazyScaleLog2 + 127 - static_cast<int>(high >> 23));
              limit[t / 2] = t % 2 == 0 ? code : limit[t / 2] | (code << 16);
              pow[t] = f2_pack(__uint_as_float(to[0]), __uint_as_float(to[1]));
              if (begun) {
                corr[t] = f2_mul(corr[t], f2_pack(alpha[0], alpha[1]));
                if (F16 && r8 == t) {
                  osum[0] *= by[0];
                  osum[1] *= by[1];
                }
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                  for (int y = 0; y < 4; ++y) o[t][u][y] *= by[y & 1];
              }
            }
            l[0] *= alpha[0];
            l[1] *= alpha[1];
          }
#pragma unroll
          for (int j = 0; j < kSub; ++j) {
            uint32_t vw[NG][2], vp[2][NG];
            load_params<NG>(vp[0], vb + (j * 16 + r8) * P);
            load_params<NG>(vp[1], vb + (j * 16 + 8 + r8) * P);
#pragma unroll
            for (int t = 0; t < NG; t += 2)
              ldmatrix_x4_trans(vw[t][0], vw[t][1], vw[t + 1][0], vw[t + 1][1],
                                vb + j * 16 * P + at + t * 16);
#pragma unroll
            for (int y = 0; y < 4; ++y)
              sv[j][y] = fast_exp2(fmaf(sv[j][y], kWhole ? fac[y & 1] : 1.f, m_neg[y & 1]));
#pragma unroll
            for (int e = 0; e < 2; ++e) l[e] += sv[j][e] + sv[j][2 + e];
#pragma unroll
            for (int t = 0; t < NG; ++t) {
              uint32_t pb[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float scale = scale_of<F16>(vp[k][t]);
                float add = min_of<F16>(vp[k][t]);
                if (F16) add = fmaf(8.f, scale, add);
                const uint64_t pp = f2_pack(sv[j][2 * k], sv[j][2 * k + 1]);
                // (In this order: a weight of zero stays one.)
                const uint64_t ww = f2_mul(f2_mul(pp, pow[t]), f2_pack(scale, scale));
                if (kWhole) {
                  corr[t] = f2_fma(pp, f2_pack(add, add), corr[t]);
                  pb[k] = movmatrix_trans(pack_f16x2(f2_lo(ww), f2_hi(ww)));
                } else {  // a hidden key's parameters may be NaN
                  const bool s0 = seen[j][2 * k], s1 = seen[j][2 * k + 1];
                  const uint64_t pa = f2_mul(pp, f2_pack(add, add));
                  corr[t] = f2_add(corr[t], f2_pack(s0 ? f2_lo(pa) : 0.f, s1 ? f2_hi(pa) : 0.f));
                  pb[k] = movmatrix_trans(pack_f16x2(s0 ? f2_lo(ww) : 0.f, s1 ? f2_hi(ww) : 0.f));
                }
              }
              const uint32_t v0 = vw[t][0] >> 8, v1 = vw[t][1] >> 8;
              mma_f16_16816(o[t][0], vw[t][0] & 0x000F000Fu, vw[t][0] & 0x00F000F0u,
                            vw[t][1] & 0x000F000Fu, vw[t][1] & 0x00F000F0u, pb[0], pb[1]);
              mma_f16_16816(o[t][1], v0 & 0x000F000Fu, v0 & 0x00F000F0u, v1 & 0x000F000Fu,
                            v1 & 0x00F000F0u, pb[0], pb[1]);
              if (F16) {  // ones in row t: the group's sum of weights
                const uint32_t one = r8 == t ? 0x3C003C00u : 0u;
                mma_f16_16816(osum, one, 0u, one, 0u, pb[0], pb[1]);
              }
            }
          }
          // The stage goes back when every word of it is in registers (the
          // products above have used them), with every lane's loads before
          // lane 0's arrival and, by the proxy fence, before the next copy, an
          // access of the async proxy that the mbarrier alone does not order.
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[s]);
        };
        if (whole)
          rest(BoolConst<true>{});
        else
          rest(BoolConst<false>{});
      }

      // ---- end of the group: the W warps' states meet in shared memory.
      if (a.trace != nullptr && threadIdx.x == 0 && vb == v_end) trace()[kTrLastTile] = globaltimer_ns();
      const bool final_group = vb == v_end;
      done += t1 - t0;
      const int n_contrib = grp.c_hi - grp.c_lo + 1;
      if (final_group && threadIdx.x == 0) {
        // The other contributors of the range's last group have mostly
        // published long ago (it was the first of their range); the producer
        // read the tickets and fenced at gpu scope, and acquiring its store
        // at CTA scope orders the loads of the partials after theirs.
        int fast = 0;
        if (n_contrib > 1 && n_contrib <= kFastMerge &&
            *peek_count == static_cast<uint32_t>(n_contrib - 1)) {
          fence_acq_rel_cta();
          fast = 1;
        }
        *fast_flag = fast;
      }
      // The scratch is free once the last group's states have been merged.
      if (n_flush > 0)
        mbar_wait(scr_free, static_cast<uint32_t>((n_flush - 1) & 1), abort_flag, a.err,
                  kErrDecodeWait, a.wait_ns);
      ++n_flush;
      float* mine = scr + warp * HP * R;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float* row = mine + (2 * c + e) * R;
        float lv = l[e];
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) lv += __shfl_xor_sync(0xffffffffu, lv, i);
#pragma unroll
        for (int t = 0; t < NG; ++t) {
          float cv = e ? f2_hi(corr[t]) : f2_lo(corr[t]);
#pragma unroll
          for (int i = 4; i < 32; i <<= 1) cv += __shfl_xor_sync(0xffffffffu, cv, i);
          const float off = power_of_two(-exponent_of(e ? f2_hi(pow[t]) : f2_lo(pow[t])));
          if (F16) cv = fmaf(-8.f * off, __shfl_sync(0xffffffffu, osum[e], 4 * t + c), cv);
          // Codes carry 2^-24, those of odd nibbles 2^-20, and the group's power.
          *reinterpret_cast<float4*>(row + 32 * t + 4 * r8) = make_float4(
              fmaf(o[t][0][e] * 0x1p24f, off, cv), fmaf(o[t][0][2 + e] * 0x1p20f, off, cv),
              fmaf(o[t][1][e] * 0x1p24f, off, cv), fmaf(o[t][1][2 + e] * 0x1p20f, off, cv));
        }
        if (r8 == 0) *reinterpret_cast<float2*>(row + D) = make_float2(m_ref[e], lv);
      }
      const int quads = grp.rows * (D / 4);
      // Row hr of the pass, dims 4 d4 .. + 3 over the W states: (M, l, O).
      auto merge_warps = [&](int hr, int d4, float& M, float& lsum, float4& acc) {
        M = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, scr[(w * HP + hr) * R + D]);
        lsum = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        const float ref = exp_ref(M);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float* row = scr + (w * HP + hr) * R;
          const float wt = fast_exp2(row[D] - ref);
          lsum = fmaf(wt, row[D + 1], lsum);
          const float4 ov = *reinterpret_cast<const float4*>(row + 4 * d4);
          acc.x = fmaf(wt, ov.x, acc.x);
          acc.y = fmaf(wt, ov.y, acc.y);
          acc.z = fmaf(wt, ov.z, acc.z);
          acc.w = fmaf(wt, ov.w, acc.w);
        }
      };
      // Quads i0, i0 + step, ...: written out (a whole group), or published as
      // this CTA's partial (a split one).
      auto merge_and_store = [&](int i0, int step) {
        const int base = n_contrib > 1 ? slot_of(blockIdx.x, grp.id) : 0;
        for (int i = i0; i < quads; i += step) {
          const int hr = i / (D / 4), d4 = i % (D / 4);
          float M, lsum;
          float4 acc;
          merge_warps(hr, d4, M, lsum, acc);
          if (n_contrib == 1) {
            write_out(grp, hr, d4, lsum, acc);
          } else {
            const int64_t at = base + hr;
            *reinterpret_cast<float4*>(&a.part_o[at * D + 4 * d4]) = acc;
            if (d4 == 0) a.part_ml[at] = make_float2(M, lsum);
          }
        }
      };
      if (!final_group) {
        // The range goes on: the warp that comes last merges the states by
        // itself, the others are already at the next group.
        __syncwarp();
        int last = 0;
        if (lane == 0) {
          fence_acq_rel_cta();
          last = atomicAdd(flushed, 1) == W - 1;
          if (last) {
            *flushed = 0;
            fence_acq_rel_cta();
          }
        }
        last = __shfl_sync(0xffffffffu, last, 0);
        if (last) {
          merge_and_store(lane, 32);
          __syncwarp();
          if (lane == 0) {
            // (The add at gpu scope publishes the warp's stores.)
            if (n_contrib > 1 &&
                atom_add_acq_rel_gpu(&counters[grp.id], 1u) == static_cast<uint32_t>(n_contrib - 1))
              *mid_last = 1;
            mbar_arrive(scr_free);
            if (a.trace != nullptr) trace()[kTrFlushes] += 1;
          }
        }
        va = vb;
        continue;
      }
      sync_consumers();
      if (a.trace != nullptr && threadIdx.x == 0) {
        trace()[kTrFlushes] += 1;
        trace()[kTrFinalMerged] = globaltimer_ns();
      }
      if (n_contrib == 1) {
        merge_and_store(threadIdx.x, W * 32);
      } else if (*fast_flag) {
        // Every other partial is published: merge them with these states.
        for (int i = threadIdx.x; i < quads; i += W * 32) {
          const int hr = i / (D / 4), d4 = i % (D / 4);
          float2 ml[kFastMerge];
          float4 ov[kFastMerge];
#pragma unroll
          for (int k = 0; k < kFastMerge; ++k) {
            const int cta = grp.c_lo + k;
            ml[k] = make_float2(-INFINITY, 0.f);
            ov[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k < n_contrib && cta != static_cast<int>(blockIdx.x)) {
              const int64_t at = slot_of(cta, grp.id) + hr;
              ml[k] = __ldcg(&a.part_ml[at]);
              ov[k] = __ldcg(reinterpret_cast<const float4*>(&a.part_o[at * D + 4 * d4]));
            }
          }
          float M, lsum;
          float4 acc;
          merge_warps(hr, d4, M, lsum, acc);
          float top = M;
#pragma unroll
          for (int k = 0; k < kFastMerge; ++k) {
            if (grp.c_lo + k == static_cast<int>(blockIdx.x)) {
              ml[k] = make_float2(M, lsum);
              ov[k] = acc;
            }
            top = fmaxf(top, ml[k].x);
          }
          // In merge_partials' order, so that the result's bits do not depend
          // on which of the two came to merge.
          const float ref = exp_ref(top);
          lsum = 0.f;
          acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < kFastMerge; ++k) {
            const float w = fast_exp2(ml[k].x - ref);
            lsum = fmaf(w, ml[k].y, lsum);
            acc.x = fmaf(w, ov[k].x, acc.x);
            acc.y = fmaf(w, ov[k].y, acc.y);
            acc.z = fmaf(w, ov[k].z, acc.z);
            acc.w = fmaf(w, ov[k].w, acc.w);
          }
          write_out(grp, hr, d4, lsum, acc);
        }
        // All have arrived: the counter goes back to zero for the next launch.
        if (threadIdx.x == 0) counters[grp.id] = 0u;
      } else {
        // Publish a partial and take a ticket; the last to do so merges.  (The
        // barrier makes every thread's partial visible to thread 0; its
        // acquire-release add publishes them and, for the last arriver, makes
        // the others' visible.)
        merge_and_store(threadIdx.x, W * 32);
        sync_consumers();
        if (threadIdx.x == 0)
          *last_flag = atom_add_acq_rel_gpu(&counters[grp.id], 1u) ==
                       static_cast<uint32_t>(n_contrib - 1);
        sync_consumers();
        if (*last_flag) merge_partials(grp);
      }
      if (a.trace != nullptr && threadIdx.x == 0 && final_group) {
        trace()[kTrFinalDone] = globaltimer_ns();
        trace()[kTrFinalKind] = n_contrib == 1 ? 0 : (*fast_flag ? 2 : 1);
      }
      va = vb;
    }
    // The range's first group, where it ended before the range did and this
    // CTA turned out to be the last of its contributors.  (Its merge, before
    // the final group's, set the flag.)
    if (v_second < v_end) {
      sync_consumers();
      if (*mid_last) merge_partials(group_at(v_begin));
    }
  }
  __syncthreads();
  if (a.trace != nullptr && threadIdx.x == 0) {
    trace()[kTrExit] = globaltimer_ns();
    trace()[kTrSm] = static_cast<uint64_t>(sm_id()) | (static_cast<uint64_t>(blockIdx.x) << 32);
    trace()[kTrUnits] = static_cast<uint64_t>(v_end - v_begin);
  }
}

template <int NG, bool MQ, bool F16>
int launch_t(const DecodeShape& s, const DecodeArgs& a, const uint32_t* mask_bits,
             const CUtensorMap& tmk, const CUtensorMap& tmv, cudaStream_t stream) {
  auto kern = gqa_decode_q4_kernel<NG, MQ, F16>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, s.smem_bytes) !=
      cudaSuccess) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(s.grid));
  cfg.blockDim = dim3(kQ4Threads);
  cfg.dynamicSmemBytes = static_cast<size_t>(s.smem_bytes);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, tmk, tmv, a, s.tiles_per_group, s.passes,
                         static_cast<int>(s.units), s.stages, s.split, s.lead, mask_bits, a.counters) != cudaSuccess) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  return GQA_OK;
}

template <int NG>
int launch_ng(const DecodeShape& s, const DecodeArgs& a, const uint32_t* mask_bits,
              const CUtensorMap& tmk, const CUtensorMap& tmv, cudaStream_t stream, bool f16) {
  if (a.Sq > 1)
    return f16 ? launch_t<NG, true, true>(s, a, mask_bits, tmk, tmv, stream)
               : launch_t<NG, true, false>(s, a, mask_bits, tmk, tmv, stream);
  return f16 ? launch_t<NG, false, true>(s, a, mask_bits, tmk, tmv, stream)
             : launch_t<NG, false, false>(s, a, mask_bits, tmk, tmv, stream);
}

template <int NG>
void fit(DecodeShape& s, int ragged_batch) {
  for (s.stages = 10;; --s.stages) {
    s.smem_bytes = Q4Layout<NG>::bytes(s.stages, ragged_batch);
    if (s.smem_bytes <= kDecodeMaxSmem || s.stages <= 2) break;
  }
}

}  // namespace

DecodeShape plan_decode_q4(const gqa_problem& p, int sm_count) {
  DecodeShape s{};
  const int64_t rows = p.heads_q / p.heads_kv * p.seq_q;
  s.D = p.head_dim <= 64 ? 64 : 128;
  // One column tile per pass: two would serve 16 rows with one unpacking, but
  // leave registers for one 16-key MMA tile at a time only (1790 ns per unit
  // against twice 640; the passes' records come out of L2 the second time).
  s.NT = 1;
  s.HP = 8;
  s.passes = static_cast<int>((rows + s.HP - 1) / s.HP);
  s.ragged = p.kv_lens != nullptr;
  s.tiles_per_group =
      s.ragged ? static_cast<int>((p.seq_k + KT - 1) / KT)
               : decode_key_range(p.seq_k, p.seq_k, p.seq_q, p.causal, p.causal_offset, p.window)
                     .tiles;
  if (s.tiles_per_group < 1) s.tiles_per_group = 1;
  s.groups = p.batch * p.heads_kv * s.passes;
  // One range per CTA, all equal, or (all groups alike) every group cut into
  // as many as the SMs allow, which saves the changes of groups inside ranges
  // and, at one range per group, the merge of partials: whichever is shorter
  // by its longest range.
  const int64_t real = s.groups * s.tiles_per_group;
  s.lead = kQ4Lead;
  s.units = real + s.groups * s.lead;
  s.grid = static_cast<int>(real < sm_count ? real : sm_count);
  if (!s.ragged && s.groups > 0 && s.groups <= sm_count) {
    int64_t split = sm_count / s.groups;
    if (split > s.tiles_per_group) split = s.tiles_per_group;
    const double apart = double((s.tiles_per_group + split - 1) / split) * q4_unit_ns(s.D) +
                         (split > 1 ? kQ4MergeNs : 0.0);
    const double even = double((s.units + sm_count - 1) / sm_count) * q4_unit_ns(s.D) + kQ4MergeNs;
    if (apart <= even) {
      s.split = static_cast<int>(split);
      s.lead = 0;
      s.units = real;
      s.grid = static_cast<int>(s.groups * split);
    }
  }
  if (s.grid < 1) s.grid = 1;
  const int rb = s.ragged ? static_cast<int>(p.batch) : 0;
  if (s.D == 128)
    fit<4>(s, rb);
  else
    fit<2>(s, rb);
  const int64_t slots = static_cast<int64_t>(s.grid) * 2 * s.HP;
  int64_t at = kScratchOffset;
  s.zero_counters = s.groups * 4 > kCounterRegionBytes;
  s.counters_offset = kWorkspaceHeadBytes;
  if (s.zero_counters) {
    s.counters_offset = at;
    at += ((s.groups * 4 + 255) / 256) * 256;
  }
  s.part_ml_offset = at;
  s.part_o_offset = s.part_ml_offset + ((slots * 8 + 255) / 256) * 256;
  s.mask_offset = s.part_o_offset + slots * s.D * 4;  // (a multiple of 256)
  s.workspace_end =
      s.mask_offset + (p.has_mask ? p.batch * p.seq_q * mask_words(p.seq_k) * 4 : 0);
  return s;
}

int launch_decode_q4(const gqa_problem& p, const DecodeShape& s, const DecodeArgs& a, uint8_t* ws,
                     const CUtensorMap& tmk, const CUtensorMap& tmv, cudaStream_t stream) {
  uint32_t* bits = nullptr;
  if (a.has_mask) {
    bits = reinterpret_cast<uint32_t*>(ws + s.mask_offset);
    const int64_t rows = p.batch * p.seq_q;
    const int64_t spans = (p.seq_k + kMaskSpan - 1) / kMaskSpan;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((spans + 7) / 8),
                       static_cast<unsigned>(rows < 65535 ? rows : 65535));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, gqa_q4_mask_bits_kernel, a, bits) != cudaSuccess) {
      cudaGetLastError();
      return GQA_ERR_CUDA;
    }
  }
  const bool f16 = p.dtype == GQA_DTYPE_F16;
  return s.D == 128 ? launch_ng<4>(s, a, bits, tmk, tmv, stream, f16)
                    : launch_ng<2>(s, a, bits, tmk, tmv, stream, f16);
}

}  // namespace gqa
