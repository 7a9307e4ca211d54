// C-ABI layer of the 4-bit cache: validation, planning and dispatch of
// append, read back and attention.  Nothing throws across the ABI.
#include <cuda_runtime.h>

#include <cstring>

#include "enqueue_turn.h"
#include "gqa.h"
#include "kernels.h"
#include "q4.cuh"

namespace gqa {
namespace {

constexpr int64_t kLim = int64_t(1) << 31;

// Times that the choice between the three ways of attending goes by (ns, this
// library's kernels; with those per unit and key tile in kernels.h): launch and
// ends of a decode; launches and ends of the 128-row kernel, and each partial
// of a group that its merge reads; a slice's launches and ends, a key tile of
// the two-tile prefill, and bytes per ns of the read back.
constexpr double kDecodeNs = 7000;
constexpr double kChunkNs = 16000, kChunkPartialNs = 300;
constexpr double kSliceNs = 9000, kReadBytesPerNs = 4500;
double two_tile_ns(int64_t head_dim) { return head_dim > 64 ? 2000 : 1700; }

bool aligned(const void* ptr, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0;
}

bool head_dim_ok(int64_t D) { return D >= 8 && D <= 128 && D % 8 == 0; }

// Byte strides of a cache of records: unit inside the record, whole 16-byte
// pieces over every dimension that is stepped (vector loads and TMA).
bool cache_strides_ok(const int64_t st[4], const int64_t sizes[3]) {
  if (st[3] != 1) return false;
  for (int d = 0; d < 3; ++d)
    if (st[d] < 0 || (sizes[d] > 1 && st[d] % 16 != 0)) return false;
  return true;
}

int validate_q4(const gqa_problem* pp) {
  if (pp == nullptr) return GQA_ERR_NULL;
  gqa_problem p = *pp;
  if (p.dtype == GQA_DTYPE_F32) return GQA_ERR_UNSUPPORTED;
  // Everything but the caches is checked as for a 16-bit problem of the same sizes.
  for (int d = 0; d < 4; ++d) p.k_stride[d] = p.v_stride[d] = d == 3 ? 1 : 8;
  const int rc = validate_problem(&p);
  if (rc != GQA_OK) return rc;
  const int64_t sizes[3] = {p.block_table ? p.num_pages : p.batch, p.heads_kv,
                            p.block_table ? p.page_size : p.seq_k};
  if (!cache_strides_ok(pp->k_stride, sizes) || !cache_strides_ok(pp->v_stride, sizes))
    return GQA_ERR_LAYOUT;
  return GQA_OK;
}

// The way over 16-bit scratch for long query blocks: entries (whole, or some
// of one's kv heads) in slices whose keys and values are read back, then
// attended to by the prefill kernels.
struct SlicePlan {
  int64_t nb, nh;            // entries and kv heads per slice (nb > 1 only with every head)
  int64_t head_bytes;        // scratch of one kv head's K (or V)
  int64_t k_offset, v_offset, workspace_end;
  int64_t slices, work;      // and the prefill's work items of all of them
  int launches;
  double ns;                 // estimated time
};

// The problem of a slice: nb entries from b0, nh kv heads from h0, contiguous
// 16-bit K and V.
gqa_problem slice_problem(const gqa_problem& p, int64_t b0, int64_t nb, int64_t nh) {
  gqa_problem c = p;
  const int64_t D = p.head_dim, S = p.seq_k;
  c.batch = nb;
  c.heads_kv = nh;
  c.heads_q = nh * (p.heads_q / p.heads_kv);
  const int64_t st[4] = {nh * S * D, S * D, D, 1};
  for (int i = 0; i < 4; ++i) c.k_stride[i] = c.v_stride[i] = st[i];
  if (p.kv_lens != nullptr) c.kv_lens = p.kv_lens + b0;
  c.block_table = nullptr;
  c.block_table_stride = c.page_size = c.num_pages = 0;
  return c;
}

constexpr int64_t kSliceL2 = int64_t(64) << 20;     // scratch that stays in L2 beside the rest
constexpr int64_t kSliceMost = int64_t(1) << 30;    // scratch of a slice, unless one head needs more

// The most keys of an entry that its queries can see.
int64_t keys_read(const gqa_problem& p) {
  const int64_t w = p.window > 0 ? p.seq_q + p.window : p.seq_k;
  return w < p.seq_k ? w : p.seq_k;
}

SlicePlan plan_slices(const gqa_problem& p, int sms) {
  SlicePlan s{};
  const int64_t g = p.heads_q / p.heads_kv;
  s.head_bytes = (p.seq_k * p.head_dim * 2 + 255) / 256 * 256;
  const int64_t qpt = 128 / g;
  const int64_t items = ((p.seq_q + qpt - 1) / qpt + 1) / 2;  // two-tile work items per kv head
  // Enough heads for two rounds of items over the SMs, or more while the
  // scratch stays in L2.
  int64_t heads = (2 * sms + items - 1) / items;
  const int64_t fit = kSliceL2 / (2 * s.head_bytes);
  if (heads < fit) heads = fit;
  const int64_t most = kSliceMost / (2 * s.head_bytes);
  if (heads > most) heads = most;
  if (heads < 1) heads = 1;
  if (heads >= p.heads_kv) {
    s.nh = p.heads_kv;
    s.nb = heads / p.heads_kv < p.batch ? heads / p.heads_kv : p.batch;
  } else {
    s.nb = 1;
    s.nh = heads;
  }
  // Slices of up to four sizes (the last of the entries and of the heads may be
  // narrower), each with a prefill plan of its own: a narrower one may need more
  // scratch (the item order that a full one is too large to sort).  K and V
  // start past all of them.
  const int64_t nbs[2] = {p.batch / s.nb, p.batch % s.nb > 0 ? 1 : 0};
  const int64_t nhs[2] = {p.heads_kv / s.nh, p.heads_kv % s.nh > 0 ? 1 : 0};
  s.slices = (nbs[0] + nbs[1]) * (nhs[0] + nhs[1]);
  for (int i = 0; i < 4; ++i) {
    const int64_t count = nbs[i & 1] * nhs[i >> 1];
    if (count == 0) continue;
    const PrefillShape f =
        plan_prefill(slice_problem(p, 0, (i & 1) != 0 ? p.batch % s.nb : s.nb,
                                   (i >> 1) != 0 ? p.heads_kv % s.nh : s.nh),
                     sms);
    if (f.workspace_end > s.k_offset) s.k_offset = f.workspace_end;
    s.launches += static_cast<int>(count) *
                  (2 + (p.has_mask ? 1 : 0) + (f.order_offset >= 0 ? 1 : 0));
    s.work += count * f.work;
  }
  s.k_offset = (s.k_offset + 255) / 256 * 256;
  s.v_offset = s.k_offset + s.nb * s.nh * s.head_bytes;
  s.workspace_end = s.v_offset + s.nb * s.nh * s.head_bytes;
  const double rounds = double((s.nb * s.nh * items + sms - 1) / sms);
  const int64_t keys = keys_read(p);
  const double bytes = 2.0 * double(p.batch * p.heads_kv) *
                       double(keys * (q4::record_bytes(static_cast<int>(p.head_dim)) +
                                         2 * p.head_dim));
  const double tiles = rounds * double((keys + 127) / 128);
  s.ns = double(s.slices) * (kSliceNs + tiles * two_tile_ns(p.head_dim)) +
         bytes / kReadBytesPerNs;
  return s;
}

// Estimated times of the other two ways over the same problem.
double decode_ns(const gqa_problem& p, const DecodeShape& s, int sms) {
  const double tiles = double((keys_read(p) + 127) / 128);
  const double places = s.split > 0 ? tiles / s.split : double(s.groups) * (tiles + s.lead) / sms;
  return kDecodeNs + places * q4_unit_ns(s.D) + (s.split == 1 ? 0.0 : kQ4MergeNs);
}

double chunk_ns(const gqa_problem& p, const ChunkShape& s, int sms) {
  const double tiles = double((keys_read(p) + 127) / 128), share = double(sms) / double(s.groups);
  return kChunkNs + double(s.groups) * (tiles + kChunkLead) / sms * chunk_tile_ns(s.D, s.nq) +
         kChunkPartialNs * (share < tiles ? share : tiles);
}

// The way to attend: a pass over the records per 8 rows of a kv head (one pass
// where it has no more), 128-row tiles that unpack each record once, or the
// two-tile prefill over 16-bit scratch: the least of the estimated times.  Over
// 468 problems (1024 to 16384 keys, 2 to 128 kv heads, 4 and 8 query heads
// each, 3 to 1024 queries, head dims 64 and 128), each timed with every way, it
// takes 0.5% longer than the fastest in the mean (10 of them 10% or more).
//
// A bf16 slice, in which keys, values and weights are rounded to bf16, has to
// save an eighth against the tiles, which keep fp16's bits of them.
//
// With per-sequence lengths a slice takes as long as its longest sequence, the
// other two as all of them together: counted as three quarters of the most.
//
// A single token always takes the first, however many query heads share a kv
// head.  At 32 of them that takes 2.7 us per 128 keys of a kv head and SM
// against 2.1 us in 128-row tiles, at 64 5.2 us.  The last two ways are
// planned, and their plans filled in, only where there is a choice: the tiles
// of a token of more than 128 query heads per kv head would hold no query
// position.
int pick_way(const gqa_problem& p, const DecodeShape& d, int sms, ChunkShape* c, SlicePlan* s) {
  if (d.passes <= 1 || p.seq_q <= 1) return GQA_KERNEL_Q4;
  *c = plan_chunk_q4(p, sms);
  *s = plan_slices(p, sms);
  const double held = p.kv_lens != nullptr ? 0.75 : 1.0;
  double best = held * decode_ns(p, d, sms);
  int way = GQA_KERNEL_Q4;
  if (c->fits && held * chunk_ns(p, *c, sms) < best) {
    best = held * chunk_ns(p, *c, sms);
    way = GQA_KERNEL_Q4_CHUNK;
  }
  const double bits = way == GQA_KERNEL_Q4_CHUNK && p.dtype == GQA_DTYPE_BF16 ? 1.15 : 1.0;
  return bits * s->ns < best ? GQA_KERNEL_Q4_PREFILL : way;
}

int fill_plan_q4(const gqa_problem& p, int sm_count, gqa_plan* plan) {
  std::memset(plan, 0, sizeof(*plan));
  const int64_t qo = p.batch * p.heads_q * p.seq_q * p.head_dim * 2;
  const int64_t kv = p.batch * p.heads_kv * p.seq_k * q4::record_bytes(static_cast<int>(p.head_dim));
  plan->algorithmic_bytes = 2 * qo + 2 * kv + (p.has_mask ? p.batch * p.seq_q * p.seq_k : 0);
  plan->algorithmic_flops = 4.0 * double(p.batch) * double(p.heads_q) * double(p.seq_q) *
                            double(p.seq_k) * double(p.head_dim) * (p.causal ? 0.5 : 1.0);
  plan->workspace_bytes = kWorkspaceHeadBytes;
  if (p.batch == 0 || p.seq_q == 0) {
    plan->kernel = GQA_KERNEL_NONE;
    return GQA_OK;
  }
  if (p.seq_k == 0 || nothing_visible(p)) {
    plan->kernel = p.seq_k == 0 ? GQA_KERNEL_ZERO : GQA_KERNEL_NAN;
    plan->grid = 592;
    plan->block = 256;
    plan->launches = 1;
    return GQA_OK;
  }
  const DecodeShape s = plan_decode_q4(p, sm_count);
  ChunkShape c{};
  SlicePlan sl{};
  plan->kernel = pick_way(p, s, sm_count, &c, &sl);
  if (plan->kernel == GQA_KERNEL_Q4_CHUNK) {
    plan->grid = c.grid;
    plan->block = kChunkThreads;
    plan->smem_bytes = c.smem_bytes;
    plan->launches = 2;
    plan->work_units = static_cast<int32_t>(c.groups * c.tiles);
    plan->workspace_bytes = (c.workspace_end + 255) / 256 * 256;
    return GQA_OK;
  }
  if (plan->kernel == GQA_KERNEL_Q4_PREFILL) {
    const PrefillShape f = plan_prefill(slice_problem(p, 0, sl.nb, sl.nh), sm_count);
    plan->grid = f.grid;
    plan->block = kPrefillThreads;
    plan->smem_bytes = f.smem_bytes;
    plan->launches = sl.launches;
    plan->work_units = static_cast<int32_t>(sl.work);
    plan->workspace_bytes = (sl.workspace_end + 255) / 256 * 256;
    return GQA_OK;
  }
  if (s.units >= kLim) return GQA_ERR_UNSUPPORTED;  // 32-bit unit indices
  plan->grid = s.grid;
  plan->block = kQ4Threads;
  plan->smem_bytes = s.smem_bytes;
  plan->launches = 1 + (s.zero_counters ? 1 : 0) + (p.has_mask ? 1 : 0);
  plan->work_units = static_cast<int32_t>(s.groups * s.tiles_per_group);
  plan->workspace_bytes = (s.workspace_end + 255) / 256 * 256;
  return GQA_OK;
}

int run_slices(const gqa_problem& p, const SlicePlan& s, int sms, const void* q,
               const uint8_t* ck, const uint8_t* cv, const uint8_t* mask, void* out, uint8_t* ws,
               cudaStream_t stream) {
  const bool f16 = p.dtype == GQA_DTYPE_F16;
  const int64_t g = p.heads_q / p.heads_kv;
  const bool paged = p.block_table != nullptr;
  for (int64_t b0 = 0; b0 < p.batch; b0 += s.nb) {
    for (int64_t h0 = 0; h0 < p.heads_kv; h0 += s.nh) {
      const int64_t nb = p.batch - b0 < s.nb ? p.batch - b0 : s.nb;
      const int64_t nh = p.heads_kv - h0 < s.nh ? p.heads_kv - h0 : s.nh;
      const gqa_problem c = slice_problem(p, b0, nb, nh);
      Q4RowsArgs a{};
      const uint8_t* caches[2] = {ck, cv};
      const int64_t* strides[2] = {p.k_stride, p.v_stride};
      const int64_t offsets[2] = {s.k_offset, s.v_offset};
      for (int i = 0; i < 2; ++i) {
        a.cache[i] = const_cast<uint8_t*>(caches[i]) + h0 * strides[i][1] +
                     (paged ? 0 : b0 * strides[i][0]);
        a.rows[i] = reinterpret_cast<uint16_t*>(ws + offsets[i]);
        for (int d = 0; d < 3; ++d) {
          a.cs[i][d] = strides[i][d];
          a.rs[i][d] = c.k_stride[d];
        }
      }
      a.lens = const_cast<int32_t*>(c.kv_lens);
      a.err = reinterpret_cast<uint32_t*>(ws);
      a.B = static_cast<int>(nb);
      a.H = static_cast<int>(nh);
      a.D = static_cast<int>(p.head_dim);
      a.n = static_cast<int>(p.seq_k);
      a.cap = p.seq_k;
      if (paged) {
        a.bt = p.block_table + b0 * p.block_table_stride;
        a.bt_stride = p.block_table_stride;
        a.page_size = p.page_size;
        a.num_pages = p.num_pages;
      }
      a.vec = true;
      // The prefill uses nothing past a length, nor key tiles below the window
      // of the first query or past the diagonal of the last.
      a.leave_tail = true;
      a.from = p.window > 0 ? p.causal_offset - p.seq_k - p.window + 1 : -kLim;
      a.to = p.causal ? p.causal_offset - p.seq_k + p.seq_q : 0;
      int rc = launch_q4_read(a, f16, stream);
      if (rc != GQA_OK) return rc;
      rc = launch_prefill_call(
          c, sms, static_cast<const uint16_t*>(q) + b0 * p.q_stride[0] + h0 * g * p.q_stride[1],
          ws + s.k_offset, ws + s.v_offset, mask != nullptr ? mask + b0 * p.mask_stride[0] : nullptr,
          static_cast<uint16_t*>(out) + b0 * p.o_stride[0] + h0 * g * p.o_stride[1], ws, stream);
      if (rc != GQA_OK) return rc;
    }
  }
  return GQA_OK;
}

// Tensor map over (byte, row, kv head, entry or page) of a cache of records:
// boxes of `rows` records, padded with zeros to the kernel's record size.
int encode_records(CUtensorMap* map, const void* base, const gqa_problem& p, const int64_t st[4],
                   int padded_dim) {
  auto enc = get_encoder();
  if (enc == nullptr) return GQA_ERR_CUDA;
  const bool paged = p.block_table != nullptr;
  const int64_t bytes = q4::record_bytes(static_cast<int>(p.head_dim));
  const int64_t S = paged ? p.page_size : p.seq_k, H = p.heads_kv;
  const int64_t B = paged ? p.num_pages : p.batch;
  // Strides of length-1 dimensions are never stepped; give them a legal value.
  const int64_t sb = S > 1 ? st[2] : bytes;
  const int64_t hb = H > 1 ? st[1] : sb * S;
  const int64_t bb = B > 1 ? st[0] : hb * H;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(bytes), static_cast<cuuint64_t>(S),
                              static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(sb), static_cast<cuuint64_t>(hb),
                                 static_cast<cuuint64_t>(bb)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(q4::record_bytes(padded_dim)),
                             static_cast<cuuint32_t>(paged ? kDecodePageBox : kDecodeKeysPerTile),
                             1, 1};
  const cuuint32_t unit[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box,
             unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? GQA_OK
             : GQA_ERR_LAYOUT;
}

// Checks shared by append and read back, and the arguments of both kernels.
int make_rows_args(const gqa_kv_q4_desc* d, void* cache_k, void* cache_v, void* k, void* v,
                   const int32_t* lens, void* workspace, size_t workspace_bytes, bool append,
                   Q4RowsArgs* out) {
  if (d == nullptr) return GQA_ERR_NULL;
  if (d->dtype == GQA_DTYPE_F32) return GQA_ERR_UNSUPPORTED;
  if (d->dtype != GQA_DTYPE_BF16 && d->dtype != GQA_DTYPE_F16) return GQA_ERR_ARG;
  if (d->batch < 0 || d->heads_kv <= 0 || d->capacity < 0 || d->head_dim <= 0 || d->n < 0 ||
      d->batch >= kLim || d->heads_kv >= kLim || d->capacity >= kLim || d->n >= kLim)
    return GQA_ERR_SHAPE;
  if (!head_dim_ok(d->head_dim)) return GQA_ERR_UNSUPPORTED;
  if (append ? (d->start != 0 || d->starts != nullptr) : (d->advance != 0 || d->counts != nullptr))
    return GQA_ERR_ARG;
  if (append && d->counts == nullptr && d->n > d->capacity) return GQA_ERR_SHAPE;
  if (!append && (d->start < 0 || d->start >= kLim)) return GQA_ERR_ARG;
  if (d->block_table != nullptr &&
      (d->page_size < 1 || d->block_table_stride < 1 || d->num_pages < 1 ||
       d->page_size >= kLim || d->block_table_stride >= kLim || d->num_pages >= kLim ||
       d->capacity > d->block_table_stride * d->page_size))
    return GQA_ERR_SHAPE;
  const int64_t csz[3] = {d->block_table ? d->num_pages : d->batch, d->heads_kv,
                          d->block_table ? d->page_size : d->capacity};
  if (!cache_strides_ok(d->cache_k_stride, csz) || !cache_strides_ok(d->cache_v_stride, csz))
    return GQA_ERR_LAYOUT;
  const int64_t* rst[2] = {d->k_stride, d->v_stride};
  for (const int64_t* s : rst)
    if (s[3] != 1 || s[0] < 0 || s[1] < 0 || s[2] < 0) return GQA_ERR_LAYOUT;
  Q4RowsArgs& a = *out;
  a = Q4RowsArgs{};
  a.B = static_cast<int>(d->batch);
  a.n = static_cast<int>(d->n);
  if (d->batch == 0 || d->n == 0) return GQA_OK;
  if (d->batch * d->heads_kv >= kLim) return GQA_ERR_UNSUPPORTED;  // 32-bit head indices
  if (cache_k == nullptr || cache_v == nullptr || k == nullptr || v == nullptr ||
      (append && lens == nullptr))
    return GQA_ERR_NULL;
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < 256)
    return GQA_ERR_WORKSPACE;
  if (!aligned(cache_k, 16) || !aligned(cache_v, 16) || !aligned(k, 2) || !aligned(v, 2) ||
      !aligned(lens, 4))
    return GQA_ERR_LAYOUT;
  a.cache[0] = static_cast<uint8_t*>(cache_k);
  a.cache[1] = static_cast<uint8_t*>(cache_v);
  a.rows[0] = static_cast<uint16_t*>(k);
  a.rows[1] = static_cast<uint16_t*>(v);
  a.vec = aligned(k, 16) && aligned(v, 16);
  const int64_t rsz[3] = {d->batch, d->heads_kv, d->n};
  for (int i = 0; i < 3; ++i) {
    a.cs[0][i] = d->cache_k_stride[i];
    a.cs[1][i] = d->cache_v_stride[i];
    a.rs[0][i] = d->k_stride[i];
    a.rs[1][i] = d->v_stride[i];
    if (rsz[i] > 1 && (d->k_stride[i] % 8 != 0 || d->v_stride[i] % 8 != 0)) a.vec = false;
  }
  a.lens = const_cast<int32_t*>(lens);  // written by an advancing append only
  a.counts = d->counts;
  a.starts = d->starts;
  a.start = d->start;
  a.err = static_cast<uint32_t*>(workspace);
  a.ticket = static_cast<uint32_t*>(workspace) + 1;
  a.H = static_cast<int>(d->heads_kv);
  a.D = static_cast<int>(d->head_dim);
  a.advance = d->advance != 0;
  a.cap = d->capacity;
  a.bt = d->block_table;
  a.bt_stride = d->block_table_stride;
  a.page_size = d->page_size;
  a.num_pages = d->num_pages;
  return GQA_OK;
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

GQA_API int64_t gqa_q4_record_bytes(int64_t head_dim) {
  return head_dim_ok(head_dim) ? q4::record_bytes(static_cast<int>(head_dim)) : 0;
}

GQA_API int gqa_kv_append_q4(const gqa_kv_q4_desc* d, void* cache_k, void* cache_v,
                             const void* k_new, const void* v_new, int32_t* kv_lens,
                             void* workspace, size_t workspace_bytes, void* stream) {
  Q4RowsArgs a;
  const int rc = make_rows_args(d, cache_k, cache_v, const_cast<void*>(k_new),
                                const_cast<void*>(v_new), kv_lens, workspace, workspace_bytes,
                                true, &a);
  if (rc != GQA_OK || a.B == 0 || a.n == 0) return rc;
  return launch_q4_append(a, d->dtype == GQA_DTYPE_F16, static_cast<cudaStream_t>(stream));
}

GQA_API int gqa_kv_read_q4(const gqa_kv_q4_desc* d, const void* cache_k, const void* cache_v,
                           void* k, void* v, const int32_t* kv_lens, void* workspace,
                           size_t workspace_bytes, void* stream) {
  Q4RowsArgs a;
  const int rc = make_rows_args(d, const_cast<void*>(cache_k), const_cast<void*>(cache_v), k, v,
                                kv_lens, workspace, workspace_bytes, false, &a);
  if (rc != GQA_OK || a.B == 0 || a.n == 0) return rc;
  return launch_q4_read(a, d->dtype == GQA_DTYPE_F16, static_cast<cudaStream_t>(stream));
}

GQA_API int gqa_query_q4(const gqa_problem* p, int sm_count, gqa_plan* plan) {
  if (plan == nullptr) return GQA_ERR_NULL;
  const int rc = validate_q4(p);
  if (rc != GQA_OK) return rc;
  if (sm_count <= 0) {
    const int drc = device_sm_count(&sm_count);
    if (drc != GQA_OK) return drc;
  }
  return fill_plan_q4(*p, sm_count, plan);
}

GQA_API int gqa_forward_q4(const gqa_problem* pp, const void* q, const void* cache_k,
                           const void* cache_v, const uint8_t* mask, void* out, void* workspace,
                           size_t workspace_bytes, void* stream_ptr) {
  const int rc = validate_q4(pp);
  if (rc != GQA_OK) return rc;
  const gqa_problem& p = *pp;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  int sms = 0;
  const int drc = device_sm_count(&sms);
  if (drc != GQA_OK) return drc;
  gqa_plan plan;
  const int prc = fill_plan_q4(p, sms, &plan);
  if (prc != GQA_OK) return prc;
  if (plan.kernel == GQA_KERNEL_NONE) return GQA_OK;
  if (out == nullptr) return GQA_ERR_NULL;
  if (plan.kernel == GQA_KERNEL_ZERO || plan.kernel == GQA_KERNEL_NAN)
    return launch_zero(p, out, stream, plan.kernel == GQA_KERNEL_NAN);
  if (q == nullptr || cache_k == nullptr || cache_v == nullptr) return GQA_ERR_NULL;
  if (p.has_mask && mask == nullptr) return GQA_ERR_NULL;
  if (workspace == nullptr || !aligned(workspace, 256) ||
      workspace_bytes < static_cast<size_t>(plan.workspace_bytes))
    return GQA_ERR_WORKSPACE;
  if (!aligned(q, 16) || !aligned(cache_k, 16) || !aligned(cache_v, 16) || !aligned(out, 16))
    return GQA_ERR_LAYOUT;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const EnqueueTurn turn(workspace);
  if (plan.kernel == GQA_KERNEL_Q4_PREFILL)
    return run_slices(p, plan_slices(p, sms), sms, q, static_cast<const uint8_t*>(cache_k),
                      static_cast<const uint8_t*>(cache_v), p.has_mask ? mask : nullptr, out, ws,
                      stream);
  const DecodeShape s = plan_decode_q4(p, sms);
  CUtensorMap tmk, tmv;
  int erc = encode_records(&tmk, cache_k, p, p.k_stride, s.D);
  if (erc != GQA_OK) return erc;
  erc = encode_records(&tmv, cache_v, p, p.v_stride, s.D);
  if (erc != GQA_OK) return erc;
  if (plan.kernel == GQA_KERNEL_Q4_CHUNK) {
    const ChunkShape c = plan_chunk_q4(p, sms);
    CUtensorMap tmq;
    erc = encode_q_map(&tmq, q, p, c.qpt);
    if (erc != GQA_OK) return erc;
    PrefillArgs f{};
    f.out = static_cast<uint16_t*>(out);
    for (int d = 0; d < 4; ++d) f.os[d] = p.o_stride[d];
    f.err = reinterpret_cast<uint32_t*>(ws);
    f.lens = p.kv_lens;
    f.Dv = static_cast<int>(p.head_dim);
    f.B = static_cast<int>(p.batch);
    f.Hq = static_cast<int>(p.heads_q);
    f.Hkv = static_cast<int>(p.heads_kv);
    f.Sq = static_cast<int>(p.seq_q);
    f.Sk = static_cast<int>(p.seq_k);
    f.g = static_cast<int>(p.heads_q / p.heads_kv);
    f.causal = p.causal;
    f.causal_offset = p.causal_offset;
    f.window = p.window;
    f.scale_log2 = static_cast<float>(static_cast<double>(p.scale) * 1.4426950408889634073599);
    return launch_chunk_q4(p, c, f, ws, tmq, tmk, tmv, stream);
  }
  const DecodeArgs a = make_decode_args(p, s, q, mask, out, ws);
  // The ticket counters must start at zero; past their region of the
  // workspace other calls may have left bytes.
  if (s.zero_counters &&
      cudaMemsetAsync(a.counters, 0, static_cast<size_t>(s.groups) * 4, stream) != cudaSuccess) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  return launch_decode_q4(p, s, a, ws, tmk, tmv, stream);
}

}  // extern "C"
