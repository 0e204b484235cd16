// The C ABI of libmla.so (declared in include/mla.h): host-side validation,
// workspace layout and kernel launches.  No allocation, no synchronisation
// (except mla_read_device_status).
#include <string.h>

#include <atomic>

#include "mla_internal.cuh"

namespace mla {

cudaError_t launch_fp8_pack(const CacheView& cv, unsigned char* out, cudaStream_t st);  // mla_fp8.cu

namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

mla_status check_geom(const mla_geom* g) {
  if (!g) return MLA_ERR_ARG;
  if (g->d_lat != kDLat || g->d_rope != kDRope || g->d_nope != kDNope || g->d_v != kDV || g->block_size != kPage)
    return MLA_ERR_SHAPE;
  if (g->H < 1 || g->H > kRowsPerBlock || (kRowsPerBlock % g->H) != 0) return MLA_ERR_SHAPE;
  if (!(g->softmax_scale > 0.f)) return MLA_ERR_ARG;
  return MLA_OK;
}

mla_status check_batch(const mla_batch* b) {
  if (!b) return MLA_ERR_ARG;
  if (b->B < 0 || b->T < 1 || b->max_pages < 1 || b->num_slots < 0 || b->num_splits_override < 0)
    return MLA_ERR_ARG;
  if ((long long)b->T * kRowsPerBlock > (1LL << 24)) return MLA_ERR_SHAPE;
  return MLA_OK;
}

mla_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

// The calls of a speculative step refuse device memory of another device than the current
// one, on which they would launch (one array of the call is looked at, ~0.2 us).
mla_status check_device(const void* p) {
  cudaPointerAttributes at;
  int dev = 0;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess || cudaGetDevice(&dev) != cudaSuccess) return MLA_ERR_CUDA;
  return at.type == cudaMemoryTypeDevice && at.device != dev ? MLA_ERR_ARG : MLA_OK;
}

}  // namespace

// Default work-range count: one per CTA pair of the decode kernel (half the SMs).
int resolve_slots(const mla_batch* b) {
  if (b->num_slots > 0) return b->num_slots;
  return decode_sm103_pairs_per_device();
}

bool compute_layout(const mla_geom* g, const mla_batch* b, WsLayout* L) {
  const long long RB = ((long long)b->T * g->H + kRowsPerBlock - 1) / kRowsPerBlock;
  const long long groups = (long long)b->B * RB;
  const int G = resolve_slots(b);
  long long cap_ranges, cap_segments, cap_partials;
  if (b->num_splits_override > 0) {
    const long long k = b->num_splits_override < b->max_pages ? b->num_splits_override : b->max_pages;
    cap_ranges = cap_segments = cap_partials = groups * k;
  } else {
    cap_ranges = G;
    cap_segments = groups + G;
    cap_partials = 2LL * G;
  }
  if (groups > (1 << 26) || cap_segments > (1 << 26)) return false;
  size_t off = align_up(MLA_HDR_WORDS * sizeof(int));
  L->off_groups = off;     off = align_up(off + (size_t)groups * kGroupWords * sizeof(int));
  L->off_segments = off;   off = align_up(off + (size_t)cap_segments * kSegWords * sizeof(int));
  L->off_range_ptr = off;  off = align_up(off + (size_t)(cap_ranges + 1) * sizeof(int));
  L->off_merge = off;      off = align_up(off + (size_t)groups * kMergeWords * sizeof(int));
  L->off_merge_sync = off; off = align_up(off + (size_t)groups * 2 * sizeof(int));
  L->off_part_lse = off;   off = align_up(off + (size_t)cap_partials * kRowsPerBlock * sizeof(float));
  L->off_part_o = off;     off = align_up(off + (size_t)cap_partials * kRowsPerBlock * kDLat * sizeof(float));
  L->total = off;
  L->cap_groups = (int)groups;
  L->cap_segments = (int)cap_segments;
  L->cap_ranges = (int)cap_ranges;
  L->cap_partials = (int)cap_partials;
  L->num_slots = G;
  return true;
}

}  // namespace mla

using namespace mla;

extern "C" {

int mla_device_sm_count(void) {
  // Filled on first use per device; concurrent first calls store the same value.
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = cached[dev].load(std::memory_order_acquire);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cached[dev].store(n, std::memory_order_release);
  }
  return n;
}

const char* mla_status_string(mla_status s) {
  switch (s) {
    case MLA_OK: return "ok";
    case MLA_ERR_ARG: return "invalid argument";
    case MLA_ERR_SHAPE: return "unsupported geometry or shape";
    case MLA_ERR_ALIGN: return "pointer or stride not 16-byte aligned";
    case MLA_ERR_WORKSPACE: return "workspace too small";
    case MLA_ERR_PLAN_STALE: return "plan built for other lengths or geometry";
    case MLA_ERR_CUDA: return "CUDA error";
    case MLA_ERR_DEVICE_CHECK: return "device check failed (block id, length or T)";
    case MLA_ERR_TIMEOUT: return "bounded wait ran out";
  }
  return "unknown status";
}

size_t mla_workspace_size(const mla_geom* geom, const mla_batch* batch) {
  if (check_geom(geom) != MLA_OK || check_batch(batch) != MLA_OK) return 0;
  WsLayout L;
  if (!compute_layout(geom, batch, &L)) return 0;
  return L.total;
}

mla_status mla_plan(const mla_geom* geom, const mla_batch* batch, const int32_t* seq_lens, void* workspace,
                    size_t ws_bytes, mla_stream_t stream) {
  mla_status s = check_geom(geom);
  if (s != MLA_OK) return s;
  if ((s = check_batch(batch)) != MLA_OK) return s;
  if (!workspace || (batch->B > 0 && !seq_lens)) return MLA_ERR_ARG;
  if (!aligned32(workspace) || !aligned16(seq_lens)) return MLA_ERR_ALIGN;
  WsLayout L;
  if (!compute_layout(geom, batch, &L)) return MLA_ERR_SHAPE;
  if (ws_bytes < L.total) return MLA_ERR_WORKSPACE;
  return cuda_status(launch_plan(seq_lens, geom, batch, L, workspace, (cudaStream_t)stream));
}

mla_status mla_absorb_q(const mla_geom* geom, const void* q_nope, const void* w_uk, void* q_lat, int BT,
                        mla_stream_t stream) {
  mla_status s = check_geom(geom);
  if (s != MLA_OK) return s;
  if (BT < 0) return MLA_ERR_ARG;
  if (BT == 0) return MLA_OK;
  if (!q_nope || !w_uk || !q_lat) return MLA_ERR_ARG;
  if (!aligned16(q_nope) || !aligned16(w_uk) || !aligned32(q_lat)) return MLA_ERR_ALIGN;
  return cuda_status(launch_absorb_sm103(static_cast<const __nv_bfloat16*>(q_nope), static_cast<const __nv_bfloat16*>(w_uk),
                                   static_cast<__nv_bfloat16*>(q_lat), BT, geom->H, (cudaStream_t)stream));
}

mla_status mla_unabsorb_o(const mla_geom* geom, const void* o_lat, const void* w_uv, void* o, int BT,
                          mla_stream_t stream) {
  mla_status s = check_geom(geom);
  if (s != MLA_OK) return s;
  if (BT < 0) return MLA_ERR_ARG;
  if (BT == 0) return MLA_OK;
  if (!o_lat || !w_uv || !o) return MLA_ERR_ARG;
  if (!aligned16(o_lat) || !aligned16(w_uv) || !aligned32(o)) return MLA_ERR_ALIGN;
  return cuda_status(launch_unabsorb_sm103(static_cast<const __nv_bfloat16*>(o_lat), static_cast<const __nv_bfloat16*>(w_uv),
                                     static_cast<__nv_bfloat16*>(o), BT, geom->H, (cudaStream_t)stream));
}

static mla_status check_cache(const mla_cache* cache, CacheView* cv);

}  // extern "C"

// Host validation of mla_decode's arguments other than the workspace.
mla_status mla::check_decode_args(const mla_geom* geom, const mla_batch* batch, const void* q_lat, const void* q_pe,
                                  const mla_cache* cache, const int32_t* block_table, int bt_stride,
                                  const int32_t* seq_lens, const void* o_lat, const float* lse, CacheView* cv) {
  mla_status s = check_geom(geom);
  if (s != MLA_OK) return s;
  if ((s = check_batch(batch)) != MLA_OK) return s;
  if (batch->B == 0) return MLA_OK;
  if (!q_lat || !q_pe || !block_table || !seq_lens || !o_lat || !lse) return MLA_ERR_ARG;
  if (bt_stride < batch->max_pages) return MLA_ERR_ARG;
  if (!aligned16(q_lat) || !aligned16(q_pe) || !aligned32(o_lat) || !aligned16(lse) || !aligned16(block_table) ||
      !aligned16(seq_lens))
    return MLA_ERR_ALIGN;
  return check_cache(cache, cv);
}

extern "C" {

static mla_status check_cache(const mla_cache* cache, CacheView* cv) {
  if (!cache || !cache->ckv || !cache->kpe || cache->num_blocks < 1) return MLA_ERR_ARG;
  if (cache->ckv_row_stride < 1 || cache->kpe_row_stride < 1 || cache->ckv_block_stride < 1 ||
      cache->kpe_block_stride < 1)
    return MLA_ERR_ARG;
  if (!aligned16(cache->ckv) || !aligned16(cache->kpe)) return MLA_ERR_ALIGN;
  if ((cache->ckv_row_stride * 2) % 16 != 0 || (cache->ckv_block_stride * 2) % 16 != 0 ||
      (cache->kpe_row_stride * 2) % 16 != 0 || (cache->kpe_block_stride * 2) % 16 != 0)
    return MLA_ERR_ALIGN;
  cv->ckv = static_cast<const __nv_bfloat16*>(cache->ckv);
  cv->kpe = static_cast<const __nv_bfloat16*>(cache->kpe);
  cv->ckv_row = cache->ckv_row_stride;
  cv->ckv_block = cache->ckv_block_stride;
  cv->kpe_row = cache->kpe_row_stride;
  cv->kpe_block = cache->kpe_block_stride;
  cv->num_blocks = cache->num_blocks;
  return MLA_OK;
}

mla_status mla_decode(const mla_geom* geom, const mla_batch* batch, const void* q_lat, const void* q_pe,
                      const mla_cache* cache, const int32_t* block_table, int bt_stride, const int32_t* seq_lens,
                      int checked, void* o_lat, float* lse, void* workspace, size_t ws_bytes, mla_stream_t stream) {
  CacheView cv;
  mla_status s = check_decode_args(geom, batch, q_lat, q_pe, cache, block_table, bt_stride, seq_lens, o_lat, lse, &cv);
  if (s != MLA_OK) return s;
  if (batch->B == 0) return MLA_OK;
  if (!workspace) return MLA_ERR_ARG;
  if (!aligned32(workspace)) return MLA_ERR_ALIGN;
  WsLayout L;
  if (!compute_layout(geom, batch, &L)) return MLA_ERR_SHAPE;
  if (ws_bytes < L.total) return MLA_ERR_WORKSPACE;
  cudaStream_t st = (cudaStream_t)stream;
  // One kernel: the split-KV decode, and (when the plan has merge records) the
  // LSE merge of each split group by the CTAs that finish its partial states last.
  return cuda_status(launch_decode_sm103(geom, batch, L, static_cast<const __nv_bfloat16*>(q_lat),
                                         static_cast<const __nv_bfloat16*>(q_pe), cv, block_table, bt_stride,
                                         seq_lens, checked, static_cast<__nv_bfloat16*>(o_lat), lse, workspace, st));
}

mla_status mla_decode_fp8(const mla_geom* geom, const mla_batch* batch, const void* q_lat, const void* q_pe,
                          const void* cache_fp8, int num_blocks, const int32_t* block_table, int bt_stride,
                          const int32_t* seq_lens, int checked, void* o_lat, float* lse, void* workspace,
                          size_t ws_bytes, mla_stream_t stream) {
  mla_status s = check_geom(geom);
  if (s != MLA_OK) return s;
  if ((s = check_batch(batch)) != MLA_OK) return s;
  if (batch->B == 0) return MLA_OK;
  if (!q_lat || !q_pe || !cache_fp8 || !block_table || !seq_lens || !o_lat || !lse || !workspace) return MLA_ERR_ARG;
  if (num_blocks < 1 || bt_stride < batch->max_pages) return MLA_ERR_ARG;
  if ((long long)num_blocks * kPage >= (1LL << 31)) return MLA_ERR_SHAPE;
  if (!aligned16(q_lat) || !aligned16(q_pe) || !aligned16(cache_fp8) || !aligned16(block_table) ||
      !aligned16(seq_lens) || !aligned32(o_lat) || !aligned16(lse) || !aligned32(workspace))
    return MLA_ERR_ALIGN;
  WsLayout L;
  if (!compute_layout(geom, batch, &L)) return MLA_ERR_SHAPE;
  if (ws_bytes < L.total) return MLA_ERR_WORKSPACE;
  CacheView cv{};
  cv.num_blocks = num_blocks;
  const Fp8Pool pool{static_cast<const unsigned char*>(cache_fp8), num_blocks};
  return cuda_status(launch_decode_sm103(geom, batch, L, static_cast<const __nv_bfloat16*>(q_lat),
                                         static_cast<const __nv_bfloat16*>(q_pe), cv, block_table, bt_stride,
                                         seq_lens, checked, static_cast<__nv_bfloat16*>(o_lat), lse, workspace,
                                         (cudaStream_t)stream, nullptr, &pool));
}

// Trees of drafted tokens: a plan of their own (the nodes' counts), then the decode.
mla_status mla_plan_tree(const mla_geom* geom, const mla_batch* batch, const int32_t* seq_lens,
                         const int32_t* node_lens, void* workspace, size_t ws_bytes, mla_stream_t stream) {
  mla_status s = check_geom(geom);
  if (s != MLA_OK) return s;
  if ((s = check_batch(batch)) != MLA_OK) return s;
  if (batch->causal) return MLA_ERR_ARG;
  if (batch->T > kMaxTreeNodes) return MLA_ERR_SHAPE;
  if (!workspace || (batch->B > 0 && !seq_lens)) return MLA_ERR_ARG;
  if (!aligned32(workspace) || !aligned16(seq_lens) || !aligned16(node_lens)) return MLA_ERR_ALIGN;
  WsLayout L;
  if (!compute_layout(geom, batch, &L)) return MLA_ERR_SHAPE;
  if (ws_bytes < L.total) return MLA_ERR_WORKSPACE;
  if (batch->B > 0 && (s = check_device(seq_lens)) != MLA_OK) return s;
  const TreeNodes tree{node_lens, nullptr};
  return cuda_status(launch_plan(seq_lens, geom, batch, L, workspace, (cudaStream_t)stream, 1, 0, &tree));
}

mla_status mla_decode_tree(const mla_geom* geom, const mla_batch* batch, const void* q_lat, const void* q_pe,
                           const mla_cache* cache, const int32_t* block_table, int bt_stride, const int32_t* seq_lens,
                           const int32_t* node_lens, const uint32_t* tree_mask, int checked, void* o_lat, float* lse,
                           void* workspace, size_t ws_bytes, mla_stream_t stream) {
  CacheView cv;
  mla_status s = check_decode_args(geom, batch, q_lat, q_pe, cache, block_table, bt_stride, seq_lens, o_lat, lse, &cv);
  if (s != MLA_OK) return s;
  if (batch->causal) return MLA_ERR_ARG;
  if (batch->T > kMaxTreeNodes) return MLA_ERR_SHAPE;
  if (batch->B == 0) return MLA_OK;
  if (!tree_mask || !workspace) return MLA_ERR_ARG;
  if (!aligned16(node_lens) || !aligned16(tree_mask) || !aligned32(workspace)) return MLA_ERR_ALIGN;
  WsLayout L;
  if (!compute_layout(geom, batch, &L)) return MLA_ERR_SHAPE;
  if (ws_bytes < L.total) return MLA_ERR_WORKSPACE;
  if ((s = check_device(q_lat)) != MLA_OK) return s;
  const TreeNodes tree{node_lens, tree_mask};
  return cuda_status(launch_decode_sm103(geom, batch, L, static_cast<const __nv_bfloat16*>(q_lat),
                                         static_cast<const __nv_bfloat16*>(q_pe), cv, block_table, bt_stride,
                                         seq_lens, checked, static_cast<__nv_bfloat16*>(o_lat), lse, workspace,
                                         (cudaStream_t)stream, nullptr, nullptr, &tree));
}

// Where an FP8 tree decode keeps converted pages: past the plan's workspace, a block
// table, then a bf16 pool of B * max_pages blocks.  False where converting ahead does
// not pay (one row group per sequence converts each page once as it is) or has no room.
static bool tree_scratch(const mla_geom* g, const mla_batch* b, size_t plan_bytes, size_t* table, size_t* pool,
                         size_t* total) {
  const long long blocks = (long long)b->B * b->max_pages;
  *total = plan_bytes;
  if ((long long)b->T * g->H <= kRowsPerBlock || b->B > 65535 || blocks * kPage >= (1LL << 31)) return false;
  *table = plan_bytes;
  *pool = align_up(*table + (size_t)blocks * sizeof(int32_t));
  *total = *pool + (size_t)blocks * kPage * kDK * sizeof(__nv_bfloat16);
  return true;
}

size_t mla_tree_fp8_workspace_size(const mla_geom* geom, const mla_batch* batch) {
  const size_t plan = mla_workspace_size(geom, batch);
  if (plan == 0 || batch->causal || batch->T > kMaxTreeNodes) return 0;
  size_t table, pool, total;
  tree_scratch(geom, batch, plan, &table, &pool, &total);
  return total;
}

mla_status mla_decode_tree_fp8(const mla_geom* geom, const mla_batch* batch, const void* q_lat, const void* q_pe,
                               const void* cache_fp8, int num_blocks, const int32_t* block_table, int bt_stride,
                               const int32_t* seq_lens, const int32_t* node_lens, const uint32_t* tree_mask,
                               int checked, void* o_lat, float* lse, void* workspace, size_t ws_bytes,
                               mla_stream_t stream) {
  mla_status s = check_geom(geom);
  if (s != MLA_OK) return s;
  if ((s = check_batch(batch)) != MLA_OK) return s;
  if (batch->causal) return MLA_ERR_ARG;
  if (batch->T > kMaxTreeNodes) return MLA_ERR_SHAPE;
  if (batch->B == 0) return MLA_OK;
  if (!q_lat || !q_pe || !cache_fp8 || !block_table || !seq_lens || !tree_mask || !o_lat || !lse || !workspace)
    return MLA_ERR_ARG;
  if (num_blocks < 1 || bt_stride < batch->max_pages) return MLA_ERR_ARG;
  if ((long long)num_blocks * kPage >= (1LL << 31)) return MLA_ERR_SHAPE;
  if (!aligned16(q_lat) || !aligned16(q_pe) || !aligned16(cache_fp8) || !aligned16(block_table) ||
      !aligned16(seq_lens) || !aligned16(node_lens) || !aligned16(tree_mask) || !aligned32(o_lat) || !aligned16(lse) ||
      !aligned32(workspace))
    return MLA_ERR_ALIGN;
  WsLayout L;
  if (!compute_layout(geom, batch, &L)) return MLA_ERR_SHAPE;
  if (ws_bytes < L.total) return MLA_ERR_WORKSPACE;
  CacheView cv{};
  cv.num_blocks = num_blocks;
  const Fp8Pool pool{static_cast<const unsigned char*>(cache_fp8), num_blocks};
  const TreeNodes tree{node_lens, tree_mask};
  if ((s = check_device(q_lat)) != MLA_OK) return s;
  size_t off_table, off_pool, total;
  if (tree_scratch(geom, batch, L.total, &off_table, &off_pool, &total) && ws_bytes >= total) {
    // each page converted once, then the decode over bf16 pages
    char* base = static_cast<char*>(workspace);
    int32_t* table = reinterpret_cast<int32_t*>(base + off_table);
    __nv_bfloat16* rows = reinterpret_cast<__nv_bfloat16*>(base + off_pool);
    if (launch_fp8_expand(pool, block_table, bt_stride, batch->B, batch->max_pages, seq_lens, checked, workspace,
                          table, rows, (cudaStream_t)stream) != cudaSuccess)
      return MLA_ERR_CUDA;
    cv.ckv = rows;
    cv.kpe = rows + kDLat;
    cv.ckv_row = cv.kpe_row = kDK;
    cv.ckv_block = cv.kpe_block = (int64_t)kPage * kDK;
    cv.num_blocks = batch->B * batch->max_pages;
    return cuda_status(launch_decode_sm103(geom, batch, L, static_cast<const __nv_bfloat16*>(q_lat),
                                           static_cast<const __nv_bfloat16*>(q_pe), cv, table, batch->max_pages,
                                           seq_lens, checked, static_cast<__nv_bfloat16*>(o_lat), lse, workspace,
                                           (cudaStream_t)stream, nullptr, nullptr, &tree));
  }
  return cuda_status(launch_decode_sm103(geom, batch, L, static_cast<const __nv_bfloat16*>(q_lat),
                                         static_cast<const __nv_bfloat16*>(q_pe), cv, block_table, bt_stride,
                                         seq_lens, checked, static_cast<__nv_bfloat16*>(o_lat), lse, workspace,
                                         (cudaStream_t)stream, nullptr, &pool, &tree));
}

// The sparse decode as a dense one over B * S_q one-token sequences of up to topk
// listed rows (non-causal), lengths topk_length[b] shared by sequence b's tokens.
static bool sparse_batch(const mla_batch* batch, int topk, mla_batch* vb) {
  if (!batch || topk < 1 || batch->B < 0 || batch->T < 1 || batch->causal) return false;
  if ((long long)batch->B * batch->T > (1LL << 26)) return false;
  *vb = *batch;
  vb->B = batch->B * batch->T;
  vb->T = 1;
  vb->causal = 0;
  vb->max_pages = (topk + kPage - 1) / kPage;
  return true;
}

size_t mla_sparse_workspace_size(const mla_geom* geom, const mla_batch* batch, int topk) {
  mla_batch vb;
  if (!sparse_batch(batch, topk, &vb)) return 0;
  return mla_workspace_size(geom, &vb);
}

mla_status mla_decode_sparse(const mla_geom* geom, const mla_batch* batch, const void* q_lat, const void* q_pe,
                             const mla_cache* cache, const int32_t* indices, int topk, const int32_t* topk_length,
                             int checked, void* o_lat, float* lse, void* workspace, size_t ws_bytes,
                             mla_stream_t stream) {
  mla_status s = check_geom(geom);
  if (s != MLA_OK) return s;
  mla_batch vb;
  if (!sparse_batch(batch, topk, &vb)) return MLA_ERR_ARG;
  if ((s = check_batch(&vb)) != MLA_OK) return s;
  if (vb.B == 0) return MLA_OK;
  if (!q_lat || !q_pe || !indices || !topk_length || !o_lat || !lse || !workspace) return MLA_ERR_ARG;
  if (!aligned16(q_lat) || !aligned16(q_pe) || !aligned16(indices) || !aligned16(topk_length) || !aligned32(o_lat) ||
      !aligned16(lse) || !aligned32(workspace))
    return MLA_ERR_ALIGN;
  CacheView cv;
  if ((s = check_cache(cache, &cv)) != MLA_OK) return s;
  // The pool's rows must be evenly spaced across blocks (one 2-D array of rows).
  if (cv.ckv_block != (int64_t)kPage * cv.ckv_row || cv.kpe_block != (int64_t)kPage * cv.kpe_row) return MLA_ERR_ARG;
  if ((long long)cv.num_blocks * kPage >= (1LL << 31)) return MLA_ERR_SHAPE;
  WsLayout L;
  if (!compute_layout(geom, &vb, &L)) return MLA_ERR_SHAPE;
  if (ws_bytes < L.total) return MLA_ERR_WORKSPACE;
  cudaStream_t st = (cudaStream_t)stream;
  if (launch_plan(topk_length, geom, &vb, L, workspace, st, batch->T, topk) != cudaSuccess) return MLA_ERR_CUDA;
  const SparseList list{indices, topk, batch->T};
  return cuda_status(launch_decode_sm103(geom, &vb, L, static_cast<const __nv_bfloat16*>(q_lat),
                                         static_cast<const __nv_bfloat16*>(q_pe), cv, nullptr, 0, topk_length,
                                         checked, static_cast<__nv_bfloat16*>(o_lat), lse, workspace, st, &list));
}

mla_status mla_split_merge(const float* part_o, const float* part_lse, const int32_t* indptr, int M, int rows, int D,
                           void* o, float* lse, mla_stream_t stream) {
  if (M < 0 || rows < 0 || D <= 0 || (D % 8) != 0) return MLA_ERR_ARG;
  if (M == 0 || rows == 0) return MLA_OK;
  if (!part_o || !part_lse || !indptr || !o || !lse) return MLA_ERR_ARG;
  if (!aligned16(part_o) || !aligned16(part_lse) || !aligned16(o) || !aligned16(lse) || !aligned16(indptr))
    return MLA_ERR_ALIGN;
  if (((size_t)rows * D * sizeof(float)) % 16 != 0) return MLA_ERR_ALIGN;
  return cuda_status(launch_split_merge(part_o, part_lse, indptr, M, rows, D, static_cast<__nv_bfloat16*>(o), lse,
                                        (cudaStream_t)stream));
}

mla_status mla_fp8_pack_cache(const mla_cache* cache, void* out, mla_stream_t stream) {
  if (!out) return MLA_ERR_ARG;
  if (!aligned16(out)) return MLA_ERR_ALIGN;
  CacheView cv;
  mla_status s = check_cache(cache, &cv);
  if (s != MLA_OK) return s;
  return cuda_status(launch_fp8_pack(cv, static_cast<unsigned char*>(out), (cudaStream_t)stream));
}

mla_status mla_debug_gather(const mla_cache* cache, const int32_t* block_table, int bt_stride, const int32_t* seq_lens,
                            int b, int path, void* out, mla_stream_t stream) {
  if (!block_table || !seq_lens || !out || b < 0 || bt_stride < 1 || (path != 0 && path != 1)) return MLA_ERR_ARG;
  if (!aligned16(out) || !aligned16(block_table) || !aligned16(seq_lens)) return MLA_ERR_ALIGN;
  CacheView cv;
  mla_status s = check_cache(cache, &cv);
  if (s != MLA_OK) return s;
  return cuda_status(launch_debug_gather(cv, block_table, bt_stride, seq_lens, b, path,
                                         static_cast<__nv_bfloat16*>(out), (cudaStream_t)stream));
}

mla_status mla_debug_set_wait_limit(long long cycles) {
  return cuda_status(set_pipeline_wait_limit(cycles));
}

int64_t mla_normal_rows_per_seq(int max_pages) { return max_pages < 1 ? 0 : normal_rows_per_seq(max_pages); }

size_t mla_normal_expanded_bytes(const mla_geom* geom, int B, int max_pages) {
  if (check_geom(geom) != MLA_OK || B < 0 || max_pages < 1) return 0;
  return (size_t)geom->H * (size_t)B * (size_t)normal_rows_per_seq(max_pages) * 256 * 2;
}

mla_status mla_normal_expand(const mla_geom* geom, const mla_cache* cache, const int32_t* block_table, int bt_stride,
                             const int32_t* seq_lens, int B, int max_pages, const void* w_uk, const void* w_uv,
                             void* kv_exp, mla_stream_t stream) {
  mla_status s = check_geom(geom);
  if (s != MLA_OK) return s;
  if (B < 0 || max_pages < 1) return MLA_ERR_ARG;
  if (B == 0) return MLA_OK;
  if (!block_table || !seq_lens || !w_uk || !w_uv || !kv_exp || bt_stride < max_pages) return MLA_ERR_ARG;
  if ((long long)B * normal_rows_per_seq(max_pages) >= (1LL << 31)) return MLA_ERR_SHAPE;
  if (!aligned16(block_table) || !aligned16(seq_lens) || !aligned16(w_uk) || !aligned16(w_uv) || !aligned32(kv_exp))
    return MLA_ERR_ALIGN;
  CacheView cv;
  if ((s = check_cache(cache, &cv)) != MLA_OK) return s;
  return cuda_status(launch_normal_expand(geom, cv, block_table, bt_stride, seq_lens, B, max_pages,
                                          static_cast<const __nv_bfloat16*>(w_uk),
                                          static_cast<const __nv_bfloat16*>(w_uv),
                                          static_cast<__nv_bfloat16*>(kv_exp), (cudaStream_t)stream));
}

mla_status mla_normal_attention(const mla_geom* geom, const mla_batch* batch, const void* q_nope, const void* q_pe,
                                const mla_cache* cache, const int32_t* block_table, int bt_stride,
                                const int32_t* seq_lens, const void* kv_exp, void* o, float* lse,
                                mla_stream_t stream) {
  mla_status s = check_geom(geom);
  if (s != MLA_OK) return s;
  if ((s = check_batch(batch)) != MLA_OK) return s;
  if (batch->B == 0) return MLA_OK;
  if (!q_nope || !q_pe || !block_table || !seq_lens || !kv_exp || !o || !lse) return MLA_ERR_ARG;
  if (bt_stride < batch->max_pages) return MLA_ERR_ARG;
  if ((long long)batch->B * normal_rows_per_seq(batch->max_pages) >= (1LL << 31) || batch->B > 65535 ||
      (batch->T + 127) / 128 > 65535)
    return MLA_ERR_SHAPE;
  if (!aligned16(q_nope) || !aligned16(q_pe) || !aligned16(block_table) || !aligned16(seq_lens) ||
      !aligned16(kv_exp) || !aligned32(o) || !aligned16(lse))
    return MLA_ERR_ALIGN;
  CacheView cv;
  if ((s = check_cache(cache, &cv)) != MLA_OK) return s;
  return cuda_status(launch_normal_attention(geom, batch, static_cast<const __nv_bfloat16*>(q_nope),
                                             static_cast<const __nv_bfloat16*>(q_pe), cv, block_table, bt_stride,
                                             seq_lens, static_cast<const __nv_bfloat16*>(kv_exp),
                                             static_cast<__nv_bfloat16*>(o), lse, (cudaStream_t)stream));
}

size_t mla_normal_chunk_bytes(const mla_geom* geom, int B, int chunk_rows) {
  if (check_geom(geom) != MLA_OK || B < 0 || chunk_rows < 128 || chunk_rows % 128 != 0) return 0;
  return (size_t)geom->H * (size_t)B * (size_t)chunk_rows * 256 * 2;
}

size_t mla_normal_chunk_state_bytes(const mla_geom* geom, const mla_batch* batch) {
  if (check_geom(geom) != MLA_OK || check_batch(batch) != MLA_OK) return 0;
  const size_t rows = (size_t)batch->B * batch->T * geom->H;
  return align_up(rows * kDV * 4) + align_up(rows * 4);
}

mla_status mla_normal_chunked(const mla_geom* geom, const mla_batch* batch, const void* q_nope, const void* q_pe,
                              const mla_cache* cache, const int32_t* block_table, int bt_stride,
                              const int32_t* seq_lens, const void* w_uk, const void* w_uv, int chunk_rows,
                              void* kv_chunk, void* state, void* o, float* lse, mla_stream_t stream) {
  mla_status s = check_geom(geom);
  if (s != MLA_OK) return s;
  if ((s = check_batch(batch)) != MLA_OK) return s;
  if (chunk_rows < 128 || chunk_rows % 128 != 0) return MLA_ERR_ARG;
  if (batch->B == 0) return MLA_OK;
  if (!q_nope || !q_pe || !block_table || !seq_lens || !w_uk || !w_uv || !kv_chunk || !state || !o || !lse)
    return MLA_ERR_ARG;
  if (bt_stride < batch->max_pages) return MLA_ERR_ARG;
  if ((long long)batch->B * chunk_rows >= (1LL << 31) || batch->B > 65535 || (batch->T + 127) / 128 > 65535)
    return MLA_ERR_SHAPE;
  if (!aligned16(q_nope) || !aligned16(q_pe) || !aligned16(block_table) || !aligned16(seq_lens) ||
      !aligned16(w_uk) || !aligned16(w_uv) || !aligned32(kv_chunk) || !aligned32(state) || !aligned32(o) ||
      !aligned16(lse))
    return MLA_ERR_ALIGN;
  CacheView cv;
  if ((s = check_cache(cache, &cv)) != MLA_OK) return s;
  const size_t rows = (size_t)batch->B * batch->T * geom->H;
  float* st_o = static_cast<float*>(state);
  float* st_lse = reinterpret_cast<float*>(static_cast<char*>(state) + align_up(rows * kDV * 4));
  return cuda_status(launch_normal_chunked(geom, batch, static_cast<const __nv_bfloat16*>(q_nope),
                                           static_cast<const __nv_bfloat16*>(q_pe), cv, block_table, bt_stride,
                                           seq_lens, static_cast<const __nv_bfloat16*>(w_uk),
                                           static_cast<const __nv_bfloat16*>(w_uv), chunk_rows,
                                           static_cast<__nv_bfloat16*>(kv_chunk), st_o, st_lse,
                                           static_cast<__nv_bfloat16*>(o), lse, (cudaStream_t)stream));
}

// An FP8 pool as a view (only its block count is used).
static mla_status check_fp8_pool(const void* cache_fp8, int num_blocks, CacheView* cv) {
  if (!cache_fp8 || num_blocks < 1) return MLA_ERR_ARG;
  if (!aligned16(cache_fp8)) return MLA_ERR_ALIGN;
  *cv = CacheView{};
  cv->num_blocks = num_blocks;
  return MLA_OK;
}
static mla_status check_rows32(const CacheView& cv) {   // physical rows as 32-bit numbers
  return (long long)cv.num_blocks * kPage >= (1LL << 31) ? MLA_ERR_SHAPE : MLA_OK;
}

// Shared by the two forms of the append: everything but the cache (fills c).
static mla_status append_args(const mla_geom* geom, int N, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                              const void* kv, int64_t kv_token_stride, const void* q_weight, const void* kv_weight,
                              float eps, const float* cos_sin, int max_pos, const int32_t* positions, int interleaved,
                              const int32_t* slots, void* q_nope, void* q_pe, AppendCall* c) {
  const mla_status s = check_geom(geom);
  if (s != MLA_OK) return s;
  if (N < 0 || !(eps >= 0.f) || max_pos < 1) return MLA_ERR_ARG;
  if (N == 0) return MLA_OK;
  if (!q || !kv || !cos_sin || !positions || !slots || !q_nope || !q_pe) return MLA_ERR_ARG;
  if (q_token_stride < 0 || q_head_stride < 0 || kv_token_stride < 0) return MLA_ERR_ARG;
  if (!aligned16(q) || !aligned16(kv) || !aligned16(q_weight) || !aligned16(kv_weight) || !aligned16(cos_sin) ||
      !aligned16(positions) || !aligned16(slots) || !aligned16(q_nope) || !aligned16(q_pe))
    return MLA_ERR_ALIGN;
  if (q_token_stride % 8 != 0 || q_head_stride % 8 != 0 || kv_token_stride % 8 != 0) return MLA_ERR_ALIGN;
  if ((long long)N * (geom->H + 1) >= (1LL << 31)) return MLA_ERR_SHAPE;
  c->N = N; c->H = geom->H;
  c->q = static_cast<const __nv_bfloat16*>(q); c->q_token = q_token_stride; c->q_head = q_head_stride;
  c->kv = static_cast<const __nv_bfloat16*>(kv); c->kv_token = kv_token_stride;
  c->q_weight = static_cast<const __nv_bfloat16*>(q_weight);
  c->kv_weight = static_cast<const __nv_bfloat16*>(kv_weight);
  c->eps = eps; c->cos_sin = cos_sin; c->max_pos = max_pos; c->positions = positions; c->slots = slots;
  c->interleaved = interleaved != 0;
  c->q_nope = static_cast<__nv_bfloat16*>(q_nope); c->q_pe = static_cast<__nv_bfloat16*>(q_pe);
  c->rows_fp8 = nullptr;
  return MLA_OK;
}

mla_status mla_rope_append(const mla_geom* geom, int N, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                           const void* kv, int64_t kv_token_stride, const void* q_weight, const void* kv_weight,
                           float eps, const float* cos_sin, int max_pos, const int32_t* positions, int interleaved,
                           const mla_cache* cache, const int32_t* slots, void* q_nope, void* q_pe,
                           mla_stream_t stream) {
  AppendCall c;
  mla_status s = append_args(geom, N, q, q_token_stride, q_head_stride, kv, kv_token_stride, q_weight, kv_weight, eps,
                             cos_sin, max_pos, positions, interleaved, slots, q_nope, q_pe, &c);
  if (s != MLA_OK || N == 0) return s;
  if ((s = check_cache(cache, &c.cv)) != MLA_OK) return s;
  if ((s = check_rows32(c.cv)) != MLA_OK) return s;
  if ((s = check_device(q)) != MLA_OK) return s;
  return cuda_status(launch_rope_append(c, (cudaStream_t)stream));
}

mla_status mla_rope_append_fp8(const mla_geom* geom, int N, const void* q, int64_t q_token_stride,
                               int64_t q_head_stride, const void* kv, int64_t kv_token_stride, const void* q_weight,
                               const void* kv_weight, float eps, const float* cos_sin, int max_pos,
                               const int32_t* positions, int interleaved, void* cache_fp8, int num_blocks,
                               const int32_t* slots, void* q_nope, void* q_pe, mla_stream_t stream) {
  AppendCall c;
  mla_status s = append_args(geom, N, q, q_token_stride, q_head_stride, kv, kv_token_stride, q_weight, kv_weight,
                                   eps, cos_sin, max_pos, positions, interleaved, slots, q_nope, q_pe, &c);
  if (s != MLA_OK || N == 0) return s;
  if ((s = check_fp8_pool(cache_fp8, num_blocks, &c.cv)) != MLA_OK) return s;
  if ((s = check_rows32(c.cv)) != MLA_OK) return s;
  c.rows_fp8 = static_cast<unsigned char*>(cache_fp8);
  if ((s = check_device(q)) != MLA_OK) return s;
  return cuda_status(launch_rope_append(c, (cudaStream_t)stream));
}

mla_status mla_verify_tree(int B, int T, int V, const void* target_probs, const void* draft_probs, mla_dtype dtype,
                           int64_t row_stride, const int32_t* tokens, const int32_t* parents,
                           const int32_t* node_lens, const float* u_accept, const float* u_sample,
                           int32_t* accept_len, int32_t* accept_idx, int32_t* out_tokens, mla_stream_t stream) {
  if (B < 0 || T < 1 || V < 1 || row_stride < V) return MLA_ERR_ARG;
  if (dtype != MLA_DTYPE_F32 && dtype != MLA_DTYPE_BF16) return MLA_ERR_ARG;
  if (T > kMaxTreeNodes || V > (1 << 30)) return MLA_ERR_SHAPE;
  if (B == 0) return MLA_OK;
  if (!target_probs || !tokens || !parents || !u_accept || !u_sample || !accept_len || !accept_idx || !out_tokens)
    return MLA_ERR_ARG;
  if (!aligned16(target_probs) || !aligned16(draft_probs) || !aligned16(tokens) || !aligned16(parents) ||
      !aligned16(node_lens) || !aligned16(u_accept) || !aligned16(u_sample) || !aligned16(accept_len) ||
      !aligned16(accept_idx) || !aligned16(out_tokens))
    return MLA_ERR_ALIGN;
  if ((row_stride * (dtype == MLA_DTYPE_BF16 ? 2 : 4)) % 16 != 0) return MLA_ERR_ALIGN;
  const mla_status s = check_device(target_probs);
  if (s != MLA_OK) return s;
  const VerifyCall c{B, T, V, target_probs, draft_probs, dtype == MLA_DTYPE_BF16, row_stride, tokens, parents,
                     node_lens, u_accept, u_sample, accept_len, accept_idx, out_tokens};
  return cuda_status(launch_verify_tree(c, (cudaStream_t)stream));
}

static mla_status cache_compact(const CacheView& cv, void* rows_fp8, const int32_t* block_table, int bt_stride,
                                int max_pages, const int32_t* seq_lens, const int32_t* node_lens,
                                const int32_t* accept_len, const int32_t* accept_idx, int B, int T, int32_t* new_lens,
                                mla_stream_t stream) {
  if (B < 0 || T < 1 || max_pages < 1 || bt_stride < max_pages) return MLA_ERR_ARG;
  if (T > kMaxTreeNodes || max_pages >= (1 << 25)) return MLA_ERR_SHAPE;
  if (B == 0) return MLA_OK;
  if (!block_table || !seq_lens || !accept_len || !accept_idx || !new_lens) return MLA_ERR_ARG;
  if (new_lens == seq_lens || new_lens == node_lens || new_lens == accept_len || new_lens == accept_idx)
    return MLA_ERR_ARG;
  if (!aligned16(block_table) || !aligned16(seq_lens) || !aligned16(node_lens) || !aligned16(accept_len) ||
      !aligned16(accept_idx) || !aligned16(new_lens))
    return MLA_ERR_ALIGN;
  mla_status s = check_rows32(cv);
  if (s != MLA_OK || (s = check_device(block_table)) != MLA_OK) return s;
  return cuda_status(launch_cache_compact(cv, static_cast<unsigned char*>(rows_fp8), block_table, bt_stride, max_pages,
                                          seq_lens, node_lens, accept_len, accept_idx, B, T, new_lens,
                                          (cudaStream_t)stream));
}

mla_status mla_cache_compact(const mla_cache* cache, const int32_t* block_table, int bt_stride, int max_pages,
                             const int32_t* seq_lens, const int32_t* node_lens, const int32_t* accept_len,
                             const int32_t* accept_idx, int B, int T, int32_t* new_lens, mla_stream_t stream) {
  CacheView cv;
  const mla_status s = check_cache(cache, &cv);
  if (s != MLA_OK) return s;
  return cache_compact(cv, nullptr, block_table, bt_stride, max_pages, seq_lens, node_lens, accept_len, accept_idx, B,
                       T, new_lens, stream);
}

mla_status mla_cache_compact_fp8(void* cache_fp8, int num_blocks, const int32_t* block_table, int bt_stride,
                                 int max_pages, const int32_t* seq_lens, const int32_t* node_lens,
                                 const int32_t* accept_len, const int32_t* accept_idx, int B, int T, int32_t* new_lens,
                                 mla_stream_t stream) {
  CacheView cv;
  const mla_status s = check_fp8_pool(cache_fp8, num_blocks, &cv);
  if (s != MLA_OK) return s;
  return cache_compact(cv, cache_fp8, block_table, bt_stride, max_pages, seq_lens, node_lens, accept_len, accept_idx,
                       B, T, new_lens, stream);
}

// What the page bookkeeping calls share.
static mla_status check_pages(const int32_t* refs, int num_blocks, const int32_t* block_table, int bt_stride,
                              int max_pages, int B) {
  if (B < 0 || num_blocks < 1 || max_pages < 1 || bt_stride < max_pages) return MLA_ERR_ARG;
  if (max_pages >= (1 << 25) || (long long)B * max_pages >= (1LL << 31)) return MLA_ERR_SHAPE;
  if (B == 0) return MLA_OK;
  if (!refs || !block_table) return MLA_ERR_ARG;
  if (!aligned16(refs) || !aligned16(block_table)) return MLA_ERR_ALIGN;
  return MLA_OK;
}

mla_status mla_pages_resize(int32_t* refs, int num_blocks, int32_t* block_table, int bt_stride, int max_pages,
                            const int32_t* cur_lens, const int32_t* new_lens, int B, int32_t* got_lens,
                            mla_stream_t stream) {
  mla_status s = check_pages(refs, num_blocks, block_table, bt_stride, max_pages, B);
  if (s != MLA_OK) return s;
  if (B > 8192) return MLA_ERR_SHAPE;
  if (B == 0) return MLA_OK;
  if (!cur_lens || !new_lens || !got_lens) return MLA_ERR_ARG;
  if (!aligned16(cur_lens) || !aligned16(new_lens) || !aligned16(got_lens)) return MLA_ERR_ALIGN;
  if ((s = check_device(refs)) != MLA_OK) return s;
  return cuda_status(launch_pages_resize(refs, num_blocks, block_table, bt_stride, max_pages, cur_lens, new_lens, B,
                                         got_lens, (cudaStream_t)stream));
}

mla_status mla_pages_fork(int32_t* refs, int num_blocks, int32_t* block_table, int bt_stride, int max_pages,
                          int32_t* seq_lens, int B, const int32_t* src, const int32_t* dst, int F, int32_t* copies,
                          mla_stream_t stream) {
  mla_status s = check_pages(refs, num_blocks, block_table, bt_stride, max_pages, B);
  if (s != MLA_OK) return s;
  if (F < 0) return MLA_ERR_ARG;
  if (B > 65536 || F > 4096) return MLA_ERR_SHAPE;
  if (F == 0) return MLA_OK;
  if (B == 0 || !seq_lens || !src || !dst || !copies) return MLA_ERR_ARG;
  if (!aligned16(seq_lens) || !aligned16(src) || !aligned16(dst) || !aligned16(copies)) return MLA_ERR_ALIGN;
  if ((s = check_device(refs)) != MLA_OK) return s;
  return cuda_status(launch_pages_fork(refs, num_blocks, block_table, bt_stride, max_pages, seq_lens, B, src, dst, F,
                                       copies, (cudaStream_t)stream));
}

static mla_status cache_copy(const CacheView& cv, void* rows_fp8, const int32_t* copies, int n, mla_stream_t stream) {
  if (n < 0) return MLA_ERR_ARG;
  if (n == 0) return MLA_OK;
  if (!copies) return MLA_ERR_ARG;
  if (!aligned16(copies)) return MLA_ERR_ALIGN;
  mla_status s = check_rows32(cv);
  if (s != MLA_OK || (s = check_device(copies)) != MLA_OK) return s;
  return cuda_status(launch_cache_copy(cv, static_cast<unsigned char*>(rows_fp8), copies, n, (cudaStream_t)stream));
}

mla_status mla_cache_copy(const mla_cache* cache, const int32_t* copies, int n, mla_stream_t stream) {
  CacheView cv;
  const mla_status s = check_cache(cache, &cv);
  return s != MLA_OK ? s : cache_copy(cv, nullptr, copies, n, stream);
}

mla_status mla_cache_copy_fp8(void* cache_fp8, int num_blocks, const int32_t* copies, int n, mla_stream_t stream) {
  CacheView cv;
  const mla_status s = check_fp8_pool(cache_fp8, num_blocks, &cv);
  return s != MLA_OK ? s : cache_copy(cv, cache_fp8, copies, n, stream);
}

mla_status mla_read_device_status(const void* workspace, int* info, mla_stream_t stream) {
  if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return MLA_ERR_CUDA;
  if (info) *info = 0;
  if (workspace) {
    int words[2] = {0, 0};
    const char* base = static_cast<const char*>(workspace) + MLA_HDR_ERROR * sizeof(int);
    if (cudaMemcpy(words, base, sizeof(words), cudaMemcpyDeviceToHost) != cudaSuccess) return MLA_ERR_CUDA;
    if (info) *info = words[1];
    if (words[0] != 0) return (mla_status)words[0];
  }
  // Kernels without a workspace keep their (rare) timeout in one word per device.
  int* bmm = bmm_status_ptr();
  if (bmm) {
    int v = 0;
    if (cudaMemcpy(&v, bmm, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return MLA_ERR_CUDA;
    if (v != 0) {
      const int zero = 0;
      cudaMemcpy(bmm, &zero, sizeof(int), cudaMemcpyHostToDevice);
      if (info) *info = -1;
      return (mla_status)v;
    }
  }
  // mla_decode_noalloc plans and decodes in the library's own scratch: its status
  // word (and detail) is read here, without a workspace, and cleared.
  if (!workspace) {
    int* na = noalloc_status_words();
    if (na) {
      int words[2] = {0, 0};
      if (cudaMemcpy(words, na, sizeof(words), cudaMemcpyDeviceToHost) != cudaSuccess) return MLA_ERR_CUDA;
      if (words[0] != 0) {
        const int zero[2] = {0, 0};
        cudaMemcpy(na, zero, sizeof(zero), cudaMemcpyHostToDevice);
        if (info) *info = words[1];
        return (mla_status)words[0];
      }
    }
  }
  return MLA_OK;
}

}  // extern "C"
